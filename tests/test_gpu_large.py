"""More than 2^31 elements in one call, beyond the forward scan: its gradients and the
norms in both directions.  The last rows are right, the first ones too."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref
from tests.test_gpu_scan import check_backward

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def need(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb << 30:
        pytest.skip(f"needs {gb} GB of free device memory")


@pytest.mark.parametrize("C", [4096, 4100])
def test_scan_gradients(C):
    """All but the last 300 tokens have no input, no gradient and a decay of exp(-0.5)."""
    need(60)
    T, tail = (1 << 19) + 40, 300
    d = ref.scan_inputs([tail], C, BF, seed=21, beta=False, h0=False)
    x, dh = (torch.zeros(1, T, C, dtype=BF, device=DEV) for _ in range(2))
    g = torch.full((1, T, C), -0.5, device=DEV)
    x[0, -tail:], g[0, -tail:], dh[0, -tail:] = d["x"].to(DEV), d["g"].to(DEV), d["dh"].to(DEV)
    dx, dg, _, _ = gdn.scan_backward(dh, x, g, dh_T=d["dh_T"].to(DEV))
    b = ref.scan_backward(d, [tail])
    check_backward((dx[:, -tail:], dg[:, -tail:], None, None), b, d, BF, (1, tail, C), "tail")
    # before it: lam decays by exp(-0.5) a token, no state to differentiate
    assert not bool(dg[0, :-tail].any()) and not bool(dx[0, :-tail - 400].any())
    lam = b["dx"][0].to(DEV) * d["g"][0].double().exp().to(DEV)
    got = dx[0, -tail - 1].double()
    assert bool(((got - lam).abs() <= 2.0 ** -8 * lam.abs() + 2e-5 * b["edx"][0].to(DEV)).all())


@pytest.mark.parametrize("D", [8, 127, 8192])
def test_norms(D):
    """Rows are independent of each other: the last ones give what they give alone, bit
    for bit, and their weight gradients are the call's, all other rows being zero."""
    need(80)
    rows, tail = (1 << 31) // D + 77, 64  # an even number of rows before the tail keeps its alignment
    rows += (rows - tail) % 2
    d = ref.norm_inputs(tail, D, x_dtype=BF, dtype=BF, seed=D)
    big = {}
    for k in ("x", "z", "dy", "r", "dr_out"):
        big[k] = torch.zeros(rows, D, dtype=BF, device=DEV)
        big[k][-tail:] = d[k].to(DEV)
    w, wp, sc = (d[k].to(DEV) for k in ("w", "w_post", "scale"))
    end = {k: v[-tail:].contiguous() for k, v in big.items()}
    y = gdn.gated_norm(big["x"], w, big["z"])
    assert torch.equal(y[-tail:], gdn.gated_norm(end["x"], w, end["z"])) and not bool(y[:-tail].any())
    del y
    dx, dz, dw = gdn.gated_norm_backward(big["dy"], big["x"], w, big["z"])
    one = gdn.gated_norm_backward(end["dy"], end["x"], w, end["z"])
    assert torch.equal(dx[-tail:], one[0]) and torch.equal(dz[-tail:], one[1])
    assert not bool(dx[:-tail].any()) and not bool(dz[:-tail].any())
    want = ref.gated_norm_backward(d)["dw"]
    ref.assert_norm(dw, want, ref.norm_steps(64 + tail, float(d["z"].abs().max())), F32, "dw")
    del dx, dz
    y, r_out = gdn.residual_norm(big["x"], big["r"], w, w_post=wp, scale=sc)
    alone = gdn.residual_norm(end["x"], end["r"], w, w_post=wp, scale=sc)
    assert torch.equal(y[-tail:], alone[0]) and torch.equal(r_out[-tail:], alone[1])
    assert not bool(y[:-tail].any())
    del y, r_out
    got = gdn.residual_norm_backward(big["dy"], big["dr_out"], big["x"], big["r"], w, w_post=wp, scale=sc)
    alone = gdn.residual_norm_backward(end["dy"], end["dr_out"], end["x"], end["r"], w, w_post=wp, scale=sc)
    for a, b in zip(got[:2], alone[:2]):
        assert torch.equal(a[-tail:], b) and not bool(a[:-tail].any())
    want = ref.residual_norm_backward({**d, "z": None})
    steps = ref.norm_steps(4 * 48 + tail, 0.0)
    for name, a in zip(("dw", "dw_post", "dscale"), got[3:]):
        ref.assert_norm(a, want[name], steps, F32, name)
