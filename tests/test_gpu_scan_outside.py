"""Gradients of packed tokens that are in no sequence are zero: before the first
offset, behind the last, and all of them without any sequence."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref
from tests.test_gpu_scan import check_backward, to_dev

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def soil(*like):
    """Leaves NaN in the memory that the call's outputs will get."""
    junk = [torch.full_like(t, NAN) for t in like for _ in range(4)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 33, 64, 520, 4096])
@pytest.mark.parametrize("head,lens,tail", [(0, [20, 13], 17), (9, [40], 0), (5, [0, 3, 0], 300), (0, [0], 21),
                                            (1, [30, 0, 700], 2), (150, [2] * 140, 90)],
                         ids=lambda x: str(len(x)) if isinstance(x, list) else str(x))
def test_gradients_outside_every_sequence(head, lens, tail, C, dtype, beta):
    if C == 4096 and len(lens) > 100:
        pytest.skip("covered by fewer channels")
    d = ref.scan_inputs(lens, C, dtype, seed=head + sum(lens) + C, beta=beta)
    b, n = ref.scan_backward(d, lens), sum(lens)
    T = head + n + tail

    def pad(t):
        return torch.cat([torch.full((head, C), NAN, dtype=t.dtype, device=DEV), t,
                          torch.full((tail, C), NAN, dtype=t.dtype, device=DEV)])

    dd = {k: pad(v) if v is not None and k not in ("h0", "dh_T") else v for k, v in to_dev(d).items()}
    cu = [head]
    for m in lens:
        cu.append(cu[-1] + m)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    soil(dd["x"], dd["g"])
    got = gdn.scan_varlen_backward(dd["dh"], dd["x"], dd["g"], cu, dd["beta"], dd["h0"], dd["dh_T"],
                                   status=status)
    assert gdn.query_status(status) == 0
    for t in got[:3]:
        if t is not None:
            assert not bool(t[:head].any()) and not bool(t[T - tail:].any())
    inner = [t[head:T - tail] if t is not None and t.shape[0] == T else t for t in got[:3]] + [got[3]]
    check_backward(inner, b, d, dtype, (n, C), "inside")


def test_no_sequences_at_all():
    T, C = 50, 70
    x, g = torch.full((T, C), NAN, dtype=BF, device=DEV), torch.full((T, C), NAN, device=DEV)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    soil(x, g)
    got = gdn.scan_varlen_backward(x, x, g, cu, x.clone(), torch.zeros(0, C, device=DEV))
    assert not any(bool(t.any()) for t in got) and got[3].shape == (0, C)


@pytest.mark.parametrize("C", [33, 520])
def test_invalid_ends_leave_other_gradients_alone(C):
    """A last or first sequence with invalid offsets: nothing is zeroed there."""
    T = 60
    d = ref.scan_inputs([30], C, F32, seed=4)
    b, dd = ref.scan_backward(d, [30]), to_dev(d)
    pad = lambda t: torch.cat([t, torch.zeros(T - 30, C, device=DEV)])  # noqa: E731
    x, g, beta, dh = (pad(dd[k]) for k in ("x", "g", "beta", "dh"))
    for cu, n in (([0, 30, 20], 0), ([0, 30, 70], 0)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        h0, dh_T = torch.zeros(2, C, device=DEV), torch.zeros(2, C, device=DEV)
        h0[n], dh_T[n] = dd["h0"][0], dd["dh_T"][0]
        got = gdn.scan_varlen_backward(dh, x, g, torch.tensor(cu, dtype=torch.int32, device=DEV), beta, h0,
                                       dh_T, status=status)
        assert gdn.query_status(status) == -3
        check_backward([t[:30] for t in got[:3]] + [got[3][n:n + 1]], b, d, F32, (30, C), str(cu))
