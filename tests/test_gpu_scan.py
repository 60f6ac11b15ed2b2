"""Channel recurrence on the GPU against the 64-bit reference, element by element
within the rounding bounds of tests/layer_reference.py."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def to_dev(d):
    return {k: v.to(DEV) if v is not None else None for k, v in d.items()}


def batch(d, B, T):
    C = d["x"].shape[1]
    return {k: (v.reshape(B, T, C) if v is not None and k not in ("h0", "dh_T") else v)
            for k, v in d.items()}


def check_forward(got, f, dtype, shape, what):
    h, h_T = got[:2]
    assert h.dtype == dtype and h_T.dtype == F32
    ref.assert_within(h, f["h"].reshape(shape), f["err"].reshape(shape), dtype, f"{what} h")
    ref.assert_within(h_T, f["h_T"], f["err_T"], F32, f"{what} h_T")


def check_backward(got, b, d, dtype, shape, what):
    for name, g, t in zip(("dx", "dg", "dbeta", "dh0"), got, (dtype, F32, dtype, F32)):
        if (name == "dbeta" and d["beta"] is None) or (name == "dh0" and d["h0"] is None):
            assert g is None
            continue
        assert g.dtype == t
        s = b[name].shape if name == "dh0" else shape
        ref.assert_within(g, b[name].reshape(s), b["e" + name].reshape(s), t, f"{what} {name}")


def offsets(lens):
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


SIZES = [  # B, T, C: one token, ends inside a slice, a tile, a cluster's tile; odd and small C
    (1, 1, 1), (3, 1, 64), (2, 2, 65), (1, 15, 32), (1, 16, 2), (2, 17, 64), (1, 127, 63),
    (1, 128, 130), (2, 129, 34), (1, 257, 100), (1, 1000, 7), (1, 1025, 66), (2, 2500, 64),
    (5, 40, 1000), (300, 3, 65), (2, 64, 5000),
    # large enough for TMA, whose boxes reach past channels, sequences and the end
    (3, 100, 1000), (1, 777, 184), (9, 33, 520), (2, 1100, 72), (70, 5, 400),
    # every launch shape over several tiles: clusters of four warps, one CTA of eight and
    # of four warps, single warps
    (1, 1100, 4096), (6, 200, 2560), (20, 70, 2048), (80, 33, 2048),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("beta,h0", [(True, False), (False, True)])
@pytest.mark.parametrize("B,T,C", SIZES)
def test_scan_and_gradients(B, T, C, beta, h0, dtype):
    lens = [T] * B
    d = ref.scan_inputs(lens, C, dtype, seed=B * 1000 + T + C, beta=beta, h0=h0)
    f, b = ref.scan(d, lens), ref.scan_backward(d, lens)
    dd = batch(to_dev(d), B, T)
    out = gdn.scan(dd["x"], dd["g"], dd["beta"], dd["h0"], save_carries=True)
    check_forward(out, f, dtype, (B, T, C), "scan")
    rows = torch.arange(0, T, 16)
    kept = f["before"].reshape(B, T, C)[:, rows]
    ref.assert_within(out[2], kept, f["err_before"].reshape(B, T, C)[:, rows], F32, "carries")
    for carries in (out[2], None):
        got = gdn.scan_backward(dd["dh"], dd["x"], dd["g"], dd["beta"], dd["h0"], dd["dh_T"],
                                carries=carries)
        check_backward(got, b, d, dtype, (B, T, C), f"carries={carries is not None}")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 64, 131, 520])
@pytest.mark.parametrize("lens", [
    [0], [1], [0, 0, 5, 0], [16, 1, 15, 17, 33], [1] * 40, [700, 3, 0, 129, 16, 2000],
    [31, 32, 0, 33, 64, 500, 1], [5, 90, 0, 1, 33, 16, 60, 2] * 15, [9, 1, 17] * 60,
], ids=lambda x: f"{len(x)}seqs{sum(x)}")
def test_scan_varlen_and_gradients(lens, C, dtype):
    d = ref.scan_inputs(lens, C, dtype, seed=sum(lens) + C)
    f, b = ref.scan(d, lens), ref.scan_backward(d, lens)
    dd, cu, T = to_dev(d), offsets(lens), sum(lens)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gdn.scan_varlen(dd["x"], dd["g"], cu, dd["beta"], dd["h0"], save_carries=True,
                          status=status)
    check_forward(out, f, dtype, (T, C), "scan_varlen")
    for carries in (out[2], None):
        got = gdn.scan_varlen_backward(dd["dh"], dd["x"], dd["g"], cu, dd["beta"], dd["h0"],
                                       dd["dh_T"], carries=carries, status=status)
        check_backward(got, b, d, dtype, (T, C), f"carries={carries is not None}")
    assert gdn.query_status(status) == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,C,beta", [(1, 1, True), (3, 7, False), (64, 4096, True), (5, 1002, True)])
def test_scan_step(B, C, beta, dtype):
    d = ref.scan_inputs([1] * B, C, dtype, seed=C, beta=beta)
    f, dd = ref.scan(d, [1] * B), to_dev(d)
    state = dd["h0"].clone()
    h = gdn.scan_step(dd["x"], dd["g"], state, dd["beta"])
    ref.assert_within(h, f["h"], f["err"], dtype, "h")
    ref.assert_within(state, f["h_T"], f["err_T"], F32, "state")


@pytest.mark.parametrize("B,T,C", [(1, 300, 64), (1, 500, 4096), (4, 200, 63), (20, 70, 2048), (3, 1, 65)])
def test_states_in_place_are_those_of_separate_ones(B, T, C):
    d = to_dev(ref.scan_inputs([T] * B, C, BF, seed=T + C))
    bt = batch(d, B, T)
    h, h_T = gdn.scan(bt["x"], bt["g"], bt["beta"], bt["h0"])
    cu = offsets([T] * B)
    for _ in range(20):
        s = d["h0"].clone()
        got, out = gdn.scan(bt["x"], bt["g"], bt["beta"], s, h_T=s)
        assert out is s and torch.equal(s, h_T) and torch.equal(got, h)
        s = d["h0"].clone()
        gdn.scan_varlen(d["x"], d["g"], cu, d["beta"], s, h_T=s)
        want = gdn.scan_varlen(d["x"], d["g"], cu, d["beta"], d["h0"])[1]
        assert torch.equal(s, want)


def test_a_run_of_calls_is_one_sequence():
    """Prefill in two calls, then single tokens, the state carried in place."""
    T, C, cut, steps = 300, 96, 173, 7
    d = ref.scan_inputs([T], C, BF, seed=5)
    f, dd = ref.scan(d, [T]), to_dev(d)
    state = dd["h0"].clone()
    hs, pos = [], 0
    for end in (cut, T - steps):
        p = slice(pos, end)
        h, s = gdn.scan(dd["x"][p][None], dd["g"][p][None], dd["beta"][p][None], state, h_T=state)
        assert s.data_ptr() == state.data_ptr()
        hs.append(h[0])
        pos = end
    for t in range(pos, T):
        hs.append(gdn.scan_step(dd["x"][t:t + 1], dd["g"][t:t + 1], state, dd["beta"][t:t + 1]))
    ref.assert_within(torch.cat(hs), f["h"], f["err"], BF, "h")
    ref.assert_within(state, f["h_T"], f["err_T"], F32, "state")


@pytest.mark.parametrize("C", [66, 4096])
def test_invalid_offsets_are_reported_and_leave_outputs_alone(C):
    T = 60
    d = to_dev(ref.scan_inputs([T], C, F32, seed=6, h0=False))
    for cu, bad in (([0, 20, 10, 60], [1]), ([0, 20, 61, 60], [1, 2]), ([-1, 20, 40, 60], [0])):
        cu_t = torch.tensor(cu, dtype=torch.int32, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        h_T = torch.full((3, C), 7.0, device=DEV)
        gdn.scan_varlen(d["x"], d["g"], cu_t, d["beta"], h_T=h_T, status=status)
        assert gdn.query_status(status) == -3
        for n in range(3):
            assert bool((h_T[n] == 7.0).all()) == (n in bad)
        status.zero_()
        h0 = torch.zeros(3, C, device=DEV)
        gdn.scan_varlen_backward(d["dh"], d["x"], d["g"], cu_t, d["beta"], h0, status=status)
        assert gdn.query_status(status) == -3


@pytest.mark.parametrize("C", [64, 4096])
def test_tokens_behind_the_last_sequence_stay(C):
    lens, T = [20, 13], 50
    d = ref.scan_inputs(lens, C, BF, seed=7)
    f = ref.scan(d, lens)
    dd, cu = to_dev(d), offsets(lens)
    pad = lambda t, v: torch.cat([t, torch.full((T - 33, C), v, dtype=t.dtype, device=DEV)])  # noqa: E731
    nan = float("nan")
    h = torch.full((T, C), 3.0, dtype=BF, device=DEV)
    x, g, beta = (pad(dd[k], nan) for k in ("x", "g", "beta"))
    _, h_T = gdn.scan_varlen(x, g, cu, beta, dd["h0"], h=h)
    assert bool((h[33:] == 3.0).all())
    check_forward((h[:33], h_T), f, BF, (33, C), "padded")
    b = ref.scan_backward(d, lens)
    got = gdn.scan_varlen_backward(pad(dd["dh"], nan), x, g, cu, beta, dd["h0"],
                                   dd["dh_T"])
    check_backward([t[:33] if t.shape[0] == T else t for t in got], b, d, BF, (33, C), "padded")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gates_at_their_ends(dtype):
    """Decays of 0 (g = -inf), of 1 (g = 0) and growth, over several tiles."""
    T, C = 400, 68
    pick = torch.randint(0, 4, (T, C), generator=torch.Generator().manual_seed(8))

    def gates(r):
        g = torch.where(pick == 0, torch.zeros(()), -r.abs())
        g = torch.where(pick == 1, 0.05 * r.abs(), g)
        return torch.where((pick == 2) & (r > 1.5), torch.tensor(-float("inf")), g)

    d = ref.scan_inputs([T], C, dtype, seed=9, g=gates)
    dd = batch(to_dev(d), 1, T)
    fin = dict(d, g=d["g"].clamp_min(-1e3))  # exp(-1000) is 0 in 64 bits too
    f, b = ref.scan(fin, [T]), ref.scan_backward(fin, [T])
    out = gdn.scan(dd["x"], dd["g"], dd["beta"], dd["h0"], save_carries=True)
    check_forward(out, f, dtype, (1, T, C), "gates")
    got = gdn.scan_backward(dd["dh"], dd["x"], dd["g"], dd["beta"], dd["h0"], dd["dh_T"],
                            carries=out[2])
    check_backward(got, b, d, dtype, (1, T, C), "gates")


def test_growth_past_the_range_starts_from_zero():
    """A run whose growth overflows fp32 does not spoil a state that is zero."""
    T, C = 512, 64
    x = torch.zeros(1, T, C, device=DEV)
    x[:, -1] = 2.0
    g = torch.full((1, T, C), 3.0, device=DEV)
    h, h_T = gdn.scan(x, g)
    assert bool((h[:, :-1] == 0).all()) and bool((h_T == 2.0).all())


def test_a_nan_stays_in_its_channel_and_behind_its_token():
    T, C = 300, 70
    d = ref.scan_inputs([T], C, F32, seed=10)
    dd = batch(to_dev(d), 1, T)
    clean = gdn.scan(dd["x"], dd["g"], dd["beta"], dd["h0"])[0]
    dd["x"][0, 150, 33] = float("nan")
    h = gdn.scan(dd["x"], dd["g"], dd["beta"], dd["h0"])[0]
    assert bool(h[0, 150:, 33].isnan().all())
    h[0, 150:, 33] = clean[0, 150:, 33]
    assert torch.equal(h, clean)


def test_unaligned_views_take_the_scalar_path():
    """Contiguous views that start on an odd element give the same numbers as a
    copy, within the bound."""
    T, C = 90, 64
    d = ref.scan_inputs([T], C, BF, seed=11)
    f, b = ref.scan(d, [T]), ref.scan_backward(d, [T])
    dd = batch(to_dev(d), 1, T)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    s = {k: shifted(v) for k, v in dd.items()}
    out = gdn.scan(s["x"], s["g"], s["beta"], s["h0"], save_carries=True)
    check_forward(out, f, BF, (1, T, C), "shifted")
    got = gdn.scan_backward(s["dh"], s["x"], s["g"], s["beta"], s["h0"], s["dh_T"], carries=out[2])
    check_backward(got, b, d, BF, (1, T, C), "shifted")
    state = shifted(dd["h0"])
    h = gdn.scan_step(s["x"][:, 0], s["g"][:, 0], state, s["beta"][:, 0])
    ref.assert_within(h, f["h"][:1], f["err"][:1], BF, "shifted step")


def test_repeatable_on_any_stream_and_in_a_graph():
    B, T, C = 2, 1100, 130
    dd = batch(to_dev(ref.scan_inputs([T] * B, C, BF, seed=12)), B, T)

    def both():
        out = gdn.scan(dd["x"], dd["g"], dd["beta"], dd["h0"], save_carries=True)
        return (*out, *gdn.scan_backward(dd["dh"], dd["x"], dd["g"], dd["beta"], dd["h0"],
                                         dd["dh_T"], carries=out[2]))

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, again, captured):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("C", [4096, 4100])
def test_elements_past_32_bits(C):
    """More than 2^31 elements in one call: the last tokens are right."""
    T = (1 << 19) + 40
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    x = torch.zeros(1, T, C, dtype=BF, device=DEV)
    g = torch.full((1, T, C), -0.5, device=DEV)
    tail = 300
    d = ref.scan_inputs([tail], C, BF, seed=13, beta=False, h0=False)
    x[0, -tail:] = d["x"].to(DEV)
    g[0, -tail:] = d["g"].to(DEV)
    h, h_T = gdn.scan(x, g)
    f = ref.scan(d, [tail])
    assert not bool(h[0, :-tail].any())
    check_forward((h[:, -tail:], h_T), f, BF, (1, tail, C), "tail")


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: nothing needs a call before."""
    import subprocess
    import sys
    code = """
import torch
import gated_deltanet_linear_20_b200 as gdn
dev = torch.device('cuda:0')
x = torch.randn(1, 600, 1024, device=dev).bfloat16()
g = -torch.rand(1, 600, 1024, device=dev)
w = torch.ones(1024, device=dev)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    h, h_T, c = gdn.scan(x, g, save_carries=True)
    dx = gdn.scan_backward(h, x, g, carries=c)[0]
    y, r = gdn.residual_norm(h, x, w, w_post=w, scale=w)
    grads = gdn.residual_norm_backward(dx, None, h, r, w, w_post=w, scale=w)
    gg = gdn.gated_norm_backward(y, r, w, h)
graph.replay()
torch.cuda.synchronize()
want = gdn.scan(x, g)[0]
assert torch.equal(h, want)
assert torch.equal(gg[0], gdn.gated_norm_backward(y, r, w, h)[0])
print('captured')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stderr[-2000:]
