"""Norms around a layer on the GPU against the 64-bit reference, element by
element within the rounding bounds of tests/layer_reference.py, and a layer of
the library's calls in a run."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def name_of(t):
    return {BF: "bf16", F32: "f32"}.get(t)


def to_dev(d):
    return {k: v.to(DEV) if v is not None else None for k, v in d.items()}


def steps(d, rows, D):
    """Steps of a row's results (two sums of D terms on the way to the last ones)
    and of a sum over the rows."""
    zmax = float(d["z"].double().abs().max()) if d["z"] is not None and d["z"].numel() else 0.0
    return ref.norm_steps(2 * D, zmax), ref.norm_steps(2 * D + rows, zmax)


SIZES = [(1, 1), (3, 8), (5, 64), (2, 65), (17, 128), (40, 200), (33, 256), (3, 257), (4, 264),
         (7, 1000), (2, 4096), (3, 4100), (5, 4104), (2, 8192), (2, 9001), (3, 16384), (1, 16383),
         (1500, 64), (700, 520),
         # odd rows (their pairs are shifted by one) and even ones that are no multiple of 4
         (37, 33), (300, 257), (301, 63), (9, 4097), (5, 16383), (33, 31), (130, 255), (2, 7),
         (21, 54), (3, 250), (4, 2770), (3, 16382), (1000, 14)]


@pytest.mark.parametrize("z,gate", [(True, "silu"), (True, "sigmoid"), (False, "silu")])
@pytest.mark.parametrize("x_dtype,dtype", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)], ids=name_of)
@pytest.mark.parametrize("rows,D", SIZES)
def test_gated_norm_and_gradients(rows, D, x_dtype, dtype, z, gate):
    d = ref.norm_inputs(rows, D, x_dtype=x_dtype, dtype=dtype, seed=rows + D, z=z)
    one, summed = steps(d, rows, D)
    dd = to_dev(d)
    kw = dict(gate=gate, eps=1e-5, weight_offset=0.25)
    y = gdn.gated_norm(dd["x"], dd["w"], dd["z"], out_dtype=dtype, **kw)
    want = ref.gated_norm(d, gate, 1e-5, 0.25)
    assert y.dtype == dtype
    ref.assert_norm(y, (want, want.abs()), one, dtype, "y")
    got = gdn.gated_norm_backward(dd["dy"], dd["x"], dd["w"], dd["z"], **kw)
    b = ref.gated_norm_backward(d, gate, 1e-5, 0.25)
    ref.assert_norm(got[0], b["dx"], one, x_dtype, "dx")
    ref.assert_norm(got[2], b["dw"], summed, F32, "dw")
    assert (got[1] is None) == (not z)
    if z:
        ref.assert_norm(got[1], b["dz"], one, dtype, "dz")


GRADS = ("dx", "dr", "dz", "dw", "dw_post", "dscale")


def check_residual_gradients(got, b, dtype, r_dtype, one, summed):
    for name, g, t, n in zip(GRADS, got, (dtype, r_dtype, dtype, F32, F32, F32),
                             (one, one, one, summed, summed, summed)):
        assert (g is None) == (name not in b), name
        if g is not None:
            ref.assert_norm(g, b[name], n, t, name)


@pytest.mark.parametrize("z,post,scale", [(True, True, True), (False, True, False),
                                          (True, False, False), (False, False, True),
                                          (False, False, False)])
@pytest.mark.parametrize("dtype,r_dtype", [(BF, BF), (BF, F32), (F32, F32)], ids=name_of)
@pytest.mark.parametrize("rows,D", SIZES)
def test_residual_norm_and_gradients(rows, D, dtype, r_dtype, z, post, scale):
    d = ref.norm_inputs(rows, D, x_dtype=dtype, dtype=dtype, r_dtype=r_dtype, seed=rows * 3 + D,
                        z=z, post=post, scale=scale)
    one, summed = steps(d, rows, D)
    dd = to_dev(d)
    kw = dict(z=dd["z"], w_post=dd["w_post"], scale=dd["scale"], eps=1e-5, weight_offset=0.25)
    y, r_out = gdn.residual_norm(dd["x"], dd["r"], dd["w"], **kw)
    f = ref.residual_norm(d, "silu", 1e-5, 0.25)
    ref.assert_norm(r_out, f["r_out"], one, r_dtype, "r_out")
    ref.assert_norm(y, f["y"], one, dtype, "y")
    for with_dr in (True, False):
        got = gdn.residual_norm_backward(dd["dy"], dd["dr_out"] if with_dr else None, dd["x"],
                                         dd["r"], dd["w"], **kw)
        b = ref.residual_norm_backward({**d, "dr_out": d["dr_out"] if with_dr else None}, "silu",
                                       1e-5, 0.25)
        check_residual_gradients(got, b, dtype, r_dtype, one, summed)


# rows of more than a CTA's registers hold with their weights, on more rows than CTAs: the
# ends of each layout, in fours, pairs, odd rows
LONG = [(5, 4098), (200, 5120), (3, 6144), (160, 6148), (2, 6150), (301, 8190), (5, 8191), (170, 4997),
        (299, 5121)]


@pytest.mark.parametrize("z,post,scale", [(True, True, True), (False, False, True), (False, True, False)])
@pytest.mark.parametrize("dtype,r_dtype", [(BF, BF), (BF, F32), (F32, F32)], ids=name_of)
@pytest.mark.parametrize("rows,D", LONG)
def test_residual_norm_of_long_rows(rows, D, dtype, r_dtype, z, post, scale):
    test_residual_norm_and_gradients(rows, D, dtype, r_dtype, z, post, scale)


@pytest.mark.parametrize("rows,D", LONG)
def test_gated_norm_of_long_rows(rows, D):
    test_gated_norm_and_gradients(rows, D, BF, BF, True, "silu")
    test_gated_norm_and_gradients(rows, D, F32, BF, True, "sigmoid")


def test_rows_of_zeros_and_no_rows():
    w = torch.ones(64, device=DEV)
    x = torch.zeros(3, 64, dtype=BF, device=DEV)
    assert not bool(gdn.gated_norm(x, w, x).any())
    dx, dz, dw = gdn.gated_norm_backward(x, x, w, x)
    assert not bool(dx.any()) and not bool(dz.any()) and not bool(dw.any())
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    assert gdn.gated_norm(e, w).shape == (0, 64)
    dx, dz, dw = gdn.gated_norm_backward(e, e, w, e)
    assert dw.shape == (64,) and not bool(dw.any())
    out = gdn.residual_norm_backward(e, e, e, e, w, z=e, w_post=w.clone(), scale=w.clone())
    assert all(not bool(g.any()) for g in out[3:])


def test_gates_far_from_zero():
    """Gates of +-300 and of infinity: no NaN from an overflowing exponential."""
    z = torch.tensor([300.0, -300.0, 88.0, -88.0, float("inf"), 0.0, -0.0, 20.0], device=DEV)
    x = torch.ones(1, 8, device=DEV)
    w = torch.ones(8, device=DEV)
    y = gdn.gated_norm(x, w, z[None], eps=0.0)[0]
    assert y[0] == 300 and abs(float(y[1])) < 1e-30 and y[2] == 88 and y[4] == float("inf")
    p = gdn.gated_norm(x, w, z[None], gate="sigmoid", eps=0.0)[0]
    assert p[0] == 1 and abs(float(p[1])) < 1e-30 and p[4] == 1 and p[5] == 0.5


def test_a_nan_stays_in_its_row():
    d = to_dev(ref.norm_inputs(50, 128, x_dtype=BF, dtype=BF, seed=4))
    clean = gdn.gated_norm(d["x"], d["w"], d["z"])
    x = d["x"].clone()
    x[17, 3] = float("nan")
    y = gdn.gated_norm(x, d["w"], d["z"])
    assert bool(y[17].isnan().all())
    y[17] = clean[17]
    assert torch.equal(y, clean)


def test_unaligned_views_take_the_scalar_path():
    d = ref.norm_inputs(20, 128, x_dtype=BF, dtype=BF, seed=5)
    one, summed = steps(d, 20, 128)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1).to(DEV)
        return flat[1:].view(t.shape)

    s = {k: shifted(v) for k, v in d.items()}
    want = ref.gated_norm(d)
    ref.assert_norm(gdn.gated_norm(s["x"], s["w"], s["z"]), (want, want.abs()), one, BF, "y")
    got = gdn.residual_norm_backward(s["dy"], s["dr_out"], s["x"], s["r"], s["w"], z=s["z"],
                                     w_post=s["w_post"], scale=s["scale"])
    check_residual_gradients(got, ref.residual_norm_backward(d), BF, BF, one, summed)


@pytest.mark.parametrize("D", [4100, 8192])
def test_unaligned_long_rows(D):
    d = ref.norm_inputs(170, D, x_dtype=BF, dtype=BF, seed=6)
    one, summed = steps(d, 170, D)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1).to(DEV)
        return flat[1:].view(t.shape)

    s = {k: shifted(v) for k, v in d.items()}
    want = ref.gated_norm(d)
    ref.assert_norm(gdn.gated_norm(s["x"], s["w"], s["z"]), (want, want.abs()), one, BF, "y")
    got = gdn.residual_norm_backward(s["dy"], s["dr_out"], s["x"], s["r"], s["w"], z=s["z"],
                                     w_post=s["w_post"], scale=s["scale"])
    check_residual_gradients(got, ref.residual_norm_backward(d), BF, BF, one, summed)


def test_in_place_sums_and_leading_dimensions():
    d = to_dev(ref.norm_inputs(24, 512, x_dtype=BF, dtype=BF, r_dtype=F32, seed=6, z=False))
    y, r_out = gdn.residual_norm(d["x"], d["r"], d["w"], w_post=d["w_post"])
    r = d["r"].clone().reshape(2, 3, 4, 512)
    y2, r2 = gdn.residual_norm(d["x"].reshape(2, 3, 4, 512), r, d["w"], w_post=d["w_post"], r_out=r)
    assert r2.data_ptr() == r.data_ptr()
    assert torch.equal(y2.reshape(24, 512), y) and torch.equal(r.reshape(24, 512), r_out)


def test_repeatable_on_any_stream_and_in_a_graph():
    d = to_dev(ref.norm_inputs(999, 640, x_dtype=BF, dtype=BF, r_dtype=F32, seed=7))

    def both():
        kw = dict(z=d["z"], w_post=d["w_post"], scale=d["scale"])
        return (gdn.gated_norm(d["x"], d["w"], d["z"]),
                *gdn.gated_norm_backward(d["dy"], d["x"], d["w"], d["z"]),
                *gdn.residual_norm(d["x"], d["r"], d["w"], **kw),
                *gdn.residual_norm_backward(d["dy"], d["dr_out"], d["x"], d["r"], d["w"], **kw))

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


def test_a_layer_prefill_then_one_token():
    """norm -> both recurrences -> gated norm -> residual norm, as a layer runs
    them (its projections left out): all tokens but the last in one call each,
    then the last one by the single-token calls.  Every stage is held to 64 bits
    on the inputs it really had, the gated delta rule to the oracle."""
    import oracle
    from gated_deltanet_linear_20_b200 import inputs
    B, T, H, Dh = 2, 70, 3, 128
    D = H * Dh
    gen = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    p = inputs.prefill_inputs(B, T, H, seed=9, s0_std=0.05)
    stream, w = rnd(B, T, D), 1 + 0.2 * rnd(D)
    z, w_head, w_post = rnd(B, T, H, Dh).to(BF), 1 + 0.2 * rnd(Dh), 1 + 0.2 * rnd(D)
    g = torch.nn.functional.logsigmoid(rnd(B, T, D) + 2)
    c = lambda t: t.to(DEV)  # noqa: E731
    runs = []
    for a, b in ((0, T - 1), (T - 1, T)):
        q, k, v, gs, be = (c(p[n][:, a:b].contiguous()) for n in ("q", "k", "v", "g", "beta"))
        s, zz, gg = (c(t[:, a:b].contiguous()) for t in (stream, z, g))
        x = gdn.gated_norm(s, c(w), out_dtype=BF)
        if a == 0:
            o, S = gdn.prefill(q, k, v, gs, be, c(p["S0"]))
            h, state = gdn.scan(x, gg)
        else:
            o = gdn.decode_step(*(t[:, 0].contiguous() for t in (q, k, v, gs, be)), S)[:, None]
            h = gdn.scan_step(x[:, 0].contiguous(), gg[:, 0].contiguous(), state)[:, None]
        u = gdn.gated_norm(o.contiguous(), c(w_head), zz).reshape(B, b - a, D)
        y, r = gdn.residual_norm(u, s, c(w), w_post=c(w_post), z=h.contiguous(), gate="sigmoid")
        runs.append((x, o, h, u, y, r))
    x, o, h, u, y, r = (torch.cat(t, 1).cpu() for t in zip(*runs))
    one = lambda n, zz: ref.norm_steps(2 * n, float(zz.double().abs().max()))  # noqa: E731
    want = ref.gated_norm(dict(x=stream, w=w, z=None))
    ref.assert_norm(x, (want, want.abs()), one(D, torch.zeros(1)), BF, "x")
    ro, _ = oracle.prefill(p["q"], p["k"], p["v"], p["g"], p["beta"], p["S0"])
    ro = torch.as_tensor(ro)
    assert float((o.double() - ro).norm() / ro.norm()) <= 2e-3
    flat = dict(x=x.reshape(-1, D), g=g.reshape(-1, D), beta=None, h0=None)
    f = ref.scan(flat, [T] * B)
    ref.assert_within(h.reshape(-1, D), f["h"], f["err"], BF, "h")
    want = ref.gated_norm(dict(x=o, w=w_head, z=z))
    ref.assert_norm(u.reshape(o.shape), (want, want.abs()), one(Dh, z), BF, "u")
    want = ref.residual_norm(dict(x=u, r=stream, w=w, z=h, w_post=w_post, scale=None), "sigmoid")
    ref.assert_norm(y, want["y"], one(D, h), BF, "y")
    ref.assert_norm(r, want["r_out"], one(D, h), F32, "r_out")
