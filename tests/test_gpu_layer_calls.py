"""Calls of the channel recurrence and the norms that their documentation allows, beside
those of the other tests: no tokens, outputs over inputs through the C calls, replayed
graphs with new inputs, calls side by side on two streams."""
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


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 64, 4096])
def test_no_tokens(C, dtype):
    x, g = torch.empty(3, 0, C, dtype=dtype, device=DEV), torch.empty(3, 0, C, device=DEV)
    h0, dh_T = torch.randn(3, C, device=DEV), torch.randn(3, C, device=DEV)
    h, h_T, kept = gdn.scan(x, g, x.clone(), h0, save_carries=True)
    assert h.shape == x.shape and torch.equal(h_T, h0) and kept.shape == (3, 0, C)
    assert not bool(gdn.scan(x, g)[1].any())
    dx, dg, dbeta, dh0 = gdn.scan_backward(x, x, g, x.clone(), h0, dh_T, carries=kept)
    assert torch.equal(dh0, dh_T) and dx.numel() == dg.numel() == dbeta.numel() == 0
    dh0 = gdn.scan_backward(x, x, g, None, h0)[3]
    assert not bool(dh0.any())


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,C", [(700, 64), (5, 64), (300, 4096), (90, 33)])
def test_the_initial_states_gradient_over_the_last_ones(T, C):
    """dh0 in the place of dh_T, as the header allows."""
    from gated_deltanet_linear_20_b200 import recurrence as r
    d = to_dev(ref.scan_inputs([T], C, BF, seed=T + C))
    x, g, beta, dh = (d[k][None] for k in ("x", "g", "beta", "dh"))
    want = gdn.scan_backward(dh, x, g, beta, d["h0"], d["dh_T"])
    both = d["dh_T"].clone()
    dx, dg, dbeta = torch.empty_like(x), torch.empty_like(g), torch.empty_like(beta)
    scratch = torch.empty(-(-T // 16), C, device=DEV)
    p = lambda t: t.data_ptr()  # noqa: E731
    rc = r._lib.gdn_scan_backward(p(x), p(g), p(beta), p(d["h0"]), p(dh), p(both), p(dx), p(dg), p(dbeta),
                                  p(both), p(scratch), 0, 1, T, C, 1, None, stream())
    torch.cuda.synchronize()
    assert rc == 0
    for a, b in zip((dx, dg, dbeta, both), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,D", [(40, 128), (7, 33), (9, 4097), (300, 255), (5, 8192)])
def test_the_streams_gradient_over_the_one_that_reaches_it(rows, D):
    """dr in the place of dr_out, as the header allows."""
    from gated_deltanet_linear_20_b200 import norms as n
    d = to_dev(ref.norm_inputs(rows, D, x_dtype=BF, dtype=BF, r_dtype=F32, seed=D))
    want = gdn.residual_norm_backward(d["dy"], d["dr_out"], d["x"], d["r"], d["w"], w_post=d["w_post"])
    both, dx = d["dr_out"].clone(), torch.empty_like(d["x"])
    dw, dwp = torch.empty_like(d["w"]), torch.empty_like(d["w"])
    ws = torch.empty(n.workspace_bytes(rows, D, 2), dtype=torch.uint8, device=DEV)
    p = lambda t: t.data_ptr()  # noqa: E731
    rc = n._lib.gdn_residual_norm_backward(p(d["dy"]), p(both), p(d["x"]), p(d["r"]), p(d["w"]), None,
                                           p(d["w_post"]), None, p(dx), p(both), None, p(dw), p(dwp), None,
                                           rows, D, 1, 0, p(ws), ws.numel(), None, stream())
    torch.cuda.synchronize()
    assert rc == 0
    for a, b in zip((dx, both, dw, dwp), (want[0], want[1], want[3], want[4])):
        assert torch.equal(a, b)


def everything(d, cu):
    """A layer's forward and backward calls on packed tokens."""
    h, h_T, kept = gdn.scan_varlen(d["x"], d["g"], cu, d["beta"], d["h0"], save_carries=True)
    y, r = gdn.residual_norm(h, d["r"], d["w"], z=d["x"], w_post=d["w_post"], scale=d["scale"])
    o = gdn.gated_norm(y, d["w"], h)
    gy, gz, gw = gdn.gated_norm_backward(d["dh"], y, d["w"], h)
    grads = gdn.residual_norm_backward(gy, r, h, r, d["w"], z=d["x"], w_post=d["w_post"], scale=d["scale"])
    back = gdn.scan_varlen_backward(grads[0], d["x"], d["g"], cu, d["beta"], d["h0"], d["dh_T"], carries=kept)
    return [h, h_T, y, r, o, gz, gw, *grads, *back]


def layer(lens, C, seed):
    T = sum(lens)
    d = ref.scan_inputs(lens, C, BF, seed=seed)
    n = ref.norm_inputs(T, C, x_dtype=BF, dtype=BF, seed=seed + 1)
    d.update({k: n[k] for k in ("r", "w", "w_post", "scale")})
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    return to_dev(d), torch.tensor(cu, dtype=torch.int32, device=DEV)


def test_a_replayed_graph_takes_new_inputs_and_offsets():
    """The offsets are read on the device: the same total length, split in another way."""
    C, first, second = 520, [300, 0, 45, 600], [1, 500, 444, 0]
    d, cu = layer(first, C, 3)
    new, new_cu = layer(second, C, 7)
    want = [everything(d, cu), everything(new, new_cu)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = everything(d, cu)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want[0]))
    for k, v in new.items():
        d[k].copy_(v)
    cu.copy_(new_cu)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want[1]))


def test_two_streams_at_once():
    """Calls in flight side by side, and two captured graphs replayed on two streams,
    give what they give alone."""
    jobs = [layer([300, 0, 45, 600], 520, 3), layer([70] * 30, 256, 5)]
    want = [everything(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(everything(*jobs[i]))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for run in o for a, b in zip(run, w))
    graphs = []
    for j in jobs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, everything(*j)))
    for _ in range(5):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))
