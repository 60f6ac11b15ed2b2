"""Norms around a layer on the CPU: the 64-bit reference gradients against
differences, and the refusals of the C ABI (nothing reaches a device)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests import layer_reference as ref


@pytest.fixture(scope="module")
def norms():
    from gated_deltanet_linear_20_b200 import build
    build.build()
    from gated_deltanet_linear_20_b200 import norms as mod
    return mod


def directional(loss, d, name, want):
    """A central difference of step 1e-5 against the gradient along a random direction."""
    v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    diff = (loss({**d, name: d[name] + 1e-5 * v}) - loss({**d, name: d[name] - 1e-5 * v})) / 2e-5
    want = float((want * v).sum())
    assert abs(diff - want) <= 1e-7 * (1 + abs(want))


@pytest.mark.parametrize("name", ["x", "z", "w"])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_reference_gated_norm_gradients_match_differences(name, gate):
    d = ref.norm_inputs(4, 9, x_dtype=torch.float32, dtype=torch.float32, seed=1)
    d = {k: v.double() for k, v in d.items()}
    want = ref.gated_norm_backward(d, gate, 1e-3, 0.5)["d" + name][0]
    directional(lambda s: float((d["dy"] * ref.gated_norm(s, gate, 1e-3, 0.5)).sum()), d, name, want)


@pytest.mark.parametrize("name,post", [(n, True) for n in ("x", "r", "z", "w", "w_post", "scale")]
                         + [(n, False) for n in ("x", "r", "z", "w", "scale")])
def test_reference_residual_norm_gradients_match_differences(name, post):
    d = ref.norm_inputs(4, 9, x_dtype=torch.float32, dtype=torch.float32, seed=2, post=post)
    d = {k: v.double() if v is not None else None for k, v in d.items()}
    kept = {**d, "r": ref.residual_norm(d, "silu", 1e-3, 0.5)["r_out"][0]}
    want = ref.residual_norm_backward(kept, "silu", 1e-3, 0.5)["d" + name][0]

    def loss(s):
        f = ref.residual_norm(s, "silu", 1e-3, 0.5)
        return float((d["dy"] * f["y"][0]).sum() + (d["dr_out"] * f["r_out"][0]).sum())

    directional(loss, d, name, want)


# ------------------------------------------------------------------ refusals
P = 0x7f0000000000  # never dereferenced
MB = 1 << 24


def opts(norms, **over):
    a = dict(size=ctypes.sizeof(norms.NormOptions), eps=1e-6, weight_offset=0.0, gate=0)
    a.update(over)
    return ctypes.byref(norms.NormOptions(*a.values()))


def gated_args(**over):
    a = dict(x=P, xt=0, w=P + MB, z=P + 2 * MB, y=P + 3 * MB, rows=8, D=128, dt=1, opts=None, st=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -3), (dict(D=-1), -3), (dict(D=16385), -3), (dict(xt=2), -4), (dict(dt=-1), -4),
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(x=P + 2), -2),
    (dict(z=P + 2 * MB + 1), -2), (dict(w=P + MB + 2), -2), (dict(y=P), -5), (dict(y=P + 2 * MB), -5),
    (dict(y=P + MB), -5),
], ids=str)
def test_gated_norm_refuses(norms, over, code):
    assert norms._lib.gdn_gated_norm(*gated_args(**over)) == code


@pytest.mark.parametrize("over", [
    dict(size=8), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(weight_offset=float("nan")), dict(gate=2), dict(gate=-1),
], ids=str)
def test_norm_options_are_checked(norms, over):
    assert norms._lib.gdn_gated_norm(*gated_args(opts=opts(norms, **over))) == -4


def gated_backward_args(**over):
    a = dict(dy=P, x=P + MB, xt=0, w=P + 2 * MB, z=P + 3 * MB, dx=P + 4 * MB, dz=P + 5 * MB,
             dw=P + 6 * MB, rows=8, D=128, dt=1, ws=P + 7 * MB, n=8 * 128 * 4, opts=None, st=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -3), (dict(D=1 << 20), -3), (dict(dt=9), -4), (dict(dy=None), -1),
    (dict(dx=None), -1), (dict(dw=None), -1), (dict(dz=None), -1), (dict(z=None), -1),
    (dict(dx=P + 4 * MB + 2), -2), (dict(dw=P + 6 * MB + 1), -2),
    (dict(ws=None), -8), (dict(ws=P + 7 * MB + 128), -8), (dict(n=8 * 128 * 4 - 1), -8),
    (dict(dx=P + MB), -5), (dict(dz=P), -5), (dict(dw=P + 2 * MB), -5), (dict(ws=P + 4 * MB), -5),
], ids=str)
def test_gated_norm_backward_refuses(norms, over, code):
    assert norms._lib.gdn_gated_norm_backward(*gated_backward_args(**over)) == code


def residual_args(**over):
    a = dict(x=P, r=P + MB, w=P + 2 * MB, z=P + 3 * MB, wp=P + 4 * MB, sc=P + 5 * MB, y=P + 6 * MB,
             ro=P + 7 * MB, rows=8, D=128, dt=1, rt=0, opts=None, st=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -3), (dict(D=16392), -3), (dict(dt=0, rt=1), -4), (dict(rt=3), -4),
    (dict(x=None), -1), (dict(r=None), -1), (dict(w=None), -1), (dict(y=None), -1),
    (dict(ro=None), -1), (dict(r=P + MB + 2), -2), (dict(sc=P + 5 * MB + 2), -2),
    (dict(y=P), -5), (dict(ro=P + MB + 4), -5), (dict(ro=P + 6 * MB), -5), (dict(y=P + 4 * MB), -5),
], ids=str)
def test_residual_norm_refuses(norms, over, code):
    assert norms._lib.gdn_residual_norm(*residual_args(**over)) == code


def residual_backward_args(**over):
    a = dict(dy=P, dro=P + MB, x=P + 2 * MB, ro=P + 3 * MB, w=P + 4 * MB, z=P + 5 * MB,
             wp=P + 6 * MB, sc=P + 7 * MB, dx=P + 8 * MB, dr=P + 9 * MB, dz=P + 10 * MB,
             dw=P + 11 * MB, dwp=P + 12 * MB, dsc=P + 13 * MB, rows=8, D=128, dt=1, rt=0,
             ws=P + 14 * MB, n=3 * 8 * 128 * 4, opts=None, st=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -3), (dict(dt=0, rt=1), -4), (dict(dy=None), -1), (dict(ro=None), -1),
    (dict(dr=None), -1), (dict(dwp=None), -1), (dict(wp=None), -1), (dict(sc=None), -1),
    (dict(dz=None), -1), (dict(dw=None), -1), (dict(dr=P + 9 * MB + 2), -2), (dict(ws=None), -8),
    (dict(n=3 * 8 * 128 * 4 - 1), -8), (dict(dr=P + MB + 4), -5), (dict(dx=P + 2 * MB), -5),
    (dict(dr=P + 3 * MB), -5), (dict(dsc=P + 12 * MB), -5), (dict(ws=P + 13 * MB), -5),
], ids=str)
def test_residual_norm_backward_refuses(norms, over, code):
    assert norms._lib.gdn_residual_norm_backward(*residual_backward_args(**over)) == code


def test_no_rows_is_a_noop(norms):
    none = dict(x=None, w=None, z=None, y=None)
    assert norms._lib.gdn_gated_norm(*gated_args(rows=0, **none)) == 0
    assert norms._lib.gdn_gated_norm(*gated_args(D=0, **none)) == 0
    assert norms._lib.gdn_residual_norm(*residual_args(rows=0, x=None, r=None, y=None, ro=None)) == 0


def test_workspace_bytes(norms):
    assert norms.workspace_bytes(8, 128, 1) == 8 * 128 * 4
    assert norms.workspace_bytes(1 << 20, 128, 1) == 592 * 128 * 4
    assert norms.workspace_bytes(1 << 20, 4096, 3) == 296 * 4096 * 12
    assert norms.workspace_bytes(0, 128) == norms.workspace_bytes(5, 0) == 0
    assert norms.workspace_bytes(5, 128, 4) == norms.workspace_bytes(-1, 128) == 0


def test_bindings_refuse_cpu_tensors_and_unknown_gates(norms):
    import gated_deltanet_linear_20_b200 as gdn
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda: gdn.gated_norm(x, w), lambda: gdn.residual_norm(x, x, w),
                 lambda: gdn.gated_norm_backward(x, x, w),
                 lambda: gdn.residual_norm_backward(x, x, x, x, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="gate"):
        norms._options(1e-6, 0.0, "tanh")
