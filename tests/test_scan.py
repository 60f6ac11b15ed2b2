"""Channel recurrence on the CPU: the 64-bit reference against its invariants and
differences, and the refusals of the C ABI (nothing reaches a device)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from tests import layer_reference as ref


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_20_b200 import build
    build.build()
    from gated_deltanet_linear_20_b200 import gdn, recurrence  # noqa: F401  (argument types)
    return gdn._lib


# ------------------------------------------------------------------ the reference itself
def test_reference_keeps_the_state_without_input_or_decay():
    d = ref.scan_inputs([7, 0, 3], 5, torch.float32, seed=0, g=torch.zeros_like)
    d["beta"] = torch.zeros_like(d["beta"])
    f = ref.scan(d, [7, 0, 3])
    assert torch.equal(f["h_T"], d["h0"].double())


def test_reference_sums_the_inputs_without_decay():
    d = ref.scan_inputs([9], 4, torch.float32, seed=1, beta=False, h0=False, g=torch.zeros_like)
    assert torch.allclose(ref.scan(d, [9])["h"], d["x"].double().cumsum(0), rtol=1e-14, atol=1e-14)


@pytest.mark.parametrize("name", ["x", "g", "beta", "h0"])
def test_reference_gradients_match_differences(name):
    """d(loss)/d(input) along a random direction, loss = <dh, h> + <dh_T, h_T>:
    a central difference of step 1e-5 is off by about 1e-10 of the third
    derivative and 1e-11 of the loss."""
    lens = [5, 0, 1, 11]
    d = ref.scan_inputs(lens, 3, torch.float32, seed=2)
    d = {k: v.double() for k, v in d.items()}
    grads = ref.scan_backward(d, lens)
    v = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)

    def loss(s):
        f = ref.scan({**d, name: d[name] + s * v}, lens)
        return float((d["dh"] * f["h"]).sum() + (d["dh_T"] * f["h_T"]).sum())

    diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
    want = float((grads["d" + name] * v).sum())
    assert abs(diff - want) <= 1e-7 * (1 + abs(want))


# ------------------------------------------------------------------ refusals
P = 0x7f0000000000  # never dereferenced: every call below is refused first
MB = 1 << 24


def scan_args(**over):
    a = dict(x=P, g=P + MB, beta=P + 2 * MB, h0=P + 3 * MB, h=P + 4 * MB, h_T=P + 5 * MB,
             carries=P + 6 * MB, B=2, T=40, C=64, dtype=1, status=None, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -3), (dict(T=-1), -3), (dict(C=-1), -3),
    (dict(B=1 << 16, T=1 << 15), -3),                       # 2^31 tokens
    (dict(B=1, T=1 << 30, C=1 << 20), -3),                  # 2^50 elements
    (dict(dtype=2), -4), (dict(dtype=-1), -4),
    (dict(x=None), -1), (dict(g=None), -1), (dict(h=None), -1), (dict(h_T=None), -1),
    (dict(x=P + 1), -2), (dict(h=P + 4 * MB + 1), -2), (dict(g=P + MB + 2), -2),
    (dict(h_T=P + 5 * MB + 2), -2), (dict(h0=P + 3 * MB + 1), -2), (dict(dtype=0, x=P + 2), -2),
    (dict(carries=P + 6 * MB + 2), -2),
    (dict(h=P), -5), (dict(h=P + MB + 64), -5), (dict(h_T=P + 2 * MB), -5),
    (dict(h_T=P + 3 * MB + 4), -5),                         # partly over h0
    (dict(h=P + 3 * MB), -5), (dict(h=P + 5 * MB), -5), (dict(carries=P + 4 * MB + 4), -5),
    (dict(status=P + 7 * MB + 1), -2), (dict(status=P + 4 * MB), -5),
], ids=str)
def test_scan_refuses(lib, over, code):
    assert lib.gdn_scan(*scan_args(**over)) == code


def varlen_args(**over):
    a = dict(x=P, g=P + MB, beta=P + 2 * MB, h0=P + 3 * MB, h=P + 4 * MB, h_T=P + 5 * MB,
             carries=P + 6 * MB, cu=P + 7 * MB, N=2, T=40, C=64, dtype=1, status=P + 8 * MB,
             stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(N=-1), -3), (dict(T=-1), -3), (dict(cu=None), -1), (dict(cu=P + 7 * MB + 2), -2),
    (dict(status=P + 8 * MB + 1), -2), (dict(cu=P + 4 * MB), -5), (dict(status=P + 7 * MB), -5),
    (dict(status=P + 5 * MB), -5), (dict(dtype=7), -4),
], ids=str)
def test_scan_varlen_refuses(lib, over, code):
    assert lib.gdn_scan_varlen(*varlen_args(**over)) == code


def step_args(**over):
    a = dict(x=P, g=P + MB, beta=P + 2 * MB, state=P + 3 * MB, h=P + 4 * MB, B=2, C=64, dtype=1,
             stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -3), (dict(C=-2), -3), (dict(dtype=3), -4), (dict(x=None), -1),
    (dict(state=None), -1), (dict(h=None), -1), (dict(g=None), -1), (dict(g=P + MB + 1), -2),
    (dict(state=P + 3 * MB + 2), -2), (dict(h=P), -5), (dict(state=P + MB), -5),
    (dict(h=P + 3 * MB + 128), -5),
], ids=str)
def test_scan_step_refuses(lib, over, code):
    assert lib.gdn_scan_step(*step_args(**over)) == code


def backward_args(**over):
    a = dict(x=P, g=P + MB, beta=P + 2 * MB, h0=P + 3 * MB, dh=P + 4 * MB, dh_T=P + 5 * MB,
             dx=P + 6 * MB, dg=P + 7 * MB, dbeta=P + 8 * MB, dh0=P + 9 * MB, carries=P + 10 * MB,
             valid=1, B=2, T=40, C=64, dtype=1, status=None, stream=None)
    a.update(over)
    return list(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -3), (dict(T=-1), -3), (dict(C=-1), -3), (dict(dtype=5), -4),
    (dict(x=None), -1), (dict(dh=None), -1), (dict(dx=None), -1), (dict(dg=None), -1),
    (dict(carries=None), -1), (dict(dbeta=None), -1), (dict(beta=None), -1),
    (dict(dx=P + 6 * MB + 1), -2), (dict(dg=P + 7 * MB + 2), -2), (dict(dh_T=P + 5 * MB + 2), -2),
    (dict(dx=P + 4 * MB), -5), (dict(dg=P + MB), -5), (dict(dbeta=P + 2 * MB), -5),
    (dict(dh0=P + 3 * MB), -5), (dict(dh0=P + 5 * MB + 4), -5), (dict(dx=P + 8 * MB), -5),
    (dict(carries=P), -5), (dict(status=P + 6 * MB), -5),
], ids=str)
def test_scan_backward_refuses(lib, over, code):
    assert lib.gdn_scan_backward(*backward_args(**over)) == code


def test_scan_empty_problems_are_noops(lib):
    none = dict(x=None, g=None, beta=None, h0=None, h=None, h_T=None, carries=None)
    assert lib.gdn_scan(*scan_args(B=0, **none)) == 0
    assert lib.gdn_scan(*scan_args(C=0, **none)) == 0
    assert lib.gdn_scan_varlen(*varlen_args(N=0, T=0, cu=None, status=None, **none)) == 0
    assert lib.gdn_scan_step(*step_args(B=0, x=None, g=None, state=None, h=None, beta=None)) == 0


def test_scan_carry_bytes(lib):
    f = lib.gdn_scan_carry_bytes
    assert f(2, 2 * 40, 64, 0) == 2 * 3 * 64 * 4
    assert f(3, 40, 64, 1) == (2 + 3) * 64 * 4
    assert f(0, 0, 64, 0) == 0 and f(-1, 5, 5, 0) == 0 and f(1, 1, 1, 1) == 4
    assert ctypes.c_size_t(f(1, 1 << 30, 4096, 0)).value == (1 << 26) * 4096 * 4


def test_bindings_refuse_cpu_tensors(lib):
    import gated_deltanet_linear_20_b200 as gdn
    x, g = torch.zeros(1, 2, 4), torch.zeros(1, 2, 4)
    for call in (lambda: gdn.scan(x, g), lambda: gdn.scan_step(x[0], g[0], g[0].clone()),
                 lambda: gdn.scan_backward(x, x, g),
                 lambda: gdn.scan_varlen(x[0], g[0], torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
