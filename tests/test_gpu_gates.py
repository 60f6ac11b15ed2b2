"""The gates' values and slopes, relative to themselves as far as they are normal fp32
numbers: rows of ones with weights of one and no eps make y the gate and dz its slope."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U32 = 2.0 ** -24


def points(D):
    """From -103 to 103, denser around zero, and tiny ones."""
    z = torch.cat([torch.linspace(-103, 103, D // 2), torch.linspace(-12, 12, D // 4),
                   torch.linspace(-1.4, 1.4, D - D // 2 - D // 4)])
    z[:4] = torch.tensor([1e-30, -1e-30, 0.0, -0.0])
    return z


@pytest.mark.parametrize("D", [64, 250, 255, 4096, 6150, 8191])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_values_and_slopes(gate, D):
    """Half steps of fp32: 4 of the power's stated error and 2.4 |z| of its exponent (as
    in tests/layer_reference.py), which act on exp(-|z|) only; 2 of the reciprocal, 2 of
    the sum before it, and 12 products, among them those with the root (two steps)."""
    z = points(D)
    ones = torch.ones(1, D, device=DEV)
    w = torch.ones(D, device=DEV)
    y = gdn.gated_norm(ones, w, z[None].to(DEV), gate=gate, eps=0.0)[0].double().cpu()
    dz = gdn.gated_norm_backward(ones, ones, w, z[None].to(DEV), gate=gate, eps=0.0)[1][0].double().cpu()
    zd = z.double()
    p, q = 1 / (1 + torch.exp(-zd)), 1 / (1 + torch.exp(zd))
    a = zd * p if gate == "silu" else p
    da = p * (1 + zd * q) if gate == "silu" else p * q
    size = p * (1 + zd.abs() * q) if gate == "silu" else da
    steps = 20 + 2.4 * zd.abs()
    # an exponential below the normal numbers, 2^-126, may count as zero; |z| times that
    least = (zd.abs() > 87) * (1 + zd.abs()) * 2.0 ** -126
    assert bool(((y - a).abs() <= steps * U32 * a.abs() + least).all())
    assert bool(((dz - da).abs() <= 2 * steps * U32 * size + least).all())


@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_the_residual_norms_gate_has_the_same_slope(gate):
    D = 512
    z, ones, w = points(D), torch.ones(1, D, device=DEV), torch.ones(D, device=DEV)
    want = gdn.gated_norm_backward(ones, ones, w, z[None].to(DEV), gate=gate, eps=0.0)[1]
    # r' of zero with an eps has no gradient of its own: dr is dr_out
    dz = gdn.residual_norm_backward(torch.zeros_like(ones), ones, ones, torch.zeros_like(ones), w,
                                    z=z[None].to(DEV), gate=gate)[2]
    assert bool(((dz - want).abs() <= 8 * U32 * want.abs() + 2.0 ** -148).all())


def test_infinite_gates():
    z = torch.tensor([float("inf"), -float("inf"), float("nan"), 3e38, -3e38], device=DEV)[None]
    x, w = torch.ones(1, 5, device=DEV), torch.ones(5, device=DEV)
    p = gdn.gated_norm(x, w, z, gate="sigmoid", eps=0.0)[0].tolist()
    assert p[0] == 1 and p[1] == 0 and p[2] != p[2] and p[3] == 1 and p[4] == 0
    dz = gdn.gated_norm_backward(x, x, w, z, gate="sigmoid", eps=0.0)[1][0].tolist()
    assert dz[0] == 0 and dz[1] == 0 and dz[3] == 0 and dz[4] == 0
    y = gdn.gated_norm(x, w, z, eps=0.0)[0].tolist()
    assert y[0] == float("inf") and y[3] > 2e38 and y[4] == 0
