"""The channel recurrence at the ends of the fp32 range: decays below the normal
numbers count, in whole sequences as in single tokens."""
from __future__ import annotations

import math

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = torch.float32


@pytest.mark.parametrize("C", [127, 299, 300, 600])
def test_a_decay_below_the_normal_numbers_then_growth(C):
    """Channel c: a decay of exp(-90) at token c, growth of exp(80) at the next, no
    input.  exp(-90) is 5.8e5 steps of the smallest fp32 numbers: rounding the
    exponential (at most 2 steps) and its product with the state (half a step, where
    it is one) leaves 4.3e-6 of it; exp(80), at most 2 units in the last place,
    products and a sum of 170 in the exponent add less than 1.1e-5 more."""
    T = C + 2
    at = torch.arange(C)
    g = torch.zeros(T, C)
    g[at, at] = -90.0
    g[at + 1, at] = 80.0
    g, x = g.to(DEV), torch.zeros(T, C, device=DEV)
    h0 = torch.full((1, C), 1.0, device=DEV)
    tol = 1.6e-5
    h, h_T, kept = gdn.scan(x[None], g[None], None, h0, save_carries=True)
    end = math.exp(-10.0)
    assert bool(((h_T - end).abs() <= tol * end).all())
    state = h0[0].clone()[None]
    for t in range(T):
        hs = gdn.scan_step(x[t:t + 1], g[t:t + 1], state)
        assert bool(((h[0, t] - hs[0]).abs() <= 2 * tol * hs[0].abs()).all()), t
    # the gradient of the last state: lam = exp(80) between the two tokens
    dh_T = torch.ones(1, C, device=DEV)
    for carries in (kept, None):
        dx, dg, _, dh0 = gdn.scan_backward(torch.zeros_like(x)[None], x[None], g[None], None, h0, dh_T,
                                           carries=carries)
        assert bool(((dh0 - end).abs() <= tol * end).all())
        # dg_t = lam_t exp(g_t) h_{t-1}: exp(-10) at every token
        assert bool(((dg - end).abs() <= 2 * tol * end).all())
        assert bool(((dx[0].diagonal() - math.exp(80.0)).abs() <= tol * math.exp(80.0)).all())
