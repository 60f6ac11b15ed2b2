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


def growth(T, C, g, h0, x_last=0.0):
    x = torch.zeros(1, T, C, device=DEV)
    x[:, -1] = x_last
    return x, torch.full((1, T, C), g, device=DEV), torch.full((1, C), h0, device=DEV)


@pytest.mark.parametrize("C", [33, 64])
def test_growth_in_range_over_a_run_is_exact(C):
    """1024 tokens that grow a small state by exp(102.4) in all, 12.8 over 128: the
    sums of 16 decays are off by at most 16 roundings of 1.6, the exponentials by 2
    units: below 64 (16 0.8 + 4) + 1024 half steps, 1.3e-4."""
    x, g, h0 = growth(1024, C, 0.1, 1e-30)
    h, h_T = gdn.scan(x, g, None, h0)
    t = torch.arange(1, 1025, dtype=torch.float64)
    want = float(h0[0, 0]) * torch.exp(t * float(g[0, 0, 0]))
    assert bool((((h[0].double().cpu() - want[:, None]) / want[:, None]).abs() <= 1.3e-4).all())
    assert bool(((h_T.double().cpu() - want[-1]).abs() <= 1.3e-4 * want[-1]).all())


@pytest.mark.parametrize("B,T,C", [(1, 2048, 64), (1, 2048, 4096), (8, 128, 64), (20, 200, 2048), (3, 500, 33)])
@pytest.mark.parametrize("g", [0.9, 2.0, 7.0])
def test_growth_past_the_range_is_right_or_infinite(B, T, C, g):
    """A state that grows past the fp32 range over neighbouring tokens: right, or
    infinite, never a wrong number; and infinite in the end."""
    x, gg, h0 = growth(T, C, g, 1e-30)
    x, gg, h0 = (t.expand(B, *t.shape[1:]).contiguous() for t in (x, gg, h0))
    h, h_T = gdn.scan(x, gg, None, h0)
    t = torch.arange(1, T + 1, dtype=torch.float64)
    want = (torch.log(h0[0, 0].double()).cpu() + t * float(gg[0, 0, 0])).exp()[:, None]
    got = h.double().cpu()
    # at most a rounding of the sums and exponents a token
    ok = ((got - want).abs() <= (1e-6 * t[:, None] + 1e-5 * g) * want) | (got == float("inf"))
    assert bool(ok.all())
    if -math.log(1e30) + g * T > 90:
        assert bool((h_T == float("inf")).all())


def test_a_decay_to_nothing_outweighs_growth():
    """Growth by exp(95) and g = -inf within the same 128 tokens, in either order: the
    state begins anew there."""
    T, C = 512, 64
    x, g, h0 = growth(T, C, -0.05, 1e-30)
    x[0, 450] = 3.0
    g = g.cpu()
    for c in range(C):
        first = c // 2
        g[0, first:first + 95, c] = 1.0
        g[0, first + 95, c] = -math.inf
        g[0, 130 + first, c] = -math.inf
        g[0, 131 + first:226 + first, c] = 1.0
    h, h_T = gdn.scan(x, g.to(DEV), None, h0)
    assert bool((h[0, 450] == 3.0).all())
    want = 3.0 * math.exp(-0.05 * 61)  # 61 decays of a few half steps each
    assert bool(((h_T - want).abs() <= 1e-4 * want).all())


@pytest.mark.parametrize("B,T,C", [(1, 1100, 64), (1, 700, 4096), (2, 300, 33)])
def test_an_infinite_state_stays_visible(B, T, C):
    """Infinite inputs and states: what single tokens leave infinite or NaN is so in
    whole sequences, the other channels and tokens are as without them."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(B, T, C, generator=gen)
    g = torch.nn.functional.logsigmoid(torch.randn(B, T, C, generator=gen) + 1)
    h0 = torch.randn(B, C, generator=gen)
    clean = gdn.scan(x.to(DEV), g.to(DEV), None, h0.to(DEV))[0]
    x[:, 50, 5], x[:, 90, 9], h0[:, 20] = math.inf, -math.inf, math.inf
    h, h_T = gdn.scan(x.to(DEV), g.to(DEV), None, h0.to(DEV))
    assert not bool(h[:, 50:, 5].isfinite().any()) and not bool(h[:, 90:, 9].isfinite().any())
    assert not bool(h[:, :, 20].isfinite().any()) and not bool(h_T[:, [5, 9, 20]].isfinite().any())
    assert bool((h[:, 50, 5] == math.inf).all()) and bool((h[:, 90, 9] == -math.inf).all())
    h[:, 50:, 5], h[:, 90:, 9], h[:, :, 20] = clean[:, 50:, 5], clean[:, 90:, 9], clean[:, :, 20]
    assert torch.equal(h, clean)
