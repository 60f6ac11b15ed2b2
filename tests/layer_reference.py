"""Plain 64-bit forms of the channel recurrence on the CPU, token by token, and
the rounding bounds that the GPU tests hold the kernels to."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24          # half a step of fp32, relative
HALF_STEP = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}


def scan_inputs(lens, C, dtype, *, seed, beta=True, h0=True, mean=2.0, g=None):
    """Packed inputs of sequences of the given lengths (CPU)."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(
        x=r(T, C).to(dtype),
        g=torch.nn.functional.logsigmoid(r(T, C) + mean) if g is None else g(r(T, C)),
        beta=torch.sigmoid(r(T, C)).to(dtype) if beta else None,
        h0=r(N, C) if h0 else None,
        dh=r(T, C).to(dtype), dh_T=r(N, C))


def scan(d, lens):
    """h, h_T, the state before every token, and err: the rounding bound of h.

    A computed state differs from the exact one by at most K * U32 * err with a
    small K.  err follows the recurrence: a token's decay is off by at most a few
    steps (its exponential, the product with the state, the sum) and, where runs
    are joined by exp(sum of g), by |g| half steps for the sum; both act on the
    magnitude mag the state can have."""
    C = d["x"].shape[1]
    x, g = d["x"].double(), d["g"].double()
    u = x * d["beta"].double() if d["beta"] is not None else x
    h, before, err, err_before = (torch.zeros_like(x) for _ in range(4))
    h_T = torch.zeros(len(lens), C, dtype=torch.float64)
    err_T = torch.zeros_like(h_T)
    t = 0
    for n, m in enumerate(lens):
        s = d["h0"][n].double() if d["h0"] is not None else torch.zeros(C, dtype=torch.float64)
        mag, e = s.abs(), torch.zeros(C, dtype=torch.float64)
        for _ in range(m):
            before[t], err_before[t] = s, e
            a = g[t].exp()
            e = a * e + (1 + g[t].abs()) * a * mag
            s = a * s + u[t]
            mag = a * mag + u[t].abs()
            e = e + mag
            h[t], err[t] = s, e
            t += 1
        h_T[n], err_T[n] = s, e
    return dict(h=h, h_T=h_T, before=before, err=err, err_T=err_T, err_before=err_before)


def scan_backward(d, lens):
    """Gradients by the formulas, and a rounding bound for each (as in scan)."""
    f = scan(d, lens)
    x, g = d["x"].double(), d["g"].double()
    beta = d["beta"].double() if d["beta"] is not None else torch.ones_like(x)
    a = g.exp()
    lam, el, maglam = (torch.zeros_like(x) for _ in range(3))
    N, C = len(lens), x.shape[1]
    dh0 = torch.zeros(N, C, dtype=torch.float64)
    eh0 = torch.zeros_like(dh0)
    end = sum(lens)
    for n in reversed(range(N)):
        mu = d["dh_T"][n].double() if d["dh_T"] is not None else torch.zeros(C, dtype=torch.float64)
        mag, e = mu.abs(), torch.zeros(C, dtype=torch.float64)
        for t in range(end - 1, end - 1 - lens[n], -1):
            lam[t] = d["dh"][t].double() + mu
            mag = mag + d["dh"][t].double().abs()
            el[t] = e + mag
            maglam[t] = mag
            mu = a[t] * lam[t]
            e = a[t] * el[t] + (1 + g[t].abs()) * a[t] * mag
            mag = a[t] * mag
        end -= lens[n]
        dh0[n], eh0[n] = mu, e
    hp = f["before"]
    dg = lam * a * hp
    edg = a * (el * hp.abs() + maglam * f["err_before"]) + (3 + g.abs()) * dg.abs()
    return dict(dx=beta * lam, dg=dg, dbeta=x * lam, dh0=dh0,
                edx=beta.abs() * (el + maglam), edg=edg, edbeta=x.abs() * (el + maglam), edh0=eh0)


#: Steps of a bound: expf is off by at most one unit in the last place (two half
#: steps), the product with the state and the sum by half a step each; a join
#: adds one exponential and one multiply-add to a run of at least 8 tokens.
STEPS = 5


def assert_within(got, ref, err, dtype, what):
    """|got - ref| <= STEPS U32 err + half a step of the output's type (and the
    smallest fp32 numbers, which results may be flushed to or rounded among)."""
    got, ref = got.detach().double().cpu(), ref.cpu()
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} != {tuple(ref.shape)}"
    half = HALF_STEP[dtype]
    tol = STEPS * U32 * err * (1 + half) + half * ref.abs() + 2.0 ** -126
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst "
                           f"{float(((got - ref).abs() / tol).nan_to_num(float('inf')).max()):.3g} x")
