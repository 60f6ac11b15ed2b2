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


#: Steps of a bound, in half steps of fp32.  A token: the approximate power of two
#: is off by 2^1.5 (its stated bound of 2^-22.5), the rounding of g log2 e adds
#: 1.5 |g|, the products with the state and of x with beta and the sum one each on
#: the magnitudes: at most 5 (1 + |g|) on the decayed state's and 5 on the new
#: one's.  A join over 16 tokens replaces their 80 + 5 |G| steps by those of one
#: power, of its product and sum, and of the sum G of their log decays (8 |G|, the
#: partial sums growing evenly): fewer as long as |G| is below 17.
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


# ---------------------------------------------------------------- norms
def act(name, z):
    """The gate's value and slope in 64 bits."""
    if z is None:
        return 1.0, None
    p = torch.sigmoid(z)
    return (z * p, p * (1 + z * (1 - p))) if name == "silu" else (p, p * (1 - p))


def slope_size(name, z):
    """Size of the terms in the gate's slope, which cancel where it crosses zero."""
    p = torch.sigmoid(z)
    return p * (1 + z.abs()) if name == "silu" else p


def norm_inputs(rows, D, *, x_dtype, dtype, r_dtype=None, seed, z=True, post=True, scale=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    rt = r_dtype or dtype
    return dict(x=(r(rows, D) * torch.exp(r(rows, 1))).to(x_dtype), w=1 + 0.3 * r(D),
                z=(2 * r(rows, D)).to(dtype) if z else None, dy=r(rows, D).to(dtype),
                r=r(rows, D).to(rt), dr_out=r(rows, D).to(rt),
                w_post=1 + 0.3 * r(D) if post else None, scale=0.5 + 0.2 * r(D) if scale else None)


def _grad(x, w, u, mu, eps):
    """Gradients of w x / rms(x) by x and by w (row by row), given the gradient u of
    the result and the size mu of u's terms; each with the size of its terms."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    dx = r * (u * w - xh * (u * w * xh).mean(-1, keepdim=True))
    m = mu * w.abs()
    mx = r * (m + xh.abs() * (m * xh.abs()).mean(-1, keepdim=True))
    return (dx, mx), (u * xh, mu * xh.abs())


def _sum(pair):
    return pair[0].sum(0), pair[1].sum(0)


def gated_norm(d, name="silu", eps=1e-6, offset=0.0):
    x, w = d["x"].double(), d["w"].double() + offset
    a, _ = act(name, d["z"].double() if d["z"] is not None else None)
    return w * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * a


def gated_norm_backward(d, name="silu", eps=1e-6, offset=0.0):
    """{gradient: (value, size of its terms)}."""
    x, w, dy = d["x"].double(), d["w"].double() + offset, d["dy"].double()
    z = d["z"].double() if d["z"] is not None else None
    a, da = act(name, z)
    u = dy * a
    dx, dw = _grad(x, w, u, u.abs(), eps)
    out = dict(dx=dx, dw=_sum(dw))
    if z is not None:
        t = dy * w * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
        out["dz"] = (t * da, t.abs() * slope_size(name, z))
    return out


def residual_norm(d, name="silu", eps=1e-6, offset=0.0):
    """y and r_out, each with the size of its terms."""
    x, r, w = d["x"].double(), d["r"].double(), d["w"].double() + offset
    u = x
    if d["w_post"] is not None:
        u = (d["w_post"].double() + offset) * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    if d["z"] is not None:
        u = u * act(name, d["z"].double())[0]
    if d["scale"] is not None:
        u = u * d["scale"].double()
    s, m = r + u, r.abs() + u.abs()
    rstd = torch.rsqrt((s * s).mean(-1, keepdim=True) + eps)
    # an error of m in the sum moves y by w rstd m, and through rstd by at most
    # |y| times the mean of |s| m over the mean of s^2
    through = (s.abs() * m).mean(-1, keepdim=True) * rstd * rstd
    y = w * s * rstd
    return dict(y=(y, w.abs() * rstd * m + y.abs() * (1 + through)), r_out=(s, m))


def residual_norm_backward(d, name="silu", eps=1e-6, offset=0.0):
    """As gated_norm_backward; d["r"] is the kept sum."""
    x, r, w, dy = (d[k].double() for k in ("x", "r", "w", "dy"))
    z = d["z"].double() if d["z"] is not None else None
    a, da = act(name, z)
    (dr, mr), dw = _grad(r, w + offset, dy, dy.abs(), eps)
    if d["dr_out"] is not None:
        dr, mr = dr + d["dr_out"].double(), mr + d["dr_out"].double().abs()
    u = x
    if d["w_post"] is not None:
        wp = d["w_post"].double() + offset
        u = wp * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    sc = d["scale"].double() if d["scale"] is not None else torch.ones_like(w)
    out = dict(dr=(dr, mr), dw=_sum(dw))
    if d["scale"] is not None:
        out["dscale"] = _sum((dr * a * u, mr * abs(a) * u.abs()))
    if z is not None:
        out["dz"] = (dr * sc * u * da, mr * sc.abs() * u.abs() * slope_size(name, z))
    v, mv = dr * sc * a, mr * sc.abs() * abs(a)
    if d["w_post"] is None:
        out["dx"] = (v, mv)
    else:
        out["dx"], dwp = _grad(x, wp, v, mv, eps)
        out["dw_post"] = _sum(dwp)
    return out


def norm_steps(n, zmax):
    """Half steps of fp32 by which a result may be off, relative to the size of its
    terms, with sums of n terms in all on its way: the terms' own roundings
    (products, two roots of two steps, means: 16), the gate's exponential (its
    stated bound of 2 + 1.2 |z| units in the last place is twice that in half
    steps) and quotient (2 units), and one rounding an addition along the
    longest chain, n at most."""
    return 16 + 2 * (4 + 1.2 * zmax) + n


def assert_norm(got, want, steps, dtype, what):
    ref, size = want
    got, half = got.detach().double().cpu(), HALF_STEP[dtype]
    assert got.shape == ref.shape, f"{what}: {tuple(got.shape)} != {tuple(ref.shape)}"
    tol = steps * U32 * size * (1 + half) + half * ref.abs() + 2.0 ** -126
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst "
                           f"{float(((got - ref).abs() / tol).nan_to_num(float('inf')).max()):.3g} x")
