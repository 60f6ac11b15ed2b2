"""Measured cases of the channel recurrence (scan) and of the norms around a layer.

Each case names one operator, its sizes and types.  ``run`` computes it in its
plain form (elementary torch operations in 32 bits, rounded once at the end)
or, with ``own``, through the library's entry points.  ``exact`` is the
definition in 64 bits: token by token for the recurrence, through autograd for
the norms' gradients.
"""
import math
import random

import torch

own = False

EPS = 1e-6
CARRY_TOKENS = 16  # tokens between saved states of a training forward
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one very long sequence read at once (prefill of a long document, 4096 channels)
        dict(name="scan_long", op="scan", dtype="bf16", B=1, T=32768, C=4096, beta=True, h0=False, carries=False),
        # the forward pass of a training step: the states that the backward pass needs are kept
        dict(name="scan_train", op="scan", dtype="bf16", B=4, T=4096, C=2048, beta=True, h0=False, carries=True),
        # a serving batch of 32 prompts of different lengths packed together, states carried on
        dict(name="scan_packed", op="scan_varlen", dtype="bf16", N=32, T=16384, C=2048, beta=False, h0=True),
        # one token of each of 64 sequences: latency
        dict(name="scan_step", op="scan_step", dtype="bf16", B=64, C=4096, beta=True),
        # the gradient of the training forward above, with the states it kept
        dict(name="scan_backward", op="scan_backward", dtype="bf16", B=4, T=4096, C=2048, beta=True, h0=False, carries=True),
        # a small ragged packed batch in 32 bits with an odd channel count, nothing kept from the forward pass
        dict(name="scan_backward_odd", op="scan_varlen_backward", dtype="f32", N=5, T=2885, C=577, beta=True, h0=True, carries=False),
        # o of a batched prefill (16384 tokens x 32 heads x 128), normalised per head and gated
        dict(name="gated_norm_prefill", op="gated_norm", rows=524288, D=128, x_dtype="bf16", dtype="bf16", z=True, act="silu"),
        # o of a decode step, 64 sequences x 16 heads, still in 32 bits: latency
        dict(name="gated_norm_decode", op="gated_norm", rows=1024, D=128, x_dtype="f32", dtype="bf16", z=True, act="silu"),
        # its gradient over 4096 tokens x 32 heads, o kept in 32 bits
        dict(name="gated_norm_backward", op="gated_norm_backward", rows=131072, D=128, x_dtype="f32", dtype="bf16", z=True, act="silu"),
        # between two layers of a prefill: norm after the block, its scale, the residual, norm before the next
        dict(name="residual_norm_prefill", op="residual_norm", rows=8192, D=4096, dtype="bf16", r_dtype="bf16", z=False, post=True, scale=True, act="silu"),
        # the same in a decode step of 64 sequences, 16 heads x 128 channels: latency
        dict(name="residual_norm_decode", op="residual_norm", rows=64, D=2048, dtype="bf16", r_dtype="bf16", z=False, post=True, scale=True, act="silu"),
        # a training step's gradient with everything on and the residual stream in 32 bits
        dict(name="residual_norm_backward", op="residual_norm_backward", rows=4096, D=4096, dtype="bf16", r_dtype="f32", z=True, post=True, scale=True, act="sigmoid"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan_varlen", "scan_step", "scan_backward", "scan_varlen_backward",
                     "gated_norm", "gated_norm_backward", "residual_norm", "residual_norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        most = 1 << 25
        C = _log(rng, 1, 8192) if rng.random() < 0.5 else 64 * _log(rng, 1, 128)
        case = dict(op=op, dtype=dtype, C=C, beta=rng.random() < 0.5)
        if op == "scan_step":
            return dict(case, B=_log(rng, 1, 512))
        case["h0"] = rng.random() < 0.5
        if "varlen" in op:
            T = _log(rng, 1, min(32768, most // C))
            case.update(N=_log(rng, 1, min(64, T)), T=T)
        else:
            T = _log(rng, 1, min(32768, most // C))
            case.update(B=_log(rng, 1, max(1, min(16, most // (C * T)))), T=T)
        if op != "scan_varlen":
            case["carries"] = rng.random() < 0.5
        return case
    most = 1 << 25
    act = rng.choice(["silu", "sigmoid"])
    if op.startswith("gated_norm"):
        D = rng.choice([64, 128, 256]) if rng.random() < 0.6 else _log(rng, 8, 4096)
        return dict(op=op, rows=_log(rng, 1, most // D), D=D, x_dtype=rng.choice(["bf16", "f32"]), dtype=dtype,
                    z=rng.random() < 0.8, act=act)
    D = 64 * _log(rng, 4, 128) if rng.random() < 0.6 else _log(rng, 8, 8192)
    return dict(op=op, rows=_log(rng, 1, most // D), D=D, dtype=dtype, r_dtype="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                z=rng.random() < 0.4, post=rng.random() < 0.7, scale=rng.random() < 0.7, act=act)


# ---------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Sequence lengths: equal ones of a batch, or a ragged split of the packed tokens (empty sequences happen)."""
    if "varlen" not in case["op"]:
        return [case["T"]] * case["B"]
    rng = random.Random(seed * 7919 + case["N"])
    cuts = sorted(rng.randint(0, case["T"]) for _ in range(case["N"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32)  # noqa: E731
    s = {"case": dict(case)}
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op.startswith("scan"):
        C = case["C"]
        if op == "scan_step":
            shape, n = (case["B"], C), case["B"]
        elif "varlen" in op:
            shape, n = (case["T"], C), case["N"]
        else:
            shape, n = (case["B"], case["T"], C), case["B"]
        # channels of short and of long memory: the decay's logit has a mean of 0 to 6 by channel
        mean = torch.rand(C, generator=gen, device="cuda") * 6
        s["g"] = torch.nn.functional.logsigmoid(randn(*shape) + mean)
        s["x"] = randn(*shape).to(dt)
        s["beta"] = torch.sigmoid(randn(*shape)).to(dt) if case["beta"] else None
        if op == "scan_step":
            s["state"] = randn(n, C)
            return s
        s["h0"] = randn(n, C) if case["h0"] else None
        lens = _lengths(case, seed)
        starts = [sum(lens[:i]) for i in range(n)]
        s["lens"], s["starts"] = lens, starts
        if "varlen" in op:
            s["cu"] = torch.tensor(starts + [case["T"]], dtype=torch.int32, device="cuda")
        full = [i for i in range(n) if lens[i]]
        index = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731
        s["full"] = index(full)
        s["first"] = index([starts[i] for i in full])
        s["last"] = index([starts[i] + lens[i] - 1 for i in full])
        rows, token = _carry_rows(case, starts, lens)
        s["carry_row"], s["carry_token"] = index(rows), index(token)
        if "backward" in op:
            s["dh"] = randn(*shape).to(dt)
            s["dh_T"] = randn(n, C)
            s["carries"] = None
            if case["carries"]:  # what the forward pass of this step kept
                h, _ = _states(s)
                s["carries"] = _carries(s, h)
        return s
    rows, D = case["rows"], case["D"]
    s["x"] = randn(rows, D)
    s["x"] = (s["x"] * torch.exp(0.5 * randn(rows, 1))).to(DTYPES[case.get("x_dtype", case["dtype"])])
    s["z"] = randn(rows, D).to(dt) if case["z"] else None
    s["w"] = 1 + 0.2 * randn(D)
    if op.startswith("residual"):
        s["r"] = (2 * randn(rows, D)).to(DTYPES[case["r_dtype"]])  # forward: the stream; backward: the kept sum
        s["w_post"] = 1 + 0.2 * randn(D) if case["post"] else None
        s["scale"] = 0.5 + 0.1 * randn(D) if case["scale"] else None
        if "backward" in op:
            s["dr"] = randn(rows, D).to(DTYPES[case["r_dtype"]])
    if "backward" in op:
        s["dy"] = randn(rows, D).to(dt)
    return s


def _carry_rows(case, starts, lens):
    """Row of the kept states and the token it precedes, for every 16th token of every sequence: a batch has
    ceil(T / 16) rows a sequence; packed sequence n begins at row start // 16 + n."""
    rows, token = [], []
    for n, (a, m) in enumerate(zip(starts, lens)):
        base = a // CARRY_TOKENS + n if "varlen" in case["op"] else n * -(-m // CARRY_TOKENS)
        for j in range(-(-m // CARRY_TOKENS)):
            rows.append(base + j)
            token.append(a + j * CARRY_TOKENS)
    return rows, token


# ---------------------------------------------------------------- plain forms
def _f(t):
    return None if t is None else t.float()


def _states(s):
    """h [tokens, C] and the decays, in 32 bits: a doubling scan whose decay is cut at each sequence's first token."""
    C = s["g"].shape[-1]
    a = torch.exp(s["g"].reshape(-1, C))
    h = _f(s["x"]).reshape(-1, C)
    h = h * _f(s["beta"]).reshape(-1, C) if s["beta"] is not None else h.clone()
    if s["h0"] is not None:
        h[s["first"]] += a[s["first"]] * s["h0"][s["full"]]
    cut = a.clone()
    cut[s["first"]] = 0
    return _double(cut, h, max(s["lens"], default=0)), a


def _double(a, h, longest):
    d = 1
    while d < longest:
        h[d:] = h[d:] + a[d:] * h[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return h


def _before(s, h):
    """h of the token before, each sequence's first token seeing its h0."""
    p = torch.zeros_like(h)
    p[1:] = h[:-1]
    p[s["first"]] = s["h0"][s["full"]] if s["h0"] is not None else 0.0
    return p


def _carries(s, h):
    case, C = s["case"], h.shape[1]
    if "varlen" in case["op"]:
        out = torch.zeros((case["T"] // CARRY_TOKENS + case["N"], C), device=h.device)
        out[s["carry_row"]] = _before(s, h)[s["carry_token"]]
        return out
    return _before(s, h)[s["carry_token"]].reshape(case["B"], -1, C)


def _plain_scan(s):
    x = s["x"]
    h, _ = _states(s)
    h_T = s["h0"].clone() if s["h0"] is not None else torch.zeros((len(s["lens"]), h.shape[1]), device=h.device)
    h_T[s["full"]] = h[s["last"]]
    out = [h.to(x.dtype).reshape(x.shape), h_T]
    if s["case"].get("carries"):
        out.append(_carries(s, h))
    return out


def _plain_scan_backward(s):
    x, C = s["x"], s["g"].shape[-1]
    h, a = _states(s)
    h = _before(s, h)
    lam = _f(s["dh"]).reshape(-1, C).clone()
    lam[s["last"]] += s["dh_T"][s["full"]]
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[s["last"]] = 0
    lam = _double(nxt.flip(0), lam.flip(0), max(s["lens"], default=0)).flip(0)
    dg = lam * a * h
    xf = _f(x).reshape(-1, C)
    dx, dbeta = lam, None
    if s["beta"] is not None:
        dx, dbeta = lam * _f(s["beta"]).reshape(-1, C), (lam * xf).to(x.dtype).reshape(x.shape)
    dh0 = None
    if s["h0"] is not None:
        dh0 = s["dh_T"].clone()
        dh0[s["full"]] = (a * lam)[s["first"]]
    return [dx.to(x.dtype).reshape(x.shape), dg.reshape(x.shape), dbeta, dh0]


def _plain_step(s):
    u = _f(s["x"]) * _f(s["beta"]) if s["beta"] is not None else _f(s["x"])
    h = torch.exp(s["g"]) * s["state"] + u
    s["state"].copy_(h)
    return [h.to(s["x"].dtype), s["state"]]


def _act(name, z):
    """The gate's value and slope."""
    if z is None:
        return 1.0, None
    p = 1 / (1 + torch.exp(-z))
    return (z * p, p * (1 + z * (1 - p))) if name == "silu" else (p, p * (1 - p))


def _rstd(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_gated_norm(s):
    x, a = _f(s["x"]), _act(s["case"]["act"], _f(s["z"]))[0]
    return [(x * _rstd(x) * s["w"] * a).to(DTYPES[s["case"]["dtype"]])]


def _norm_grad(x, w, u):
    """Gradient of w xh with respect to x (xh = x / rms) and to w, u the gradient of the result."""
    r = _rstd(x)
    xh, uw = x * r, u * w
    return r * (uw - xh * (uw * xh).mean(-1, keepdim=True)), (u * xh).sum(0)


def _plain_gated_norm_backward(s):
    x, z, dy, w = _f(s["x"]), _f(s["z"]), _f(s["dy"]), s["w"]
    a, da = _act(s["case"]["act"], z)
    dx, dw = _norm_grad(x, w, dy * a)
    dz = (dy * w * x * _rstd(x) * da).to(s["dy"].dtype) if z is not None else None
    return [dx.to(s["x"].dtype), dz, dw]


def _plain_residual_norm(s):
    x, r = _f(s["x"]), _f(s["r"])
    a = _act(s["case"]["act"], _f(s["z"]))[0]
    u = x * _rstd(x) * s["w_post"] if s["w_post"] is not None else x
    u = u * a
    r = r + (u * s["scale"] if s["scale"] is not None else u)
    return [(r * _rstd(r) * s["w"]).to(s["x"].dtype), r.to(s["r"].dtype)]


def _plain_residual_norm_backward(s):
    x, r, z, dy = _f(s["x"]), _f(s["r"]), _f(s["z"]), _f(s["dy"])
    a, da = _act(s["case"]["act"], z)
    dr, dw = _norm_grad(r, s["w"], dy)
    dr = dr + _f(s["dr"])
    u = x * _rstd(x) * s["w_post"] if s["w_post"] is not None else x
    dscale = (dr * a * u).sum(0) if s["scale"] is not None else None
    d = dr * s["scale"] if s["scale"] is not None else dr
    dz = (d * u * da).to(s["dy"].dtype) if z is not None else None
    dx, dw_post = (d * a), None
    if s["w_post"] is not None:
        dx, dw_post = _norm_grad(x, s["w_post"], d * a)
    return [dx.to(s["x"].dtype), dr.to(s["r"].dtype), dz, dw, dw_post, dscale]


_PLAIN = {"scan": _plain_scan, "scan_varlen": _plain_scan, "scan_step": _plain_step,
          "scan_backward": _plain_scan_backward, "scan_varlen_backward": _plain_scan_backward,
          "gated_norm": _plain_gated_norm, "gated_norm_backward": _plain_gated_norm_backward,
          "residual_norm": _plain_residual_norm, "residual_norm_backward": _plain_residual_norm_backward}


# ---------------------------------------------------------------- one pass
def _own_run(s):
    import gated_deltanet_linear_20_b200 as gdn
    case, op = s["case"], s["case"]["op"]
    if op == "scan":
        return list(gdn.scan(s["x"], s["g"], s["beta"], s["h0"], save_carries=case["carries"]))
    if op == "scan_varlen":
        return list(gdn.scan_varlen(s["x"], s["g"], s["cu"], s["beta"], s["h0"]))
    if op == "scan_step":
        return [gdn.scan_step(s["x"], s["g"], s["state"], s["beta"]), s["state"]]
    if op == "scan_backward":
        return list(gdn.scan_backward(s["dh"], s["x"], s["g"], s["beta"], s["h0"], s["dh_T"], carries=s["carries"]))
    if op == "scan_varlen_backward":
        return list(gdn.scan_varlen_backward(s["dh"], s["x"], s["g"], s["cu"], s["beta"], s["h0"], s["dh_T"],
                                             carries=s["carries"]))
    if op == "gated_norm":
        return [gdn.gated_norm(s["x"], s["w"], s["z"], gate=case["act"], eps=EPS, out_dtype=DTYPES[case["dtype"]])]
    if op == "gated_norm_backward":
        return list(gdn.gated_norm_backward(s["dy"], s["x"], s["w"], s["z"], gate=case["act"], eps=EPS))
    if op == "residual_norm":
        return list(gdn.residual_norm(s["x"], s["r"], s["w"], z=s["z"], w_post=s["w_post"], scale=s["scale"],
                                      gate=case["act"], eps=EPS))
    return list(gdn.residual_norm_backward(s["dy"], s["dr"], s["x"], s["r"], s["w"], z=s["z"], w_post=s["w_post"],
                                           scale=s["scale"], gate=case["act"], eps=EPS))


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["case"]["op"]](state)


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op.startswith("scan"):
        C, b = case["C"], int(case["beta"])
        if op == "scan_step":
            n = case["B"] * C
            return {"bytes": n * ((2 + b) * e + 12), "flops": n * 6}
        seqs = case["N"] if "varlen" in op else case["B"]
        tokens = case["T"] * (1 if "varlen" in op else case["B"])
        cu = 4 * (seqs + 1) if "varlen" in op else 0
        h0 = 4 * C * seqs * int(case["h0"])
        kept = tokens // CARRY_TOKENS * C * 4 if case.get("carries") else 0
        if "backward" in op:
            return {"bytes": tokens * C * (8 + (3 + 2 * b) * e) + 2 * h0 + 4 * C * seqs + kept + cu, "flops": tokens * C * 14}
        return {"bytes": tokens * C * (4 + (2 + b) * e) + h0 + 4 * C * seqs + kept + cu, "flops": tokens * C * 6}
    rows, D, z = case["rows"], case["D"], int(case["z"])
    n = rows * D
    if op == "gated_norm":
        return {"bytes": n * (SIZE[case["x_dtype"]] + (1 + z) * e) + 4 * D, "flops": n * 10}
    if op == "gated_norm_backward":
        return {"bytes": n * (2 * SIZE[case["x_dtype"]] + (1 + 2 * z) * e) + 8 * D, "flops": n * 24}
    er, small = SIZE[case["r_dtype"]], 4 * D * (1 + int(case["post"]) + int(case["scale"]))
    if op == "residual_norm":
        return {"bytes": n * (2 * er + (2 + z) * e) + small, "flops": n * 14}
    return {"bytes": n * (3 * er + (3 + 2 * z) * e) + 2 * small, "flops": n * 34}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan_step":
        h = s["state"].double() * s["g"].double().exp()
        h += s["x"].double() * (s["beta"].double() if s["beta"] is not None else 1)
        return [h, h]
    if op.startswith("scan"):
        return _exact_recurrence(case, s)
    return _exact_norm(case, s)


def _exact_recurrence(case, s):
    C, n = case["C"], len(s["lens"])
    flat = lambda t: None if t is None else t.reshape(-1, C)  # noqa: E731
    x, g, beta = flat(s["x"]), flat(s["g"]), flat(s["beta"])
    backward = "backward" in case["op"]
    order = sorted(range(n), key=lambda i: -s["lens"][i])  # longest first: the running ones are a prefix
    lens = [s["lens"][i] for i in order]
    at = torch.tensor([s["starts"][i] for i in order], dtype=torch.int64, device="cuda")
    ends = torch.tensor([s["starts"][i] + s["lens"][i] - 1 for i in order], dtype=torch.int64, device="cuda")
    state = torch.zeros((n, C), dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        state += s["h0"].double()[order]
    h = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    before = torch.empty_like(h) if backward or case.get("carries") else None
    k = n
    for t in range(lens[0] if n else 0):
        while k and lens[k - 1] <= t:
            k -= 1
        row = at[:k] + t
        if before is not None:
            before[row] = state[:k]
        u = x[row].double()
        if beta is not None:
            u = u * beta[row].double()
        state[:k] = torch.exp(g[row].double()) * state[:k] + u
        h[row] = state[:k]
    back = torch.empty_like(state)
    back[order] = state
    if not backward:
        out = [h.reshape(s["x"].shape), back]
        if case["op"] == "scan" and case["carries"]:
            out.append(before[s["carry_token"]].reshape(case["B"], -1, C))
        return out
    lam = torch.empty_like(h)
    mu = s["dh_T"].double()[order]
    k = n
    for t in range(lens[0] if n else 0):  # from each sequence's end
        while k and lens[k - 1] <= t:
            k -= 1
        row = ends[:k] - t
        v = flat(s["dh"])[row].double() + mu[:k]
        lam[row] = v
        mu[:k] = torch.exp(g[row].double()) * v
    dg = lam * torch.exp(g.double()) * before
    shape = s["x"].shape
    dx = lam if beta is None else lam * beta.double()
    dbeta = None if beta is None else (lam * x.double()).reshape(shape)
    dh0 = torch.empty_like(state)
    dh0[order] = mu
    return [dx.reshape(shape), dg.reshape(shape), dbeta, dh0 if s["h0"] is not None else None]


def _exact_norm(case, s):
    backward = "backward" in case["op"]
    v = {k: t.double().requires_grad_(backward and k not in ("dy", "dr"))
         for k, t in s.items() if isinstance(t, torch.Tensor)}
    get = v.get
    norm = lambda t, w: t / torch.sqrt(t.pow(2).mean(-1, keepdim=True) + EPS) * w  # noqa: E731
    gate = None
    if get("z") is not None:
        gate = torch.sigmoid(v["z"]) * (v["z"] if case["act"] == "silu" else 1)
    if case["op"].startswith("gated_norm"):
        y = norm(v["x"], v["w"])
        y = y if gate is None else y * gate
        if not backward:
            return [y]
        y.backward(v["dy"])
        return [v["x"].grad, get("z").grad if get("z") is not None else None, v["w"].grad]
    u = norm(v["x"], v["w_post"]) if get("w_post") is not None else v["x"]
    u = u if gate is None else u * gate
    u = u if get("scale") is None else u * v["scale"]
    if not backward:
        r = v["r"] + u
        return [norm(r, v["w"]), r]
    # the kept sum is the point at which the next norm is differentiated
    norm(v["r"], v["w"]).backward(v["dy"])
    dr = v["r"].grad + v["dr"]
    u.backward(dr)
    grad = lambda k: v[k].grad if get(k) is not None else None  # noqa: E731
    return [grad("x"), dr, grad("z"), grad("w"), grad("w_post"), grad("scale")]
