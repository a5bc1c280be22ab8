"""The operators of a whole MoE sublayer as cases that can be timed and compared.

Five operators beside the router and the recalibrated backward: the forward of the
routed experts (gated feed-forward block), its backward up to the first projection's
output, the layer norm in both directions, and dropout with a residual.  ``run``
computes them in plain torch operations, or with ``own`` through the library.
"""

import math

import torch

own = False

F32, BF16 = "f32", "bf16"
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
SIZE = {F32: 4, BF16: 2}
EPS = 1e-5

_context = None  # the library context a program keeps


def _lib():
    from backward_token_expert_gb300 import lrm

    global _context
    if _context is None:
        _context = lrm.lrm_create(0)
    return lrm, _context


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # experts, forward: one token of the benchmark's layer, as an answer is generated; an odd-sized layer with
        # padding tokens; the benchmark's layer in training, which saves what its backward reads
        dict(name="ffn token", op="ffn", T=1, E=128, k=8, h=2048, I=768, masked=False, save=False),
        dict(name="ffn ragged", op="ffn", T=5003, E=20, k=3, h=1496, I=1000, masked=True, save=True),
        dict(name="ffn layer", op="ffn", T=32768, E=128, k=8, h=2048, I=768, masked=False, save=True),
        # experts, backward of the retained pairs: the tiny layer, an odd-sized one, the benchmark's layer
        dict(name="ffn_bwd tiny", op="ffn_bwd", N=512, E=8, h=64, I=32, rows=333, spare=40),
        dict(name="ffn_bwd ragged", op="ffn_bwd", N=30011, E=20, h=1000, I=1496, rows=15013, spare=1000),
        dict(name="ffn_bwd layer", op="ffn_bwd", N=262144, E=128, h=2048, I=768, rows=87204, spare=8192),
        # layer norm: a few sequences' single tokens, an odd width, the benchmark's tokens; padding rows in one
        dict(name="norm tokens bf16", op="norm", rows=8, width=2048, dtype=BF16, masked=False),
        dict(name="norm layer bf16", op="norm", rows=32768, width=2048, dtype=BF16, masked=False),
        dict(name="norm_bwd ragged bf16", op="norm_bwd", rows=20011, width=1497, dtype=BF16, masked=True, residual=False),
        dict(name="norm_bwd layer f32", op="norm_bwd", rows=32768, width=2048, dtype=F32, masked=False, residual=True),
        # dropout: an odd number of elements behind a residual, and the gradient of the benchmark's tokens (no residual)
        dict(name="dropout ragged f32", op="dropout", n=1000003, p=0.2, dtype=F32, residual=True),
        dict(name="dropout layer bf16", op="dropout", n=67108864, p=0.1, dtype=BF16, residual=False),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn_bwd", "norm", "norm_bwd", "dropout"])
    dtype = rng.choice([F32, BF16])
    if op in ("ffn", "ffn_bwd"):
        h, I = 8 * _log(rng, 8, 640), 8 * _log(rng, 4, 192)
        E = min(_log(rng, 2, 160), max(2, 128 * 2048 * 768 // (h * I)))
        most = 262144 * 2048 * 768 // (h * I)
        if op == "ffn":
            k = rng.randint(1, min(E, 8))
            return dict(op=op, T=min(_log(rng, 1, 32768), most // k), E=E, k=k, h=h, I=I, masked=rng.random() < 0.4,
                        save=rng.random() < 0.6)
        rows = min(_log(rng, 100, 100000), most // 3)
        return dict(op=op, N=rows + rng.randint(0, 2 * rows), E=E, h=h, I=I, rows=rows, spare=rng.randint(0, rows // 4))
    if op == "dropout":
        return dict(op=op, n=_log(rng, 500, 60000000), p=round(rng.uniform(0.0, 0.6), 2), dtype=dtype,
                    residual=rng.random() < 0.6)
    width = _log(rng, 16, 8192)
    if rng.random() < 0.6:
        width = 8 * max(2, width // 8)
    case = dict(op=op, rows=min(_log(rng, 1, 40000), 32768 * 2048 // width), width=width, dtype=dtype,
                masked=rng.random() < 0.4)
    return dict(case, residual=rng.random() < 0.5) if op == "norm_bwd" else case


# ---------------------------------------------------------------------------
# inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _segments(pairs, experts, E, room):
    """The pairs grouped by expert, ascending within one: ids [room], offsets [E+1]."""
    ids = torch.zeros(max(1, room), dtype=torch.int32, device="cuda")
    ids[:pairs.numel()] = pairs[experts.sort(stable=True).indices].to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(experts, minlength=E).cumsum(0)
    return ids, offsets


def _prepare_ffn(case, g):
    # a skewed router's choice (random logits plus an expert's own bias) and its gates; tokens of padding have no pair
    # in the segments and gate 0
    T, E, k, h, I = (case[n] for n in ("T", "E", "k", "h", "I"))
    rank = torch.randperm(E, generator=g, device="cuda").float()
    logits = torch.randn(T, E, generator=g, device="cuda") - 0.8 * torch.log(rank + 1.0)
    top = logits.topk(k, dim=1)
    alpha = torch.softmax(top.values, 1)
    pairs, experts = torch.arange(T * k, device="cuda"), top.indices.reshape(-1)
    if case["masked"]:
        counted = torch.rand(T, generator=g, device="cuda") < 0.9
        alpha *= counted[:, None]
        kept = counted.repeat_interleave(k)
        pairs, experts = pairs[kept], experts[kept]
    ids, offsets = _segments(pairs, experts, E, T * k)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    state = dict(x=_normal(g, T, h), W1=_normal(g, E, 2 * I, h, scale=h ** -0.5), W=_normal(g, E, h, I, scale=I ** -0.5),
                 alpha=alpha.reshape(-1), ids=ids, offsets=offsets, bounds=offsets.tolist(),
                 phi=torch.zeros(T * k, I, **bf), rows=torch.zeros(T * k, h, **bf), y=torch.zeros(T, h, **bf))
    state["ab"] = torch.zeros(T * k, 2 * I, **bf) if case["save"] else None
    return state


def _prepare_ffn_bwd(case, g):
    # the retained pairs' weighted output gradients, as small as a mean loss gives, and the saved projections of all pairs
    N, E, h, I, rows = (case[n] for n in ("N", "E", "h", "I", "rows"))
    room = rows + case["spare"]
    u = torch.randperm(N, generator=g, device="cuda")[:rows].sort().values
    e = torch.randint(0, E, (rows,), generator=g, device="cuda")
    ids, offsets = _segments(u, e, E, room)
    delta = _normal(g, room, h, scale=1e-3, dtype=torch.float32)
    delta = delta.mul_(torch.rand(room, 1, generator=g, device="cuda")).to(torch.bfloat16)
    state = dict(delta=delta, W=_normal(g, E, h, I, scale=I ** -0.5), ab=_normal(g, N, 2 * I), ids=ids, offsets=offsets,
                 bounds=offsets.tolist(), dh1=torch.zeros(room, 2 * I, dtype=torch.bfloat16, device="cuda"),
                 dgate=torch.zeros(N, device="cuda"))
    return state


def _prepare_norm(case, g):
    # a residual stream: rows of their own scale and mean, a few channels far larger than the rest
    rows, width, dt = case["rows"], case["width"], TORCH[case["dtype"]]
    x = torch.randn(rows, width, generator=g, device="cuda")
    x.mul_(0.5 + 2.0 * torch.rand(rows, 1, generator=g, device="cuda"))
    x[:, ::97] *= 12.0
    x.add_(0.3 * torch.randn(rows, 1, generator=g, device="cuda"))
    state = dict(x=x.to(dt), gamma=1.0 + 0.2 * torch.randn(width, generator=g, device="cuda"),
                 beta=0.1 * torch.randn(width, generator=g, device="cuda"),
                 y=torch.zeros(rows, width, dtype=dt, device="cuda"), stats=torch.zeros(rows, 2, device="cuda"))
    valid = (torch.rand(rows, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["masked"] else None
    return dict(state, valid=valid)


def _prepare_norm_bwd(case, g):
    state = _prepare_norm(case, g)
    rows, width, dt = case["rows"], case["width"], TORCH[case["dtype"]]
    stats = _plain_norm(dict(state, case=case))["stats"]
    dy = _normal(g, rows, width, scale=0.01, dtype=dt)
    dres = _normal(g, rows, width, scale=0.01, dtype=dt) if case["residual"] else None
    return dict(x=state["x"], dy=dy, gamma=state["gamma"], stats=stats, valid=state["valid"], dres=dres,
                dx=torch.zeros(rows, width, dtype=dt, device="cuda"), dgamma=torch.zeros(width, device="cuda"),
                dbeta=torch.zeros(width, device="cuda"))


def _prepare_dropout(case, g):
    n, dt = case["n"], TORCH[case["dtype"]]
    seed = int(torch.randint(0, 2 ** 62, (1,), generator=g, device="cuda"))
    offset = int(torch.randint(0, 2 ** 40, (1,), generator=g, device="cuda"))
    step = torch.randint(0, 100000, (1,), generator=g, device="cuda")  # the training step, which a program counts up
    return dict(x=_normal(g, n, dtype=dt), residual=_normal(g, n, dtype=dt) if case["residual"] else None,
                out=torch.zeros(n, dtype=dt, device="cuda"), seed=seed, offset=offset, step=step)


def _plan(case, state):
    """What a program that uses the library keeps beside its tensors."""
    if not own:
        return None
    lrm, ctx = _lib()
    op = case["op"]
    if op == "ffn":
        return lrm.dims_of(case["T"], case["E"], case["k"], case["h"], case["I"])
    if op == "ffn_bwd":
        dims = lrm.dims_of(case["N"], case["E"], 1, case["h"], case["I"])
        need = lrm.lrm_ffn_backward_workspace(ctx, dims, state["delta"].shape[0])
        return dims, torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    if op == "norm_bwd":
        need = lrm.lrm_layer_norm_workspace(ctx, case["rows"], case["width"])
        return torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return None


def prepare(case, seed):
    g = _generator(seed)
    make = dict(ffn=_prepare_ffn, ffn_bwd=_prepare_ffn_bwd, norm=_prepare_norm, norm_bwd=_prepare_norm_bwd,
                dropout=_prepare_dropout)[case["op"]]
    state = make(case, g)
    state["case"] = case
    state["plan"] = _plan(case, state)
    return state


# ---------------------------------------------------------------------------
# the plain forms


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _plain_ffn(state):
    case, I = state["case"], state["case"]["I"]
    x = state["x"].float()
    y = torch.zeros(case["T"], case["h"], device="cuda")
    at = state["bounds"]
    for e in range(case["E"]):
        if at[e + 1] > at[e]:
            u = state["ids"][at[e]:at[e + 1]].long()
            t = u // case["k"]
            h1 = x[t] @ state["W1"][e].float().T
            phi = _silu(h1[:, :I]) * h1[:, I:]
            r = phi @ state["W"][e].float().T
            y[t] += state["alpha"][u][:, None] * r  # a token has an expert once
            if case["save"]:
                state["ab"][u] = h1.to(torch.bfloat16)
                state["phi"][u] = phi.to(torch.bfloat16)
    out = dict(y=y.to(torch.bfloat16))
    return dict(out, ab=state["ab"], phi=state["phi"]) if case["save"] else out


def _plain_ffn_bwd(state):
    case, I, at = state["case"], state["case"]["I"], state["bounds"]
    dgate = torch.zeros(case["N"], device="cuda")
    for e in range(case["E"]):
        a, b = at[e], at[e + 1]
        if b > a:
            u = state["ids"][a:b].long()
            d = state["delta"][a:b].float() @ state["W"][e].float()
            gate, up = state["ab"][u].float().split(I, 1)
            s = 1.0 / (1.0 + torch.exp(-gate))
            state["dh1"][a:b, :I] = (d * up * s * (1.0 + gate * (1.0 - s))).to(torch.bfloat16)
            state["dh1"][a:b, I:] = (d * gate * s).to(torch.bfloat16)
            dgate[u] = (d * gate * s * up).sum(1)
    return dict(dh1=state["dh1"], dgate=dgate)


def _plain_norm(state):
    x = state["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    counted = torch.ones_like(mean) if state["valid"] is None else state["valid"].float()[:, None]
    y = (c * rstd * state["gamma"] + state["beta"]) * counted
    return dict(y=y.to(state["x"].dtype), stats=torch.cat([mean, rstd], 1) * counted)


def _plain_norm_bwd(state):
    mean, rstd = state["stats"][:, :1], state["stats"][:, 1:]
    counted = torch.ones_like(mean) if state["valid"] is None else state["valid"].float()[:, None]
    xhat = (state["x"].float() - mean) * rstd
    dy = state["dy"].float() * counted
    d = dy * state["gamma"]
    dx = rstd * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))
    if state["dres"] is not None:
        dx = dx + state["dres"].float() * counted
    # long sums over the rows
    return dict(dx=dx.to(state["x"].dtype), dgamma=(dy * xhat).sum(0, dtype=torch.float64).float(),
                dbeta=dy.sum(0, dtype=torch.float64).float())


_M = 0xFFFFFFFF


def _philox(seed, offset, n):
    """The first n 32-bit words of Philox4x32-10 with the given key and the upper half of its counter (a tensor of
    one element): word i is word i % 4 of counter (i // 4, offset)."""
    q = torch.arange((n + 3) // 4, device="cuda")
    c = [q & _M, q >> 32, (offset & _M).expand_as(q), ((offset >> 32) & _M).expand_as(q)]
    k0, k1 = seed & _M, (seed >> 32) & _M
    for _ in range(10):
        # a product of two 32-bit words, modulo 2^64 in int64: both halves are exact
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & _M) ^ c[1] ^ k0, p1 & _M, ((p0 >> 32) & _M) ^ c[3] ^ k1, p0 & _M]
        k0, k1 = (k0 + 0x9E3779B9) & _M, (k1 + 0xBB67AE85) & _M
    return torch.stack(c, 1).reshape(-1)[:n]


def _plain_dropout(state):
    p = state["case"]["p"]
    r = _philox(state["seed"], state["offset"] + state["step"], state["case"]["n"])
    out = torch.where(r < int(p * 2 ** 32), 0.0, state["x"].float() * (1.0 / (1.0 - p)))
    if state["residual"] is not None:
        out = out + state["residual"].float()
    return dict(out=out.to(state["x"].dtype))


# ---------------------------------------------------------------------------
# the library's calls


def _own_ffn(state):
    lrm, ctx = _lib()
    dims, n = state["plan"], state["ids"].shape[0]
    lrm.lrm_ffn_up(ctx, state["x"], state["W1"], state["offsets"], state["ids"], dims, n, state["ab"], state["phi"])
    lrm.lrm_ffn_down(ctx, state["phi"], state["W"], state["offsets"], state["ids"], dims, n, state["rows"])
    lrm.lrm_ffn_combine(ctx, state["rows"], state["alpha"], dims, state["y"])
    out = dict(y=state["y"])
    return dict(out, ab=state["ab"], phi=state["phi"]) if state["case"]["save"] else out


def _own_ffn_bwd(state):
    lrm, ctx = _lib()
    dims, ws = state["plan"]
    lrm.lrm_ffn_backward(ctx, state["delta"], state["W"], state["ab"], state["offsets"], state["ids"], dims,
                         state["delta"].shape[0], state["dh1"], state["dgate"], ws, ws.numel())
    return dict(dh1=state["dh1"], dgate=state["dgate"])


def _dtype(lrm, case):
    return lrm.DTYPE_F32 if case["dtype"] == F32 else lrm.DTYPE_BF16


def _own_norm(state):
    lrm, ctx = _lib()
    case = state["case"]
    lrm.lrm_layer_norm(ctx, state["x"], _dtype(lrm, case), state["gamma"], state["beta"], state["valid"], case["rows"],
                       case["width"], EPS, state["y"], state["stats"])
    return dict(y=state["y"], stats=state["stats"])


def _own_norm_bwd(state):
    lrm, ctx = _lib()
    case, ws = state["case"], state["plan"]
    lrm.lrm_layer_norm_backward(ctx, state["x"], _dtype(lrm, case), state["dy"], state["gamma"], state["stats"],
                                state["valid"], state["dres"], case["rows"], case["width"], state["dx"],
                                state["dgamma"], state["dbeta"], ws, ws.numel())
    return dict(dx=state["dx"], dgamma=state["dgamma"], dbeta=state["dbeta"])


def _own_dropout(state):
    lrm, ctx = _lib()
    case = state["case"]
    lrm.lrm_dropout_add(ctx, state["x"], state["residual"], _dtype(lrm, case), case["n"], case["p"], state["seed"],
                        state["offset"], state["step"], state["out"])
    return dict(out=state["out"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(ffn=_own_ffn, ffn_bwd=_own_ffn_bwd, norm=_own_norm, norm_bwd=_own_norm_bwd,
                    dropout=_own_dropout)[op](state)
    return dict(ffn=_plain_ffn, ffn_bwd=_plain_ffn_bwd, norm=_plain_norm, norm_bwd=_plain_norm_bwd,
                dropout=_plain_dropout)[op](state)


# ---------------------------------------------------------------------------
# work and the 64-bit values


def work(case):
    op = case["op"]
    if op == "ffn":
        T, E, k, h, I = (case[n] for n in ("T", "E", "k", "h", "I"))
        N = T * k * (0.9 if case["masked"] else 1.0)
        saved = 6 * N * I if case["save"] else 0
        return dict(bytes=int(6 * min(E, T * k) * h * I + 4 * T * h + 8 * T * k + saved), flops=int(6 * N * h * I))
    if op == "ffn_bwd":
        N, E, h, I, rows = (case[n] for n in ("N", "E", "h", "I", "rows"))
        return dict(bytes=2 * rows * h + 8 * rows * I + 2 * min(E, rows) * h * I + 4 * rows + 4 * N,
                    flops=2 * rows * h * I + 12 * rows * I)
    size = SIZE[case["dtype"]]
    if op == "dropout":
        return dict(bytes=(3 if case["residual"] else 2) * case["n"] * size, flops=30 * case["n"])
    n = case["rows"] * case["width"]
    if op == "norm":
        return dict(bytes=2 * n * size + 8 * case["width"] + 8 * case["rows"], flops=8 * n)
    return dict(bytes=(4 if case["residual"] else 3) * n * size + 12 * case["width"] + 8 * case["rows"], flops=14 * n)


def _exact_ffn(st, case):
    # pair by pair: the rows of every pair, zeros for a pair in no segment, then the gated sum over the slots
    T, k, h, I, at = case["T"], case["k"], case["h"], case["I"], st["bounds"]
    h1 = torch.zeros(T * k, 2 * I, dtype=torch.float64, device="cuda")
    r = torch.zeros(T * k, h, dtype=torch.float64, device="cuda")
    phi = torch.zeros(T * k, I, dtype=torch.float64, device="cuda")
    for e in [e for e in range(case["E"]) if at[e + 1] > at[e]]:
        u = st["ids"][at[e]:at[e + 1]].long()
        z = torch.einsum("rh,ch->rc", st["x"].index_select(0, u.div(k, rounding_mode="floor")).double(),
                         st["W1"][e].double())
        h1[u] = z
        phi[u] = 0.5 * z[:, :I] * (1.0 + torch.tanh(0.5 * z[:, :I])) * z[:, I:]
        r[u] = torch.einsum("ri,hi->rh", phi[u], st["W"][e].double())
    y = torch.einsum("tk,tkh->th", st["alpha"].double().reshape(T, k), r.reshape(T, k, h))
    return dict(y=y, ab=h1, phi=phi) if case["save"] else dict(y=y)


def _exact_ffn_bwd(st, case):
    # the activation's derivative from its logistic form: silu'(a) = s + a s (1 - s)
    I, at = case["I"], st["bounds"]
    dh1 = torch.zeros(st["dh1"].shape, dtype=torch.float64, device="cuda")
    dgate = torch.zeros(case["N"], dtype=torch.float64, device="cuda")
    for e in [e for e in range(case["E"]) if at[e + 1] > at[e]]:
        seg = slice(at[e], at[e + 1])
        u = st["ids"][seg].long()
        d = torch.einsum("rh,hi->ri", st["delta"][seg].double(), st["W"][e].double())
        a, b = st["ab"][u, :I].double(), st["ab"][u, I:].double()
        s = torch.sigmoid(a)
        dh1[seg] = torch.cat([d * b * (s + a * s * (1.0 - s)), d * (a * s)], 1)
        dgate[u] = torch.einsum("ri,ri->r", d, a * s * b)
    return dict(dh1=dh1, dgate=dgate)


def _exact_norm(st, case):
    x = st["x"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = (var + EPS).rsqrt()
    y = (x - mean[:, None]) * rstd[:, None] * st["gamma"].double() + st["beta"].double()
    stats = torch.stack([mean, rstd], 1)
    if st["valid"] is not None:
        y[st["valid"] == 0] = 0.0
        stats[st["valid"] == 0] = 0.0
    return dict(y=y, stats=stats)


def _exact_norm_bwd(st, case):
    # through the centred rows: d/dx of (x - mean) rstd, with the saved statistics
    rows = torch.arange(case["rows"], device="cuda") if st["valid"] is None else st["valid"].nonzero()[:, 0]
    mean, rstd = st["stats"][rows].double().unbind(1)
    xhat = torch.einsum("rw,r->rw", st["x"][rows].double() - mean[:, None], rstd)
    dy = st["dy"][rows].double()
    d = dy * st["gamma"].double()
    along = torch.einsum("rw,rw->r", d, xhat) / case["width"]
    dx = torch.zeros(case["rows"], case["width"], dtype=torch.float64, device="cuda")
    dx[rows] = torch.einsum("rw,r->rw", d - d.mean(1)[:, None] - xhat * along[:, None], rstd)
    if st["dres"] is not None:
        dx[rows] += st["dres"][rows].double()
    return dict(dx=dx, dgamma=torch.einsum("rw,rw->w", dy, xhat), dbeta=torch.einsum("rw->w", dy))


def _mulhilo(a, m):
    """High and low words of a m for 32-bit words, by 16-bit halves."""
    ah, al, mh, ml = a >> 16, a & 0xFFFF, m >> 16, m & 0xFFFF
    mid = ah * ml + ((al * ml) >> 16)
    mid2 = al * mh + (mid & 0xFFFF)
    return ah * mh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((al * ml) & 0xFFFF)


def _exact_dropout(st, case):
    n, p = case["n"], case["p"]
    step = st["offset"] + int(st["step"])
    i = torch.arange(n, device="cuda")
    q = (i[::4] // 4)
    x0, x1 = q % 2 ** 32, q // 2 ** 32
    x2, x3 = torch.zeros_like(q) + step % 2 ** 32, torch.zeros_like(q) + step // 2 ** 32 % 2 ** 32
    for r in range(10):
        h0, l0 = _mulhilo(x0, 0xD2511F53)
        h1, l1 = _mulhilo(x2, 0xCD9E8D57)
        key0 = (st["seed"] + r * 0x9E3779B9) % 2 ** 32
        key1 = (st["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        x0, x1, x2, x3 = h1 ^ x1 ^ key0, l1, h0 ^ x3 ^ key1, l0
    word = torch.stack([x0, x1, x2, x3]).T.reshape(-1)[:n]
    kept = (word >= math.floor(p * 2.0 ** 32)).double()
    out = st["x"].double() * kept / (1.0 - p)
    return dict(out=out if st["residual"] is None else out + st["residual"].double())


def exact(case, seed):
    st = prepare(case, seed)
    return dict(ffn=_exact_ffn, ffn_bwd=_exact_ffn_bwd, norm=_exact_norm, norm_bwd=_exact_norm_bwd,
                dropout=_exact_dropout)[case["op"]](st, case)
