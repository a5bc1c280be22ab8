"""The router's and the gradient clip's operators as cases that can be timed and compared.

Four operators around the experts' backward: the router's forward (top-k, gates,
balance and z losses, counts), its backward, the gate gradient of the retained
pairs, and the global gradient norm with clipping.  ``run`` computes them in
plain torch operations, or with ``own`` through the library.
"""

import math

import torch

own = False

F32, BF16 = "f32", "bf16"
TORCH = {F32: torch.float32, BF16: torch.bfloat16}
SIZE = {F32: 4, BF16: 2}
AUX_COEF, Z_COEF = 0.01, 0.001

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
        # the smallest layer of the repository: a few hundred tokens, latency only
        dict(name="router_fwd tiny", op="fwd", T=256, E=8, k=2, dtype=F32, masked=False, renorm=True),
        # the benchmark's layer: 4 sequences of 8192 tokens
        dict(name="router_fwd layer", op="fwd", T=32768, E=128, k=8, dtype=F32, masked=False, renorm=True),
        # E and k that are no powers of two, bf16 logits with ties, padding tokens, gates not renormalised
        dict(name="router_fwd ragged bf16", op="fwd", T=20011, E=160, k=6, dtype=BF16, masked=True, renorm=False),
        # the same three kinds of layer in the backward direction; the last one is the large batch
        dict(name="router_bwd tiny", op="bwd", T=256, E=8, k=2, dtype=F32, masked=False, renorm=True),
        dict(name="router_bwd ragged bf16", op="bwd", T=20011, E=160, k=6, dtype=BF16, masked=True, renorm=False),
        dict(name="router_bwd stress", op="bwd", T=131072, E=128, k=8, dtype=F32, masked=False, renorm=True),
        # gate gradients: the tiny layer, an odd-sized layer with wide rows, the benchmark's layer
        dict(name="gate_grad tiny", op="gate", N=512, E=8, I=32, rows=333, spare=40),
        dict(name="gate_grad ragged", op="gate", N=60003, E=20, I=1496, rows=30011, spare=1000),
        dict(name="gate_grad layer", op="gate", N=262144, E=128, I=768, rows=87204, spare=8192),
        # clipping: the weight gradients of one tiny layer with its router and norms; several hundred odd-sized
        # tensors of both types (a whole model's small parameters); the two expert gradients of the benchmark's layer
        dict(name="grad_clip tiny", op="clip", tensors=6, largest=32768, dtype=F32, spread=True, clipped=True),
        dict(name="grad_clip many bf16", op="clip", tensors=400, largest=1000003, dtype=BF16, spread=True, clipped=True),
        dict(name="grad_clip layer", op="clip", tensors=2, largest=402653184, dtype=F32, spread=False, clipped=True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "gate", "clip"])
    dtype = rng.choice([F32, BF16])
    if op in ("fwd", "bwd"):
        E = _log(rng, 2, 512)
        T = min(_log(rng, 64, 131072), 131072 * 128 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 12)), dtype=dtype, masked=rng.random() < 0.5,
                    renorm=rng.random() < 0.5)
    if op == "gate":
        I = 8 * _log(rng, 2, 256)
        rows = min(_log(rng, 200, 200000), 131072 * 1024 // I)
        return dict(op=op, N=rows + rng.randint(0, 2 * rows), E=_log(rng, 2, 256), I=I, rows=rows,
                    spare=rng.randint(0, rows // 4))
    tensors = _log(rng, 1, 500)
    return dict(op=op, tensors=tensors, largest=_log(rng, 2000, 200000000 // tensors), dtype=dtype,
                spread=rng.random() < 0.7, clipped=rng.random() < 0.8)


def _sizes(case):
    """Element counts of the clipped tensors: the largest, then (spread) sizes over the
    whole range below it, odd ones and single elements among them, else halves of it."""
    n, top = case["tensors"], case["largest"]
    if not case["spread"]:
        return [top if i == 0 else top // 2 for i in range(n)]
    return [max(1, int(top ** (1.0 - ((i * 7) % n) / n))) for i in range(n)]


# ---------------------------------------------------------------------------
# inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _logits(case, g):
    # random logits plus an expert's own bias: a skewed router, as the workloads' Zipf prior gives
    T, E = case["T"], case["E"]
    rank = torch.randperm(E, generator=g, device="cuda").float()
    x = torch.randn(T, E, generator=g, device="cuda") - 0.8 * torch.log(rank + 1.0)
    valid = (torch.rand(T, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["masked"] else None
    return x.to(TORCH[case["dtype"]]), valid


def _prepare_fwd(case, g):
    logits, valid = _logits(case, g)
    T, E, k = case["T"], case["E"], case["k"]
    state = dict(logits=logits, valid=valid)
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    state["out"] = dict(expert_idx=torch.empty(T, k, **i32), alpha=torch.empty(T, k, **f32),
                        row_stats=torch.empty(T, 2, **f32), counts=torch.empty(E, **i32), f=torch.empty(E, **f32),
                        P=torch.empty(E, **f32), losses=torch.empty(4, **f32))
    return state


def _prepare_bwd(case, g):
    # what the forward left for the backward, and gate gradients as small as a mean loss gives
    state = _prepare_fwd(case, g)
    saved = _plain_fwd(dict(state, case=case))
    losses = torch.zeros(4, device="cuda")
    losses[:3] = saved["losses"]
    losses.view(torch.int32)[3:] = saved["tokens"]
    dgate = torch.randn(case["T"], case["k"], generator=g, device="cuda") * saved["alpha"] * 0.01
    return dict(logits=state["logits"], expert_idx=saved["expert_idx"], alpha=saved["alpha"],
                row_stats=saved["row_stats"], f=saved["f"], losses=losses, dgate=dgate,
                dlogits=torch.empty_like(state["logits"]))


def _prepare_gate(case, g):
    N, E, I, rows = case["N"], case["E"], case["I"], case["rows"]
    room = rows + case["spare"]
    phi = torch.randn(room, I, generator=g, device="cuda").mul_(
        0.5 + 1.5 * torch.rand(room, 1, generator=g, device="cuda")).to(torch.bfloat16)
    dphi = torch.randn(room, I, generator=g, device="cuda").mul_(
        torch.rand(room, 1, generator=g, device="cuda")).to(torch.bfloat16)
    # the retained pairs, expert-major, ascending within an expert
    u = torch.randperm(N, generator=g, device="cuda")[:rows].sort().values
    e = torch.randint(0, E, (rows,), generator=g, device="cuda")
    ids = torch.zeros(room, dtype=torch.int32, device="cuda")
    ids[:rows] = u[e.sort(stable=True).indices].to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, e, torch.ones_like(e)).cumsum(0)
    return dict(dphi=dphi, phi=phi, ids=ids, offsets=offsets, dgate=torch.empty(N, device="cuda"))


def _prepare_clip(case, g):
    # the gradients lie in one buffer a type, each at a 256-byte boundary, as a program that owns its
    # gradients keeps them; the clipped ones go to a second buffer
    sizes = _sizes(case)
    dt = TORCH[case["dtype"]]
    step = 256 // SIZE[case["dtype"]]
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // step) * step
    src = torch.zeros(at, dtype=dt, device="cuda")
    for n, a in zip(sizes, starts):
        src[a:a + n].normal_(0.0, 0.01, generator=g)
    dst = torch.zeros_like(src)
    expected = 0.01 * math.sqrt(sum(sizes))
    state = dict(src=src, dst=dst, max_norm=expected * (0.1 if case["clipped"] else 10.0),
                 grads=[src[a:a + n] for n, a in zip(sizes, starts)],
                 clipped=[dst[a:a + n] for n, a in zip(sizes, starts)])
    return state


def _plan(case, state):
    """What a program that uses the library keeps beside its tensors."""
    if not own:
        return None
    lrm, ctx = _lib()
    if case["op"] == "clip":
        from backward_token_expert_gb300.pipeline import GradClip

        return GradClip(state["grads"], state["clipped"])
    if case["op"] == "gate":
        return lrm.dims_of(case["N"], case["E"], 1, 8, case["I"])
    dims = lrm.dims_of(case["T"], case["E"], case["k"], 8, 8)
    need = lrm.lrm_workspace_size(ctx, lrm.LRM_OP_ROUTER, dims) if case["op"] == "fwd" else 0
    return dims, torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    make = dict(fwd=_prepare_fwd, bwd=_prepare_bwd, gate=_prepare_gate, clip=_prepare_clip)[case["op"]]
    state = make(case, g)
    state["case"] = case
    state["plan"] = _plan(case, state)
    return state


# ---------------------------------------------------------------------------
# the plain forms


def _plain_fwd(state):
    case, k = state["case"], state["case"]["k"]
    x = state["logits"].float()
    T, E = x.shape
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    p = e / s
    ids = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    alpha = p.gather(1, ids)
    if case["renorm"]:
        alpha = alpha / alpha.sum(1, keepdim=True)
    stats = torch.cat([m, s], 1)
    counted = torch.ones(T, 1, device="cuda") if state["valid"] is None else state["valid"].float()[:, None]
    alpha, stats = alpha * counted, stats * counted
    tokens = counted.sum()
    one = counted.to(torch.int32).expand(T, k).reshape(-1)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda").scatter_add_(0, ids.reshape(-1), one)
    f = counts.float() / (tokens * k).clamp(min=1.0)
    P = (p * counted).sum(0) / tokens.clamp(min=1.0)
    aux = E * (f * P).sum()
    lse = m + torch.log(s)
    z = (lse * lse * counted).sum() / tokens.clamp(min=1.0)
    return dict(expert_idx=ids.to(torch.int32), alpha=alpha, row_stats=stats, counts=counts, f=f, P=P,
                losses=torch.stack([AUX_COEF * aux + Z_COEF * z, aux, z]), tokens=tokens.to(torch.int32).reshape(1))


def _plain_bwd(state):
    case, E = state["case"], state["case"]["E"]
    x = state["logits"].float()
    m, s = state["row_stats"][:, :1], state["row_stats"][:, 1:]
    counted = (s > 0).float()
    s = torch.where(s > 0, s, 1.0)
    p = torch.exp(x - m) / s
    tokens = state["losses"].view(torch.int32)[3:].float().clamp(min=1.0)
    fp = (p * state["f"]).sum(1, keepdim=True)
    d = p * ((AUX_COEF * E / tokens) * (state["f"] - fp) + (2.0 * Z_COEF / tokens) * (m + torch.log(s)))
    dg = state["dgate"]
    S = dg.sum(1, keepdim=True)
    ids = state["expert_idx"].long()
    if case["renorm"]:
        d = d.scatter_add(1, ids, dg - state["alpha"] * S)
    else:
        d = (d - p * S).scatter_add(1, ids, dg)
    return dict(dlogits=(d * counted).to(state["logits"].dtype))


def _plain_gate(state):
    N, rows = state["case"]["N"], state["phi"].shape[0]
    dots = (state["dphi"].float() * state["phi"].float()).sum(1)
    kept = torch.arange(rows, device="cuda") < state["offsets"][-1]
    at = torch.where(kept, state["ids"].long(), N)
    out = torch.zeros(N + 1, device="cuda")
    out[at] = dots
    return dict(dgate=out[:N])


def _plain_clip(state):
    squares = [(t.float() * t.float()).sum() for t in state["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    finite = torch.isfinite(norm)
    coef = torch.where(finite & (norm > state["max_norm"]), state["max_norm"] / norm, 1.0)
    [d.copy_(t.float() * coef) for t, d in zip(state["grads"], state["clipped"])]
    return dict(norm=norm.reshape(1), coef=coef.reshape(1), grads=state["dst"])


# ---------------------------------------------------------------------------
# the library's calls


def _own_fwd(state):
    lrm, ctx = _lib()
    case, o, (dims, ws) = state["case"], state["out"], state["plan"]
    dt = lrm.DTYPE_F32 if case["dtype"] == F32 else lrm.DTYPE_BF16
    lrm.lrm_router_forward(ctx, state["logits"], dt, state["valid"], dims, case["renorm"], AUX_COEF, Z_COEF,
                           o["expert_idx"], o["alpha"], o["row_stats"], o["counts"], o["f"], o["P"], o["losses"], ws,
                           ws.numel())
    return dict(expert_idx=o["expert_idx"], alpha=o["alpha"], row_stats=o["row_stats"], counts=o["counts"], f=o["f"],
                P=o["P"], losses=o["losses"][:3], tokens=o["losses"].view(torch.int32)[3:])


def _own_bwd(state):
    lrm, ctx = _lib()
    case, (dims, _) = state["case"], state["plan"]
    dt = lrm.DTYPE_F32 if case["dtype"] == F32 else lrm.DTYPE_BF16
    lrm.lrm_router_backward(ctx, state["logits"], dt, state["expert_idx"], state["alpha"], state["row_stats"],
                            state["dgate"], state["f"], state["losses"], dims, case["renorm"], AUX_COEF, Z_COEF,
                            state["dlogits"], dt)
    return dict(dlogits=state["dlogits"])


def _own_gate(state):
    lrm, ctx = _lib()
    lrm.lrm_gate_grad(ctx, state["dphi"], state["phi"], state["offsets"], state["ids"], state["plan"],
                      state["phi"].shape[0], state["dgate"])
    return dict(dgate=state["dgate"])


def _own_clip(state):
    clip = state["plan"]
    clip.clip(state["max_norm"])
    return dict(norm=clip.norm, coef=clip.coef, grads=state["dst"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(fwd=_own_fwd, bwd=_own_bwd, gate=_own_gate, clip=_own_clip)[op](state)
    return dict(fwd=_plain_fwd, bwd=_plain_bwd, gate=_plain_gate, clip=_plain_clip)[op](state)


# ---------------------------------------------------------------------------
# work and the 64-bit values


def work(case):
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return dict(bytes=2 * n * SIZE[case["dtype"]], flops=3 * n)
    if case["op"] == "gate":
        return dict(bytes=4 * case["rows"] * case["I"] + 4 * case["rows"] + 4 * case["N"],
                    flops=2 * case["rows"] * case["I"])
    T, E, k, es = case["T"], case["E"], case["k"], SIZE[case["dtype"]]
    if case["op"] == "fwd":
        return dict(bytes=T * E * es + 8 * T * k + 8 * T + (T if case["masked"] else 0) + 12 * E, flops=5 * T * E)
    return dict(bytes=2 * T * E * es + 12 * T * k + 8 * T + 4 * E, flops=8 * T * E)


def _exact_fwd(st, case):
    l = st["logits"].double()
    T, E, k = case["T"], case["E"], case["k"]
    ok = torch.ones(T, dtype=torch.bool, device="cuda") if st["valid"] is None else st["valid"] != 0
    # rank of an expert: how many are larger, or equal with a lower index; by a 64-bit sort key free of ties
    ids = (-l).argsort(dim=1, stable=True)[:, :k]
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    picked = torch.gather(l, 1, ids)
    base = torch.logsumexp(picked, 1) if case["renorm"] else lse
    alpha = torch.where(ok[:, None], torch.exp(picked - base[:, None]), 0.0)
    m = l.max(1).values
    stats = torch.where(ok[:, None], torch.stack([m, torch.exp(lse - m)], 1), 0.0)
    tokens = int(ok.sum())
    counts = torch.bincount(ids[ok].reshape(-1), minlength=E)
    f = counts.double() / max(1, tokens * k)
    P = p[ok].sum(0) / max(1, tokens)
    aux, z = E * torch.dot(f, P), lse[ok].square().sum() / max(1, tokens)
    return dict(expert_idx=ids.int(), alpha=alpha, row_stats=stats, counts=counts.int(), f=f, P=P,
                losses=torch.stack([AUX_COEF * aux + Z_COEF * z, aux, z]),
                tokens=torch.tensor([tokens], dtype=torch.int32))


def _exact_bwd(st, case):
    # the softmax's Jacobian applied to dL/dp (balance, gates) and the z loss's own gradient
    l = st["logits"].double()
    m, s = st["row_stats"].double().unbind(1)
    ok = s > 0
    tokens = max(1, int(st["losses"].view(torch.int32)[3]))
    lse = torch.where(ok, m + torch.log(torch.where(ok, s, 1.0)), 0.0)
    p = torch.exp(l - lse[:, None])
    up = (AUX_COEF * case["E"] / tokens) * st["f"].double().expand_as(p)
    grad = p * (up - (p * up).sum(1, keepdim=True)) + p * (2.0 * Z_COEF / tokens * lse)[:, None]
    dg, alpha, ids = st["dgate"].double(), st["alpha"].double(), st["expert_idx"].long()
    total = dg.sum(1, keepdim=True)
    at = torch.zeros_like(grad).scatter_(1, ids, dg - alpha * total if case["renorm"] else dg)
    grad = grad + at - (0.0 if case["renorm"] else p * total)
    return dict(dlogits=torch.where(ok[:, None], grad, 0.0))


def _exact_gate(st, case):
    rows = int(st["offsets"][-1])
    out = torch.zeros(case["N"], dtype=torch.float64, device="cuda")
    for a in range(0, rows, 65536):
        b = min(rows, a + 65536)
        out[st["ids"][a:b].long()] = torch.einsum("ri,ri->r", st["dphi"][a:b].double(), st["phi"][a:b].double())
    return dict(dgate=out)


def _exact_clip(st, case):
    total = sum(float(t.double().square().sum()) for t in st["grads"])
    norm = math.sqrt(total)
    coef = min(1.0, st["max_norm"] / norm)
    one = dict(dtype=torch.float64)
    return dict(norm=torch.tensor([norm], **one), coef=torch.tensor([coef], **one), grads=st["src"].double() * coef)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(fwd=_exact_fwd, bwd=_exact_bwd, gate=_exact_gate, clip=_exact_clip)[case["op"]](st, case)
