"""The experts' sub-layer, as cases to be measured.

What a served token goes through after attention: routing to experts (``route``), their gated up
projection with an 8-bit output (``up``), their down projection with the weighted sum over a
token's experts (``down``), and the product that both stand on, as a plain projection through 8-bit
weights with a scale per 128 x 128 block (``f8``).  ``run`` computes them in plain torch operations
in 32 bits (the routing in 64, whose choices are whole numbers), or, where ``own`` is true, through
this package's entry points."""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode token: latency
        dict(name="route_one", op="route", T=1, E=256, k=8, softmax=False, bias=True, groups=8, top=4, best=2, bf16=False, pad=0, shut=0),
        # a long prompt over many experts in groups, with a balance bias
        dict(name="route_prompt", op="route", T=16384, E=256, k=8, softmax=False, bias=True, groups=8, top=4, best=2, bf16=False, pad=0, shut=0),
        # an odd batch over an odd number of experts, some of them shut, its last rows padding
        dict(name="route_softmax_odd", op="route", T=777, E=60, k=4, softmax=True, bias=False, groups=1, top=1, best=1, bf16=True, pad=7, shut=3),
        # one decode token through the query, key and value weights
        dict(name="f8_one", op="f8", T=1, K=4096, N=6144, xs="e8m0"),
        # an odd number of sequences' tokens
        dict(name="f8_odd", op="f8", T=37, K=4096, N=14336, xs="f32"),
        # a short prompt through weights whose last block of 128 outputs is a short one
        dict(name="f8_chunk", op="f8", T=500, K=2048, N=5200, xs="e8m0"),
        # a prompt through weights of the engram projection's shape
        dict(name="f8_prompt", op="f8", T=4096, K=6144, N=20480, xs="e8m0"),
        # one decode token's experts: latency, and the experts' weights once
        dict(name="up_one", op="up", T=1, E=256, k=8, K=4096, I=2048, xs="e8m0"),
        # a decode step of 64 sequences, which meets most of the experts
        dict(name="up_step", op="up", T=64, E=256, k=8, K=4096, I=2048, xs="e8m0"),
        # a prompt over fewer experts: some hundred rows each, unevenly
        dict(name="up_prompt", op="up", T=4096, E=64, k=8, K=4096, I=2048, xs="e8m0"),
        dict(name="down_step", op="down", T=64, E=256, k=8, K=2048, N=4096, xs="e8m0"),
        dict(name="down_prompt", op="down", T=4096, E=64, k=8, K=2048, N=4096, xs="e8m0"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "f8", "up", "down"])
    if op == "route":
        E = rng.choice([8, 60, 64, 160, 256, 384])
        groups = rng.choice([1, 1, 4] if E in (8, 60) else [1, 4, 8])
        T = _log(rng, 1, 16384 * 256 // max(E, 256))
        return dict(op=op, T=T, E=E, k=rng.choice([1, 2, 4, 6, 8] if E > 8 else [1, 2]), softmax=rng.random() < 0.5, bias=rng.random() < 0.6, groups=groups,
                    top=rng.randint(1, max(1, groups // 2)), best=rng.choice([1, 2]), bf16=rng.random() < 0.4, pad=rng.choice([0, 0, T // 5]), shut=rng.choice([0, 0, E // 8]))
    T, xs = _log(rng, 1, 4096), rng.choice(["e8m0", "f32"])
    if op == "f8":
        return dict(op=op, T=T, K=128 * _log(rng, 1, 48), N=16 * _log(rng, 16, 1280), xs=xs)
    E = rng.choice([4, 8, 16, 60, 64, 160, 256])
    k = rng.choice([1, 2, 4] if E < 8 else [1, 2, 4, 6, 8])
    if op == "up":
        return dict(op=op, T=T, E=E, k=k, K=128 * _log(rng, 1, 32), I=128 * _log(rng, 1, 16), xs=xs)
    return dict(op=op, T=T, E=E, k=k, K=128 * _log(rng, 1, 16), N=16 * _log(rng, 16, 256), xs=xs)


def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        return {"bytes": T * case["E"] * (2 if case["bf16"] else 4) + 4 * case["E"] * (2 if case["bias"] else 1) + 12 * T * case["k"], "flops": 8 * T * case["E"]}
    K = case["K"]
    if op == "f8":
        return {"bytes": case["N"] * K * (1 + 1 / 4096) + T * K * (1 + 1 / 32) + 2 * T * case["N"], "flops": 2 * T * K * case["N"]}
    E, R = case["E"], T * case["k"]
    met = E * (1 - (1 - case["k"] / E) ** T)  # experts that an even routing meets
    if op == "up":
        return {"bytes": met * 2 * case["I"] * K * (1 + 1 / 4096) + T * K * (1 + 1 / 32) + R * case["I"] * (1 + 1 / 32), "flops": 4 * R * K * case["I"]}
    return {"bytes": met * case["N"] * K * (1 + 1 / 4096) + R * K * (1 + 1 / 32) + 2 * T * case["N"], "flops": 2 * R * K * case["N"]}


# ------------------------------------------------------------------------------------ inputs
def _weights(g, *shape):
    """e4m3 codes [..., N, K], normal, with an f32 scale per 128 x 128 block, all blocks different."""
    N, K = shape[-2:]
    w = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(96).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    blocks = (*shape[:-2], (N + BLOCK - 1) // BLOCK, (K + BLOCK - 1) // BLOCK)
    return w, (0.5 + torch.rand(*blocks, generator=g, device="cuda")) / (96 * math.sqrt(K))


def _rows(g, rows, K, kind):
    """Normal rows, some channels louder, in e4m3 with a power of two per 32 values or an f32 scale per 128."""
    x = torch.randn(rows, K, generator=g, device="cuda") * torch.exp2(torch.rand(K, generator=g, device="cuda") * 2 - 1)
    b = x.view(rows, K // (32 if kind == "e8m0" else BLOCK), -1)
    if kind == "e8m0":
        e = torch.ceil(torch.log2(b.abs().amax(2) / E4M3_MAX))
        return (b / torch.exp2(e)[:, :, None]).view(rows, K).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)
    s = b.abs().amax(2) / E4M3_MAX
    return (b / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, K).to(torch.float8_e4m3fn).view(torch.uint8), s


def _logits(g, T, E):
    """Normal logits over experts that are not equally liked."""
    return torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, bf, i32 = case["op"], case["T"], torch.bfloat16, torch.int32
    st = dict(case, w=None)
    if op == "f8":
        st["x"], st["s"] = _rows(g, T, case["K"], case["xs"])
        st["w"], st["ws"] = _weights(g, case["N"], case["K"])
        st["y"] = torch.empty(T, case["N"], dtype=bf, device="cuda")
    else:
        E, k = case["E"], case["k"]
        st["ids"] = torch.zeros(T, k, dtype=i32, device="cuda")
        st["weights"] = torch.zeros(T, k, device="cuda")
        st["offsets"] = torch.zeros(E + 1, dtype=i32, device="cuda")
        st["order"] = torch.zeros(T * k, dtype=i32, device="cuda")
        x = _logits(g, T, E)
    if op == "route":
        x[:, torch.randperm(E, generator=g, device="cuda")[:case["shut"]]] = -math.inf
        if case["pad"]:
            x[T - case["pad"]:] = -math.inf
        st["logits"] = x.to(bf) if case["bf16"] else x
        st["b"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
    elif op != "f8":
        # the plan that the routing made
        top = torch.topk(x, k, 1)
        st["ids"], st["weights"] = top.indices.to(i32), torch.softmax(top.values, 1)
        flat = top.indices.view(-1)
        counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
        st["offsets"][1:] = counts.cumsum(0)
        st["order"] = torch.sort(flat, stable=True).indices.to(i32)
        st["most"] = int(counts.max())
        if op == "up":
            st["x"], st["s"] = _rows(g, T, case["K"], case["xs"])
            st["w"], st["ws"] = _weights(g, E, 2, case["I"], case["K"])
            st["h"] = torch.empty(T * k, case["I"], dtype=torch.uint8, device="cuda")
            st["hs"] = torch.empty(T * k, case["I"] // 32, dtype=torch.uint8, device="cuda")
        else:
            st["x"], st["s"] = _rows(g, T * k, case["K"], case["xs"])
            st["w"], st["ws"] = _weights(g, E, case["N"], case["K"])
            st["y"] = torch.empty(T, case["N"], dtype=bf, device="cuda")
    if own:
        import gram_hashed_embedding_engram_amd as M
        st["wf8"] = None if st["w"] is None else M.F8(st["w"], st["ws"])
        if op != "f8":
            st["routes"] = M.Routes(st["ids"], st["weights"], st["offsets"], st["order"])
            need = M.route_bytes(st["routes"]) if op == "route" else M.experts_down_bytes(st["wf8"], st["routes"]) if op == "down" else 0
            st["space"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return st


# -------------------------------------------------------------------------------- plain forms
def _route(st):
    T, E, k = st["T"], st["E"], st["k"]
    x = st["logits"].double()
    free = torch.isfinite(x)
    low = torch.full_like(x, -math.inf)
    if st["softmax"]:
        top = torch.where(free, x, low).amax(1, keepdim=True)
        p = torch.where(free, torch.exp(x - torch.where(torch.isfinite(top), top, torch.zeros_like(top))), torch.zeros_like(x))
        score = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = torch.where(free, 1 / (1 + torch.exp(-x)), torch.zeros_like(x))
    liked = score if st["b"] is None else score + st["b"].double()
    key = torch.where(free, x if st["b"] is None else liked, low)
    if st["groups"] > 1:
        inside = torch.where(free, liked, low).view(T, st["groups"], -1)
        best = torch.sort(inside, dim=2, descending=True).values[:, :, :st["best"]]
        total = torch.where(torch.isfinite(best), best, torch.zeros_like(best)).sum(2)
        total = torch.where(torch.isfinite(best[:, :, 0]), total, torch.full_like(total, -math.inf))
        kept = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :st["top"]]
        mask = torch.zeros_like(total, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(mask.repeat_interleave(E // st["groups"], 1), key, low)
    first = torch.sort(key, dim=1, descending=True, stable=True)
    ids = first.indices[:, :k]
    some = torch.isfinite(first.values[:, :k])
    w = torch.where(some, torch.gather(score, 1, ids), torch.zeros_like(score[:, :k]))
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = torch.where(some, ids, torch.full_like(ids, -1))
    flat = torch.where(some, ids, torch.full_like(ids, E)).view(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat((torch.zeros_like(counts[:1]), counts[:E].cumsum(0)))
    order = torch.sort(flat, stable=True).indices
    order = torch.where(torch.arange(T * k, device=x.device) < offsets[E], order, torch.zeros_like(order))
    return ids.int(), w.float(), offsets.int(), order.int()


def _values(codes, scales):
    """Rows of codes times their scales, as f32."""
    v = codes.view(torch.float8_e4m3fn).float()
    s = scales if scales.dtype == torch.float32 else torch.exp2(scales.float() - 127)
    return (v.view(*s.shape, -1) * s[..., None]).view_as(v)


def _matrix(w, s):
    """Weights as f32: codes times their block's scale."""
    N, K = w.shape[-2:]
    v = w.view(torch.float8_e4m3fn).float()
    wide = s.repeat_interleave(BLOCK, -2)[..., :N, :]
    return v.view(*v.shape[:-1], K // BLOCK, BLOCK).mul_(wide[..., None]).view_as(v)


def _grouped(rows, st):
    """Row p of the plan (already in its order) times its expert's weights, [rows, outputs]."""
    E, R = st["E"], st["T"] * st["k"]
    w, s = st["w"].view(E, -1, st["K"]), st["ws"]
    expert = torch.searchsorted(st["offsets"].long(), torch.arange(R, device=rows.device), right=True) - 1
    if R < E:  # each row's own matrix
        m = _matrix(st["w"][expert], s[expert]).view(R, -1, st["K"])
        return torch.bmm(m, rows[:, :, None])[:, :, 0]
    at = torch.arange(R, device=rows.device) - st["offsets"].long()[expert]
    wide = torch.zeros(E, st["most"], st["K"], device=rows.device)
    wide[expert, at] = rows
    out = torch.bmm(wide, _matrix(st["w"], s).view_as(w).transpose(1, 2))
    return out[expert, at]


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), 2^-126 at least."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126))


def _f8(st):
    return torch.mm(_values(st["x"], st["s"]), _matrix(st["w"], st["ws"]).t()).to(torch.bfloat16)


def _up(st):
    x = _values(st["x"], st["s"])[st["order"].long() // st["k"]]
    gate, up = _grouped(x, st).chunk(2, 1)
    h = gate / (1 + torch.exp(-gate)) * up
    b = h.reshape(h.shape[0], -1, 32)
    s = _pow2_scale(b.abs().amax(2))
    return (b / s[:, :, None]).view_as(h).to(torch.float8_e4m3fn), s.to(torch.float8_e8m0fnu)


def _down(st):
    p = _grouped(_values(st["x"], st["s"]), st)
    slot = st["order"].long()
    mine = torch.zeros_like(p)
    mine[slot] = p * st["weights"].view(-1)[slot][:, None]
    return mine.view(st["T"], st["k"], -1).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------------- 64-bit definitions
def _rows64(codes, scales):
    s = scales.to(torch.float64) if scales.dtype == torch.float32 else torch.exp2(scales.to(torch.float64) - 127)
    return codes.view(torch.float8_e4m3fn).to(torch.float64) * s.repeat_interleave(codes.shape[1] // s.shape[1], 1)


def _weights64(codes, scales):
    N, K = codes.shape
    blocks = scales.to(torch.float64)[torch.arange(N, device="cuda") // BLOCK][:, torch.arange(K, device="cuda") // BLOCK]
    return codes.view(torch.float8_e4m3fn).to(torch.float64) * blocks


def _nearest_e4m3(v):
    """The e4m3 values nearest to v (|v| <= 448), ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _scale64(amax):
    """2^k, k the least whole number with amax <= 448 * 2^k."""
    k = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -117) / E4M3_MAX))
    k = torch.where(E4M3_MAX * torch.exp2(k - 1) >= amax, k - 1, k)
    return torch.exp2(torch.where(E4M3_MAX * torch.exp2(k) < amax, k + 1, k).clamp(min=-126.0))


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]

    def route_weights():
        """On the host, row by row, by a comparison of whole entries."""
        x = st["logits"].double().cpu().numpy()
        T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
        b = None if st["b"] is None else st["b"].double().cpu().numpy()
        out = np.zeros((T, k))
        for t in range(T):
            some = np.flatnonzero(np.isfinite(x[t]))
            if not some.size:
                continue
            v = x[t, some]
            score = np.exp(v - v.max()) / np.exp(v - v.max()).sum() if st["softmax"] else 1 / (1 + np.exp(-v))
            liked = score if b is None else score + b[some]
            key = v if b is None else liked
            if G > 1:
                of = some // (E // G)
                total = [(-sum(sorted(liked[of == j], reverse=True)[:st["best"]]), j) for j in sorted(set(of.tolist()))]
                kept = np.isin(of, [j for _, j in sorted(total)[:st["top"]]])
                some, score, key = some[kept], score[kept], key[kept]
            chosen = sorted(range(some.size), key=lambda i: (-key[i], some[i]))[:k]
            total = sum(score[i] for i in chosen)
            out[t, :len(chosen)] = [score[i] / total for i in chosen]
        return torch.from_numpy(out)

    if op == "route":
        return None, route_weights(), None, None
    x = _rows64(st["x"], st["s"])
    if op == "f8":
        return x @ _weights64(st["w"], st["ws"]).t()
    offsets, order, k = st["offsets"].tolist(), st["order"].long(), case["k"]
    if op == "up":
        h = torch.empty(case["T"] * k, case["I"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            p, q = offsets[e], offsets[e + 1]
            if q > p:
                mine = x[order[p:q] // k]
                gate, up = (mine @ _weights64(st["w"][e, i], st["ws"][e, i]).t() for i in range(2))
                h[p:q] = gate * torch.sigmoid(gate) * up
        s = _scale64(h.abs().view(h.shape[0], -1, 32).amax(2))
        return _nearest_e4m3(h / s.repeat_interleave(32, 1)), s
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
    weights = st["weights"].double().view(-1)
    for e in range(case["E"]):
        p, q = offsets[e], offsets[e + 1]
        if q > p:
            slot = order[p:q]
            y[slot // k] += (x[p:q] @ _weights64(st["w"][e], st["ws"][e]).t()) * weights[slot][:, None]
    return y


# ---------------------------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if not own:
        return {"route": _route, "f8": _f8, "up": _up, "down": _down}[op](state)
    import gram_hashed_embedding_engram_amd as M
    if op == "route":
        M.route(state["logits"], state["routes"], state["b"], softmax=state["softmax"], groups=state["groups"], top_groups=state["top"], group_best=state["best"], d_ws=state["space"])
        return state["ids"], state["weights"], state["offsets"], state["order"]
    if op == "f8":
        M.project_f8(state["x"], state["wf8"], state["y"], state["s"])
        return state["y"]
    if op == "up":
        M.experts_up(state["x"], state["s"], state["wf8"], state["routes"], state["h"], state["hs"])
        return state["h"].view(torch.float8_e4m3fn), state["hs"].view(torch.float8_e8m0fnu)
    M.experts_down(state["x"], state["s"], state["wf8"], state["routes"], state["y"], d_ws=state["space"])
    return state["y"]
