"""The attention sub-layer beside the engram layer, as cases to be measured.

Four operators that a served token goes through after the engram has been added to the highway:
the residual's addition with the root-mean-square norm and an 8-bit output (``norm``), the
projection of few tokens through 4-bit weights with a scale per 32 values (``w4``), the position
rotation with the append to a paged 8-bit cache (``append``), and attention over that cache
(``attend``).  ``run`` computes them in plain torch operations in 32 bits, or, where ``own`` is
true, through this package's entry points."""
import math
import random

import torch

own = False

PAGE = 64
E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence on one highway stream: latency
        dict(name="norm_one", op="norm", rows=1, dim=4096, res="f32", add=True),
        # a 4096-token prompt on the four FP32 highway streams
        dict(name="norm_prompt", op="norm", rows=16384, dim=4096, res="f32", add=True),
        # a batch of tokens on a bf16 residual of a width that is no power of two
        dict(name="norm_bf16_odd", op="norm", rows=777, dim=7200, res="bf16", add=True),
        # one decode token through the query, key and value weights
        dict(name="w4_one", op="w4", T=1, K=4096, N=6144, x="e4m3"),
        # sixteen sequences' tokens through weights of the engram projection's shape
        dict(name="w4_sixteen", op="w4", T=16, K=6144, N=20480, x="e4m3"),
        # an odd number of sequences through an output projection: bf16 activations
        dict(name="w4_bf16_odd", op="w4", T=37, K=4096, N=14336, x="bf16"),
        # a decode step of 64 sequences of ragged lengths
        dict(name="append_step", op="append", B=64, n=1, ragged=False, past=8192, kv=8, q=32, d=128, rot=128, halves=True),
        # ragged prompts, after a cached prefix that ends inside a page
        dict(name="append_prompt", op="append", B=5, n=4096, ragged=True, past=200, kv=8, q=32, d=128, rot=64, halves=False),
        # one sequence's token over a short cache: latency
        dict(name="attend_short", op="attend", B=1, n=1, ragged=False, past=500, kv=8, q=32, d=128, window=0),
        # a decode step of 64 sequences of ragged lengths
        dict(name="attend_step", op="attend", B=64, n=1, ragged=False, past=8192, kv=8, q=32, d=128, window=0),
        # one sequence's token over a long cache with few, wide heads
        dict(name="attend_long", op="attend", B=1, n=1, ragged=False, past=131071, kv=4, q=32, d=256, window=0),
        # two ragged prompt chunks over what is cached already
        dict(name="attend_prompt", op="attend", B=2, n=4096, ragged=True, past=1500, kv=8, q=32, d=128, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "w4", "append", "attend", "attend"])
    if op == "norm":
        dim = 32 * _log(rng, 8, 320)
        return dict(op=op, rows=_log(rng, 1, max(1, (16384 * 4096) // dim)), dim=dim, res=rng.choice(["f32", "bf16"]), add=rng.random() < 0.8)
    if op == "w4":
        return dict(op=op, T=_log(rng, 1, 64), K=128 * _log(rng, 4, 48), N=16 * _log(rng, 16, 1280), x=rng.choice(["e4m3", "bf16"]))
    d = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    q = kv * rng.choice([1, 3, 4, 6, 8])
    if op == "append":
        if rng.random() < 0.5:
            return dict(op=op, B=_log(rng, 1, 128), n=1, ragged=False, past=_log(rng, 1, 8192), kv=kv, q=q, d=d, rot=rng.choice([d, d // 2]), halves=rng.random() < 0.5)
        return dict(op=op, B=rng.randint(1, 4), n=_log(rng, 2, 800), ragged=rng.random() < 0.7, past=_log(rng, 1, 2000), kv=kv, q=q, d=d, rot=rng.choice([d, d // 2]), halves=rng.random() < 0.5)
    if rng.random() < 0.65:
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, n=1, ragged=False, past=_log(rng, 1, max(2, 130000 // B)), kv=kv, q=q, d=d, window=rng.choice([0, 0, 1000]))
    return dict(op=op, B=rng.randint(1, 3), n=_log(rng, 2, 900), ragged=rng.random() < 0.7, past=_log(rng, 1, 1500), kv=kv, q=q, d=d, window=rng.choice([0, 0, 500]))


def _lengths(case):
    """(new tokens, cached positions before them) of each sequence: fixed by the case."""
    r = random.Random(case["B"] * 7919 + case["n"] * 31 + case["past"])
    B, n, past = case["B"], case["n"], case["past"]
    new = [n if b == 0 or not case["ragged"] else max(1, int(n * r.uniform(0.05, 1.0))) for b in range(B)]
    old = [past if b == 0 else int(past * r.uniform(0.1, 1.0)) for b in range(B)]
    return new, old


def _visible(case):
    """How many (query, position) pairs the mask leaves, and how many positions are read at all."""
    new, old = _lengths(case)
    w = case["window"]
    pairs = reach = 0
    for n, p in zip(new, old):
        pairs += sum(min(p + i + 1, w) for i in range(n)) if w else n * p + n * (n + 1) // 2
        reach += min(p + n, w + n - 1) if w else p + n
    return pairs, reach


def work(case):
    op = case["op"]
    if op == "norm":
        v = case["rows"] * case["dim"]
        r = 4 if case["res"] == "f32" else 2
        return {"bytes": v * ((2 * r + 2 if case["add"] else r) + 1 + 1 / 32) + 2 * case["dim"], "flops": 6 * v}
    if op == "w4":
        T, K, N = case["T"], case["K"], case["N"]
        x = T * K * 2 if case["x"] == "bf16" else T * K * (1 + 1 / 32)
        return {"bytes": N * K * (0.5 + 1 / 32) + x + 2 * T * N, "flops": 2 * T * K * N}
    T = sum(_lengths(case)[0])
    if op == "append":
        v = T * case["kv"] * case["d"]
        return {"bytes": 2 * v * 3 + 4 * T * case["q"] * case["d"], "flops": 8 * v + 4 * T * case["q"] * case["d"]}
    pairs, reach = _visible(case)
    return {"bytes": 2 * reach * case["kv"] * case["d"] + 4 * T * case["q"] * case["d"], "flops": 4 * pairs * case["q"] * case["d"]}


# ------------------------------------------------------------------------------------ inputs
def _cache(case, g, width, n_pages):
    """A paged cache of values as they come from key and value projections: normal, each head of a
    loudness of its own, each page under the scale that its largest value asks for."""
    kv, d = case["kv"], case["d"]
    out = []
    for loud in (1.0, 0.6):
        v = torch.randn(n_pages, kv, PAGE, d, generator=g, device="cuda")
        v *= loud * torch.exp2(torch.rand(1, kv, 1, 1, generator=g, device="cuda") * 2 - 1)
        s = torch.exp2(torch.ceil(torch.log2(v.abs().amax((2, 3)) / E4M3_MAX)))
        out += [(v / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s]
        del v
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    bf = torch.bfloat16
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if op == "norm":
        rows, dim = case["rows"], case["dim"]
        st = dict(op=op, eps=EPS, res=randn(rows, dim) * 2, w=(1 + 0.1 * randn(dim)).to(bf))
        st["res"] = st["res"].to(bf) if case["res"] == "bf16" else st["res"]
        # beside the residual, so that a pass can be repeated on the same inputs
        st["sum"] = torch.empty_like(st["res"]) if case["add"] else st["res"]
        st["x"] = (0.02 * randn(rows, dim)).to(bf) if case["add"] else None
        st["codes"] = torch.empty(rows, dim, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(rows, dim // 32, dtype=torch.uint8, device="cuda")
        return st
    if op == "w4":
        T, K, N = case["T"], case["K"], case["N"]
        w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        ws = torch.randint(119, 123, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        x = randn(T, K)
        st = dict(op=op, w=w, ws=ws, y=torch.empty(T, N, dtype=bf, device="cuda"), xs=None)
        if case["x"] == "bf16":
            st["x"] = x.to(bf)
        else:
            b = x.view(T, K // 32, 32)
            e = torch.ceil(torch.log2(b.abs().amax(2) / E4M3_MAX))
            st["x"] = (b / torch.exp2(e)[:, :, None]).view(T, K).to(torch.float8_e4m3fn).view(torch.uint8)
            st["xs"] = (e + 127).to(torch.uint8)
        if own:
            import gram_hashed_embedding_engram_amd as E
            st["weights"] = E.W4(w, ws)
        return st
    new, old = _lengths(case)
    B, kv, q, d, T = case["B"], case["kv"], case["q"], case["d"], sum(new)
    width = max((p + n + PAGE - 1) // PAGE for p, n in zip(old, new)) + 1
    used = sum((p + n + PAGE - 1) // PAGE for p, n in zip(old, new))
    n_pages = used + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").int()
    pages = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        m = (old[b] + new[b] + PAGE - 1) // PAGE
        pages[b, :m] = perm[at:at + m]
        at += m
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    kc, ks, vc, vs = _cache(case, g, width, n_pages)
    st = dict(op=op, pages=pages, start=torch.tensor(old, dtype=torch.int32, device="cuda"), kc=kc, ks=ks, vc=vc, vs=vs, kv=kv, q=q, d=d, T=T, B=B, max_new=max(new),
              cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), ragged=case["ragged"])
    if op == "append":
        # one projection's output holds the queries, keys and values side by side
        st["qkv"] = randn(T, (q + 2 * kv) * d).to(bf)
        rot = case["rot"]
        st["rot"], st["halves"] = rot, case["halves"]
        st["freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        st["qout"] = torch.empty(T, q, d, dtype=bf, device="cuda")
    else:
        st["query"] = randn(T, q, d).to(bf)
        st["out"] = torch.empty(T, q, d, dtype=bf, device="cuda")
        st["window"], st["scale"] = case["window"], 1.0 / math.sqrt(d)
    if own:
        import gram_hashed_embedding_engram_amd as E
        st["cache"] = E.Cache(kc, vc, ks, vs)
        st["seqs"] = E.Sequences(pages, st["start"], st["cu"] if case["ragged"] else None)
        if op == "attend":
            st["ws"] = torch.empty(E.cache_attend_bytes(st["cache"], st["seqs"], q, T), dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------------------------- plain forms
def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), 2^-126 at least."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126))


def _norm(st):
    r = st["res"].float()
    if st["x"] is not None:
        r = r + st["x"].float()
    total = r.to(st["res"].dtype)
    r = total.float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + st["eps"]) * st["w"].float()
    b = y.view(y.shape[0], -1, 32)
    s = _pow2_scale(b.abs().amax(2))
    codes = (b / s[:, :, None]).view_as(y).to(torch.float8_e4m3fn)
    return total, codes, s.to(torch.float8_e8m0fnu)


def _e2m1(w):
    """Packed 4-bit codes (the even value in the low nibble) as f32: sign, two exponent bits, one of mantissa."""
    c = torch.stack((w & 15, w >> 4), -1).view(w.shape[0], -1)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=w.device)
    return values[c.int()]


def _groups(v, s):
    """v [rows, K] times 2^(s - 127), one scale per 32 values."""
    return (v.view(v.shape[0], -1, 32) * torch.exp2(s.float() - 127)[:, :, None]).view_as(v)


def _w4(st):
    w = _groups(_e2m1(st["w"]), st["ws"])
    x = st["x"].float() if st["xs"] is None else _groups(st["x"].view(torch.float8_e4m3fn).float(), st["xs"])
    return torch.mm(x, w.t()).to(torch.bfloat16)


def _rotate(x, cos, sin, rot, halves):
    """x [T, heads, d] f32 with the first `rot` values of each head rotated in pairs."""
    r = x[..., :rot]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if halves else (r[..., 0::2], r[..., 1::2])
    c, s = cos[:, None], sin[:, None]
    p, t = a * c - b * s, a * s + b * c
    r = torch.cat((p, t), -1) if halves else torch.stack((p, t), -1).flatten(-2)
    return torch.cat((r, x[..., rot:]), -1)


def _append(st):
    T, q, kv, d = st["T"], st["q"], st["kv"], st["d"]
    dev = st["qkv"].device
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(st["cu"].long(), t, right=True) - 1
    pos = st["start"].long()[seq] + t - st["cu"].long()[seq]
    page, slot = st["pages"].long()[seq, pos // PAGE], pos % PAGE
    angle = pos[:, None].double() * st["freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    x = st["qkv"].float().view(T, q + 2 * kv, d)
    qr = _rotate(x[:, :q], cos, sin, st["rot"], st["halves"])
    # how many older positions the token's page holds
    older = (st["start"].long()[seq] - (pos - slot)).clamp(0, PAGE)
    out = [qr.to(torch.bfloat16)]
    for codes, scales, v in ((st["kc"], st["ks"], _rotate(x[:, q:q + kv], cos, sin, st["rot"], st["halves"])), (st["vc"], st["vs"], x[:, q + kv:])):
        need = torch.zeros_like(scales).index_reduce_(0, page, v.abs().amax(2), "amax")
        had = torch.where(older[:, None] > 0, scales[page], torch.zeros_like(scales[page]))
        s = torch.maximum(had, _pow2_scale(need)[page])
        # the older positions under the page's new scale, each token's page for itself
        vals = codes.view(torch.float8_e4m3fn)[page[older > 0]].float() * (scales[page] / s)[older > 0][:, :, None, None]
        keep = torch.arange(PAGE, device=dev)[None, :] < older[older > 0][:, None]
        codes[page[older > 0]] = torch.where(keep[:, None, :, None], vals.to(torch.float8_e4m3fn).view(torch.uint8), codes[page[older > 0]])
        codes[page, :, slot] = (v / s[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[page] = s
        out += [codes.view(torch.float8_e4m3fn), scales]
    return tuple(out)


def _attend(st):
    T, B, q, kv, d, n = st["T"], st["B"], st["q"], st["kv"], st["d"], st["max_new"]
    dev = st["query"].device
    cu, start = st["cu"].long(), st["start"].long()
    L = st["pages"].shape[1] * PAGE

    def taken(codes, scales):  # [B, kv, L, d]
        p = st["pages"].long()
        v = codes.view(torch.float8_e4m3fn)[p].float() * scales[p][..., None, None]
        return v.permute(0, 2, 1, 3, 4).reshape(B * kv, L, d)

    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[seq]
    g = q // kv
    query = torch.zeros(B, n, q, d, device=dev)
    query[seq, i] = st["query"].float()
    query = query.view(B, n, kv, g, d).permute(0, 2, 1, 3, 4).reshape(B * kv, n * g, d)
    s = torch.bmm(query, taken(st["kc"], st["ks"]).transpose(1, 2).contiguous()).mul_(st["scale"]).view(B, kv, n, g, L)
    pos = (start[:, None] + torch.arange(n, device=dev))[:, None, :, None, None]
    j = torch.arange(L, device=dev)
    hide = j > pos
    if st["window"]:
        hide = hide | (j <= pos - st["window"])
    s = s.masked_fill_(hide, float("-inf"))
    s = (s - s.amax(-1, keepdim=True)).exp_()
    s = s.div_(s.sum(-1, keepdim=True))
    o = torch.bmm(s.view(B * kv, n * g, L), taken(st["vc"], st["vs"]))
    o = o.view(B, kv, n, g, d).permute(0, 2, 1, 3, 4).reshape(B, n, q, d)
    return o[seq, i].to(torch.bfloat16)


# ------------------------------------------------------------------------- 64-bit definitions
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
    f64 = torch.float64
    if op == "norm":
        total = st["res"].to(f64) if st["x"] is None else st["res"].to(f64) + st["x"].to(f64)
        r = total.to(st["res"].dtype).to(f64)  # the norm is that of the residual as it is kept
        y = r / torch.sqrt(torch.einsum("ti,ti->t", r, r)[:, None] / case["dim"] + st["eps"]) * st["w"].to(f64)
        s = _scale64(y.abs().view(y.shape[0], -1, 32).amax(2))
        wide = s.repeat_interleave(32, 1)
        return total, _nearest_e4m3(y / wide), s
    if op == "w4":
        def magnitude(c):  # exponent field 0: halves; otherwise 2^(e-1) times 1 or 1.5
            e, m = ((c >> 1) & 3).to(f64), (c & 1).to(f64)
            return torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2)) * (1 - 2 * (c >> 3).to(f64))
        w = torch.empty(case["N"], case["K"], dtype=f64, device="cuda")
        w[:, 0::2], w[:, 1::2] = magnitude(st["w"] & 15), magnitude(st["w"] >> 4)
        w *= torch.exp2(st["ws"].to(f64) - 127).repeat_interleave(32, 1)
        x = st["x"].to(f64) if st["xs"] is None else st["x"].view(torch.float8_e4m3fn).to(f64) * torch.exp2(st["xs"].to(f64) - 127).repeat_interleave(32, 1)
        return x @ w.t()
    new, old = _lengths(case)
    kv, q, d = case["kv"], case["q"], case["d"]
    g, at = q // kv, 0
    if op == "append":
        x = st["qkv"].to(f64).view(-1, q + 2 * kv, d)
        T, rot = x.shape[0], case["rot"]
        where = torch.cat([torch.arange(p, p + n, device="cuda") for n, p in zip(new, old)])
        turn = torch.polar(torch.ones(T, rot // 2, dtype=f64, device="cuda"), where.to(f64)[:, None] * st["freq"].to(f64)[None])[:, None]
        z = x[:, :q + kv, :rot]
        z = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:].contiguous()) if case["halves"] else torch.view_as_complex(z.reshape(T, q + kv, rot // 2, 2).contiguous())
        z = torch.view_as_real(z * turn)
        x[:, :q + kv, :rot] = torch.cat((z[..., 0], z[..., 1]), -1) if case["halves"] else z.flatten(-2)
        out = [x[:, :q]]
        for codes, scales, h0 in ((st["kc"], st["ks"], q), (st["vc"], st["vs"], q + kv)):
            c, s = codes.view(torch.float8_e4m3fn).to(f64), scales.to(f64)
            first = 0
            for b, (n, p) in enumerate(zip(new, old)):
                for blk in range(p // PAGE, (p + n - 1) // PAGE + 1):
                    pg = int(st["pages"][b, blk])
                    lo, hi = max(p, blk * PAGE), min(p + n, (blk + 1) * PAGE)
                    v = x[first + lo - p:first + hi - p, h0:h0 + kv].transpose(0, 1)  # [kv, tokens, d]
                    sc, a = _scale64(v.abs().amax((1, 2))), lo - blk * PAGE
                    if a:
                        sc = torch.maximum(sc, s[pg])
                        c[pg, :, :a] = _nearest_e4m3(c[pg, :, :a] * (s[pg] / sc)[:, None, None])
                    c[pg, :, a:a + hi - lo] = _nearest_e4m3(v / sc[:, None, None])
                    s[pg] = sc
                first += n
            out += [c, s]
        return tuple(out)
    out = torch.empty(sum(new), q, d, dtype=f64, device="cuda")
    for b, (n, p) in enumerate(zip(new, old)):
        pg = st["pages"][b, :(p + n + PAGE - 1) // PAGE].long()
        i, j = torch.arange(p, p + n, device="cuda"), torch.arange(p + n, device="cuda")
        seen = j[None] <= i[:, None]
        if case["window"]:
            seen &= i[:, None] - j[None] < case["window"]
        for h in range(kv):
            k, v = ((c[pg, h].view(torch.float8_e4m3fn).to(f64) * s[pg, h].to(f64)[:, None, None]).reshape(-1, d)[:p + n] for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
            for u in range(h * g, (h + 1) * g):
                logits = torch.where(seen, st["query"][at:at + n, u].to(f64) @ k.t() * st["scale"], -math.inf)
                out[at:at + n, u] = torch.softmax(logits, 1) @ v
        at += n
    return out


# ---------------------------------------------------------------------------------- one pass
def run(state):
    op = state["op"]
    if not own:
        return {"norm": _norm, "w4": _w4, "append": _append, "attend": _attend}[op](state)
    import gram_hashed_embedding_engram_amd as E
    if op == "norm":
        E.add_norm(state["x"], state["res"], state["w"], state["eps"], state["codes"], state["scales"], d_sum=state["sum"])
        return state["sum"], state["codes"].view(torch.float8_e4m3fn), state["scales"].view(torch.float8_e8m0fnu)
    if op == "w4":
        E.project_w4(state["x"], state["weights"], state["y"], state["xs"])
        return state["y"]
    if op == "append":
        T, q, kv, d = state["T"], state["q"], state["kv"], state["d"]
        qkv = state["qkv"].view(T, q + 2 * kv, d)
        E.cache_append(state["cache"], state["seqs"], qkv[:, q:q + kv], qkv[:, q + kv:], state["freq"], qkv[:, :q], state["qout"], halves=state["halves"])
        return state["qout"], state["kc"].view(torch.float8_e4m3fn), state["ks"], state["vc"].view(torch.float8_e4m3fn), state["vs"]
    E.cache_attend(state["cache"], state["seqs"], state["query"], state["out"], state["scale"], state["window"], d_ws=state["ws"])
    return state["out"]
