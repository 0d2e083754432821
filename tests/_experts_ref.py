"""Plain 64-bit forms of the experts' operators and the inputs of their tests.
Written from the formulas; nothing here calls the library."""
import math

import numpy as np
import torch

from _attention_ref import e4m3, grouped

F64 = torch.float64
BLOCK = 128


# -------------------------------------------------------------------- routing
def route(logits, bias, k, softmax, groups, top_groups, best, renorm, factor):
    """(ids, weights, offsets, order) of numpy f64 logits [T, E]: a token at a
    time, by a comparison of whole entries."""
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        some = np.isfinite(logits[t])
        if bias is not None:
            some &= np.isfinite(bias)
        some = np.flatnonzero(some)
        if not some.size:
            continue
        x = logits[t, some]
        with np.errstate(over="ignore"):
            if softmax:
                score = np.exp(x - x.max()) / np.exp(x - x.max()).sum()
            else:
                score = 1 / (1 + np.exp(-x))
        liked = score if bias is None else score + bias[some]
        key = x if bias is None else liked
        if groups > 1:
            of = some // (E // groups)
            sums = [(-sum(sorted(liked[of == g].tolist(), reverse=True)[:best]), g) for g in np.unique(of)]
            kept = np.isin(of, [g for _, g in sorted(sums)[:top_groups]])
            some, score, key = some[kept], score[kept], key[kept]
        chosen = sorted(range(some.size), key=lambda i: (-key[i], some[i]))[:k]
        got = score[chosen]
        total = got.sum()
        ids[t, :len(chosen)] = some[chosen]
        weights[t, :len(chosen)] = factor * ((got / total if total > 0 else 0 * got) if renorm else got)
    return ids, weights, *plan(ids, E)


def plan(ids, E):
    """offsets [E + 1] and the slots in their order."""
    flat = ids.reshape(-1)
    slots = np.flatnonzero(flat >= 0)
    order = slots[np.argsort(flat[slots], kind="stable")]
    counts = np.bincount(flat[slots], minlength=E)
    return np.concatenate(([0], counts.cumsum())), order


# ------------------------------------------------------------------- products
def weights8(g, *shape, spread=2.0):
    """e4m3 codes [..., N, K] and block scales of different sizes and signs."""
    N, K = shape[-2:]
    w = (torch.randn(*shape, generator=g, device="cuda") * 60).clamp_(-448, 448).to(torch.float8_e4m3fn)
    blocks = (*shape[:-2], -(-N // BLOCK), -(-K // BLOCK))
    s = torch.exp2((torch.rand(*blocks, generator=g, device="cuda") * 2 - 1) * spread) / (60 * math.sqrt(K))
    s *= torch.where(torch.rand(*blocks, generator=g, device="cuda") < 0.2, -1.0, 1.0)
    return w.view(torch.uint8), s


def rows8(g, rows, K, f32):
    """e4m3 rows with scales of either kind, and their values in 64 bits."""
    x = (torch.randn(rows, K, generator=g, device="cuda") * 60).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if f32:
        s = torch.exp2(torch.rand(rows, K // BLOCK, generator=g, device="cuda") * 3 - 1) / 60
        return x, s, e4m3(x) * s.to(F64).repeat_interleave(BLOCK, 1)
    s = torch.randint(119, 124, (rows, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    return x, s, grouped(e4m3(x), s)


def matrix(w, s):
    N, K = w.shape
    return e4m3(w) * s.to(F64).repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def product(x, w):
    """(x w^T, how far f32 sums of it may be off).  The matrix instruction cuts
    the products of eight neighbours below 2^-13 of the largest: at most 7 * 2^-13
    of it, so of the root of their squares' sum; the products' signs are
    independent, so such errors add like a random walk, and six times the root of
    their squares' sum is not passed but once in e^18 outputs.  Everything is then
    added in f32, K / 8 terms and the blocks' factors."""
    K = x.shape[1]
    walk = 6 * 7 * 2.0 ** -13 * ((x * x) @ (w * w).t()).sqrt()
    return x @ w.t(), walk + (K / 8 + 8) * 2.0 ** -24 * (x.abs() @ w.abs().t())


def up(x, w, s, offsets, order, k):
    """(h, its tolerance before the 8-bit rounding) in the plan's order."""
    R, I = len(order), w.shape[2]
    h = torch.zeros(R, I, dtype=F64, device=x.device)
    tol = torch.zeros_like(h)
    for e in range(w.shape[0]):
        p, q = int(offsets[e]), int(offsets[e + 1])
        if q > p:
            mine = x[torch.as_tensor(order[p:q], device=x.device) // k]
            (g, dg), (u, du) = (product(mine, matrix(w[e, i], s[e, i])) for i in range(2))
            silu = g * torch.sigmoid(g)
            h[p:q] = silu * u
            # |silu'| < 1.1; e^-g by an ulp or two, a quotient and a product
            tol[p:q] = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -21 * h[p:q].abs()
    return h, tol


def down(h, w, s, offsets, order, weights):
    """(y, its tolerance before the bf16 rounding)."""
    T, k = weights.shape
    y = torch.zeros(T, w.shape[1], dtype=F64, device=h.device)
    tol = torch.zeros_like(y)
    flat = weights.reshape(-1).to(F64)
    for e in range(w.shape[0]):
        p, q = int(offsets[e]), int(offsets[e + 1])
        if q > p:
            slot = torch.as_tensor(order[p:q], device=h.device)
            v, d = product(h[p:q], matrix(w[e], s[e]))
            y.index_add_(0, slot // k, v * flat[slot][:, None])
            # a product as f16 under a shared power of two (2^-11 of itself, or 2^-39 of
            # its row's largest), times its weight and added to k, each rounded in f32
            f16 = 2.0 ** -11 * v.abs() + 2.0 ** -39 * v.abs().amax(1, keepdim=True)
            tol.index_add_(0, slot // k, ((1 + 2.0 ** -11) * d + f16 + (k + 1) * 2.0 ** -24 * v.abs()) * flat[slot].abs()[:, None])
    return y, tol
