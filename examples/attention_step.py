"""A prompt and single-token steps through engram layers with their attention sub-layer.

    python examples/attention_step.py

Each layer gates its engram onto the FP32 highway, then runs the attention sub-layer on it:
norm with 8-bit output, 4-bit projection to queries, keys and values, rotation and append to the
paged 8-bit cache, attention over the cache, 4-bit output projection, and the residual's addition
with the norm that the next sub-layer takes.  Synthetic weights; one highway stream.
"""
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gram_hashed_embedding_engram_amd as E  # noqa: E402
import synth  # noqa: E402
from synth import generate as G  # noqa: E402

KV_HEADS, Q_HEADS, HEAD_DIM = 2, 8, 64
WINDOW = 0


def random_w4(gen, N, K):
    """[N, K] in 4 bits whose products keep the size of what they are fed."""
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8)
    exponent = 127 - round(math.log2(3 * math.sqrt(K)))     # e2m1 values are about 3 in size
    scales = torch.full((N, K // E.NORM_GROUP), exponent, dtype=torch.uint8)
    return E.W4(codes.cuda(), scales.cuda())


class Attention:
    """One layer's weights, cache and buffers for calls of up to max_tokens."""

    def __init__(self, gen, dim, eps, max_tokens, n_pages):
        bf16, u8 = torch.bfloat16, torch.uint8
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        self.eps = eps
        self.norms = [(1 + 0.1 * torch.randn(dim, generator=gen)).to(bf16).cuda() for _ in range(2)]
        self.qkv_w = random_w4(gen, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM, dim)
        self.out_w = random_w4(gen, dim, Q_HEADS * HEAD_DIM)
        shape = (n_pages, KV_HEADS, E.PAGE_TOKENS, HEAD_DIM)
        self.cache = E.Cache(new(*shape, dtype=u8), new(*shape, dtype=u8),
                             new(*shape[:2], dtype=torch.float32), new(*shape[:2], dtype=torch.float32))
        self.freq = (10000.0 ** (-torch.arange(0, HEAD_DIM, 2, dtype=torch.float64) / HEAD_DIM)).float().cuda()
        self.codes = new(max_tokens, dim, dtype=u8)
        self.scales = new(max_tokens, dim // E.NORM_GROUP, dtype=u8)
        self.qkv = new(max_tokens, Q_HEADS + 2 * KV_HEADS, HEAD_DIM, dtype=bf16)
        self.q = new(max_tokens, Q_HEADS, HEAD_DIM, dtype=bf16)
        self.o = new(max_tokens, Q_HEADS, HEAD_DIM, dtype=bf16)
        self.y = new(max_tokens, dim, dtype=bf16)

    def __call__(self, seqs, h, ws):
        """h [T, dim] f32, in place; returns the next sub-layer's 8-bit input and its scales."""
        T = h.shape[0]
        codes, scales, qkv, q, o, y = (t[:T] for t in (self.codes, self.scales, self.qkv, self.q, self.o, self.y))
        E.add_norm(None, h, self.norms[0], self.eps, codes, scales)
        E.project_w4(codes, self.qkv_w, qkv.view(T, -1), scales)
        E.cache_append(self.cache, seqs, qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:],
                       self.freq, qkv[:, :Q_HEADS], q)
        E.cache_attend(self.cache, seqs, q, o, 1 / math.sqrt(HEAD_DIM), WINDOW, ws)
        E.project_w4(o.view(T, -1), self.out_w, y)
        E.add_norm(y, h, self.norms[1], self.eps, codes, scales)
        return codes, scales


def run(w=synth.HC1_Q2K, steps=None, seed=0):
    """Highway rows [tokens, dim] after the last layer: the prompt's, then one a step."""
    gen = torch.Generator().manual_seed(seed)
    dev = torch.device("cuda")
    steps = w.decode_steps if steps is None else steps
    tokens = w.prompt + steps
    ht = G.hash_tables(w)
    tables = E.HashTables(torch.from_numpy(ht["token_map"]).to(dev), ht["pad_id"], ht["multipliers"],
                          ht["primes"], ht["offsets"])
    ctx = E.Context(tables, w.hc, w.dim, w.head_dim, w.eps, w.prompt, tokens)
    keep, layers = [], []
    max_pages = (tokens + E.PAGE_TOKENS - 1) // E.PAGE_TOKENS
    for i in range(w.n_layers):
        L = G.layer_inputs(w, ht, i)
        scales = L.get("scales")
        table = E.Table(torch.from_numpy(L["table"]).to(dev),
                        None if scales is None else torch.from_numpy(scales).to(dev),
                        head_dim=w.head_dim, scale_block=w.scale_block)
        qk = torch.empty(w.hc, w.dim, dtype=torch.float32, device=dev)
        E.qk_product(torch.from_numpy(L["q"].view(np.int16)).to(dev),
                     torch.from_numpy(L["k"].view(np.int16)).to(dev), qk)
        wkv = torch.from_numpy(L["wkv"].view(np.int16)).to(dev)
        ctx.add_layer(i, table, wkv, qk)
        keep.append((table, wkv, qk))
        layers.append(Attention(gen, w.dim, w.eps, w.prompt, max_pages))
    ctx.reset()
    # one sequence, whose pages lie in any order
    pages = torch.randperm(max_pages, generator=gen).int().view(1, -1).to(dev)
    start = torch.zeros(1, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    seqs = E.Sequences(pages, start, d_err=err)
    need = max(E.cache_attend_bytes(layers[0].cache, seqs, Q_HEADS, T) for T in (w.prompt, 1))
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    ids = torch.from_numpy(G.token_ids(w).astype(np.int32)).to(dev)
    rows = torch.from_numpy(G.highway(w, tokens)).to(dev).view(tokens, w.dim)
    at = 0
    while at < tokens:
        T = w.prompt if at == 0 else 1
        h = rows[at:at + T]
        for i, layer in enumerate(layers):
            ctx.forward(i, ids[at:at + T], T, h)
            layer(seqs, h, ws)
        start += T                              # on the stream, like the step itself
        at += T
    ctx.check()
    if int(err):
        raise RuntimeError(f"sequence or page errors: {int(err)}")
    return rows


if __name__ == "__main__":
    out = run()
    print(f"{out.shape[0]} tokens of {out.shape[1]} values, root mean square "
          f"{float(out.square().mean().sqrt()):.4f}")
