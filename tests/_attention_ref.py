"""Plain 64-bit forms of the attention sub-layer's operators and the inputs
of their tests.  Written from the formulas; nothing here calls the library."""
import math

import torch

PAGE = 64
F64 = torch.float64


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32).to(F64)


def scale_of(amax):
    """The least 2^k, k >= -126, with amax <= 448 * 2^k."""
    k = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448)).clamp(min=-126)
    k = torch.where(448 * torch.exp2(k - 1) >= amax, k - 1, k).clamp(min=-126)
    k = torch.where(448 * torch.exp2(k) < amax, k + 1, k)
    return torch.exp2(k)


def near_border(amax, rel):
    """Whether a relative change of `rel` in amax can change its scale."""
    return scale_of(amax * (1 + rel)) != scale_of(amax * (1 - rel))


def e2m1(w):
    """[N, K/2] packed codes -> [N, K] values."""
    c = torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], -1).long()
    mag = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=w.device)
    return mag[c & 7] * torch.where(c >= 8, -1.0, 1.0).to(F64)


def grouped(v, s):
    """v [rows, K] times 2^(s - 127) per 32 values (255: NaN)."""
    f = torch.where(s == 255, torch.full_like(s, 0, dtype=F64) + math.nan, torch.exp2(s.to(F64) - 127))
    return v * f.repeat_interleave(32, 1)


class Step:
    """A cache, its sequences and a step's tokens.  Bytes of the cache that no
    token has written are NaN codes and their pages' scales NaN, so whatever
    reads them shows."""

    def __init__(self, seed, new, old, kv, g, d, qstride=0, width=None, device="cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.new, self.old, self.kv, self.g, self.q, self.d = new, old, kv, g, kv * g, d
        self.B, self.T = len(new), sum(new)
        need = [(o + n + PAGE - 1) // PAGE for o, n in zip(old, new)]
        self.width = width or max(max(need), 1) + 1
        self.n_pages = sum(need) + 2
        perm = torch.randperm(self.n_pages, generator=gen, device=device).int().cpu()
        pages = torch.full((self.B, self.width), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            pages[b, :m] = perm[at:at + m]
            at += m
        self.pages = pages.to(device)
        self.start = torch.tensor(old, dtype=torch.int32, device=device)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        shape = (self.n_pages, kv, PAGE, d)
        self.codes, self.scales = [], []
        for _ in range(2):
            c = torch.full(shape, 0x7F, dtype=torch.uint8, device=device)
            s = torch.full((self.n_pages, kv), math.nan, dtype=torch.float32, device=device)
            for b in range(self.B):
                self._fill(gen, c, s, b, 0, old[b])
            self.codes.append(c)
            self.scales.append(s)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        # the heads side by side in one projection's output, `qstride` values wider
        self.row = (self.q + 2 * kv) * d + qstride
        self.qkv = torch.randn(self.T, self.row, generator=gen, device=device).bfloat16()
        self.gen = gen

    def _fill(self, gen, c, s, b, lo, hi):
        """Positions lo..hi-1 of sequence b get values and their pages scales."""
        for blk in range(lo // PAGE, (hi + PAGE - 1) // PAGE):
            p = int(self.pages[b, blk])
            n = min(hi - blk * PAGE, PAGE)
            v = torch.randn(self.kv, n, self.d, generator=gen, device=c.device)
            v *= torch.exp2(torch.rand(self.kv, 1, 1, generator=gen, device=c.device) * 4 - 2)
            sc = scale_of(v.abs().amax((1, 2)).to(F64)).float()
            c[p, :, :n] = (v / sc[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s[p] = sc

    def fill_new(self):
        """As if the step's tokens had been appended."""
        for c, s in zip(self.codes, self.scales):
            for b in range(self.B):
                o, n = self.old[b], self.new[b]
                if n:
                    first = o // PAGE * PAGE
                    self._fill(self.gen, c, s, b, first, o + n)

    def heads(self):
        x = self.qkv[:, :(self.q + 2 * self.kv) * self.d].view(self.T, self.q + 2 * self.kv, self.d)
        return x[:, :self.q], x[:, self.q:self.q + self.kv], x[:, self.q + self.kv:]

    def objects(self, E, cu=True, err=True):
        cache = E.Cache(self.codes[0], self.codes[1], self.scales[0], self.scales[1])
        seqs = E.Sequences(self.pages, self.start, self.cu if cu else None,
                           self.err if err else None)
        return cache, seqs


def freq_of(rot, device="cuda"):
    return (10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=F64) / rot)).float()


def rotate(x, pos, freq, halves):
    """x [T, heads, d] rotated by its positions, in 64 bits; also |a| + |b| of
    the pair behind each value (what an angle's rounding is multiplied with)."""
    x = x.to(F64)
    rot = 2 * freq.numel()
    out, size = x.clone(), x.abs()
    if rot:
        a = pos.to(F64)[:, None, None] * freq.to(F64)
        c, s = a.cos(), a.sin()
        i = torch.arange(rot // 2, device=x.device)
        u, v = (i, i + rot // 2) if halves else (2 * i, 2 * i + 1)
        p, t = x[..., u], x[..., v]
        out[..., u], out[..., v] = p * c - t * s, p * s + t * c
        size = size.clone()
        size[..., u] = size[..., v] = p.abs() + t.abs()
    return out, size


def attend(step, q, scale, window, causal_bad=()):
    """(out [T, q, d], tolerance) in 64 bits; pages outside the cache masked."""
    kv, g, d = step.kv, step.g, step.d
    out = torch.zeros(step.T, step.q, d, dtype=F64, device=q.device)
    tol = torch.zeros_like(out)
    at = 0
    for b, (n, o) in enumerate(zip(step.new, step.old)):
        if n == 0:
            continue
        L = o + n
        pg = step.pages[b, :(L + PAGE - 1) // PAGE].long()
        ok = (pg >= 0) & (pg < step.n_pages)
        pc = torch.where(ok, pg, torch.zeros_like(pg))
        i, j = torch.arange(o, L, device=q.device), torch.arange(L, device=q.device)
        seen = (j[None] <= i[:, None]) & ok.repeat_interleave(PAGE)[:L][None]
        if window:
            seen &= j[None] > i[:, None] - window
        for h in range(kv):
            k, v = ((e4m3(c[pc, h]) * s[pc, h].to(F64)[:, None, None]).reshape(-1, d)[:L]
                    for c, s in zip(step.codes, step.scales))
            any_seen = seen.any(0)
            k = torch.where(any_seen[:, None], k, torch.zeros_like(k))
            v = torch.where(any_seen[:, None], v, torch.zeros_like(v))
            for u in range(h * g, (h + 1) * g):
                x = q[at:at + n, u].to(F64)
                a = torch.where(seen, x @ k.t() * scale, torch.full((), -math.inf, dtype=F64, device=q.device))
                m = a.amax(1, keepdim=True)
                m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
                p = torch.exp(a - m)
                l = p.sum(1, keepdim=True)
                p = torch.where(l > 0, p / l, torch.zeros_like(p))
                r = p @ v
                out[at:at + n, u] = r
                # logits: f32 sums of d products and a query held to 2^-17 of
                # its largest value; exponents of up to some hundred binary
                # digits in f32: relative error of a probability `delta`
                size = (x.abs() @ k.abs().t()) + x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None]
                big = torch.where(seen, size, torch.zeros_like(size)).amax(1, keepdim=True)
                delta = abs(scale) * big * (d * 2.0 ** -24 + 2.0 ** -17) + 2.0 ** -16
                # probabilities rounded to bf16 (2^-8), sums in f32, out to bf16 (2^-8)
                tol[at:at + n, u] = (2.0 ** -8 * r.abs() + (2.0 ** -8 + 2 * delta + L * 2.0 ** -24) *
                                     (p @ v.abs()) + 1e-30)
        at += n
    return out, tol
