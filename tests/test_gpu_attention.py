"""The attention sub-layer's operators on the GPU against their 64-bit forms
(tests/_attention_ref.py).  Tolerances count roundings: half a step of the
result's type (bf16 2^-8, e4m3 2^-4 relative), f32 sums of n terms n * 2^-24 of
the sum of their magnitudes."""
import math

import pytest

torch = pytest.importorskip("torch")

import _attention_ref as R  # noqa: E402
from _gpu_util import log  # noqa: E402

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def E():
    import gram_hashed_embedding_engram_amd as E
    E.lib()
    return E


def seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def within(got, want, tol, what):
    got, want = got.to(F64), want.to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    same = torch.isnan(want) | (torch.isinf(want) & (got == want))
    off = torch.where(same, torch.zeros_like(want), (got - want).abs() - tol)
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} past the tolerance at {int(off.argmax())}"


# ------------------------------------------------------------------- norm
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("rows,dim", [(1, 32), (3, 64), (1, 4096), (5, 96), (64, 1056), (7, 7200),
                                      (300, 512), (2, 65536), (2, 16416), (9, 10240)])
def test_add_norm(E, rows, dim, add, bf16):
    log(f"add_norm {rows} x {dim} add {add} bf16 {bf16}")
    g = seeded(rows * 7 + dim)
    t = torch.bfloat16 if bf16 else torch.float32
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    res = (rn(rows, dim) * torch.exp2(rn(rows, 1) * 4)).to(t)
    x = (rn(rows, dim) * 0.3).bfloat16() if add else None
    w = (1 + 0.3 * rn(dim)).bfloat16()
    if rows > 2:
        res[1] = 0                                     # scales at their floor
        if x is not None:
            x[1] = 0
        res[2, dim // 2] = math.inf if rows % 2 else math.nan
        w[:32] = 0                                     # a group of zeros
    codes = torch.zeros(rows, dim, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, dim // 32, dtype=torch.uint8, device="cuda")
    total = torch.empty_like(res) if rows % 2 else None
    keep = res.clone()
    E.add_norm(x, res, w, 1e-6, codes, scales, d_sum=total)
    torch.cuda.synchronize()
    s = res if total is None else total
    if total is not None:
        assert torch.equal(res.nan_to_num(), keep.nan_to_num())
    want_s = (keep.float() + (x.float() if add else 0)).to(t)      # one rounding: the same bits
    assert torch.equal(s.nan_to_num(), want_s.nan_to_num())
    r = want_s.to(F64)
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6) * w.to(F64)
    # sum of squares: a thread's chain and a tree of ten; then root, quotient, products
    rel = (dim / 256 + 32) * 2.0 ** -24
    got_s = torch.exp2(scales.to(F64) - 127)
    # NaN (a NaN in the row, or an infinity over the infinite norm) is outside a scale
    amax = y.nan_to_num().abs().view(rows, -1, 32).amax(2)
    ok = (got_s == R.scale_of(amax)) | R.near_border(amax, 2 * rel)
    assert bool(ok.all())
    wide = got_s.repeat_interleave(32, 1)
    tol = y.abs() * (2.0 ** -4 * (1 + 2 * rel) + rel) + 2.0 ** -10 * wide
    within(R.e4m3(codes) * wide, y, tol, "codes")


@pytest.mark.parametrize("bf16", [False, True])
def test_add_norm_without_eps(E, bf16):
    """eps = 0: rows whose squares f32 holds are normed whatever their size;
    where all vanish in f32 the norm is nothing to divide by."""
    t = torch.bfloat16 if bf16 else torch.float32
    size = torch.tensor([1.0, 2.0 ** -60, 2.0 ** 50, 2.0 ** -90, 0.0], device="cuda")
    res = (torch.randn(5, 96, generator=seeded(33), device="cuda") * size[:, None]).to(t)
    w = torch.ones(96, dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros(5, 96, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(5, 3, dtype=torch.uint8, device="cuda")
    E.add_norm(None, res, w, 0.0, codes, scales)
    got = R.grouped(R.e4m3(codes), scales)
    assert bool(torch.isnan(got[3:]).all())
    r = res[:3].to(F64)
    y = r / (r * r).mean(1, keepdim=True).sqrt()
    # squares of 2^-120 and their sum keep 24 bits in f32
    wide = torch.exp2(scales[:3].to(F64) - 127).repeat_interleave(32, 1)
    within(got[:3], y, y.abs() * (2.0 ** -4 + 2.0 ** -18) + 2.0 ** -10 * wide, "codes")


# --------------------------------------------------------------------- w4
def w4_case(seed, T, K, N, fp8, lo=110, hi=130):
    g = seeded(seed)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(lo, hi, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(T, K, generator=g, device="cuda")
    if fp8:
        codes = (x * 100).to(torch.float8_e4m3fn).view(torch.uint8)
        xs = torch.randint(lo, hi, (T, K // 32), generator=g, device="cuda", dtype=torch.uint8)
        return w, ws, codes, xs, R.grouped(R.e4m3(codes), xs)
    return w, ws, x.bfloat16(), None, x.bfloat16().to(F64)


def check_w4(E, w, ws, x, xs, x64):
    T, K, N = x.shape[0], x.shape[1], w.shape[0]
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    E.project_w4(x, E.W4(w, ws), y, xs)
    torch.cuda.synchronize()
    w64 = R.grouped(R.e2m1(w), ws)
    if xs is None:                       # a weight past f32's range is infinite
        w64 = w64.float().to(F64)
    want = x64 @ w64.t()
    tol = 2.0 ** -8 * want.abs() + K * 2.0 ** -24 * (x64.abs() @ w64.abs().t()) + 1e-38
    within(y, want, tol, "y")
    return y


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (1, 4096, 6144), (2, 512, 48), (5, 640, 1040),
                                   (16, 2048, 256), (17, 896, 272), (33, 1152, 4112), (48, 384, 16),
                                   (64, 6144, 512), (65, 256, 64), (130, 768, 80), (200, 1024, 1296),
                                   (1, 16384, 32)])
def test_project_w4(E, T, K, N, fp8):
    log(f"project_w4 T {T} K {K} N {N} fp8 {fp8}")
    check_w4(E, *w4_case(T + K + N, T, K, N, fp8))


@pytest.mark.parametrize("fp8", [True, False])
def test_project_w4_single_products(E, fp8):
    """One non-zero value a token: every code, every scale byte at both ends of
    its range, each k in its own place."""
    K, N, T = 256, 16, 64
    g = seeded(3)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(64, 191, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    for first in range(0, K, T):
        x = torch.zeros(T, K, device="cuda")
        x[torch.arange(T), first + torch.arange(T)] = 1.0
        if fp8:
            codes = x.to(torch.float8_e4m3fn).view(torch.uint8)
            xs = torch.full((T, K // 32), 127, device="cuda", dtype=torch.uint8)
            y = check_w4(E, w, ws, codes, xs, x.to(F64))
        else:
            y = check_w4(E, w, ws, x.bfloat16(), None, x.to(F64))
        want = R.grouped(R.e2m1(w), ws)[:, first:first + T].t()
        assert torch.equal(y.to(F64), want)           # a power of two times a code: exact


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("lo,hi", [(1, 5), (245, 255)])
def test_project_w4_far_scales(E, fp8, lo, hi):
    """Scale bytes at both ends, against activations at the other."""
    w, ws, x, xs, x64 = w4_case(9, 3, 256, 32, fp8, lo, hi)
    if fp8:
        xs = (254 - (ws[:3] if xs is None else xs).int()).to(torch.uint8)
        x64 = R.grouped(R.e4m3(x), xs)
    else:
        x = (x.float() * (2.0 ** 120 if lo == 1 else 2.0 ** -120)).bfloat16()
        x64 = x.to(F64)
    check_w4(E, w, ws, x, xs, x64)


@pytest.mark.parametrize("fp8", [True, False])
def test_project_w4_nan(E, fp8):
    """A NaN scale or value reaches its own outputs and no others."""
    w, ws, x, xs, x64 = w4_case(11, 20, 512, 64, fp8)
    ws[5, 3] = 255
    if fp8:
        xs[7, 2] = 255
        x[9, 100] = 0x7F
        x64 = R.grouped(R.e4m3(x), xs)
    else:
        x[7, 64] = math.nan
        x[9, 100] = math.nan
        x64 = x.to(F64)
    y = torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda")
    E.project_w4(x, E.W4(w, ws), y, xs)
    bad = torch.zeros(20, 64, dtype=torch.bool, device="cuda")
    bad[:, 5] = True
    bad[7] = bad[9] = True
    assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("T,K,N", [(3, 128, 16), (20, 640, 64), (40, 1152, 80), (60, 4096, 1296)])
def test_project_w4_infinite(E, T, K, N):
    """An infinite value meets its own weights only, wherever in K it stands:
    infinities of the weights' signs, NaN over zero weights."""
    w, ws, x, xs, _ = w4_case(13 + K, T, K, N, False)
    for t, at in ((0, K - 1), (1, K // 2), (2, 0)):
        x[t, at] = math.inf
    x[T - 1, K - 128] = -math.inf
    check_w4(E, w, ws, x, xs, x.to(F64))


def cut_products(x, w):
    """Sums over k of products x[t][k] w[n][k] as the scaled 8-bit instruction
    forms them: the products of eight neighbours are cut towards zero below
    2^-13 of the largest one's power of two (the operands' exponents added;
    zeros have none), then everything is added in f32 (here exactly)."""
    T, K, N = x.shape[0], x.shape[1], w.shape[0]
    low = torch.full((), -1000.0, dtype=F64, device=x.device)
    ex = torch.where(x == 0, low, x.abs().clamp(min=2.0 ** -6).log2().floor())
    ew = torch.where(w == 0, low, w.abs().clamp(min=1.0).log2().floor())
    p = (x[:, None, :] * w[None]).view(T, N, K // 8, 8)
    top = (ex[:, None, :] + ew[None]).view(T, N, K // 8, 8).amax(-1, keepdim=True)
    unit = torch.exp2(top.clamp(min=-100) - 13)
    return (torch.trunc(p / unit) * unit).sum((-1, -2)), p.abs().sum((-1, -2))


@pytest.mark.parametrize("spread", [0, 8, 14])
@pytest.mark.parametrize("fp8", [True, False])
def test_project_w4_sums(E, fp8, spread):
    """What a sum keeps beside large values that cancel: with bf16 activations
    what f32 keeps, with 8-bit ones what the instruction does."""
    T, K, N = 32, 128, 256
    g = seeded(spread + 17)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    w[:, 0::4] = 0xF7                                   # 6 and -6 for the first two of every eight
    ws = torch.full((N, K // 32), 127, device="cuda", dtype=torch.uint8)
    x = torch.randn(T, K, generator=g, device="cuda")
    x *= torch.exp2(torch.rand(T, K, generator=g, device="cuda") * spread - spread + 6)
    x = x.clamp(-448, 448)
    x[:, 0::8] = x[:, 1::8] = 448
    x = x.to(torch.float8_e4m3fn)
    w64, x64 = R.e2m1(w), x.float().to(F64)
    cut, size = cut_products(x64, w64)
    exact = x64 @ w64.t()
    assert bool(((cut - exact).abs() <= K / 8 * 7 * 2.0 ** -13 * 448 * 6).all())
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    if fp8:
        E.project_w4(x.view(torch.uint8), E.W4(w, ws), y, torch.full((T, K // 32), 127, device="cuda", dtype=torch.uint8))
    else:
        E.project_w4(x.to(torch.bfloat16), E.W4(w, ws), y)
    want = cut if fp8 else exact
    within(y, want, 2.0 ** -8 * want.abs() + K * 2.0 ** -24 * size, "y")


# ----------------------------------------------------------------- append
STEPS = [  # new tokens, older positions, kv heads, queries a key head, head_dim
    ([1], [0], 1, 1, 64), ([1], [63], 2, 4, 128), ([1], [64], 2, 3, 64), ([1, 1, 1], [5, 127, 300], 4, 8, 256),
    ([3, 0, 70], [62, 10, 0], 2, 4, 128), ([130, 1, 64, 0], [1, 200, 64, 7], 1, 6, 64),
    ([257], [40], 2, 1, 256), ([2] * 70, [3 * i for i in range(70)], 1, 2, 64),
    ([0, 5], [0, 60], 3, 1, 128)]


def check_append(E, st, freq, halves, cu=True, with_q=True):
    q, k, v = st.heads()
    out = torch.full((st.T, st.q, st.d), 9.0, dtype=torch.bfloat16, device="cuda") if with_q else None
    old_c = [c.clone() for c in st.codes]
    old_s = [s.clone() for s in st.scales]
    cache, seqs = st.objects(E, cu=cu)
    E.cache_append(cache, seqs, k, v, freq, q if with_q else None, out, halves=halves)
    torch.cuda.synchronize()
    assert int(st.err) == 0
    f = freq if freq is not None else torch.zeros(0, device="cuda")
    pos = torch.cat([torch.arange(o, o + n, device="cuda") for n, o in zip(st.new, st.old)])
    # an angle is formed in 64 bits, its cosine and sine are f32 of 2^-22, two products and a sum
    if with_q:
        want, size = R.rotate(q, pos, f, halves)
        within(out, want, 2.0 ** -8 * want.abs() + 2.0 ** -21 * size, "q")
    kr, ksize = R.rotate(k, pos, f, halves)
    touched = torch.zeros(st.n_pages, dtype=torch.bool, device="cuda")
    for which, (vals, size) in enumerate(((kr, ksize), (v.to(F64), None))):
        c, s = st.codes[which], st.scales[which]
        rel = 2.0 ** -20 if which == 0 and f.numel() else 0.0
        first = 0
        for b, (n, o) in enumerate(zip(st.new, st.old)):
            for blk in range(o // 64, (o + n + 63) // 64 if n else 0):
                pg = int(st.pages[b, blk])
                touched[pg] = True
                lo, hi = max(o, blk * 64), min(o + n, blk * 64 + 64)
                x = vals[first + lo - o:first + hi - o].transpose(0, 1)
                a = lo - blk * 64
                amax = x.abs().amax((1, 2))
                need = R.scale_of(amax)
                had = old_s[which][pg].to(F64) if a else torch.zeros_like(need)
                now = s[pg].to(F64)
                ok = now == torch.maximum(need, had)
                if rel:
                    ok |= R.near_border(amax, rel) & (now >= had)
                assert bool(ok.all()), f"scales of page {pg}"
                got = R.e4m3(c[pg, :, a:a + hi - lo]) * now[:, None, None]
                if which:                       # values: the exact nearest code
                    exact = (x / now[:, None, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
                    assert torch.equal(c[pg, :, a:a + hi - lo], exact)
                tol = 2.0 ** -4 * x.abs() + 2.0 ** -10 * now[:, None, None]
                if rel:
                    tol = tol + 2.0 ** -20 * size[first + lo - o:first + hi - o].transpose(0, 1)
                within(got, x, tol, f"codes of page {pg}")
                if a:                           # older codes: rounded once more where the scale rose
                    ratio = (had / now).float()
                    exact = (R.e4m3(old_c[which][pg, :, :a]).float() * ratio[:, None, None]) \
                        .to(torch.float8_e4m3fn).view(torch.uint8)
                    assert torch.equal(c[pg, :, :a], exact)
                if a + hi - lo < 64:
                    assert torch.equal(c[pg, :, a + hi - lo:], old_c[which][pg, :, a + hi - lo:])
            first += n
        assert torch.equal(c[~touched], old_c[which][~touched])
        assert torch.equal(s[~touched].nan_to_num(), old_s[which][~touched].nan_to_num())


@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("part", [0, 1, 2])
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_append(E, case, part, halves):
    new, old, kv, g, d = STEPS[case]
    log(f"append {new[:6]} after {old[:6]} kv {kv} g {g} d {d} part {part} halves {halves}")
    st = R.Step(case * 10 + part, new, old, kv, g, d, qstride=8 * (case % 3))
    if case % 2:
        st.qkv *= 30                                   # scales rise
    freq = None if part == 0 else R.freq_of(d // part)
    check_append(E, st, freq, halves, with_q=case != 2)


def test_append_uniform(E):
    """No token bounds: each sequence brings as many."""
    for n in (1, 5, 64):
        st = R.Step(n, [n] * 3, [7, 64, 130], 2, 4, 128)
        check_append(E, st, R.freq_of(128), True, cu=False)


def test_append_far_positions(E):
    """Angles of far positions: the position times the frequency in 64 bits."""
    st = R.Step(5, [3, 2], [1000001, 131070], 1, 2, 64)
    check_append(E, st, R.freq_of(64), True)


def test_append_repeats(E):
    """The same step again finds its own scales: the same bytes."""
    st = R.Step(6, [3, 70], [62, 1], 2, 4, 128)
    check_append(E, st, R.freq_of(128), True)
    c = [x.clone() for x in st.codes + st.scales]
    q, k, v = st.heads()
    cache, seqs = st.objects(E)
    E.cache_append(cache, seqs, k, v, R.freq_of(128), halves=True)
    for x, y in zip(c, st.codes + st.scales):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())


def test_append_not_finite(E):
    """A NaN or an infinity becomes a NaN code; the scale covers the rest."""
    st = R.Step(7, [4], [62], 1, 1, 64)
    q, k, v = st.heads()
    v[1, 0, 5] = math.inf
    v[2, 0, 6] = math.nan
    v[3] = 0
    old = [s.clone() for s in st.scales]
    cache, seqs = st.objects(E)
    E.cache_append(cache, seqs, k, v, None)
    p0, p1 = int(st.pages[0, 0]), int(st.pages[0, 1])
    got = R.e4m3(st.codes[1])
    assert bool(torch.isnan(got[p0, 0, 63, 5])) and bool(torch.isnan(got[p1, 0, 0, 6]))
    nan = torch.isnan(got[p1, 0, :2])
    assert int(nan.sum()) == 1
    need = torch.maximum(R.scale_of(v[0].abs().amax().to(F64)),
                         R.scale_of(v[1, 0][torch.isfinite(v[1, 0])].abs().amax().to(F64)))
    assert float(st.scales[1][p0, 0]) == max(float(need), float(old[1][p0, 0]))
    # a page of zeros takes the lowest scale
    st = R.Step(8, [2], [0], 1, 1, 64)
    st.qkv.zero_()
    cache, seqs = st.objects(E)
    q, k, v = st.heads()
    E.cache_append(cache, seqs, k, v, R.freq_of(64))
    assert float(st.scales[0][int(st.pages[0, 0]), 0]) == 2.0 ** -126


def bad_steps():
    """(what, its error bit, whether tokens of sequence 0 stay out)."""
    return [("start", 16), ("width", 16), ("cu_falls", 16), ("cu_past", 16), ("page_high", 8),
            ("page_low", 8)]


def spoil(st, what):
    if what == "start":
        st.start[0] = -1
    elif what == "width":
        st.start[0] = st.width * 64 - st.new[0] + 1
    elif what == "cu_falls":
        st.cu[1] = -2
    elif what == "cu_past":
        st.cu[-1] = st.T + 5
    elif what == "page_high":
        st.pages[0, st.old[0] // 64] = st.n_pages
    else:
        st.pages[0, st.old[0] // 64] = -7


@pytest.mark.parametrize("what,bit", bad_steps())
def test_append_bad_sequences(E, what, bit):
    """Bad bounds and pages set their bit and write nothing of theirs; the
    other sequences are appended as ever."""
    good, st = (R.Step(9, [3, 2, 4], [30, 62, 0], 2, 2, 64) for _ in range(2))
    spoil(st, what)
    before = [x.clone() for x in st.codes + st.scales]
    for s in (good, st):
        q, k, v = s.heads()
        cache, seqs = s.objects(E)
        E.cache_append(cache, seqs, k, v, R.freq_of(64))
    torch.cuda.synchronize()
    assert int(st.err) == bit and int(good.err) == 0
    whole = {0: [what not in ("start", "width", "cu_falls", "page_high", "page_low")],
             1: [what != "cu_falls"], 2: [what != "cu_past"]}
    for b in range(3):
        for blk in range((st.old[b] + st.new[b] + 63) // 64):
            pg = int(good.pages[b, blk])
            for x, y, z in zip(st.codes + st.scales, good.codes + good.scales, before):
                want = y if whole[b][0] else z
                assert torch.equal(x[pg].nan_to_num(), want[pg].nan_to_num()), (b, blk)


# ----------------------------------------------------------------- attend
def check_attend(E, st, window=0, scale=None, cu=True, q=None, bits=0):
    scale = scale or 1 / math.sqrt(st.d)
    q = st.heads()[0] if q is None else q
    out = torch.full((st.T, st.q, st.d), 9.0, dtype=torch.bfloat16, device="cuda")
    cache, seqs = st.objects(E, cu=cu)
    ws = torch.full((E.cache_attend_bytes(cache, seqs, st.q, st.T),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    E.cache_attend(cache, seqs, q, out, scale, window, ws)
    torch.cuda.synchronize()
    assert int(st.err) == bits
    want, tol = R.attend(st, q, scale, window)
    within(out, want, tol, "out")
    again = torch.empty_like(out)
    E.cache_attend(cache, seqs, q, again, scale, window, ws)
    assert torch.equal(out, again)                      # no order of arrival in the results
    return out


@pytest.mark.parametrize("window", [0, 1, 7, 64, 100])
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_attend(E, case, window):
    new, old, kv, g, d = STEPS[case]
    log(f"attend {new[:6]} after {old[:6]} kv {kv} g {g} d {d} window {window}")
    st = R.Step(100 + case, new, old, kv, g, d, qstride=8 * (case % 3))
    st.fill_new()
    check_attend(E, st, window)


@pytest.mark.parametrize("new,old,kv,g,d,window", [
    ([1], [5000], 2, 4, 128, 0), ([1], [131071], 1, 3, 64, 0), ([1], [40000], 2, 8, 256, 0),
    ([1] * 9, [4096 + 511 * i for i in range(9)], 4, 4, 128, 0), ([4], [9000], 1, 4, 128, 0),
    ([4, 1], [9000, 3], 2, 8, 64, 500), ([1], [20000], 1, 32, 128, 0), ([1, 1], [30000, 5], 1, 1, 256, 1000),
    ([3], [6000], 2, 5, 64, 0), ([17], [3000], 1, 20, 128, 0)])
def test_attend_long(E, new, old, kv, g, d, window):
    log(f"attend long {new} after {old} kv {kv} g {g} d {d} window {window}")
    st = R.Step(sum(old), new, old, kv, g, d)
    st.fill_new()
    check_attend(E, st, window)


@pytest.mark.parametrize("new,old,kv,g,d,window", [
    # units of even pieces, over more sequences than a wavefront's lanes
    ([1] * 70, [1030 + 29 * (i % 7) for i in range(70)], 2, 4, 64, 0),
    ([0, 1] * 50, [40 * i for i in range(100)], 1, 2, 64, 0),
    ([1] * 66, [20000 if i in (3, 65) else 3 * i for i in range(66)], 2, 4, 128, 0),
    # more units than workgroups; one long sequence among many short ones
    ([1] * 150, [1100 + (i % 3) for i in range(150)], 4, 1, 64, 0),
    ([1] * 40, [60000] + [70] * 39, 8, 2, 128, 0), ([1] * 90, [1500 + i for i in range(90)], 4, 2, 256, 300),
    # units that end one page past, on and before a piece
    ([1, 1, 1], [64 * 32, 64 * 32 - 1, 64 * 31 - 1], 1, 4, 256, 0), ([2, 1], [1020, 63], 3, 8, 256, 0)])
def test_attend_shares(E, new, old, kv, g, d, window):
    log(f"attend shares {len(new)} sequences, longest {max(old)}, kv {kv} g {g} d {d} window {window}")
    st = R.Step(len(new) + d, new, old, kv, g, d)
    st.fill_new()
    check_attend(E, st, window)


def empty_run(B, lo, hi, past):
    """One token for each of B sequences, none for sequences lo .. hi-1."""
    return ([0 if lo <= i < hi else 1 for i in range(B)],
            [70 if lo <= i < hi else past + 5 * (i % 9) for i in range(B)])


@pytest.mark.parametrize("B,lo,hi,past,kv,g,d", [
    (140, 40, 64, 1100, 8, 1, 64), (140, 40, 65, 1100, 8, 4, 128), (140, 63, 66, 1100, 8, 2, 64),
    (140, 10, 64, 1100, 4, 1, 256), (230, 50, 130, 1100, 8, 2, 64), (260, 30, 200, 1100, 8, 1, 128),
    (300, 1, 299, 40000, 2, 4, 64), (200, 64, 128, 1090, 4, 2, 256)])
def test_attend_shares_over_empty_sequences(E, B, lo, hi, past, kv, g, d):
    """Workgroups whose share walks on over runs of sequences without tokens,
    inside and across groups of 64 sequences."""
    log(f"attend over empty sequences {lo}..{hi} of {B}, kv {kv} g {g} d {d}")
    new, old = empty_run(B, lo, hi, past)
    st = R.Step(B + lo, new, old, kv, g, d)
    st.fill_new()
    check_attend(E, st)


@pytest.mark.parametrize("new,old,kv,g,d,window", [
    ([300], [100], 2, 4, 128, 0), ([513, 60, 0, 129], [0, 700, 5, 63], 1, 4, 64, 0),
    ([200, 33], [77, 1000], 2, 3, 256, 0), ([400], [900], 1, 8, 128, 150), ([350, 90], [64, 300], 2, 1, 128, 0),
    ([150], [0], 8, 8, 64, 40), ([100], [1030], 1, 20, 128, 0), ([130], [70], 1, 6, 256, 1),
    ([1100], [33], 2, 4, 128, 0), ([700, 300], [77, 200], 4, 3, 256, 0), ([600], [64], 4, 8, 64, 90),
    ([700], [300], 4, 4, 256, 64), ([800, 3], [5, 90], 4, 6, 64, 0), ([600], [130], 8, 3, 128, 33),
    ([90] * 5, [11 * i for i in range(5)], 2, 4, 128, 0),
    # tiles whose pages are shared out: long caches, short ones among them, windows
    ([300], [3000], 8, 2, 128, 0), ([520, 64], [2500, 3], 4, 4, 64, 700), ([200, 129, 0], [2000, 1, 9], 8, 3, 256, 0),
    ([257], [6000], 8, 4, 128, 100), ([150], [1200], 8, 8, 256, 0), ([1, 600], [4000, 2100], 4, 4, 64, 0)])
def test_attend_prompt(E, new, old, kv, g, d, window):
    log(f"attend prompt {new} after {old} kv {kv} g {g} d {d} window {window}")
    st = R.Step(sum(old) + 1, new, old, kv, g, d)
    st.fill_new()
    check_attend(E, st, window)


def test_attend_uniform(E):
    for n in (1, 3, 100):
        st = R.Step(n, [n] * 3, [7, 640, 130], 2, 4, 128)
        st.fill_new()
        check_attend(E, st, cu=False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,kv", [(1, 2), (90, 2), (400, 4)])
def test_attend_peaked(E, d, n, kv):
    """Queries of very different sizes within a head and large logits (one key
    takes nearly all), and all-zero queries (an even mean)."""
    st = R.Step(n + d, [n, n], [700, 64], kv, 4, d)
    st.fill_new()
    q = st.heads()[0].contiguous()
    q *= torch.exp2(torch.randint(-6, 5, q.shape, generator=st.gen, device="cuda")).bfloat16()
    q[:, 1] = 0
    q[:, 2, 3] = 100
    check_attend(E, st, q=q)
    check_attend(E, st, q=q * 2.0 ** -100)
    check_attend(E, st, q=q, scale=2.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([1, 1], 2), ([20, 30], 2), ([300, 90], 8)])
@pytest.mark.parametrize("loud", [1, 8])
def test_attend_logits(E, loud, new, kv, d):
    """Logits within what the 8-bit instructions keep: of each eight neighbours'
    products, seven may lose up to 2^-13 of the largest, for the query's first
    part (at most 1 + 2^-4 of it) and its second (2^-4 of that)."""
    st = R.Step(d + loud, new, [200, 70], kv, 2, d)
    st.fill_new()
    q = (st.heads()[0] * loud).contiguous()
    scale = 1 / math.sqrt(d)
    out = torch.empty_like(q)
    cache, seqs = st.objects(E)
    ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, st.T), dtype=torch.uint8, device="cuda")
    E.cache_attend(cache, seqs, q, out, scale, 0, ws)
    torch.cuda.synchronize()
    at = 0
    for b, (n, o) in enumerate(zip(st.new, st.old)):
        L = o + n
        pg = st.pages[b, :(L + 63) // 64].long()
        seen = visible(st, b, 0)
        for u in range(st.q):
            k, v = ((R.e4m3(c[pg, u // st.g]) * s[pg, u // st.g].to(F64)[:, None, None]).reshape(-1, d)[:L]
                    for c, s in zip(st.codes, st.scales))
            x = q[at:at + n, u].to(F64)
            a = torch.where(seen, x @ k.t() * scale, torch.full((), -math.inf, dtype=F64, device="cuda"))
            p = torch.softmax(a, 1)
            largest = (x[:, None, :] * k[None]).abs().view(n, L, d // 8, 8).amax(-1).sum(-1)
            off = 7 * 2.0 ** -13 * (1 + 2.0 ** -4) ** 2 * largest           # what is cut
            # the query's parts (2^-21 of its largest value), f32 sums of 2d products
            off += 2.0 ** -21 * x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] + 2 * d * 2.0 ** -24 * (x.abs() @ k.abs().t())
            off = torch.where(seen, off, torch.zeros_like(off)).amax(1, keepdim=True) * scale + 2.0 ** -16
            want = p @ v
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + torch.expm1(2 * off) + L * 2.0 ** -24) * (p @ v.abs())
            within(out[at:at + n, u], want, tol, f"out of head {u}")
        at += n


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,kv", [(1, 2), (90, 2), (400, 4)])
@pytest.mark.parametrize("far", [-100, -61, 61, 100])
def test_attend_far_value_scales(E, far, d, n, kv):
    """Values near both ends of f32's range, under large logits."""
    st = R.Step(n + d + 1, [n, n], [700, 64], kv, 4, d)
    st.fill_new()
    st.scales[1] *= 2.0 ** far
    q = st.heads()[0].contiguous()
    q[:, ::2] *= 16
    check_attend(E, st, q=q)


@pytest.mark.parametrize("n,kv,d", [(1, 2, 128), (90, 2, 128), (90, 2, 64), (30, 2, 256), (600, 8, 128),
                                   (500, 8, 64), (500, 8, 256)])
def test_attend_not_finite(E, n, kv, d):
    """NaN and infinite queries reach their own rows; NaN keys and values the
    queries that see them, and no others."""
    st = R.Step(n, [n, n], [100, 64], kv, 2, d)
    st.fill_new()
    clean = check_attend(E, st)
    q = st.heads()[0].contiguous()
    q[0, 0, 3] = math.nan
    q[-1, 3, 5] = math.inf
    out = torch.empty_like(clean)
    cache, seqs = st.objects(E)
    ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, st.T), dtype=torch.uint8, device="cuda")
    E.cache_attend(cache, seqs, q, out, 0.1, 0, ws)
    E.cache_attend(cache, seqs, st.heads()[0].contiguous(), clean, 0.1, 0, ws)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 0] = bad[-1, 3] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])
    # position 100 + n//2 of sequence 0: seen by its token and the later ones
    at = 100 + n // 2
    pg = int(st.pages[0, at // 64])
    for which in (0, 1):
        keep = st.codes[which][pg, 1, at % 64, 9].clone()
        st.codes[which][pg, 1, at % 64, 9] = 0xFF
        E.cache_attend(cache, seqs, st.heads()[0].contiguous(), out, 0.1, 0, ws)
        bad = torch.zeros_like(out, dtype=torch.bool)
        if which:
            bad[n // 2:n, 2:4, 9] = True
        else:
            bad[n // 2:n, 2:4] = True
        assert torch.equal(torch.isnan(out), bad)
        assert torch.equal(out[~bad], clean[~bad])
        # a window that ends before it: nobody but the nearest tokens see it
        E.cache_attend(cache, seqs, st.heads()[0].contiguous(), out, 0.1, 5, ws)
        bad = torch.zeros_like(out, dtype=torch.bool)
        if which:
            bad[n // 2:min(n, n // 2 + 5), 2:4, 9] = True
        else:
            bad[n // 2:min(n, n // 2 + 5), 2:4] = True
        assert torch.equal(torch.isnan(out), bad)
        st.codes[which][pg, 1, at % 64, 9] = keep


@pytest.mark.parametrize("n,kv", [(1, 2), (90, 2), (600, 8)])
def test_attend_bad_sequences(E, n, kv):
    """Sequences with bad bounds give zeros, positions of bad pages are masked
    (a row without any is zeros), tokens of no sequence are left alone."""
    make = lambda: R.Step(n + 20, [n, n, n], [100, 64, 0], kv, 2, 128)  # noqa: E731
    st = make()
    st.fill_new()
    st.pages[0, 0] = -1                                  # 64 positions of sequence 0
    check_attend(E, st, bits=8)
    st.pages[2] = st.n_pages                             # all of sequence 2
    st.err.zero_()
    out = check_attend(E, st, bits=8)
    assert not out[2 * n:].any()
    for what in ("start", "width", "cu_past", "cu_falls"):
        st = make()
        st.fill_new()
        good = check_attend(E, st)
        spoil(st, what)
        out = torch.full_like(good, 9.0)
        cache, seqs = st.objects(E)
        ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, st.T), dtype=torch.uint8, device="cuda")
        E.cache_attend(cache, seqs, st.heads()[0], out, 1 / math.sqrt(128), 0, ws)
        torch.cuda.synchronize()
        assert int(st.err) == 16
        if what in ("start", "width"):
            assert not out[:n].any() and torch.equal(out[n:], good[n:])
        elif what == "cu_past":
            assert torch.equal(out[:2 * n], good[:2 * n]) and bool((out[2 * n:] == 9).all())
        else:
            assert torch.equal(out[2 * n:], good[2 * n:]) and bool((out[:2 * n] == 9).all())


# -------------------------------------------- every page and position, once each
def visible(st, b, window):
    """[new, positions] of sequence b: what each of its tokens sees."""
    n, o = st.new[b], st.old[b]
    i, j = torch.arange(o, o + n, device="cuda"), torch.arange(o + n, device="cuda")
    seen = j[None] <= i[:, None]
    return seen & (j[None] > i[:, None] - window) if window else seen


def page_marks(d, step):
    """Each page's positions mark one dimension; pages d apart share it (at
    most 32 of the longest cache's), and another step pairs other pages."""
    def dims(st, b, j):
        blk = j // 64
        return (blk * step + (blk // d if step > 1 else 0)) % d
    return dims


def position_marks(d, window):
    """Up to d single positions, each in a dimension of its own: both ends of
    pages, cache and windows, and others between; the rest mark none (-1)."""
    def dims(st, b, j):
        L, o = len(j), st.old[b]
        at = [0, 1, 63, 64, 65, L - 1, L - 2, o, o - 1, o + 1, L // 2, L // 64 * 64, L // 64 * 64 - 1,
              o // 64 * 64, o // 64 * 64 - 1]
        at += [x - window + k for x in (o, L - 1) for k in (-1, 0, 1) if window]
        at += [64 * k + (7 * k) % 64 for k in range(0, L // 64 + 1, max(1, L // 64 // (d // 3)))]
        at = sorted({x for x in at if 0 <= x < L})[:d]
        out = torch.full((L,), -1, dtype=torch.long, device="cuda")
        out[torch.tensor(at, device="cuda")] = torch.arange(len(at), device="cuda")
        return out
    return dims


def check_marks(E, st, window, dims):
    """Zero queries weigh what they see evenly, and the values are zeros but for
    the marks: an output is a count over the positions seen, so a page or a
    position that is lost, doubled, another sequence's or another head's is off
    by 2^-5 of it and more.  Weights, products and sums are exact in f32; the
    quotient's two roundings (2^-24) and the result's (bf16, 2^-8) remain."""
    d = st.d
    want = torch.zeros(st.T, st.q, d, dtype=F64, device="cuda")
    at = 0
    for b, (n, o) in enumerate(zip(st.new, st.old)):
        L = o + n
        j = torch.arange(L, device="cuda")
        pg, slot = st.pages[b].long()[j // 64], j % 64
        size = 1 + b % 4 / 4                                     # an e4m3 value, 0x38 is 1
        code = 0x38 + 2 * (b % 4)
        at_d = dims(st, b, j) if L else j
        st.codes[1][pg, :, slot] = 0
        on = at_d >= 0
        st.codes[1][pg[on], :, slot[on], at_d[on]] = code
        for h in range(st.kv):
            st.scales[1][pg, h] = 2.0 ** (h % 4)
        if n == 0:
            continue
        marks = torch.zeros(L, d, dtype=F64, device="cuda")
        marks[j[on], at_d[on]] = size
        seen = visible(st, b, window).to(F64)
        mean = (seen @ marks) / seen.sum(1, keepdim=True)
        for h in range(st.kv):
            want[at:at + n, h * st.g:(h + 1) * st.g] = mean[:, None] * 2.0 ** (h % 4)
        at += n
    q = torch.zeros(st.T, st.q, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9.0)
    cache, seqs = st.objects(E)
    ws = torch.full((E.cache_attend_bytes(cache, seqs, st.q, st.T),), 0xFF, dtype=torch.uint8, device="cuda")
    E.cache_attend(cache, seqs, q, out, 0.7, window, ws)
    torch.cuda.synchronize()
    assert int(st.err) == 0
    within(out, want, (2.0 ** -8 + 2.0 ** -22) * want, "out")


def check_all_marks(E, new, old, kv, g, d, window, width=None):
    st = R.Step(len(new) + sum(old) % 1000, new, old, kv, g, d, width=width)
    st.fill_new()
    for dims in (page_marks(d, 1), page_marks(d, 5), position_marks(d, window)):
        check_marks(E, st, window, dims)


@pytest.mark.parametrize("window", [0, 1, 7, 64, 100])
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_marks_short(E, case, window):
    new, old, kv, g, d = STEPS[case]
    log(f"marks {new[:6]} after {old[:6]} kv {kv} g {g} d {d} window {window}")
    check_all_marks(E, new, old, kv, g, d, window)


MARKED = [
    # short tables: many units, whose values one workgroup takes
    ([1] * 300, [900 - (i % 40) for i in range(300)], 4, 2, 128, 0), ([1] * 90, [1000 - i for i in range(90)], 4, 1, 256, 0),
    ([2] * 200, [7 * i % 900 for i in range(200)], 2, 16, 64, 0), ([1] * 150, [1000 - i for i in range(150)], 8, 1, 64, 200),
    # one or few sequences: even pieces, joined by rows
    ([1], [131071], 1, 3, 64, 0), ([1], [40000], 2, 8, 256, 0), ([1], [20000], 1, 32, 128, 0), ([1], [1025], 1, 1, 64, 0),
    ([1] * 9, [4096 + 511 * i for i in range(9)], 4, 4, 128, 0), ([4, 1], [9000, 3], 2, 8, 64, 500), ([3], [6000], 2, 5, 64, 0),
    ([1, 1], [30000, 5], 1, 1, 256, 1000), ([17], [3000], 1, 20, 128, 0),
    ([1, 1, 1], [64 * 32, 64 * 32 - 1, 64 * 31 - 1], 1, 4, 256, 0), ([1] * 70, [1030 + 29 * (i % 7) for i in range(70)], 2, 4, 64, 0),
    # shares that cross units, groups of 64 sequences and sequences without tokens
    ([1] * 150, [1100 + (i % 3) for i in range(150)], 4, 1, 64, 0), ([1] * 200, [1030 + 90 * (i % 5) for i in range(200)], 8, 2, 128, 0),
    ([1] * 40, [60000] + [70] * 39, 8, 2, 128, 0), ([1] * 90, [1500 + i for i in range(90)], 4, 2, 256, 300),
    ([1] * 66, [20000 if i in (3, 65) else 3 * i for i in range(66)], 2, 4, 128, 0), (*empty_run(230, 50, 130, 1100), 8, 2, 64, 0),
    ([1] * 51, [1113] * 51, 8, 4, 128, 0),
    # tiles of 128 rows, whole and with their pages shared out
    ([300], [100], 2, 4, 128, 0), ([513, 60, 0, 129], [0, 700, 5, 63], 1, 4, 64, 0), ([700, 300], [77, 200], 4, 3, 256, 0),
    ([400], [900], 1, 8, 128, 150), ([600], [64], 4, 8, 64, 90), ([700], [300], 4, 4, 256, 64), ([1100], [33], 2, 4, 128, 0),
    ([300], [3000], 8, 2, 128, 0), ([520, 64], [2500, 3], 4, 4, 64, 700), ([200, 129, 0], [2000, 1, 9], 8, 3, 256, 0),
    ([257], [6000], 8, 4, 128, 100), ([1, 600], [4000, 2100], 4, 4, 64, 0), ([512], [30000], 8, 4, 128, 0),
    # prompts and single tokens in one step, by either kind of tile
    ([700] + [1] * 63, [50] + [1200 + 31 * i for i in range(63)], 8, 4, 128, 0), ([1] * 40 + [500], [300] * 40 + [2000], 4, 8, 64, 0),
    ([130] + [1] * 63, [900] + [40 * i for i in range(63)], 2, 4, 128, 0), ([100] + [1] * 90, [1500] + [1100] * 90, 4, 4, 256, 0)]


@pytest.mark.parametrize("case", range(len(MARKED)))
def test_marks(E, case):
    new, old, kv, g, d, window = MARKED[case]
    log(f"marks {len(new)} sequences of up to {max(new)} after up to {max(old)}, kv {kv} g {g} d {d} window {window}")
    check_all_marks(E, new, old, kv, g, d, window)


@pytest.mark.parametrize("new,old,kv,g,d,window", [
    ([1], [500], 8, 4, 128, 0), ([1] * 20, [800 - i for i in range(20)], 4, 4, 256, 0), ([3, 1], [62, 10], 2, 4, 64, 0),
    ([600], [130], 4, 4, 128, 0), ([300, 40], [0, 64], 4, 4, 256, 90), ([90] * 5, [11 * i for i in range(5)], 8, 4, 64, 0)])
def test_marks_wide_table(E, new, old, kv, g, d, window):
    """Tables of many more columns than the sequences fill, as a server keeps
    them: other kernels than a tight table's, the same outputs."""
    log(f"marks {new[:6]} after {old[:6]} kv {kv} g {g} d {d} in a table of 2048 columns")
    check_all_marks(E, new, old, kv, g, d, window, width=2048)


def test_workspace_is_asked_for(E):
    """What splits its pages needs a workspace; what does not needs none."""
    for new, old, kv, g, d, some in (([1], [5000], 2, 4, 128, True), ([1], [500], 2, 4, 128, False),
                                     ([512], [30000], 8, 4, 128, True), ([4096], [100], 8, 4, 128, False)):
        st = R.Step(1, new, old, kv, g, d)
        assert (E.cache_attend_bytes(*st.objects(E), st.q, st.T) > 0) == some


# ------------------------------------------------------- tensors in host memory
def test_one_host_tensor(E):
    """Each tensor of each call alone in host memory is refused, by name."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    norm = dict(d_x=z(4, 64), d_res=z(4, 64, dt=f32), d_w=z(64), d_codes=z(4, 64, dt=u8),
                d_scales=z(4, 2, dt=u8), d_sum=z(4, 64, dt=f32))
    w4 = dict(d_w=z(16, 64, dt=u8), d_scales=z(16, 4, dt=u8))
    project = dict(d_x=z(2, 128, dt=u8), d_xs=z(2, 4, dt=u8), d_y=z(2, 16))
    keys = dict(d_k=z(3, 1, 64, 64, dt=u8), d_v=z(3, 1, 64, 64, dt=u8), d_k_scales=z(3, 1, dt=f32),
                d_v_scales=z(3, 1, dt=f32))
    seqs = dict(d_pages=z(2, 1, dt=i32), d_start=z(2, dt=i32), d_cu=z(3, dt=i32), d_err=z(1, dt=i32))
    append = dict(d_k=z(4, 1, 64), d_v=z(4, 1, 64), d_freq=z(32, dt=f32), d_q=z(4, 2, 64), d_q_out=z(4, 2, 64))
    attend = dict(d_q=z(4, 2, 64), d_out=z(4, 2, 64), d_ws=z(1 << 20, dt=u8))
    seqs["d_cu"] += torch.tensor([0, 2, 4], dtype=i32, device="cuda")

    def calls(norm=norm, w4=w4, project=project, keys=keys, seqs=seqs, append=append, attend=attend):
        s, c = E.Sequences(**seqs), E.Cache(**keys)
        return {"norm": lambda: E.add_norm(eps=1e-6, **norm),
                "project": lambda: E.project_w4(weights=E.W4(**w4), **project),
                "append": lambda: E.cache_append(c, s, **append),
                "attend": lambda: E.cache_attend(c, s, scale=1.0, **attend)}

    for call in calls().values():
        call()
    torch.cuda.synchronize()
    uses = dict(norm=["norm"], w4=["project"], project=["project"], keys=["append", "attend"],
                seqs=["append", "attend"], append=["append"], attend=["attend"])
    for group, names in uses.items():
        have = dict(norm=norm, w4=w4, project=project, keys=keys, seqs=seqs, append=append, attend=attend)[group]
        for name in have:
            bad = calls(**{group: {**have, name: have[name].cpu()}})
            for call in names:
                with pytest.raises(E.EngramError, match="on the GPU is needed"):
                    bad[call]()


def test_outputs_beside_inputs(E):
    """An output that begins where its input ends, or ends where it begins, is
    no overlap: the same bits as in a buffer of its own."""
    st = R.Step(81, [3, 2], [70, 1200], 2, 4, 128)
    st.fill_new()
    n = st.T * st.q * st.d
    cache, seqs = st.objects(E)
    ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, st.T), dtype=torch.uint8, device="cuda")
    q = st.heads()[0].contiguous()
    want = torch.empty_like(q)
    E.cache_attend(cache, seqs, q, want, 0.1, 0, ws)
    for at in (0, n):
        both = torch.empty(2 * n, dtype=torch.bfloat16, device="cuda")
        x, out = both[at:at + n].view_as(q), both[n - at:2 * n - at].view_as(q)
        x.copy_(q)
        E.cache_attend(cache, seqs, x, out, 0.1, 0, ws)
        assert torch.equal(out, want) and torch.equal(x, q)
        with pytest.raises(E.EngramError, match="overlaps"):
            E.cache_attend(cache, seqs, x, x, 0.1, 0, ws)
    w, ws4, x, xs, _ = w4_case(82, 5, 256, 256, False)
    want = torch.empty(5, 256, dtype=torch.bfloat16, device="cuda")
    E.project_w4(x, E.W4(w, ws4), want)
    for at in (0, 1):
        both = torch.empty(2, 5, 256, dtype=torch.bfloat16, device="cuda")
        both[at].copy_(x)
        E.project_w4(both[at], E.W4(w, ws4), both[1 - at])
        assert torch.equal(both[1 - at], want)
        with pytest.raises(E.EngramError, match="overlaps"):
            E.project_w4(both[at], E.W4(w, ws4), both[at])


# ------------------------------------------- token bounds that are not in order
def overlapping(B, first, last):
    """Bounds whose first sequence brings tokens 0 .. first-1 and whose last
    brings the `last` after them; those between begin again at 0, or fall."""
    return [0] + [first if i % 2 else 0 for i in range(1, B)] + [first + last]


@pytest.mark.parametrize("B,first,last,old,kv,g,d", [
    (4, 6, 3, 10, 2, 2, 64), (4, 1, 1, 1100, 2, 4, 128), (200, 16, 3, 1100, 8, 2, 64),
    (66, 2, 1, 1500, 1, 1, 256), (4, 600, 90, 70, 8, 2, 128), (130, 400, 300, 5, 8, 4, 64)])
def test_overlapping_bounds(E, B, first, last, old, kv, g, d):
    """A sequence that begins before an earlier one's end is bad: its tokens
    count once, whatever the bounds between say."""
    log(f"overlapping bounds, {B} sequences, {first} + {last} tokens after {old}, kv {kv} g {g} d {d}")
    new, olds = [first] + [0] * (B - 2) + [last], [old] + [9] * (B - 2) + [old // 2]
    good, st = (R.Step(B + first, new, olds, kv, g, d) for _ in range(2))
    bounds = overlapping(B, first, last)
    st.cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    outs = []
    for s in (good, st):
        q, k, v = s.heads()
        cache, seqs = s.objects(E)
        outs.append(torch.full((s.T, s.q, s.d), 9.0, dtype=torch.bfloat16, device="cuda"))
        E.cache_append(cache, seqs, k, v, R.freq_of(d), q, outs[-1])
    torch.cuda.synchronize()
    assert int(good.err) == 0 and int(st.err) == 16
    assert torch.equal(*outs)
    for x, y in zip(st.codes + st.scales, good.codes + good.scales):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())
    st.err.zero_()
    check_attend(E, st, bits=16)


# ----------------------------------------------------- a cache past 32 bits
@pytest.mark.parametrize("new,old", [([1, 1], [100, 900]), ([1, 1], [1500, 70]), ([300, 260], [200, 33])])
def test_pages_past_4_gib(E, new, old):
    """Pages behind 4 GiB of codes: the same bits as in a cache of their own."""
    st = R.Step(60, new, old, 8, 4, 256)
    freq = R.freq_of(256)

    def step():
        q, k, v = st.heads()
        qo, out = (torch.empty(st.T, st.q, st.d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache, seqs = st.objects(E)
        ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, st.T), dtype=torch.uint8, device="cuda")
        E.cache_append(cache, seqs, k, v, freq, q, qo)
        E.cache_attend(cache, seqs, qo, out, 1 / 16, 0, ws)
        torch.cuda.synchronize()
        assert int(st.err) == 0
        return out

    first = ((1 << 32) // (8 * 64 * 256)) + 5
    codes, scales, n = [c.clone() for c in st.codes], [x.clone() for x in st.scales], st.n_pages
    want = step()
    appended = [c.clone() for c in st.codes] + [x.clone() for x in st.scales]
    for which in (0, 1):
        for kept, now in ((codes, st.codes), (scales, st.scales)):
            big = torch.empty(first + n, *kept[which].shape[1:], dtype=kept[which].dtype, device="cuda")
            big[first:] = kept[which]
            now[which] = big
    st.pages = (st.pages + first).int()
    st.n_pages = first + n
    assert torch.equal(step(), want)
    for big, small in zip(st.codes + st.scales, appended):
        assert torch.equal(big[first:].nan_to_num() if big.dtype == torch.float32 else big[first:],
                           small.nan_to_num() if big.dtype == torch.float32 else small)


# ------------------------------------------------------ the far end of the sizes
@pytest.mark.parametrize("dim,bf16", [(32, False), (544, True)])
def test_add_norm_many_rows(E, dim, bf16):
    """More rows than workgroups: each takes rows in turn.  The same bits as in
    calls of fewer."""
    rows, some = (1 << 20) + 1037, 4096
    t = torch.bfloat16 if bf16 else torch.float32
    g = seeded(dim)
    few = torch.randn(some, dim, generator=g, device="cuda")
    w = (1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).bfloat16()
    at = torch.arange(rows, device="cuda") % some
    x = (0.3 * few).bfloat16()

    def call(res, x):
        total, codes = torch.empty_like(res), torch.zeros(res.shape, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(res.shape[0], dim // 32, dtype=torch.uint8, device="cuda")
        E.add_norm(x, res, w, 1e-6, codes, scales, d_sum=total)
        return total, codes, scales

    want = call(few.to(t), x)
    for got, one in zip(call(few.to(t)[at], x[at]), want):
        assert torch.equal(got, one[at])


@pytest.mark.parametrize("fp8", [True, False])
def test_project_w4_most_tokens(E, fp8):
    """2^22 tokens, which repeat sixty-four: the same bits for each."""
    T, K, N = 1 << 22, 128, 16
    w, ws, x, xs, x64 = w4_case(91, 64, K, N, fp8)
    want = check_w4(E, w, ws, x, xs, x64)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    E.project_w4(x.repeat(T // 64, 1), E.W4(w, ws), y, None if xs is None else xs.repeat(T // 64, 1))
    assert bool((y.view(T // 64, 64, N) == want).all())


def test_append_most_tokens(E):
    """2^22 tokens of one sequence at once, and in two calls that meet at a page's
    border: the same bytes (each page has all its tokens in one call)."""
    n, d = 1 << 22, 64
    pages = torch.randperm(n // 64, device="cuda").int().view(1, -1)
    k, v = (torch.randn(n, 1, d, generator=seeded(s), device="cuda", dtype=torch.bfloat16) for s in (1, 2))
    freq = R.freq_of(d)
    made = []
    for cuts in ((0, n), (0, n // 2 + 64 * 77, n)):
        codes = [torch.zeros(n // 64, 1, 64, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(n // 64, 1, device="cuda") for _ in range(2)]
        cache, err = E.Cache(*codes, *scales), torch.zeros(1, dtype=torch.int32, device="cuda")
        for lo, hi in zip(cuts, cuts[1:]):
            start = torch.tensor([lo], dtype=torch.int32, device="cuda")
            E.cache_append(cache, E.Sequences(pages, start, d_err=err), k[lo:hi], v[lo:hi], freq)
        torch.cuda.synchronize()
        assert int(err) == 0
        made.append(codes + scales)
    for x, y in zip(*made):
        assert torch.equal(x, y)
    # the last page against the formula
    at = slice(n - 64, n)
    want, _ = R.rotate(k[at], torch.arange(n - 64, n, device="cuda"), freq, True)
    p = int(pages[0, -1])
    got = R.e4m3(made[0][0][p, 0]) * made[0][2][p].to(F64)
    within(got, want[:, 0], 2.0 ** -4 * want[:, 0].abs() + 2.0 ** -10 * made[0][2][p].to(F64) + 2.0 ** -20 * 8, "keys")


@pytest.mark.parametrize("fp8", [True, False])
def test_project_w4_lowest_scale(E, fp8):
    """Scale byte 0 is 2^-127, below f32's normal numbers."""
    w, ws, x, xs, x64 = w4_case(19, 5, 256, 32, fp8, 0, 1)
    if fp8:
        xs = (254 - xs.int()).to(torch.uint8)
        x64 = R.grouped(R.e4m3(x), xs)
    else:
        x = (x.float() * 2.0 ** 120).bfloat16()
        x64 = x.to(F64)
    check_w4(E, w, ws, x, xs, x64)


FORMS = [([1], [500], 2, 4, 128), ([1, 1], [1500, 70], 2, 8, 256), ([3], [5000], 1, 4, 64), ([300, 7], [90, 64], 4, 4, 128),
         ([90, 60], [700, 3], 8, 4, 256), ([260], [2500], 8, 4, 64)]      # short, even pieces, tiles, split tiles


@pytest.mark.parametrize("case", range(len(FORMS)))
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30])
def test_attend_scales(E, scale, case):
    """Negative scales turn the order of the logits round, zero ones level it."""
    st = R.Step(70 + case, *FORMS[case])
    st.fill_new()
    q = st.heads()[0]
    out = torch.empty(st.T, st.q, st.d, dtype=torch.bfloat16, device="cuda")
    cache, seqs = st.objects(E)
    ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, st.T), dtype=torch.uint8, device="cuda")
    E.cache_attend(cache, seqs, q, out, scale, 0, ws)
    want, tol = R.attend(st, q, scale, 0)
    within(out, want, tol, "out")


@pytest.mark.parametrize("case", range(len(FORMS)))
def test_attend_any_page_scale(E, case):
    """Page scales that are no powers of two, as a caller's own cache may have."""
    st = R.Step(80 + case, *FORMS[case])
    st.fill_new()
    for i in (0, 1):
        st.scales[i] *= 1 + torch.rand(st.scales[i].shape, generator=st.gen, device="cuda")
    check_attend(E, st)
    check_attend(E, st, window=77)


@pytest.mark.parametrize("case", range(len(FORMS)))
def test_attend_far_windows(E, case):
    """A window past every position is none, however large it is."""
    st = R.Step(90 + case, *FORMS[case])
    st.fill_new()
    none = check_attend(E, st)
    for window in (max(st.old) + max(st.new), (1 << 30) + 5, (1 << 31) - 1, 1 << 31, (1 << 40) + 1):
        out = check_attend(E, st, window)
        if window > 1 << 30:                            # shared out as without one: the same bits
            assert torch.equal(out, none)


@pytest.mark.parametrize("case", range(len(FORMS)))
def test_heads_side_by_token(E, case):
    """Queries, keys and values whose tokens lie side by side within a head."""
    st, same = (R.Step(100 + case, *FORMS[case]) for _ in range(2))
    freq, outs = R.freq_of(st.d), []
    for s, far in ((st, True), (same, False)):
        heads = [x.transpose(0, 1).contiguous().transpose(0, 1) if far else x for x in s.heads()]
        q, k, v = heads
        assert not far or s.T == 1 or q.stride(0) == s.d
        qo, out = (torch.empty(s.T, s.q, s.d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache, seqs = s.objects(E)
        E.cache_append(cache, seqs, k, v, freq, q, qo)
        ws = torch.empty(E.cache_attend_bytes(cache, seqs, s.q, s.T), dtype=torch.uint8, device="cuda")
        E.cache_attend(cache, seqs, qo.transpose(0, 1).contiguous().transpose(0, 1) if far else qo, out, 0.1, 0, ws)
        outs += [qo, out]
        assert int(s.err) == 0
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    for x, y in zip(st.codes + st.scales, same.codes + same.scales):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())


# ------------------------------------------------------- streams and graphs
def test_stream_and_graph(E):
    """The four operators on a stream of their own, and captured into a graph
    that is replayed with eager work between: the same bits each time."""
    st = R.Step(50, [1, 1, 1], [100, 1000, 3000], 2, 4, 128)
    T, dim = st.T, 512
    g = seeded(51)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    res, x, w = rn(T, dim), rn(T, dim).bfloat16(), (1 + 0.1 * rn(dim)).bfloat16()
    N = (st.q + 2 * st.kv) * st.d
    wt = E.W4(torch.randint(0, 256, (N, dim // 2), generator=g, device="cuda", dtype=torch.uint8),
              torch.randint(119, 123, (N, dim // 32), generator=g, device="cuda", dtype=torch.uint8))
    total, codes = torch.empty_like(res), torch.empty(T, dim, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, dim // 32, dtype=torch.uint8, device="cuda")
    qkv = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    heads = qkv.view(T, st.q + 2 * st.kv, st.d)
    qo, out = (torch.empty(T, st.q, st.d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache, seqs = st.objects(E)
    ws = torch.empty(E.cache_attend_bytes(cache, seqs, st.q, T), dtype=torch.uint8, device="cuda")
    freq = R.freq_of(128)

    def step(stream=None):
        E.add_norm(x, res, w, 1e-6, codes, scales, d_sum=total, stream=stream)
        E.project_w4(codes, wt, qkv, scales, stream=stream)
        E.cache_append(cache, seqs, heads[:, st.q:st.q + st.kv], heads[:, st.q + st.kv:], freq,
                       heads[:, :st.q], qo, stream=stream)
        E.cache_attend(cache, seqs, qo, out, 1 / math.sqrt(128), 0, ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    assert bool(torch.isfinite(want).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        out.zero_()
        qkv.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
        x.copy_(rn(T, dim).bfloat16())               # another step between, eager
        step()
        want = out.clone()


def test_example(E):
    """The example's prompt and steps: finite, and the same bits again."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "attention_step.py")
    spec = importlib.util.spec_from_file_location("attention_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rows = example.run()
    assert bool(torch.isfinite(rows).all())
    assert torch.equal(rows, example.run())
