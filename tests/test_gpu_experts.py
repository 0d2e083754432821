"""The experts' operators on the GPU against their 64-bit forms
(tests/_experts_ref.py).  Tolerances count roundings: half a step of the
result's type (bf16 2^-8, e4m3 2^-4 relative) beside what the form states."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import _attention_ref as A  # noqa: E402
import _experts_ref as R  # noqa: E402
from _gpu_util import log  # noqa: E402

pytestmark = pytest.mark.gpu
F64 = torch.float64
INF, NAN = math.inf, math.nan


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


# -------------------------------------------------------------------- routing
def new_routes(E, T, n, k, fill=-7):
    i32 = torch.int32
    return E.Routes(torch.full((T, k), fill, dtype=i32, device="cuda"), torch.full((T, k), NAN, device="cuda"),
                    torch.full((n + 1,), fill, dtype=i32, device="cuda"),
                    torch.full((T * k,), fill, dtype=i32, device="cuda"), torch.zeros(1, dtype=i32, device="cuda"))


def space(E, need):
    return torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") if need else None


def check_route(E, x, bias, k, softmax=False, groups=1, top=1, best=2, renorm=True, factor=1.0, err=0, what=""):
    T, n = x.shape
    r = new_routes(E, T, n, k)
    E.route(x, r, bias, softmax, groups, top, best, renorm, factor, space(E, E.route_bytes(r)))
    torch.cuda.synchronize()
    ids, w, offsets, order = R.route(x.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy(),
                                     k, softmax, groups, top, best, renorm, factor)
    got_ids, got_w, got_offsets, got_order, got_err = (t.cpu().numpy() for t in r.keep)
    assert np.array_equal(got_ids, ids), f"{what}: ids differ in {(got_ids != ids).any(1).sum()} tokens"
    # a softmax score is off by (|x - max| + 6) * 2^-24 of itself, at most e^-104 long; a sigmoid by less
    off = np.abs(got_w - w) - (2.0 ** -17 * np.abs(w) + 2.0 ** -149)
    assert off.max() <= 0, f"{what}: weights {off.max():.2e} past the tolerance"
    assert np.array_equal(got_offsets, offsets), f"{what}: offsets"
    assert np.array_equal(got_order[:len(order)], order), f"{what}: order"
    assert (got_order[len(order):] == -7).all(), f"{what}: rows past the plan are written"
    assert int(got_err[0]) == err, f"{what}: error word {int(got_err[0])}"
    return r


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T,n,k,groups,top,best", [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 5, 5, 1, 1, 1), (2, 8, 2, 1, 1, 2), (63, 60, 4, 4, 2, 1),
    (64, 64, 6, 1, 1, 1), (65, 65, 8, 5, 2, 2), (130, 160, 6, 8, 3, 1), (777, 60, 4, 1, 1, 1), (40, 384, 8, 1, 1, 1),
    (70, 384, 8, 64, 5, 2), (129, 1024, 32, 16, 4, 2), (9, 512, 32, 2, 1, 2), (31, 96, 3, 48, 2, 2), (5, 64, 1, 64, 1, 2),
    (1000, 256, 8, 8, 4, 2)])
def test_route(E, T, n, k, groups, top, best, softmax):
    g = seeded(T * 31 + n)
    for bf16 in (False, True):
        for with_bias in (False, True):
            x = torch.randn(T, n, generator=g, device="cuda") * (1 + 2 * with_bias)
            x = x.bfloat16() if bf16 else x
            bias = torch.randn(n, generator=g, device="cuda") * 0.2 if with_bias else None
            renorm = (T + with_bias) % 2 == 0
            what = f"T {T} n {n} k {k} groups {groups} bf16 {bf16} bias {with_bias} softmax {softmax} renorm {renorm}"
            log(what)
            check_route(E, x, bias, k, softmax, groups, top, best, renorm, 2.5 if renorm else 1.0, what=what)


@pytest.mark.parametrize("T", [64 * 256, 64 * 256 + 1, 64 * 320 + 17])
def test_route_many_tokens(E, T):
    """Calls whose blocks are counted once, and once more by segments."""
    log(f"route T {T}")
    g = seeded(T)
    check_route(E, torch.randn(T, 24, generator=g, device="cuda"), 0.1 * torch.randn(24, generator=g, device="cuda"), 3)


@pytest.mark.parametrize("softmax", [False, True])
def test_route_ties(E, softmax):
    """Equal keys go to the lowest expert and group, with and without a bias."""
    zero = torch.zeros(100, 96, device="cuda")
    flat = torch.full((96,), 0.25, device="cuda")
    g = seeded(5)
    few = torch.randint(-2, 3, (100, 96), generator=g, device="cuda").float() / 2
    signed = torch.where(torch.rand(100, 96, generator=g, device="cuda") < 0.5, -zero, zero)
    signed[:, 7] = -1e-30
    for x in (zero, few, few.bfloat16(), signed):
        for bias in (None, flat):
            for groups, top, best in ((1, 1, 1), (8, 3, 2), (12, 2, 1)):
                check_route(E, x, bias, 8, softmax, groups, top, best, what=f"groups {groups}")


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_route_near_keys(E, softmax, groups, top):
    """Keys that f32 cannot tell apart are told apart all the same: the biases
    undo one token's scores up to their rounding."""
    g = seeded(11)
    x = torch.randn(50, 64, generator=g, device="cuda")
    score = torch.softmax(x.double(), 1) if softmax else torch.sigmoid(x.double())
    for t in (0, 17):
        check_route(E, x, (0.7 - score[t]).float(), 8, softmax, groups, top, 2)
    # a group's two keys against another's
    x[:, 1::2] = x[:, ::2]
    check_route(E, x, (0.7 - score[3]).float(), 8, softmax, groups, top, 2)


@pytest.mark.parametrize("softmax", [False, True])
def test_route_shut(E, softmax):
    """Shut experts, shut groups, rows of nothing, padding; values of any size."""
    g = seeded(3)
    x = torch.randn(140, 48, generator=g, device="cuda")
    bias = 0.1 * torch.randn(48, generator=g, device="cuda")
    x[:, 5] = -INF
    x[3] = -INF
    x[4, 2:] = -INF                                    # fewer open than asked for
    x[5, :24] = -INF                                   # whole groups
    x[130:] = -INF
    lowest = x.clone()
    lowest[6:9] = torch.finfo(torch.float32).min       # the type's lowest value is a value
    lowest[9, ::2] = torch.finfo(torch.float32).max
    lowest[10] *= 100                                  # sigmoids that vanish in f32
    lowest[11] = -60 - lowest[11].abs().clamp(max=10)
    lowest[12] = -200 - lowest[12].abs().clamp(max=10)
    for b in (None, bias):
        for groups, top, best in ((1, 1, 1), (6, 2, 2), (6, 1, 1), (48, 3, 2)):
            check_route(E, x, b, 6, softmax, groups, top, best)
            check_route(E, lowest, b, 6, softmax, groups, top, best)
    shut = bias.clone()
    shut[7] = -INF
    check_route(E, x, shut, 6, softmax, 6, 2)
    shut[:] = -INF
    r = check_route(E, x, shut, 6, softmax)
    assert int(r.keep[2][-1]) == 0
    for bad in (NAN, INF):
        y = x.clone()
        y[20, 9] = bad
        err = E.DEVERR_ROUTE
        check_route(E, y, None, 6, softmax, err=err)
        check_route(E, y, bias, 6, softmax, 6, 2, err=err)
        shut = bias.clone()
        shut[2] = bad
        check_route(E, x, shut, 6, softmax, err=err)


def test_route_views(E):
    """Rows of wider rows; a stream of their own."""
    g = seeded(8)
    wide = torch.randn(90, 200, generator=g, device="cuda")
    check_route(E, wide[:, 13:77], None, 4)
    check_route(E, wide.bfloat16()[:, 13:76], None, 4, True)
    check_route(E, wide[::2, :64], None, 4)
    check_route(E, wide[:1].expand(30, 200)[:, :1][:1], None, 1)


# ------------------------------------------------------------------- products
SIZES = [(1, 128, 16), (1, 4096, 6144), (2, 512, 48), (5, 640, 1040), (16, 2048, 256), (17, 896, 272), (33, 1152, 4112),
         (48, 384, 16), (64, 6144, 512), (65, 256, 64), (130, 768, 80), (200, 1024, 1296), (1, 16384, 32), (300, 128, 400),
         (257, 384, 528), (513, 256, 272), (1000, 512, 256), (129, 2048, 5200)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_project_f8(E, T, K, N, f32):
    log(f"project_f8 T {T} K {K} N {N} f32 {f32}")
    g = seeded(T + K + N)
    w, s = R.weights8(g, N, K)
    x, xs, x64 = R.rows8(g, T, K, f32)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    E.project_f8(x, E.F8(w, s), y, xs)
    torch.cuda.synchronize()
    want, tol = R.product(x64, R.matrix(w, s))
    within(y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")


def some_plan(g, T, n, k, empty=0.0, skew=1.0):
    """ids [T, k] (some -1), weights, offsets, order: experts not equally liked."""
    x = torch.randn(T, n, generator=g, device="cuda") + skew * torch.randn(n, generator=g, device="cuda")
    top = torch.topk(x, k, 1)
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < empty, -1, top.indices)
    weights = torch.where(ids >= 0, torch.softmax(top.values, 1), torch.zeros_like(top.values))
    offsets, order = R.plan(ids.cpu().numpy(), n)
    i32 = torch.int32
    filled = np.full(T * k, 1 << 30)                   # past the plan: not to be read
    filled[:len(order)] = order
    return (ids.to(i32), weights, torch.tensor(offsets, dtype=i32, device="cuda"),
            torch.tensor(filled, dtype=i32, device="cuda")), offsets, order


PLANS = [(1, 4, 1, 0.0), (1, 8, 8, 0.0), (1, 16, 2, 0.0), (3, 5, 2, 0.0), (7, 64, 6, 0.2), (16, 4, 2, 0.0), (40, 2, 1, 0.0),
         (64, 16, 4, 0.1), (200, 3, 2, 0.0), (333, 8, 2, 0.3), (600, 2, 2, 0.0), (500, 1, 1, 0.0), (128, 60, 4, 0.0),
         (1100, 12, 3, 0.05), (9, 4, 2, 1.0)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("K,I", [(128, 128), (640, 256), (1024, 384)])
@pytest.mark.parametrize("T,n,k,empty", PLANS)
def test_experts_up(E, T, n, k, empty, K, I, f32):
    log(f"experts_up T {T} experts {n} k {k} empty {empty} K {K} I {I} f32 {f32}")
    g = seeded(T * 7 + n + K + I)
    arrays, offsets, order = some_plan(g, T, n, k, empty)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w, s = R.weights8(g, n, 2, I, K)
    x, xs, x64 = R.rows8(g, T, K, f32)
    h = torch.full((T * k, I), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((T * k, I // 32), 0x55, dtype=torch.uint8, device="cuda")
    E.experts_up(x, xs, E.F8(w, s), E.Routes(*arrays, err), h, hs)
    torch.cuda.synchronize()
    m = len(order)
    want, tol = R.up(x64, w, s, offsets, order, k)
    check_h(h[:m], hs[:m], want, tol)
    assert bool((h[m:] == 0x55).all()) and bool((hs[m:] == 0x55).all()), "rows past the plan are written"
    assert int(err) == 0


def check_h(h, hs, want, tol):
    m, I = want.shape
    if not m:
        return
    got_s = torch.exp2(hs.to(F64) - 127)
    amax, slack = (v.view(m, -1, 32).amax(2) for v in (want.abs(), tol))
    lo, hi = A.scale_of((amax - slack).clamp(min=0)), A.scale_of(amax + slack)
    assert bool(((got_s == lo) | (got_s == hi)).all()), "scales"
    wide = got_s.repeat_interleave(32, 1)
    within(A.e4m3(h) * wide, want, 2.0 ** -4 * want.abs() + (1 + 2.0 ** -4) * tol + 2.0 ** -10 * wide, "h")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("K,N", [(128, 16), (640, 272), (1024, 528), (384, 2064)])
@pytest.mark.parametrize("T,n,k,empty", PLANS)
def test_experts_down(E, T, n, k, empty, K, N, f32):
    log(f"experts_down T {T} experts {n} k {k} empty {empty} K {K} N {N} f32 {f32}")
    g = seeded(T * 5 + n + K + N)
    arrays, offsets, order = some_plan(g, T, n, k, empty)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w, s = R.weights8(g, n, N, K)
    h, hs, h64 = R.rows8(g, T * k, K, f32)
    h[len(order):] = 0x7F                              # NaN codes past the plan: not to be read
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    weights, routes = E.F8(w, s), E.Routes(*arrays, err)
    need = E.experts_down_bytes(weights, routes)
    E.experts_down(h, hs, weights, routes, y, torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None)
    torch.cuda.synchronize()
    want, tol = R.down(h64, w, s, offsets, order, arrays[1])
    within(y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")
    assert int(err) == 0


# --------------------------------------------------- tile sizes and their borders
@pytest.mark.parametrize("T,K,N", [(4090, 256, 4080), (2040, 256, 4080), (2040, 384, 2032), (1000, 256, 2032), (1000, 1152, 1008),
                                   (97, 2048, 336), (4090, 128, 4096)])
def test_project_f8_tiles(E, T, K, N):
    log(f"project_f8 T {T} K {K} N {N}")
    g = seeded(T + K + N)
    w, s = R.weights8(g, N, K)
    for f32 in (False, True):
        x, xs, x64 = R.rows8(g, T, K, f32)
        y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        E.project_f8(x, E.F8(w, s), y[:T], xs)
        torch.cuda.synchronize()
        want, tol = R.product(x64, R.matrix(w, s))
        within(y[:T], want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")
        assert bool((y[T] == 7).all()), "a row past the last is written"


# tiles of 256 x 256, 128 x 256, 128 x 128 and 64 x 128 over more blocks than a load of scales
# covers, of 128 x 128 and 64 x 128 over one, few rows of weights that no cache keeps
@pytest.mark.parametrize("T,K,N", [(4090, 1152, 4080), (2000, 1152, 4080), (961, 1152, 10000), (2000, 1408, 2064),
                                   (1000, 128, 10240), (2040, 128, 2032), (100, 6144, 16400), (35, 6144, 16400)])
def test_project_f8_long_tiles(E, T, K, N):
    test_project_f8_tiles(E, T, K, N)


def counted_plan(g, counts, shuffled=False):
    """One expert a token, so many tokens each."""
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(sum(counts)))]
    offsets, order = R.plan(ids[:, None].numpy(), len(counts))
    if shuffled:                                       # an expert's slots in any order
        rng = np.random.default_rng(1)
        order = np.concatenate([rng.permutation(order[p:q]) for p, q in zip(offsets[:-1], offsets[1:])])
    i32 = torch.int32
    weights = torch.rand(len(ids), 1, generator=g, device="cuda") - 0.3
    return (ids[:, None].to(i32).cuda(), weights, torch.tensor(offsets, dtype=i32, device="cuda"),
            torch.tensor(order, dtype=i32, device="cuda")), offsets, order


def check_experts(E, g, arrays, offsets, order, n, K, I, N, f32=False, err=0):
    """Both products over a plan, from rows and from h of their own."""
    T, k = arrays[0].shape
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    routes = E.Routes(*arrays, word)
    m = len(order)
    w, s = R.weights8(g, n, 2, I, K)
    x, xs, x64 = R.rows8(g, T, K, f32)
    h = torch.full((T * k, I), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((T * k, I // 32), 0x55, dtype=torch.uint8, device="cuda")
    E.experts_up(x, xs, E.F8(w, s), routes, h, hs)
    want, tol = R.up(x64, w, s, offsets, order, k)
    check_h(h[:m], hs[:m], want, tol)
    assert bool((h[m:] == 0x55).all()) and bool((hs[m:] == 0x55).all()), "rows past the plan are written"
    w, s = R.weights8(g, n, N, K)
    down = E.F8(w, s)
    h, hs, h64 = R.rows8(g, T * k, K, f32)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    E.experts_down(h, hs, down, routes, y, space(E, E.experts_down_bytes(down, routes)))
    want, tol = R.down(h64, w, s, offsets, order, arrays[1])
    within(y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")
    assert int(word) == err


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts", [[0, 1, 15, 16, 17, 3], [0, 0, 9, 0], [64, 65, 0, 128, 1, 63], [100, 128, 129, 43], [33, 31],
                                    [129, 256, 257, 0, 512, 300], [255, 193, 192, 320, 321], [1000]])
def test_experts_borders(E, counts, f32):
    log(f"experts with {counts} rows f32 {f32}")
    g = seeded(sum(counts))
    arrays, offsets, order = counted_plan(g, counts, shuffled=True)
    check_experts(E, g, arrays, offsets, order, len(counts), 384, 256, 528, f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("counts", [[300, 200, 129], [100, 64, 50], [20, 9, 3], [2, 0, 1]])
def test_experts_long_rows(E, counts, f32):
    """More blocks of K than one load of rows' scales covers, at every tile's height."""
    log(f"experts' rows {counts} of 1408 and 1152 values")
    g = seeded(sum(counts) + 1)
    arrays, offsets, order = counted_plan(g, counts)
    check_experts(E, g, arrays, offsets, order, len(counts), 1408, 256, 272, f32)
    check_experts(E, g, arrays, offsets, order, len(counts), 1152, 128, 2064, f32)


def test_experts_many(E):
    """The most experts, the most of them a token."""
    g = seeded(12)
    arrays, offsets, order = some_plan(g, 20, 1024, 32, 0.1)
    check_experts(E, g, arrays, offsets, order, 1024, 128, 128, 48)
    arrays, offsets, order = some_plan(g, 700, 32, 32, 0.1)
    check_experts(E, g, arrays, offsets, order, 32, 128, 128, 48)


def test_experts_one_twice(E):
    """A token's slots may name one expert twice: a row each."""
    g = seeded(13)
    for T in (1, 5, 60):
        ids = torch.full((T, 3), 2, dtype=torch.int32)
        ids[:, 1] = 0
        offsets, order = R.plan(ids.numpy(), 4)
        weights = torch.rand(T, 3, generator=g, device="cuda")
        arrays = (ids.cuda(), weights, *(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, order)))
        check_experts(E, g, arrays, offsets, order, 4, 256, 128, 2048 if T == 5 else 64)


# --------------------------------------------------------- values at their ends
@pytest.mark.parametrize("T", [3, 40, 300])
def test_project_f8_nan(E, T):
    """NaN codes and scales reach their own row and output alone; an infinite
    block scale its own outputs."""
    g = seeded(T)
    w, s = R.weights8(g, 400, 512)
    x, xs, x64 = R.rows8(g, T, 512, False)
    x[1, 77] = 0x7F
    xs[2, 3] = 255
    w[5, 200] = 0xFF
    s[3, 1] = INF
    x64 = A.grouped(A.e4m3(x), xs)
    y = torch.zeros(T, 400, dtype=torch.bfloat16, device="cuda")
    E.project_f8(x, E.F8(w, s), y, xs)
    bad = torch.zeros(T, 400, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    bad[:, 5] = True
    assert bool(torch.isnan(y[bad]).all())
    far = torch.zeros_like(bad)
    far[:, 384:] = True
    assert not bool(torch.isfinite(y[far]).any())
    s[3, 1], w[5, 200], x[1, 77], xs[2, 3] = 1.0, 0, 0, 127
    x64 = A.grouped(A.e4m3(x), xs)
    want, tol = R.product(x64, R.matrix(w, s))
    rest = ~(bad | far)
    within(y[rest], want[rest], (2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol)[rest], "y")


@pytest.mark.parametrize("T", [2, 60])
def test_project_f8_scales(E, T):
    """Scales from one end of their bytes to the other, undone by the weights'."""
    g = seeded(T + 1)
    K, N = 512, 160
    w, _ = R.weights8(g, N, K)
    for byte in (1, 40, 127, 200, 250):
        x, xs, _ = R.rows8(g, T, K, False)
        xs[:] = byte
        s = torch.full((2, 4), 2.0 ** (127 - max(byte, 3)) / 4096, device="cuda")
        y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        E.project_f8(x, E.F8(w, s), y, xs)
        want, tol = R.product(A.grouped(A.e4m3(x), xs), R.matrix(w, s))
        # (byte 1: products reach below f32's normal numbers)
        within(y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol + 2.0 ** -126 * K * s[0, 0].double(), f"scale byte {byte}")


def test_experts_nan(E):
    """A NaN or infinity in one token's rows stays with that token."""
    g = seeded(21)
    for T in (4, 90):
        arrays, offsets, order = some_plan(g, T, 3, 2)
        w, s = R.weights8(g, 3, 2, 128, 256)
        x, xs, _ = R.rows8(g, T, 256, False)
        out = []
        for bad in (False, True):
            if bad:
                x[2, 100] = 0x7F
            h = torch.zeros(2 * T, 128, dtype=torch.uint8, device="cuda")
            hs = torch.zeros(2 * T, 4, dtype=torch.uint8, device="cuda")
            E.experts_up(x, xs, E.F8(w, s), E.Routes(*arrays), h, hs)
            out.append((h, hs))
        mine = torch.tensor(order // 2 == 2, device="cuda")
        (h0, hs0), (h1, hs1) = out
        assert torch.equal(h0[~mine], h1[~mine]) and torch.equal(hs0[~mine], hs1[~mine])
        assert bool(torch.isnan(A.e4m3(h1[mine])).all())
        wd, sd = R.weights8(g, 3, 64, 128)
        down, routes = E.F8(wd, sd), E.Routes(*arrays)
        ys = []
        for h, hs in out:
            y = torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")
            E.experts_down(h, hs, down, routes, y, space(E, E.experts_down_bytes(down, routes)))
            ys.append(y)
        others = torch.arange(T, device="cuda") != 2
        assert torch.equal(ys[0][others], ys[1][others]) and bool(torch.isnan(ys[1][2]).all())


def test_experts_down_infinite(E):
    """Products past f16's and f32's range: large ones keep their size, infinite
    ones are infinite."""
    g = seeded(22)
    for T in (3, 70):
        ids = torch.zeros(T, 1, dtype=torch.int32)
        offsets, order = R.plan(ids.numpy(), 2)
        arrays = (ids.cuda(), torch.ones(T, 1, device="cuda"),
                  *(torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, order)))
        w, s = R.weights8(g, 2, 64, 128)
        h, hs, _ = R.rows8(g, T, 128, True)
        hs[0] *= 2.0 ** 60
        hs[1] = 2.0 ** 127
        s[:] = 2.0 ** 20
        down, routes = E.F8(w, s), E.Routes(*arrays)
        y = torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")
        E.experts_down(h, hs, down, routes, y, space(E, E.experts_down_bytes(down, routes)))
        h64 = A.e4m3(h) * hs.double()
        want, tol = R.down(h64, w, s, offsets, order, arrays[1])
        fine = torch.arange(T, device="cuda") != 1
        within(y[fine], want[fine], (2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol)[fine], "y")
        assert not bool(torch.isfinite(y[1]).any())


# ------------------------------------------------------------------- bad plans
@pytest.mark.parametrize("T,k,n", [(6, 2, 4), (40, 2, 3), (400, 2, 3), (1200, 1, 2)])
def test_bad_plans(E, T, k, n):
    """Spans and slots out of range set the error bit, and what they do not
    touch is computed as ever."""
    log(f"bad plans T {T} k {k} experts {n}")
    g = seeded(T)
    (ids, weights, offsets, order), *_ = some_plan(g, T, n, k, skew=0.0)
    w, s = R.weights8(g, n, 2, 128, 256)
    up = E.F8(w, s)
    N = 2048 if T == 6 else 64                         # one launch, and two
    wd, sd = R.weights8(g, n, N, 128)
    down = E.F8(wd, sd)
    x, xs, _ = R.rows8(g, T, 256, False)

    def both(offsets, order):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        routes = E.Routes(ids, weights, offsets, order, err)
        h = torch.full((T * k, 128), 0x55, dtype=torch.uint8, device="cuda")
        hs = torch.full((T * k, 4), 0x7F, dtype=torch.uint8, device="cuda")
        E.experts_up(x, xs, up, routes, h, hs)
        torch.cuda.synchronize()
        first = int(err)
        err.zero_()
        y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
        E.experts_down(h, hs, down, routes, y, space(E, E.experts_down_bytes(down, routes)))
        torch.cuda.synchronize()
        return h, hs, y, first, int(err)

    h0, hs0, y0, *errs = both(offsets, order)
    assert errs == [0, 0]
    cut = int(offsets[1])
    for bad in (-5, T * k + 1, 1 << 30):
        o = offsets.clone()
        o[0] = bad                                     # the first expert's span does not hold
        h, hs, _, *errs = both(o, order)
        assert errs == [E.DEVERR_ROUTE] * 2
        assert bool((h[:cut] == 0x55).all()) and torch.equal(h[cut:], h0[cut:]) and torch.equal(hs[cut:], hs0[cut:])
    for bad in (-1, T * k, 1 << 30, -(1 << 31)):
        p = order.clone()
        p[cut] = bad                                   # one slot of the second expert
        h, hs, y, *errs = both(offsets, p)
        assert errs == [E.DEVERR_ROUTE] * 2
        keep = torch.arange(T * k, device="cuda") != cut
        assert bool((h[cut] == 0x55).all()) and torch.equal(h[keep], h0[keep]) and torch.equal(hs[keep], hs0[keep])
        others = torch.arange(T, device="cuda") != int(order[cut]) // k
        assert torch.equal(y[others], y0[others])


# ------------------------------------------------------------------ far offsets
def test_weights_past_4_gib(E):
    g = seeded(31)
    n, I, K = 520, 1024, 4096
    w = torch.zeros(n, 2, I, K, dtype=torch.uint8, device="cuda")
    s = torch.ones(n, 2, I // 128, K // 128, device="cuda") / 4096
    last, ls = R.weights8(g, 2, 2, I, K)
    w[-2:], s[-2:] = last, ls
    for T in (2, 40):
        ids = torch.arange(T)[:, None] % 2 + n - 2
        offsets, order = R.plan(ids.numpy(), n)
        i32 = torch.int32
        routes = E.Routes(ids.to(i32).cuda(), torch.ones(T, 1, device="cuda"), torch.tensor(offsets, dtype=i32, device="cuda"),
                          torch.tensor(order, dtype=i32, device="cuda"))
        x, xs, x64 = R.rows8(g, T, K, False)
        h = torch.zeros(T, I, dtype=torch.uint8, device="cuda")
        hs = torch.zeros(T, I // 32, dtype=torch.uint8, device="cuda")
        E.experts_up(x, xs, E.F8(w, s), routes, h, hs)
        want, tol = R.up(x64, last, ls, offsets[-3:], order, 1)
        check_h(h, hs, want, tol)


def test_results_past_4_gib(E):
    g = seeded(32)
    T, K, N = 70000, 128, 32768
    w, s = R.weights8(g, N, K)
    x, xs, x64 = R.rows8(g, T, K, True)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    E.project_f8(x, E.F8(w, s), y, xs)
    for rows in (slice(0, 40), slice(T // 2, T // 2 + 40), slice(T - 40, T)):
        want, tol = R.product(x64[rows], R.matrix(w, s))
        within(y[rows], want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")


# --------------------------------------------------------- the sub-layer together
class SubLayer:
    """Norm, router, experts and the next norm, over buffers of a step."""

    def __init__(self, E, seed, T, dim=256, n=12, k=3, I=128):
        g = self.g = seeded(seed)
        self.E, self.T, self.k, self.n = E, T, k, n
        z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        bf, i32 = torch.bfloat16, torch.int32
        self.h = torch.randn(T, dim, generator=g, device="cuda")
        self.norm = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(bf)
        self.gate, self.up, self.down = (R.weights8(g, *s, spread=0.5) for s in ((n + 4, dim), (n, 2, I, dim), (n, dim, I)))
        self.bias = 0.1 * torch.randn(n, generator=g, device="cuda")
        self.w = [E.F8(*p) for p in (self.gate, self.up, self.down)]
        self.codes, self.scales = z(T, dim), z(T, dim // 32)
        self.logits = z(T, n + 4, dt=bf)
        self.routes = E.Routes(z(T, k, dt=i32), z(T, k, dt=torch.float32), z(n + 1, dt=i32), z(T * k, dt=i32), z(1, dt=i32))
        self.act, self.act_s, self.y = z(T * k, I), z(T * k, I // 32), z(T, dim, dt=bf)
        self.out, self.out_s, self.sum = z(T, dim), z(T, dim // 32), z(T, dim, dt=torch.float32)
        self.ws = [space(E, b) for b in (E.route_bytes(self.routes), E.experts_down_bytes(self.w[2], self.routes))]

    def run(self):
        E = self.E
        E.add_norm(None, self.h, self.norm, 1e-6, self.codes, self.scales)
        E.project_f8(self.codes, self.w[0], self.logits, self.scales)
        E.route(self.logits[:, :self.n], self.routes, self.bias, groups=4, top_groups=2, factor=1.5, d_ws=self.ws[0])
        E.experts_up(self.codes, self.scales, self.w[1], self.routes, self.act, self.act_s)
        E.experts_down(self.act, self.act_s, self.w[2], self.routes, self.y, self.ws[1])
        E.add_norm(self.y, self.h, self.norm, 1e-6, self.out, self.out_s, d_sum=self.sum)

    def results(self):
        return [t.clone() for t in (self.logits, *self.routes.keep[:4], self.act, self.act_s, self.y, self.out, self.out_s, self.sum)]


@pytest.mark.parametrize("T", [1, 3, 37, 300, 1500])
def test_together(E, T):
    """Each step against its 64-bit form on what the step before left."""
    L = SubLayer(E, T, T)
    L.run()
    torch.cuda.synchronize()
    x64 = A.grouped(A.e4m3(L.codes), L.scales)
    want, tol = R.product(x64, R.matrix(*L.gate))
    within(L.logits, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "logits")
    ids, weights, offsets, order = R.route(L.logits[:, :L.n].double().cpu().numpy(), L.bias.double().cpu().numpy(), L.k, False, 4, 2, 2,
                                           True, 1.5)
    got = [t.cpu().numpy() for t in L.routes.keep]
    assert np.array_equal(got[0], ids) and np.array_equal(got[2], offsets) and np.array_equal(got[3], order)
    assert np.abs(got[1] - weights).max() <= 2.0 ** -17 * 1.5 and got[4][0] == 0
    want, tol = R.up(x64, *L.up, offsets, order, L.k)
    check_h(L.act, L.act_s, want, tol)
    want, tol = R.down(A.grouped(A.e4m3(L.act), L.act_s), *L.down, offsets, order, L.routes.keep[1])
    within(L.y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")
    assert torch.equal(L.sum, L.h + L.y.float())


@pytest.mark.parametrize("T", [1, 50, 300])
def test_captured(E, T):
    """A step captured into a graph and replayed on new tokens, with work of the
    program's own between the replays, gives the eager step's bits."""
    L = SubLayer(E, T + 5, T)
    L.run()                                            # (code is loaded before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run()
    for i in range(4):
        L.h.copy_(torch.randn(L.h.shape, generator=L.g, device="cuda") * (i + 1))
        L.run()
        eager = L.results()
        for t in (L.logits, L.y, L.out, L.act):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, L.results()):
            assert torch.equal(a, b)


def test_two_streams(E):
    """Two steps side by side, each with its own buffers on a stream of its own,
    and repeated: the bits of the step alone."""
    steps = [SubLayer(E, 40 + i, T) for i, T in enumerate((64, 700))]
    alone = []
    for L in steps:
        L.run()
        torch.cuda.synchronize()
        alone.append(L.results())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for L, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                L.run()
    torch.cuda.synchronize()
    for L, want in zip(steps, alone):
        assert all(torch.equal(a, b) for a, b in zip(want, L.results()))


def test_stream_argument(E):
    """A call goes to the stream it is given, not to the current one."""
    L = SubLayer(E, 50, 30)
    L.run()
    torch.cuda.synchronize()
    want = L.results()
    stream = torch.cuda.Stream()
    h = L.h.clone()
    L.h.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        L.h.copy_(h)
        E.add_norm(None, L.h, L.norm, 1e-6, L.codes, L.scales)
    E.project_f8(L.codes, L.w[0], L.logits, L.scales, stream=stream)
    E.route(L.logits[:, :L.n], L.routes, L.bias, groups=4, top_groups=2, factor=1.5, d_ws=L.ws[0], stream=stream.cuda_stream)
    E.experts_up(L.codes, L.scales, L.w[1], L.routes, L.act, L.act_s, stream=stream)
    E.experts_down(L.act, L.act_s, L.w[2], L.routes, L.y, L.ws[1], stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[:8], L.results()[:8]))


@pytest.mark.parametrize("T", [4096, 4097])
def test_route_blocks(E, T):
    g = seeded(T)
    check_route(E, torch.randn(T, 12, generator=g, device="cuda"), None, 2, True)


# ------------------------------------------------- group sums at the ends of f32
LOWEST, MOST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("n,groups,top,k", [(8, 4, 2, 3), (48, 6, 2, 6), (256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 3, 5)])
def test_route_lowest_bias(E, n, groups, top, k, softmax):
    """Biases of the type's lowest or largest value are values: the experts stay
    open, and two such keys of a group add up to what f32 cannot hold."""
    g = seeded(n + groups)
    x = torch.randn(70, n, generator=g, device="cuda")
    size = n // groups
    for large in (LOWEST, MOST):
        for first in (2, size, size + 1, n - 1):       # the experts from here on
            bias = 0.1 * torch.randn(n, generator=g, device="cuda")
            bias[first:] = large
            for best in (1, 2):
                check_route(E, x, bias, k, softmax, groups, top, best, what=f"{large} from {first} on, best {best}")
        bias = 0.1 * torch.randn(n, generator=g, device="cuda")
        bias[::2] = large                              # one key of a group, against the other's own size
        check_route(E, x, bias, k, softmax, groups, top, 2, what=f"{large} at every second")
        bias[1::2] = -large                            # sums near zero
        check_route(E, x, bias, k, softmax, groups, top, 2, what=f"{large} and its negative")


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("size", [64.0, 1000.0, 1e5])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_group_sums_that_cancel(E, size, softmax, bf16):
    """Groups whose two keys are large and of opposite signs: what their sum keeps
    is as far off as the keys' own rounding, however small it is."""
    log(f"groups of two, biases of +-{size} softmax {softmax} bf16 {bf16}")
    g = seeded(int(size))
    T, n, k, top = 150000, 16, 3, 4
    x = torch.randn(T, n, generator=g, device="cuda")
    x = x.bfloat16() if bf16 else x
    bias = 0.1 * torch.randn(n, generator=g, device="cuda")
    bias[::2] += size
    bias[1::2] -= size
    r = new_routes(E, T, n, k)
    E.route(x, r, bias, softmax, n // 2, top, 2, d_ws=space(E, E.route_bytes(r)))
    got = r.keep[0].cpu().numpy()
    x, b = x.double().cpu().numpy(), bias.double().cpu().numpy()
    score = np.exp(x - x.max(1, keepdims=True))
    score = score / score.sum(1, keepdims=True) if softmax else 1 / (1 + np.exp(-x))
    key = score + b
    sums = key[:, ::2] + key[:, 1::2]
    kept = np.zeros(sums.shape, dtype=bool)
    np.put_along_axis(kept, np.argsort(-sums, 1, kind="stable")[:, :top], True, 1)
    key[~kept.repeat(2, 1)] = -INF
    want = np.argsort(-key, 1, kind="stable")[:, :k]
    assert np.array_equal(got, want), f"ids differ in {(got != want).any(1).sum()} tokens"


# ----------------------------------------- few rows: every number of outputs a workgroup
# 32, 48, 64 and 80 outputs a workgroup (of 256 CUs) over up to 16 and up to 32 rows; last
# workgroups part filled, workgroups that meet two blocks of scales, last blocks of 16 outputs
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,K,N", [(1, 256, 8208), (3, 384, 12304), (16, 1152, 16400), (16, 640, 20480), (9, 128, 20496),
                                   (17, 384, 8208), (19, 128, 12272), (24, 896, 12304), (32, 384, 16400), (32, 256, 20496),
                                   (31, 1152, 20480), (1, 2048, 40976), (20, 256, 41008)])
def test_project_f8_few_rows(E, T, K, N, f32):
    log(f"project_f8 T {T} K {K} N {N} f32 {f32}")
    g = seeded(T + K + N)
    w, s = R.weights8(g, N, K)
    x, xs, x64 = R.rows8(g, T, K, f32)
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    E.project_f8(x, E.F8(w, s), y[:T], xs)
    torch.cuda.synchronize()
    want, tol = R.product(x64, R.matrix(w, s))
    within(y[:T], want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")
    assert bool((y[T] == 7).all()), "a row past the last is written"


# ---------------------------------------------- tiles over more than 64 experts
def many_counts(n, rows):
    """Rows of n experts, `rows` on average at least, some experts without any
    where the experts are looked through 64 at a time."""
    counts = np.random.default_rng(n + rows).integers(rows // 2, 2 * rows, n)
    counts[[e for e in (0, 63, 64, 128, 129, 191, 255) if e < n - 1]] = 0
    counts[-1] += max(0, rows * n - int(counts.sum()))
    return counts.tolist()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows", [9, 64, 192])
@pytest.mark.parametrize("n", [65, 130, 256])
def test_experts_many_rows(E, n, rows, f32):
    """Every tile height, the rows found across several 64s of experts."""
    log(f"{n} experts of {rows} rows f32 {f32}")
    g = seeded(n + rows)
    arrays, offsets, order = counted_plan(g, many_counts(n, rows))
    check_experts(E, g, arrays, offsets, order, n, 256, 128, 144, f32)


@pytest.mark.parametrize("T", [3, 40, 8400])
def test_down_weights_past_4_gib(E, T):
    """In one launch, through few rows and through tiles."""
    log(f"experts_down past 4 GiB T {T}")
    g = seeded(T)
    n, N, K = 520, 2048, 4096
    w = torch.zeros(n, N, K, dtype=torch.uint8, device="cuda")
    s = torch.ones(n, N // 128, K // 128, device="cuda") / 4096
    w[-2:], s[-2:] = R.weights8(g, 2, N, K)
    ids = torch.arange(T)[:, None] % 2 + n - 2
    offsets, order = R.plan(ids.numpy(), n)
    i32 = torch.int32
    arrays = (ids.to(i32).cuda(), torch.rand(T, 1, generator=g, device="cuda"), torch.tensor(offsets, dtype=i32, device="cuda"),
              torch.tensor(order, dtype=i32, device="cuda"))
    routes, down = E.Routes(*arrays), E.F8(w, s)
    h, hs, h64 = R.rows8(g, T, K, False)
    y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    E.experts_down(h, hs, down, routes, y, space(E, E.experts_down_bytes(down, routes)))
    want, tol = R.down(h64, w[-2:], s[-2:], offsets[-3:], order, arrays[1])
    within(y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")


def test_up_weights_past_4_gib_in_tiles(E):
    log("experts_up past 4 GiB in tiles")
    g = seeded(33)
    n, I, K, T = 520, 1024, 4096, 4200
    w = torch.zeros(n, 2, I, K, dtype=torch.uint8, device="cuda")
    s = torch.ones(n, 2, I // 128, K // 128, device="cuda") / 4096
    w[-2:], s[-2:] = R.weights8(g, 2, 2, I, K)
    ids = torch.arange(T)[:, None] % 2 + n - 2
    offsets, order = R.plan(ids.numpy(), n)
    i32 = torch.int32
    routes = E.Routes(ids.to(i32).cuda(), torch.ones(T, 1, device="cuda"), torch.tensor(offsets, dtype=i32, device="cuda"),
                      torch.tensor(order, dtype=i32, device="cuda"))
    x, xs, x64 = R.rows8(g, T, K, False)
    h = torch.zeros(T, I, dtype=torch.uint8, device="cuda")
    hs = torch.zeros(T, I // 32, dtype=torch.uint8, device="cuda")
    E.experts_up(x, xs, E.F8(w, s), routes, h, hs)
    want, tol = R.up(x64, w[-2:], s[-2:], offsets[-3:], order, 1)
    check_h(h, hs, want, tol)


# --------------------------------------------------------- products that cancel
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,n,N", [(1, 4, 64), (8, 4, 2048), (2, 4, 64), (5, 4, 144), (9, 6, 2048), (40, 12, 272), (300, 90, 80)])
def test_down_products_that_cancel(E, T, n, N, f32):
    """A token's two experts have the same codes under scales that differ by 2^-9,
    and its weights are each other's negatives: what is left is as good as f32's
    products for calls of few rows, of one launch or of two."""
    log(f"experts_down, cancelling T {T} experts {n} N {N} f32 {f32}")
    g = seeded(T + n)
    K = 512
    assert 2 * T // n < 8
    ids = 2 * (torch.arange(T) % (n // 2))[:, None] + torch.arange(2)
    offsets, order = R.plan(ids.numpy(), n)
    first = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    weights = torch.cat((first, -first), 1).contiguous()
    i32 = torch.int32
    arrays = (ids.to(i32).cuda(), weights, *(torch.tensor(v, dtype=i32, device="cuda") for v in (offsets, order)))
    w, s = R.weights8(g, n, N, K)
    w[1::2], s[1::2] = w[::2], s[::2] * (1 + 2.0 ** -9)
    h, hs, h64 = (v[torch.as_tensor(order, device="cuda") // 2].contiguous() for v in R.rows8(g, T, K, f32))
    y = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    down, routes = E.F8(w, s), E.Routes(*arrays)
    E.experts_down(h, hs, down, routes, y, space(E, E.experts_down_bytes(down, routes)))
    want = torch.zeros(T, N, dtype=F64, device="cuda")
    tol = torch.zeros_like(want)
    place = np.argsort(order)
    for t in range(T):
        e = 2 * (t % (n // 2))
        x = h64[place[2 * t]:place[2 * t] + 1]
        (v, d), (u, _) = (R.product(x, R.matrix(w[i], s[i])) for i in (e, e + 1))
        size = x.abs() @ R.matrix(w[e], s[e]).abs().t()
        want[t] = (v - u)[0] * first[t].double()
        # the sums of a block are the same but for a power of two, so that what they are
        # off by cancels as they do; the block's factors, the sums over K / 128 blocks, the
        # weights and the sum of two are rounded in f32, each for two products
        tol[t] = (2.0 ** -8 * d[0] + 2 * (K / 128 + 4) * 2.0 ** -24 * size[0]) * first[t].double()
    within(y, want, 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * tol, "y")


# ------------------------------------------------- what a block's sum keeps
def cut_sums(x, w):
    """Sums of products of e4m3 values as the 8-bit matrix instruction forms
    them: the products of eight neighbours are cut towards zero below 2^-13 of
    the largest one's power of two (the operands' exponents added), then
    everything is added in f32 (here exactly).  And the sums of their sizes."""
    (T, K), N = x.shape, w.shape[0]
    low = torch.full((), -1000.0, dtype=F64, device=x.device)
    ex, ew = (torch.where(v == 0, low, v.abs().clamp(min=2.0 ** -6).log2().floor()) for v in (x, w))
    p = (x[:, None, :] * w[None]).view(T, N, K // 8, 8)
    top = (ex[:, None, :] + ew[None]).view(T, N, K // 8, 8).amax(-1, keepdim=True)
    unit = torch.exp2(top.clamp(min=-100) - 13)
    cut = torch.trunc(p / unit) * unit
    assert bool(((cut - p).sum(-1).abs() <= 7 * 2.0 ** -13 * torch.exp2(top.squeeze(-1))).all())
    return cut.sum((-1, -2)), p.abs().sum((-1, -2))


@pytest.mark.parametrize("spread", [0, 8, 14])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T", [3, 20, 40, 130])
def test_project_f8_sums(E, T, f32, spread):
    """What a sum keeps beside large values that cancel, of few rows and in tiles:
    what the instruction does, whatever the rows' scales."""
    log(f"sums T {T} f32 {f32} spread {spread}")
    g = seeded(spread + T)
    K, N = 256, 128
    x, w = (torch.randn(n, K, generator=g, device="cuda") for n in (T, N))
    x *= torch.exp2(torch.rand(T, K, generator=g, device="cuda") * spread - spread + 6)
    x[:, 0::8] = x[:, 1::8] = 448                       # the first two of every eight cancel
    w = w * 60
    w[:, 0::8], w[:, 1::8] = 400, -400
    x, w = (v.clamp(-448, 448).to(torch.float8_e4m3fn) for v in (x, w))
    want, size = cut_sums(x.to(F64), w.to(F64))
    xs = torch.ones(T, K // 128, device="cuda") if f32 else torch.full((T, K // 32), 127, dtype=torch.uint8, device="cuda")
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    E.project_f8(x.view(torch.uint8), E.F8(w.view(torch.uint8), torch.ones(1, K // 128, device="cuda")), y, xs)
    within(y, want, 2.0 ** -8 * want.abs() + K * 2.0 ** -24 * size, "y")


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("softmax", [False, True])
def test_route_small_scores(E, softmax, renorm):
    """Scores near and below f32's normal numbers, chosen beside larger ones."""
    g = seeded(41)
    T = 400
    depth = torch.rand(T, 1, generator=g, device="cuda") * 70
    x = torch.full((T, 8), -INF, device="cuda")
    x[:, 1] = 0.3
    x[:, 4:7] = -torch.rand(T, 3, generator=g, device="cuda") * 50 - 45 - depth
    check_route(E, x, None, 4, softmax, renorm=renorm, what="beside one of a common size")
    bias = torch.zeros(8, device="cuda")
    bias[4:] = 5                                       # the second group is kept, the first has the largest score
    x = torch.rand(T, 8, generator=g, device="cuda")
    x[:, 4:] = -torch.sort(torch.rand(T, 4, generator=g, device="cuda"), 1).values * 50 - 50 * torch.rand(T, 1, generator=g, device="cuda")
    check_route(E, x, bias, 4, softmax, 2, 1, 1, renorm=renorm, what="all small")


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("n,groups,top", [(256, 4, 2), (512, 32, 11), (65, 13, 2), (64, 16, 5), (60, 12, 7), (3, 3, 1)])
def test_route_equal_scores_of_groups(E, n, groups, top, softmax):
    """A group's one best score, without a bias: logits that differ and whose scores
    are one number of 64 bits, among equal logits, go by the group's index."""
    g = seeded(n + top)
    T, size = 300, n // groups
    whole = torch.randint(0, 6, (T, n), generator=g, device="cuda").float()
    for what, x in (("tiny", whole * 1e-30), ("about 0.5", 0.5 + whole * 2.0 ** -24), ("sigmoids of 1", 40 + whole),
                    ("vanishing", -2000 - 100 * whole), ("lowest", torch.where(whole < 3, whole * 1e30 - 3e38, -whole))):
        if what == "vanishing":
            x[:, 0] = 0                                # (a softmax's largest)
        for v in (x, x.bfloat16()):
            check_route(E, v, None, min(5, size), softmax, groups, top, 1, what=what)
