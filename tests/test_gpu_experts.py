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
