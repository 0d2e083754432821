"""The experts' entry points on the host, without a GPU: what they refuse,
before any launch (fake device addresses are never read)."""
import ctypes
import os

import pytest

import gram_hashed_embedding_engram_amd as E

torch = pytest.importorskip("torch")

FAKE = 0x7F0000000000          # 256-byte aligned stand-ins for device memory, far apart
OUT, IDS, WTS, OFF, ORD, WS, SC = (FAKE + (i << 40) for i in range(1, 8))
HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "engram.h")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(E.LIB_PATH):
        import gram_hashed_embedding_engram_amd.build as B
        B.build()
    return E.lib()


def test_constants(L):
    text = open(HEADER).read()
    assert "#define ENGRAM_F8_BLOCK %d" % E.F8_BLOCK in text
    assert "#define ENGRAM_DEVERR_ROUTE %d " % E.DEVERR_ROUTE in text


def routes_c(**k):
    a = dict(experts=64, chosen=4, tokens=6, d_ids=IDS, d_weights=WTS, d_offsets=OFF, d_order=ORD, d_err=None)
    a.update(k)
    return E.RoutesC(**a)


def f8(L, **k):
    a = dict(x=FAKE, xs=SC, f32=0, w=WS, ws=WS, y=OUT, T=4, K=256, N=64)
    a.update(k)
    return L.engram_project_f8(*a.values(), None)


def route(L, routes=None, **k):
    a = dict(x=FAKE, bf16=0, stride=64, bias=None, softmax=0, groups=1, top=1, best=2, renorm=1, factor=1.0, ws=WS,
             nws=1 << 40)
    a.update(k)
    return L.engram_route(ctypes.byref(routes or routes_c()), *a.values(), None)


def up(L, routes=None, **k):
    a = dict(x=FAKE, xs=SC, f32=0, w=WS, ws=WS, h=OUT, hs=OUT + (1 << 38), K=256, I=128)
    a.update(k)
    return L.engram_experts_up(ctypes.byref(routes or routes_c()), *a.values(), None)


def down(L, routes=None, **k):
    a = dict(h=FAKE, hs=SC, f32=0, w=WS, ws=WS, y=OUT, K=256, N=64, space=WS, n=1 << 40)
    a.update(k)
    return L.engram_experts_down(ctypes.byref(routes or routes_c()), *a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), E.E_ARG), (dict(T=(1 << 22) + 1), E.E_RANGE), (dict(K=0), E.E_UNSUPPORTED),
    (dict(K=192), E.E_UNSUPPORTED), (dict(K=(1 << 20) + 128), E.E_UNSUPPORTED),
    (dict(K=-128), E.E_UNSUPPORTED), (dict(N=0), E.E_UNSUPPORTED), (dict(N=24), E.E_UNSUPPORTED),
    (dict(N=(1 << 24) + 16), E.E_UNSUPPORTED), (dict(x=None), E.E_ARG), (dict(xs=None), E.E_ARG),
    (dict(w=None), E.E_ARG), (dict(ws=None), E.E_ARG), (dict(y=None), E.E_ARG), (dict(x=FAKE + 8), E.E_ARG),
    (dict(w=FAKE + 8), E.E_ARG), (dict(xs=SC + 2), E.E_ARG), (dict(ws=WS + 1), E.E_ARG), (dict(y=OUT + 4), E.E_ARG)])
def test_f8_refusals(L, change, code):
    assert f8(L, **change) == code and E.last_error()


BAD_ROUTES = [(dict(tokens=-1), E.E_ARG), (dict(tokens=(1 << 22) + 1), E.E_RANGE), (dict(experts=0), E.E_UNSUPPORTED),
              (dict(experts=1025), E.E_UNSUPPORTED), (dict(chosen=0), E.E_UNSUPPORTED), (dict(chosen=33), E.E_UNSUPPORTED),
              (dict(experts=3, chosen=4), E.E_UNSUPPORTED), (dict(tokens=1 << 22, chosen=8), E.E_RANGE),
              (dict(d_ids=None), E.E_ARG), (dict(d_weights=None), E.E_ARG), (dict(d_offsets=None), E.E_ARG),
              (dict(d_order=None), E.E_ARG), (dict(d_ids=IDS + 2), E.E_ARG), (dict(d_weights=WTS + 1), E.E_ARG),
              (dict(d_offsets=OFF + 2), E.E_ARG), (dict(d_order=ORD + 2), E.E_ARG), (dict(d_err=IDS + 2), E.E_ARG)]


@pytest.mark.parametrize("call", [route, up, down])
@pytest.mark.parametrize("change,code", BAD_ROUTES)
def test_routes_refusals(L, call, change, code):
    more = dict(stride=1 << 20) if call is route else {}
    assert call(L, routes_c(**change), **more) == code and E.last_error()


@pytest.mark.parametrize("change,code", [
    (dict(groups=0), E.E_UNSUPPORTED), (dict(groups=3), E.E_UNSUPPORTED), (dict(groups=128), E.E_UNSUPPORTED),
    (dict(groups=4, top=5), E.E_ARG), (dict(top=0), E.E_ARG), (dict(best=0), E.E_UNSUPPORTED),
    (dict(best=3), E.E_UNSUPPORTED), (dict(factor=float("nan")), E.E_ARG), (dict(factor=float("inf")), E.E_ARG),
    (dict(stride=63), E.E_ARG), (dict(stride=-64), E.E_ARG), (dict(stride=1 << 41), E.E_ARG), (dict(x=None), E.E_ARG),
    (dict(x=FAKE + 2), E.E_ARG), (dict(x=FAKE + 1, bf16=1), E.E_ARG), (dict(bias=FAKE + 2), E.E_ARG)])
def test_route_refusals(L, change, code):
    assert route(L, **change) == code and E.last_error()


def test_workspace_refusals(L):
    many = routes_c(tokens=1000)
    need = L.engram_route_bytes(ctypes.byref(many))
    assert need > 0 and L.engram_route_bytes(ctypes.byref(routes_c(tokens=64))) == 0
    assert route(L, many, nws=need - 1) == E.E_RANGE and E.last_error()
    assert route(L, many, ws=None, nws=need) == E.E_ARG
    assert route(L, many, ws=WS + 16, nws=need) == E.E_ARG
    need = L.engram_experts_down_bytes(ctypes.byref(many), 64)
    assert need > 0
    assert down(L, many, n=need - 1) == E.E_RANGE and E.last_error()
    assert down(L, many, space=None, n=need) == E.E_ARG
    assert down(L, many, space=WS + 16, n=need) == E.E_ARG
    for bad in (routes_c(experts=0), routes_c(tokens=-1), routes_c(tokens=0)):
        assert L.engram_route_bytes(ctypes.byref(bad)) == 0
        assert L.engram_experts_down_bytes(ctypes.byref(bad), 64) == 0
    assert L.engram_experts_down_bytes(ctypes.byref(many), 24) == 0


@pytest.mark.parametrize("change,code", [
    (dict(K=192), E.E_UNSUPPORTED), (dict(K=0), E.E_UNSUPPORTED), (dict(I=192), E.E_UNSUPPORTED),
    (dict(I=(1 << 20) + 128), E.E_UNSUPPORTED), (dict(x=None), E.E_ARG), (dict(xs=None), E.E_ARG),
    (dict(w=None), E.E_ARG), (dict(ws=None), E.E_ARG), (dict(h=None), E.E_ARG), (dict(hs=None), E.E_ARG),
    (dict(x=FAKE + 8), E.E_ARG), (dict(w=FAKE + 8), E.E_ARG), (dict(xs=SC + 2), E.E_ARG), (dict(ws=WS + 2), E.E_ARG),
    (dict(h=OUT + 8), E.E_ARG), (dict(hs=OUT + 2), E.E_ARG)])
def test_up_refusals(L, change, code):
    assert up(L, **change) == code and E.last_error()


@pytest.mark.parametrize("change,code", [
    (dict(K=192), E.E_UNSUPPORTED), (dict(K=-128), E.E_UNSUPPORTED), (dict(N=24), E.E_UNSUPPORTED),
    (dict(N=0), E.E_UNSUPPORTED), (dict(h=None), E.E_ARG), (dict(hs=None), E.E_ARG), (dict(w=None), E.E_ARG),
    (dict(ws=None), E.E_ARG), (dict(y=None), E.E_ARG), (dict(h=FAKE + 8), E.E_ARG), (dict(w=FAKE + 8), E.E_ARG),
    (dict(hs=SC + 2), E.E_ARG), (dict(ws=WS + 2), E.E_ARG), (dict(y=OUT + 8), E.E_ARG)])
def test_down_refusals(L, change, code):
    assert down(L, **change) == code and E.last_error()


def test_sizes_past_32_bits(L):
    """Rows that a product's 32-bit offsets could not reach are refused."""
    assert up(L, routes_c(tokens=1 << 21, chosen=1), K=1024) == E.E_RANGE and E.last_error()


def test_outputs_over_inputs_are_refused(L):
    for shift in (-248, 0, 8, 504):
        assert f8(L, y=FAKE + 2 * shift) == E.E_ARG and "overlap" in E.last_error()
        assert f8(L, y=SC + 16 * (shift > 0)) == E.E_ARG and "overlap" in E.last_error()
        assert down(L, y=FAKE + 2 * shift) == E.E_ARG and "overlap" in E.last_error()
    for name in ("h", "hs"):
        assert up(L, **{name: FAKE + 16}) == E.E_ARG and "overlap" in E.last_error()
        assert up(L, **{name: SC + 16}) == E.E_ARG and "overlap" in E.last_error()
    for name in ("d_ids", "d_weights", "d_offsets", "d_order"):
        assert route(L, routes_c(**{name: FAKE + 64})) == E.E_ARG and "overlap" in E.last_error()


def test_workspaces_over_other_arrays_are_refused(L):
    """A workspace that reaches into the rows, the results or the routes, and h
    that reaches into its scales."""
    many = routes_c(tokens=1000)
    need = L.engram_route_bytes(ctypes.byref(many))
    for at in (FAKE, IDS, WTS, OFF, ORD):
        assert route(L, many, ws=at, nws=need) == E.E_ARG and "workspace overlaps" in E.last_error()
    need = L.engram_experts_down_bytes(ctypes.byref(many), 64)
    for at in (FAKE, SC, OUT):
        assert down(L, many, space=at, n=need) == E.E_ARG and "workspace overlaps" in E.last_error()
    assert up(L, hs=OUT + 64) == E.E_ARG and "overlaps" in E.last_error()


def test_empty_calls_touch_nothing(L):
    none = routes_c(tokens=0, d_ids=None, d_weights=None, d_offsets=None, d_order=None)
    assert f8(L, T=0, x=None, xs=None, w=None, ws=None, y=None) == E.OK
    assert route(L, none, x=None, ws=None, nws=0) == E.OK
    assert up(L, none, x=None, xs=None, w=None, ws=None, h=None, hs=None) == E.OK
    assert down(L, none, h=None, hs=None, w=None, ws=None, y=None, space=None, n=0) == E.OK


Z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
F32, I32, BF = torch.float32, torch.int32, torch.bfloat16


def some():
    routes = E.Routes(Z(6, 2, dt=I32), Z(6, 2, dt=F32), Z(5, dt=I32), Z(12, dt=I32))
    return (routes, E.F8(Z(64, 256), Z(1, 2, dt=F32)), E.F8(Z(4, 2, 128, 256), Z(4, 2, 1, 2, dt=F32)),
            E.F8(Z(4, 208, 256), Z(4, 2, 2, dt=F32)))


def test_binding_refusals():
    """Types, shapes and views the binding sees and the library cannot."""
    routes, w, w_up, w_down = some()
    x, s8, s32, y = Z(6, 256), Z(6, 8), Z(6, 2, dt=F32), Z(6, 64, dt=BF)
    h, hs, k8 = Z(12, 128), Z(12, 4), Z(12, 256)
    calls = [
        lambda: E.F8(Z(64, 256, dt=F32), Z(1, 2, dt=F32)), lambda: E.F8(Z(64, 256), Z(1, 2)),
        lambda: E.F8(Z(144, 256), Z(1, 2, dt=F32)), lambda: E.F8(Z(4, 64, 256), Z(1, 2, dt=F32)),
        lambda: E.F8(Z(256, 64).t(), Z(1, 2, dt=F32)),
        lambda: E.Routes(Z(6, 2), Z(6, 2, dt=F32), Z(5, dt=I32), Z(12, dt=I32)),
        lambda: E.Routes(Z(6, 2, dt=I32), Z(6, 3, dt=F32), Z(5, dt=I32), Z(12, dt=I32)),
        lambda: E.Routes(Z(6, 2, dt=I32), Z(6, 2, dt=F32), Z(1, dt=I32), Z(12, dt=I32)),
        lambda: E.Routes(Z(6, 2, dt=I32), Z(6, 2, dt=F32), Z(5, dt=I32), Z(11, dt=I32)),
        lambda: E.Routes(Z(2, 6, dt=I32).t(), Z(6, 2, dt=F32), Z(5, dt=I32), Z(12, dt=I32)),
        lambda: E.Routes(Z(6, 2, dt=I32), Z(6, 2, dt=F32), Z(5, dt=I32), Z(12, dt=I32), Z(0, dt=I32)),
        lambda: E.project_f8(x, w_down, y, s8), lambda: E.project_f8(x.float(), w, y, s8),
        lambda: E.project_f8(x, w, y, Z(6, 4)), lambda: E.project_f8(x, w, y, Z(6, 8, dt=F32)),
        lambda: E.project_f8(x, w, Z(6, 60, dt=BF), s8), lambda: E.project_f8(x, w, y.float(), s8),
        lambda: E.project_f8(Z(6, 512)[:, ::2], w, y, s8), lambda: E.project_f8(x, w, y, Z(6, 16)[:, ::2]),
        lambda: E.route(Z(6, 5, dt=F32), routes), lambda: E.route(Z(6, 4), routes),
        lambda: E.route(Z(4, 6, dt=F32).t(), routes), lambda: E.route(Z(6, 4, dt=F32), routes, Z(4, dt=BF)),
        lambda: E.route(Z(6, 4, dt=F32), routes, Z(5, dt=F32)), lambda: E.route(Z(6, 4, dt=F32), routes, d_ws=Z(4, dt=F32)),
        lambda: E.experts_up(x, s8, w, routes, h, hs), lambda: E.experts_up(x, s8, w_down, routes, h, hs),
        lambda: E.experts_up(Z(5, 256), s8, w_up, routes, h, hs), lambda: E.experts_up(x, s8, w_up, routes, Z(6, 128), hs),
        lambda: E.experts_up(x, s8, w_up, routes, h, Z(12, 1)), lambda: E.experts_up(x, s8, w_up, routes, h, Z(12, 4, dt=F32)),
        lambda: E.experts_down(k8, Z(12, 8), w_up, routes, Z(6, 208, dt=BF)),
        lambda: E.experts_down(Z(6, 256), Z(6, 8), w_down, routes, Z(6, 208, dt=BF)),
        lambda: E.experts_down(k8, Z(12, 8), w_down, routes, Z(6, 200, dt=BF)),
        lambda: E.experts_down(k8, Z(12, 8), w_down, routes, Z(6, 208, dt=BF), Z(8, dt=F32))]
    for i, call in enumerate(calls):
        with pytest.raises(E.EngramError):
            call()
            pytest.fail(f"call {i} is not refused")


def test_host_tensors_are_refused():
    """A tensor in host memory, right in type and shape, ends in the binding."""
    routes, w, w_up, w_down = some()
    assert (routes.host, w.host) == ("ids", "w")
    x, s8, h, hs = Z(6, 256), Z(6, 8), Z(12, 128), Z(12, 4)
    calls = [lambda: E.project_f8(x, w, Z(6, 64, dt=BF), s8, stream=0),
             lambda: E.project_f8(x, w, Z(6, 64, dt=BF), Z(6, 2, dt=F32), stream=0),
             lambda: E.route(Z(6, 4, dt=F32), routes, Z(4, dt=F32), stream=0),
             lambda: E.experts_up(x, s8, w_up, routes, h, hs, stream=0),
             lambda: E.experts_down(Z(12, 256), Z(12, 8), w_down, routes, Z(6, 208, dt=BF), stream=0)]
    for call in calls:
        with pytest.raises(E.EngramError, match="on the GPU is needed"):
            call()
    for kept in (routes, w, w_up, w_down):
        kept.host = None
    for call in calls:
        with pytest.raises(E.EngramError, match="on the GPU is needed"):
            call()


def test_other_device_is_refused(monkeypatch):
    """Tensors that are not on the device whose stream a call would use."""
    monkeypatch.setattr(E, "_device", lambda: 1)
    with pytest.raises(E.EngramError, match="current one is 1"):
        E._here(0)
    E._here(1)
    with pytest.raises(E.EngramError, match="not on the call's device"):
        E._same_device(1, x=type("T", (), dict(is_cuda=True, device="cuda:0", get_device=lambda self: 0))())


# addresses of their own for every array of a call, far apart
FAR = {name: FAKE + ((16 + i) << 44) for i, name in enumerate(
    ("x", "xs", "w", "ws", "y", "h", "hs", "space", "logits", "bias", "d_ids", "d_weights", "d_offsets", "d_order", "d_err"))}
PLAN = ("d_ids", "d_weights", "d_offsets", "d_order")


def far_call(L, op, moved, T=1000, k=4, n=64, K=256, I=256, N=208, f32=0):
    """A call whose arrays are far apart but for those in `moved`."""
    at = dict(FAR, **moved)
    r = routes_c(experts=n, chosen=k, tokens=T, **{name: at[name] for name in (*PLAN, "d_err")})
    ref = ctypes.byref(r)
    if op == "route":
        return L.engram_route(ref, at["logits"], 0, n, at["bias"], 0, 1, 1, 2, 1, 1.0, at["space"],
                              L.engram_route_bytes(ref), None)
    if op == "f8":
        return L.engram_project_f8(at["x"], at["xs"], f32, at["w"], at["ws"], at["y"], T, K, N, None)
    if op == "up":
        return L.engram_experts_up(ref, at["x"], at["xs"], f32, at["w"], at["ws"], at["h"], at["hs"], K, I, None)
    return L.engram_experts_down(ref, at["x"], at["xs"], f32, at["w"], at["ws"], at["y"], K, N, at["space"],
                                 L.engram_experts_down_bytes(ref, N), None)


def far_bytes(L, op, T=1000, k=4, n=64, K=256, I=256, N=208, f32=0):
    """(what a call writes, what it reads), with their sizes."""
    R, width = T * k, (lambda v: v // 128 * 4 if f32 else v // 32)
    r = routes_c(experts=n, chosen=k, tokens=T)
    plan = dict(d_ids=4 * R, d_weights=4 * R, d_offsets=4 * (n + 1), d_order=4 * R)
    err = dict(d_err=4)
    if op == "route":
        return dict(space=L.engram_route_bytes(ctypes.byref(r)), **plan, **err), dict(logits=4 * T * n, bias=4 * n)
    if op == "f8":
        return dict(y=2 * T * N), dict(x=T * K, xs=T * width(K), w=N * K, ws=2 * (K // 128) * 4)
    if op == "up":
        return (dict(h=R * I, hs=R * I // 32, **err),
                dict(x=T * K, xs=T * width(K), w=n * 2 * I * K, ws=n * 2 * (I // 128) * (K // 128) * 4, **plan))
    return (dict(space=L.engram_experts_down_bytes(ctypes.byref(r), N), y=2 * T * N, **err),
            dict(x=R * K, xs=R * width(K), w=n * N * K, ws=n * 2 * (K // 128) * 4, **plan))


@pytest.mark.parametrize("f32", [0, 1])
@pytest.mark.parametrize("op", ["route", "f8", "up", "down"])
def test_every_overlap_is_refused(L, op, f32):
    """What a call writes, over the first and over the last bytes of everything
    else of the call."""
    writes, reads = far_bytes(L, op, f32=f32)
    assert all(writes.values()) and all(reads.values())
    for out, size in writes.items():
        for other, theirs in {**reads, **writes}.items():
            if other == out:
                continue
            last = (theirs - 1) // 256 * 256           # the last aligned place in it
            for place in {0, last, -(size - 1) // 256 * 256}:
                start = FAR[other] + place
                if start + size <= FAR[other]:
                    continue
                assert far_call(L, op, {out: start}, f32=f32) == E.E_ARG, (op, out, other, place)
                assert "overlaps" in E.last_error(), (op, out, other, place, E.last_error())


@pytest.mark.parametrize("op", ["route", "up", "down"])
def test_neighbours_are_not_refused(L, op):
    """An array right behind another: only the error word, which lies in the
    plan's order, ends such a call."""
    writes, reads = far_bytes(L, op)
    for out in writes:
        for other, theirs in {**reads, **writes}.items():
            if out in (other, "d_err") or other == "d_err":
                continue
            start = FAR[other] + (theirs + 255) // 256 * 256
            moved = {out: start, "d_err": FAR["d_order"] + 400}
            if out == "d_order":
                moved["d_err"] = start + 400
            assert far_call(L, op, moved) == E.E_ARG and "error word" in E.last_error(), (op, out, other)


def test_a_workspace_serves_fewer_tokens(L):
    """A workspace made for a call of the most tokens is enough for any call of
    fewer: what a call needs does not fall as tokens are added."""
    steps = sorted({*range(1, 1300), *(64 * i + d for i in range(1, 400) for d in (-1, 0, 1)), 40000, 300000, 1 << 20})
    for n, k in ((1, 1), (4, 2), (60, 4), (256, 8), (1024, 32)):
        for need in (lambda r: L.engram_route_bytes(ctypes.byref(r)), lambda r: L.engram_experts_down_bytes(ctypes.byref(r), 64),
                     lambda r: L.engram_experts_down_bytes(ctypes.byref(r), 4112)):
            last = (0, 0)
            for T in steps:
                if T * k > 1 << 24:
                    break
                now = need(routes_c(experts=n, chosen=k, tokens=T))
                assert now >= last[1], f"{n} experts, {k} a token: {T} tokens need {now} bytes, {last[0]} {last[1]}"
                last = (T, now)
