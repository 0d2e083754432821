"""The attention sub-layer's entry points on the host, without a GPU: what
they refuse, before any launch (fake device addresses are never read)."""
import ctypes
import os
import subprocess

import pytest

import gram_hashed_embedding_engram_amd as E

torch = pytest.importorskip("torch")

FAKE = 0x7F0000000000          # 256-byte aligned stand-in for device memory
HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "engram.h")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(E.LIB_PATH):
        import gram_hashed_embedding_engram_amd.build as B
        B.build()
    return E.lib()


def test_constants(L):
    text = open(HEADER).read()
    assert "#define ENGRAM_PAGE_TOKENS %d" % E.PAGE_TOKENS in text
    assert "#define ENGRAM_NORM_GROUP %d" % E.NORM_GROUP in text
    assert "#define ENGRAM_DEVERR_PAGE %d " % E.DEVERR_PAGE in text
    assert "#define ENGRAM_DEVERR_SEQUENCE %d " % E.DEVERR_SEQUENCE in text


def norm(L, **k):
    a = dict(x=FAKE, res=FAKE, bf=0, w=FAKE, eps=1e-6, sum=FAKE, codes=FAKE, scales=FAKE, rows=4,
             dim=256)
    a.update(k)
    return L.engram_add_norm(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), E.E_ARG), (dict(rows=1 << 31), E.E_RANGE), (dict(dim=0), E.E_UNSUPPORTED),
    (dict(dim=48), E.E_UNSUPPORTED), (dict(dim=65536 + 32), E.E_UNSUPPORTED),
    (dict(dim=-32), E.E_UNSUPPORTED), (dict(eps=-1.0), E.E_ARG),
    (dict(eps=float("nan")), E.E_ARG), (dict(eps=float("inf")), E.E_ARG),
    (dict(res=None), E.E_ARG), (dict(w=None), E.E_ARG), (dict(sum=None), E.E_ARG),
    (dict(codes=None), E.E_ARG), (dict(scales=None), E.E_ARG), (dict(x=FAKE + 2), E.E_ARG),
    (dict(res=FAKE + 4), E.E_ARG), (dict(w=FAKE + 8), E.E_ARG), (dict(sum=FAKE + 4), E.E_ARG),
    (dict(codes=FAKE + 4), E.E_ARG)])
def test_norm_refusals(L, change, code):
    assert norm(L, **change) == code and E.last_error()


def w4(L, **k):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, y=FAKE, T=4, K=256, N=64)
    a.update(k)
    return L.engram_project_w4(*a.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), E.E_ARG), (dict(T=(1 << 22) + 1), E.E_RANGE), (dict(K=0), E.E_UNSUPPORTED),
    (dict(K=192), E.E_UNSUPPORTED), (dict(K=(1 << 20) + 128), E.E_UNSUPPORTED),
    (dict(K=-128), E.E_UNSUPPORTED), (dict(N=0), E.E_UNSUPPORTED), (dict(N=24), E.E_UNSUPPORTED),
    (dict(N=(1 << 24) + 16), E.E_UNSUPPORTED), (dict(x=None), E.E_ARG), (dict(w=None), E.E_ARG),
    (dict(ws=None), E.E_ARG), (dict(y=None), E.E_ARG), (dict(x=FAKE + 8), E.E_ARG),
    (dict(w=FAKE + 8), E.E_ARG), (dict(xs=FAKE + 2), E.E_ARG), (dict(ws=FAKE + 1), E.E_ARG),
    (dict(y=FAKE + 4), E.E_ARG)])
def test_w4_refusals(L, change, code):
    assert w4(L, **change) == code and E.last_error()


def cache_c(**k):
    a = dict(kv_heads=2, head_dim=128, n_pages=10, d_k=FAKE, d_v=FAKE, d_k_scales=FAKE,
             d_v_scales=FAKE)
    a.update(k)
    return E.CacheC(**a)


def seqs_c(**k):
    a = dict(batch=3, max_pages=5, d_pages=FAKE, d_start=FAKE, d_cu=FAKE, d_err=None)
    a.update(k)
    return E.SequencesC(**a)


def append(L, cache=None, seqs=None, **k):
    a = dict(k=FAKE, kt=1024, kh=128, v=FAKE, vt=1024, vh=128, q=FAKE, qt=1024, qh=128, qo=FAKE,
             heads=4, freq=FAKE, rot=128, halves=1, T=6)
    a.update(k)
    return L.engram_cache_append(ctypes.byref(cache or cache_c()), ctypes.byref(seqs or seqs_c()),
                                 *a.values(), None)


def attend(L, cache=None, seqs=None, **k):
    a = dict(q=FAKE, qt=1024, qh=128, out=FAKE, heads=4, T=6, scale=0.1, window=0, ws=FAKE,
             nws=1 << 40)
    a.update(k)
    return L.engram_cache_attend(ctypes.byref(cache or cache_c()), ctypes.byref(seqs or seqs_c()),
                                 *a.values(), None)


BAD_CACHE = [(dict(head_dim=96), E.E_UNSUPPORTED), (dict(head_dim=0), E.E_UNSUPPORTED),
             (dict(kv_heads=0), E.E_UNSUPPORTED), (dict(kv_heads=2048), E.E_UNSUPPORTED),
             (dict(n_pages=0), E.E_ARG), (dict(n_pages=1 << 31), E.E_ARG), (dict(d_k=None), E.E_ARG),
             (dict(d_v=None), E.E_ARG), (dict(d_k_scales=None), E.E_ARG),
             (dict(d_v_scales=None), E.E_ARG), (dict(d_k=FAKE + 8), E.E_ARG),
             (dict(d_v=FAKE + 8), E.E_ARG), (dict(d_k_scales=FAKE + 2), E.E_ARG)]
BAD_SEQS = [(dict(batch=0), E.E_ARG), (dict(batch=-1), E.E_ARG), (dict(batch=1 << 17), E.E_ARG),
            (dict(max_pages=0), E.E_ARG), (dict(max_pages=1 << 25), E.E_ARG),
            (dict(d_pages=None), E.E_ARG), (dict(d_start=None), E.E_ARG),
            (dict(d_cu=FAKE + 2), E.E_ARG), (dict(batch=4, d_cu=None), E.E_ARG)]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("change,code", BAD_CACHE)
def test_cache_refusals(L, call, change, code):
    assert call(L, cache=cache_c(**change)) == code and E.last_error()


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("change,code", BAD_SEQS)
def test_sequence_refusals(L, call, change, code):
    assert call(L, seqs=seqs_c(**change)) == code and E.last_error()


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), E.E_ARG), (dict(T=(1 << 22) + 1), E.E_RANGE), (dict(heads=-1), E.E_ARG),
    (dict(rot=8), E.E_UNSUPPORTED), (dict(rot=144), E.E_UNSUPPORTED), (dict(rot=-16), E.E_UNSUPPORTED),
    (dict(freq=None), E.E_ARG), (dict(k=None), E.E_ARG), (dict(v=None), E.E_ARG),
    (dict(q=None), E.E_ARG), (dict(qo=None), E.E_ARG), (dict(k=FAKE + 8), E.E_ARG),
    (dict(kt=1020), E.E_UNSUPPORTED), (dict(vh=132), E.E_UNSUPPORTED), (dict(vh=-128), E.E_UNSUPPORTED),
    (dict(qh=64), E.E_ARG), (dict(kt=64), E.E_ARG), (dict(qo=FAKE + 8), E.E_ARG)])
def test_append_refusals(L, change, code):
    assert append(L, **change) == code and E.last_error()


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), E.E_ARG), (dict(T=(1 << 22) + 1), E.E_RANGE), (dict(heads=3), E.E_UNSUPPORTED),
    (dict(heads=0), E.E_UNSUPPORTED), (dict(heads=2048), E.E_UNSUPPORTED),
    (dict(scale=float("nan")), E.E_ARG), (dict(scale=float("inf")), E.E_ARG),
    (dict(window=-1), E.E_ARG), (dict(q=None), E.E_ARG), (dict(out=None), E.E_ARG),
    (dict(q=FAKE + 8), E.E_ARG), (dict(qt=1020), E.E_UNSUPPORTED), (dict(qh=64), E.E_ARG),
    (dict(out=FAKE + 4), E.E_ARG)])
def test_attend_refusals(L, change, code):
    assert attend(L, **change) == code and E.last_error()


def test_attend_workspace_refusals(L):
    # long sequences of few rows: the keys are split, so there is a workspace
    seqs = seqs_c(batch=1, max_pages=4096)
    need = L.engram_cache_attend_bytes(ctypes.byref(cache_c()), ctypes.byref(seqs), 4, 1)
    if need:
        assert attend(L, seqs=seqs, T=1, nws=need - 1) == E.E_RANGE and E.last_error()
        assert attend(L, seqs=seqs, T=1, ws=None, nws=need) == E.E_ARG
        assert attend(L, seqs=seqs, T=1, ws=FAKE + 16, nws=need) == E.E_ARG
    # bad arguments need no bytes
    for c, s, h, T in ((cache_c(head_dim=7), seqs, 4, 1), (cache_c(), seqs_c(batch=0), 4, 1),
                       (cache_c(), seqs, 3, 1), (cache_c(), seqs, 4, -1), (cache_c(), seqs, 4, 0)):
        assert L.engram_cache_attend_bytes(ctypes.byref(c), ctypes.byref(s), h, T) == 0


def test_empty_calls_touch_nothing(L):
    assert norm(L, rows=0, x=None, res=None, w=None, sum=None, codes=None, scales=None) == E.OK
    assert w4(L, T=0, x=None, xs=None, w=None, ws=None, y=None) == E.OK
    none = dict(k=None, v=None, q=None, qo=None, freq=None)
    assert append(L, T=0, **none) == E.OK
    assert attend(L, T=0, q=None, out=None, ws=None, nws=0) == E.OK


def test_binding_refusals():
    """Types, shapes and views the binding sees and the library cannot."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    bad = pytest.raises(E.EngramError)
    with bad:
        E.add_norm(z(4, 64, dt=f32), z(4, 64, dt=f32), z(64), 1e-6, z(4, 64, dt=u8), z(4, 2, dt=u8))
    with bad:
        E.add_norm(z(4, 64), z(4, 64, dt=f32), z(64), 1e-6, z(4, 64, dt=u8), z(4, 3, dt=u8))
    with bad:
        E.add_norm(z(3, 64), z(4, 64, dt=f32), z(64), 1e-6, z(4, 64, dt=u8), z(4, 2, dt=u8))
    with bad:
        E.add_norm(z(4, 64), z(4, 64, dt=f32), z(32), 1e-6, z(4, 64, dt=u8), z(4, 2, dt=u8))
    with bad:
        E.add_norm(z(4, 64), z(4, 64, dt=f32), z(64), 1e-6, z(4, 64, dt=u8), z(4, 2, dt=u8),
                   d_sum=z(4, 64))
    with bad:
        E.add_norm(z(64, 4).t(), z(4, 64, dt=f32), z(64), 1e-6, z(4, 64, dt=u8), z(4, 2, dt=u8))
    with bad:
        E.W4(z(16, 64, dt=u8), z(16, 3, dt=u8))
    w = E.W4(z(16, 64, dt=u8), z(16, 4, dt=u8))
    with bad:
        E.project_w4(z(2, 64), w, z(2, 16))
    with bad:
        E.project_w4(z(2, 128), w, z(2, 32))
    with bad:
        E.project_w4(z(2, 128), w, z(2, 16), z(2, 4, dt=u8))       # scales with bf16 x
    with bad:
        E.project_w4(z(2, 128, dt=u8), w, z(2, 16))                # codes without scales
    with bad:
        E.Cache(z(3, 2, 32, 64, dt=u8), z(3, 2, 32, 64, dt=u8), z(3, 2, dt=f32), z(3, 2, dt=f32))
    with bad:
        E.Cache(z(3, 2, 64, 64, dt=u8), z(3, 2, 64, 64, dt=u8), z(2, 3, dt=f32), z(3, 2, dt=f32))
    c = E.Cache(z(3, 2, 64, 64, dt=u8), z(3, 2, 64, 64, dt=u8), z(3, 2, dt=f32), z(3, 2, dt=f32))
    with bad:
        E.Sequences(z(2, 3, dt=torch.int64), z(2, dt=i32))
    with bad:
        E.Sequences(z(2, 3, dt=i32), z(2, dt=i32), z(2, dt=i32))
    s = E.Sequences(z(2, 3, dt=i32), z(2, dt=i32))
    with bad:
        E.cache_append(c, s, z(4, 3, 64), z(4, 2, 64), None)
    with bad:
        E.cache_append(c, s, z(4, 2, 64), z(2, 2, 64), None)
    with bad:
        E.cache_append(c, s, z(4, 2, 64), z(4, 2, 64), None, z(4, 4, 64))
    with bad:
        E.cache_append(c, s, z(4, 2, 128)[:, :, ::2], z(4, 2, 64), None)
    with bad:
        E.cache_attend(c, s, z(4, 4, 64), z(4, 4, 32), 1.0)
    with bad:
        E.cache_attend(c, s, z(4, 4, 64, dt=f32), z(4, 4, 64), 1.0)


def test_host_tensors_are_refused():
    """A tensor in host memory, right in type and shape, ends in the binding."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    cache = E.Cache(z(3, 2, 64, 64, dt=u8), z(3, 2, 64, 64, dt=u8), z(3, 2, dt=f32), z(3, 2, dt=f32))
    seqs = E.Sequences(z(2, 3, dt=i32), z(2, dt=i32))
    weights = E.W4(z(16, 64, dt=u8), z(16, 4, dt=u8))
    assert cache.host == "k" and seqs.host == "pages" and weights.host == "w"
    calls = [
        lambda: E.add_norm(z(4, 64), z(4, 64, dt=f32), z(64), 1e-6, z(4, 64, dt=u8), z(4, 2, dt=u8),
                           stream=0),
        lambda: E.project_w4(z(2, 128), weights, z(2, 16), stream=0),
        lambda: E.project_w4(z(2, 128, dt=u8), weights, z(2, 16), z(2, 4, dt=u8), stream=0),
        lambda: E.cache_append(cache, seqs, z(4, 2, 64), z(4, 2, 64), z(32, dt=f32), stream=0),
        lambda: E.cache_attend(cache, seqs, z(4, 4, 64), z(4, 4, 64), 1.0, stream=0)]
    for call in calls:
        with pytest.raises(E.EngramError, match="on the GPU is needed"):
            call()
    # the step's own tensors, where what the program keeps is on the GPU
    cache.host = seqs.host = weights.host = None
    for call in calls:
        with pytest.raises(E.EngramError, match="on the GPU is needed"):
            call()


@pytest.mark.parametrize("version,message", [(E.ABI_VERSION - 1, "ABI version"), (E.ABI_VERSION, "has no engram_")])
def test_stale_library(tmp_path, monkeypatch, version, message):
    """A library built before this binding is named as that, whether its
    version differs or entry points were only added since."""
    src, so = tmp_path / "stale.c", tmp_path / "stale.so"
    src.write_text(f"int engram_abi_version(void) {{ return {version}; }}\n"
                   "const char *engram_last_error(void) { return \"\"; }\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(E, "_lib", None)
    monkeypatch.setattr(E, "LIB_PATH", str(so))
    with pytest.raises(RuntimeError, match=f"{message}.*rebuild"):
        E.lib()
    assert E._lib is None


@pytest.mark.parametrize("gone", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_current_stream_by_the_public_way(monkeypatch, gone):
    """Without torch's own short cut the current stream is asked for publicly."""
    asked = []

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: asked.append(1) or Stream)
    monkeypatch.delattr(torch._C, gone, raising=False)
    monkeypatch.setattr(E, "_current", None)
    assert [E._stream(None) for _ in range(3)] == [77] * 3 and len(asked) == 3
    assert E._stream(5) == 5 and E._stream(Stream) == 77


def test_outputs_over_inputs_are_refused(L):
    """Workgroups read what another would have written: refused, in place or
    shifted by a few bytes (a call that starts where the other ends is not)."""
    for shift in (-256, 0, 8, 1024):
        assert w4(L, T=4, K=256, N=64, xs=None, y=FAKE + shift) == E.E_ARG and "overlaps" in E.last_error()
        # q spans 5 strides of 1024 values, 3 of 128 and a head
        assert attend(L, out=FAKE + shift) == E.E_ARG and "overlaps" in E.last_error()
    assert attend(L, out=FAKE + 2 * (5 * 1024 + 3 * 128 + 128) - 16) == E.E_ARG and "overlaps" in E.last_error()
    assert attend(L, out=FAKE - 6 * 4 * 128 * 2 + 16) == E.E_ARG and "overlaps" in E.last_error()


def test_attend_asks_for_a_workspace(L):
    """A long table of few rows has its keys split over workgroups, on any
    device: never 0 bytes, and one byte less is refused."""
    for dim in (64, 128, 256):
        cache, seqs = cache_c(head_dim=dim), seqs_c(batch=1, max_pages=4096)
        need = L.engram_cache_attend_bytes(ctypes.byref(cache), ctypes.byref(seqs), 4, 1)
        assert need > 0
        call = dict(cache=cache, seqs=seqs, T=1, qh=dim)
        assert attend(L, nws=need - 1, **call) == E.E_RANGE and E.last_error()
        assert attend(L, ws=None, nws=need, **call) == E.E_ARG and E.last_error()
        assert attend(L, ws=FAKE + 16, nws=need, **call) == E.E_ARG and E.last_error()
    assert L.engram_cache_attend_bytes(ctypes.byref(cache_c()), ctypes.byref(seqs_c(batch=1, max_pages=16)), 4, 1) == 0


def test_append_grid_is_checked(L):
    """More workgroups than a grid holds threads for: refused before a launch."""
    cache, seqs = cache_c(head_dim=256, kv_heads=32), seqs_c(batch=65536)
    strides = dict(kt=32 * 256, kh=256, vt=32 * 256, vh=256, q=None, heads=0, rot=0, freq=None)
    assert append(L, cache=cache, seqs=seqs, T=1024, **strides) == E.E_RANGE
    assert "workgroups" in E.last_error()
    assert append(L, cache=cache_c(head_dim=256, kv_heads=64), seqs=seqs, T=1024, **dict(strides, kt=64 * 256, vt=64 * 256)) == E.E_RANGE
