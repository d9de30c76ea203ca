"""The entry points of the 8-bit paged cache without a GPU (a process that sees one does not run this file):
refusals of the C ABI (fake pointers, nothing is dereferenced) and of the Python binding, and the references
of the GPU tests on hand-worked cases."""
import ctypes
import os

import numpy as np
import pytest

import _paged8 as p8

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def xs():
    from conftest import build_library
    build_library()
    import dit_attention_ulysses_gb300 as xs
    # the calls that pass the checks below must not reach a GPU with their made-up addresses
    nbytes = ctypes.c_size_t(0)
    assert xs.lib.xs_attn_paged_workspace_bytes(1, 1, 1, 64, ctypes.byref(nbytes)) != xs.XS_OK, "run this file without a GPU"
    return xs


def A(i):
    """A fake device address, far from the others."""
    return 0x10_0000_0000 * (i + 1)


def _passed(xs, code):
    return code in (xs.XS_ERR_CUDA, xs.XS_ERR_UNSUPPORTED_DEVICE)   # the checks passed, and there is no GPU


def S3(*v):
    return (ctypes.c_longlong * 3)(*v)


class Cache8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "ksc", "vsc")] + \
               [(n, ctypes.c_longlong * 3) for n in ("ks", "vs", "kss", "vss")] + \
               [(n, ctypes.c_int) for n in ("pages", "page", "Hkv", "D", "block", "dtype")]


class AppendArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "pos", "slots", "qo", "rope")] + [("cache", Cache8)] + \
               [(n, ctypes.c_longlong) for n in ("qs", "ks", "vs", "os_")] + [("T", ctypes.c_int), ("H", ctypes.c_int)]


class ReadArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "cu", "first", "ko", "vo")] + [("cache", Cache8)] + \
               [(n, ctypes.c_longlong) for n in ("ks", "vs", "ts")] + [(n, ctypes.c_int) for n in ("T", "n", "width")]


class AttnArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "table", "lse", "ws")] + [("nbytes", ctypes.c_size_t)] + \
               [("outs", ctypes.c_void_p * 16), ("cache", Cache8), ("qs", ctypes.c_longlong), ("ts", ctypes.c_longlong)] + \
               [(n, ctypes.c_int) for n in ("layout", "P", "T", "H", "n", "width", "max_q", "causal", "window")] + \
               [("scale", ctypes.c_float)]


def test_the_binding_packs_the_structs(xs):
    assert ctypes.sizeof(Cache8) == 152
    assert xs._APPEND8_ARGS.size == ctypes.sizeof(AppendArgs) and AppendArgs.cache.offset == 56
    assert xs._READ8_ARGS.size == ctypes.sizeof(ReadArgs) and ReadArgs.T.offset == 216
    assert {p.size for p in xs._ATTN8_ARGS.values()} == {ctypes.sizeof(AttnArgs)} and set(xs._ATTN8_ARGS) == set(range(1, 17))
    assert AttnArgs.cache.offset == 168 and AttnArgs.scale.offset == 372


# 8 pages of 32 tokens, 2 KV heads of 128, blocks of 16
CACHE = dict(kc=A(10), vc=A(11), ksc=A(12), vsc=A(13), kst=S3(32 * 256, 256, 128), vst=S3(32 * 256, 256, 128),
             kss=S3(4, 2, 1), vss=S3(4, 2, 1), pages=8, page=32, Hkv=2, D=128, block=16, dtype=0)


def _cache(a):
    return Cache8(*(a[n] for n in ("kc", "vc", "ksc", "vsc", "kst", "vst", "kss", "vss", "pages", "page", "Hkv", "D", "block",
                                   "dtype")))


def _append(xs, rotate=True, **kw):
    a = dict(CACHE, q=A(0), k=A(1), v=A(2), pos=A(3), slots=A(4), qo=A(5), T=10, H=4, qs=512, ks=256, vs=256, os_=512)
    keep = xs._RopeStruct()
    assert xs.lib.xs_rope_init(ctypes.addressof(keep), 128, 128, 0, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0) == xs.XS_OK
    a["rope"] = ctypes.addressof(keep)
    if not rotate:
        a.update(rope=None, q=None, pos=None, qo=None, H=0)
    a.update(kw)
    g = AppendArgs(*(a[n] for n in ("q", "k", "v", "pos", "slots", "qo", "rope")), _cache(a), a["qs"], a["ks"], a["vs"], a["os_"],
                   a["T"], a["H"])
    return xs.lib.xs_rope_append_paged8(bytes(g), None)


def _read(xs, **kw):
    a = dict(CACHE, table=A(0), cu=A(1), first=A(2), ko=A(3), vo=A(4), ks=256, vs=256, ts=10, T=16, n=4, width=10)
    a.update(kw)
    g = ReadArgs(*(a[n] for n in ("table", "cu", "first", "ko", "vo")), _cache(a),
                 *(a[n] for n in ("ks", "vs", "ts", "T", "n", "width")))
    return xs.lib.xs_paged_read8(bytes(g), None)


def _attn(xs, **kw):
    a = dict(CACHE, q=A(0), table=A(3), layout=1, outs=[A(20) + (i << 28) for i in range(16)], lse=A(5), T=16, H=8, P=1,
             qs=1024, n=4, width=10, ts=10, max_q=1, causal=1, window=0, scale=0.1, ws=A(6), nbytes=1 << 30)
    a.update(kw)
    g = AttnArgs(a["q"], a["table"], a["lse"], a["ws"], a["nbytes"], (ctypes.c_void_p * 16)(*a["outs"]), _cache(a), a["qs"],
                 a["ts"], *(a[n] for n in ("layout", "P", "T", "H", "n", "width", "max_q", "causal", "window", "scale")))
    return xs.lib.xs_attn_paged8_fwd(bytes(g), None)


CALLS = {"append": _append, "append, not rotated": lambda xs, **kw: _append(xs, rotate=False, **kw), "read": _read, "attn": _attn}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS)
def test_refusals_of_a_cache(xs, call):
    f = lambda **k: call(xs, **k)   # noqa: E731
    assert _passed(xs, f())
    for name in ("kc", "vc", "ksc", "vsc"):
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert f(D=96) == f(D=0) == xs.XS_ERR_HEAD_DIM
    for page in (8, 48, 2048, 0, -32):
        assert f(page=page) == xs.XS_ERR_PAGE, page
    for block in (8, 0, -16, 24, 64, 256):      # 64: more than a page
        assert f(block=block) == xs.XS_ERR_PAGE, block
    big = dict(page=256, kst=S3(256 * 256, 256, 128), vst=S3(256 * 256, 256, 128))
    assert f(block=256, **big) == xs.XS_ERR_PAGE and _passed(xs, f(block=128, **big))
    assert f(pages=0) == f(pages=2 ** 27) == f(Hkv=0) == f(Hkv=4097) == xs.XS_ERR_SHAPE
    assert f(kst=S3(8192, 120, 128)) == f(vst=S3(2 ** 35 + 16, 256, 128)) == f(kst=S3(8192, 256, 0)) == xs.XS_ERR_SHAPE
    assert f(kss=S3(4, 0, 1)) == f(vss=S3(4, 2, -1)) == f(kss=S3(2 ** 35 + 1, 2, 1)) == xs.XS_ERR_SHAPE
    assert f(kst=S3(8200, 256, 128)) == f(vst=S3(8192, 256, 136)) == f(kc=A(10) + 8) == f(vc=A(11) + 4) == xs.XS_ERR_ALIGNMENT
    assert f(dtype=2) == f(dtype=-1) == xs.XS_ERR_DTYPE
    assert _passed(xs, f(ksc=A(12) + 1, vsc=A(13) + 3, kss=S3(5, 2, 1), vss=S3(8, 1, 4)))   # scales: any address, any strides


@pytest.mark.parametrize("rotate", [True, False])
def test_append_refusals(xs, rotate):
    f = lambda **k: _append(xs, rotate=rotate, **k)   # noqa: E731
    for name in ("k", "v", "slots") + (("q", "pos", "qo") if rotate else ()):
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert xs.lib.xs_rope_append_paged8(None, None) == xs.XS_ERR_NULL
    assert f(T=0) == f(T=-1) == f(ks=255) == f(vs=0) == f(ks=2 ** 40) == xs.XS_ERR_SHAPE
    assert f(ks=260) == f(slots=A(4) + 4) == f(k=A(1) + 2) == f(v=A(2) + 8) == xs.XS_ERR_ALIGNMENT
    assert f(vc=A(10)) == f(kc=A(1) + 64) == f(slots=A(11) + 1024) == f(vc=A(2) + 16) == xs.XS_ERR_OVERLAP
    # the scales: apart from each other, from the numbers and from what is read
    assert f(vsc=A(12)) == f(vsc=A(12) + 7) == f(ksc=A(10) + 100) == f(vsc=A(10)) == f(ksc=A(4) + 79) == xs.XS_ERR_OVERLAP
    assert f(ksc=A(1) + 10) == f(vsc=A(2) + 5119) == xs.XS_ERR_OVERLAP and _passed(xs, f(vsc=A(2) + 5120))
    both = S3(2 * 32 * 256, 256, 128)
    assert _passed(xs, f(vc=A(10) + 32 * 256, kst=both, vst=both))                          # one buffer, by pages
    assert f(vc=A(10) + 32 * 256 - 16, kst=both, vst=both) == f(vc=A(10) + 16 * 256, kst=both, vst=both) == xs.XS_ERR_OVERLAP
    sc = S3(8, 2, 1)
    assert _passed(xs, f(vsc=A(12) + 4, kss=sc, vss=sc)) and f(vsc=A(12) + 3, kss=sc, vss=sc) == xs.XS_ERR_OVERLAP
    assert f(vsc=A(12) + 4, kss=sc, vss=S3(8, 1, 2)) == xs.XS_ERR_OVERLAP                   # unlike strides: not told apart
    assert _passed(xs, f(k=A(0) + 1024, v=A(0) + 1536, ks=1024, vs=1024, **(dict(qo=A(0), qs=1024, os_=1024) if rotate else {})))
    assert _passed(xs, f(Hkv=1, ks=128, vs=128, kst=S3(4096, 128, 1), vst=S3(4096, 128, 0), kss=S3(2, 1, 0), vss=S3(2, 1, -5)))
    assert _passed(xs, f(page=16, kst=S3(4096, 256, 128), vst=S3(4096, 256, 128), kss=S3(2, 0, 1), vss=S3(2, -9, 1)))   # one block


def test_append_with_or_without_a_rotation(xs):
    f = lambda **k: _append(xs, **k)   # noqa: E731
    assert f(D=64) == xs.XS_ERR_HEAD_DIM                                                    # not the rotation's
    assert f(H=0) == f(H=4097) == f(qs=511) == f(os_=0) == xs.XS_ERR_SHAPE
    assert f(qs=516) == f(qo=A(5) + 8) == f(pos=A(3) + 2) == xs.XS_ERR_ALIGNMENT
    assert f(qo=A(1)) == f(qo=A(0) + 16) == f(qo=A(10)) == f(qo=A(12)) == f(qo=A(3)) == f(pos=A(13) + 4) == xs.XS_ERR_OVERLAP
    assert f(qo=A(4) + 16) == f(qo=A(2)) == f(ksc=A(5) + 3) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f(qo=A(0)))                                                          # in place
    g = lambda **k: _append(xs, rotate=False, **k)   # noqa: E731
    assert g(q=A(0)) == g(pos=A(3)) == g(qo=A(5)) == g(H=1) == xs.XS_ERR_ROPE
    assert _passed(xs, g(qs=0, os_=-7))                                                     # strides of nothing
    assert _passed(xs, g(D=64, kst=S3(8192, 256, 128), vst=S3(8192, 256, 128)))


def test_read_refusals(xs):
    f = lambda **k: _read(xs, **k)   # noqa: E731
    for name in ("table", "cu", "ko", "vo"):
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert xs.lib.xs_paged_read8(None, None) == xs.XS_ERR_NULL
    assert f(T=0) == f(n=0) == f(n=8193) == f(width=0) == f(ts=9) == f(ts=2 ** 36) == f(ks=255) == f(vs=2 ** 40) == xs.XS_ERR_SHAPE
    assert f(ks=260) == f(ko=A(3) + 8) == f(vo=A(4) + 2) == f(cu=A(1) + 2) == f(first=A(2) + 1) == f(table=A(0) + 2) \
        == xs.XS_ERR_ALIGNMENT
    assert f(vo=A(3)) == f(ko=A(0) + 16) == f(ko=A(1)) == f(vo=A(2)) == f(ko=A(10) + 64) == f(vo=A(11)) == xs.XS_ERR_OVERLAP
    assert f(ksc=A(3) + 5) == f(vsc=A(4) + 16 * 512 - 1) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f(first=None)) and _passed(xs, f(n=1, ts=0)) and _passed(xs, f(n=1, ts=-3))
    assert _passed(xs, f(vo=A(3) + 512, ks=512, vs=512))                                    # columns of one matrix
    assert _passed(xs, f(vc=A(10), vsc=A(12)))                                              # reads may be of one buffer


def test_plan_refusals(xs):
    def f(**kw):
        a = dict(cu=A(0), kv=A(1), n=4, H=8, Hkv=2, D=128, max_q=1, causal=1, window=0, ws=A(2), nbytes=1 << 30)
        a.update(kw)
        return xs.lib.xs_attn_paged8_plan(*a.values(), None)
    assert f(cu=None) == f(kv=None) == f(ws=None) == xs.XS_ERR_NULL
    assert f(n=0) == f(n=8193) == f(H=0) == f(Hkv=0) == f(max_q=0) == f(window=-1) == f(window=5, causal=0) == xs.XS_ERR_SHAPE
    assert f(H=129, Hkv=1) == xs.XS_ERR_SHAPE and f(D=96) == xs.XS_ERR_HEAD_DIM and f(Hkv=3) == xs.XS_ERR_DIVISIBILITY
    assert f(cu=A(0) + 2) == f(ws=A(2) + 128) == xs.XS_ERR_ALIGNMENT and f(cu=A(2) + 256) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f(window=1)) and _passed(xs, f(max_q=2 ** 31 - 1))


def test_attention_refusals(xs):
    f = lambda **k: _attn(xs, **k)   # noqa: E731
    for name in ("q", "table", "ws"):
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert xs.lib.xs_attn_paged8_fwd(None, None) == xs.XS_ERR_NULL
    assert f(outs=[]) == f(outs=[A(20), A(21)], layout=0, P=4) == xs.XS_ERR_NULL
    assert f(T=0) == f(qs=1000) == f(width=0) == f(ts=9) == f(n=0) == f(max_q=0) == f(window=3, causal=0) == xs.XS_ERR_SHAPE
    assert f(layout=3) == xs.XS_ERR_LAYOUT and f(layout=0, P=17) == xs.XS_ERR_TOO_MANY_RANKS
    assert f(layout=0, P=3) == f(layout=2, P=3) == f(H=7, qs=1024) == xs.XS_ERR_DIVISIBILITY
    assert f(scale=float("nan")) == f(scale=-1.0) == xs.XS_ERR_SCALE
    assert f(q=A(0) + 8) == f(qs=1028) == f(lse=A(5) + 2) == f(ws=A(6) + 16) == f(outs=[A(20) + 8]) == xs.XS_ERR_ALIGNMENT
    assert f(lse=A(20)) == f(ws=A(0)) == f(lse=A(10) + 64) == f(outs=[A(11) + 16]) == xs.XS_ERR_OVERLAP
    assert f(lse=A(12)) == f(outs=[A(13) + 0]) == f(ksc=A(6) + 999) == f(vsc=A(20) + 3) == xs.XS_ERR_OVERLAP
    assert f(outs=[A(20), A(20)], layout=0, P=2) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f(lse=None)) and _passed(xs, f(layout=0, P=4)) and _passed(xs, f(n=1, ts=0))


def test_python_refuses_host_tensors_and_wrong_types(xs):
    rows, pos, slots = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    code, scale = torch.zeros((3, 32, 2, 64)).to(torch.float8_e4m3fn), torch.zeros((3, 2, 2), dtype=torch.uint8)
    cache = (code, code.clone(), scale, scale.clone())
    table = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(TypeError, match="current device"):
        xs.xs_rope_append_paged8(rows, rows, rows, pos, slots, rows, *cache, xs.Rope(64))
    with pytest.raises(TypeError, match="current device"):
        xs.xs_rope_append_paged8(None, rows, rows, None, slots, None, *cache, None)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        xs.xs_rope_append_paged8(None, rows.float(), rows.float(), None, slots, None, *cache, None)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        xs.xs_rope_append_paged8(None, rows, rows, None, slots, None, rows[:, None], *cache[1:], None)
    with pytest.raises(TypeError, match="current device"):
        xs.xs_paged_read8(*cache, table, pos[:3], None, rows, rows.clone())
    with pytest.raises(TypeError):
        xs.xs_attn_paged8_plan(pos[:3], pos[:2], 1, type("W", (), dict(_buf=slots, _dims=(2, 2, 2, 64), n=2, H=2, Hkv=2, D=64,
                                                                      ptr=0, nbytes=32))())


def test_native_binding_leaves_host_tensors_to_python(xs):
    xs._device()
    if xs._native is None:
        assert not os.path.exists(os.path.join(os.path.dirname(xs.__file__), "_binding.so"))
        return
    x, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    rope, n = xs.Rope(64), xs._native
    assert n.append8(x, x, x, pos, pos, x, x, x, x, x, rope.ptr, 64, None) is None
    assert n.append8(None, x, x, None, pos, None, x, x, x, x, 0, 64, None) is None and n.append8(1) is None
    assert n.read8(x, x, x, x, pos, pos, None, x, x, None) is None and n.read8() is None
    assert n.plan8(pos, pos, 1, pos, (1, 1, 1, 64, 0, 0), 1, 0, None) is None
    assert n.attn8(x, x, x, x, x, pos, 1, [x], 0.1, pos, (), (1, 1, 0), None, None) is None


# -------------------------------------------------------------- the tests' references
def test_numbers_by_hand():
    values = np.array([0.0, 1.0, 1.0625, 1.1875, 447.0, 448.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, -3.4, 17.0])
    want = np.array([0.0, 1.0, 1.0, 1.25, 448.0, 448.0, 2.0 ** -9, 0.0, 2.0 ** -8, -3.5, 16.0])
    assert np.array_equal(p8.nearest(values), want)
    assert np.array_equal(p8.numbers(p8.codes(want)), want)
    every = np.arange(256, dtype=np.uint8)
    x = p8.numbers(torch.from_numpy(every))
    finite = np.isfinite(x)
    assert finite.sum() == 254 and np.array_equal(p8.nearest(x[finite]), x[finite])
    # needs: 448 fits 2^0, 449 does not
    a = np.array([0.0, 448.0, 449.0, 224.0, 225.0, 1.0, 2.0 ** -80, 3e38])
    e = p8.need(a)
    assert e.tolist()[:5] == [-64, 0, 1, -1, 0] and e[6] == -64
    assert (a[1:] <= 448 * np.exp2(e[1:].astype(float))).all()
    assert (a[[1, 2, 3, 4, 5, 7]] > 448 * np.exp2(e[[1, 2, 3, 4, 5, 7]] - 1.0)).all()


def test_append_reference_by_hand():
    """Blocks of 16 in pages of 32, one head, one channel: a run that begins a block, one that joins it and needs a
    larger scale, one that does not, padding, and a run that goes on in the next block."""
    num, exp = np.full((2, 32, 1, 1), np.nan), np.full((2, 2, 1), 128.0)
    x = np.array([448.0, 1.0, 2.0 ** -9 * 448, 900.0, 5.0, 7.0, 3.0]).reshape(-1, 1, 1)
    p8.append_reference(num, exp, x[:1], [32], 16)
    assert exp[1, 0, 0] == 0 and num[1, 0, 0, 0] == 448
    p8.append_reference(num, exp, x[1:3], [33, 34], 16)      # 1, 0.875
    assert exp[1, 0, 0] == 0 and num[1, :3, 0, 0].tolist() == [448, 1, 0.875]
    p8.append_reference(num, exp, x[3:5], [35, -1], 16)      # 900 = 448 * 2.009: two steps up
    assert exp[1, 0, 0] == 2 and num[1, :4, 0, 0].tolist() == [112, 0.25, 0.21875, 224]
    p8.append_reference(num, exp, x[5:], [15, 16], 16)       # the last of block 0 (kept: what it held), the first of block 1
    assert exp[0, 1, 0] == -7 and num[0, 16, 0, 0] == 384 and exp[0, 0, 0] == 128
    assert np.isnan(num[1, 4:]).all()


def test_attention_reference_takes_the_elements():
    c = p8.Paged8Case([1, 2], [20, 5], 2, 1, 64, 16, 16, device="cpu", spread=2)
    k = p8.numbers(c.k.view(torch.uint8))
    e = c.ks.view(torch.uint8).double().numpy() - 127
    for i, kv in enumerate(c.kv_lens):
        for t in range(kv):
            at = int(c.table[i, t // 16])
            assert np.array_equal(k[at, t % 16] * 2.0 ** e[at, 0][:, None], c.keys[i][t])
    out, mass, lse = c.reference(True, 0, 0.1)
    s = c.q64[0, 0] @ c.keys[0][:, 0].T * 0.1
    w = np.exp(s - s.max())
    np.testing.assert_allclose(out[0, 0], w @ c.values[0][:, 0] / w.sum(), rtol=1e-12)
