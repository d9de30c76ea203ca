"""The paged-cache entry points without a GPU (a process that sees one does not run this file):
refusals of the C ABI (fake pointers, nothing is dereferenced) and of the Python binding, the frequencies of xs_rope_init, the division of
the attention's work (host program over the kernels' own geometry), and the references of the
GPU tests on hand-worked cases."""
import ctypes
import math
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

import _paged as pg

torch = pytest.importorskip("torch")
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dit_attention_ulysses_gb300", "csrc")


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


REFUSED_LATER = ("XS_ERR_CUDA", "XS_ERR_UNSUPPORTED_DEVICE")   # the checks passed, and there is no GPU


def _passed(xs, code):
    return code in tuple(getattr(xs, n) for n in REFUSED_LATER)


def S3(*v):
    return (ctypes.c_longlong * 3)(*v)


# ------------------------------------------------------------------------------- rope
def _init(xs, **kw):
    a = dict(D=128, rot=128, layout=0, base=1e4, scaling=0, factor=1.0, context=0.0, low=1.0, high=32.0, magnitude=1.0)
    a.update(kw)
    s = xs._RopeStruct()
    return xs.lib.xs_rope_init(ctypes.addressof(s), *a.values()), s


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), "XS_ERR_HEAD_DIM"), (dict(rot=0), "XS_ERR_ROPE"), (dict(rot=24), "XS_ERR_ROPE"),
    (dict(D=64, rot=80), "XS_ERR_ROPE"), (dict(layout=2), "XS_ERR_LAYOUT"), (dict(layout=-1), "XS_ERR_LAYOUT"),
    (dict(base=0.5), "XS_ERR_ROPE"), (dict(base=float("nan")), "XS_ERR_ROPE"), (dict(base=float("inf")), "XS_ERR_ROPE"),
    (dict(scaling=4), "XS_ERR_ROPE"), (dict(scaling=-1), "XS_ERR_ROPE"),
    (dict(scaling=1, factor=0.5), "XS_ERR_ROPE"), (dict(scaling=2, factor=float("nan")), "XS_ERR_ROPE"),
    (dict(scaling=3, factor=2.0), "XS_ERR_ROPE"), (dict(scaling=3, factor=2.0, context=100.0, low=3.0, high=3.0), "XS_ERR_ROPE"),
    (dict(magnitude=float("inf")), "XS_ERR_ROPE")])
def test_rope_init_refusals(xs, kw, code):
    assert _init(xs, **kw)[0] == getattr(xs, code)
    assert xs.lib.xs_rope_init(None, 64, 64, 0, 1e4, 0, 1.0, 0.0, 1.0, 2.0, 1.0) == xs.XS_ERR_NULL
    with pytest.raises(xs.XsError):
        xs.Rope(kw.get("D", 128), **{k: v for k, v in {"rot": 128, **kw}.items() if k != "D"})


@pytest.mark.parametrize("rot", [16, 48, 128])
@pytest.mark.parametrize("kw", [{}, dict(scaling="linear", factor=3.0), dict(scaling="stretch", factor=4.0, base=1e6),
                                dict(scaling="by_parts", factor=8.0, context=8192.0), dict(base=1.0)], ids=str)
def test_rope_init_frequencies(xs, rot, kw):
    k = dict(kw)
    k["scaling"] = ("plain", "linear", "stretch", "by_parts").index(k.get("scaling", "plain"))
    code, s = _init(xs, rot=rot, magnitude=1.5, **k)
    assert code == xs.XS_OK and s.magnitude == 1.5 and s.rot == rot and s.D == 128
    theta = np.array(list(s.turns)[:rot // 2], dtype=np.float64) * 2.0 ** -64 * 2 * math.pi
    # pow and a few products: some steps of 2^-53; the table's own step is 2^-64 turns
    np.testing.assert_allclose(theta, pg.frequencies(rot, **kw), rtol=1e-13, atol=2 * math.pi * 2.0 ** -64)
    assert not any(list(s.turns)[rot // 2:])


def test_angles_are_exact_at_far_positions(xs):
    """position * turns mod 2^64 against exact integers: an angle off by less than 2^-31 turns."""
    from fractions import Fraction
    _, s = _init(xs, rot=32)
    for pos in (1, -1, 12345, 2 ** 31 - 1, -2 ** 31):
        for t in list(s.turns)[:16]:
            got = (pos * t) % 2 ** 64 >> 32
            got -= 2 ** 32 * (got >= 2 ** 31)
            exact = Fraction(pos * t, 2 ** 64)
            d = (Fraction(got, 2 ** 32) - exact) % 1
            assert min(d, 1 - d) <= Fraction(1, 2 ** 32)


def _rope_fwd(xs, x=A(0), pos=A(1), out=A(2), T=10, H=4, xs_=None, os_=None, dtype=0, rope=True, D=128):
    s = _init(xs, D=D, rot=D)[1]
    return xs.lib.xs_rope_fwd(x, pos, out, T, H, H * D if xs_ is None else xs_, H * D if os_ is None else os_, dtype, 0,
                              ctypes.addressof(s) if rope else None, None)


def test_rope_fwd_refusals(xs):
    f = lambda **k: _rope_fwd(xs, **k)   # noqa: E731
    assert f(x=None) == f(pos=None) == f(out=None) == f(rope=False) == xs.XS_ERR_NULL
    assert f(T=0) == f(H=0) == f(T=-1) == f(xs_=511) == f(os_=0) == f(xs_=2 ** 50) == f(T=2 ** 30, H=4096) == xs.XS_ERR_SHAPE
    assert f(dtype=2) == f(dtype=-1) == xs.XS_ERR_DTYPE
    assert f(xs_=516) == f(x=A(0) + 8) == f(out=A(2) + 2) == f(pos=A(1) + 2) == xs.XS_ERR_ALIGNMENT
    assert f(out=A(0) + 16) == xs.XS_ERR_OVERLAP                        # shifted by 16 bytes
    assert f(out=A(0), os_=1024) == xs.XS_ERR_OVERLAP                   # the same rows at another stride
    assert f(out=A(0) + 512, xs_=1536, os_=1536) == xs.XS_ERR_OVERLAP   # columns that overlap
    assert f(pos=A(2) + 64) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f(out=A(0)))                                     # in place
    assert _passed(xs, f(out=A(0) + 1024, xs_=1536, os_=1536))          # other columns of one matrix
    assert _passed(xs, f(x=A(0) + 1024, out=A(0), xs_=1536, os_=1536))
    bad = xs._RopeStruct()
    assert xs.lib.xs_rope_fwd(A(0), A(1), A(2), 1, 1, 64, 64, 0, 0, ctypes.addressof(bad), None) == xs.XS_ERR_HEAD_DIM


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_longlong * 3),
                ("vs", ctypes.c_longlong * 3), ("pages", ctypes.c_int), ("page", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("reserved", ctypes.c_int)]


class AppendArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "pos", "slots", "qo", "rope")] + [("cache", Cache)] + \
               [(n, ctypes.c_longlong) for n in ("qs", "ks", "vs", "os_")] + [("T", ctypes.c_int), ("H", ctypes.c_int)]


class AttnArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "table", "lse", "ws")] + [("nbytes", ctypes.c_size_t)] + \
               [("outs", ctypes.c_void_p * 16), ("cache", Cache), ("qs", ctypes.c_longlong), ("ts", ctypes.c_longlong)] + \
               [(n, ctypes.c_int) for n in ("layout", "P", "T", "H", "n", "width", "max_q", "causal", "window")] + \
               [("scale", ctypes.c_float)]


def test_the_binding_packs_the_structs(xs):
    assert xs._APPEND_ARGS.size == ctypes.sizeof(AppendArgs)
    assert {p.size for p in xs._ATTN_ARGS.values()} == {ctypes.sizeof(AttnArgs)} and set(xs._ATTN_ARGS) == set(range(1, 17))
    assert Cache.dtype.offset == 80 and AttnArgs.cache.offset == 168 and AttnArgs.scale.offset == 308


def _append(xs, **kw):
    a = dict(q=A(0), k=A(1), v=A(2), pos=A(3), slots=A(4), qo=A(5), kc=A(6), vc=A(7), T=10, H=4, Hkv=2, qs=512, ks=256,
             vs=256, os_=512, pages=8, page=16, kst=S3(16 * 256, 256, 128), vst=S3(16 * 256, 256, 128), dtype=0, D=128)
    keep = _init(xs)[1]
    a["rope"] = ctypes.addressof(keep)
    a.update(kw)
    c = Cache(a["kc"], a["vc"], a["kst"], a["vst"], a["pages"], a["page"], a["Hkv"], a["D"], a["dtype"], 0)
    g = AppendArgs(*(a[n] for n in ("q", "k", "v", "pos", "slots", "qo", "rope")), c, a["qs"], a["ks"], a["vs"], a["os_"],
                   a["T"], a["H"])
    return xs.lib.xs_rope_append_paged(bytes(g), None)


def test_append_refusals(xs):
    f = lambda **k: _append(xs, **k)   # noqa: E731
    for name in ("q", "k", "v", "pos", "slots", "qo", "kc", "vc", "rope"):
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert xs.lib.xs_rope_append_paged(None, None) == xs.XS_ERR_NULL
    assert f(D=64) == f(D=96) == xs.XS_ERR_HEAD_DIM      # not the rotation's
    assert f(page=8) == f(page=48) == f(page=2048) == f(page=0) == xs.XS_ERR_PAGE
    assert f(pages=0) == f(pages=2 ** 28) == f(Hkv=0) == f(ks=255) == f(kst=S3(4096, 120, 128)) == xs.XS_ERR_SHAPE
    assert f(kst=S3(4100, 256, 128)) == f(vst=S3(4096, 260, 128)) == f(slots=A(4) + 4) == f(kc=A(6) + 8) == xs.XS_ERR_ALIGNMENT
    assert f(vc=A(6)) == f(kc=A(0) + 64) == f(qo=A(1)) == f(qo=A(0) + 16) == f(slots=A(7) + 1024) == xs.XS_ERR_OVERLAP
    assert f(qo=A(7)) == xs.XS_ERR_OVERLAP
    assert f(dtype=5) == xs.XS_ERR_DTYPE
    assert _passed(xs, f(qo=A(0)))
    assert _passed(xs, f(k=A(0) + 1024, v=A(0) + 1536, qo=A(0), qs=1024, ks=1024, vs=1024, os_=1024))   # a fused projection
    both = S3(2 * 16 * 256, 256, 128)
    assert _passed(xs, f(vc=A(6) + 2 * 16 * 256, kst=both, vst=both))                                   # one buffer, by pages
    assert f(vc=A(6) + 2 * 16 * 256 - 16, kst=both, vst=both) == f(vc=A(6) + 16 * 256, kst=both, vst=both) == xs.XS_ERR_OVERLAP
    tok = S3(16 * 512, 512, 128)
    assert _passed(xs, f(vc=A(6) + 512, kst=tok, vst=tok)) and _passed(xs, f(kc=A(6) + 512, vc=A(6), kst=tok, vst=tok))
    assert f(vc=A(6) + 256, kst=tok, vst=tok) == f(vc=A(6) + 16 * 1024, kst=tok, vst=tok) == xs.XS_ERR_OVERLAP
    head = S3(16 * 512, 512, 256)
    assert _passed(xs, f(vc=A(6) + 256, kst=head, vst=head)) and f(vc=A(6) + 512, kst=head, vst=head) == xs.XS_ERR_OVERLAP
    assert f(vc=A(6) + 512, kst=tok, vst=S3(16 * 512, 512, 136)) == xs.XS_ERR_OVERLAP                   # unlike strides: not told apart
    assert _passed(xs, f(Hkv=1, ks=128, vs=128, kst=S3(2048, 128, 1), vst=S3(2048, 128, 0)))            # one head: its stride is not used


# ------------------------------------------------------------------------------- step
def _step(xs, **kw):
    a = dict(cached=A(0), new=A(1), table=A(2), free=A(3), count=A(4), n=10, width=5, pages=100, page=16, rows=20, kv=A(5),
             cu=A(6), pos=A(7), slots=A(8), count_out=A(9), status=A(10))
    a.update(kw)
    return xs.lib.xs_paged_step(*a.values(), None)


def test_step_refusals(xs):
    f = lambda **k: _step(xs, **k)   # noqa: E731
    names = ("cached", "new", "table", "free", "count", "kv", "cu", "pos", "slots", "count_out", "status")
    for name in names:
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert f(n=0) == f(n=8193) == f(width=0) == f(rows=0) == f(width=2 ** 28) == f(pages=0) == xs.XS_ERR_SHAPE
    assert f(page=15) == f(page=2048) == f(page=24) == xs.XS_ERR_PAGE
    assert f(slots=A(8) + 4) == f(cached=A(0) + 1) == xs.XS_ERR_ALIGNMENT
    assert f(kv=A(0)) == f(count_out=A(4)) == f(cu=A(5)) == f(pos=A(8) + 156) == f(table=A(3) + 396) == xs.XS_ERR_OVERLAP
    assert f(free=A(2)) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f()) and _passed(xs, f(n=8192, width=2 ** 20))


# -------------------------------------------------------------------------- attention
def _plan(xs, **kw):
    a = dict(cu=A(0), kv=A(1), n=4, H=8, Hkv=2, D=128, max_q=1, causal=1, window=0, ws=A(2), nbytes=1 << 30)
    a.update(kw)
    return xs.lib.xs_attn_paged_plan(*a.values(), None)


def _attn(xs, **kw):
    a = dict(q=A(0), kc=A(1), vc=A(2), table=A(3), layout=1, outs=[A(4) + (i << 28) for i in range(16)],
             lse=A(5), T=16, H=8, Hkv=2, D=128, P=1, qs=1024, n=4, width=10, ts=10, pages=64, page=16,
             kst=S3(4096, 256, 128), vst=S3(4096, 256, 128), dtype=0, max_q=1, causal=1, window=0, scale=0.1, ws=A(6),
             nbytes=1 << 30)
    a.update(kw)
    c = Cache(a["kc"], a["vc"], a["kst"], a["vst"], a["pages"], a["page"], a["Hkv"], a["D"], a["dtype"], 0)
    g = AttnArgs(a["q"], a["table"], a["lse"], a["ws"], a["nbytes"], (ctypes.c_void_p * 16)(*a["outs"]), c, a["qs"], a["ts"],
                 *(a[n] for n in ("layout", "P", "T", "H", "n", "width", "max_q", "causal", "window", "scale")))
    return xs.lib.xs_attn_paged_fwd(bytes(g), None)


def test_plan_refusals(xs):
    f = lambda **k: _plan(xs, **k)   # noqa: E731
    assert f(cu=None) == f(kv=None) == f(ws=None) == xs.XS_ERR_NULL
    assert f(n=0) == f(n=8193) == f(H=0) == f(Hkv=0) == f(max_q=0) == f(window=-1) == xs.XS_ERR_SHAPE
    assert f(window=5, causal=0) == xs.XS_ERR_SHAPE
    assert f(D=96) == xs.XS_ERR_HEAD_DIM
    assert f(Hkv=3) == xs.XS_ERR_DIVISIBILITY
    assert f(cu=A(0) + 2) == f(ws=A(2) + 128) == xs.XS_ERR_ALIGNMENT
    assert f(cu=A(2) + 256) == xs.XS_ERR_OVERLAP
    assert _passed(xs, f(window=1))


def test_attention_refusals(xs):
    f = lambda **k: _attn(xs, **k)   # noqa: E731
    for name in ("q", "kc", "vc", "table", "ws"):
        assert f(**{name: None}) == xs.XS_ERR_NULL, name
    assert xs.lib.xs_attn_paged_fwd(None, None) == xs.XS_ERR_NULL
    assert f(outs=[]) == f(outs=[A(4), A(7)], layout=0, P=4) == xs.XS_ERR_NULL
    assert f(T=0) == f(qs=1000) == f(width=0) == f(ts=9) == f(n=0) == f(max_q=0) == f(window=3, causal=0) == xs.XS_ERR_SHAPE
    assert f(pages=0) == f(pages=2 ** 28) == f(kst=S3(4096, 64, 128)) == xs.XS_ERR_SHAPE
    assert f(layout=3) == xs.XS_ERR_LAYOUT
    assert f(layout=0, P=17) == xs.XS_ERR_TOO_MANY_RANKS
    assert f(layout=0, P=3) == f(layout=2, P=3) == f(H=8, Hkv=3) == xs.XS_ERR_DIVISIBILITY
    assert f(page=20) == xs.XS_ERR_PAGE
    assert f(dtype=2) == xs.XS_ERR_DTYPE
    assert f(scale=float("nan")) == f(scale=-1.0) == xs.XS_ERR_SCALE
    assert f(q=A(0) + 8) == f(qs=1028) == f(kst=S3(4100, 256, 128)) == f(lse=A(5) + 2) == f(ws=A(6) + 16) == xs.XS_ERR_ALIGNMENT
    assert f(lse=A(4)) == f(ws=A(0)) == f(lse=A(1) + 64) == xs.XS_ERR_OVERLAP
    assert f(outs=[A(2) + 16]) == f(outs=[A(4), A(4)], layout=0, P=2) == xs.XS_ERR_OVERLAP
    assert f(D=96) == xs.XS_ERR_HEAD_DIM
    assert _passed(xs, f(lse=None)) and _passed(xs, f(layout=0, P=4)) and _passed(xs, f(n=1, ts=0))


def test_workspace_bytes_refusals(xs):
    b = ctypes.c_size_t(0)
    f = lambda *a: xs.lib.xs_attn_paged_workspace_bytes(*a, ctypes.byref(b))   # noqa: E731
    assert xs.lib.xs_attn_paged_workspace_bytes(1, 1, 1, 64, None) == xs.XS_ERR_NULL
    assert f(0, 1, 1, 64) == xs.XS_ERR_SHAPE and f(1, 1, 1, 48) == xs.XS_ERR_HEAD_DIM and f(1, 3, 2, 64) == xs.XS_ERR_DIVISIBILITY


def test_python_refuses_host_tensors_and_wrong_types(xs):
    x, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    rope = xs.Rope(64)
    with pytest.raises(TypeError, match="current device"):
        xs.xs_rope_fwd(x, pos, x, rope)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        xs.xs_rope_fwd(x.float(), pos, x, rope)
    with pytest.raises(TypeError, match="D = 128"):
        xs.xs_rope_fwd(x, pos, x, xs.Rope(128))
    with pytest.raises(TypeError):
        xs.xs_paged_step(*([pos] * 5), 16, *([pos] * 6))


def test_native_binding_leaves_host_tensors_to_python(xs):
    xs._device()
    if xs._native is None:
        from importlib import util
        assert util.find_spec("torch") is None or xs.__file__ is None or not os.path.exists(
            os.path.join(os.path.dirname(xs.__file__), "_binding.so"))
        return
    x, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    rope, n = xs.Rope(64), xs._native
    assert n.rope(x, pos, x, rope.ptr, 64, 0, None) is None
    assert n.rope(x, pos) is None and n.rope(None, 1, 2, 3, 4, 5, 6) is None         # too few; not tensors
    assert n.step(*([pos] * 5), 16, *([pos] * 6), None) is None
    assert n.plan(pos, pos, 1, pos, (1, 1, 1, 64, 0, 0), 1, 0, None) is None
    assert n.append(x, x, x, pos, pos, x, x, x, rope.ptr, 64, None) is None
    assert n.attn(x, x, x, pos, 1, [x], 0.1, pos, (), (1, 1, 0), None, None) is None
    with pytest.raises(ValueError):
        n.bind(1, 2, 3, 4, 0)


def test_copies_of_a_rope_stand_alone(xs):
    import copy
    import pickle
    a = xs.Rope(128, 48, base=5e5, scaling=xs.XS_ROPE_LINEAR, factor=2.0)
    want = bytes(a._struct)
    for b in (copy.copy(a), copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        assert b.ptr != a.ptr and bytes(b._struct) == want and ctypes.addressof(b._struct) == b.ptr


# ------------------------------------------------------------------- division of work
def test_division_of_work(tmp_path):
    """Every block of every tile once, pieces in CTA order, the record of cut tiles right, for
    random batches; the closed forms of the cost against sums over tiles and rows."""
    cxx, nvcc = shutil.which("g++"), shutil.which("nvcc")
    root = os.path.dirname(os.path.dirname(os.path.realpath(nvcc))) if nvcc else "/usr/local/cuda"
    if cxx is None or not os.path.exists(os.path.join(root, "include", "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = str(tmp_path / "paged_plan_check")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, "-I", os.path.join(root, "include"),
                    os.path.join(HERE, "paged_plan_check.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    r = random.Random(5)
    log = lambda lo, hi: min(hi, int(math.exp(r.uniform(math.log(lo), math.log(hi + 1)))))   # noqa: E731
    cases = []
    for _ in range(1500):
        G = r.choice([1, 2, 3, 4, 5, 8, 16, 32])
        rows, block, grid, cost, snap, whole, least = r.choice([
            (16, 32, 304, 256, 4, 16, 512), (32, 32, 304, 64, 4, 16, 160), (128, 128, 152, 384, 2, 4, 1024),
            (128, 128, 148, 0, 1, 0, 128), (16, 64, 304, 16, 1, 3, 64), (128, 128, 152, 300, 5, 2, 512)])
        causal = r.randint(0, 1)
        window = log(1, 5000) if causal and r.random() < 0.4 else 0
        n = log(1, 40)
        lens = []
        for _ in range(n):
            q = r.choice([0, 1, 1, log(1, 3000)])
            lens += [q, max(0, r.choice([q + log(1, 20000), q, q - r.randint(0, q), 0]))]
        cases.append(" ".join(map(str, [max(1, rows // G), block, grid, cost, snap, whole, least, r.choice([1, 2, 8, 24]), causal, window,
                                n]
                                  + lens)))
    p = subprocess.run([exe], input="\n".join(cases), capture_output=True, text=True)
    out = p.stdout.strip().split("\n")
    assert p.returncode == 0 and len(out) == len(cases), (out[-1], cases[len(out) - 1])
    assert all(line.startswith("ok") for line in out)


# -------------------------------------------------------------- the tests' references
def test_step_reference_by_hand():
    """Pages of 4 tokens: request 0 decodes into its page, 1 ends, 2 needs two pages, 3 one, 4 none left."""
    ref = pg.step_reference(np.array([2, 5, 0, 4, 8]), np.array([1, -1, 5, 1, 1]),
                            np.array([[6, 0, 0], [3, 1, 0], [0, 0, 0], [2, 0, 0], [7, 8, 0]]), np.array([5, 0, 0, 0, 0, 0, 0, 0, 0]), 1, 4, 20)
    # list: 5, 3, 1 -> request 2 takes 1, 3; request 3 takes 5; request 4 finds nothing
    assert ref["status"].tolist() == [0, 0, 0, 0, 1] and ref["free_count"] == 0
    assert ref["table"].tolist() == [[6, 0, 0], [3, 1, 0], [1, 3, 0], [2, 5, 0], [7, 8, 0]]
    assert ref["free"][:3].tolist() == [5, 3, 1] and ref["cu_q"].tolist() == [0, 1, 1, 6, 7, 7]
    assert ref["kv_lens"].tolist() == [3, 0, 5, 5, 8]
    assert ref["positions"][:8].tolist() == [2, 0, 1, 2, 3, 4, 4, 0]
    assert ref["slots"][:8].tolist() == [26, 4, 5, 6, 7, 12, 20, -1]


def test_attention_reference_by_hand():
    q, k, v = np.array([[1.0], [1.0]]), np.array([[0.0], [np.log(2.0)], [np.log(4.0)]]), np.array([[1.0], [10.0], [100.0]])
    out, mass, lse = pg.attention_reference(q, k, v, 3, True, 0, 1.0)
    np.testing.assert_allclose(out[:, 0], [21 / 3, 421 / 7])
    np.testing.assert_allclose(lse, np.log([3.0, 7.0]))
    out, _, lse = pg.attention_reference(q, k, v, 3, True, 2, 1.0)
    np.testing.assert_allclose(out[:, 0], [21 / 3, 420 / 6])
    out, _, lse = pg.attention_reference(q, k[:1], v[:1], 1, True, 0, 1.0)
    assert out[:, 0].tolist() == [0.0, 1.0] and lse.tolist() == [-np.inf, 0.0]


def test_rope_reference_by_hand():
    x = np.zeros((1, 1, 64))
    x[0, 0, 0] = 1.0
    y, _ = pg.rope_reference(x, np.array([1]), pg.frequencies(64), False)
    assert abs(y[0, 0, 0] - math.cos(1)) < 1e-15 and abs(y[0, 0, 32] - math.sin(1)) < 1e-15
    y, _ = pg.rope_reference(x, np.array([1]), pg.frequencies(64), True)
    assert abs(y[0, 0, 1] - math.sin(1)) < 1e-15
