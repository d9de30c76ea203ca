"""Fused sequence-parallel attention + Ulysses All-to-All layout for GB300.

Python binding of ``libxsattn.so`` (hand-written sm_103a CUDA kernels behind a
C ABI, declared in ``include/xsattn.h``).  This module only marshals
arguments: it turns torch tensors into pointers and sizes, picks the current
CUDA stream, and raises :class:`XsError` on a non-zero return code.  Every
step of the computation runs in the library's kernels; there is no fallback.
PyTorch is used for device memory and streams only.

Method: X-Stage (arXiv 2607.23264), abstract and the gist.science technical
summary, "Key Contributions" item 3: the attention output-tile owner stores
each finished tile straight into the post-attention Ulysses All-to-All layout
(the sequence shard of the rank that owns the tile's rows) and resumes its next
tile.  On one GPU the P ranks are P device buffers.
"""
from __future__ import annotations

import ctypes
import os
import struct

__all__ = [
    "XsError",
    "lib",
    "xs_attn_a2a_fwd",
    "xs_attn_fwd",
    "xs_attn_heads_fwd",
    "xs_relayout_a2a",
    "xs_relayout_a2a_inverse",
    "xs_attn_ulysses_fwd",
    "xs_attn_ulysses_rank_fwd",
    "xs_burst_gap",
    "xs_attn_a2a_fwd_staged",
    "xs_attn_workspace_bytes",
    "xs_attn_fwd_balanced",
    "xs_attn_fwd_balanced_noalloc",
    "xs_attn_causal_fwd",
    "xs_attn_varlen_fwd",
    "Workspace",
    "Rope",
    "xs_rope_init",
    "xs_rope_fwd",
    "xs_rope_append_paged",
    "xs_paged_step",
    "PagedWorkspace",
    "xs_attn_paged_workspace_bytes",
    "xs_attn_paged_plan",
    "xs_attn_paged_fwd",
    "xs_attn_get_device_error",
    "xs_attn_get_device_error_info",
    "xs_attn_error_string",
    "attn_a2a",
    "LIB_PATH",
    "EXPORTS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libxsattn.so")

# Error codes of include/xsattn.h
XS_OK = 0
XS_ERR_NULL = -1
XS_ERR_SHAPE = -2
XS_ERR_HEAD_DIM = -3
XS_ERR_DIVISIBILITY = -4
XS_ERR_TOO_MANY_RANKS = -5
XS_ERR_ALIGNMENT = -6
XS_ERR_OVERLAP = -7
XS_ERR_SCALE = -8
XS_ERR_CUDA = -9
XS_ERR_DEVICE_TIMEOUT = -10
XS_ERR_UNSUPPORTED_DEVICE = -11
XS_ERR_WORKSPACE = -12
XS_ERR_LAYOUT = -13
XS_ERR_DEVICE_DRAIN = -14
XS_ERR_DEVICE_BOUNDS = -15
XS_ERR_UNAVAILABLE = -16
XS_ERR_DTYPE = -17
XS_ERR_PAGE = -18
XS_ERR_ROPE = -19
XS_DTYPE_BF16 = 0
XS_DTYPE_FP16 = 1
XS_ROPE_HALF = 0
XS_ROPE_INTERLEAVED = 1
XS_ROPE_PLAIN = 0
XS_ROPE_LINEAR = 1
XS_ROPE_STRETCH = 2
XS_ROPE_BY_PARTS = 3
XS_MAX_P = 16
XS_LAYOUT_A2A = 0
XS_LAYOUT_CONTIGUOUS = 1
XS_LAYOUT_HEADS = 2

_vp = ctypes.c_void_p
_int = ctypes.c_int
_f32 = ctypes.c_float
_size = ctypes.c_size_t
_i64 = ctypes.c_longlong
_f64 = ctypes.c_double


class _RopeStruct(ctypes.Structure):
    """``xs_rope`` of include/xsattn.h."""

    _fields_ = [("turns", ctypes.c_ulonglong * 64), ("magnitude", _f32), ("layout", _int), ("rot", _int), ("D", _int)]


# name -> (restype, argtypes); the full exported C ABI
EXPORTS = {
    "xs_attn_a2a_fwd": (_int, [_vp, _vp, _vp, ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _f32, _vp]),
    "xs_attn_fwd": (_int, [_vp, _vp, _vp, _vp, _int, _int, _int, _int, _f32, _vp]),
    "xs_attn_heads_fwd": (_int, [_vp, _vp, _vp, ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _f32, _vp]),
    "xs_relayout_a2a": (_int, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _vp]),
    "xs_attn_a2a_fwd_staged": (_int, [_vp, _vp, _vp, ctypes.POINTER(_vp), _vp, _vp, _vp, ctypes.POINTER(_vp),
                                      _int, _int, _int, _int, _int, _f32, _vp, _size, _vp]),
    "xs_attn_workspace_bytes": (_int, [_int, _int, _int, _int, ctypes.POINTER(_size)]),
    "xs_attn_fwd_balanced": (_int, [_vp, _vp, _vp, _int, ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _f32,
                                    _vp, _size, _vp]),
    "xs_attn_fwd_balanced_noalloc": (_int, [_vp, _vp, _vp, _int, ctypes.POINTER(_vp), _int, _int, _int, _int, _int,
                                            _f32, _vp]),
    "xs_attn_causal_fwd": (_int, [_vp, _vp, _vp, _int, ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _f32,
                                  _vp]),
    "xs_attn_varlen_fwd": (_int, [_vp, _vp, _vp, ctypes.POINTER(_int), _int, _int, _int, ctypes.POINTER(_vp), _int,
                                  _int, _int, _int, _f32, _vp]),
    "xs_attn_ulysses_fwd": (_int, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                   ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _f32, _vp, _size, _vp]),
    "xs_relayout_a2a_inverse": (_int, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _int, _int, _int, _int, _int,
                                       _vp]),
    "xs_attn_ulysses_rank_fwd": (_int, [_vp, _vp, _vp, ctypes.POINTER(_vp), _int, _int, _int, _int, _int, _int, _f32,
                                        _vp, _size, _vp]),
    "xs_rope_init": (_int, [_vp, _int, _int, _int, _f64, _int, _f64, _f64, _f64, _f64, _f64]),
    "xs_rope_fwd": (_int, [_vp, _vp, _vp, _int, _int, _i64, _i64, _int, _int, _vp, _vp]),
    "xs_rope_append_paged": (_int, [ctypes.c_char_p, _vp]),
    "xs_paged_step": (_int, [_vp] * 5 + [_int] * 5 + [_vp] * 7),
    "xs_attn_paged_workspace_bytes": (_int, [_int, _int, _int, _int, ctypes.POINTER(_size)]),
    "xs_attn_paged_plan": (_int, [_vp, _vp] + [_int] * 7 + [_vp, _size, _vp]),
    "xs_attn_paged_fwd": (_int, [ctypes.c_char_p, _vp]),
    "xs_burst_gap": (_int, [_vp, _size, _int, _size, _int, ctypes.c_longlong, ctypes.c_longlong, _vp, _vp]),
    "xs_attn_get_device_error": (_int, [_vp]),
    "xs_attn_get_device_error_info": (_int, [_vp, ctypes.POINTER(_int), _int]),
    "xs_attn_error_string": (ctypes.c_char_p, [_int]),
    "xs_attn_last_cuda_error": (_int, []),
    "xs_attn_version": (_int, []),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: the CUDA library has not been built "
            "(run `python -c 'import __graft_entry__ as g; g.build()'`); there is no fallback")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in EXPORTS.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


lib = _load()


class XsError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = lib.xs_attn_error_string(code).decode()
        if code == XS_ERR_CUDA:
            msg += f" (cudaError {lib.xs_attn_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{code}]")


def _check(code: int, where: str) -> None:
    if code != XS_OK:
        raise XsError(code, where)


def _c_int(x: int, code: int, where: str) -> int:
    """``x`` if a C int holds it (ctypes would pass its lower 32 bits on), else the refusal ``code``."""
    if not -0x80000000 <= x <= 0x7fffffff:
        raise XsError(code, where)
    return x


def _ptr_array(ptrs):
    arr = (_vp * max(1, len(ptrs)))()
    for i, p in enumerate(ptrs):
        arr[i] = p
    return arr


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _bshd(t, name):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
        raise TypeError(f"{name} must be a contiguous CUDA bfloat16 tensor [B,S,H,D]")
    return t


def xs_attn_a2a_fwd(q, k, v, out_ptrs, scale: float, stream=None) -> None:
    """Fused attention; writes P sequence shards ``out_ptrs[p]`` of shape [B,S/P,H,D]."""
    B, S, H, D = _bshd(q, "q").shape
    _bshd(k, "k"), _bshd(v, "v")
    outs = [_bshd(o, "out") for o in out_ptrs]
    _check(lib.xs_attn_a2a_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr_array([o.data_ptr() for o in outs]),
                               B, S, H, D, len(outs), scale, _stream_handle(stream)), "xs_attn_a2a_fwd")


def xs_attn_fwd(q, k, v, out, scale: float, stream=None) -> None:
    """Same attention kernel, one contiguous [B,S,H,D] output."""
    B, S, H, D = _bshd(q, "q").shape
    _bshd(k, "k"), _bshd(v, "v"), _bshd(out, "out")
    _check(lib.xs_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, S, H, D, scale,
                           _stream_handle(stream)), "xs_attn_fwd")


def xs_attn_heads_fwd(q, k, v, heads, scale: float, stream=None) -> None:
    """Same attention kernel, writing the P Ulysses head shards [B,S,H/P,D]."""
    B, S, H, D = _bshd(q, "q").shape
    _bshd(k, "k"), _bshd(v, "v")
    hs = [_bshd(x, "heads") for x in heads]
    _check(lib.xs_attn_heads_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr_array([x.data_ptr() for x in hs]),
                                 B, S, H, D, len(hs), scale, _stream_handle(stream)), "xs_attn_heads_fwd")


def xs_relayout_a2a(heads, out_ptrs, stream=None) -> None:
    """Separate All-to-All re-layout: head shards [B,S,H/P,D] -> sequence shards [B,S/P,H,D]."""
    hs = [_bshd(x, "heads") for x in heads]
    outs = [_bshd(o, "out") for o in out_ptrs]
    P = len(hs)
    B, S, Hl, D = hs[0].shape
    _check(lib.xs_relayout_a2a(_ptr_array([x.data_ptr() for x in hs]), _ptr_array([o.data_ptr() for o in outs]),
                               B, S, Hl * P, D, P, _stream_handle(stream)), "xs_relayout_a2a")


def xs_attn_ulysses_fwd(q_shards, k_shards, v_shards, out_shards, scale: float, workspace=None,
                        stream=None) -> None:
    """The Ulysses attention step of P virtual ranks in one launch: inputs are the P sequence
    shards [B,S/P,H,D] of Q, K and V, outputs the P sequence shards [B,S/P,H,D] of O."""
    qs = [_bshd(x, "q_shards") for x in q_shards]
    ks = [_bshd(x, "k_shards") for x in k_shards]
    vs = [_bshd(x, "v_shards") for x in v_shards]
    os_ = [_bshd(x, "out_shards") for x in out_shards]
    P = len(qs)
    B, Sl, H, D = qs[0].shape
    wp, wn = _ws(workspace)
    _check(lib.xs_attn_ulysses_fwd(_ptr_array([x.data_ptr() for x in qs]), _ptr_array([x.data_ptr() for x in ks]),
                                   _ptr_array([x.data_ptr() for x in vs]), _ptr_array([x.data_ptr() for x in os_]),
                                   B, Sl * P, H, D, P, scale, wp, wn, _stream_handle(stream)), "xs_attn_ulysses_fwd")


def xs_attn_ulysses_rank_fwd(q_heads, k_heads, v_heads, out_shard_ptrs, H: int, rank: int, scale: float,
                             workspace=None, stream=None) -> None:
    """Attention of Ulysses rank ``rank`` over its head shard [B,S,H/P,D] (q, k, v), storing
    every output row straight into ``out_shard_ptrs[p]`` (device addresses of the P ranks'
    sequence shards [B,S/P,H,D], which may belong to other processes) at global head
    rank*H/P + j.  ``out_shard_ptrs``: ints (device pointers) or CUDA tensors."""
    B, S, Hl, D = _bshd(q_heads, "q_heads").shape
    _bshd(k_heads, "k_heads"), _bshd(v_heads, "v_heads")
    ptrs = [p if isinstance(p, int) else _bshd(p, "out_shards").data_ptr() for p in out_shard_ptrs]
    P = len(ptrs)
    wp, wn = _ws(workspace)
    _check(lib.xs_attn_ulysses_rank_fwd(q_heads.data_ptr(), k_heads.data_ptr(), v_heads.data_ptr(), _ptr_array(ptrs),
                                        B, S, H, D, P, rank, scale, wp, wn, _stream_handle(stream)),
           "xs_attn_ulysses_rank_fwd")


def xs_relayout_a2a_inverse(seq_shards, heads, stream=None) -> None:
    """Separate pre-attention All-to-All: sequence shards [B,S/P,H,D] -> head shards [B,S,H/P,D]."""
    ss = [_bshd(x, "seq_shards") for x in seq_shards]
    hs = [_bshd(x, "heads") for x in heads]
    P = len(ss)
    B, Sl, H, D = ss[0].shape
    _check(lib.xs_relayout_a2a_inverse(_ptr_array([x.data_ptr() for x in ss]), _ptr_array([x.data_ptr() for x in hs]),
                                       B, Sl * P, H, D, P, _stream_handle(stream)), "xs_relayout_a2a_inverse")


def xs_burst_gap(dst, producers: int, burst_bytes: int, bursts: int, gap_ns: int, stream=None, lead_ns: int = 0):
    """Run the Burst-Gap store microbenchmark into the CUDA tensor ``dst`` (any dtype, contiguous);
    returns the device int64 tensor [bursts, producers] of burst issue times in ns."""
    import torch
    if not dst.is_cuda or not dst.is_contiguous():
        raise TypeError("dst must be a contiguous CUDA tensor")
    times = torch.empty((bursts, producers), dtype=torch.int64, device=dst.device)
    _check(lib.xs_burst_gap(dst.data_ptr(), dst.numel() * dst.element_size(), producers, burst_bytes, bursts,
                            lead_ns, gap_ns, times.data_ptr(), _stream_handle(stream)), "xs_burst_gap")
    return times


def xs_attn_a2a_fwd_staged(q_host, k_host, v_host, out_host, q_dev, k_dev, v_dev, out_dev, scale: float,
                           workspace=None, stream=None) -> None:
    """Host-resident variant: H2D copies, fused kernel and D2H copies of the shards, all on ``stream``.
    ``workspace``: a :class:`Workspace` (balanced schedule) or None (plain schedule)."""
    B, S, H, D = q_host.shape
    P = len(out_dev)
    wp, wn = _ws(workspace)
    _check(lib.xs_attn_a2a_fwd_staged(
        q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(), _ptr_array([o.data_ptr() for o in out_host]),
        q_dev.data_ptr(), k_dev.data_ptr(), v_dev.data_ptr(), _ptr_array([o.data_ptr() for o in out_dev]),
        B, S, H, D, P, scale, wp, wn, _stream_handle(stream)), "xs_attn_a2a_fwd_staged")


def xs_attn_workspace_bytes(B: int, S: int, H: int, D: int) -> int:
    """Workspace bytes the balanced schedule needs for this shape on the current device (0: no split)."""
    n = _size(0)
    _check(lib.xs_attn_workspace_bytes(B, S, H, D, ctypes.byref(n)), "xs_attn_workspace_bytes")
    return n.value


class Workspace:
    """A zero-filled device workspace for :func:`xs_attn_fwd_balanced` (torch-allocated,
    256-byte aligned).  ``Workspace.for_shape(B, S, H, D)`` sizes it for one shape;
    ``None`` is returned there when the shape needs none."""

    def __init__(self, nbytes: int, device="cuda"):
        import torch
        self.nbytes = int(nbytes)
        self._buf = torch.zeros(self.nbytes + 256, dtype=torch.uint8, device=device)
        base = self._buf.data_ptr()
        self.ptr = (base + 255) & ~255

    @classmethod
    def for_shape(cls, B: int, S: int, H: int, D: int, device="cuda"):
        n = xs_attn_workspace_bytes(B, S, H, D)
        return cls(n, device) if n else None


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.ptr, workspace.nbytes


def xs_attn_fwd_balanced(q, k, v, layout: int, outs, scale: float, workspace, stream=None) -> None:
    """The attention kernel with the last partial wave of tiles balanced over all SMs.
    ``layout``: XS_LAYOUT_A2A (P sequence shards), XS_LAYOUT_CONTIGUOUS (one [B,S,H,D]
    tensor) or XS_LAYOUT_HEADS (P head shards); ``workspace``: a :class:`Workspace` or None."""
    B, S, H, D = _bshd(q, "q").shape
    _bshd(k, "k"), _bshd(v, "v")
    os_ = [_bshd(o, "out") for o in outs]
    wp, wn = _ws(workspace)
    _check(lib.xs_attn_fwd_balanced(q.data_ptr(), k.data_ptr(), v.data_ptr(), layout,
                                    _ptr_array([o.data_ptr() for o in os_]), B, S, H, D, len(os_), scale, wp, wn,
                                    _stream_handle(stream)), "xs_attn_fwd_balanced")


def xs_attn_get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status code."""
    return lib.xs_attn_get_device_error(_stream_handle(stream))


def xs_attn_get_device_error_info(stream=None):
    """Synchronise the stream; return (status code, record of the first device error as a
    dict) and clear both (see include/xsattn.h for the fields)."""
    info = (_int * 8)()
    code = lib.xs_attn_get_device_error_info(_stream_handle(stream), info, 8)
    keys = ("kind", "cta", "warp", "lane", "site", "detail0", "detail1", "detail2")
    return code, dict(zip(keys, list(info)))


def xs_attn_error_string(code: int) -> str:
    return lib.xs_attn_error_string(code).decode()


def xs_attn_fwd_balanced_noalloc(q, k, v, layout: int, outs, scale: float, stream=None) -> None:
    """:func:`xs_attn_fwd_balanced` with the library's own scratch array as workspace (no
    allocation on the call path; calls that overlap in time race on the one array)."""
    B, S, H, D = _bshd(q, "q").shape
    _bshd(k, "k"), _bshd(v, "v")
    os_ = [_bshd(o, "out") for o in outs]
    _check(lib.xs_attn_fwd_balanced_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), layout,
                                            _ptr_array([o.data_ptr() for o in os_]), B, S, H, D, len(os_), scale,
                                            _stream_handle(stream)), "xs_attn_fwd_balanced_noalloc")


def xs_attn_causal_fwd(q, k, v, layout: int, outs, scale: float, stream=None) -> None:
    """Causal attention (row s attends to keys 0 .. s) with the fused output layouts:
    ``layout`` XS_LAYOUT_A2A (P sequence shards), XS_LAYOUT_CONTIGUOUS (one [B,S,H,D]
    tensor) or XS_LAYOUT_HEADS (P head shards)."""
    B, S, H, D = _bshd(q, "q").shape
    _bshd(k, "k"), _bshd(v, "v")
    os_ = [_bshd(o, "out") for o in outs]
    _check(lib.xs_attn_causal_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), layout,
                                  _ptr_array([o.data_ptr() for o in os_]), B, S, H, D, len(os_), scale,
                                  _stream_handle(stream)), "xs_attn_causal_fwd")


def _thd(t, name):
    import torch
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
        raise TypeError(f"{name} must be a contiguous CUDA bfloat16 tensor [T,H,D]")
    return t


def xs_attn_varlen_fwd(q, k, v, seqlens, layout: int, outs, scale: float, causal: bool = False,
                       stream=None) -> None:
    """Attention over packed variable-length sequences: ``q``, ``k``, ``v`` are
    [T, H, D] bf16 holding sequences of lengths ``seqlens`` (host integers) back to
    back; each row attends to its own sequence (``causal=True``: to its own
    sequence's keys up to its own position; run as one causal launch per
    sequence).
    ``layout`` XS_LAYOUT_A2A (P shards [T/P, H, D]), XS_LAYOUT_CONTIGUOUS (one
    [T, H, D] tensor) or XS_LAYOUT_HEADS (P head shards [T, H/P, D])."""
    T, H, D = _thd(q, "q").shape
    _thd(k, "k"), _thd(v, "v")
    os_ = [_thd(o, "out") for o in outs]
    lens = (ctypes.c_int * max(1, len(seqlens)))(*[int(n) for n in seqlens])
    _check(lib.xs_attn_varlen_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), lens, len(seqlens), int(bool(causal)),
                                  layout, _ptr_array([o.data_ptr() for o in os_]), T, H, D, len(os_), scale,
                                  _stream_handle(stream)), "xs_attn_varlen_fwd")


# ---- serving: new tokens over a paged cache


class Rope:
    """Rotary positions of a model (``xs_rope`` of the C ABI): head dimension ``D``, the first
    ``rot`` channels of a head rotated, ``layout`` XS_ROPE_HALF or XS_ROPE_INTERLEAVED, ``base``,
    and the scaling of long contexts (``scaling`` XS_ROPE_PLAIN, _LINEAR, _STRETCH or _BY_PARTS
    with ``factor``, ``context``, ``low``, ``high``; ``magnitude`` multiplies cos and sin)."""

    def __init__(self, D: int, rot: int | None = None, layout: int = XS_ROPE_HALF, base: float = 10000.0,
                 scaling: int = XS_ROPE_PLAIN, factor: float = 1.0, context: float = 0.0, low: float = 1.0,
                 high: float = 32.0, magnitude: float = 1.0):
        self._struct = _RopeStruct()
        self.ptr = ctypes.addressof(self._struct)
        xs_rope_init(self, D, D if rot is None else rot, layout, base, scaling, factor, context, low, high, magnitude)

    def __reduce__(self):   # copies have a table of their own
        return Rope, self._args


def xs_rope_init(rope: Rope, D: int, rot: int, layout: int, base: float, scaling: int, factor: float,
                 context: float, low: float, high: float, magnitude: float) -> None:
    """Fill ``rope`` on the host (``Rope(...)`` calls it); a refused call leaves it as it was."""
    where = "xs_rope_init"
    _check(lib.xs_rope_init(rope.ptr, _c_int(D, XS_ERR_HEAD_DIM, where), _c_int(rot, XS_ERR_ROPE, where),
                            _c_int(layout, XS_ERR_LAYOUT, where), base, _c_int(scaling, XS_ERR_ROPE, where), factor, context,
                            low, high, magnitude), where)
    rope.D, rope.rot = D, rot
    rope._args = (D, rot, layout, base, scaling, factor, context, low, high, magnitude)


# The checks below run on every call of a decoding loop, where they cost more than the
# kernels: the accepted case takes a few attribute reads per tensor, and the reason of a
# refusal is worked out only once there is one.  Where the native binding (csrc/binding.cpp)
# has been built for this torch, it reads the tensors and makes the call itself; what it does
# not accept (it returns None) goes through the checks here.
_I32 = _I64 = _F32 = None
_DTYPES = {}
_current_device = _raw_stream = None
_native = None


def _bind_native(torch):
    try:
        from . import _binding
    except ImportError:     # not built here, or for another torch
        return None
    if _binding.torch_version != torch.__version__.partition("+")[0]:
        return None
    names = ("xs_rope_fwd", "xs_rope_append_paged", "xs_paged_step", "xs_attn_paged_plan", "xs_attn_paged_fwd")
    _binding.bind(*(ctypes.cast(getattr(lib, name), _vp).value for name in names))
    return _binding


def _bind_torch():
    global _I32, _I64, _F32, _current_device, _raw_stream, _native
    import torch
    _native = _bind_native(torch)
    _DTYPES.update({torch.bfloat16: XS_DTYPE_BF16, torch.float16: XS_DTYPE_FP16})
    if torch.cuda.is_available():
        torch.cuda.init()
        _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    else:
        _current_device, _raw_stream = (lambda: -2), (lambda dev: 0)   # no tensor is on device -2
    _I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _device():
    """The current device's index (-2 without CUDA)."""
    if _I32 is None:
        _bind_torch()
    return _current_device()


def _stream_of(stream, dev):
    return _raw_stream(dev) if stream is None else _stream_handle(stream)


def _handle(stream):
    return None if stream is None else _stream_handle(stream)


def _dtype_of(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be bfloat16 or float16, not {t.dtype}")
    return d


def _on_device(t, name, dev):
    if t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on the current device")


def _rows(t, name, dtype, D, dev):
    """A [T, H, D] tensor whose heads are contiguous; returns (T, H, row stride)."""
    if t.dim() != 3 or t.dtype is not dtype or t.shape[2] != D:
        raise TypeError(f"{name} must be a {dtype} tensor [T, H, D] with D = {D}")
    _on_device(t, name, dev)
    T, H, _ = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and H > 1):
        raise TypeError(f"{name}: the heads of a row must be contiguous")
    return T, H, s0 if T > 1 else H * D


def _vec(t, name, dtype, n, dev):
    """Address of a contiguous vector of n integers."""
    if t.dtype is dtype and t.dim() == 1 and t.numel() == n and t.is_contiguous():
        if t.get_device() == dev:
            return t.data_ptr()
        _on_device(t, name, dev)
    raise TypeError(f"{name} must be a contiguous {dtype} tensor of shape [{n}]")


# The argument structs of include/xsattn.h, packed in one go (no field of theirs needs padding):
# xs_paged_cache is "2Q6q6i".
_APPEND_ARGS = struct.Struct("=7Q2Q6q6i4q2i")
_ATTN_ARGS = {P: struct.Struct(f"=5Q{P}Q{8 * (XS_MAX_P - P)}x2Q6q6i2q9if") for P in range(1, XS_MAX_P + 1)}


def _cache(t, name, dtype, dev):
    """Strides of a cache [n_pages, page_size, Hkv, D] with D contiguous."""
    if t.dim() != 4 or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor [n_pages, page_size, Hkv, D]")
    _on_device(t, name, dev)
    s0, s1, s2, s3 = t.stride()
    if s3 != 1:
        raise TypeError(f"{name}: the channels of a head must be contiguous")
    return s0, s1, s2


def _same(what, a, b):
    if a != b:
        raise TypeError(f"{what}: shapes do not match ({a} against {b})")


def xs_rope_fwd(x, positions, out, rope: Rope, grad: bool = False, stream=None) -> None:
    """Rotary positions of ``x`` [T, H, D] (bf16 or fp16; rows may be slices of a wider matrix)
    into ``out`` (``out`` may be ``x``); ``grad=True`` applies the transposed map, which takes
    the gradient of ``out`` to the gradient of ``x``.  ``positions``: int32 [T]."""
    if _native is not None:
        code = _native.rope(x, positions, out, rope.ptr, rope.D, 1 if grad else 0, _handle(stream))
        if code is not None:
            return _check(code, "xs_rope_fwd") if code else None
    dev, D, dt = _device(), rope.D, x.dtype
    dtype = _dtype_of(x, "x")
    T, H, x_stride = _rows(x, "x", dt, D, dev)
    To, Ho, out_stride = _rows(out, "out", dt, D, dev)
    if T != To or H != Ho:
        _same("xs_rope_fwd", (T, H), (To, Ho))
    code = lib.xs_rope_fwd(x.data_ptr(), _vec(positions, "positions", _I32, T, dev), out.data_ptr(), T, H, x_stride,
                           out_stride, dtype, 1 if grad else 0, rope.ptr, _stream_of(stream, dev))
    if code:
        _check(code, "xs_rope_fwd")


def xs_rope_append_paged(q, k, v, positions, slots, q_out, k_cache, v_cache, rope: Rope, stream=None) -> None:
    """Rotate the new tokens' ``q`` [T, H, D] into ``q_out`` and their ``k`` [T, Hkv, D] into the
    slots of ``k_cache`` [n_pages, page_size, Hkv, D], and copy ``v`` into those of ``v_cache``.
    ``positions`` int32 [T], ``slots`` int64 [T] (outside the cache: not stored)."""
    if _native is not None:
        code = _native.append(q, k, v, positions, slots, q_out, k_cache, v_cache, rope.ptr, rope.D, _handle(stream))
        if code is not None:
            return _check(code, "xs_rope_append_paged") if code else None
    dev, D, dt = _device(), rope.D, q.dtype
    dtype = _dtype_of(q, "q")
    T, H, qs = _rows(q, "q", dt, D, dev)
    Tk, Hkv, ks = _rows(k, "k", dt, D, dev)
    Tv, Hv, vs = _rows(v, "v", dt, D, dev)
    To, Ho, os_ = _rows(q_out, "q_out", dt, D, dev)
    kc, vc = _cache(k_cache, "k_cache", dt, dev), _cache(v_cache, "v_cache", dt, dev)
    shape = k_cache.shape
    n_pages, page_size, Hc, Dc = shape
    if T != Tk or T != Tv or T != To or H != Ho or Hkv != Hv or Hc != Hkv or Dc != D or v_cache.shape != shape:
        _same("xs_rope_append_paged", [(T, H), (T, Hkv), (T, Hkv), (To, Ho), (n_pages, page_size, Hkv, D)] * 2,
              [(To, Ho), (Tk, Hkv), (Tv, Hv), (T, H), tuple(shape), (T, H), (T, Hkv), (T, Hkv), (To, Ho),
               tuple(v_cache.shape)])
    args = _APPEND_ARGS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), _vec(positions, "positions", _I32, T, dev),
                             _vec(slots, "slots", _I64, T, dev), q_out.data_ptr(), rope.ptr, k_cache.data_ptr(),
                             v_cache.data_ptr(), *kc, *vc, n_pages, page_size, Hkv, D, dtype, 0, qs, ks, vs, os_, T, H)
    code = lib.xs_rope_append_paged(args, _stream_of(stream, dev))
    if code:
        _check(code, "xs_rope_append_paged")


def xs_paged_step(cache_lens, new_lens, block_table, free_pages, free_count, page_size: int, kv_lens, cu_q, positions,
                  slots, free_count_out, status, stream=None) -> None:
    """Lay out one step on the device: pages for the new tokens of every request (from
    ``free_pages``, whose first ``free_count`` entries are free) into ``block_table``, pages of
    ended requests (``new_lens < 0``) back to the list, and ``kv_lens``, ``cu_q``, ``positions``,
    ``slots``, ``free_count_out`` and ``status`` (include/xsattn.h has the rules).  All int32
    device tensors, ``slots`` int64; ``free_pages`` has one entry per page of the cache."""
    if _native is not None:
        code = _native.step(cache_lens, new_lens, block_table, free_pages, free_count, page_size, kv_lens, cu_q,
                            positions, slots, free_count_out, status, _handle(stream))
        if code is not None:
            return _check(code, "xs_paged_step") if code else None
    dev, i32 = _device(), _I32
    if block_table.dim() != 2 or block_table.dtype is not i32 or not block_table.is_contiguous():
        raise TypeError(f"block_table must be a contiguous {i32} tensor [n, width]")
    _on_device(block_table, "block_table", dev)
    n, width = block_table.shape
    rows, n_pages = positions.numel(), free_pages.numel()
    page_size = _c_int(page_size, XS_ERR_PAGE, "xs_paged_step")
    code = lib.xs_paged_step(_vec(cache_lens, "cache_lens", i32, n, dev), _vec(new_lens, "new_lens", i32, n, dev),
                             block_table.data_ptr(), _vec(free_pages, "free_pages", i32, n_pages, dev),
                             _vec(free_count, "free_count", i32, 1, dev), n, width, n_pages, page_size, rows,
                             _vec(kv_lens, "kv_lens", i32, n, dev), _vec(cu_q, "cu_q", i32, n + 1, dev),
                             _vec(positions, "positions", i32, rows, dev), _vec(slots, "slots", _I64, rows, dev),
                             _vec(free_count_out, "free_count_out", i32, 1, dev), _vec(status, "status", i32, n, dev),
                             _stream_of(stream, dev))
    if code:
        _check(code, "xs_paged_step")


def xs_attn_paged_workspace_bytes(n: int, H: int, Hkv: int, D: int) -> int:
    """Workspace bytes of the paged attention of up to ``n`` sequences."""
    b = _size(0)
    _check(lib.xs_attn_paged_workspace_bytes(n, H, Hkv, D, ctypes.byref(b)), "xs_attn_paged_workspace_bytes")
    return b.value


class PagedWorkspace:
    """Plan and scratch memory of the paged attention of ``n`` sequences with ``H`` query and
    ``Hkv`` KV heads of dimension ``D`` (torch-allocated, 256-byte aligned).  Filled by
    :func:`xs_attn_paged_plan`, used by every :func:`xs_attn_paged_fwd` of the step; calls that
    may overlap in time need one each."""

    def __init__(self, n: int, H: int, Hkv: int, D: int, device="cuda"):
        import torch
        self.n, self.H, self.Hkv, self.D = n, H, Hkv, D
        self.nbytes = xs_attn_paged_workspace_bytes(n, H, Hkv, D)
        self._buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        self.ptr = (self._buf.data_ptr() + 255) & ~255
        self._dims = (n, H, Hkv, D, self.ptr, self.nbytes)
        self.planned = None   # (max_q, causal, window) of the plan

    def __reduce__(self):   # a copy is a new workspace without a plan
        return PagedWorkspace, (self.n, self.H, self.Hkv, self.D, self._buf.device)


def xs_attn_paged_plan(cu_q, kv_lens, max_q: int, workspace: PagedWorkspace, causal: bool = True, window: int = 0,
                       stream=None) -> None:
    """Divide the attention of a step among the SMs: ``cu_q`` int32 [n + 1], ``kv_lens`` int32 [n]
    on the device; ``max_q`` an upper estimate of a sequence's new tokens; ``causal`` and
    ``window`` (0: none) as the attention is to use them."""
    w, causal = workspace, 1 if causal else 0
    code = None
    if _native is not None:
        code = _native.plan(cu_q, kv_lens, max_q, w._buf, w._dims, causal, window, _handle(stream))
    if code is None:
        dev = _device()
        _on_device(w._buf, "workspace", dev)
        for x in (max_q, window):
            _c_int(x, XS_ERR_SHAPE, "xs_attn_paged_plan")
        code = lib.xs_attn_paged_plan(_vec(cu_q, "cu_q", _I32, w.n + 1, dev), _vec(kv_lens, "kv_lens", _I32, w.n, dev),
                                      w.n, w.H, w.Hkv, w.D, max_q, causal, window, w.ptr, w.nbytes,
                                      _stream_of(stream, dev))
    if code:
        _check(code, "xs_attn_paged_plan")
    w.planned = (max_q, causal, window)


def xs_attn_paged_fwd(q, k_cache, v_cache, block_table, layout: int, outs, scale: float, workspace: PagedWorkspace,
                      lse=None, stream=None) -> None:
    """Attention of the new tokens ``q`` [T, H, D] over a paged cache ([n_pages, page_size, Hkv, D]
    each, any strides with D contiguous) as ``workspace`` plans it.  ``block_table`` int32 [n, width];
    ``layout`` XS_LAYOUT_A2A (P shards [T/P, H, D]), XS_LAYOUT_CONTIGUOUS (one [T, H, D] tensor) or
    XS_LAYOUT_HEADS (P head shards [T, H/P, D]); ``lse``: fp32 [T, H] or None."""
    if _native is not None:
        code = _native.attn(q, k_cache, v_cache, block_table, layout, outs, scale, workspace._buf, workspace._dims,
                            workspace.planned, lse, _handle(stream))
        if code is not None:
            return _check(code, "xs_attn_paged_fwd") if code else None
    w, dev, dt = workspace, _device(), q.dtype
    if w.planned is None:
        raise ValueError("xs_attn_paged_fwd: the workspace has no plan (call xs_attn_paged_plan first)")
    max_q, causal, window = w.planned
    D, n = w.D, w.n
    dtype = _dtype_of(q, "q")
    T, H, qs = _rows(q, "q", dt, D, dev)
    _on_device(w._buf, "workspace", dev)
    kc, vc = _cache(k_cache, "k_cache", dt, dev), _cache(v_cache, "v_cache", dt, dev)
    shape = k_cache.shape
    n_pages, page_size, Hkv, Dc = shape
    if H != w.H or Hkv != w.Hkv or Dc != D or v_cache.shape != shape:
        _same("xs_attn_paged_fwd", (H, Hkv, Dc, tuple(shape)), (w.H, w.Hkv, D, tuple(v_cache.shape)))
    if block_table.dim() != 2 or block_table.dtype is not _I32 or block_table.shape[0] != n:
        raise TypeError(f"block_table must be an int32 tensor [{n}, width]")
    _on_device(block_table, "block_table", dev)
    width = block_table.shape[1]
    ts, ts1 = block_table.stride()
    if ts1 != 1 and width > 1:
        raise TypeError("block_table: the entries of a row must be contiguous")
    P = len(outs)
    if layout == XS_LAYOUT_CONTIGUOUS or P == 0:
        want = (T, H, D)
    else:
        want = (T // P, H, D) if layout == XS_LAYOUT_A2A else (T, H // P, D)
    for o in outs:
        if o.shape != want or o.dtype is not dt or not o.is_contiguous():
            raise TypeError(f"out must be a contiguous {dt} tensor of shape {list(want)}")
        _on_device(o, "out", dev)
    z = 0
    if lse is not None:
        if lse.dtype is not _F32 or lse.shape != (T, H) or not lse.is_contiguous():
            raise TypeError("lse must be a contiguous float32 tensor [T, H]")
        _on_device(lse, "lse", dev)
        z = lse.data_ptr()
    pack = _ATTN_ARGS.get(P)
    if pack is None:
        raise XsError(XS_ERR_SHAPE if P < 1 else XS_ERR_TOO_MANY_RANKS, "xs_attn_paged_fwd")
    args = pack.pack(q.data_ptr(), block_table.data_ptr(), z, w.ptr, w.nbytes, *[o.data_ptr() for o in outs],
                     k_cache.data_ptr(), v_cache.data_ptr(), *kc, *vc, n_pages, page_size, Hkv, D, dtype, 0, qs, ts,
                     layout, P, T, H, n, width, max_q, causal, window, scale)
    code = lib.xs_attn_paged_fwd(args, _stream_of(stream, dev))
    if code:
        _check(code, "xs_attn_paged_fwd")


def attn_a2a(q, k, v, P: int, scale: float | None = None, stream=None, workspace=None):
    """Allocate the P output shards with torch and run the fused path; returns the list of shards.
    With a :class:`Workspace` the balanced schedule is used."""
    import torch
    B, S, H, D = q.shape
    if scale is None:
        scale = D ** -0.5
    outs = [torch.empty((B, S // P, H, D), dtype=torch.bfloat16, device=q.device) for _ in range(P)]
    if workspace is None:
        xs_attn_a2a_fwd(q, k, v, outs, scale, stream)
    else:
        xs_attn_fwd_balanced(q, k, v, XS_LAYOUT_A2A, outs, scale, workspace, stream)
    return outs
