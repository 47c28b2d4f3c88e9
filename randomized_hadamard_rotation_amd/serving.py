"""What uses 4-bit rows when a model answers: products with quantised weights and a paged 4-bit key-value cache.

The functions carry the names of the C entry points in include/serving/rhtq_serving.h and, like the others, only
marshal arguments: torch provides device memory and the current HIP stream, every step runs in the library's
kernels, and nothing is read back to the host.  They are exported by the package itself.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import (_DEFAULT_GROUP, _DEFAULT_SCALE, _FMT, _SCALE, RHTQ_IN_BF16, RHTQ_IN_F16, RHTQ_IN_F32, RHTQ_SCALE_F16,
               RHTQ_SCALE_F32, _check, _expect, _resolve_stream, _same_device, _scale_torch_dtype, _signs_tensor, lib, scale_shape)

EXPORTED_SERVING = ["rhtq_serving_version", "rhtq_matvec_workspace", "rhtq_matvec", "rhtq_cache_append", "rhtq_cache_read",
                    "rhtq_paged_attention_workspace", "rhtq_paged_attention", "rhtq_pages_workspace", "rhtq_pages_reserve",
                    "rhtq_pages_free", "rhtq_pages_trim", "rhtq_pages_fork", "rhtq_pages_copy", "rhtq_pages_compact"]

_IN = {torch.bfloat16: RHTQ_IN_BF16, torch.float16: RHTQ_IN_F16, torch.float32: RHTQ_IN_F32}
_SCALE_OF = {torch.float32: RHTQ_SCALE_F32, torch.float16: RHTQ_SCALE_F16}
_U8, _I8, _I32 = torch.uint8, torch.int8, torch.int32
_SCALE_TORCH = {"f32": torch.float32, "f16": torch.float16, "e4m3": torch.uint8, "e8m0": torch.uint8}


# A decode step makes a few of these calls per layer, each a few microseconds of kernels, so the host's share counts: every check below
# first takes a short form that only reads attributes, and goes to the spelled-out one, which raises, when that fails.

class _On:
    """The device and stream a call runs on.  Makes the tensors' device current; copies and fills of the wrapper go to its current
    stream, which a caller's other stream then waits for (follow), and that one keeps what the wrapper allocated (keep)."""
    __slots__ = ("raw", "stream", "before")

    def __init__(self, index):
        self.before = -1
        now = torch.cuda.current_device()
        if now != index:
            self.before = now
            torch.cuda.set_device(index)
        self.stream = None
        self.raw = _raw_stream(index)

    def follow(self, stream):
        st, other = _resolve_stream(stream)
        if other:
            self.raw, self.stream = st.cuda_stream, st

    def keep(self, *owned):
        if self.stream is not None:
            for t in owned:
                if t is not None:
                    t.record_stream(self.stream)

    def leave(self):
        if self.before >= 0:
            torch.cuda.set_device(self.before)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _one_device(index, named):
    """Every tensor on device `index`; raises as the other calls do."""
    if index >= 0:
        for t in named.values():
            if t is not None and t.get_device() != index:
                break
        else:
            return
    first = next(t for t in named.values() if t is not None)
    _same_device(first.device, **named)


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("layers", ctypes.c_int32), ("pages", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32)]


# the same struct as bytes, which a pointer argument takes as they are (a third of the time of a Structure)
_pack_cache = struct.Struct("@4P6i").pack
assert struct.calcsize("@4P6i") == ctypes.sizeof(_CacheStruct)


def _declare():
    vp, i32, i64, ci, fl = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    cache = vp
    args = {
        "rhtq_serving_version": (ci, []),
        "rhtq_matvec_workspace": (i64, [i64, i32, i64]),
        "rhtq_matvec": (ci, [vp, ci, i64, i32, i32, vp, ci, vp, vp, vp, i64, ci, i32, ci, vp, ci, vp, i64, vp]),
        "rhtq_cache_append": (ci, [cache, vp, vp, ci, i64, i64, i64, i64, i64, vp, i32, vp, vp, i32, vp, vp, vp]),
        "rhtq_cache_read": (ci, [cache, vp, vp, ci, i64, vp, i32, vp, vp, i32, vp, vp, vp]),
        "rhtq_paged_attention_workspace": (i64, [i32] * 8),
        "rhtq_paged_attention": (ci, [vp, ci, i32, i32, i64, i64, cache, vp, i32, vp, vp, vp, fl, i32, i32, vp, vp, i64, vp]),
        "rhtq_pages_workspace": (i64, [i32, i32, i32]),
        "rhtq_pages_reserve": (ci, [vp, i32, vp, i32, vp, i32, i32, vp, vp, vp, i64, vp]),
        "rhtq_pages_free": (ci, [vp, i32, vp, i32, vp, i32, vp, i32, vp]),
        "rhtq_pages_trim": (ci, [vp, i32, vp, i32, vp, i32, i32, i32, i32, vp]),
        "rhtq_pages_fork": (ci, [cache, vp, i32, vp, i32, vp, vp, vp, i32, vp, vp, i64, vp]),
        "rhtq_pages_copy": (ci, [cache, vp, vp, i32, vp]),
        "rhtq_pages_compact": (ci, [cache, vp, i32, i32, vp, vp, vp, i64, vp]),
    }
    for name, (res, types) in args.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, types


_declare()


class RhtqCache(NamedTuple):
    """One layer's paged cache, or with a leading axis every layer's: codes uint8 [.., pages, kv_heads, page, head_dim/2], scales
    float16 or float32 [.., pages, kv_heads, page].  Page calls take every layer at once; append, read and attention one."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor

    def layer(self, i: int) -> "RhtqCache":
        return RhtqCache(*(t[i] for t in self))


def rhtq_cache_new(pages: int, kv_heads: int, page: int, head_dim: int, scale_dtype: str = "f16", layers: int | None = None,
                   device="cuda") -> RhtqCache:
    """A cache of zero rows, with a leading axis if `layers` is given."""
    if scale_dtype not in ("f16", "f32"):
        raise ValueError("scale_dtype must be 'f16' or 'f32'")
    if head_dim not in (64, 128, 256):
        raise ValueError("head_dim must be 64, 128 or 256")
    if page < 16 or page > 256 or page & (page - 1):
        raise ValueError("page must be a power of two from 16 to 256")
    shape = (() if layers is None else (layers,)) + (pages, kv_heads, page)
    sdt = _scale_torch_dtype(scale_dtype)
    return RhtqCache(*(torch.zeros(s, dtype=d, device=device) for s, d in
                       2 * (((*shape, head_dim // 2), torch.uint8), (shape, sdt))))


def _cache_struct(cache, layered):
    """(C struct, pages, kv_heads, page, head_dim) of a cache whose four tensors agree; with `layered`, a leading axis is taken."""
    k, ks, v, vs = cache
    shape = k.shape
    dims = len(shape)
    sdt = ks.dtype
    if not (k.dtype is _U8 and v.dtype is _U8 and vs.dtype is sdt and sdt in _SCALE_OF and (dims == 4 or layered and dims == 5)
            and v.shape == shape and ks.shape == shape[:-1] and vs.shape == ks.shape and k.is_contiguous() and ks.is_contiguous()
            and v.is_contiguous() and vs.is_contiguous()):
        if dims != 4 and not (layered and dims == 5):
            raise ValueError("k_codes must be [pages][kv_heads][page][head_dim/2]" + (", with layers in front or not" if layered else ""))
        if sdt not in _SCALE_OF:
            raise ValueError(f"k_scales: dtype {sdt}, expected float16 or float32")
        for t, name, dtype, want in ((k, "k_codes", _U8, shape), (ks, "k_scales", sdt, shape[:-1]), (v, "v_codes", _U8, shape),
                                     (vs, "v_scales", sdt, shape[:-1])):
            _expect(t, name, dtype, want)
    pages, kv_heads, page, half = shape[-4:]
    return (_pack_cache(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(), shape[0] if dims == 5 else 1, pages, kv_heads, page,
                        2 * half, _SCALE_OF[sdt]), pages, kv_heads, page, 2 * half)


def _int32(t, name, shape):
    if not (t.dtype is _I32 and t.shape == shape and t.is_contiguous()):
        _expect(t, name, _I32, shape)


def _rows16(t):
    """t contiguous from an address of 16 bytes on: a copy where it is not (views may start anywhere)."""
    if t.is_contiguous() and not t.data_ptr() & 15:
        return t
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def _signs(signs, n, x):
    """Device int8 [n] (marshalling only)."""
    if signs is None or (type(signs) is torch.Tensor and signs.dtype is _I8 and signs.dim() == 1 and signs.shape[0] == n
                         and signs.is_contiguous() and signs.get_device() == x.get_device() and not signs.data_ptr() & 15):
        return signs
    return _rows16(_signs_tensor(signs, n, x.device))


def _bounded(v):
    """A count as int32, which ctypes would cut to its low 32 bits: beyond 2^31 - 1 positions there are none."""
    return max(-1, min(v, 0x7FFFFFFF))


def _p(t):
    return None if t is None else t.data_ptr()


def rhtq_serving_version() -> int:
    return lib.rhtq_serving_version()


def rhtq_matvec(packed, scales, x, signs=None, fmt: str = "int4", group: int = 0, scale_dtype: str | None = None,
                tensor_scale=None, rotated: bool = False, block=None, out=None, out_dtype=None, stream=None):
    """y [tokens][rows] = x [tokens][n] times the transpose of the matrix that rhtq_inverse(packed, scales, n, signs, ...) gives:
    rows quantised by rhtq_forward are weights, used as they lie.  x is bfloat16, float16 or float32; y has its type unless `out`
    or out_dtype says otherwise.  rotated = True: x is rhtq_rotate(x, signs) already (one rotation serves several weights).
    fmt, group, scale_dtype, tensor_scale and block as in rhtq_forward."""
    if fmt not in _FMT:
        raise ValueError(f"unknown fmt {fmt!r}")
    if x.dim() != 2 or packed.dim() != 2:
        raise ValueError("x must be 2-D [tokens][n] and packed 2-D [rows][n/2]")
    in_type = _IN.get(x.dtype)
    if in_type is None:
        raise ValueError("x must be bfloat16, float16 or float32")
    tokens, n = x.shape
    rows = packed.shape[0]
    if scale_dtype is None:
        scale_dtype = _DEFAULT_SCALE[fmt]
    if group == 0:
        group = _DEFAULT_GROUP.get(fmt, 0)
    if packed.dtype is not _U8 or packed.shape[1] * 2 != n:
        raise ValueError(f"packed: {packed.dtype} {tuple(packed.shape)}, expected uint8 {(rows, n // 2)}")
    sshape = scale_shape(rows, n, fmt, group)
    sdt = _SCALE_TORCH.get(scale_dtype) or _scale_torch_dtype(scale_dtype)
    if scales.dtype is not sdt or scales.shape != sshape:
        raise ValueError(f"scales: {scales.dtype} {tuple(scales.shape)}, expected {sdt} {sshape}")
    if fmt == "nvfp4":
        if tensor_scale is None:
            raise ValueError("NVFP4 needs its tensor_scale")
        if tensor_scale.dtype != torch.float32 or tensor_scale.numel() != 1:
            raise ValueError("tensor_scale must be one float32")
    else:
        tensor_scale = None
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    out_type = _IN.get(out_dtype)
    if out_type is None:
        raise ValueError("out_dtype must be bfloat16, float16 or float32")
    if out is not None:
        _expect(out, "out", out_dtype, (tokens, rows))
    index = x.get_device()
    _one_device(index, {"x": x, "packed": packed, "scales": scales, "tensor_scale": tensor_scale, "out": out})
    on = _On(index)
    try:
        xc, pc, sc = x, packed, scales
        xp, pp, sp = x.data_ptr(), packed.data_ptr(), scales.data_ptr()
        if (xp | pp) & 15 or sp & 1 or not (x.is_contiguous() and packed.is_contiguous() and scales.is_contiguous()):
            xc, pc = _rows16(x), _rows16(packed)
            sc = _rows16(scales) if sp & 1 else scales.contiguous()          # E4M3 bytes are loaded in pairs, others one by one
            xp, pp, sp = xc.data_ptr(), pc.data_ptr(), sc.data_ptr()
        s = None if rotated else _signs(signs, n, x)
        own = out is None
        if own:
            out = x.new_empty((tokens, rows), dtype=out_dtype)
        need = lib.rhtq_matvec_workspace(tokens, n, rows)
        work = x.new_empty(need, dtype=_U8)
        if stream is not None:
            on.follow(stream)
        _check(lib.rhtq_matvec(xp, in_type, tokens, n, n if block is None else block, _p(s), rotated,
                               pp, sp, _p(tensor_scale), rows, _FMT[fmt], group, _SCALE[scale_dtype],
                               out.data_ptr(), out_type, work.data_ptr(), need, on.raw), "rhtq_matvec")
        on.keep(xc if xc is not x else None, pc if pc is not packed else None, sc if sc is not scales else None, s, work,
                out if own else None)
    finally:
        on.leave()
    return out


def _rows_of(cache, table, lengths, starts, tokens):
    """(struct, seqs, width) of an append or read call after its checks; the device is checked last, by the caller."""
    c = _cache_struct(cache, False)
    if table.dim() != 2:
        raise ValueError("table must be 2-D [seqs][width]")
    shape = table.shape
    seqs, width = shape
    _int32(table, "table", shape)
    _int32(lengths, "lengths", (seqs,))
    if starts is not None:
        _int32(starts, "starts", (seqs + 1,))
    elif tokens != seqs:
        raise ValueError(f"without starts there is one row for each of {seqs} sequences: got {tokens}")
    return c, seqs, width


def _row_strides(x):
    """x with rows that start on 16 bytes (a copy where they do not), and its strides in elements; 0 along an axis of one entry, whose stride
    may be anything."""
    per16 = 16 // x.element_size()
    tokens, heads, dim = x.shape
    of_token, of_head, of_value = x.stride()
    if tokens < 2:
        of_token = 0
    if heads < 2:
        of_head = 0
    if of_value != 1 or of_token % per16 or of_head % per16 or x.data_ptr() & 15:
        return x.clone(memory_format=torch.contiguous_format), heads * dim, dim
    return x, of_token, of_head


def rhtq_cache_append(cache: RhtqCache, k, v, table, lengths, starts=None, k_signs=None, v_signs=None, stream=None):
    """Rotate, quantise (INT4, one scale a row) and store new keys and values [tokens][kv_heads][head_dim] (bfloat16, float16 or
    float32; any strides) in the pages that `table` int32 [seqs][width] names.  Rows starts[s] .. starts[s+1]-1 are the last positions
    of sequence s, up to lengths[s] - 1; starts None: one row for each sequence.  Rows of no sequence, or on no page, are passed over."""
    if k.dim() != 3 or v.dim() != 3 or k.shape != v.shape:
        raise ValueError("k and v must be 3-D [tokens][kv_heads][head_dim], alike")
    in_type = _IN.get(k.dtype)
    if in_type is None or v.dtype != k.dtype:
        raise ValueError("k and v must both be bfloat16, float16 or float32")
    tokens, kv_heads, dim = k.shape
    c, seqs, width = _rows_of(cache, table, lengths, starts, tokens)
    if c[2] != kv_heads or c[4] != dim:
        raise ValueError(f"k: {tuple(k.shape)}, expected {(tokens, c[2], c[4])}")
    index = k.get_device()
    _one_device(index, {"k": k, "v": v, "k_codes": cache[0], "k_scales": cache[1], "v_codes": cache[2], "v_scales": cache[3],
                        "table": table, "lengths": lengths, "starts": starts})
    on = _On(index)
    try:
        ks, vs = _signs(k_signs, dim, k), _signs(v_signs, dim, k)
        (kc, k_token, k_head), (vc, v_token, v_head) = _row_strides(k), _row_strides(v)
        if stream is not None:
            on.follow(stream)
        _check(lib.rhtq_cache_append(c[0], kc.data_ptr(), vc.data_ptr(), in_type, tokens, k_token, k_head,
                                     v_token, v_head, table.data_ptr(), width, lengths.data_ptr(), _p(starts), seqs,
                                     _p(ks), _p(vs), on.raw), "rhtq_cache_append")
        on.keep(ks, vs, kc if kc is not k else None, vc if vc is not v else None)
    finally:
        on.leave()


def rhtq_cache_read(cache: RhtqCache, table, lengths, starts, tokens: int, k_signs=None, v_signs=None, dtype=torch.bfloat16,
                    k_out=None, v_out=None, stream=None):
    """Read rows back, dequantised and with the rotation undone: (k, v) [tokens][kv_heads][head_dim] of `dtype`.  Rows belong to
    sequences as in rhtq_cache_append: starts from the running sum of lengths reads whole sequences, shorter lengths read earlier rows.
    Rows of no sequence, or on no page, are zero."""
    if dtype not in _IN:
        raise ValueError("dtype must be bfloat16, float16 or float32")
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    c, seqs, width = _rows_of(cache, table, lengths, starts, tokens)
    dim = c[4]
    shape = (tokens, c[2], dim)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None:
            _expect(t, name, dtype, shape)
    first = cache[0]
    index = first.get_device()
    _one_device(index, {"k_codes": first, "k_scales": cache[1], "v_codes": cache[2], "v_scales": cache[3], "table": table,
                        "lengths": lengths, "starts": starts, "k_out": k_out, "v_out": v_out})
    on = _On(index)
    try:
        ks, vs = _signs(k_signs, dim, first), _signs(v_signs, dim, first)
        own_k, own_v = k_out is None, v_out is None
        if own_k:
            k_out = first.new_empty(shape, dtype=dtype)
        if own_v:
            v_out = first.new_empty(shape, dtype=dtype)
        if stream is not None:
            on.follow(stream)
        _check(lib.rhtq_cache_read(c[0], k_out.data_ptr(), v_out.data_ptr(), _IN[dtype], tokens, table.data_ptr(), width,
                                   lengths.data_ptr(), _p(starts), seqs, _p(ks), _p(vs), on.raw), "rhtq_cache_read")
        on.keep(ks, vs, k_out if own_k else None, v_out if own_v else None)
    finally:
        on.leave()
    return k_out, v_out


def rhtq_paged_attention(q, cache: RhtqCache, table, lengths, k_signs=None, v_signs=None, scale: float | None = None,
                         window: int = 0, sinks: int = 0, out=None, stream=None):
    """Attention of one new token per sequence, q [seqs][q_heads][head_dim] (bfloat16 or float16, any strides; q_heads a multiple of the
    cache's kv_heads), over its cached positions [0, lengths[s]); the token's own row has been appended.  scale: 1/sqrt(head_dim)
    unless given.  window > 0: only the last `window` positions and the first `sinks` are visible.  A sequence with no visible
    position gets zeros.  Returns [seqs][q_heads][head_dim] in q's type."""
    if q.dim() != 3:
        raise ValueError("q must be 3-D [seqs][q_heads][head_dim]")
    in_type = _IN.get(q.dtype, RHTQ_IN_F32)
    if in_type == RHTQ_IN_F32:
        raise ValueError("q must be bfloat16 or float16")
    c, seqs, width = _rows_of(cache, table, lengths, None, q.shape[0])
    q_heads, dim = q.shape[1:]
    kv_heads = c[2]
    if dim != c[4] or q_heads < 1 or q_heads % max(kv_heads, 1):
        raise ValueError(f"q: {tuple(q.shape)} does not fit {kv_heads} key-value heads of {c[4]}")
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    window, sinks = _bounded(window), _bounded(sinks)
    if out is not None:
        _expect(out, "out", q.dtype, q.shape)
    index = q.get_device()
    _one_device(index, {"q": q, "k_codes": cache[0], "k_scales": cache[1], "v_codes": cache[2], "v_scales": cache[3], "table": table,
                        "lengths": lengths, "out": out})
    on = _On(index)
    try:
        ks, vs = _signs(k_signs, dim, q), _signs(v_signs, dim, q)
        qc, of_seq, of_head = _row_strides(q)
        own = out is None
        if own:
            out = q.new_empty(q.shape)
        need = lib.rhtq_paged_attention_workspace(seqs, q_heads, kv_heads, dim, width, c[3], window, sinks)
        work = q.new_empty(need, dtype=_U8) if need else None
        if stream is not None:
            on.follow(stream)
        _check(lib.rhtq_paged_attention(qc.data_ptr(), in_type, seqs, q_heads, of_seq, of_head, c[0],
                                        table.data_ptr(), width, lengths.data_ptr(), _p(ks), _p(vs),
                                        1.0 / math.sqrt(dim) if scale is None else scale, window, sinks, out.data_ptr(), _p(work),
                                        need, on.raw), "rhtq_paged_attention")
        on.keep(ks, vs, work, qc if qc is not q else None, out if own else None)
    finally:
        on.leave()
    return out


def _paging(table, lengths, refs):
    if table.dim() != 2 or refs.dim() != 1:
        raise ValueError("table must be 2-D [seqs][width] and refs 1-D [pages]")
    shape = table.shape
    _int32(table, "table", shape)
    if lengths is not None:
        _int32(lengths, "lengths", shape[:1])
    _int32(refs, "refs", refs.shape)
    return shape


def _paged_cache(cache, refs):
    c = _cache_struct(cache, True)
    if c[1] != refs.shape[0]:
        raise ValueError(f"refs has {refs.shape[0]} entries, the cache {c[1]} pages")
    return c


def _index_list(t, name, shape=None):
    if t.dim() != 1:
        raise ValueError(f"{name} must be 1-D")
    _int32(t, name, t.shape if shape is None else shape)
    return t.shape[0]


def _page_call(name, named, stream, call, pages=None, seqs=0, count=0, word=False):
    """call(raw stream, word, workspace, its size) on the tensors' device: with `pages`, a workspace of the page calls; with `word`, the
    device int32 [1] that comes back."""
    first = next(iter(named.values()))
    index = first.get_device()
    _one_device(index, named)
    on = _On(index)
    try:
        told = first.new_empty(1, dtype=_I32) if word else None
        need = 0 if pages is None else lib.rhtq_pages_workspace(pages, seqs, count)
        work = first.new_empty(need, dtype=_U8) if need else None
        if stream is not None:
            on.follow(stream)
        _check(call(on.raw, _p(told), _p(work), need), name)
        on.keep(told, work)
    finally:
        on.leave()
    return told


def _tensors(cache):
    return {"k_codes": cache[0], "k_scales": cache[1], "v_codes": cache[2], "v_scales": cache[3]}


def rhtq_pages_reserve(table, lengths, refs, add, page: int, stream=None):
    """Room for add[s] more positions of every sequence: lengths grow, and where `table` int32 [seqs][width] has no page yet the lowest
    free ones (refs int32 [pages] == 0) are taken.  All or nothing; returns a device int32 [1]: 0 done, otherwise the number of
    pages missing, or -1 for a negative amount or a new position on a page that another sequence shares (after lengths were lowered: fork
    the sequence at its new length and go on with the fork)."""
    seqs, width = _paging(table, lengths, refs)
    _int32(add, "add", lengths.shape)
    pages = refs.shape[0]
    return _page_call("rhtq_pages_reserve", {"table": table, "lengths": lengths, "refs": refs, "add": add}, stream,
                      lambda raw, word, work, size: lib.rhtq_pages_reserve(table.data_ptr(), width, lengths.data_ptr(), seqs, refs.data_ptr(),
                                                                           pages, _bounded(page), add.data_ptr(), word, work, size, raw),
                      pages, seqs, 0, True)


def rhtq_pages_free(table, lengths, refs, seqs, stream=None):
    """Give up every page of the listed sequences (int32 [count]) and set their lengths to 0."""
    all_seqs, width = _paging(table, lengths, refs)
    count = _index_list(seqs, "seqs")
    _page_call("rhtq_pages_free", {"table": table, "lengths": lengths, "refs": refs, "seqs": seqs}, stream,
               lambda raw, word, work, size: lib.rhtq_pages_free(table.data_ptr(), width, lengths.data_ptr(), all_seqs, refs.data_ptr(),
                                                                 refs.shape[0], seqs.data_ptr(), count, raw))


def rhtq_pages_trim(table, lengths, refs, page: int, window: int, sinks: int = 0, stream=None):
    """Give up the pages that attention with this window and these first positions can never see again."""
    seqs, width = _paging(table, lengths, refs)
    _page_call("rhtq_pages_trim", {"table": table, "lengths": lengths, "refs": refs}, stream,
               lambda raw, word, work, size: lib.rhtq_pages_trim(table.data_ptr(), width, lengths.data_ptr(), seqs, refs.data_ptr(),
                                                                 refs.shape[0], _bounded(page), _bounded(window), _bounded(sinks), raw))


def rhtq_pages_fork(cache: RhtqCache, table, lengths, refs, src, dst, stream=None):
    """Sequences dst (int32 [count], empty ones) become copies of src: full pages are shared, a partly filled last page is copied.
    All or nothing; returns a device int32 [1]: 0 done, otherwise the number of pages missing, or -1 for an invalid index."""
    c = _paged_cache(cache, refs)
    seqs, width = _paging(table, lengths, refs)
    count = _index_list(src, "src")
    _index_list(dst, "dst", src.shape)
    return _page_call("rhtq_pages_fork", {"table": table, "lengths": lengths, "refs": refs, "src": src, "dst": dst, **_tensors(cache)}, stream,
                      lambda raw, word, work, size: lib.rhtq_pages_fork(c[0], table.data_ptr(), width, lengths.data_ptr(), seqs,
                                                                        refs.data_ptr(), src.data_ptr(), dst.data_ptr(), count, word, work,
                                                                        size, raw),
                      refs.shape[0], seqs, count, True)


def rhtq_pages_copy(cache: RhtqCache, src, dst, stream=None):
    """Copy whole pages src[i] -> dst[i] (int32 [count]) in every layer; a page may be written once and not read by the same call."""
    c = _cache_struct(cache, True)
    count = _index_list(src, "src")
    _index_list(dst, "dst", src.shape)
    _page_call("rhtq_pages_copy", {**_tensors(cache), "src": src, "dst": dst}, stream,
               lambda raw, word, work, size: lib.rhtq_pages_copy(c[0], src.data_ptr(), dst.data_ptr(), count, raw))


def rhtq_pages_compact(cache: RhtqCache, table, refs, stream=None):
    """Move live pages into lower free ones until they fill [0, live); table and refs follow.  Returns live, a device int32 [1]."""
    c = _paged_cache(cache, refs)
    seqs, width = _paging(table, None, refs)
    return _page_call("rhtq_pages_compact", {"table": table, "refs": refs, **_tensors(cache)}, stream,
                      lambda raw, word, work, size: lib.rhtq_pages_compact(c[0], table.data_ptr(), width, seqs, refs.data_ptr(), word,
                                                                           work, size, raw),
                      refs.shape[0], seqs, 0, True)
