"""Serving with an INT4 KV cache: binding of the library's kv calls.

    cache = KVCache.empty(pages, page_size, kv_heads, head_dim, "cuda")
    step = kv_slots(ctx_len, new_len, block_table, free_pages, free_state, page_size, tokens)
    q = kv_append(cache, k, v, step.slot_map, q, q_weight, k_weight, cos_sin, step.positions)
    o = kv_attention(q, cache, block_table, step.kv_len, step.cu_new, max_q_len=largest)

where `largest` is the largest number of new tokens of a request (1 in a decode step), which chooses the kernel.

Rows that a call skips (padding of a batch: no position, no slot, no request) are left as they were.  In an output
that the binding allocates that is whatever the memory held before, so where such rows go on into a call that mixes
tokens (the Rotated Runtime Smooth quantizer's maxima), pass an output that was filled (`q_out`, `out`).

Marshalling and argument checks only, like the rest of the package; every
call has a prepare_ form that checks once and launches again on each call.
"""
from __future__ import annotations

import collections
import ctypes
import functools

import numpy as np

import torch

from . import RW4_BF16, RW4_F32, RW4_OK, Call, RW4Error, _on_gpu, _out, _stream, lib

__all__ = ["KVCache", "KVSlots", "kv_slots", "prepare_kv_slots", "rope_table", "qk_norm_rope", "prepare_qk_norm_rope",
           "kv_append", "prepare_kv_append", "kv_attention", "prepare_kv_attention", "kv_attention_workspace_bytes"]

_p, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", _p), ("k_scales", _p), ("v_codes", _p), ("v_scales", _p), ("pages", _i64),
                ("page_size", _i32), ("heads", _i32), ("head_dim", _i32), ("code_page", _i64), ("code_head", _i64),
                ("code_slot", _i64), ("scale_page", _i64), ("scale_head", _i64), ("scale_slot", _i64)]


lib.rw4_kv_slots.argtypes = [_p, _p, _i64, _i32, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _p, _p, _i64, _p]
lib.rw4_qk_norm_rope.argtypes = [_p, _i64, _i64, _p, _i64, _i64, ctypes.c_int, _i64, _i32, _i32, _i32, _p, _p, _f32,
                                 _p, _i64, _i32, _i32, _p, _i32, _p, _i64, _i64, _p, _i64, _i64, ctypes.c_int, _p]
lib.rw4_kv_append.argtypes = [_p, _p, _i64, _i64, _p, _i64, _i64, _p, _p, _i64, _i64, _i32, ctypes.c_int, _i64, _p, _p,
                              _f32, _p, _i64, _i32, _i32, _p, _i32, _p, _i64, _i64, ctypes.c_int, _p]
lib.rw4_kv_attention_workspace_bytes.argtypes = [_i64, _i64, _i32, _i32, _i32]
lib.rw4_kv_attention_workspace_bytes.restype = _i64
lib.rw4_kv_attention.argtypes = [_p, _p, ctypes.c_int, _i64, _i64, _i64, _i32, _p, _i64, _p, _p, _i64, _i64, _f32, _i32,
                                 _i64, _i32, _p, ctypes.c_int, _i64, _i64, _p, _p, _i64, _p]
for _name in ("rw4_kv_slots", "rw4_qk_norm_rope", "rw4_kv_append", "rw4_kv_attention"):
    getattr(lib, _name).restype = ctypes.c_int


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_DTYPES = {torch.bfloat16: RW4_BF16, torch.float32: RW4_F32}


def _launch(fn, args, dev, what):
    """The library call on the current stream of GPU `dev`, with that GPU current."""
    if _current_device() != dev:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(dev))
    else:
        status = fn(*args, _stream(dev))
    if status != RW4_OK:
        raise RW4Error(status, what)


class KVCall(Call):
    """A prepared call that also makes its tensors' GPU current while it launches."""

    __slots__ = ()

    def __call__(self):
        _launch(self._fn, self._args, self._dev, self._what)
        return self.result


def _code(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return code


def _vec(name, t, dtype, n, dev):
    """A contiguous one-dimensional tensor of n entries (None: any number); its pointer."""
    if t.get_device() != dev or not t.is_cuda:
        _on_gpu(name, t, dev)
    if t.dtype is not dtype or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + ("" if n is None else f" of {n} entries"))
    return t.data_ptr()


def _table(t, B, dev):
    """A block table: its pointer and width."""
    if t.get_device() != dev or not t.is_cuda:
        _on_gpu("block_table", t, dev)
    if t.dtype is not torch.int32 or t.dim() != 2 or t.shape[0] != B or not t.is_contiguous():
        raise ValueError(f"block_table must be a contiguous int32 tensor of {B} rows")
    return t.data_ptr(), t.shape[1]


def _rows(name, t, dev, shape=None):
    """A [tokens, heads, D] tensor with unit stride in a head: (pointer, token stride, head stride)."""
    if t.get_device() != dev or not t.is_cuda:
        _on_gpu(name, t, dev)
    size = t.shape
    if len(size) != 3 or (shape is not None and size != shape):
        raise ValueError(f"{name} must be " + ("[tokens, heads, head_dim]" if shape is None else str(list(shape))))
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must have unit stride along the head's channels")
    return t.data_ptr(), (st if size[0] > 1 else 0), (sh if size[1] > 1 else 0)


class KVCache:
    """A paged INT4 KV cache over caller-owned tensors.

    k, v: uint8 [pages, kv_heads, page_size, head_dim / 2], one stored row per
    token; k_scale, v_scale: fp32 [pages, kv_heads, page_size].  Any strides
    with unit stride in a row (equal for k and v), so the rows that
    quantize_act writes are a cache too (from_rows).
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "page_size", "kv_heads", "head_dim", "device", "_dev",
                 "_struct", "_ptr")

    def __init__(self, k, v, k_scale, v_scale):
        self._dev = _on_gpu("k", k)
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            _on_gpu(name, t, self._dev)
        if k.dim() != 4 or k.dtype is not torch.uint8 or v.dtype is not torch.uint8 or v.shape != k.shape \
                or k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32 \
                or k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3]:
            raise ValueError("k and v must be uint8 [pages, kv_heads, page_size, head_dim / 2] and their scales "
                             "float32 [pages, kv_heads, page_size]")
        # the stride of a dimension of one entry is not used
        cs, cv, ss, sv = ([x if n > 1 else 0 for x, n in zip(t.stride(), k.shape[:3])] for t in (k, v, k_scale, v_scale))
        if cv != cs or sv != ss or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must have the same strides, with unit stride in a row (their scales likewise)")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.kv_heads, self.page_size, half = k.shape
        self.head_dim, self.device = 2 * half, k.device
        self._struct = _CacheStruct(k.data_ptr(), k_scale.data_ptr(), v.data_ptr(), v_scale.data_ptr(), self.pages,
                                    self.page_size, self.kv_heads, self.head_dim, *cs, *ss)
        self._ptr = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda") -> "KVCache":
        """A cache of zeros, pages contiguous by head."""
        k, v = (torch.zeros((pages, kv_heads, page_size, head_dim // 2), dtype=torch.uint8, device=device)
                for _ in range(2))
        ks, vs = (torch.zeros((pages, kv_heads, page_size), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    @classmethod
    def from_rows(cls, qk, sk, qv, sv, page_size: int, kv_heads: int) -> "KVCache":
        """The rows [pages * page_size, kv_heads * head_dim / 2] and scales [pages * page_size, kv_heads] that
        quantize_act writes (group = Hadamard block = head_dim), seen as pages."""
        rows, width = qk.shape
        if rows % page_size or width % kv_heads:
            raise ValueError("rows must be a multiple of page_size and hold kv_heads heads")
        codes = [t.view(rows // page_size, page_size, kv_heads, width // kv_heads).transpose(1, 2) for t in (qk, qv)]
        scales = [t.view(rows // page_size, page_size, kv_heads).transpose(1, 2) for t in (sk, sv)]
        return cls(codes[0], codes[1], scales[0], scales[1])


KVSlots = collections.namedtuple("KVSlots", "kv_len cu_new served slot_map positions free_state")


def kv_slots(ctx_len, new_len, block_table, free_pages, free_state, page_size: int, tokens: int, **out) -> KVSlots:
    """Pages and slots for one step's new tokens (new_len < 0: finished, its pages return to the free list).

    ctx_len, new_len int32 [B]; block_table int32 [B, width] and free_pages int32 [capacity] are updated in place;
    free_state int32 [2] (head, count of the ring free_pages).  Returns KVSlots(kv_len, cu_new, served, slot_map,
    positions, free_state); `out` may hold any of these by name (kv_len may be ctx_len, free_state_out free_state).
    """
    fn, args, dev, what, _, result = _slots(ctx_len, new_len, block_table, free_pages, free_state, page_size, tokens,
                                            **out)
    _launch(fn, args, dev, what)
    return result


def prepare_kv_slots(ctx_len, new_len, block_table, free_pages, free_state, page_size: int, tokens: int, **out) -> Call:
    """kv_slots checked and marshalled once; calling the result runs it."""
    return KVCall(*_slots(ctx_len, new_len, block_table, free_pages, free_state, page_size, tokens, **out))


def _slots(ctx_len, new_len, block_table, free_pages, free_state, page_size, tokens, *, kv_len=None, cu_new=None,
           served=None, slot_map=None, positions=None, free_state_out=None):
    i32, dev, device = torch.int32, _on_gpu("ctx_len", ctx_len), ctx_len.device
    if ctx_len.dim() != 1:
        raise ValueError("ctx_len must be one-dimensional")
    B, tokens = ctx_len.shape[0], int(tokens)
    table, width = _table(block_table, B, dev)
    if kv_len is None and cu_new is None and served is None and positions is None and free_state_out is None:
        # one allocation for the small outputs
        kv_len, cu_new, served, free_state_out, positions = torch.empty(
            (3 * B + 3 + tokens,), dtype=i32, device=device).split_with_sizes((B, B + 1, B, 2, tokens))
    else:
        kv_len, cu_new, served, free_state_out, positions = (
            torch.empty((n,), dtype=i32, device=device) if t is None else t
            for t, n in ((kv_len, B), (cu_new, B + 1), (served, B), (free_state_out, 2), (positions, tokens)))
    if slot_map is None:
        slot_map = torch.empty((tokens,), dtype=torch.int64, device=device)
    args = (_vec("ctx_len", ctx_len, i32, None, dev), _vec("new_len", new_len, i32, B, dev), B, int(page_size), table,
            width, _vec("free_pages", free_pages, i32, None, dev), free_pages.shape[0],
            _vec("free_state", free_state, i32, 2, dev), _vec("free_state_out", free_state_out, i32, 2, dev),
            _vec("kv_len", kv_len, i32, B, dev), _vec("cu_new", cu_new, i32, B + 1, dev),
            _vec("served", served, i32, B, dev), _vec("slot_map", slot_map, torch.int64, tokens, dev),
            _vec("positions", positions, i32, tokens, dev), tokens)
    return (lib.rw4_kv_slots, args, dev, "rw4_kv_slots", (ctx_len, new_len, block_table, free_pages, free_state),
            KVSlots(kv_len, cu_new, served, slot_map, positions, free_state_out))


def rope_table(max_pos: int, rot: int, base: float = 10000.0, device="cuda"):
    """cos_sin fp32 [max_pos, rot] for qk_norm_rope and kv_append: rot / 2 cosines, then rot / 2 sines of the angles
    p * base^(-2 i / rot), evaluated in float64."""
    angle = np.arange(max_pos, dtype=np.float64)[:, None] * float(base) ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(device)


def _weight(name, w, D, dev):
    return None if w is None else _vec(name, w, torch.float32, D, dev)


def _rope_args(cos_sin, positions, T, dev):
    """(cos_sin pointer, max_pos, rot, positions pointer)."""
    if cos_sin is None:
        return None, 0, 0, None
    _on_gpu("cos_sin", cos_sin, dev)
    if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 tensor [max_pos, rot]")
    if positions is None:
        raise ValueError("cos_sin needs positions")
    return cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], _vec("positions", positions, torch.int32, T, dev)


def qk_norm_rope(q, k=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, *, eps: float = 1e-6,
                 interleaved: bool = False, rotate: bool = False, q_out=None, k_out=None, out_dtype=None):
    """Per-head RMS norm (weights fp32 [D], None: no norm) and rotary positions (cos_sin [max_pos, rot], None: none)
    of queries [T, heads, D] and keys [T, kv_heads, D] in one pass, then the head's Hadamard when `rotate`.

    Returns (q_out, k_out); with q_out = q and k_out = k in place.  k may be None.  Rows of tokens without a position are
    not written."""
    fn, args, dev, what, _, result = _norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, rotate,
                                                q_out, k_out, out_dtype)
    _launch(fn, args, dev, what)
    return result


def prepare_qk_norm_rope(q, k=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, *, eps: float = 1e-6,
                         interleaved: bool = False, rotate: bool = False, q_out=None, k_out=None,
                         out_dtype=None) -> Call:
    """qk_norm_rope checked and marshalled once; calling the result runs it."""
    return KVCall(*_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, rotate, q_out, k_out,
                              out_dtype))


def _norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, rotate, q_out, k_out, out_dtype):
    dev = _on_gpu("q", q)
    qp, qt, qh = _rows("q", q, dev)
    T, heads, D = q.shape
    if q_out is None:
        q_out = torch.empty((T, heads, D), dtype=q.dtype if out_dtype is None else out_dtype, device=q.device)
    elif out_dtype is not None and q_out.dtype is not out_dtype:
        raise TypeError(f"q_out must be {out_dtype}")
    qop, qot, qoh = _rows("q_out", q_out, dev, (T, heads, D))
    kv_heads, kp, kt, kh, kop, kot, koh = 0, None, 0, 0, None, 0, 0
    if k is not None:
        kv_heads = k.shape[1] if k.dim() == 3 else 0
        kp, kt, kh = _rows("k", k, dev, (T, kv_heads, D))
        if k_out is None:
            k_out = torch.empty((T, kv_heads, D), dtype=q_out.dtype, device=q.device)
        kop, kot, koh = _rows("k_out", k_out, dev, (T, kv_heads, D))
        if k.dtype is not q.dtype or k_out.dtype is not q_out.dtype:
            raise TypeError("q and k (and their outputs) must have the same dtype")
    elif k_out is not None:
        raise ValueError("k_out needs k")
    cs, max_pos, rot, pos = _rope_args(cos_sin, positions, T, dev)
    args = (qp, qt, qh, kp, kt, kh, _code(q.dtype), T, heads, kv_heads, D, _weight("q_weight", q_weight, D, dev),
            _weight("k_weight", k_weight, D, dev), eps, cs, max_pos, rot, int(interleaved), pos, int(rotate), qop, qot,
            qoh, kop, kot, koh, _code(q_out.dtype))
    return (lib.rw4_qk_norm_rope, args, dev, "rw4_qk_norm_rope", (q, k, q_weight, k_weight, cos_sin, positions),
            (q_out, k_out))


def kv_append(cache: KVCache, k, v, slot_map, q=None, q_weight=None, k_weight=None, cos_sin=None, positions=None, *,
              eps: float = 1e-6, interleaved: bool = False, rotate: bool = True, q_out=None, out_dtype=None):
    """New tokens into the cache: keys [T, kv_heads, D] normed and given their positions (as qk_norm_rope), keys and
    values rotated by the head's Hadamard (`rotate`) and stored as INT4 in rows slot_map (int64 [T]).  Queries, if
    given, go through qk_norm_rope in the same launch; returns q_out (None without q; rows of tokens without a position
    are not written)."""
    fn, args, dev, what, _, result = _append(cache, k, v, slot_map, q, q_weight, k_weight, cos_sin, positions, eps,
                                             interleaved, rotate, q_out, out_dtype)
    _launch(fn, args, dev, what)
    return result


def prepare_kv_append(cache: KVCache, k, v, slot_map, q=None, q_weight=None, k_weight=None, cos_sin=None,
                      positions=None, *, eps: float = 1e-6, interleaved: bool = False, rotate: bool = True,
                      q_out=None, out_dtype=None) -> Call:
    """kv_append checked and marshalled once; calling the result runs it."""
    return KVCall(*_append(cache, k, v, slot_map, q, q_weight, k_weight, cos_sin, positions, eps, interleaved, rotate,
                           q_out, out_dtype))


def _append(cache, k, v, slot_map, q, q_weight, k_weight, cos_sin, positions, eps, interleaved, rotate, q_out,
            out_dtype):
    dev, D, kv_heads = cache._dev, cache.head_dim, cache.kv_heads
    T = k.shape[0]
    kp, kt, kh = _rows("k", k, dev, (T, kv_heads, D))
    vp, vt, vh = _rows("v", v, dev, (T, kv_heads, D))
    dtype = k.dtype
    if v.dtype is not dtype:
        raise TypeError("k and v must have the same dtype")
    qp, qt, qh, qop, qot, qoh, heads, out_code = None, 0, 0, None, 0, 0, 0, RW4_F32
    if q is not None:
        heads = q.shape[1] if q.dim() == 3 else 0
        qp, qt, qh = _rows("q", q, dev, (T, heads, D))
        if q.dtype is not dtype:
            raise TypeError("q and k must have the same dtype")
        if q_out is None:
            q_out = torch.empty((T, heads, D), dtype=dtype if out_dtype is None else out_dtype, device=q.device)
        elif out_dtype is not None and q_out.dtype is not out_dtype:
            raise TypeError(f"q_out must be {out_dtype}")
        qop, qot, qoh = _rows("q_out", q_out, dev, (T, heads, D))
        out_code = _code(q_out.dtype)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    cs, max_pos, rot, pos = _rope_args(cos_sin, positions, T, dev)
    args = (cache._ptr, kp, kt, kh, vp, vt, vh, _vec("slot_map", slot_map, torch.int64, T, dev), qp, qt, qh, heads,
            _code(dtype), T, _weight("q_weight", q_weight, D, dev), _weight("k_weight", k_weight, D, dev), eps, cs,
            max_pos, rot, int(interleaved), pos, int(rotate), qop, qot, qoh, out_code)
    return (lib.rw4_kv_append, args, dev, "rw4_kv_append",
            (cache, k, v, slot_map, q, q_weight, k_weight, cos_sin, positions), q_out)


@functools.lru_cache(maxsize=256)
def kv_attention_workspace_bytes(tokens: int, requests: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace kv_attention needs; 0 for invalid sizes."""
    return int(lib.rw4_kv_attention_workspace_bytes(tokens, requests, heads, kv_heads, head_dim))


def kv_attention(q, cache: KVCache, block_table, kv_len, cu_q, *, max_q_len=None, scale=None, causal: bool = True,
                 window: int = 0, unrotate: bool = True, out=None, out_dtype=None, return_lse: bool = False, lse=None,
                 workspace=None):
    """Softmax attention of q [T, heads, D] over the cache: request b owns query tokens cu_q[b]:cu_q[b + 1] and the
    first kv_len[b] cached tokens, in the pages block_table[b].

    causal: a request's queries are its last tokens; window > 0: the last `window` keys only.  scale defaults to
    1 / sqrt(D); unrotate applies the head's Hadamard to the output (for a cache of rotated values).  Returns out [T,
    heads, D], with return_lse (out, lse fp32 [T, heads]).  A row that sees no key gives 0 and -inf, one of no request is
    not written.

    max_q_len is the largest number of query tokens of a request (default: all tokens).  It chooses the kernel for the
    whole call and nothing else, but say it: a decode step of 32 requests without it takes the kernel for many rows, 2 to
    4 times as long, and so do single tokens in one call with a prompt's chunk; two calls can be the faster way there."""
    fn, args, dev, what, _, result = _attention(q, cache, block_table, kv_len, cu_q, max_q_len, scale, causal, window,
                                                unrotate, out, out_dtype, return_lse, lse, workspace)
    _launch(fn, args, dev, what)
    return result


def prepare_kv_attention(q, cache: KVCache, block_table, kv_len, cu_q, *, max_q_len=None, scale=None,
                         causal: bool = True, window: int = 0, unrotate: bool = True, out=None, out_dtype=None,
                         return_lse: bool = False, lse=None, workspace=None) -> Call:
    """kv_attention checked and marshalled once; calling the result runs it.

    Without `workspace` it has one of its own (7 to 68 MB, kv_attention_workspace_bytes), so do not let two runs of it
    overlap in time (two streams, two graphs); prepared calls that run one after the other can be given one together."""
    return KVCall(*_attention(q, cache, block_table, kv_len, cu_q, max_q_len, scale, causal, window, unrotate, out,
                              out_dtype, return_lse, lse, workspace))


def _attention(q, cache, block_table, kv_len, cu_q, max_q_len, scale, causal, window, unrotate, out, out_dtype,
               return_lse, lse, workspace):
    i32, dev, D, kv_heads = torch.int32, cache._dev, cache.head_dim, cache.kv_heads
    qp, qt, qh = _rows("q", q, dev)
    T, heads, dq = q.shape
    if dq != D or heads % kv_heads:
        raise ValueError(f"q must be [tokens, a multiple of {kv_heads}, {D}]")
    if kv_len.dim() != 1:
        raise ValueError("kv_len must be one-dimensional")
    B = kv_len.shape[0]
    table, width = _table(block_table, B, dev)
    if out is None:
        out = torch.empty((T, heads, D), dtype=q.dtype if out_dtype is None else out_dtype, device=q.device)
    elif out_dtype is not None and out.dtype is not out_dtype:
        raise TypeError(f"out must be {out_dtype}")
    op, ot, oh = _rows("out", out, dev, (T, heads, D))
    if lse is not None:
        _out("lse", lse, (T, heads), torch.float32, dev)
    elif return_lse:
        lse = torch.empty((T, heads), dtype=torch.float32, device=q.device)
    nbytes = kv_attention_workspace_bytes(T, B, heads, kv_heads, D)
    if workspace is None:
        wbytes = nbytes if nbytes > 16 else 16
        workspace = torch.empty((wbytes,), dtype=torch.uint8, device=q.device)
    else:
        _on_gpu("workspace", workspace, dev)
        wbytes = workspace.numel() * workspace.element_size()
        if not workspace.is_contiguous() or wbytes < nbytes:
            raise ValueError(f"workspace must be a contiguous tensor of at least {nbytes} bytes")
    args = (cache._ptr, qp, _code(q.dtype), qt, qh, T, heads, table, width, _vec("kv_len", kv_len, i32, B, dev),
            _vec("cu_q", cu_q, i32, B + 1, dev), B, T if max_q_len is None else int(max_q_len),
            D ** -0.5 if scale is None else scale, int(causal), int(window), int(unrotate), op, _code(out.dtype), ot, oh,
            None if lse is None else lse.data_ptr(), workspace.data_ptr(), wbytes)
    return (lib.rw4_kv_attention, args, dev, "rw4_kv_attention",
            (q, cache, block_table, kv_len, cu_q, workspace, lse), (out, lse) if return_lse else out)
