"""Binding of the step operators (``include/paged_gqa_step.h``).

What one step of a model runs around paged attention on a cache held in 8 bits
with one scale for each block of tokens and KV head.  As in the rest of the
package, nothing is computed here: tensors are checked, and their addresses and
strides handed to the library's kernels.

* ``paged_gqa_rope`` / ``paged_gqa_rope_frequencies`` -- rotary positions;
* ``paged_gqa_append_scaled`` -- new K/V rows quantised into the cache;
* ``paged_gqa_decode_scaled`` -- attention of single tokens over it;
* ``paged_gqa_sparse_prefill_scaled`` -- attention of prompt rows over it;
* ``paged_gqa_logits_process`` -- penalties, biases and grammar masks on logits.

A block-scaled cache is a pair of pools [num_pages, page_size, Hkv, 256] of
E4M3 (uint8 or float8_e4m3fn) or INT8 codes with equal strides, and a pair of
float32 scale tensors [num_pages, page_size / scale_block, Hkv] with equal
strides.

Tensors have to be on one CUDA device, which need not be the current one; the
call runs on ``stream``, or on that device's current stream.  Wrong types raise
TypeError, wrong shapes, strides or devices ValueError, and what the library
itself refuses PagedGQAError.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import fp8_kv_cache_gb300 as _P

__all__ = [
    "ROPE_HALF", "ROPE_INTERLEAVED", "paged_gqa_rope", "paged_gqa_rope_frequencies",
    "KV_INT8", "FLAG_BAD_VALUE", "paged_gqa_append_scaled", "paged_gqa_decode_scaled",
    "paged_gqa_decode_scaled_workspace_size", "paged_gqa_sparse_prefill_scaled",
    "FLAG_BAD_INDEX", "paged_gqa_logits_process",
]

KV_INT8 = 2
FLAG_BAD_VALUE = 256
FLAG_BAD_INDEX = 512

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
_ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
_I32, _F16, _F32, _F64 = torch.int32, torch.float16, torch.float32, torch.float64
_FLOAT = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}

_i32, _f64 = ctypes.c_int, ctypes.c_double


# The argument structures of the library's _call functions, packed as C lays them
# out ("P" an address, "q" int64, "i" int, "f" float).
_ROPE_ROWS = "PPqqqqi4x"
_LAYOUTS = "qqq"
_ARGS = {
    "paged_gqa_rope": struct.Struct("@" + 2 * _ROPE_ROWS + "PPP" + "5ifi"),
    "paged_gqa_append_scaled": struct.Struct("@PqqPqqPP" + _LAYOUTS + "PP" + _LAYOUTS + "PqPPPP" + "10i"),
    "paged_gqa_decode_scaled": struct.Struct("@PPP" + _LAYOUTS + "PP" + _LAYOUTS + "PqPPPNPPPP" + "10if"),
    "paged_gqa_sparse_prefill_scaled": struct.Struct("@PPP" + _LAYOUTS + "PP" + _LAYOUTS + "PPPPPP"
                                                     + "10if"),
    "paged_gqa_logits_process": struct.Struct("@PqPq" + "Pqi4xPPPPPPPqi4xPqi4xP" + "PP" + "3i"),
}


def _declare(L):
    """Argument types of the entry points of the loaded library L."""
    L.paged_gqa_rope_frequencies.argtypes = [ctypes.POINTER(_f64), _i32, _f64, _i32, _f64, _f64,
                                             _f64, _f64]
    L.paged_gqa_rope_frequencies.restype = _i32
    L.paged_gqa_decode_scaled_workspace_size.argtypes = [_i32] * 5
    L.paged_gqa_decode_scaled_workspace_size.restype = ctypes.c_size_t
    for name in _ARGS:
        fn = getattr(L, name + "_call")
        fn.argtypes = [ctypes.c_char_p]
        fn.restype = _i32


# ------------------------------------------------------------------ helpers
#
# A call's checks are a good part of what a small call costs, so they look at
# each property once and name what is wrong only when something is.

try:                                   # the current stream's address without a Stream object
    from torch._C import _cuda_getCurrentRawStream as _current_stream
    from torch._C import _cuda_getDevice as _current_device
except ImportError:                    # pragma: no cover
    _current_device = torch.cuda.current_device

    def _current_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _of_type(name, t, dtype):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")


def _device(first, *others):
    """The index of the CUDA device that all tensors share (None is skipped)."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"all tensors must be on one CUDA device: one is on cuda:{dev}, "
                             f"one on {t.device}")
    return dev


def _ids(name, t, n):
    """Address of a contiguous int32 tensor [n]."""
    if t.dtype is not _I32:
        raise TypeError(f"{name} must be torch.int32, not {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape [{n}]")
    return t.data_ptr()


def _stream_of(dev, stream):
    """The address of `stream`, or of the device's current stream."""
    if stream is None:
        return _current_stream(dev)
    if isinstance(stream, int):
        return stream
    _need(stream.device.index == dev, f"stream must belong to cuda:{dev}")
    return stream.cuda_stream


def _call(name, dev, args):
    """Calls the library's `name` on packed arguments with device `dev` current."""
    fn = getattr(_P._lib or _P.lib(), name + "_call")
    if _current_device() == dev:
        st = fn(args)
    else:
        with torch.cuda.device(dev):
            st = fn(args)
    if st != 0:
        raise _P.PagedGQAError(st, name)


def _empty(shape, dtype, dev, stream):
    """A new tensor whose memory belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                  else torch.cuda.default_stream(dev))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")


# ------------------------------------------------------------------ rotary positions

def paged_gqa_rope_frequencies(rot_dim, base=10000.0, *, scaling="none", factor=1.0,
                               original_len=0, low=1.0, high=32.0, device=None):
    """Radians per position of the rot_dim / 2 pairs, float64 on ``device``
    (a host tensor by default): base ** (-2 i / rot_dim), scaled for long
    contexts by ``scaling``: "none", "linear" (divided by factor), "base" (a
    larger base) or "ramp" (pairs of fewer than ``low`` turns over
    ``original_len`` positions divided by factor, those of more than ``high``
    kept, linear between)."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling {scaling!r} is none of {sorted(_ROPE_SCALING)}")
    out = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float64)
    st = _P.lib().paged_gqa_rope_frequencies(
        ctypes.cast(out.data_ptr(), ctypes.POINTER(_f64)), int(rot_dim), float(base),
        _ROPE_SCALING[scaling], float(factor), float(original_len), float(low), float(high))
    if st != 0:
        raise _P.PagedGQAError(st, "paged_gqa_rope_frequencies")
    return out if device is None else out.to(device)


_NO_ROWS = (0, 0, 0, 0, 0, 0, 0)
_pack_rope = _ARGS["paged_gqa_rope"].pack


def _rope_rows(name, x, out, dtype, T, D):
    shape = x.shape
    if len(shape) != 3 or out.shape != shape or shape[0] != T or shape[2] != D:
        raise ValueError(f"{name} and {name}_out must be [T, heads, D], with q's T and D")
    if x.dtype is not dtype or out.dtype is not dtype:
        raise TypeError("q, k and their outputs must have one type")
    s0, s1, s2 = x.stride()
    o0, o1, o2 = out.stride()
    if (s2 != 1 or o2 != 1) and D > 1:
        raise ValueError(f"{name} and {name}_out must have a unit stride along D")
    return x.data_ptr(), out.data_ptr(), s0, s1, o0, o1, shape[1]


def paged_gqa_rope(q, k, positions, inv_freq, *, layout=ROPE_HALF, scale=1.0, inverse=False,
                   q_out=None, k_out=None, stream=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (float16, bfloat16 or
    float32, any strides with unit stride along D; k may be None).

    positions int32 [T]; inv_freq float64 [rot_dim / 2], radians per position
    (paged_gqa_rope_frequencies); elements from rot_dim on pass through.
    ``layout``: ROPE_HALF pairs (i, i + rot_dim / 2), ROPE_INTERLEAVED pairs
    (2i, 2i + 1).  ``scale`` multiplies the rotated elements; ``inverse``
    rotates back.  ``q_out=q`` rotates in place.  Returns (q_out, k_out)."""
    dtype = q.dtype
    kind = _FLOAT.get(dtype)
    if kind is None:
        raise TypeError(f"q must be float16, bfloat16 or float32, not {dtype}")
    dev = _device(q, k, positions, inv_freq, q_out, k_out)
    _need(q.dim() == 3, "q must be [T, heads, D]")
    T, _, D = q.shape
    if q_out is None:
        q_out = _empty(q.shape, dtype, dev, stream)
    rows_q, rows_k = _rope_rows("q", q, q_out, dtype, T, D), _NO_ROWS
    if k is not None:
        if k_out is None:
            k_out = _empty(k.shape, dtype, dev, stream)
        rows_k = _rope_rows("k", k, k_out, dtype, T, D)
        if rows_k[6] == 0:
            rows_k = _NO_ROWS
    else:
        _need(k_out is None, "k_out without k")
    pos = _ids("positions", positions, T)
    if inv_freq.dtype is not _F64:
        raise TypeError(f"inv_freq must be torch.float64, not {inv_freq.dtype}")
    _need(inv_freq.dim() == 1 and inv_freq.is_contiguous(), "inv_freq must be contiguous and 1-D")
    if layout not in (ROPE_HALF, ROPE_INTERLEAVED):
        raise ValueError("layout must be ROPE_HALF or ROPE_INTERLEAVED")
    if T > 0:
        _call("paged_gqa_rope", dev, _pack_rope(
            *rows_q, *rows_k, pos, inv_freq.data_ptr(), _stream_of(dev, stream), T, D, kind,
            2 * inv_freq.shape[0], layout, scale, bool(inverse)))
    return q_out, k_out


# ------------------------------------------------------------------ block-scaled caches

_CODES = {torch.uint8: 1, torch.float8_e4m3fn: 1, torch.int8: 2}


def _scaled_cache(k_cache, v_cache, k_scales, v_scales, page_size):
    """Checks a block-scaled cache: (k_cache .. scale_layout as packed, kv_dtype,
    scale_block, num_pages, Hkv, D)."""
    dtype = k_cache.dtype
    kind = _CODES.get(dtype)
    if kind is None or v_cache.dtype is not dtype:
        raise TypeError("k_cache and v_cache must both be uint8 / float8_e4m3fn (E4M3) or int8")
    if k_scales.dtype is not _F32 or v_scales.dtype is not _F32:
        raise TypeError("k_scales and v_scales must be float32")
    shape, st = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or v_cache.stride() != st or st[3] != 1:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, Hkv, D] of equal "
                         "strides, with a unit stride along D")
    sh, ss = k_scales.shape, k_scales.stride()
    pages, page, Hkv, D = shape
    if (len(sh) != 3 or v_scales.shape != sh or v_scales.stride() != ss or sh[0] != pages or
            sh[2] != Hkv):
        raise ValueError("k_scales and v_scales must be [num_pages, blocks per page, Hkv] of "
                         "equal strides")
    per = sh[1]
    if page_size != page or per < 1 or page % per != 0:
        raise ValueError("page_size must be the cache's, and a multiple of the scales' blocks "
                         "per page")
    return ((k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2], k_scales.data_ptr(),
             v_scales.data_ptr(), *ss), kind, page // per, pages, Hkv, D)


def _block_table(t, B, max_seq_len, page_size):
    """Checks the int32 block table [B, n]: its address, its row stride, and
    max_seq_len, by default all it covers."""
    shape, st = t.shape, t.stride()
    if t.dtype is not _I32:
        raise TypeError(f"block_table must be torch.int32, not {t.dtype}")
    if len(shape) != 2 or shape[0] != B or (st[1] != 1 and shape[1] > 1):
        raise ValueError("block_table must be [B, pages] with a unit column stride")
    most = shape[1] * page_size
    if max_seq_len is None:
        max_seq_len = min(most, 0x7fffffff)
    elif not 0 <= max_seq_len <= most:
        raise ValueError("block_table must have ceil(max_seq_len / page_size) columns")
    return t.data_ptr(), st[0], max_seq_len


def _err(err_flag):
    if err_flag is None:
        return 0
    _of_type("err_flag", err_flag, torch.int32)
    _need(err_flag.numel() >= 1, "err_flag must hold an int32")
    return err_flag.data_ptr()


_pack_append = _ARGS["paged_gqa_append_scaled"].pack


def paged_gqa_append_scaled(k, v, k_cache, v_cache, k_scales, v_scales, block_table, seq_starts,
                            page_size, *, new_offsets=None, max_seq_len=None, num_pages=None,
                            err_flag=None, stream=None):
    """Quantises new rows into a block-scaled cache, in place.

    k, v [T, Hkv, 256] float16, bfloat16 or float32: sequence b's new tokens
    are rows new_offsets[b] .. new_offsets[b + 1] - 1 (int32 [B + 1]; without
    it row b alone), stored at positions seq_starts[b] and on (int32 [B], the
    tokens stored before).  A scale block that already holds rows keeps the
    larger scale, and its rows are coded again when it grows.  block_table
    int32 [B, pages]; rows at positions from max_seq_len (default: all the
    table covers) on are dropped.  No page may be written for two sequences, or
    in two places of one, in a call.  Returns (k_cache, v_cache)."""
    kind = _FLOAT.get(k.dtype)
    if kind is None or v.dtype is not k.dtype:
        raise TypeError("k and v must both be float16, bfloat16 or float32")
    dev = _device(k, v, k_cache, v_cache, k_scales, v_scales, block_table, seq_starts, new_offsets,
                  err_flag)
    cache, codes, block, pages, Hkv, D = _scaled_cache(k_cache, v_cache, k_scales, v_scales, page_size)
    _need(seq_starts.dim() == 1, "seq_starts must be [B]")
    B = seq_starts.shape[0]
    starts = _ids("seq_starts", seq_starts, B)
    shape, ks, vs = k.shape, k.stride(), v.stride()
    if len(shape) != 3 or v.shape != shape or shape[1:] != (Hkv, D) or ks[2] != 1 or vs[2] != 1:
        raise ValueError("k and v must be [T, Hkv, D], with a unit stride along D")
    T = shape[0]
    if new_offsets is None:
        offsets = 0
        _need(T == B, "without new_offsets there is one row for each sequence")
    else:
        offsets = _ids("new_offsets", new_offsets, B + 1)
    table, stride, most = _block_table(block_table, B, max_seq_len, page_size)
    if num_pages is not None:
        pages = _pages(num_pages, pages)
    if T > 0 and B > 0:
        _call("paged_gqa_append_scaled", dev, _pack_append(
            k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], *cache, table, stride, starts,
            offsets, _err(err_flag), _stream_of(dev, stream), kind, T, codes, block, B, Hkv, D,
            page_size, pages, most))
    return k_cache, v_cache


def _pages(num_pages, pool):
    """num_pages, at most the pool's."""
    if not 1 <= num_pages <= pool:
        raise ValueError("num_pages must be within the pool")
    return num_pages


def _q_out(q, out, dev, stream, Hkv, D):
    """Checks contiguous float16 q [rows, Hq, D]; out, made when not given."""
    if q.dtype is not _F16:
        raise TypeError(f"q must be torch.float16, not {q.dtype}")
    shape = q.shape
    if len(shape) != 3 or shape[2] != D or not q.is_contiguous() or Hkv < 1 or shape[1] % Hkv != 0:
        raise ValueError("q must be a contiguous [rows, Hq, D] tensor, Hq a multiple of the "
                         "cache's heads")
    if out is None:
        return _empty(shape, torch.float16, dev, stream)
    if out.dtype is not _F16:
        raise TypeError(f"out must be torch.float16, not {out.dtype}")
    if out.shape != shape or not out.is_contiguous():
        raise ValueError("out must be contiguous and of q's shape")
    return out


def paged_gqa_decode_scaled_workspace_size(B, Hq, Hkv, D, splits=0) -> int:
    """Bytes of workspace of a call on the current device (splits: force_splits)."""
    return int(_P.lib().paged_gqa_decode_scaled_workspace_size(B, Hq, Hkv, D, splits))


_pack_decode = _ARGS["paged_gqa_decode_scaled"].pack


def paged_gqa_decode_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens,
                            page_size, softmax_scale, out=None, *, max_seq_len=None,
                            num_pages=None, workspace=None, force_splits=0, err_flag=None,
                            split_events=None, stream=None):
    """Batched paged decode over a block-scaled cache: paged_gqa_decode with a
    scale for each block of tokens and KV head.

    q [B, Hq, 256] float16; block_table int32 [B, pages]; seq_lens int32 [B],
    at most max_seq_len (default: all the table covers).  ``workspace``: a
    CUDA uint8 tensor of paged_gqa_decode_scaled_workspace_size bytes, None to
    allocate one, False for none (long contexts are slower without); calls that
    may overlap need one each.  ``force_splits`` CTAs share all tokens; without
    effect where there is no workspace, or more than 4096 sequences.  Returns out."""
    dev = q.get_device()
    if not (dev == k_cache.get_device() == v_cache.get_device() == k_scales.get_device() ==
            v_scales.get_device() == block_table.get_device() == seq_lens.get_device() >= 0):
        _device(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens)
    if out is not None or err_flag is not None:
        _device(q, out, err_flag)
    cache, codes, block, pages, Hkv, D = _scaled_cache(k_cache, v_cache, k_scales, v_scales, page_size)
    out = _q_out(q, out, dev, stream, Hkv, D)
    B, Hq, _ = q.shape
    lens = _ids("seq_lens", seq_lens, B)
    table, stride, most = _block_table(block_table, B, max_seq_len, page_size)
    if num_pages is not None:
        pages = _pages(num_pages, pages)
    if B == 0:
        return out
    if workspace is None:
        with torch.cuda.device(dev):
            n = paged_gqa_decode_scaled_workspace_size(B, Hq, Hkv, D, force_splits)
        workspace = _empty((max(n, 256),), torch.uint8, dev, stream)
    ws, n = 0, 0
    if workspace is not False:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
        ws, n = workspace.data_ptr(), workspace.nbytes
    e0, e1 = (0, 0) if split_events is None else [e.cuda_event for e in split_events]
    _call("paged_gqa_decode_scaled", dev, _pack_decode(
        q.data_ptr(), *cache, table, stride, lens, out.data_ptr(), ws, n, _err(err_flag), e0, e1,
        _stream_of(dev, stream), codes, block, B, Hq, Hkv, D, page_size, pages, most, force_splits,
        softmax_scale))
    return out


_pack_prefill = _ARGS["paged_gqa_sparse_prefill_scaled"].pack


def paged_gqa_sparse_prefill_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, kv_len,
                                    sel_idx, q_pos, page_size, softmax_scale, out=None, *,
                                    num_pages=None, err_flag=None, stream=None):
    """Selected-sparse prefill of one sequence over a block-scaled cache:
    paged_gqa_sparse_prefill with a scale for each block of tokens and KV head.

    q [R, Hq, 256] float16; block_table int32 [pages of the sequence]; sel_idx
    int32 [R, n_sel] four-token block ids; q_pos int32 [R].  Returns out."""
    dev = _device(q, k_cache, v_cache, k_scales, v_scales, block_table, sel_idx, q_pos, out,
                  err_flag)
    cache, codes, block, pages, Hkv, D = _scaled_cache(k_cache, v_cache, k_scales, v_scales, page_size)
    out = _q_out(q, out, dev, stream, Hkv, D)
    R, Hq, _ = q.shape
    if sel_idx.dtype is not _I32:
        raise TypeError(f"sel_idx must be torch.int32, not {sel_idx.dtype}")
    if sel_idx.dim() != 2 or sel_idx.shape[0] != R or not sel_idx.is_contiguous():
        raise ValueError("sel_idx must be a contiguous tensor [R, n_sel]")
    pos = _ids("q_pos", q_pos, R)
    n_table, n_sel = block_table.numel(), sel_idx.shape[1]
    table = _ids("block_table", block_table, n_table)
    if not 0 <= kv_len <= n_table * page_size:
        raise ValueError("block_table must have ceil(kv_len / page_size) entries")
    if num_pages is not None:
        pages = _pages(num_pages, pages)
    if R > 0:
        _call("paged_gqa_sparse_prefill_scaled", dev, _pack_prefill(
            q.data_ptr(), *cache, table, sel_idx.data_ptr() if n_sel else 0, pos, out.data_ptr(),
            _err(err_flag), _stream_of(dev, stream), codes, block, pages, kv_len, n_sel, R, Hq, Hkv,
            D, page_size, softmax_scale))
    return out


# ------------------------------------------------------------------ logits

def _rows(name, t, dtype, B):
    """Checks [B, n] with unit column stride: its address, row stride and n."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != B or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be [{B}, n] with a unit column stride")
    return t.data_ptr(), st[0], shape[1]


def _per_row(name, t, dtype, B):
    """Address of a contiguous [B] tensor, or 0."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {B}")
    return t.data_ptr()


_pack_logits = _ARGS["paged_gqa_logits_process"].pack


def paged_gqa_logits_process(logits, *, history=None, history_lens=None, prompt_lens=None,
                             repetition=None, frequency=None, presence=None, bias_tokens=None,
                             bias_values=None, mask=None, mask_rows=None, out=None, err_flag=None,
                             stream=None):
    """Penalties, biases and a grammar mask on logits [B, V] (float32, float16
    or bfloat16), as float32; what paged_gqa_topk_topp_mask takes.

    history int32 [B, n]: the token ids so far, history_lens int32 [B] of them
    (default n; negative ids are padding), the first prompt_lens int32 [B]
    (default 0) of the prompt.  repetition float32 [B] divides positive and
    multiplies other logits of all those tokens; frequency and presence float32
    [B] take frequency * count + presence from tokens generated count times.
    bias_tokens int32 and bias_values float32 [B, m] are added (negative tokens
    are padding).  mask int32 [rows, ceil(V / 32)]: bit v % 32 of word v / 32
    allows token v; mask_rows int32 [B] names each row's (negative: none;
    default row b).  ``out=logits`` works in place.  Returns out."""
    kind = _FLOAT.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be float32, float16 or bfloat16, not {logits.dtype}")
    dev = _device(logits, history, history_lens, prompt_lens, repetition, frequency, presence,
                  bias_tokens, bias_values, mask, mask_rows, out, err_flag)
    _need(logits.dim() == 2 and logits.shape[1] >= 1, "logits must be [B, V]")
    B, V = logits.shape
    if out is None:
        out = _empty((B, V), torch.float32, dev, stream)
    x, x_stride, _ = _rows("logits", logits, logits.dtype, B)
    y, y_stride, n = _rows("out", out, torch.float32, B)
    _need(n == V, "out must be of logits' shape")
    i32, f32 = _I32, _F32
    hist = (0, 0, 0, 0, 0, 0, 0, 0)
    if history is not None:
        hist = (*_rows("history", history, i32, B), _per_row("history_lens", history_lens, i32, B),
                _per_row("prompt_lens", prompt_lens, i32, B),
                _per_row("repetition", repetition, f32, B),
                _per_row("frequency", frequency, f32, B), _per_row("presence", presence, f32, B))
    elif not (history_lens is prompt_lens is repetition is frequency is presence is None):
        raise ValueError("penalties need the history")
    bias = (0, 0, 0, 0)
    if bias_tokens is not None and bias_values is not None:
        tokens, b_stride, m = _rows("bias_tokens", bias_tokens, i32, B)
        values, stride, n = _rows("bias_values", bias_values, f32, B)
        if n != m or (B > 1 and stride != b_stride):
            raise ValueError("bias_tokens and bias_values must share shape and row stride")
        bias = (tokens, values, b_stride, m)
    elif bias_tokens is not bias_values:
        raise ValueError("bias_tokens and bias_values come together")
    masks = (0, 0, 0, 0)
    if mask is not None:
        rows = mask.shape[0]
        words, stride, n = _rows("mask", mask, i32, rows)
        if n < (V + 31) // 32:
            raise ValueError("mask must have ceil(V / 32) words a row")
        if mask_rows is None and rows < B:
            raise ValueError("without mask_rows there is a mask row for each row")
        masks = (words, stride, rows, _per_row("mask_rows", mask_rows, i32, B))
    else:
        _need(mask_rows is None, "mask_rows without a mask")
    if B > 0:
        _call("paged_gqa_logits_process", dev, _pack_logits(
            x, x_stride, y, y_stride, *hist, *bias, *masks, _err(err_flag), _stream_of(dev, stream),
            kind, B, V))
    return out
