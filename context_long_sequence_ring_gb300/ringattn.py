"""Thin Python binding of libringattn.so (argument marshalling only).

Every computation runs in the library's CUDA kernels; this module checks
shapes/dtypes, passes raw device pointers and the current CUDA stream, and
turns a non-zero ``ra_status`` into ``RingAttnError``.  There is no fallback:
if the library is not built, or no GPU is present, calls fail loudly.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

from .build import LIB

RA_OK, RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED, RA_ERR_CUDA, RA_ERR_TIMEOUT, RA_ERR_DEVICE_BOUNDS = range(6)
RA_F32, RA_BF16 = 0, 1
LAYOUTS = {"natural": 0, "zigzag": 1}
ROPE_STYLES = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

_c = ctypes
_vp, _i32, _i64, _u64, _f32, _sz = _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_uint64, _c.c_float, _c.c_size_t

# name -> argument types (restype is ra_status unless noted)
SIGNATURES = {
    "ra_device_status": [_vp],
    "ra_zigzag_partition": [_c.POINTER(_i64), _i32, _i32, _vp, _vp, _c.POINTER(_i64), _c.POINTER(_i64), _vp],
    "ra_gather_rows": [_vp, _i64, _vp, _vp, _i64, _i64, _vp],
    "ra_rope_gather": [_vp, _i64, _i32, _i32, _c.c_int, _vp, _i64, _vp, _c.c_double, _vp, _vp],
    "ra_ring_attn_fwd": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _c.c_int, _i32, _i32, _f32,
                         _c.c_int, _vp],
    "ra_ring_attn_fwd_ex": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _c.c_int, _i32, _i32, _f32,
                            _c.c_int, _i32, _vp],
    "ra_ring_attn_fwd_varlen": [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _c.c_int, _i32, _i32, _f32,
                                _vp],
    "ra_ring_schedule_counts": [_i32, _i32, _i32, _vp, _vp],
    "ra_ring_schedule_counts_ex": [_i32, _i32, _i32, _i32, _vp, _vp],
    "ra_lse_merge": [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _c.c_int, _vp, _vp],
    "ra_ring_step_fwd": [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _vp,
                         _c.c_int, _vp, _vp],
    "ra_attn_block_fwd": [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i64, _i64, _i32, _f32, _vp, _vp, _vp],
    "ra_segmented_prefill_workspace_size": [_i32, _i32, _i32, _i32, _i32, _c.POINTER(_sz)],
    "ra_segmented_prefill_fwd": [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i64, _i32, _f32, _i32, _vp,
                                 _c.c_int, _vp, _vp, _sz, _vp],
    "ra_cp_slot_mapping": [_vp, _vp, _vp, _i32, _i32, _i64, _i32, _i32, _i32, _i32, _vp, _vp],
    "ra_cp_kv_scatter": [_vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i64, _c.c_int, _vp],
    "ra_cp_kv_gather": [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                        _c.c_int, _vp, _vp, _vp],
    "ra_cp_decode_workspace_size": [_i32, _i32, _i32, _i32, _i32, _i32, _i32, _c.POINTER(_sz)],
    "ra_cp_decode": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64, _f32,
                     _i32, _vp, _c.c_int, _vp, _vp, _sz, _vp],
    "ra_cp_decode_noalloc": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                             _f32, _i32, _vp, _c.c_int, _vp, _vp],
    "ra_cp_decode_partials": [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                              _i32, _i64, _f32, _i32, _vp, _vp, _c.POINTER(_i32), _vp],
    "ra_cp_lse_rescale": [_vp, _vp, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _vp],
    "ra_cp_head_split": [_vp, _vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp],
    "ra_rope_apply": [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _c.c_int, _c.c_int, _vp, _vp, _vp,
                      _c.c_double, _i32, _vp],
    "ra_rope_frequencies": [_c.c_int, _c.c_double, _i32, _c.c_double, _c.c_double, _vp, _c.POINTER(_c.c_double)],
    "ra_cp_chunk_attn_workspace_size": [_i32, _i32, _i32, _c.POINTER(_sz)],
    "ra_cp_chunk_attn": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                         _i32, _f32, _vp, _c.c_int, _vp, _vp, _sz, _vp],
    "ra_cp_attn_weights": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                           _i64, _i32, _f32, _vp, _vp, _vp],
    "ra_cp_evict": [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _c.c_int, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                    _i32, _i32, _i32, _vp, _vp, _vp],
    "ra_rope_apply_axes": [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _c.c_int, _c.c_int, _vp, _i32, _vp,
                           _vp, _c.c_double, _i32, _vp],
    "ra_cp_rope_append": [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64,
                          _i32, _i32, _i32, _i32, _c.c_int, _i32, _i32, _i32, _i32, _i32, _i64, _vp, _i32, _i32, _c.c_int,
                          _vp, _vp, _c.c_double, _vp],
    "ra_cp_window_attn_workspace_size": [_i32, _i32, _i32, _c.POINTER(_sz)],
    "ra_cp_window_attn": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64,
                          _i32, _i32, _f32, _vp, _c.c_int, _vp, _vp, _sz, _vp],
    "ra_window_attn_workspace_size": [_i64, _i32, _i32, _i32, _i32, _c.POINTER(_sz)],
    "ra_window_attn_fwd": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp,
                           _c.c_int, _vp, _vp, _sz, _vp],
    "ra_window_attn_bwd": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _i32,
                           _f32, _vp, _i64, _vp, _i64, _vp, _i64, _c.c_int, _vp, _sz, _vp],
    "ra_selftest_wait_timeout": [_i64, _vp],
    "ra_synth_fill": [_u64, _i64, _vp, _i32, _vp, _vp],
}
STRING_FUNCS = ["ra_last_error", "ra_version"]


class RingAttnError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("ra_status %d: %s" % (status, msg))
        self.status = status


_lib = None


def lib():
    """The loaded library (ctypes), with argument types set."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError("libringattn.so is not built: run __graft_entry__.build() "
                               "(python -m context_long_sequence_ring_gb300.build)")
        L = ctypes.CDLL(LIB)
        for name, args in SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = _c.c_int
        for name in STRING_FUNCS:
            getattr(L, name).restype = _c.c_char_p
            getattr(L, name).argtypes = []
        _lib = L
    return _lib


class _Entries:
    """Entry points as attributes, each looked up in the library the first time."""

    def __getattr__(self, name):
        f = getattr(lib(), name)
        setattr(self, name, f)
        return f


_LIB = _Entries()


def last_error() -> str:
    return lib().ra_last_error().decode()


def version() -> str:
    return lib().ra_version().decode()


def _check(status: int):
    if status != RA_OK:
        raise RingAttnError(status, last_error())


def _stream() -> int:
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensor must be on a CUDA device")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensor must be contiguous")


def _here(first, *ts) -> int:
    """The current CUDA device, which all the (contiguous) tensors must be on; None is left out."""
    dev = first.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or not first.is_contiguous():
        raise ValueError("tensors must be contiguous and on the current CUDA device")
    for t in ts:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on the current CUDA device")
    return dev


def _of(dtype, *ts):
    for t in ts:
        if t is not None and t.dtype != dtype:
            raise ValueError("dtype must be %s, not %s" % (dtype, t.dtype))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return RA_BF16
    if t.dtype == torch.float32:
        return RA_F32
    raise ValueError("dtype must be bfloat16 or float32")


def device_status() -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    return lib().ra_device_status(_stream())


# ---------------------------------------------------------------------- partition

def zigzag_partition(seq_lens: Sequence[int], n_ranks: int, device="cuda"):
    """(perm int32 [G], restore int32 [sum L]) of the head-tail partition."""
    n = len(seq_lens)
    arr = (_i64 * max(n, 1))(*[int(x) for x in seq_lens])
    G, T = _i64(0), _i64(0)
    _check(lib().ra_zigzag_partition(arr, n, n_ranks, None, None, _c.byref(G), _c.byref(T), _stream()))
    perm = torch.empty(G.value, dtype=torch.int32, device=device)
    restore = torch.empty(T.value, dtype=torch.int32, device=device)
    if G.value > 0:
        _check(lib().ra_zigzag_partition(arr, n, n_ranks, _ptr(perm), _ptr(restore), None, None, _stream()))
    return perm, restore


def gather_rows(src: torch.Tensor, idx: torch.Tensor, out: Optional[torch.Tensor] = None):
    """out[i] = src[idx[i]] (zero rows where idx < 0); rows are the first dim."""
    _need_cuda(src, idx, out)
    if idx.dtype != torch.int32:
        raise ValueError("idx must be int32")
    rows = idx.numel()
    if out is None:
        out = torch.empty((rows,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    row_bytes = src[0].numel() * src.element_size() if src.shape[0] > 0 else 0
    _check(lib().ra_gather_rows(_ptr(src), src.shape[0], _ptr(idx), _ptr(out), rows, row_bytes, _stream()))
    return out


def rope_gather(src: torch.Tensor, positions: torch.Tensor, idx: Optional[torch.Tensor] = None,
                base: float = 10000.0, out: Optional[torch.Tensor] = None):
    """Rotary position embedding fused with a row gather: out[r] = RoPE(src[idx[r]],
    positions[idx[r]]), zero rows where idx < 0.  src [rows, H, d]; positions int32, one per
    source row.  Without idx the rows keep their order (out may be src: in place)."""
    _need_cuda(src, positions, idx, out)
    if src.dim() != 3:
        raise ValueError("src must be [rows, H, d]")
    if positions.dtype != torch.int32 or (idx is not None and idx.dtype != torch.int32):
        raise ValueError("positions and idx must be int32")
    if positions.numel() != src.shape[0]:
        raise ValueError("one position per source row")
    rows = idx.numel() if idx is not None else src.shape[0]
    if out is None:
        out = torch.empty((rows,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    _check(lib().ra_rope_gather(_ptr(src), src.shape[0], src.shape[1], src.shape[2], _dt(src),
                                _ptr(idx) if idx is not None else None, rows, _ptr(positions), float(base),
                                _ptr(out), _stream()))
    return out


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_len: float = 32768.0):
    """Frequency table of ``rope_apply``: (inv_freq float64 [rot/2] on the host, mscale), base^(-2i/rot) as it
    is ("none") or changed for contexts ``factor`` times the trained length ("linear", "ntk", "yarn")."""
    f, m = torch.empty(max(rot // 2, 0), dtype=torch.float64), _c.c_double(1.0)
    _check(lib().ra_rope_frequencies(ROPE_SCALINGS[scaling], float(base), rot, float(factor), float(trained_len),
                                     _ptr(f), _c.byref(m)))
    return f, m.value


def rope_apply(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, mscale: float = 1.0,
               style: str = "half", idx: Optional[torch.Tensor] = None, backward: bool = False,
               out: Optional[torch.Tensor] = None):
    """Rotary positions of x [rows, H, d] (any strides with the last one 1): the first 2*len(inv_freq)
    components of each head are turned, the others copied.  inv_freq float64 on the host
    (``rope_frequencies``); positions int32, one per OUTPUT row.  out[r] comes from x[idx[r]] with idx
    (zero rows where idx < 0), else from x[r]; without idx, out may be x (in place).  ``backward`` turns
    by the negative angles: the gradient of x from the gradient of out."""
    dev = _here(positions, idx)
    if positions.dtype != torch.int32 or (idx is not None and idx.dtype != torch.int32):
        raise ValueError("positions and idx must be int32")
    if x.get_device() != dev:
        raise ValueError("x must be on the current CUDA device")
    _frequency_table(inv_freq)
    if x.dim() != 3:
        raise ValueError("x must be [rows, H, d]")
    rows, H, d = x.shape
    rs, hs, es = x.stride()
    n = rows if idx is None else idx.numel()
    if positions.numel() != n:
        raise ValueError("one position per output row")
    if out is None:
        out = torch.empty((n, H, d), dtype=x.dtype, device=positions.device)
        ors, ohs, oes = H * d, d, 1
    else:
        if out.shape != (n, H, d) or out.dtype != x.dtype or out.get_device() != dev:
            raise ValueError("out must be %s of x's dtype, on its device" % ((n, H, d),))
        ors, ohs, oes = out.stride()
    if (es != 1 or oes != 1) and d > 1:
        raise ValueError("the elements of a head must be contiguous")
    _check(lib().ra_rope_apply(x.data_ptr(), rows, rs, hs, out.data_ptr(), ors, ohs, n, H, d, 2 * inv_freq.numel(),
                               _dt(x), ROPE_STYLES[style], _ptr(idx), positions.data_ptr(), inv_freq.data_ptr(), mscale,
                               1 if backward else 0, torch._C._cuda_getCurrentRawStream(dev)))
    return out


def _frequency_table(inv_freq):
    if inv_freq.dtype != torch.float64 or inv_freq.is_cuda or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 vector on the host")


def _heads_of(x, what, dev, dtype):
    """Row and head stride of [rows, heads, d] with dense heads' elements."""
    if x.dim() != 3 or x.get_device() != dev or x.dtype != dtype:
        raise ValueError("%s must be [rows, heads, d] of %s on the current CUDA device" % (what, dtype))
    rs, hs, es = x.stride()
    if es != 1 and x.shape[2] > 1:
        raise ValueError("the elements of a head of %s must be contiguous" % what)
    return rs, hs


def rope_apply_axes(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, axis: torch.Tensor,
                    mscale: float = 1.0, style: str = "half", backward: bool = False, out: Optional[torch.Tensor] = None):
    """Rotary positions with several axes: ``rope_apply`` of x [rows, H, d] (any strides with the last one 1)
    with pair i turned by positions[axis[i]] * inv_freq[i].  positions int32 [axes, rows] (e.g. time, height
    and width); inv_freq float64 and axis int32, both [rot/2] on the host.  out may be x (in place).
    ``backward`` turns by the negative angles: the gradient of x from the gradient of out."""
    rows, H, d = x.shape
    rs, hs, es = x.stride()
    dt, dev, n_axes, half = x.dtype, x.get_device(), positions.shape[0], axis.numel()
    if out is None:
        out = torch.empty((rows, H, d), dtype=dt, device=x.device)
    ors, ohs, oes = out.stride()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and positions.get_device() == dev and out.get_device() == dev):
        raise ValueError("tensors must be on the current CUDA device")
    if not (out.dtype == dt and out.shape == x.shape and ((es == 1 and oes == 1) or d <= 1)):
        raise ValueError("x and out must be alike, [rows, H, d], the elements of a head contiguous")
    if not (positions.dtype == torch.int32 and positions.shape == (n_axes, rows) and positions.is_contiguous()):
        raise ValueError("positions must be contiguous int32 [axes, rows]")
    if not (inv_freq.dtype == torch.float64 and axis.dtype == torch.int32 and inv_freq.shape == (half,) and axis.dim() == 1
            and inv_freq.get_device() < 0 and axis.get_device() < 0 and inv_freq.is_contiguous() and axis.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous float64 vector on the host, axis an int32 one as long")
    st = _LIB.ra_rope_apply_axes(x.data_ptr(), rs, hs, out.data_ptr(), ors, ohs, rows, H, d, 2 * half, _dt(x),
                                 ROPE_STYLES[style], positions.data_ptr(), n_axes, inv_freq.data_ptr(), axis.data_ptr(),
                                 mscale, 1 if backward else 0, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st)
    return out


# ---------------------------------------------------------------------- attention

def ring_attn_fwd(q, k, v, causal: bool, n_ranks: int, B: int = 1, scale: Optional[float] = None,
                  layout: str = "natural", o=None, lse=None, variant: int = 0):
    """Ring-order attention forward.  q [B*S, Hq, d], k/v [B*S, Hkv, d] token-major.

    Returns (O [B*S, Hq, d] in q's dtype, LSE float32 [B*S, Hq]).  ``variant`` picks the
    bf16 kernel (0 automatic, 1 one head per CTA, 2 two GQA heads per CTA, 3 two adjacent query
    tiles of one head per CTA)."""
    _need_cuda(q, k, v, o, lse)
    rows, Hq, d = q.shape
    Hkv = k.shape[1]
    if rows % B != 0:
        raise ValueError("rows of q must be a multiple of B")
    S = rows // B
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_ring_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, S, d, _dt(q),
                                     1 if causal else 0, n_ranks, float(scale or 0.0), LAYOUTS[layout], variant,
                                     _stream()))
    return o, lse


def ring_schedule_counts(S: int, n_ranks: int, causal: bool, kv_tile: int = 128, device="cuda"):
    """Per rank: (unmasked, causally masked, skipped) (query tile, key tile) pairs of the kernels' schedule."""
    out = torch.empty((n_ranks, 3), dtype=torch.int64, device=device)
    _check(lib().ra_ring_schedule_counts_ex(S, n_ranks, 1 if causal else 0, kv_tile, _ptr(out), _stream()))
    return out


def ring_attn_fwd_varlen(q, k, v, seq_lens: Sequence[int], causal: bool, n_ranks: int,
                         scale: Optional[float] = None, o=None, lse=None):
    """Ring-order attention over requests of different lengths, on the head-tail gathered layout
    (``zigzag_partition(seq_lens, n_ranks)`` then ``gather_rows``).  q [G, Hq, d], k/v [G, Hkv, d]
    bf16 with G the padded total; returns (O [G, Hq, d], LSE float32 [G, Hq]) in the same order."""
    _need_cuda(q, k, v, o, lse)
    rows, Hq, d = q.shape
    n = len(seq_lens)
    G = sum(-(-int(L) // (2 * n_ranks)) * 2 * n_ranks for L in seq_lens)
    if rows != G or k.shape[0] != G or v.shape[0] != G:
        raise ValueError("q, k, v must have the %d rows of the padded gathered layout" % G)
    arr = (_i64 * max(n, 1))(*[int(x) for x in seq_lens])
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_ring_attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), arr, n, Hq, k.shape[1], d,
                                         _dt(q), 1 if causal else 0, n_ranks, float(scale or 0.0), _stream()))
    return o, lse


def ring_step_fwd(q, k, v, n_ranks: int, rank: int, src: int, causal: bool, o_in=None, lse_in=None,
                  o_out=None, lse_out=None, B: int = 1, scale: Optional[float] = None):
    """One ring step of rank ``rank``: its local queries q [B*2c, Hq, d] (chunks rank and 2N-1-rank
    of each sequence) against the held block k/v [B*2c, Hkv, d] of rank ``src``, folded into the
    running result (o_in fp32 [B*2c, Hq, d], lse_in [B*2c, Hq]; None at the first step).  o_out
    (fp32 or bf16; may be o_in when fp32) and lse_out (may be lse_in) receive the result; fp32
    buffers are made when they are not given.  Returns (o_out, lse_out)."""
    _need_cuda(q, k, v, o_in, lse_in, o_out, lse_out)
    rows, Hq, d = q.shape
    if rows % (2 * B) != 0 or k.shape[0] != rows or v.shape[0] != rows:
        raise ValueError("q, k, v must hold B sequences of 2c local rows each")
    if o_out is None:
        o_out = torch.empty((rows, Hq, d), dtype=torch.float32, device=q.device)
    if lse_out is None:
        lse_out = torch.empty((rows, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_ring_step_fwd(_ptr(q), _ptr(k), _ptr(v), B, Hq, k.shape[1], rows // (2 * B), d, n_ranks, rank,
                                  src, 1 if causal else 0, float(scale or 0.0), _ptr(o_in), _ptr(lse_in),
                                  _ptr(o_out), _dt(o_out), _ptr(lse_out), _stream()))
    return o_out, lse_out


def ring_step_fn(n_ranks: int, rank: int, causal: bool, B: int = 1, scale: Optional[float] = None):
    """The step callable of ``cp_dist.ring_attention`` for rank ``rank``, on ra_ring_step_fwd."""
    def step(q, k, v, src, o_in, lse_in, o_out, lse_out):
        ring_step_fwd(q, k, v, n_ranks, rank, src, causal, o_in, lse_in, o_out, lse_out, B=B, scale=scale)
    return step


def attn_block_fwd(q, k, v, q_pos0: int, k_pos0: int, causal: bool, scale: Optional[float] = None,
                   o_part=None, lse_part=None):
    """Partial attention of q [Tq, Hq, d] (positions q_pos0..) over k/v [Tk, Hkv, d] (positions k_pos0..)
    -> (O_part fp32 [Tq, Hq, d], LSE_part [Tq, Hq]); -inf / 0 for rows with no visible key."""
    _need_cuda(q, k, v, o_part, lse_part)
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    if o_part is None:
        o_part = torch.empty((Tq, Hq, d), dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty((Tq, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_attn_block_fwd(_ptr(q), _ptr(k), _ptr(v), Tq, Tk, Hq, Hkv, d, int(q_pos0), int(k_pos0),
                                   1 if causal else 0, float(scale or 0.0), _ptr(o_part), _ptr(lse_part),
                                   _stream()))
    return o_part, lse_part


def segmented_prefill_fwd(q, k, v, q_pos0: int, seg_tokens: int, causal: bool = True,
                          scale: Optional[float] = None, out_dtype=torch.bfloat16, workspace=None, o=None, lse=None):
    """Chunked prefill of q [Tq, Hq, d] (positions q_pos0..) over k/v [Tk, Hkv, d] (positions 0..) in
    key segments of seg_tokens -> (O [Tq, Hq, d], LSE [Tq, Hq]).  O takes out_dtype, or the dtype of a
    given ``o``."""
    _need_cuda(q, k, v, workspace, o, lse)
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    n = _sz(0)
    _check(lib().ra_segmented_prefill_workspace_size(Tq, Tk, Hq, d, seg_tokens, _c.byref(n)))
    if workspace is None:
        workspace = torch.empty(n.value, dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty((Tq, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((Tq, Hq), dtype=torch.float32, device=q.device)
    out_dtype = o.dtype
    _check(lib().ra_segmented_prefill_fwd(_ptr(q), _ptr(k), _ptr(v), Tq, Tk, Hq, Hkv, d, int(q_pos0),
                                          1 if causal else 0, float(scale or 0.0), seg_tokens, _ptr(o),
                                          RA_BF16 if out_dtype == torch.bfloat16 else RA_F32, _ptr(lse),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream()))
    return o, lse


def allgather_attend_fn(seq_len: int, n_ranks: int, rank: int, causal: bool = True, B: int = 1,
                        seg_tokens: int = 32768, scale: Optional[float] = None):
    """The attend callable of ``cp_dist.allgather_kv_attention`` for rank ``rank``: each of its local
    chunks (per sequence chunk rank and chunk 2N-1-rank, c = seq_len/2N rows each) attends over the
    sequence's keys in token order, in key segments of seg_tokens (ra_segmented_prefill_fwd), into
    the rank's output rows."""
    c = seq_len // (2 * n_ranks)

    def attend(q, k_nat, v_nat, o, lse):
        for b in range(B):
            for half, ch in enumerate((rank, 2 * n_ranks - 1 - rank)):
                rows = slice((b * 2 + half) * c, (b * 2 + half + 1) * c)
                tk = (ch + 1) * c if causal else seq_len      # keys after the chunk are never visible
                keys = slice(b * seq_len, b * seq_len + tk)
                segmented_prefill_fwd(q[rows], k_nat[keys], v_nat[keys], ch * c, seg_tokens, causal, scale,
                                      o=o[rows], lse=lse[rows])
    return attend


def lse_merge(o_parts, lse_parts, out_dtype=torch.float32, o=None, lse=None):
    """Merge partials o_parts [P, T, H, d] fp32 with lse_parts [P, T, H] -> (O [T, H, d], LSE [T, H]).
    O takes out_dtype, or the dtype of a given ``o``."""
    _need_cuda(o_parts, lse_parts, o, lse)
    P, T, H, d = o_parts.shape
    if o is None:
        o = torch.empty((T, H, d), dtype=out_dtype, device=o_parts.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=o_parts.device)
    _check(lib().ra_lse_merge(_ptr(o_parts), _ptr(lse_parts), P, T, H, d, _ptr(o),
                              RA_BF16 if o.dtype == torch.bfloat16 else RA_F32, _ptr(lse), _stream()))
    return o, lse


# ---------------------------------------------------------------------- KV cache

def cp_slot_mapping(query_start_loc, positions, block_table, block_size: int, interleave: int, pcp: int,
                    dcp: int, out=None):
    _need_cuda(query_start_loc, positions, block_table, out)
    R = query_start_loc.numel() - 1
    T = positions.numel()
    W = pcp * dcp
    if out is None:
        out = torch.empty((W, T), dtype=torch.int32, device=positions.device)
    _check(lib().ra_cp_slot_mapping(_ptr(query_start_loc), _ptr(positions), _ptr(block_table),
                                    block_table.shape[1], R, T, block_size, interleave, pcp, dcp, _ptr(out),
                                    _stream()))
    return out


def cp_kv_scatter(k, v, slot, k_cache, v_cache):
    _need_cuda(k, v, slot, k_cache, v_cache)
    W, NB, Hkv, bs, d = k_cache.shape
    _check(lib().ra_cp_kv_scatter(_ptr(k), _ptr(v), _ptr(slot), _ptr(k_cache), _ptr(v_cache), k.shape[0], W, Hkv,
                                  d, bs, NB, _dt(k), _stream()))


def cp_kv_gather(k_cache, v_cache, block_table, query_start_loc, positions, interleave: int, pcp: int, dcp: int,
                 k_out=None, v_out=None):
    """Token rows out of the sharded cache: row t = token positions[t] of its request -> (k [T, Hkv, d], v)."""
    _need_cuda(k_cache, v_cache, block_table, query_start_loc, positions, k_out, v_out)
    W, NB, Hkv, bs, d = k_cache.shape
    T = positions.numel()
    if k_out is None:
        k_out = torch.empty((T, Hkv, d), dtype=k_cache.dtype, device=k_cache.device)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    _check(lib().ra_cp_kv_gather(_ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
                                 _ptr(query_start_loc), _ptr(positions), query_start_loc.numel() - 1, T, Hkv, d, bs,
                                 interleave, pcp, dcp, NB, _dt(k_cache), _ptr(k_out), _ptr(v_out), _stream()))
    return k_out, v_out


def cp_decode_workspace_size(R, Hq, d, max_vblocks, pcp, dcp, split_blocks) -> int:
    n = _sz(0)
    _check(lib().ra_cp_decode_workspace_size(R, Hq, d, max_vblocks, pcp, dcp, split_blocks, _c.byref(n)))
    return n.value


def cp_decode(q, k_cache, v_cache, block_table, ctx_lens, interleave: int, pcp: int, dcp: int,
              split_blocks: int = 8, scale: Optional[float] = None, out_dtype=torch.bfloat16,
              workspace=None, o=None, lse=None):
    """Decode of one query token per request over the sharded cache -> (O [R, Hq, d], LSE [R, Hq])."""
    _need_cuda(q, k_cache, v_cache, block_table, ctx_lens, workspace, o, lse)
    R, Hq, d = q.shape
    W, NB, Hkv, bs, _ = k_cache.shape
    if W != pcp * dcp:
        raise ValueError("cache has %d devices, pcp*dcp = %d" % (W, pcp * dcp))
    max_vb = block_table.shape[1]
    need = cp_decode_workspace_size(R, Hq, d, max_vb, pcp, dcp, split_blocks)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty((R, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((R, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_cp_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), R, Hq, Hkv,
                              d, bs, interleave, pcp, dcp, max_vb, NB, float(scale or 0.0), split_blocks, _ptr(o),
                              RA_BF16 if o.dtype == torch.bfloat16 else RA_F32, _ptr(lse), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream()))
    return o, lse


def cp_decode_noalloc(q, k_cache, v_cache, block_table, ctx_lens, interleave: int, pcp: int, dcp: int,
                      split_blocks: int = 8, scale: Optional[float] = None, out_dtype=torch.bfloat16, o=None,
                      lse=None):
    """cp_decode without a workspace, for callers that cannot allocate device memory on the decode
    path: the partials live in a fixed 32 MiB scratch array inside the library (shared by all
    calls; calls that overlap on the GPU race).  Outputs o/lse may be passed in preallocated."""
    _need_cuda(q, k_cache, v_cache, block_table, ctx_lens, o, lse)
    R, Hq, d = q.shape
    W, NB, Hkv, bs, _ = k_cache.shape
    if o is None:
        o = torch.empty((R, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None:
        lse = torch.empty((R, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_cp_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), R,
                                      Hq, Hkv, d, bs, interleave, pcp, dcp, block_table.shape[1], NB,
                                      float(scale or 0.0), split_blocks, _ptr(o),
                                      RA_BF16 if o.dtype == torch.bfloat16 else RA_F32, _ptr(lse), _stream()))
    return o, lse


def cp_decode_partials(q, k_cache, v_cache, block_table, ctx_lens, interleave: int, pcp: int, dcp: int,
                       dev0: int = 0, split_blocks: int = 8, scale: Optional[float] = None, o_parts=None,
                       lse_parts=None):
    """Split-KV partials of the devices whose shards k_cache/v_cache [n_dev, NB, Hkv, bs, d] hold
    (devices dev0 .. dev0+n_dev-1 of pcp*dcp) -> (O_parts fp32 [P, R, Hq, d], LSE_parts [P, R, Hq]),
    partial p = (w - dev0) * n_splits + s.  A partial with LSE -inf has no token and unwritten O."""
    _need_cuda(q, k_cache, v_cache, block_table, ctx_lens, o_parts, lse_parts)
    R, Hq, d = q.shape
    n_dev, NB, Hkv, bs, _ = k_cache.shape
    max_vb = block_table.shape[1]
    P = _i32(0)
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(ctx_lens), R, Hq, Hkv, d, bs, interleave,
            pcp, dcp, dev0, n_dev, max_vb, NB, float(scale or 0.0), split_blocks)
    _check(lib().ra_cp_decode_partials(*args, None, None, _c.byref(P), _stream()))
    if o_parts is None:
        o_parts = torch.empty((P.value, R, Hq, d), dtype=torch.float32, device=q.device)
    if lse_parts is None:
        lse_parts = torch.empty((P.value, R, Hq), dtype=torch.float32, device=q.device)
    _check(lib().ra_cp_decode_partials(*args, _ptr(o_parts), _ptr(lse_parts), None, _stream()))
    return o_parts, lse_parts


def cp_lse_rescale(o_local, lse_all, w: int, o_scaled=None, lse_total=None):
    """Step 2 of cp_lse_ag_out_rs on device w: o_local fp32 [R, Hq, d], lse_all [W, R, Hq] ->
    (o_scaled [W, R, Hq/W, d], lse_total [R, Hq/W])."""
    _need_cuda(o_local, lse_all, o_scaled, lse_total)
    R, Hq, d = o_local.shape
    W = lse_all.shape[0]
    if o_scaled is None:
        o_scaled = torch.empty((W, R, Hq // W, d), dtype=torch.float32, device=o_local.device)
    if lse_total is None:
        lse_total = torch.empty((R, Hq // W), dtype=torch.float32, device=o_local.device)
    _check(lib().ra_cp_lse_rescale(_ptr(o_local), _ptr(lse_all), W, w, R, Hq, d, _ptr(o_scaled), _ptr(lse_total),
                                   _stream()))
    return o_scaled, lse_total


def cp_head_split(o_local, lse_local, W: int, o_split=None, lse_split=None):
    """All-to-all form of the decode merge: o_local fp32 [R, Hq, d], lse_local [R, Hq] ->
    (o_split [W, R, Hq/W, d], lse_split [W, R, Hq/W]) laid out by the device that keeps each head."""
    _need_cuda(o_local, lse_local, o_split, lse_split)
    R, Hq, d = o_local.shape
    if o_split is None:
        o_split = torch.empty((W, R, Hq // W, d), dtype=torch.float32, device=o_local.device)
    if lse_split is None:
        lse_split = torch.empty((W, R, Hq // W), dtype=torch.float32, device=o_local.device)
    _check(lib().ra_cp_head_split(_ptr(o_local), _ptr(lse_local), W, R, Hq, d, _ptr(o_split), _ptr(lse_split),
                                  _stream()))
    return o_split, lse_split


def cp_head_split_fn():
    """The split callable of ``cp_dist.cp_lse_a2a``, on ra_cp_head_split."""
    def split(o_local, lse_local, W, o_split, lse_split):
        cp_head_split(o_local, lse_local, W, o_split, lse_split)
    return split


def lse_merge_fn(out_dtype=torch.float32):
    """The merge callable of ``cp_dist.cp_lse_a2a``, on ra_lse_merge."""
    def merge(o_parts, lse_parts, o, lse):
        lse_merge(o_parts, lse_parts, out_dtype=out_dtype, o=o, lse=lse)
    return merge


def cp_lse_rescale_fn():
    """The rescale callable of ``cp_dist.cp_lse_ag_out_rs``, on ra_cp_lse_rescale."""
    def rescale(o_local, lse_all, w, o_scaled, lse_total):
        cp_lse_rescale(o_local, lse_all, w, o_scaled, lse_total)
    return rescale


def _need_paged(q, cache, block_table, query_start_loc, ctx_lens, pcp: int, dcp: int):
    """Checks of types and sizes shared by the operators on a packed batch of queries and the paged cache."""
    _of(torch.bfloat16, q, cache)
    _of(torch.int32, block_table, query_start_loc, ctx_lens)
    if q.dim() != 3 or cache.dim() != 5 or block_table.dim() != 2:
        raise ValueError("q must be [T, Hq, d], the cache [W, NB, Hkv, bs, d], block_table [R, max_vblocks]")
    T, Hq, d = q.shape
    W, NB, Hkv, bs, dk = cache.shape
    R, max_vb = block_table.shape
    if W != pcp * dcp:
        raise ValueError("cache has %d devices, pcp*dcp = %d" % (W, pcp * dcp))
    if dk != d:
        raise ValueError("q and the cache must have the same head dim")
    if query_start_loc.numel() != R + 1 or ctx_lens.numel() != R:
        raise ValueError("block_table has %d requests: query_start_loc needs R+1 entries, ctx_lens R" % R)
    return T, Hq, d, NB, Hkv, bs, R, max_vb


def cp_chunk_attn_workspace_size(Hq: int, Hkv: int, d: int) -> int:
    n = _sz(0)
    _check(lib().ra_cp_chunk_attn_workspace_size(Hq, Hkv, d, _c.byref(n)))
    return n.value


def cp_chunk_attn(q, k_cache, v_cache, block_table, query_start_loc, ctx_lens, interleave: int, pcp: int, dcp: int,
                  causal: bool = True, scale: Optional[float] = None, out_dtype=torch.bfloat16, workspace=None,
                  o=None, lse=None):
    """Attention of a packed batch of new tokens, q [T, Hq, d] (request r has rows query_start_loc[r] ..
    query_start_loc[r+1], the last ones of its ctx_lens[r] cached tokens), over the sharded paged cache
    -> (O [T, Hq, d], LSE [T, Hq]).  Rows of no request are left as they were (undefined in a new O).  The
    probabilities are rounded to bf16 for the product with V, for out_dtype float32 too."""
    dev = _here(q, k_cache, v_cache, block_table, query_start_loc, ctx_lens, workspace, o, lse)
    T, Hq, d, NB, Hkv, bs, R, max_vb = _need_paged(q, k_cache, block_table, query_start_loc, ctx_lens, pcp, dcp)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("v_cache must be like k_cache")
    if workspace is None:
        workspace = torch.empty(cp_chunk_attn_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device=q.device)
    if o is None:
        o = torch.empty((T, Hq, d), dtype=out_dtype, device=q.device)
    elif o.shape != q.shape:
        raise ValueError("o must be [T, Hq, d]")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    elif lse.shape != (T, Hq) or lse.dtype != torch.float32:
        raise ValueError("lse must be float32 [T, Hq]")
    _check(lib().ra_cp_chunk_attn(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                  query_start_loc.data_ptr(), ctx_lens.data_ptr(), T, R, Hq, Hkv, d, bs, interleave,
                                  pcp, dcp, max_vb, NB, 1 if causal else 0, scale or 0.0, o.data_ptr(), _dt(o),
                                  lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  torch._C._cuda_getCurrentRawStream(dev)))
    return o, lse


def cp_attn_weights(q, lse, k_cache, block_table, query_start_loc, ctx_lens, interleave: int, pcp: int, dcp: int,
                    w_in=None, w_out=None, causal: bool = True, scale: Optional[float] = None):
    """Accumulated attention weight of every cached token, per K/V head -> w_out fp32 [W, NB, Hkv, bs]: w_in
    (None: 0; the chunk's own tokens start from 0) plus the softmax weights of the queries q [T, Hq, d] with
    their lse [T, Hq] (a query of lse -inf adds nothing).  w_out may be w_in; slots of no token are left as they
    were (0 in a new w_out).  A block that several requests share gets the value of one of them."""
    dev = _here(q, lse, k_cache, block_table, query_start_loc, ctx_lens, w_in, w_out)
    T, Hq, d, NB, Hkv, bs, R, max_vb = _need_paged(q, k_cache, block_table, query_start_loc, ctx_lens, pcp, dcp)
    _of(torch.float32, lse, w_in, w_out)
    shape = k_cache.shape[:4]
    if w_out is None:
        w_out = torch.zeros(shape, dtype=torch.float32, device=q.device)
    if lse.shape != (T, Hq):
        raise ValueError("lse must be [T, Hq]")
    if w_out.shape != shape or (w_in is not None and w_in.shape != shape):
        raise ValueError("the weights must be [W, NB, Hkv, bs]")
    _check(lib().ra_cp_attn_weights(q.data_ptr(), lse.data_ptr(), k_cache.data_ptr(), block_table.data_ptr(),
                                    query_start_loc.data_ptr(), ctx_lens.data_ptr(), T, R, Hq, Hkv, d, bs, interleave,
                                    pcp, dcp, max_vb, NB, 1 if causal else 0, scale or 0.0, _ptr(w_in),
                                    w_out.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)))
    return w_out


def cp_evict(k_cache, v_cache, weights, block_table, ctx_lens, keep: int, interleave: int, pcp: int, dcp: int,
             n_sink: int = 0, n_recent: int = 0, dst_block_table=None, kept=None, new_lens=None):
    """Cut every request's cached context to ``keep`` tokens per K/V head (the first n_sink, the last n_recent
    and the heaviest of the others by ``weights`` fp32 [W, NB, Hkv, bs]) and pack them in order, with their
    weights, into the blocks of dst_block_table [R, .] (None: the request's own blocks; else none of the blocks
    that hold a context), no block being two requests'.  Returns (kept int32
    [R, Hkv, keep]: former positions, -1 past the end; new_lens int32 [R])."""
    dev = _here(k_cache, v_cache, weights, block_table, ctx_lens, dst_block_table, kept, new_lens)
    _of(torch.float32, weights)
    _of(torch.int32, block_table, ctx_lens, dst_block_table, kept, new_lens)
    if k_cache.dim() != 5 or block_table.dim() != 2:
        raise ValueError("the cache must be [W, NB, Hkv, bs, d], block_table [R, max_vblocks]")
    shape = k_cache.shape
    W, NB, Hkv, bs, d = shape
    R, max_vb = block_table.shape
    if W != pcp * dcp:
        raise ValueError("cache has %d devices, pcp*dcp = %d" % (W, pcp * dcp))
    if v_cache.shape != shape or v_cache.dtype != k_cache.dtype or weights.shape != shape[:4]:
        raise ValueError("v_cache must be like k_cache, weights [W, NB, Hkv, bs]")
    dst_vb = 0
    if dst_block_table is not None:
        if dst_block_table.dim() != 2 or dst_block_table.shape[0] != R:
            raise ValueError("dst_block_table must be [R, dst_max_vblocks]")
        dst_vb = dst_block_table.shape[1]
    if ctx_lens.numel() != R:
        raise ValueError("ctx_lens must have one entry per request")
    if kept is None:
        kept = torch.empty((R, Hkv, max(keep, 0)), dtype=torch.int32, device=k_cache.device)
    elif kept.numel() != R * Hkv * keep:
        raise ValueError("kept must be [R, Hkv, keep]")
    if new_lens is None:
        new_lens = torch.empty(R, dtype=torch.int32, device=k_cache.device)
    elif new_lens.numel() != R:
        raise ValueError("new_lens must be [R]")
    _check(lib().ra_cp_evict(k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(), block_table.data_ptr(),
                             _ptr(dst_block_table), ctx_lens.data_ptr(), R, Hkv, d, _dt(k_cache), bs, interleave, pcp,
                             dcp, max_vb, dst_vb, NB, keep, n_sink, n_recent, kept.data_ptr(), new_lens.data_ptr(),
                             torch._C._cuda_getCurrentRawStream(dev)))
    return kept, new_lens


def cp_rope_append(k, v, k_cache, v_cache, block_table, query_start_loc, ctx_lens, interleave: int, pcp: int, dcp: int,
                   positions=None, inv_freq=None, axis=None, mscale: float = 1.0, style: str = "half", q=None,
                   q_out=None):
    """New tokens into the sharded paged cache: k and v [T, Hkv, d] (any strides with the last one 1; request r's
    are rows query_start_loc[r] .. query_start_loc[r+1], the last ones of its ctx_lens[r] tokens), k turned by its
    rotary positions.  q [T, Hq, d] is turned beside them into q_out (new if not given; may be q) and returned.
    positions int32 [T], or [axes, T] with axis int32 [rot/2] on the host; None: the token's place in its context.
    inv_freq float64 [rot/2] on the host; None: nothing is turned."""
    W, NB, Hkv, bs, d = shape = k_cache.shape
    R, max_vb = block_table.shape
    T, heads, dk = k.shape
    dt, dev, i32 = k_cache.dtype, k_cache.get_device(), torch.int32
    krs, khs, kes = k.stride()
    vrs, vhs, ves = v.stride()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and v_cache.get_device() == dev
            and block_table.get_device() == dev and query_start_loc.get_device() == dev and ctx_lens.get_device() == dev
            and k.get_device() == dev and v.get_device() == dev):
        raise ValueError("tensors must be on the current CUDA device")
    if not (W == pcp * dcp and v_cache.shape == shape and v_cache.dtype == dt and k_cache.is_contiguous()
            and v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be alike, contiguous [pcp*dcp, NB, Hkv, bs, d]")
    if not (query_start_loc.numel() == R + 1 and ctx_lens.numel() == R and block_table.dtype == i32
            and query_start_loc.dtype == i32 and ctx_lens.dtype == i32 and block_table.is_contiguous()
            and query_start_loc.is_contiguous() and ctx_lens.is_contiguous()):
        raise ValueError("block_table [R, max_vblocks], query_start_loc [R+1] and ctx_lens [R] must be contiguous int32")
    if not (heads == Hkv and dk == d and v.shape == k.shape and k.dtype == dt and v.dtype == dt
            and ((kes == 1 and ves == 1) or d == 1)):
        raise ValueError("k and v must be [T, Hkv, d] of the caches' heads and dtype, the elements of a head contiguous")
    n_axes, half, at = 1, 0, None
    if inv_freq is not None:
        half = inv_freq.numel()
        if not (inv_freq.dtype == torch.float64 and inv_freq.dim() == 1 and inv_freq.get_device() < 0
                and inv_freq.is_contiguous()):
            raise ValueError("inv_freq must be a contiguous float64 vector on the host")
        if axis is not None and not (axis.dtype == i32 and axis.shape == (half,) and axis.get_device() < 0
                                     and axis.is_contiguous() and positions is not None):
            raise ValueError("axis must be a contiguous int32 vector on the host as long as inv_freq, with positions")
    if positions is not None:
        at = positions.data_ptr()
        n_axes = positions.shape[0] if axis is not None else 1
        if not (positions.dtype == i32 and positions.get_device() == dev and positions.is_contiguous()
                and positions.shape == ((n_axes, T) if axis is not None else (T,))):
            raise ValueError("positions must be contiguous int32 [T], or [axes, T] with axis")
    qp, op, Hq, qrs, qhs, ors, ohs = None, None, 0, 0, 0, 0, 0
    if q is not None:
        _, Hq, _ = q.shape
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dt, device=q.device)
        qrs, qhs, qes = q.stride()
        ors, ohs, oes = q_out.stride()
        if not (q.shape == (T, Hq, d) and q_out.shape == q.shape and q.dtype == dt and q_out.dtype == dt
                and q.get_device() == dev and q_out.get_device() == dev and ((qes == 1 and oes == 1) or d == 1)):
            raise ValueError("q and q_out must be alike, [T, Hq, d] of the caches' dtype, the elements of a head contiguous")
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    st = _LIB.ra_cp_rope_append(k.data_ptr(), krs, khs, v.data_ptr(), vrs, vhs, qp, qrs, qhs, op, ors, ohs,
                                k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), query_start_loc.data_ptr(),
                                ctx_lens.data_ptr(), T, R, Hq, Hkv, d, _dt(k_cache), bs, interleave, pcp, dcp, max_vb, NB,
                                at, n_axes, 2 * half, ROPE_STYLES[style], None if inv_freq is None else inv_freq.data_ptr(),
                                None if axis is None else axis.data_ptr(), mscale, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _check(st)
    return q_out


def _reach(tokens: int) -> int:
    """A window or a number of first tokens for the library, whose integers have 32 bits: no sequence is as long."""
    return max(-1, min(tokens, 2 ** 31 - 1))


def _out_rows(o, lse, T: int, Hq: int, d: int, out_dtype, device):
    if o is None:
        o = torch.empty((T, Hq, d), dtype=out_dtype, device=device)
    elif o.shape != (T, Hq, d):
        raise ValueError("o must be [T, Hq, d]")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=device)
    elif lse.shape != (T, Hq) or lse.dtype != torch.float32:
        raise ValueError("lse must be float32 [T, Hq]")
    return o, lse


def cp_window_attn_workspace_size(Hq: int, Hkv: int, d: int) -> int:
    n = _sz(0)
    _check(lib().ra_cp_window_attn_workspace_size(Hq, Hkv, d, _c.byref(n)))
    return n.value


def cp_window_attn(q, k_cache, v_cache, block_table, query_start_loc, ctx_lens, window: int, interleave: int, pcp: int,
                   dcp: int, n_sink: int = 0, scale: Optional[float] = None, out_dtype=torch.bfloat16, workspace=None,
                   o=None, lse=None):
    """``cp_chunk_attn`` with a sliding window: the query at position p sees the tokens x <= p with x > p - window or
    x < n_sink -> (O [T, Hq, d], LSE [T, Hq]).  Blocks that no query of the request sees are not looked at (their
    entries in block_table may hold anything)."""
    dev = _here(q, k_cache, v_cache, block_table, query_start_loc, ctx_lens, workspace, o, lse)
    T, Hq, d, NB, Hkv, bs, R, max_vb = _need_paged(q, k_cache, block_table, query_start_loc, ctx_lens, pcp, dcp)
    if v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("v_cache must be like k_cache")
    if workspace is None:
        workspace = torch.empty(cp_window_attn_workspace_size(Hq, Hkv, d), dtype=torch.uint8, device=q.device)
    o, lse = _out_rows(o, lse, T, Hq, d, out_dtype, q.device)
    _check(lib().ra_cp_window_attn(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                   query_start_loc.data_ptr(), ctx_lens.data_ptr(), T, R, Hq, Hkv, d, bs, interleave, pcp,
                                   dcp, max_vb, NB, _reach(window), _reach(n_sink), scale or 0.0, o.data_ptr(), _dt(o),
                                   lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   torch._C._cuda_getCurrentRawStream(dev)))
    return o, lse


def window_attn_workspace_size(T: int, R: int, Hq: int, Hkv: int, d: int) -> int:
    n = _sz(0)
    _check(lib().ra_window_attn_workspace_size(T, R, Hq, Hkv, d, _c.byref(n)))
    return n.value


def _packed_rows(x, what, dev, dtype, shape=None):
    """Row stride of [rows, heads, d] whose rows are dense."""
    rs, hs = _heads_of(x, what, dev, dtype)
    if shape is not None and x.shape != shape:
        raise ValueError("%s must be %s" % (what, tuple(shape)))
    if hs != x.shape[2] and x.shape[1] > 1:
        raise ValueError("the heads of a row of %s must be contiguous" % what)
    # a single row's stride is of no account
    return rs if x.shape[0] > 1 else x.shape[1] * x.shape[2]


def _need_packed(q, k, v, query_start_loc, workspace, *others):
    dev = _here(query_start_loc, workspace, *others)
    _of(torch.int32, query_start_loc)
    bf = torch.bfloat16
    qrs = _packed_rows(q, "q", dev, bf)
    T, Hq, d = q.shape
    krs, vrs = _packed_rows(k, "k", dev, bf), _packed_rows(v, "v", dev, bf, k.shape)
    if k.shape[0] != T or k.shape[2] != d:
        raise ValueError("k and v must be [T, Hkv, d] with q's tokens and head dim")
    R, Hkv = query_start_loc.numel() - 1, k.shape[1]
    if workspace is None:
        workspace = torch.empty(window_attn_workspace_size(T, R, Hq, Hkv, d), dtype=torch.uint8, device=q.device)
    return dev, qrs, krs, vrs, T, R, Hq, Hkv, d, workspace


def window_attn_fwd(q, k, v, query_start_loc, window: int, n_sink: int = 0, scale: Optional[float] = None,
                    out_dtype=torch.bfloat16, workspace=None, o=None, lse=None):
    """Causal attention of packed sequences (rows query_start_loc[r] .. query_start_loc[r+1] of q [T, Hq, d] and
    k, v [T, Hkv, d] bf16, rows any multiple of 8 elements apart) with a sliding window: position p sees x <= p with
    x > p - window or x < n_sink -> (O [T, Hq, d], LSE [T, Hq]).  Rows of no sequence are left as they were."""
    dev, qrs, krs, vrs, T, R, Hq, Hkv, d, workspace = _need_packed(q, k, v, query_start_loc, workspace, o, lse)
    o, lse = _out_rows(o, lse, T, Hq, d, out_dtype, q.device)
    _check(lib().ra_window_attn_fwd(q.data_ptr(), qrs, k.data_ptr(), krs, v.data_ptr(), vrs, query_start_loc.data_ptr(), T,
                                    R, Hq, Hkv, d, _reach(window), _reach(n_sink), scale or 0.0, o.data_ptr(), _dt(o),
                                    lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    torch._C._cuda_getCurrentRawStream(dev)))
    return o, lse


def window_attn_bwd(do, q, k, v, o, lse, query_start_loc, window: int, n_sink: int = 0, scale: Optional[float] = None,
                    out_dtype=torch.bfloat16, workspace=None, dq=None, dk=None, dv=None):
    """Gradient of ``window_attn_fwd``: do, o [T, Hq, d] bf16 and lse [T, Hq] (what it gave) -> (dQ [T, Hq, d],
    dK, dV [T, Hkv, d]) in out_dtype, or in the dtype of given outputs, whose rows may be any multiple of 16 bytes
    apart (parts of the gradient of a fused projection)."""
    dev, qrs, krs, vrs, T, R, Hq, Hkv, d, workspace = _need_packed(q, k, v, query_start_loc, workspace, do, o, lse)
    _of(torch.bfloat16, do, o)
    _of(torch.float32, lse)
    if do.shape != q.shape or o.shape != q.shape or lse.shape != (T, Hq):
        raise ValueError("do and o must be [T, Hq, d], lse [T, Hq]")
    given = [x for x in (dq, dk, dv) if x is not None]
    dt = given[0].dtype if given else out_dtype
    new = lambda x: torch.empty(x.shape, dtype=dt, device=q.device)
    dq, dk, dv = (new(x) if g is None else g for x, g in ((q, dq), (k, dk), (v, dv)))
    rs = [_packed_rows(g, what, dev, dt, x.shape) for g, what, x in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v))]
    _check(lib().ra_window_attn_bwd(q.data_ptr(), qrs, k.data_ptr(), krs, v.data_ptr(), vrs, o.data_ptr(), lse.data_ptr(),
                                    do.data_ptr(), query_start_loc.data_ptr(), T, R, Hq, Hkv, d, _reach(window),
                                    _reach(n_sink), scale or 0.0, dq.data_ptr(), rs[0], dk.data_ptr(), rs[1], dv.data_ptr(), rs[2],
                                    _dt(dq), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    torch._C._cuda_getCurrentRawStream(dev)))
    return dq, dk, dv


# ---------------------------------------------------------------------- misc

def selftest_wait_timeout(limit_cycles: int):
    _check(lib().ra_selftest_wait_timeout(int(limit_cycles), _stream()))


_TABLES = {}


def synth_fill(key: int, table_cpu: torch.Tensor, shape, device="cuda"):
    """Device tensor of the counter-based draw (see inputs.py) with the given key and value table."""
    dev = torch.device(device)
    tk = (table_cpu.dtype, dev)
    if tk not in _TABLES:
        _TABLES[tk] = table_cpu.to(dev)
    table = _TABLES[tk]
    out = torch.empty(tuple(shape), dtype=table_cpu.dtype, device=dev)
    _check(lib().ra_synth_fill(_u64(key), out.numel(), _ptr(table), table.element_size(), _ptr(out), _stream()))
    return out
