"""Python entry points with the names of the C interface (``include/dsa.h``).

Marshalling only: each function checks the tensors' device, dtype and shape,
passes their device pointers and torch's current CUDA stream to the C library
and returns.  Every step of the hot path runs in the library's CUDA kernels;
nothing here computes on the host or falls back to torch operations.
"""
from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import _lib

D_K, D_V = 576, 512


@dataclass
class Dims:
    B: int
    Nq: int
    H_I: int
    d_I: int
    H: int
    k: int
    T_max: int
    idx_dtype: int
    kv_dtype: int
    ld_scores: int

    def c(self) -> _lib.DsaDims:
        return _lib.DsaDims(self.B, self.Nq, self.H_I, self.d_I, self.H, self.k, self.T_max, self.idx_dtype,
                            self.kv_dtype, 0, self.ld_scores)


def dims_of(inp, ld_scores: Optional[int] = None, Nq: Optional[int] = None) -> Dims:
    """Dims for an ``inputs.DSAInputs`` workload (ld_scores defaults to T_max rounded up to 4)."""
    ld = ld_scores if ld_scores is not None else (inp.T_max + 3) // 4 * 4
    return Dims(inp.B, inp.Nq if Nq is None else Nq, inp.H_I, inp.d_I, inp.H, inp.k, inp.T_max, inp.idx_dtype,
                inp.kv_dtype, ld)


def _stream_ptr(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def workspace_size(dims: Dims, op: int) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    d = dims.c()
    _lib.check(lib, lib.dsa_workspace_size(ctypes.byref(d), op, ctypes.byref(n)), "dsa_workspace_size")
    return int(n.value)


def make_workspace(dims: Dims, op: int, device=None) -> torch.Tensor:
    """A zero-initialised uint8 device buffer sized for `op` (torch allocates; the library never does)."""
    lib = _lib.load()
    nbytes = workspace_size(dims, op)
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device or "cuda")
    _lib.check(lib, lib.dsa_workspace_init(ws.data_ptr(), ws.numel(), _stream_ptr()), "dsa_workspace_init")
    return ws


def get_device_status(ws: torch.Tensor) -> int:
    lib = _lib.load()
    v = ctypes.c_int32(0)
    _lib.check(lib, lib.dsa_get_device_status(ws.data_ptr(), _stream_ptr(), ctypes.byref(v)), "dsa_get_device_status")
    return int(v.value)


def status_string(code: int) -> str:
    return _lib.load().dsa_status_string(code).decode()


def indexer_scores(dims: Dims, q_I, q_scale, w, k_I, k_scale, q_seq, q_len, scores, ws=None):
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_indexer_scores(ctypes.byref(d), _ptr(q_I), _ptr(q_scale), _ptr(w), _ptr(k_I), _ptr(k_scale),
                                _ptr(q_seq), _ptr(q_len), _ptr(scores), _ptr(ws),
                                0 if ws is None else ws.numel(), _stream_ptr())
    _lib.check(lib, rc, "dsa_indexer_scores")
    return scores


def prefill_indexer_scores(dims: Dims, q_I, q_scale, w, k_I, k_scale, q_seq, q_len, scores, ws=None):
    """Indexer scores for rows of one prompt: four consecutive rows per tensor-core pass."""
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_prefill_indexer_scores(ctypes.byref(d), _ptr(q_I), _ptr(q_scale), _ptr(w), _ptr(k_I), _ptr(k_scale),
                                        _ptr(q_seq), _ptr(q_len), _ptr(scores), _ptr(ws),
                                        0 if ws is None else ws.numel(), _stream_ptr())
    _lib.check(lib, rc, "dsa_prefill_indexer_scores")
    return scores


def topk(dims: Dims, scores, q_len, idx, ws=None):
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_topk(ctypes.byref(d), _ptr(scores), _ptr(q_len), _ptr(idx), _ptr(ws),
                      0 if ws is None else ws.numel(), _stream_ptr())
    _lib.check(lib, rc, "dsa_topk")
    return idx


def dense_mla_attn(dims: Dims, q, kv, q_seq, q_len, softmax_scale, out, lse, ws):
    """Attention over every position s < q_len[t] (the dense comparison of the sparse path)."""
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_dense_mla_attn(ctypes.byref(d), _ptr(q), _ptr(kv), _ptr(q_seq), _ptr(q_len),
                                ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                _stream_ptr())
    _lib.check(lib, rc, "dsa_dense_mla_attn")
    return out


def sparse_mla_attn(dims: Dims, q, kv, idx, q_seq, q_len, softmax_scale, out, lse, ws):
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_sparse_mla_attn(ctypes.byref(d), _ptr(q), _ptr(kv), _ptr(idx), _ptr(q_seq), _ptr(q_len),
                                 ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                 _stream_ptr())
    _lib.check(lib, rc, "dsa_sparse_mla_attn")
    return out, lse


@dataclass
class PagedCache:
    """Block pools and block table of a paged cache (device tensors)."""
    k_I: Optional[torch.Tensor]      # [num_blocks, block_size, d_I] e4m3 (uint8); None for chunk_attn_paged alone
    k_scale: Optional[torch.Tensor]  # [num_blocks, block_size] fp32; None for chunk_attn_paged alone
    kv: torch.Tensor           # [num_blocks, block_size, 576] bf16 or [.., 656] FP8 entries (uint8)
    block_table: torch.Tensor  # [B, max_blocks] int32
    block_size: int

    def c(self) -> _lib.DsaPagedCache:
        return _lib.DsaPagedCache(_ptr(self.k_I), _ptr(self.k_scale), _ptr(self.kv), _ptr(self.block_table),
                                  self.block_size, self.kv.shape[0], self.block_table.shape[1], 0)


def append_tokens(dims: Dims, seq, pos, kv_new, k_new, kv=None, k_I=None, k_scale=None,
                  cache: Optional["PagedCache"] = None, ws=None):
    """Write new tokens (bf16 latent rows, fp32 indexer keys) into the caches, quantising as
    the caches' types require; contiguous caches (kv, k_I, k_scale) or a paged cache."""
    lib = _lib.load()
    d = dims.c()
    pc = cache.c() if cache is not None else None
    rc = lib.dsa_append_tokens(ctypes.byref(d), int(seq.numel()), _ptr(seq), _ptr(pos), _ptr(kv_new), _ptr(k_new),
                               _ptr(kv), _ptr(k_I), _ptr(k_scale), ctypes.byref(pc) if pc is not None else None,
                               _ptr(ws), 0 if ws is None else ws.numel(), _stream_ptr())
    _lib.check(lib, rc, "dsa_append_tokens")


@dataclass
class Rope:
    """Position rotation: 32 frequencies (radians a position, fp32, on the device) and the pair layouts
    (``_lib.DSA_ROPE_*``) of the latent rows' 64 rope values and of the indexer's first 64 values."""
    inv_freq: torch.Tensor
    latent: int = _lib.DSA_ROPE_INTERLEAVED
    index: int = _lib.DSA_ROPE_HALVES


def _refuse(t: torch.Tensor, name: str, dtypes: tuple, numel: int, dev: Optional[int]) -> None:
    """The error of a tensor argument that failed a check (the order of the checks is theirs)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.get_device() != (torch.cuda.current_device() if dev is None else dev):
        raise ValueError(f"{name} lives on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    raise ValueError(f"{name} must be contiguous")


def _first(t: torch.Tensor, name: str, dtypes: tuple, numel: int) -> int:
    """A call's first tensor: on the current device, whose index the other checks use."""
    try:
        dev = t.get_device()
        if t.dtype not in dtypes or t.numel() != numel or dev < 0 or dev != _current_device():
            _refuse(t, name, dtypes, numel, None)
        return dev
    except AttributeError:  # (no tensor; the try costs the others nothing)
        _refuse(t, name, dtypes, numel, None)


def _dense(t: torch.Tensor, name: str, dtypes: tuple, numel: int, dev: int) -> int:
    """Device pointer of a contiguous tensor argument of one of `dtypes` with `numel` elements."""
    try:
        if t.dtype not in dtypes or t.numel() != numel or t.get_device() != dev or not t.is_contiguous():
            _refuse(t, name, dtypes, numel, dev)
        return t.data_ptr()
    except AttributeError:
        _refuse(t, name, dtypes, numel, dev)


def _strided(t: torch.Tensor, name: str, dtypes: tuple, numel: int, dev: int) -> int:
    """The same for a tensor whose strides are passed on."""
    try:
        if t.dtype not in dtypes or t.numel() != numel or t.get_device() != dev:
            _refuse(t, name, dtypes, numel, dev)
        return t.data_ptr()
    except AttributeError:
        _refuse(t, name, dtypes, numel, dev)


def _workspace(ws: torch.Tensor, dev: int) -> tuple:
    """Device pointer and bytes of a workspace."""
    n = ws.numel() if isinstance(ws, torch.Tensor) else 0
    return _dense(ws, "ws", _U8, n, dev), n


# The C structures as bytes: a third of the time of a ctypes structure.
_pack_dims = struct.Struct("10iq").pack
_pack_cache = struct.Struct("4P4i").pack
_pack_rope = struct.Struct("P2i").pack


def _dims_arg(d: Dims) -> bytes:
    return _pack_dims(d.B, d.Nq, d.H_I, d.d_I, d.H, d.k, d.T_max, d.idx_dtype, d.kv_dtype, 0, d.ld_scores)


def _pools(d: Dims, kv, k_I, k_scale, tokens: int, dev: int, index: bool) -> tuple:
    """Device pointers (0: not used) of caches with room for `tokens`, of the types that dims names."""
    if d.kv_dtype == _lib.DSA_FP8_E4M3:
        p_kv = _dense(kv, "the latent cache kv", _U8, tokens * 656, dev)
    else:
        p_kv = _dense(kv, "the latent cache kv", _BF16, tokens * D_K, dev)
    if not index:
        return p_kv, 0, 0
    if d.idx_dtype == _lib.DSA_F32:
        return p_kv, _dense(k_I, "the key cache k_I", _F32, tokens * d.d_I, dev), 0
    return (p_kv, _dense(k_I, "the key cache k_I", _CODES, tokens * d.d_I, dev),
            _dense(k_scale, "the key cache k_scale", _F32, tokens, dev))


def _cache_arg(d: Dims, c: PagedCache, dev: int, index: bool) -> bytes:
    """The paged cache of a call that uses its latent pool, its block table and (index) its key pool."""
    try:
        table, kv, block = c.block_table, c.kv, c.block_size
        blocks, width = kv.size(0), table.size(1)
    except (AttributeError, IndexError):
        raise ValueError("cache: expected a PagedCache with a latent pool and a [B, max_blocks] block table") from None
    p_kv, p_k, p_s = _pools(d, kv, c.k_I, c.k_scale, blocks * block, dev, index)
    return _pack_cache(p_k, p_s, p_kv, _dense(table, "the block table", _I32, d.B * width, dev), block, blocks, width, 0)


def _rope_arg(r: Rope, dev: int) -> bytes:
    try:
        freq, latent, index = r.inv_freq, r.latent, r.index
    except AttributeError:
        raise ValueError(f"rope: expected a Rope, got {type(r).__name__}") from None
    return _pack_rope(_dense(freq, "inv_freq", _F32, 32, dev), latent, index)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_I32, _F32, _BF16, _U8 = (torch.int32,), (torch.float32,), (torch.bfloat16,), (torch.uint8,)
_CODES = (torch.uint8, torch.float8_e4m3fn)
_RAW = (torch.float32, torch.bfloat16)
_ROW_DTYPES = {torch.float32: _lib.DSA_F32, torch.bfloat16: _lib.DSA_BF16}


def _row_stride(t: torch.Tensor, name: str, shape: tuple) -> int:
    """Row stride (elements) of a tensor of `shape` whose rows hold contiguous values."""
    stride = t.stride()
    if tuple(t.shape) != shape or stride[-1] != 1 or (len(shape) == 3 and shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name}: expected {list(shape)} with contiguous rows, got {list(t.shape)} with strides {stride}")
    return stride[0] if shape[0] > 1 else math.prod(shape[1:])


def append_tokens_rope(dims: Dims, seq, pos, kv_new, k_new, rope: Rope, kv=None, k_I=None, k_scale=None,
                       cache: Optional["PagedCache"] = None, ws=None):
    """Write new tokens into the caches from the raw projections, rotated to `pos` on the way: kv_new
    [n, 576] bf16 and k_new [n, d_I] fp32 or bf16, each with any row stride (a multiple of 16 bytes)."""
    lib = _lib.load()
    n = seq.numel() if isinstance(seq, torch.Tensor) else 0
    dev = _first(seq, "seq", _I32, n)
    p_pos = _dense(pos, "pos", _I32, n, dev)
    p_kv = _strided(kv_new, "kv_new", _BF16, n * D_K, dev)
    p_k = _strided(k_new, "k_new", _RAW, n * dims.d_I, dev)
    if n == 0:
        return
    kv_stride = _row_stride(kv_new, "kv_new", (n, D_K))
    k_stride = _row_stride(k_new, "k_new", (n, dims.d_I))
    if not seq.is_contiguous():
        raise ValueError("seq must be contiguous")
    paged = p_ckv = p_cki = p_cks = None
    if cache is not None:
        paged = _cache_arg(dims, cache, dev, True)
    else:
        p_ckv, p_cki, p_cks = _pools(dims, kv, k_I, k_scale, dims.B * dims.T_max, dev, True)
    rc = lib.dsa_append_tokens_rope(_dims_arg(dims), n, seq.data_ptr(), p_pos, p_kv, kv_stride, p_k, k_stride,
                                    _ROW_DTYPES[k_new.dtype], _rope_arg(rope, dev), p_ckv, p_cki, p_cks, paged,
                                    *((None, 0) if ws is None else _workspace(ws, dev)), _raw_stream(dev))
    if rc:
        _lib.check(lib, rc, "dsa_append_tokens_rope")


def rope_queries(dims: Dims, pos, rope: Rope, q=None, q_pe=None, q_nope=None, qi_new=None, q_I=None, q_scale=None):
    """The raw queries of dims.Nq rows at positions `pos`: q_pe [Nq, H, 64] (strided) rotated into
    q[..., 512:576] (and q_nope [Nq, H, 512] copied into q[..., :512] when given); qi_new [Nq, H_I, d_I]
    fp32 or bf16 rotated and quantised into q_I and q_scale.  Either half may be left out."""
    lib = _lib.load()
    n, H = dims.Nq, dims.H
    dev = _first(pos, "pos", _I32, n)
    p_q = p_pe = p_nope = p_new = p_qi = p_scale = None
    pe_row = pe_head = qi_row = qi_dtype = 0
    if q_pe is not None:
        p_pe = _strided(q_pe, "q_pe", _BF16, n * H * 64, dev)
        p_q = _dense(q, "q", _BF16, n * H * D_K, dev)
        if q_nope is not None:
            p_nope = _dense(q_nope, "q_nope", _BF16, n * H * D_V, dev)
        if tuple(q_pe.shape) != (n, H, 64) or q_pe.stride(2) != 1:
            raise ValueError(f"q_pe: expected [{n}, {H}, 64] with contiguous values, got {list(q_pe.shape)}")
        pe_head = q_pe.stride(1) if H > 1 else 64
        pe_row = q_pe.stride(0) if n > 1 else H * pe_head
    if qi_new is not None:
        numel = n * dims.H_I * dims.d_I
        p_new = _strided(qi_new, "qi_new", _RAW, numel, dev)
        if dims.idx_dtype == _lib.DSA_F32:
            p_qi = _dense(q_I, "q_I", _F32, numel, dev)
        else:
            p_qi = _dense(q_I, "q_I", _CODES, numel, dev)
            p_scale = _dense(q_scale, "q_scale", _F32, n * dims.H_I, dev)
        qi_row = _row_stride(qi_new, "qi_new", (n, dims.H_I, dims.d_I))
        qi_dtype = _ROW_DTYPES[qi_new.dtype]
    rc = lib.dsa_rope_queries(_dims_arg(dims), _dense(pos, "pos", _I32, n, dev), _rope_arg(rope, dev), p_nope, p_pe, pe_row, pe_head, p_q, p_new,
                              qi_row, qi_dtype, p_qi, p_scale, _raw_stream(dev))
    if rc:
        _lib.check(lib, rc, "dsa_rope_queries")
    return q, q_I, q_scale


def chunk_attn_paged(dims: Dims, q, cache: PagedCache, q_seq, q_len, softmax_scale, out, lse, ws):
    """Attention of a chunk of new tokens over every cached position s < q_len[t] of their sequences,
    read through the block table (ws sized for ``_lib.DSA_OP_CHUNK_ATTN``)."""
    lib = _lib.load()
    n, H = dims.Nq, dims.H
    dev = _first(q, "q", _BF16, n * H * D_K)
    rc = lib.dsa_chunk_attn_paged(_dims_arg(dims), _dense(q, "q", _BF16, n * H * D_K, dev),
                                  _cache_arg(dims, cache, dev, False), _dense(q_seq, "q_seq", _I32, n, dev),
                                  _dense(q_len, "q_len", _I32, n, dev), softmax_scale,
                                  _dense(out, "out", _BF16, n * H * D_V, dev),
                                  None if lse is None else _dense(lse, "lse", _F32, n * H, dev),
                                  *_workspace(ws, dev), _raw_stream(dev))
    if rc:
        _lib.check(lib, rc, "dsa_chunk_attn_paged")
    return out, lse


def decode_step_paged(dims: Dims, q_I, q_scale, w, cache: PagedCache, q, q_seq, q_len, softmax_scale, out, lse, ws,
                      scores_out=None, idx_out=None):
    """One decode step over a paged cache on torch's current stream."""
    lib = _lib.load()
    d = dims.c()
    pc = cache.c()
    rc = lib.dsa_decode_step_paged(ctypes.byref(d), _ptr(q_I), _ptr(q_scale), _ptr(w), ctypes.byref(pc), _ptr(q),
                                   _ptr(q_seq), _ptr(q_len), ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse),
                                   _ptr(scores_out), _ptr(idx_out), _ptr(ws), ws.numel(), _stream_ptr(), None)
    _lib.check(lib, rc, "dsa_decode_step_paged")
    return out, lse


def decode_step(dims: Dims, q_I, q_scale, w, k_I, k_scale, q, kv, q_seq, q_len, softmax_scale, out, lse, ws,
                scores_out=None, idx_out=None, events: Optional[Sequence] = None):
    """One decode step (indexer -> top-k -> sparse MLA) on torch's current stream.

    events: optional 5 ``torch.cuda.Event(enable_timing=True)`` recorded before
    the first stage and after each stage (indexer, top-k, attention, merge).
    """
    lib = _lib.load()
    d = dims.c()
    evp = None
    if events is not None:
        evs = _lib.DsaStageEvents()
        for i, e in enumerate(events):
            if e is not None and not e.cuda_event:
                e.record()  # torch creates the CUDA event lazily, on its first record
            evs.ev[i] = None if e is None else e.cuda_event
        evp = ctypes.byref(evs)
    rc = lib.dsa_decode_step(ctypes.byref(d), _ptr(q_I), _ptr(q_scale), _ptr(w), _ptr(k_I), _ptr(k_scale), _ptr(q),
                             _ptr(kv), _ptr(q_seq), _ptr(q_len), ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse),
                             _ptr(scores_out), _ptr(idx_out), _ptr(ws), ws.numel(), _stream_ptr(), evp)
    _lib.check(lib, rc, "dsa_decode_step")
    return out, lse


def prefill(dims: Dims, q_I, q_scale, w, k_I, k_scale, q, kv, q_seq, q_len, softmax_scale, out, lse, ws,
            idx_out=None):
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_prefill(ctypes.byref(d), _ptr(q_I), _ptr(q_scale), _ptr(w), _ptr(k_I), _ptr(k_scale), _ptr(q),
                         _ptr(kv), _ptr(q_seq), _ptr(q_len), ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse),
                         _ptr(idx_out), _ptr(ws), ws.numel(), _stream_ptr())
    _lib.check(lib, rc, "dsa_prefill")
    return out, lse


def selftest_wait_timeout(ws: torch.Tensor, timeout_us: int = 200000):
    lib = _lib.load()
    rc = lib.dsa_selftest_wait_timeout(ws.data_ptr(), ws.numel(), int(timeout_us), _stream_ptr())
    _lib.check(lib, rc, "dsa_selftest_wait_timeout")


def selftest_attention_stall(dims: Dims, q, kv, idx, q_seq, q_len, softmax_scale, out, lse, ws,
                             timeout_us: int = 100000):
    """The attention kernel with its first tile never signalled: its bounded wait runs out."""
    lib = _lib.load()
    d = dims.c()
    rc = lib.dsa_selftest_attention_stall(ctypes.byref(d), _ptr(q), _ptr(kv), _ptr(idx), _ptr(q_seq), _ptr(q_len),
                                          ctypes.c_float(softmax_scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                          int(timeout_us), _stream_ptr())
    _lib.check(lib, rc, "dsa_selftest_attention_stall")


# ---- conveniences over an inputs.DSAInputs workload --------------------------

def alloc_outputs(inp, device=None):
    dev = device or inp.device
    odt = torch.float32 if inp.kv_dtype == _lib.DSA_F32 else torch.bfloat16
    out = torch.empty((inp.Nq, inp.H, D_V), dtype=odt, device=dev)
    lse = torch.empty((inp.Nq, inp.H), dtype=torch.float32, device=dev)
    return out, lse


def run_decode(inp, ws=None, scores_out=None, idx_out=None, events=None, dims=None, out=None, lse=None):
    """decode_step over a device-resident ``DSAInputs``; returns (out, lse)."""
    dims = dims or dims_of(inp)
    if ws is None:
        ws = make_workspace(dims, _lib.DSA_OP_DECODE, inp.device)
    if out is None:
        out, lse = alloc_outputs(inp)
    return decode_step(dims, inp.q_I, inp.q_scale, inp.w, inp.k_I, inp.k_scale, inp.q, inp.kv, inp.q_seq, inp.q_len,
                       inp.softmax_scale, out, lse, ws, scores_out=scores_out, idx_out=idx_out, events=events)
