"""Binding of libclo's paged KV cache held in 16 bits (include/clo_paged.h):
argument marshalling only, like the rest of the package, which re-exports
everything here.

A serving step on a paged cache (clo_paged_plan gives slots, offsets, lengths):

    clo_paged_rope_append(q, k, v, ...)   # positions, and K and V into the cache, each layer
    clo_paged_chunk_attn(q, kc, vc, ...)  # attention of prompts, chunks and decoding requests, each layer

and for long contexts, decode attention over selected blocks:

    clo_paged_block_bounds(kc, slots, bounds)        # the ranges of the blocks that were written to
    clo_paged_block_select(q, bounds, ..., sel, ws)  # the blocks each KV head attends to
    clo_paged_sparse_decode_attn(q, kc, vc, ..., sel, out, ws)

The ``prepare_*`` forms check a call once and re-issue it on the same buffers.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import (_F, _I, _P, _SIGS, _SZ, CLO_ERR_INVALID_ARG, HEAD_DIM, CloError, PreparedCall, _check, _dev, _opts, _run,
               lib)
from .kv4 import _device_of, _dtype, _LL, _Prepared, _rows

PAGED_BLOCK_SIZE = 16


class RopeAppendArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("q", "k", "v", "q_out")] + \
               [(n, _LL) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")] + \
               [(n, _P) for n in ("pos", "pairs", "slot_map", "kc", "vc", "err_flag")] + \
               [(n, _I) for n in ("dtype", "N", "axes", "rot", "interleaved", "Hq", "Hkv", "d", "num_blocks", "block_size")]


class ChunkAttnArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("q", "kc", "vc")] + [(n, _LL) for n in ("q_stride", "kv_block", "kv_head", "kv_token")] + \
               [(n, _P) for n in ("block_table", "ctx_len", "offsets", "out", "lse", "workspace")] + \
               [("ws_bytes", _SZ), ("err_flag", _P), ("opts", _P), ("dtype", _I), ("scale", _F)] + \
               [(n, _I) for n in ("B", "N", "Hq", "Hkv", "d", "num_blocks", "block_size", "max_blocks")]


class BlockBoundsArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("kc", "slot_map", "bounds", "err_flag")] + \
               [(n, _I) for n in ("dtype", "N", "Hkv", "d", "num_blocks", "block_size")]


class BlockSelectArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("q", "bounds", "block_table", "ctx_len", "sel", "workspace")] + \
               [("ws_bytes", _SZ), ("err_flag", _P)] + \
               [(n, _I) for n in ("dtype", "B", "Hq", "Hkv", "d", "num_blocks", "block_size", "max_blocks", "n_sel", "n_first",
                                  "n_last")]


class SparseAttnArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("q", "kc", "vc", "block_table", "ctx_len", "sel", "out", "lse", "workspace")] + \
               [("ws_bytes", _SZ), ("err_flag", _P), ("opts", _P), ("dtype", _I), ("scale", _F)] + \
               [(n, _I) for n in ("B", "Hq", "Hkv", "d", "num_blocks", "block_size", "max_blocks", "n_sel")]


_SIGS.update({
    "clo_rope_pairs": ([_P, _P, _I, _P], _I),
    "clo_paged_rope_append": ([_P, _P], _I),
    "clo_paged_chunk_workspace_size": ([_I, _I, _I, _I], _SZ),
    "clo_paged_chunk_attn": ([_P, _P], _I),
    "clo_paged_bounds_bytes": ([_I, _I], _SZ),
    "clo_paged_block_bounds": ([_P, _P], _I),
    "clo_paged_select_workspace_size": ([_I, _I, _I], _SZ),
    "clo_paged_block_select": ([_P, _P], _I),
    "clo_paged_sparse_decode_attn": ([_P, _P], _I),
})


def _caches(kc, vc, dtype, strided=False):
    """Pointers of a cache [num_blocks][Hkv][16][128] and its strides."""
    for t, name in ((kc, "kc"), (vc, "vc")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4 or t.dtype != dtype:
            raise CloError(f"{name} must be a {dtype} CUDA tensor [num_blocks][Hkv][16][{HEAD_DIM}]", CLO_ERR_INVALID_ARG)
        if not strided and not t.is_contiguous():
            raise CloError(f"{name} must be contiguous", CLO_ERR_INVALID_ARG)
    if kc.shape != vc.shape or kc.shape[2] != PAGED_BLOCK_SIZE or kc.shape[3] != HEAD_DIM:
        raise CloError(f"kc and vc must be [num_blocks][Hkv][{PAGED_BLOCK_SIZE}][{HEAD_DIM}], got {tuple(kc.shape)} and "
                       f"{tuple(vc.shape)}", CLO_ERR_INVALID_ARG)
    nb, Hkv, bs, d = kc.shape
    # The strides of dimensions of size 1 say nothing.
    strides = [x if n > 1 else y for x, n, y in zip(kc.stride(), kc.shape, (Hkv * bs * d, bs * d, d, 1))]
    if strided and ([x for x, n in zip(kc.stride(), kc.shape) if n > 1] != [x for x, n in zip(vc.stride(), vc.shape) if n > 1] or
                    strides[3] != 1):
        raise CloError("kc and vc must have the same strides and contiguous rows", CLO_ERR_INVALID_ARG)
    return kc.data_ptr(), vc.data_ptr(), nb, Hkv, strides[:3]


# ---------------------------------------------------------------- positions and append

def clo_rope_pairs(inv_freq, axis=None) -> torch.Tensor:
    """The table of a model's pairs for clo_paged_rope_append, on the host: int64
    [n][2], 16 bytes a pair (copy it to the GPU once).  inv_freq: n radians a
    position (float64 tensor or sequence); axis: n position axes (None: all 0)."""
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
    ax = None if axis is None else torch.as_tensor(axis, device="cpu").to(torch.int32).contiguous()
    if f.dim() != 1 or (ax is not None and ax.shape != f.shape):
        raise CloError("inv_freq and axis must be 1-d and of one length", CLO_ERR_INVALID_ARG)
    out = torch.zeros(f.numel(), 2, dtype=torch.int64)
    _check(lib().clo_rope_pairs(f.data_ptr(), None if ax is None else ax.data_ptr(), f.numel(), out.data_ptr()),
           "clo_rope_pairs")
    return out


def clo_paged_rope_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, pairs: torch.Tensor,
                          slot_map: torch.Tensor, kc: torch.Tensor, vc: torch.Tensor, q_out: Optional[torch.Tensor],
                          interleaved: bool = False, err_flag: Optional[torch.Tensor] = None, stream=None):
    """Turns queries q [N][Hq][128] (into q_out, which may be q) and keys k
    [N][Hkv][128] by their positions pos [N] or [axes][N] int32, and writes k and v
    to the slots slot_map [N] int32 of the cache kc, vc [num_blocks][Hkv][16][128];
    slot -1 skips a token's K and V.  float16 or bfloat16; tokens may be strided, as
    in a fused projection's output.  pairs: clo_rope_pairs(...) on the GPU, one row
    for each pair of channels.  q and q_out None: keys and values alone."""
    call, _ = _rope_call(q, k, v, pos, pairs, slot_map, kc, vc, q_out, interleaved, err_flag)
    _run(call, stream)


def prepare_paged_rope_append(q, k, v, pos, pairs, slot_map, kc, vc, q_out, interleaved=False, err_flag=None,
                              stream=None) -> PreparedCall:
    """clo_paged_rope_append on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_rope_call(q, k, v, pos, pairs, slot_map, kc, vc, q_out, interleaved, err_flag), stream)


def _rope_call(q, k, v, pos, pairs, slot_map, kc, vc, q_out, interleaved, err_flag):
    dt = _dtype(k, "k")
    pk, ks = _rows(k, "k")
    pv, vs = _rows(v, "v")
    if (q is None) != (q_out is None):
        raise CloError("q and q_out go together", CLO_ERR_INVALID_ARG)
    pq, qs = (None, 0) if q is None else _rows(q, "q")
    po, os_ = (None, 0) if q is None else _rows(q_out, "q_out")
    ppos = _dev(pos, "pos", torch.int32)
    ppr = _dev(pairs, "pairs", torch.int64, 2)
    psl = _dev(slot_map, "slot_map", torch.int32, 1)
    pkc, pvc, nb, Hkv, _ = _caches(kc, vc, k.dtype)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    N = k.shape[0]
    axes = 1 if pos.dim() == 1 else pos.shape[0]
    if v.dtype != k.dtype or v.shape != k.shape or slot_map.numel() != N or k.shape[1] != Hkv or pos.dim() not in (1, 2) or \
            pos.shape[-1] != N or pairs.shape[1] != 2:
        raise CloError("append shapes do not match", CLO_ERR_INVALID_ARG)
    if q is not None and (q.dtype != k.dtype or q_out.dtype != k.dtype or q.shape != q_out.shape or q.shape[0] != N):
        raise CloError("q and q_out do not match", CLO_ERR_INVALID_ARG)
    args = RopeAppendArgs(pq, pk, pv, po, qs, ks, vs, os_, ppos, ppr or None, psl, pkc, pvc, pe or None, dt, N, axes,
                          2 * pairs.shape[0], int(bool(interleaved)), 0 if q is None else q.shape[1], Hkv, k.shape[2], nb,
                          PAGED_BLOCK_SIZE)
    keepalive = (q, k, v, pos, pairs, slot_map, kc, vc, q_out, err_flag)
    return ("clo_paged_rope_append", (ctypes.byref(args),), keepalive + (args,)), _device_of(*keepalive)


# ---------------------------------------------------------------- attention of chunks

def clo_paged_chunk_workspace_size(Hq: int, Hkv: int, d: int = HEAD_DIM, num_ctas: int = 0) -> int:
    return int(lib().clo_paged_chunk_workspace_size(Hq, Hkv, d, num_ctas))


def clo_paged_chunk_attn(q: torch.Tensor, kc: torch.Tensor, vc: torch.Tensor, block_table: torch.Tensor, ctx_len: torch.Tensor,
                         offsets: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, lse: Optional[torch.Tensor] = None,
                         err_flag: Optional[torch.Tensor] = None, scale: Optional[float] = None, num_ctas: int = 0,
                         events: Optional[Sequence] = None, stream=None):
    """Causal attention of each request's last tokens over its cached ones: rows
    offsets[r] .. offsets[r + 1] - 1 of q and out [N][Hq][128] (q's tokens may be
    strided) are the last of ctx_len[r] tokens in the blocks block_table[r] of the
    cache kc, vc [num_blocks][Hkv][16][128] (float16 or bfloat16; any strides that kc
    and vc share, with contiguous rows, such as clo_kv4_gather's output
    k.view(-1, 16, Hkv, 128).transpose(1, 2)).  offsets [B + 1], ctx_len [B] and
    block_table [B][max_blocks] int32; lse [N][Hq] fp32; workspace uint8,
    clo_paged_chunk_workspace_size(...) bytes."""
    call, _ = _chunk_call(q, kc, vc, block_table, ctx_len, offsets, out, workspace, lse, err_flag, scale, num_ctas, events)
    _run(call, stream)


def prepare_paged_chunk_attn(q, kc, vc, block_table, ctx_len, offsets, out, workspace, lse=None, err_flag=None, scale=None,
                             num_ctas: int = 0, events=None, stream=None) -> PreparedCall:
    """clo_paged_chunk_attn on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_chunk_call(q, kc, vc, block_table, ctx_len, offsets, out, workspace, lse, err_flag, scale, num_ctas,
                                  events), stream)


def _chunk_call(q, kc, vc, block_table, ctx_len, offsets, out, workspace, lse, err_flag, scale, num_ctas, events):
    dt = _dtype(q, "q")
    pq, qs = _rows(q, "q")
    N, Hq, d = q.shape
    pkc, pvc, nb, Hkv, strides = _caches(kc, vc, q.dtype, strided=True)
    pt = _dev(block_table, "block_table", torch.int32, 2)
    pc = _dev(ctx_len, "ctx_len", torch.int32, 1)
    pof = _dev(offsets, "offsets", torch.int32, 1)
    po = _dev(out, "out", q.dtype, 3)
    plse = _dev(lse, "lse", torch.float32, optional=True)
    pws = _dev(workspace, "workspace", torch.uint8)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    B = ctx_len.numel()
    if out.shape != q.shape or block_table.shape[0] != B or offsets.numel() != B + 1 or \
            (lse is not None and lse.numel() != N * Hq):
        raise CloError("attention buffer shapes do not match", CLO_ERR_INVALID_ARG)
    opts = _opts(num_ctas, events)
    args = ChunkAttnArgs(pq, pkc, pvc, qs, *strides, pt, pc, pof, po, plse or None, pws, workspace.numel(), pe or None,
                         ctypes.addressof(opts) if opts is not None else None, dt,
                         1.0 / math.sqrt(d) if scale is None else float(scale), B, N, Hq, Hkv, d, nb, PAGED_BLOCK_SIZE,
                         block_table.shape[1])
    keepalive = (q, kc, vc, block_table, ctx_len, offsets, out, workspace, lse, err_flag)
    return ("clo_paged_chunk_attn", (ctypes.byref(args),), keepalive + (opts, args)), _device_of(*keepalive)


# ---------------------------------------------------------------- selected blocks

def clo_paged_bounds_bytes(block_size: int = PAGED_BLOCK_SIZE, d: int = HEAD_DIM) -> int:
    """Bytes of one record of bounds (the key ranges of one block and KV head)."""
    return int(lib().clo_paged_bounds_bytes(block_size, d))


def _bounds(bounds):
    p = _dev(bounds, "bounds", torch.uint8, 3)
    if bounds.shape[2] != clo_paged_bounds_bytes():
        raise CloError(f"bounds must be [num_blocks][Hkv][{clo_paged_bounds_bytes()}], got {tuple(bounds.shape)}",
                       CLO_ERR_INVALID_ARG)
    return p


def clo_paged_block_bounds(kc: torch.Tensor, slot_map: torch.Tensor, bounds: torch.Tensor,
                           err_flag: Optional[torch.Tensor] = None, stream=None):
    """Updates the key ranges bounds [num_blocks][Hkv][272] uint8 of the blocks that
    the new tokens in slots slot_map [N] int32 went to, from the cache kc
    [num_blocks][Hkv][16][128]."""
    call, _ = _bounds_call(kc, slot_map, bounds, err_flag)
    _run(call, stream)


def prepare_paged_block_bounds(kc, slot_map, bounds, err_flag=None, stream=None) -> PreparedCall:
    """clo_paged_block_bounds on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_bounds_call(kc, slot_map, bounds, err_flag), stream)


def _bounds_call(kc, slot_map, bounds, err_flag):
    dt = _dtype(kc, "kc")
    pkc, _, nb, Hkv, _ = _caches(kc, kc, kc.dtype)
    psl = _dev(slot_map, "slot_map", torch.int32, 1)
    pb = _bounds(bounds)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    if bounds.shape[:2] != kc.shape[:2]:
        raise CloError("bounds do not match the cache", CLO_ERR_INVALID_ARG)
    args = BlockBoundsArgs(pkc, psl, pb, pe or None, dt, slot_map.numel(), Hkv, HEAD_DIM, nb, PAGED_BLOCK_SIZE)
    keepalive = (kc, slot_map, bounds, err_flag)
    return ("clo_paged_block_bounds", (ctypes.byref(args),), keepalive + (args,)), _device_of(*keepalive)


def clo_paged_select_workspace_size(B: int, Hkv: int, max_blocks: int) -> int:
    return int(lib().clo_paged_select_workspace_size(B, Hkv, max_blocks))


def clo_paged_block_select(q: torch.Tensor, bounds: torch.Tensor, block_table: torch.Tensor, ctx_len: torch.Tensor,
                           sel: torch.Tensor, workspace: torch.Tensor, n_first: int = 1, n_last: int = 1,
                           err_flag: Optional[torch.Tensor] = None, stream=None):
    """Selects the blocks that the queries q [B][Hq][128] attend to: sel
    [B][Hkv][n_sel] int32 gets columns of block_table, ascending, then -1.  The
    first n_first and last n_last blocks of a request are always among them.
    workspace: uint8, clo_paged_select_workspace_size(...) bytes."""
    call, _ = _select_call(q, bounds, block_table, ctx_len, sel, workspace, n_first, n_last, err_flag)
    _run(call, stream)


def prepare_paged_block_select(q, bounds, block_table, ctx_len, sel, workspace, n_first=1, n_last=1, err_flag=None,
                               stream=None) -> PreparedCall:
    """clo_paged_block_select on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_select_call(q, bounds, block_table, ctx_len, sel, workspace, n_first, n_last, err_flag), stream)


def _select_call(q, bounds, block_table, ctx_len, sel, workspace, n_first, n_last, err_flag):
    dt = _dtype(q, "q")
    pq = _dev(q, "q", q.dtype, 3)
    B, Hq, d = q.shape
    pb = _bounds(bounds)
    nb, Hkv = bounds.shape[:2]
    pt = _dev(block_table, "block_table", torch.int32, 2)
    pc = _dev(ctx_len, "ctx_len", torch.int32, 1)
    ps = _dev(sel, "sel", torch.int32, 3)
    pws = _dev(workspace, "workspace", torch.uint8)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    if ctx_len.numel() != B or block_table.shape[0] != B or sel.shape[:2] != (B, Hkv):
        raise CloError("selection buffer shapes do not match", CLO_ERR_INVALID_ARG)
    args = BlockSelectArgs(pq, pb, pt, pc, ps, pws, workspace.numel(), pe or None, dt, B, Hq, Hkv, d, nb, PAGED_BLOCK_SIZE,
                           block_table.shape[1], sel.shape[2], int(n_first), int(n_last))
    keepalive = (q, bounds, block_table, ctx_len, sel, workspace, err_flag)
    return ("clo_paged_block_select", (ctypes.byref(args),), keepalive + (args,)), _device_of(*keepalive)


def clo_paged_sparse_decode_attn(q: torch.Tensor, kc: torch.Tensor, vc: torch.Tensor, block_table: torch.Tensor,
                                 ctx_len: torch.Tensor, sel: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                                 lse: Optional[torch.Tensor] = None, err_flag: Optional[torch.Tensor] = None,
                                 scale: Optional[float] = None, num_ctas: int = 0, events: Optional[Sequence] = None,
                                 stream=None):
    """Decode attention of q [B][Hq][128] over the blocks sel [B][Hkv][n_sel] int32
    (columns of block_table) of the cache kc, vc [num_blocks][Hkv][16][128].
    workspace: uint8, clo_paged_chunk_workspace_size(...) bytes."""
    call, _ = _sparse_call(q, kc, vc, block_table, ctx_len, sel, out, workspace, lse, err_flag, scale, num_ctas, events)
    _run(call, stream)


def prepare_paged_sparse_decode_attn(q, kc, vc, block_table, ctx_len, sel, out, workspace, lse=None, err_flag=None, scale=None,
                                     num_ctas: int = 0, events=None, stream=None) -> PreparedCall:
    """clo_paged_sparse_decode_attn on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_sparse_call(q, kc, vc, block_table, ctx_len, sel, out, workspace, lse, err_flag, scale, num_ctas,
                                   events), stream)


def _sparse_call(q, kc, vc, block_table, ctx_len, sel, out, workspace, lse, err_flag, scale, num_ctas, events):
    dt = _dtype(q, "q")
    pq = _dev(q, "q", q.dtype, 3)
    B, Hq, d = q.shape
    pkc, pvc, nb, Hkv, _ = _caches(kc, vc, q.dtype)
    pt = _dev(block_table, "block_table", torch.int32, 2)
    pc = _dev(ctx_len, "ctx_len", torch.int32, 1)
    ps = _dev(sel, "sel", torch.int32, 3)
    po = _dev(out, "out", q.dtype, 3)
    plse = _dev(lse, "lse", torch.float32, optional=True)
    pws = _dev(workspace, "workspace", torch.uint8)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    if out.shape != q.shape or ctx_len.numel() != B or block_table.shape[0] != B or sel.shape[:2] != (B, Hkv) or \
            (lse is not None and lse.numel() != B * Hq):
        raise CloError("attention buffer shapes do not match q", CLO_ERR_INVALID_ARG)
    opts = _opts(num_ctas, events)
    args = SparseAttnArgs(pq, pkc, pvc, pt, pc, ps, po, plse or None, pws, workspace.numel(), pe or None,
                          ctypes.addressof(opts) if opts is not None else None, dt,
                          1.0 / math.sqrt(d) if scale is None else float(scale), B, Hq, Hkv, d, nb, PAGED_BLOCK_SIZE,
                          block_table.shape[1], sel.shape[2])
    keepalive = (q, kc, vc, block_table, ctx_len, sel, out, workspace, lse, err_flag)
    return ("clo_paged_sparse_decode_attn", (ctypes.byref(args),), keepalive + (opts, args)), _device_of(*keepalive)
