"""Binding of libclo's paged KV cache held in 4 bits (include/clo_kv4.h):
argument marshalling only, like the rest of the package, which re-exports
everything here.

A decode step of a paged cache:

    clo_paged_plan(...)                  # block table, slots of the new tokens, lengths
    clo_kv4_append(k, v, slots, pool)    # the new tokens' K and V into the cache, each layer
    clo_kv4_paged_decode_attn(q, ...)    # attention of the new queries, each layer

``clo_kv4_gather`` reads cached rows back in 16 bits.  The ``prepare_*`` forms
check a call once and re-issue it on the same buffers.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from . import (_F, _I, _P, _SIGS, _SZ, CLO_ERR_INVALID_ARG, CLO_OK, HEAD_DIM, CloError, PreparedCall, _check, _dev,
               _opts, _run, lib)

FLAG_NO_ROOM = 0x10
KV4_BLOCK_SIZE = 16
KV4_GROUPS = (32, 64, 128)

_LL = ctypes.c_longlong


class PlanArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("len_in", "keep", "add", "block_table", "free_ring", "ring_in", "ring_out", "len_out",
                                  "start", "offsets", "slot_map", "err_flag")] + \
               [(n, _I) for n in ("B", "block_size", "max_blocks", "ring_size", "max_new")]


class AppendArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_stride", _LL), ("v_stride", _LL), ("slot_map", _P), ("pool", _P),
                ("err_flag", _P)] + \
               [(n, _I) for n in ("dtype", "N", "Hkv", "d", "num_blocks", "block_size", "group")]


class GatherArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("pool", "slot_map", "k", "v", "err_flag")] + \
               [(n, _I) for n in ("dtype", "N", "Hkv", "d", "num_blocks", "block_size", "group")]


class AttnArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("q", "pool", "block_table", "ctx_len", "out", "lse", "workspace")] + \
               [("ws_bytes", _SZ), ("err_flag", _P), ("opts", _P), ("dtype", _I), ("scale", _F)] + \
               [(n, _I) for n in ("B", "n_q", "Hq", "Hkv", "d", "num_blocks", "block_size", "max_blocks", "group")]


_SIGS.update({
    "clo_kv4_block_bytes": ([_I, _I, _I], _SZ),
    "clo_paged_plan": ([_P, _P], _I),
    "clo_kv4_append": ([_P, _P], _I),
    "clo_kv4_gather": ([_P, _P], _I),
    "clo_kv4_paged_workspace_size": ([_I, _I, _I, _I, _I, _I], _SZ),
    "clo_kv4_paged_decode_attn": ([_P, _P], _I),
})

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_GROUP_OF_RECORD = {2048 + 128 * (HEAD_DIM // g): g for g in KV4_GROUPS}


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # as current_stream(), without the object


class _Prepared(PreparedCall):
    """A PreparedCall that is refused while another device is current: its
    kernels would start there."""

    __slots__ = ("_device",)

    def __init__(self, call, device: int, stream=None):
        super().__init__(*call, stream)
        self._device = device

    def __call__(self):
        if torch.cuda.current_device() != self._device:
            raise CloError(f"the call's tensors are on cuda:{self._device}, which is not the current device",
                           CLO_ERR_INVALID_ARG)
        st = self._stream
        if st is None:
            st = torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(self._device)
        status = self._fn(self._args[0], st)
        if status != CLO_OK:
            _check(status, self._what)


def _device_of(*tensors) -> int:
    """The one device of the tensors, which has to be the current one."""
    devices = {t.device.index for t in tensors if t is not None}
    if len(devices) != 1:
        raise CloError("tensors are on more than one device", CLO_ERR_INVALID_ARG)
    device = devices.pop()
    if device != torch.cuda.current_device():
        raise CloError(f"tensors are on cuda:{device}, which is not the current device", CLO_ERR_INVALID_ARG)
    return device


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise CloError(f"{name} must be a float16 or bfloat16 tensor", CLO_ERR_INVALID_ARG)
    return _DTYPES[t.dtype]


def _pool(pool: torch.Tensor):
    """(pointer, num_blocks, Hkv, group) of a cache."""
    p = _dev(pool, "pool", torch.uint8, 3)
    group = _GROUP_OF_RECORD.get(pool.shape[2])
    if group is None:
        raise CloError(f"pool must be [num_blocks][Hkv][R] with R of clo_kv4_block_bytes, got {tuple(pool.shape)}",
                       CLO_ERR_INVALID_ARG)
    return p, pool.shape[0], pool.shape[1], group


def clo_kv4_block_bytes(group: int, block_size: int = KV4_BLOCK_SIZE, d: int = HEAD_DIM) -> int:
    """Bytes of one record (16 tokens of one KV head) with channel groups of `group`."""
    return int(lib().clo_kv4_block_bytes(block_size, d, group))


# ---------------------------------------------------------------- block plan

def clo_paged_plan(len_in: torch.Tensor, add: torch.Tensor, block_table: torch.Tensor, free_ring: torch.Tensor,
                   ring_in: torch.Tensor, ring_out: torch.Tensor, len_out: torch.Tensor, start: torch.Tensor,
                   offsets: torch.Tensor, slot_map: torch.Tensor, keep: Optional[torch.Tensor] = None,
                   err_flag: Optional[torch.Tensor] = None, block_size: int = KV4_BLOCK_SIZE, stream=None):
    """The block table, lengths, free ring and slot map of a step in which
    request r keeps its first keep[r] tokens (None: all) and gets add[r] new
    ones.  int32 tensors: len_in, add, keep, len_out, start [B]; block_table
    [B][max_blocks] and free_ring, in place; ring_in, ring_out [2] (first
    entry, count); offsets [B + 1]; slot_map [max_new].  len_out may be len_in
    and ring_out may be ring_in."""
    call, _ = _plan_call(len_in, add, block_table, free_ring, ring_in, ring_out, len_out, start, offsets, slot_map,
                         keep, err_flag, block_size)
    _run(call, stream)


def prepare_paged_plan(len_in, add, block_table, free_ring, ring_in, ring_out, len_out, start, offsets, slot_map,
                       keep=None, err_flag=None, block_size: int = KV4_BLOCK_SIZE, stream=None) -> PreparedCall:
    """clo_paged_plan on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_plan_call(len_in, add, block_table, free_ring, ring_in, ring_out, len_out, start, offsets,
                                 slot_map, keep, err_flag, block_size), stream)


def _plan_call(len_in, add, block_table, free_ring, ring_in, ring_out, len_out, start, offsets, slot_map, keep,
               err_flag, block_size):
    i32 = torch.int32
    pl, pa = _dev(len_in, "len_in", i32, 1), _dev(add, "add", i32, 1)
    pk = _dev(keep, "keep", i32, 1, optional=True)
    pt, pr = _dev(block_table, "block_table", i32, 2), _dev(free_ring, "free_ring", i32, 1)
    pi, po = _dev(ring_in, "ring_in", i32, 1), _dev(ring_out, "ring_out", i32, 1)
    plo, ps = _dev(len_out, "len_out", i32, 1), _dev(start, "start", i32, 1)
    pof, psl = _dev(offsets, "offsets", i32, 1), _dev(slot_map, "slot_map", i32, 1)
    pe = _dev(err_flag, "err_flag", i32, optional=True)
    B = len_in.numel()
    if any(t.numel() != B for t in (add, len_out, start)) or (keep is not None and keep.numel() != B) or \
            block_table.shape[0] != B or offsets.numel() != B + 1 or ring_in.numel() != 2 or ring_out.numel() != 2:
        raise CloError("plan buffer sizes do not match len_in", CLO_ERR_INVALID_ARG)
    keepalive = (len_in, add, block_table, free_ring, ring_in, ring_out, len_out, start, offsets, slot_map, keep,
                 err_flag)
    args = PlanArgs(pl, pk or None, pa, pt, pr, pi, po, plo, ps, pof, psl, pe or None, B, int(block_size),
                    block_table.shape[1], free_ring.numel(), slot_map.numel())
    return ("clo_paged_plan", (ctypes.byref(args),), keepalive + (args,)), _device_of(*keepalive)


# ---------------------------------------------------------------- append and gather

def _rows(t: torch.Tensor, name: str):
    """(pointer, elements between tokens) of [N][Hkv][128] rows: contiguous in
    a token, any stride between tokens that is a multiple of 8."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3 or t.shape[2] != HEAD_DIM:
        raise CloError(f"{name} must be a CUDA tensor [N][Hkv][{HEAD_DIM}]", CLO_ERR_INVALID_ARG)
    N, Hkv, d = t.shape
    if N * Hkv > 0 and (t.stride(2) != 1 or (Hkv > 1 and t.stride(1) != d)):
        raise CloError(f"{name} must be contiguous within a token", CLO_ERR_INVALID_ARG)
    return t.data_ptr(), t.stride(0) if N > 1 else Hkv * d


def clo_kv4_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, pool: torch.Tensor,
                   err_flag: Optional[torch.Tensor] = None, stream=None):
    """Quantises K and V rows [N][Hkv][128] (float16 or bfloat16; tokens may be
    strided, as in a fused projection's output) into the slots slot_map [N]
    int32 of the cache pool [num_blocks][Hkv][R] uint8; slot -1 skips a row."""
    call, _ = _append_call(k, v, slot_map, pool, err_flag)
    _run(call, stream)


def prepare_kv4_append(k, v, slot_map, pool, err_flag=None, stream=None) -> PreparedCall:
    """clo_kv4_append on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_append_call(k, v, slot_map, pool, err_flag), stream)


def _append_call(k, v, slot_map, pool, err_flag):
    dt = _dtype(k, "k")
    pk, ks = _rows(k, "k")
    pv, vs = _rows(v, "v")
    psl = _dev(slot_map, "slot_map", torch.int32, 1)
    pp, nb, Hkv, group = _pool(pool)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    if v.dtype != k.dtype or v.shape != k.shape or slot_map.numel() != k.shape[0] or k.shape[1] != Hkv:
        raise CloError("append shapes do not match", CLO_ERR_INVALID_ARG)
    args = AppendArgs(pk, pv, ks, vs, psl, pp, pe or None, dt, k.shape[0], Hkv, k.shape[2], nb, KV4_BLOCK_SIZE, group)
    keepalive = (k, v, slot_map, pool, err_flag)
    return ("clo_kv4_append", (ctypes.byref(args),), keepalive + (args,)), _device_of(*keepalive)


def clo_kv4_gather(pool: torch.Tensor, slot_map: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   err_flag: Optional[torch.Tensor] = None, stream=None):
    """Reads the slots slot_map [N] int32 of the cache back into k, v
    [N][Hkv][128] (float16 or bfloat16, contiguous); slot -1 gives zeros."""
    call, _ = _gather_call(pool, slot_map, k, v, err_flag)
    _run(call, stream)


def prepare_kv4_gather(pool, slot_map, k, v, err_flag=None, stream=None) -> PreparedCall:
    """clo_kv4_gather on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_gather_call(pool, slot_map, k, v, err_flag), stream)


def _gather_call(pool, slot_map, k, v, err_flag):
    dt = _dtype(k, "k")
    pk, pv = _dev(k, "k", k.dtype, 3), _dev(v, "v", k.dtype, 3)
    psl = _dev(slot_map, "slot_map", torch.int32, 1)
    pp, nb, Hkv, group = _pool(pool)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    if v.shape != k.shape or slot_map.numel() != k.shape[0] or k.shape[1] != Hkv:
        raise CloError("gather shapes do not match", CLO_ERR_INVALID_ARG)
    args = GatherArgs(pp, psl, pk, pv, pe or None, dt, k.shape[0], Hkv, k.shape[2], nb, KV4_BLOCK_SIZE, group)
    keepalive = (pool, slot_map, k, v, err_flag)
    return ("clo_kv4_gather", (ctypes.byref(args),), keepalive + (args,)), _device_of(*keepalive)


# ---------------------------------------------------------------- attention

def clo_kv4_paged_workspace_size(B: int, n_q: int, Hq: int, Hkv: int, d: int = HEAD_DIM, num_ctas: int = 0) -> int:
    return int(lib().clo_kv4_paged_workspace_size(B, n_q, Hq, Hkv, d, num_ctas))


def clo_kv4_paged_decode_attn(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor, ctx_len: torch.Tensor,
                              out: torch.Tensor, workspace: torch.Tensor, lse: Optional[torch.Tensor] = None,
                              err_flag: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                              num_ctas: int = 0, events: Optional[Sequence] = None, stream=None):
    """Decode attention over the 4-bit paged cache: q and out [B][n_q][Hq][128]
    (or [B][Hq][128] for one query a request), float16 or bfloat16; pool
    [num_blocks][Hkv][R] uint8; block_table [B][max_blocks] and ctx_len [B]
    int32.  ctx_len counts the last n_q tokens, whose queries q holds: query i
    sees the first ctx_len - (n_q - 1 - i).  lse: [B][n_q][Hq] fp32; workspace:
    uint8, clo_kv4_paged_workspace_size(...) bytes."""
    call, _ = _attn_call(q, pool, block_table, ctx_len, out, workspace, lse, err_flag, scale, num_ctas, events)
    _run(call, stream)


def prepare_kv4_paged_decode_attn(q, pool, block_table, ctx_len, out, workspace, lse=None, err_flag=None, scale=None,
                                  num_ctas: int = 0, events=None, stream=None) -> PreparedCall:
    """clo_kv4_paged_decode_attn on fixed buffers, checked once (see PreparedCall)."""
    return _Prepared(*_attn_call(q, pool, block_table, ctx_len, out, workspace, lse, err_flag, scale, num_ctas,
                                 events), stream)


def _attn_call(q, pool, block_table, ctx_len, out, workspace, lse, err_flag, scale, num_ctas, events):
    dt = _dtype(q, "q")
    pq = _dev(q, "q", q.dtype)
    if q.dim() not in (3, 4):
        raise CloError(f"q must be [B][n_q][Hq][d] or [B][Hq][d], got {tuple(q.shape)}", CLO_ERR_INVALID_ARG)
    B, Hq, d = q.shape[0], q.shape[-2], q.shape[-1]
    n_q = q.shape[1] if q.dim() == 4 else 1
    pp, nb, Hkv, group = _pool(pool)
    pt = _dev(block_table, "block_table", torch.int32, 2)
    pc = _dev(ctx_len, "ctx_len", torch.int32, 1)
    po = _dev(out, "out", q.dtype)
    plse = _dev(lse, "lse", torch.float32, optional=True)
    pws = _dev(workspace, "workspace", torch.uint8)
    pe = _dev(err_flag, "err_flag", torch.int32, optional=True)
    if out.shape != q.shape or ctx_len.numel() != B or block_table.shape[0] != B or \
            (lse is not None and lse.numel() != B * n_q * Hq):
        raise CloError("attention buffer shapes do not match q", CLO_ERR_INVALID_ARG)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    opts = _opts(num_ctas, events)
    keepalive = (q, pool, block_table, ctx_len, out, workspace, lse, err_flag)
    args = AttnArgs(pq, pp, pt, pc, po, plse or None, pws, workspace.numel(), pe or None,
                    ctypes.addressof(opts) if opts is not None else None, dt, float(scale), B, n_q, Hq, Hkv, d, nb,
                    KV4_BLOCK_SIZE, block_table.shape[1], group)
    return ("clo_kv4_paged_decode_attn", (ctypes.byref(args),), keepalive + (opts, args)), _device_of(*keepalive)
