"""The 16-bit paged cache's entry points without a GPU: the exported symbols, the
structs' layout, the rotary table and what each call refuses before it launches
anything."""
import ctypes
import math
import os
import re
import subprocess
from fractions import Fraction

import pytest
import torch

import offloaded_kv_decode_gb300 as clo
import paged_ref as ref
from offloaded_kv_decode_gb300 import build as libbuild
from offloaded_kv_decode_gb300 import paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned non-null stand-in pointer: never dereferenced on these paths
OK, INVALID, UNSUPPORTED, WORKSPACE = clo.CLO_OK, clo.CLO_ERR_INVALID_ARG, clo.CLO_ERR_UNSUPPORTED, clo.CLO_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return clo.lib()


def test_header_and_library_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "clo_paged.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(clo_[a-z0-9_]+)\s*\(", text))
    assert names == {"clo_rope_pairs", "clo_paged_rope_append", "clo_paged_chunk_workspace_size", "clo_paged_chunk_attn",
                     "clo_paged_bounds_bytes", "clo_paged_block_bounds", "clo_paged_select_workspace_size",
                     "clo_paged_block_select", "clo_paged_sparse_decode_attn"}
    for n in names:
        assert hasattr(L, n) and hasattr(clo, n)


STRUCTS = {"clo_paged_rope_append_args": paged.RopeAppendArgs, "clo_paged_chunk_attn_args": paged.ChunkAttnArgs,
           "clo_paged_block_bounds_args": paged.BlockBoundsArgs, "clo_paged_block_select_args": paged.BlockSelectArgs,
           "clo_paged_sparse_attn_args": paged.SparseAttnArgs}


def test_structs_match_the_header(tmp_path):
    """Sizes and offsets of the argument structs as a C compiler lays them out."""
    lines = ['printf("%zu\\n", sizeof(clo_rope_pair));']
    for name, t in STRUCTS.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in t._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "clo_paged.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0; }\n")
    cuda = os.path.join(os.path.dirname(os.path.dirname(libbuild.nvcc_path())), "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src),
                    "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, check=True).stdout.split()]
    want = [16]
    for t in STRUCTS.values():
        want.append(ctypes.sizeof(t))
        want += [getattr(t, f[0]).offset for f in t._fields_]
    assert got == want


def call(L, what, struct, values):
    return getattr(L, what)(ctypes.byref(struct(**values)), None)


def test_no_arguments(L):
    for what in ("clo_paged_rope_append", "clo_paged_chunk_attn", "clo_paged_block_bounds", "clo_paged_block_select",
                 "clo_paged_sparse_decode_attn"):
        assert getattr(L, what)(None, None) == INVALID


# ---------------------------------------------------------------- the rotary table

def over_two_pi(f):
    """f / (2 pi) * 2^64 rounded, modulo 2^64, in whole numbers: pi by Machin's series."""
    bits = 400

    def arctan_inverse(x):
        term = total = (1 << bits) // x
        k, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    v = Fraction(f) * (1 << (64 + bits)) / (2 * pi)
    return math.floor(v + Fraction(1, 2)) % (1 << 64)


def test_rope_pairs(L):
    f = [1.0, 10000.0 ** (-1 / 64), 10000.0 ** (-63 / 64), 1e-300, 0.0, -0.3, 5e5 ** (-17 / 64), 1048575.9, 2.0 ** -30, math.pi]
    got = clo.clo_rope_pairs(f, list(range(4)) + [0] * 6)
    for x, (turns, rest), a in zip(f, got.tolist(), list(range(4)) + [0] * 6):
        assert (turns - over_two_pi(x)) % (1 << 64) in (0, 1, (1 << 64) - 1), x  # a tie may fall either way
        assert rest == a  # the axis, and a reserved word of 0
    assert clo.clo_rope_pairs([]).shape == (0, 2)
    assert torch.equal(clo.clo_rope_pairs(f)[:, 0], got[:, 0]) and torch.all(clo.clo_rope_pairs(f)[:, 1] == 0)


def test_rope_pairs_rejects(L):
    for bad in ([math.nan], [math.inf], [1048576.0], [-1e30]):
        with pytest.raises(clo.CloError):
            clo.clo_rope_pairs(bad)
    for axis in ([4], [-1]):
        with pytest.raises(clo.CloError):
            clo.clo_rope_pairs([1.0], axis)
    with pytest.raises(clo.CloError):
        clo.clo_rope_pairs([1.0, 2.0], [0])
    assert L.clo_rope_pairs(None, None, 0, None) == OK
    assert L.clo_rope_pairs(None, None, 1, FAKE) == INVALID and L.clo_rope_pairs(FAKE, None, -1, FAKE) == INVALID


# ---------------------------------------------------------------- refusals

def _append(L, **kw):
    p = dict(q=FAKE, k=FAKE * 2, v=FAKE * 3, q_out=FAKE, q_stride=1024, k_stride=256, v_stride=256, q_out_stride=1024, pos=FAKE,
             pairs=FAKE, slot_map=FAKE, kc=FAKE, vc=FAKE, err_flag=None, dtype=0, N=4, axes=1, rot=128, interleaved=0, Hq=8, Hkv=2,
             d=128, num_blocks=8, block_size=16)
    p.update(kw)
    return call(L, "clo_paged_rope_append", paged.RopeAppendArgs, p)


def test_append_rejects(L):
    for name in ("k", "v", "pos", "pairs", "slot_map", "kc", "vc", "q", "q_out"):
        assert _append(L, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "q_out", "pairs", "kc", "vc"):
        assert _append(L, **{name: FAKE + 8}) == INVALID, name
    for name in ("pos", "slot_map", "err_flag"):
        assert _append(L, **{name: FAKE + 2}) == INVALID, name
    for kw in (dict(N=-1), dict(Hkv=0), dict(Hq=-1), dict(num_blocks=0), dict(axes=0), dict(rot=-16), dict(dtype=2), dict(dtype=-1),
               dict(q_stride=1016), dict(k_stride=255), dict(v_stride=260), dict(q_out_stride=1028), dict(k_stride=(1 << 40) + 8)):
        assert _append(L, **kw) == INVALID, kw
    for kw in (dict(d=64), dict(block_size=32), dict(rot=144), dict(rot=24), dict(axes=5), dict(N=1 << 28), dict(num_blocks=1 << 27)):
        assert _append(L, **kw) == UNSUPPORTED, kw
    assert _append(L, N=0, k=None, v=None, q=None, q_out=None, pos=None, pairs=None, slot_map=None, kc=None, vc=None) == OK


def test_append_rejects_overlaps(L):
    """q_out is q, or apart from all inputs; columns of the same fused rows are apart."""
    row = 8 * 256  # bytes of a query row
    assert _append(L, q_out=FAKE + 256) == INVALID
    assert _append(L, q_out=FAKE, q_stride=2048) == INVALID
    assert _append(L, q_out=FAKE * 2) == INVALID and _append(L, q_out=FAKE * 3 - 256) == INVALID
    fused = dict(q=FAKE, k=FAKE + row, v=FAKE + row + 512, q_stride=1536, k_stride=1536, v_stride=1536)
    assert _append(L, **fused, q_out=FAKE + 256, q_out_stride=1536) == INVALID   # over k
    assert _append(L, **fused, q_out=FAKE + row - 512, q_out_stride=1536) == INVALID
    assert _append(L, **fused, q_out=FAKE, q_out_stride=1024) == INVALID
    wide = dict(q=FAKE, k=FAKE + row, v=FAKE + row + 512, q_stride=4096, k_stride=4096, v_stride=4096)
    assert _append(L, **wide, q_out=FAKE + row + 256, q_out_stride=4096) == INVALID


def _chunk(L, **kw):
    p = dict(q=FAKE, kc=FAKE, vc=FAKE, q_stride=1024, kv_block=0, kv_head=0, kv_token=0, block_table=FAKE, ctx_len=FAKE,
             offsets=FAKE, out=FAKE * 2, lse=None, workspace=FAKE, ws_bytes=1 << 40, err_flag=None, opts=None, dtype=0, scale=0.1,
             B=2, N=4, Hq=8, Hkv=2, d=128, num_blocks=8, block_size=16, max_blocks=4)
    p.update(kw)
    return call(L, "clo_paged_chunk_attn", paged.ChunkAttnArgs, p)


def _sparse(L, **kw):
    p = dict(q=FAKE, kc=FAKE, vc=FAKE, block_table=FAKE, ctx_len=FAKE, sel=FAKE, out=FAKE * 2, lse=None, workspace=FAKE,
             ws_bytes=1 << 40, err_flag=None, opts=None, dtype=0, scale=0.1, B=2, Hq=8, Hkv=2, d=128, num_blocks=8, block_size=16,
             max_blocks=4, n_sel=3)
    p.update(kw)
    return call(L, "clo_paged_sparse_decode_attn", paged.SparseAttnArgs, p)


@pytest.mark.parametrize("fn,lists", [(_chunk, "offsets"), (_sparse, "sel")])
def test_attention_rejects(L, fn, lists):
    for name in ("q", "kc", "vc", "block_table", "ctx_len", lists, "out"):
        assert fn(L, **{name: None}) == INVALID, name
    for name in ("q", "kc", "vc", "out"):
        assert fn(L, **{name: FAKE + 8}) == INVALID, name
    for name in ("block_table", "ctx_len", lists, "lse", "err_flag"):
        assert fn(L, **{name: FAKE + 2}) == INVALID, name
    for kw in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(num_blocks=0), dict(max_blocks=0), dict(dtype=3), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf)):
        assert fn(L, **kw) == INVALID, kw
    for kw in (dict(d=64), dict(block_size=32), dict(Hq=18), dict(B=4097), dict(max_blocks=(1 << 20) + 1), dict(num_blocks=(1 << 26) + 1)):
        assert fn(L, **kw) == UNSUPPORTED, kw
    opts = clo.AttnOpts(-1, None, None)
    assert fn(L, opts=ctypes.addressof(opts)) == INVALID
    opts = clo.AttnOpts(4096, None, None)
    assert fn(L, opts=ctypes.addressof(opts)) == UNSUPPORTED
    opts = clo.AttnOpts(8, None, None)
    assert fn(L, opts=ctypes.addressof(opts), workspace=None) == WORKSPACE
    assert fn(L, opts=ctypes.addressof(opts), workspace=FAKE + 8) == WORKSPACE
    size = clo.clo_paged_chunk_workspace_size(8, 2, num_ctas=8)
    assert size > 0 and fn(L, opts=ctypes.addressof(opts), ws_bytes=size - 1) == WORKSPACE
    assert fn(L, B=0, q=None, kc=None, vc=None, out=None, workspace=None) == OK


def test_chunk_rejects(L):
    opts = clo.AttnOpts(8, None, None)
    o = dict(opts=ctypes.addressof(opts))
    for kw in (dict(N=-1), dict(q_stride=1016), dict(q_stride=1028), dict(kv_block=4096), dict(kv_block=4096, kv_head=2048, kv_token=64),
               dict(kv_block=4096, kv_head=2048, kv_token=130), dict(out=FAKE), dict(out=FAKE + 4 * 2048 - 16),
               dict(kv_block=1 << 39, kv_head=2048, kv_token=128)):
        assert _chunk(L, **o, **kw) == INVALID, kw
    assert _chunk(L, N=1 << 29) == UNSUPPORTED
    assert _chunk(L, N=0, q=None, out=None, workspace=None) == OK


def test_sparse_rejects(L):
    opts = clo.AttnOpts(8, None, None)
    o = dict(opts=ctypes.addressof(opts))
    assert _sparse(L, **o, out=FAKE) == INVALID and _sparse(L, **o, out=FAKE + 4080) == INVALID
    assert _sparse(L, **o, n_sel=0) == INVALID and _sparse(L, **o, n_sel=1 << 30) == UNSUPPORTED


def test_workspace_sizes(L):
    assert clo.clo_paged_chunk_workspace_size(8, 2, num_ctas=4) < clo.clo_paged_chunk_workspace_size(8, 2, num_ctas=400)
    for kw in (dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(Hq=18), dict(d=64), dict(num_ctas=-1), dict(num_ctas=4096)):
        a = dict(Hq=8, Hkv=2, d=128, num_ctas=4)
        a.update(kw)
        assert clo.clo_paged_chunk_workspace_size(**a) == 0, kw
    assert clo.clo_paged_select_workspace_size(2, 3, 100) >= 2400
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (4097, 1, 1), (4096, 16, 1), (100, 100, 1 << 20), (1, 1, (1 << 20) + 1)):
        assert clo.clo_paged_select_workspace_size(*bad) == 0, bad
    assert clo.clo_paged_bounds_bytes() == ref.RECORD
    assert clo.clo_paged_bounds_bytes(32) == 0 and clo.clo_paged_bounds_bytes(16, 64) == 0


def _bounds(L, **kw):
    p = dict(kc=FAKE, slot_map=FAKE, bounds=FAKE, err_flag=None, dtype=0, N=4, Hkv=2, d=128, num_blocks=8, block_size=16)
    p.update(kw)
    return call(L, "clo_paged_block_bounds", paged.BlockBoundsArgs, p)


def test_bounds_rejects(L):
    for name in ("kc", "slot_map", "bounds"):
        assert _bounds(L, **{name: None}) == INVALID, name
    for kw in (dict(kc=FAKE + 8), dict(bounds=FAKE + 8), dict(slot_map=FAKE + 2), dict(err_flag=FAKE + 1), dict(N=-1), dict(Hkv=0),
               dict(num_blocks=0), dict(dtype=5)):
        assert _bounds(L, **kw) == INVALID, kw
    for kw in (dict(d=64), dict(block_size=8), dict(Hkv=65536), dict(num_blocks=1 << 27)):
        assert _bounds(L, **kw) == UNSUPPORTED, kw
    assert _bounds(L, N=0, kc=None, slot_map=None, bounds=None) == OK


def _select(L, **kw):
    p = dict(q=FAKE, bounds=FAKE, block_table=FAKE, ctx_len=FAKE, sel=FAKE, workspace=FAKE, ws_bytes=1 << 20, err_flag=None, dtype=0,
             B=2, Hq=8, Hkv=2, d=128, num_blocks=8, block_size=16, max_blocks=4, n_sel=3, n_first=1, n_last=1)
    p.update(kw)
    return call(L, "clo_paged_block_select", paged.BlockSelectArgs, p)


def test_select_rejects(L):
    for name in ("q", "bounds", "block_table", "ctx_len", "sel"):
        assert _select(L, **{name: None}) == INVALID, name
    for kw in (dict(q=FAKE + 8), dict(bounds=FAKE + 8), dict(block_table=FAKE + 2), dict(ctx_len=FAKE + 2), dict(sel=FAKE + 2),
               dict(err_flag=FAKE + 2), dict(B=-1), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(num_blocks=0), dict(max_blocks=0),
               dict(n_sel=0), dict(n_first=-1), dict(n_last=-1), dict(n_first=2, n_last=2), dict(n_first=(1 << 31) - 1, n_last=1),
               dict(dtype=2)):
        assert _select(L, **kw) == INVALID, kw
    for kw in (dict(d=64), dict(block_size=32), dict(Hq=18), dict(B=4097), dict(num_blocks=1 << 27), dict(n_sel=(1 << 20) + 1),
               dict(max_blocks=(1 << 20) + 1), dict(B=4096, Hkv=16, Hq=16)):
        assert _select(L, **kw) == UNSUPPORTED, kw
    need = clo.clo_paged_select_workspace_size(2, 2, 4)
    for kw in (dict(workspace=None), dict(workspace=FAKE + 8), dict(ws_bytes=need - 1)):
        assert _select(L, **kw) == WORKSPACE, kw
    assert _select(L, B=0, q=None, bounds=None, workspace=None) == OK


def test_binding_checks_before_the_library():
    """Host tensors and shapes that do not match are refused in Python."""
    t = torch.zeros(4, 2, 128).half()
    i = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros(8, 2, 16, 128).half()
    for fn, args in ((clo.clo_paged_rope_append, (t, t, t, i, torch.zeros(64, 2, dtype=torch.int64), i, cache, cache, t)),
                     (clo.clo_paged_chunk_attn, (t, cache, cache, i[None], i, i, t, i)),
                     (clo.clo_paged_block_bounds, (cache, i, i)),
                     (clo.clo_paged_block_select, (t, i, i, i, i, i)),
                     (clo.clo_paged_sparse_decode_attn, (t, cache, cache, i, i, i, t, i))):
        with pytest.raises(clo.CloError):
            fn(*args)


# ---------------------------------------------------------------- the references' own sense

def test_bounds_reference_is_an_upper_bound():
    """The score of a block is at least every exact score of its keys, up to the roundings of the codes."""
    g = torch.Generator().manual_seed(1)
    k, q = torch.randn(16, 128, generator=g).half(), torch.randn(1, 128, generator=g).half()
    codes, scale = ref.bounds_record(k)
    assert torch.equal(ref.unpack_record(ref.pack_records(codes, scale))[0], codes)
    code = ref.query_codes(q)
    step = float(q[0].float().abs().max()) / 127
    upper = float(torch.maximum(code * codes[0], code * codes[1]).sum()) * float(scale) * step
    rounding = 0.5 * step * float(k.float().abs().sum(1).max())
    assert upper >= float((k.double() @ q[0].double()).max()) - rounding
