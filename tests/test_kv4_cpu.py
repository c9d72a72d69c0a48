"""The 4-bit paged cache's entry points without a GPU: the exported symbols,
what each call refuses before it launches anything, and the reference's own
layout and quantiser."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from offloaded_kv_decode_gb300 import build as libbuild
from offloaded_kv_decode_gb300 import kv4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned non-null stand-in pointer: never dereferenced on these paths
INVALID, UNSUPPORTED = clo.CLO_ERR_INVALID_ARG, clo.CLO_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return clo.lib()


def test_header_and_library_agree(L):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "clo_kv4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(clo_[a-z0-9_]+)\s*\(", text))
    assert names == {"clo_kv4_block_bytes", "clo_paged_plan", "clo_kv4_append", "clo_kv4_gather",
                     "clo_kv4_paged_workspace_size", "clo_kv4_paged_decode_attn"}
    for n in names:
        assert hasattr(L, n) and hasattr(clo, n)
    assert int(re.search(r"CLO_FLAG_NO_ROOM (0x[0-9a-f]+)", text).group(1), 16) == clo.FLAG_NO_ROOM == ref.NO_ROOM
    assert clo.check_error_flag(clo.FLAG_NO_ROOM) == clo.CLO_ERR_BAD_INDEX


def test_structs_match_the_header(tmp_path):
    """Sizes and offsets of the argument structs as a C compiler lays them out."""
    structs = {"clo_paged_plan_args": kv4.PlanArgs, "clo_kv4_append_args": kv4.AppendArgs,
               "clo_kv4_gather_args": kv4.GatherArgs, "clo_kv4_attn_args": kv4.AttnArgs}
    lines = []
    for name, t in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f[0]}));' for f in t._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "clo_kv4.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0; }\n")
    cuda = os.path.join(os.path.dirname(os.path.dirname(libbuild.nvcc_path())), "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", cuda, str(src),
                    "-o", str(tmp_path / "layout")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, check=True).stdout.split()]
    want = []
    for t in structs.values():
        want.append(ctypes.sizeof(t))
        want += [getattr(t, f[0]).offset for f in t._fields_]
    assert got == want


def test_record_sizes(L):
    for group in clo.KV4_GROUPS:
        assert clo.clo_kv4_block_bytes(group) == ref.record_bytes(group)
        assert clo.clo_kv4_block_bytes(group) % 128 == 0
    assert clo.clo_kv4_block_bytes(16) == 0
    assert clo.clo_kv4_block_bytes(64, block_size=32) == 0
    assert clo.clo_kv4_block_bytes(64, d=64) == 0


def call(L, what, struct, values):
    return getattr(L, what)(ctypes.byref(struct(**values)), None)


def _plan(L, B=4, bs=16, mb=8, rs=64, mn=32, **kw):
    p = dict(len_in=FAKE, keep=None, add=FAKE, block_table=FAKE, free_ring=FAKE, ring_in=FAKE, ring_out=FAKE,
             len_out=FAKE, start=FAKE, offsets=FAKE, slot_map=FAKE, B=B, block_size=bs, max_blocks=mb, ring_size=rs,
             max_new=mn)
    p.update(kw)
    return call(L, "clo_paged_plan", kv4.PlanArgs, p)


def test_no_arguments(L):
    for what in ("clo_paged_plan", "clo_kv4_append", "clo_kv4_gather", "clo_kv4_paged_decode_attn"):
        assert getattr(L, what)(None, None) == INVALID


def test_plan_rejects(L):
    for name in ("len_in", "add", "block_table", "free_ring", "ring_in", "ring_out", "len_out", "start", "offsets",
                 "slot_map"):
        assert _plan(L, **{name: None}) == INVALID, name
        assert _plan(L, **{name: FAKE + 2}) == INVALID, name
    assert _plan(L, keep=FAKE + 1) == INVALID
    assert _plan(L, B=-1) == INVALID
    assert _plan(L, mb=0) == INVALID
    assert _plan(L, rs=0) == INVALID
    assert _plan(L, mn=-1) == INVALID
    assert _plan(L, bs=32) == UNSUPPORTED
    assert _plan(L, B=4097) == UNSUPPORTED
    assert _plan(L, B=4096, mb=1 << 15) == UNSUPPORTED  # positions past 32 bits
    assert _plan(L, mn=(1 << 30) + 1) == UNSUPPORTED
    assert _plan(L, rs=(1 << 30) + 1) == UNSUPPORTED


def _append(L, k=FAKE, v=FAKE, ks=1024, vs=1024, dt=0, slots=FAKE, N=4, Hkv=8, d=128, pool=FAKE, nb=16, bs=16,
            group=64, err=None):
    return call(L, "clo_kv4_append", kv4.AppendArgs, dict(
        k=k, v=v, k_stride=ks, v_stride=vs, slot_map=slots, pool=pool, err_flag=err, dtype=dt, N=N, Hkv=Hkv, d=d,
        num_blocks=nb, block_size=bs, group=group))


def test_append_rejects(L):
    for name in ("k", "v", "slots", "pool"):
        assert _append(L, **{name: None}) == INVALID, name
    assert _append(L, k=FAKE + 8) == INVALID
    assert _append(L, pool=FAKE + 8) == INVALID
    assert _append(L, slots=FAKE + 2) == INVALID
    assert _append(L, err=FAKE + 2) == INVALID
    assert _append(L, ks=1016) == INVALID       # rows overlap
    assert _append(L, vs=1028) == INVALID       # rows off the 16-byte grid
    assert _append(L, dt=2) == INVALID
    assert _append(L, N=-1) == INVALID
    assert _append(L, Hkv=0) == INVALID
    assert _append(L, nb=0) == INVALID
    assert _append(L, d=64) == UNSUPPORTED
    assert _append(L, bs=32) == UNSUPPORTED
    assert _append(L, group=16) == UNSUPPORTED
    assert _append(L, N=1 << 30) == UNSUPPORTED
    assert _append(L, N=0, k=None, v=None, slots=None, pool=None) == clo.CLO_OK
    assert _append(L, N=0, ks=0, vs=0) == clo.CLO_OK


def _gather(L, k=FAKE, v=FAKE, dt=0, slots=FAKE, N=4, Hkv=8, d=128, pool=FAKE, nb=16, bs=16, group=64):
    return call(L, "clo_kv4_gather", kv4.GatherArgs, dict(
        pool=pool, slot_map=slots, k=k, v=v, dtype=dt, N=N, Hkv=Hkv, d=d, num_blocks=nb, block_size=bs, group=group))


def test_gather_rejects(L):
    for name in ("k", "v", "slots", "pool"):
        assert _gather(L, **{name: None}) == INVALID, name
    assert _gather(L, v=FAKE + 8) == INVALID
    assert _gather(L, dt=-1) == INVALID
    assert _gather(L, N=-1) == INVALID
    assert _gather(L, d=96) == UNSUPPORTED
    assert _gather(L, group=256) == UNSUPPORTED
    assert _gather(L, N=0) == clo.CLO_OK


def _attn(L, q=FAKE, dt=0, pool=FAKE, bt=FAKE, mb=8, cl=FAKE, nb=64, B=4, n_q=1, Hq=32, Hkv=8, d=128, bs=16,
          group=64, scale=0.088, out=FAKE, lse=None, ws=FAKE, wsb=1 << 40, num_ctas=7):
    opts = clo.AttnOpts(num_ctas, None, None)
    return call(L, "clo_kv4_paged_decode_attn", kv4.AttnArgs, dict(
        q=q, pool=pool, block_table=bt, ctx_len=cl, out=out, lse=lse, workspace=ws, ws_bytes=wsb,
        opts=ctypes.addressof(opts), dtype=dt, scale=scale, B=B, n_q=n_q, Hq=Hq, Hkv=Hkv, d=d, num_blocks=nb,
        block_size=bs, max_blocks=mb, group=group))


def test_attention_rejects(L):
    for name in ("q", "pool", "bt", "cl", "out"):
        assert _attn(L, **{name: None}) == INVALID, name
    assert _attn(L, q=FAKE + 8) == INVALID
    assert _attn(L, lse=FAKE + 2) == INVALID
    assert _attn(L, Hq=30) == INVALID
    assert _attn(L, n_q=0) == INVALID
    assert _attn(L, mb=0) == INVALID
    assert _attn(L, nb=0) == INVALID
    assert _attn(L, dt=3) == INVALID
    assert _attn(L, num_ctas=-1) == INVALID
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _attn(L, scale=scale) == INVALID
    assert _attn(L, d=64) == UNSUPPORTED
    assert _attn(L, bs=32) == UNSUPPORTED
    assert _attn(L, group=8) == UNSUPPORTED
    assert _attn(L, n_q=9) == UNSUPPORTED            # 4 * 9 query rows
    assert _attn(L, Hq=264, Hkv=8) == UNSUPPORTED    # 33 query rows
    assert _attn(L, B=4097) == UNSUPPORTED
    assert _attn(L, B=4096, Hkv=64, Hq=64, mb=1 << 14) == UNSUPPORTED
    assert _attn(L, ws=None) == clo.CLO_ERR_WORKSPACE
    assert _attn(L, ws=FAKE + 8) == clo.CLO_ERR_WORKSPACE
    need = clo.clo_kv4_paged_workspace_size(4, 1, 32, 8, 128, 7)
    assert need > 0 and _attn(L, wsb=need - 1) == clo.CLO_ERR_WORKSPACE
    assert _attn(L, B=0) == clo.CLO_OK


def test_workspace_size_of_invalid_sizes(L):
    assert clo.clo_kv4_paged_workspace_size(1, 1, 30, 8, 128, 4) == 0
    assert clo.clo_kv4_paged_workspace_size(1, 0, 32, 8, 128, 4) == 0
    assert clo.clo_kv4_paged_workspace_size(1, 9, 32, 8, 128, 4) == 0
    assert clo.clo_kv4_paged_workspace_size(1, 1, 32, 8, 64, 4) == 0
    assert clo.clo_kv4_paged_workspace_size(1, 1, 32, 8, 128, -1) == 0


def test_binding_checks_tensors():
    """Host tensors, wrong types and shapes never reach the library."""
    i32 = torch.zeros(4, dtype=torch.int32)
    kv = torch.zeros(4, 2, 128, dtype=torch.float16)
    pool = torch.zeros(3, 2, 2304, dtype=torch.uint8)
    for call in (lambda: clo.clo_kv4_append(kv, kv, i32, pool),
                 lambda: clo.clo_kv4_append(kv.float(), kv, i32, pool),
                 lambda: clo.clo_kv4_gather(pool, i32, kv, kv),
                 lambda: clo.clo_kv4_paged_decode_attn(kv, pool, i32.view(2, 2), i32, kv, pool),
                 lambda: clo.clo_paged_plan(i32, i32, i32.view(2, 2), i32, i32[:2], i32[:2], i32, i32, i32, i32)):
        with pytest.raises(clo.CloError) as e:
            call()
        assert e.value.status == INVALID


@pytest.mark.parametrize("group", [32, 64, 128])
def test_reference_layout_covers_every_nibble_once(group):
    seen = set()
    for places in (ref.KB, ref.VB):
        seen |= {(int(b), int(s)) for b, s in zip(places.ravel(), ref.SH.ravel())}
    assert seen == {(b, s) for b in range(2048) for s in (0, 4)}


@pytest.mark.parametrize("group", [32, 64, 128])
def test_reference_quantiser_bounds(group):
    """Codes 0..15, no element off by more than half a scale, and the same rows
    read back from the layout."""
    rng = np.random.Generator(np.random.PCG64(group))
    k = rng.standard_normal((20, 3, 128)).astype(np.float16).astype(np.float64)
    k[3, 1] = 2.5                      # a constant row
    k[4, 0, :group] = np.nan
    v = 1e-6 * k                       # scales among the smallest fp16 values
    v = v.astype(np.float16).astype(np.float64)
    codes, scale, zero, _ = ref.quantise(k, group)
    assert codes.min() >= 0 and codes.max() <= 15
    pool = np.zeros((3, 3, ref.record_bytes(group)), np.uint8)
    slots = rng.permutation(48)[:20]
    ref.write_rows(pool, slots, k, v, group)
    kk, vv = ref.values(pool, group)
    for x, got in ((k, kk), (v, vv)):
        _, s, _, _ = ref.quantise(x, group)
        back = got[slots // 16, :, slots % 16]
        half = np.repeat(s.astype(np.float64), group, -1) / 2
        bad = np.isnan(half)
        assert np.array_equal(np.isnan(back), bad)
        assert np.all(np.abs(back - x)[~bad] <= half[~bad] * (1 + 1e-12))


def test_reference_plan_on_a_worked_example():
    """Two requests: one grows over a block's end, one drops a draft and ends a block earlier."""
    table = np.array([[4, -1], [2, 3]])
    ring = np.array([9, 7, 5, -1, -1, -1])
    got, err = ref.plan([16, 18], [16, 15], [2, 0], table, ring, [1, 2], 4)
    assert err == 0
    assert got["len_out"].tolist() == [18, 15] and got["start"].tolist() == [16, 15]
    assert got["block_table"].tolist() == [[4, 7], [2, 3]]
    assert got["slot_map"].tolist() == [7 * 16, 7 * 16 + 1, -1, -1]
    assert got["offsets"].tolist() == [0, 2, 2]
    assert got["free_ring"].tolist() == [9, 7, 5, 3, -1, -1] and got["ring_out"].tolist() == [2, 2]
