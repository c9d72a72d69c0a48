"""What the 4-bit cache's calls leave alone, that a repeated call gives the same
bits, and that a long draft may be scored in parts."""
import numpy as np
import pytest
import torch

import kv4_case
import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev
from test_kv4_attention_gpu import assert_matches, inputs
from test_kv4_cache_gpu import append, rows

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def row_bytes(shape, slots, group):
    """Mask of a pool's bytes that the rows of `slots` own: (codes, pairs)."""
    codes, pairs = np.zeros(shape, bool), np.zeros(shape, bool)
    ng = 128 // group
    for s in slots:
        b, t = s // 16, s % 16
        codes[b, :, t * 64:(t + 1) * 64] = True
        codes[b, :, 1024 + t * 64:1024 + (t + 1) * 64] = True
        pairs[b, :, 2048 + t * 8 * ng:2048 + (t + 1) * 8 * ng] = True
    return codes, pairs


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,Hkv,fused", [(1, 1, True), (17, 3, False), (133, 8, True), (700, 2, False), (250, 5, True)])
def test_append_writes_its_rows_and_no_other_byte(N, Hkv, fused, group, dtype):
    k, v = rows(N, Hkv, DT[dtype], 7 * N + group, fused)
    nb = N // 16 + 3
    g = torch.Generator().manual_seed(N + 1)
    slots = torch.randperm(nb * 16, generator=g)[:N].to(torch.int32)
    slots[N // 2:N // 2 + N // 10] = -1
    pool = torch.randint(0, 256, (nb, Hkv, ref.record_bytes(group)), dtype=torch.uint8, generator=g)
    want = pool.numpy().copy()
    pool = pool.to(dev())
    assert append(k, v, slots.to(dev()), pool) == 0
    ref.write_rows(want, slots.numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), group)
    differ = pool.cpu().numpy() != want
    codes, pairs = row_bytes(want.shape, [s for s in slots.tolist() if s >= 0], group)
    assert not differ[~codes].any()   # other rows' bytes, and the pairs bit for bit
    assert pairs.sum() == (slots >= 0).sum().item() * Hkv * 8 * (128 // group)
    assert differ[codes].sum() <= 2   # quotients next to the border between two codes


@pytest.mark.parametrize("num_ctas", [0, 5])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_writes_its_outputs_and_no_other_byte(dtype, num_ctas):
    """Guards around out, lse and the workspace stay as they are, and so do the
    inputs; every output is written."""
    dt = DT[dtype]
    for ctx, n_q, Hq, Hkv in (([300, 0, 17], 1, 8, 2), ([5, 600], 3, 10, 2), ([2000], 1, 7, 7), ([40, 700], 4, 8, 1)):
        q, pool, table, c = inputs(ctx, n_q, Hq, Hkv, 64, dt, 5)
        q, pool = q.to(dev()), torch.as_tensor(pool).to(dev())
        table, c = (torch.as_tensor(x, dtype=torch.int32).to(dev()) for x in (table, c))
        held = [x.clone() for x in (q, pool, table, c)]
        size = clo.clo_kv4_paged_workspace_size(len(ctx), n_q, Hq, Hkv, 128, num_ctas)
        buffers = []
        for n, t in ((q.numel(), dt), (q.numel() // 128, torch.float32), (size, torch.uint8)):
            whole = torch.full((n + 512,), 77, dtype=t, device=dev())
            buffers.append((whole, whole[256:256 + n]))
        out, lse = buffers[0][1].view(q.shape), buffers[1][1]
        for _ in range(3):
            buffers[0][1].fill_(float("nan"))
            lse.fill_(float("nan"))
            clo.clo_kv4_paged_decode_attn(q, pool, table, c, out, buffers[2][1], lse=lse, num_ctas=num_ctas)
        for whole, mine in buffers:
            assert torch.all(whole[:256] == 77) and torch.all(whole[-256:] == 77)
        assert torch.all(torch.isfinite(out)) and not torch.isnan(lse).any()
        for x, y in zip((q, pool, table, c), held):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gather_writes_its_rows_and_no_other_byte(dtype):
    dt = DT[dtype]
    for N, Hkv in ((1, 1), (13, 3), (130, 8)):
        pool = torch.zeros(9, Hkv, ref.record_bytes(32), dtype=torch.uint8, device=dev())
        slots = torch.arange(N, dtype=torch.int32, device=dev())
        whole = [torch.full((N * Hkv * 128 + 512,), 77.0, dtype=dt, device=dev()) for _ in range(2)]
        k, v = (w[256:-256].view(N, Hkv, 128) for w in whole)
        clo.clo_kv4_gather(pool, slots, k, v)
        for w in whole:
            assert torch.all(w[:256] == 77) and torch.all(w[-256:] == 77) and torch.all(w[256:-256] == 0)


@pytest.mark.parametrize("num_ctas", [0, 1, 7, 150, 700])
def test_a_repeated_call_gives_the_same_bits(num_ctas):
    """Also where the tokens are shared out evenly and pieces are merged, and with
    another workspace's contents."""
    q, pool, table, ctx = inputs([5000, 17, 1200, 0, 640, 3333], 1, 32, 8, 64, torch.float16, 18, mb=900)
    q, pool = q.to(dev()), torch.as_tensor(pool).to(dev())
    table, ctx = (torch.as_tensor(x, dtype=torch.int32).to(dev()) for x in (table, ctx))
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=dev())
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(6, 1, 32, 8, 128, num_ctas), dtype=torch.uint8, device=dev())
    first = None
    for i in range(12):
        ws.fill_(i * 23)
        out.fill_(float("nan"))
        clo.clo_kv4_paged_decode_attn(q, pool, table, ctx, out, ws, lse=lse, num_ctas=num_ctas)
        now = out.view(torch.int16).clone(), lse.view(torch.int32).clone()
        first = first or now
        assert torch.equal(now[0], first[0]) and torch.equal(now[1], first[1])


def test_a_long_draft_in_two_calls():
    """5 drafted tokens with 8 query heads a KV head: 40 query rows are refused,
    and are 24 with two tokens less and 16."""
    q, pool, table, ctx = inputs([0, 1, 2, 3, 4, 5, 17, 300], 5, 16, 2, 64, torch.float16, 3)
    want = ref.attention(q.double().numpy(), pool, table, ctx, 64, ref.scale_for(), torch.float16)
    qd, pool = q.to(dev()), torch.as_tensor(pool).to(dev())
    table, c = (torch.as_tensor(x, dtype=torch.int32).to(dev()) for x in (table, ctx))
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(8, 3, 16, 2), dtype=torch.uint8, device=dev())
    with pytest.raises(clo.CloError):
        clo.clo_kv4_paged_decode_attn(qd, pool, table, c, torch.empty_like(qd), ws)
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    got, lse = [], []
    for lo, hi in ((0, 3), (3, 5)):
        part = qd[:, lo:hi].contiguous()
        out, ls = torch.empty_like(part), torch.empty(part.shape[:3], device=dev())
        clo.clo_kv4_paged_decode_attn(part, pool, table, (c - (5 - hi)).clamp_(min=0), out, ws, lse=ls, err_flag=err)
        got.append(out)
        lse.append(ls)
    assert int(err.item()) == 0
    assert_matches(torch.cat(got, 1).double().cpu().numpy(), torch.cat(lse, 1).double().cpu().numpy(), want)


@pytest.mark.parametrize("name", ["gather_1000", "attn_b1_1k"])
def test_a_case_runs_for_a_profiler(name):
    assert kv4_case.main(name, 2) == 0
