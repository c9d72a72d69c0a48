"""The paged 4-bit cache as a decode loop uses it: plan, append and attention
of each step, with prompts, drafts and ended requests, against attention in 64
bits over the rows as the reference quantises them."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("group,dt", [(64, torch.float16), (32, torch.bfloat16)])
def test_decode_loop(group, dt, captured):
    B, Hq, Hkv, mb, n_q, max_new, layers = 5, 8, 2, 10, 2, 120, 2
    rng = np.random.Generator(np.random.PCG64(group))
    nb = 64
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev())  # noqa: E731
    length, keep, add, start, offsets = i32(B), i32(B), i32(B), i32(B), i32(B + 1)
    table, slots, err = torch.full((B, mb), -1, dtype=torch.int32, device=dev()), i32(max_new), i32(1)
    ring, state = torch.randperm(nb, device=dev()).to(torch.int32), torch.tensor([nb - 3, nb], dtype=torch.int32, device=dev())
    pools = [torch.zeros(nb, Hkv, ref.record_bytes(group), dtype=torch.uint8, device=dev()) for _ in range(layers)]
    qkv = [torch.zeros(max_new, (Hq + 2 * Hkv) * 128, dtype=dt, device=dev()) for _ in range(layers)]
    q = [torch.zeros(B, n_q, Hq, 128, dtype=dt, device=dev()) for _ in range(layers)]
    out = [torch.zeros_like(x) for x in q]
    lse = [torch.zeros(B, n_q, Hq, device=dev()) for _ in range(layers)]
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(B, n_q, Hq, Hkv), dtype=torch.uint8, device=dev())
    ko, vo = (torch.zeros(max_new, Hkv, 128, dtype=dt, device=dev()) for _ in range(2))
    calls = [clo.prepare_paged_plan(length, add, table, ring, state, state, length, start, offsets, slots, keep=keep,
                                    err_flag=err)]
    for i in range(layers):
        k = qkv[i][:, Hq * 128:(Hq + Hkv) * 128].view(max_new, Hkv, 128)
        v = qkv[i][:, (Hq + Hkv) * 128:].view(max_new, Hkv, 128)
        calls.append(clo.prepare_kv4_append(k, v, slots, pools[i], err_flag=err))
        calls.append(clo.prepare_kv4_paged_decode_attn(q[i], pools[i], table, length, out[i], ws, lse=lse[i],
                                                       err_flag=err))
    calls.append(clo.prepare_kv4_gather(pools[-1], slots, ko, vo, err_flag=err))

    def step():
        for c in calls:
            c()

    graph = None
    held = [[[] for _ in range(B)] for _ in range(layers)]  # rows (k, v) of each request, as appended
    now = np.zeros(B, int)
    for s in range(9):
        if s == 0:
            kp, ad = np.zeros(B, int), np.array([37, 1, 16, 0, 45])
        else:
            kp = np.maximum(now - rng.integers(0, n_q, B), 0)
            ad = np.where(now > 0, rng.integers(1, n_q + 1, B), rng.integers(0, 20, B))
            if s % 4 == 0:
                kp[s % B], ad[s % B] = 0, 0  # a request ends
        keep.copy_(torch.from_numpy(kp).to(torch.int32))
        add.copy_(torch.from_numpy(ad).to(torch.int32))
        for i in range(layers):
            qkv[i].copy_(torch.from_numpy(rng.standard_normal(qkv[i].shape)))
            q[i].copy_(torch.from_numpy(rng.standard_normal(q[i].shape)))
        if captured and s == 1:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        now = kp + ad
        assert length.cpu().numpy().tolist() == now.tolist()
        off = np.concatenate([[0], np.cumsum(ad)])
        for i in range(layers):
            rows = qkv[i].double().cpu().numpy()[:, Hq * 128:].reshape(max_new, 2, Hkv, 128)
            for r in range(B):
                held[i][r] = held[i][r][:kp[r]] + [rows[n] for n in range(off[r], off[r + 1])]
            # The same rows in a cache of the reference's, request after request.
            mine = np.zeros((B * mb, Hkv, ref.record_bytes(group)), np.uint8)
            tab = np.arange(B * mb).reshape(B, mb)
            for r in range(B):
                if now[r]:
                    kv = np.stack(held[i][r])
                    ref.write_rows(mine, r * mb * 16 + np.arange(now[r]), kv[:, 0], kv[:, 1], group)
            o, l, tol, ltol = ref.attention(q[i].double().cpu().numpy(), mine, tab, now, group, ref.scale_for(), dt)
            got, gl = out[i].double().cpu().numpy(), lse[i].double().cpu().numpy()
            assert np.all(np.abs(got - o) <= tol)
            seen = np.isfinite(l)
            assert np.array_equal(np.isneginf(gl), ~seen) and np.all(np.abs(gl[seen] - l[seen]) <= ltol[seen])
        # The last layer's new rows read back; the padding is zeros.
        n = off[-1]
        got = ko.double().cpu().numpy()
        _, sc, z, _ = ref.quantise(rows[:n, 0], group)
        half = np.repeat(sc.astype(np.float64), group, -1) / 2
        assert np.all(np.abs(got[:n] - rows[:n, 0]) <= half * (1 + 1e-6) + ref.U16[dt] * (np.abs(rows[:n, 0]) + half) + 1e-7)
        assert np.all(got[n:] == 0) and torch.all(vo[n:] == 0)
