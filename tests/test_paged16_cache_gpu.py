"""clo_paged_rope_append, clo_paged_block_bounds and clo_paged_block_select on the
GPU: rotations against 64 bits, records and selections exactly."""
import math

import pytest
import torch

import offloaded_kv_decode_gb300 as clo
import paged_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


def rand(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def freqs(rot, theta=10000.0):
    n = rot // 2
    return [theta ** (-i / n) for i in range(n)]


def append(q, k, v, pos, inv, axis, slots, num_blocks, inter, q_out=None):
    Hkv = k.shape[1]
    kc, vc = (torch.full((num_blocks, Hkv, 16, ref.D), 9.0, dtype=k.dtype, device="cuda") for _ in range(2))
    if q is not None and q_out is None:
        q_out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    clo.clo_paged_rope_append(q, k, v, pos, clo.clo_rope_pairs(inv, axis).cuda(), slots, kc, vc, q_out, interleaved=inter,
                              err_flag=err)
    torch.cuda.synchronize()
    return q_out, kc, vc, int(err.item())


def check_append(q, k, v, pos, inv, axis, slots, num_blocks, inter, q_in=None):
    got_q, kc, vc, err = append(q, k, v, pos, inv, axis, slots, num_blocks, inter)
    assert err == 0
    p2 = pos if pos.dim() == 2 else pos[None]
    ax = axis if axis is not None else [0] * len(inv)
    if q is not None:
        ref.check_rotated(got_q, *ref.rotate(q, p2, inv, ax, inter))
    want, size = ref.rotate(k, p2, inv, ax, inter)
    live = slots >= 0
    s = slots[live].long()
    rows = kc.transpose(1, 2).reshape(-1, k.shape[1], ref.D)
    ref.check_rotated(rows[s], want[live], size[live])
    vrows = vc.transpose(1, 2).reshape(-1, k.shape[1], ref.D)
    assert torch.equal(vrows[s], v[live])
    rest = torch.ones(len(rows), dtype=torch.bool, device="cuda")
    rest[s] = False
    assert torch.all(rows[rest] == 9) and torch.all(vrows[rest] == 9)  # nothing else is written


def scattered(N, seed, every=9):
    nb = N // 16 + 3
    g = torch.Generator().manual_seed(seed)
    slots = (torch.randperm(nb * 16, generator=g)[:N]).to(torch.int32)
    slots[::every] = -1
    return slots.cuda(), nb


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 64, 96, 112, 128])
def test_rotation(rot, inter, dtype):
    N = 33
    q, k, v = (rand(N, h, ref.D, dtype=dtype, seed=rot + i) for i, h in enumerate((6, 2, 2)))
    slots, nb = scattered(N, rot)
    pos = torch.randint(0, 5000, (N,), dtype=torch.int32, generator=torch.Generator().manual_seed(rot)).cuda()
    check_append(q, k, v, pos, freqs(rot), None, slots, nb, inter)


@pytest.mark.parametrize("N", [1, 2, 7, 100, 1000])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (40, 8), (3, 1), (32, 32), (7, 5)])
def test_sizes(N, Hq, Hkv):
    dtype = DTYPES[N % 2]
    q, k, v = (rand(N, h, ref.D, dtype=dtype, seed=N + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    slots, nb = scattered(N, N, every=N + 1)
    check_append(q, k, v, torch.arange(N, dtype=torch.int32, device="cuda"), freqs(128, 5e5), None, slots, nb, False)


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_and_negative_positions(dtype):
    N = 12
    k, v = (rand(N, 2, ref.D, dtype=dtype, seed=i) for i in range(2))
    pos = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 20 + 1, 10 ** 7, 2 ** 30, 2 ** 31 - 1, -2 ** 31, -12345, 131072, 999999], dtype=torch.int64)
    slots, nb = scattered(N, 3, every=100)
    check_append(None, k, v, pos.to(torch.int32).cuda(), freqs(128, 1e6), None, slots, nb, False)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_several_axes(axes, inter):
    N, n = 50, 48
    q, k, v = (rand(N, h, ref.D, dtype=torch.bfloat16, seed=axes + i) for i, h in enumerate((4, 2, 2)))
    pos = torch.randint(-100, 100000, (axes, N), dtype=torch.int32, generator=torch.Generator().manual_seed(axes)).cuda()
    slots, nb = scattered(N, axes)
    check_append(q, k, v, pos, freqs(2 * n), [i % axes for i in range(n)], slots, nb, inter)
    check_append(q, k, v, pos, freqs(2 * n), [min(i * axes // n, axes - 1) for i in range(n)], slots, nb, inter)


def test_parts_of_a_fused_projection_in_place():
    N, Hq, Hkv, dtype = 200, 8, 2, torch.float16
    qkv = rand(N, Hq + 2 * Hkv + 1, ref.D, dtype=dtype, seed=4)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:Hq + 2 * Hkv]
    slots, nb = scattered(N, 5)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    want_q, kc0, vc0, _ = append(q, k.contiguous(), v.contiguous(), pos, freqs(128), None, slots, nb, False)
    before = qkv.clone()
    got_q, kc, vc, err = append(q, k, v, pos, freqs(128), None, slots, nb, False, q_out=q)
    assert err == 0 and torch.equal(got_q, want_q) and torch.equal(kc, kc0) and torch.equal(vc, vc0)
    assert torch.equal(qkv[:, Hq:], before[:, Hq:])


def test_bad_slots_and_axes():
    N, dtype = 20, torch.float16
    q, k, v = (rand(N, 2, ref.D, dtype=dtype, seed=i) for i in range(3))
    slots, nb = scattered(N, 6, every=100)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    good = append(q, k, v, pos, freqs(64), None, slots, nb, False)
    s2 = slots.clone()
    s2[3], s2[4] = nb * 16, -2
    got = append(q, k, v, pos, freqs(64), None, s2, nb, False)
    assert got[3] == clo.FLAG_BAD_INDEX and torch.equal(got[0], good[0])
    rows = got[1].transpose(1, 2).reshape(-1, 2, ref.D)
    assert torch.all(rows[slots[3].long()] == 9) and torch.all(rows[slots[4].long()] == 9)
    keep = torch.tensor([i for i in range(N) if i not in (3, 4)], device="cuda")
    assert torch.equal(rows[slots[keep].long()], good[1].transpose(1, 2).reshape(-1, 2, ref.D)[slots[keep].long()])
    got = append(q, k, v, pos, freqs(64), [3] * 32, slots, nb, False)  # an axis that pos does not have counts as 0
    assert got[3] == clo.FLAG_BAD_INDEX and torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])


# ---------------------------------------------------------------- bounds

def runs(specs, seed):
    """Slots of requests with (first position in a block, tokens), blocks scattered; the number of blocks."""
    used, slots = 0, []
    for first, n in specs:
        slots.append(used * 16 + first + torch.arange(n))
        used += (first + n + 15) // 16
    slots = torch.cat(slots)
    perm = torch.randperm(used + 2, generator=torch.Generator().manual_seed(seed))
    return (perm[slots // 16] * 16 + slots % 16).to(torch.int32), used + 2


def bounds_ref(kc, slots, bounds):
    """The records after the call, on the host."""
    out = bounds.clone()
    sl = slots.tolist()
    for i, s in enumerate(sl):
        if s < 0 or s >= kc.shape[0] * 16 or not (s % 16 == 15 or i + 1 == len(sl) or sl[i + 1] != s + 1):
            continue
        for h in range(kc.shape[1]):
            codes, scale = ref.bounds_record(kc[s // 16, h, :s % 16 + 1])
            out[s // 16, h] = ref.pack_records(codes, scale)
    return out


def check_bounds(kc, slots, seed=0, want_err=0):
    bounds = torch.randint(0, 256, (*kc.shape[:2], ref.RECORD), dtype=torch.uint8, generator=torch.Generator().manual_seed(seed))
    got = bounds.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    clo.clo_paged_block_bounds(kc.cuda(), slots.cuda(), got, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == want_err
    assert torch.equal(got.cpu(), bounds_ref(kc, slots, bounds))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("specs", [[(0, 1)], [(0, 16)], [(15, 1)], [(3, 40), (0, 5), (15, 18)], [(r % 16, 1 + r % 20) for r in range(60)]])
def test_bounds(specs, dtype):
    slots, nb = runs(specs, len(specs))
    kc = torch.randn(nb, 3, 16, ref.D, generator=torch.Generator().manual_seed(nb)).to(dtype)
    kc += torch.randn(1, 3, 1, ref.D, generator=torch.Generator().manual_seed(1)).to(dtype) * 4
    check_bounds(kc, slots)


def test_bounds_of_many_tokens():
    """More tokens than the form for single tokens takes."""
    slots, nb = runs([(5, 4400)], 2)
    kc = torch.randn(nb, 8, 16, ref.D, generator=torch.Generator().manual_seed(2)).half()
    check_bounds(kc, slots)


@pytest.mark.parametrize("dtype", DTYPES)
def test_bounds_of_odd_keys(dtype):
    """Blocks of zeros, of one value, of the smallest and largest ones, of NaN and infinities, in and behind the tokens."""
    slots, nb = runs([(0, 16)] * 9 + [(0, 5)] * 3, 3)
    kc = torch.randn(nb, 2, 16, ref.D, generator=torch.Generator().manual_seed(3)).to(dtype)
    order = list(dict.fromkeys((slots // 16).tolist()))
    top, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    kc[order[0]] = 0
    kc[order[1]] = -0.0
    kc[order[2]] = 3.0
    kc[order[3]] = -2.5
    kc[order[4], :, 3] = top
    kc[order[5]] = tiny / 64 if dtype == torch.float16 else tiny / 128
    kc[order[6], 0, 2, 7] = math.nan
    kc[order[7], 1, 15, 127] = math.inf
    kc[order[8], 1, 0, 0] = -math.inf
    kc[order[9], :, 5:] = math.nan     # behind the last token
    kc[order[10], :, 5] = math.inf
    kc[order[11], :, 4] = math.nan     # the last token itself
    check_bounds(kc, slots)


def test_bounds_skip_and_report():
    kc = torch.randn(6, 2, 16, ref.D, generator=torch.Generator().manual_seed(3)).half()
    check_bounds(kc, torch.tensor([16, 17, -1, -5, 40, 41, 42], dtype=torch.int32))
    check_bounds(kc, torch.tensor([16, 17, 96, 40, 1 << 30], dtype=torch.int32), want_err=clo.FLAG_BAD_INDEX)


# ---------------------------------------------------------------- selection

def select(q, bounds, table, lens, n_sel, n_first, n_last):
    Hkv = bounds.shape[1]
    sel = torch.full((len(lens), Hkv, n_sel), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((clo.clo_paged_select_workspace_size(len(lens), Hkv, table.shape[1]),), 0xff, dtype=torch.uint8, device="cuda")
    clo.clo_paged_block_select(q, bounds, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), sel, ws, n_first, n_last,
                               err_flag=err)
    torch.cuda.synchronize()
    return sel.cpu(), int(err.item())


def random_bounds(nb, Hkv, seed, levels=127, scales=True):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(-levels, levels + 1, (nb, Hkv, 2, ref.D), generator=g)
    codes = torch.stack([c.amax(2), c.amin(2)], 2)
    scale = torch.rand(nb, Hkv, generator=g) * 0.1 if scales else torch.ones(nb, Hkv)
    return ref.pack_records(codes, scale)


def check_select(lens, G, Hkv, n_sel, n_first, n_last, dtype, seed, levels=127, scales=True, q=None):
    nb = [ref.blocks_of(n) for n in lens]
    g = torch.Generator().manual_seed(seed)
    total = sum(nb) + 2
    bounds = random_bounds(total, Hkv, seed, levels, scales)
    mb = max(max(nb), 1) + 2
    table = torch.full((len(lens), mb), -1, dtype=torch.int32)
    ids, at = torch.randperm(total, generator=g), 0
    for r, n in enumerate(nb):
        table[r, :n] = ids[at:at + n].to(torch.int32)
        at += n
    if q is None:
        q = torch.randn(len(lens), G * Hkv, ref.D, generator=g).to(dtype)
    sel, err = select(q.cuda(), bounds.cuda(), table.cuda(), lens, n_sel, n_first, n_last)
    assert err == 0
    for r, n in enumerate(nb):
        for h in range(Hkv):
            want = ref.select(q[r, h * G:(h + 1) * G], bounds[table[r, :n].long(), h], n, n_sel, n_first, n_last)
            assert sel[r, h].tolist() == want, (r, h)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,Hkv,n_sel,n_first,n_last", [(4, 2, 5, 1, 1), (1, 1, 1, 0, 0), (8, 3, 17, 4, 8), (5, 2, 64, 0, 1), (3, 1, 2, 1, 1)])
def test_select(G, Hkv, n_sel, n_first, n_last, dtype):
    check_select([1, 0, 300, 16 * n_sel, 16 * n_sel + 1, 2000, 90], G, Hkv, n_sel, n_first, n_last, dtype, n_sel)


def test_select_many_equal_scores():
    """Few different codes and one scale: most scores are equal, the lower blocks win."""
    q = torch.zeros(3, 4, ref.D).half()
    q[:, :, 3] = 1.0
    check_select([4000, 1700, 5000], 2, 2, 40, 1, 2, torch.float16, 5, levels=1, scales=False, q=q)


def test_select_queries_without_an_order():
    """Zero queries and queries that are not finite: all scores are equal."""
    q = torch.zeros(3, 2, ref.D).half()
    q[1, 0, 5] = math.nan
    q[2, :, 0], q[2, 0, 1] = 1.0, math.inf
    check_select([700, 700, 700], 1, 2, 10, 0, 1, torch.float16, 6, q=q)
    q = (q * 0 + 65504).nan_to_num(65504.0).bfloat16()
    check_select([700, 700, 700], 1, 2, 10, 0, 1, torch.bfloat16, 7, q=q)


def test_select_long_context():
    """More blocks than the selection holds in registers, and in one round."""
    check_select([16 * 9000 - 3], 2, 1, 300, 1, 1, torch.float16, 8)


def test_select_whole_tables_and_errors():
    bounds = random_bounds(40, 2, 9).cuda()
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    q = rand(2, 4, ref.D, dtype=torch.float16, seed=1)
    sel, err = select(q, bounds, table, [320, -1], 6, 1, 1)
    assert err == clo.FLAG_BAD_CTX and torch.all(sel[1] == -1) and torch.all(sel[0] >= 0)
    sel, err = select(q, bounds, table, [321, 100], 6, 1, 1)
    assert err == clo.FLAG_BAD_CTX and torch.all(sel[0] == -1)
    t2 = table.clone()
    t2[0, 11] = 40
    sel2, err = select(q, bounds, t2, [320, 100], 6, 1, 1)
    assert err == clo.FLAG_BAD_INDEX and (sel2[0] == 11).any(1).all()
    # a block with the scale of keys that are not finite is always selected
    b2 = bounds.clone()
    b2[7, :, :256] = 0
    b2[7, :, 256:260] = torch.tensor([math.inf]).view(torch.uint8).cuda()
    sel3, err = select(q, b2, table, [320, 100], 6, 1, 1)
    assert err == 0 and (sel3[0] == 7).any(1).all()


# ---------------------------------------------------------------- a run of them

def test_serving_steps():
    """Plan, append, chunk attention for two steps of ragged prompts and decoding
    tokens, then bounds, selection and sparse attention: every part against 64 bits,
    in one captured graph a step."""
    B, Hq, Hkv, dtype, mb = 3, 8, 2, torch.float16, 24
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table = torch.zeros(B, **i32), torch.full((B, mb), -1, **i32)
    ring = torch.randperm(80, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    state = torch.tensor([70, 80], **i32)
    start, offs, add = torch.empty(B, **i32), torch.empty(B + 1, **i32), torch.zeros(B, **i32)
    N = 400
    slots, pos = torch.empty(N, **i32), torch.zeros(N, **i32)
    kc, vc = (torch.full((80, Hkv, 16, ref.D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    bounds = torch.zeros(80, Hkv, ref.RECORD, dtype=torch.uint8, device="cuda")
    q, k, v = (torch.zeros(N, h, ref.D, dtype=dtype, device="cuda") for h in (Hq, Hkv, Hkv))
    q_rot, out = torch.zeros_like(q), torch.zeros_like(q)
    err = torch.zeros(1, **i32)
    ws = torch.empty(clo.clo_paged_chunk_workspace_size(Hq, Hkv), dtype=torch.uint8, device="cuda")
    pairs = clo.clo_rope_pairs(freqs(128)).cuda()
    calls = [clo.prepare_paged_plan(lens, add, table, ring, state, state, lens, start, offs, slots, err_flag=err),
             clo.prepare_paged_rope_append(q, k, v, pos, pairs, slots, kc, vc, q_rot, err_flag=err),
             clo.prepare_paged_block_bounds(kc, slots, bounds, err_flag=err),
             clo.prepare_paged_chunk_attn(q_rot, kc, vc, table, lens, offs, out, ws, err_flag=err)]
    graph = torch.cuda.CUDAGraph()
    for c in calls:  # loads the kernels
        c()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    host = [0] * B
    all_k = [torch.zeros(0, Hkv, ref.D, dtype=torch.float64, device="cuda") for _ in range(B)]
    for step, new in enumerate(([150, 1, 37], [60, 20, 1], [1, 1, 1])):
        g = torch.Generator().manual_seed(step)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(dtype))
        p = torch.cat([torch.arange(h, h + n) for h, n in zip(host, new)])
        pos[:len(p)] = p.to(torch.int32).cuda()
        add.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        host = [h + n for h, n in zip(host, new)]
        assert int(err.item()) == 0 and lens.tolist() == host and offs.tolist()[-1] == sum(new)
        n = sum(new)
        ref.check_rotated(q_rot[:n], *ref.rotate(q[:n], pos[None, :n], freqs(128), [0] * 64, False))
        ref.check_attention(out[:n], None, ref.chunk_attention(q_rot[:n], kc, vc, table, host, new), max(host))
        turned, size = ref.rotate(k[:n], pos[None, :n], freqs(128), [0] * 64, False)
        at = 0
        for r, m in enumerate(new):
            all_k[r] = torch.cat([all_k[r], turned[at:at + m]])
            have = ref.cached(kc, table, r, host[r]).transpose(0, 1)
            assert (have - all_k[r]).abs().max() < 4e-3  # half a step at 4 to 8, and the angle
            at += m
    # the last step again, over selected blocks
    q1 = q_rot[:B].contiguous()
    sel = torch.empty(B, Hkv, 4, **i32)
    sws = torch.empty(clo.clo_paged_select_workspace_size(B, Hkv, mb), dtype=torch.uint8, device="cuda")
    o1 = torch.empty_like(q1)
    clo.clo_paged_block_select(q1, bounds, table, lens, sel, sws, 1, 1, err_flag=err)
    clo.clo_paged_sparse_decode_attn(q1, kc, vc, table, lens, sel, o1, ws, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    G = Hq // Hkv
    for r in range(B):
        nb = ref.blocks_of(host[r])
        for h in range(Hkv):
            rec = torch.stack([ref.pack_records(*ref.bounds_record(kc[table[r, p], h, :min(16, host[r] - 16 * p)].cpu()))
                               for p in range(nb)])
            assert torch.equal(rec, bounds[table[r, :nb].long(), h].cpu())
            assert sel[r, h].tolist() == ref.select(q1[r, h * G:(h + 1) * G].cpu(), rec, nb, 4, 1, 1)
            tok = [c * 16 + i for c in sel[r, h].tolist() if c >= 0 for i in range(16) if c * 16 + i < host[r]]
            kk, vv = (ref.cached(x, table, r, host[r])[h][tok] for x in (kc, vc))
            o, e, mag, size = ref.attend_clean(q1[r, h * G:(h + 1) * G].double(), kk, vv, 1 / math.sqrt(ref.D))
            ref.check_attention(o1[r, h * G:(h + 1) * G], None, (o, e, mag, size), 64)
