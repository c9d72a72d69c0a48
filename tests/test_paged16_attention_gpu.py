"""clo_paged_chunk_attn and clo_paged_sparse_decode_attn against attention in 64 bits."""
import math

import pytest
import torch

import offloaded_kv_decode_gb300 as clo
import paged_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


def offsets_of(n_new):
    return torch.tensor([0] + n_new, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def chunk(q, kc, vc, table, lens, n_new, num_ctas=0, scale=None, lse=True, offsets=None, fill=float("nan")):
    out = torch.full(q.shape, fill, dtype=q.dtype, device="cuda")
    e = torch.full(q.shape[:2], fill, device="cuda") if lse else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((clo.clo_paged_chunk_workspace_size(q.shape[1], kc.shape[1], num_ctas=num_ctas),), 0xff, dtype=torch.uint8,
                    device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clo.clo_paged_chunk_attn(q, kc, vc, table, ctx, offsets_of(n_new) if offsets is None else offsets, out, ws, lse=e,
                             err_flag=err, num_ctas=num_ctas, scale=scale)
    torch.cuda.synchronize()
    return out, e, int(err.item())


def queries(N, Hq, dtype, seed, size=1.0):
    return (torch.randn(N, Hq, ref.D, generator=torch.Generator().manual_seed(seed)) * size).to(dtype).cuda()


def check(lens, n_new, Hq, Hkv, dtype, seed=1, num_ctas=0, size=1.0, fill=float("nan"), scale=None):
    kc, vc, table = ref.make_cache(lens, Hkv, dtype, seed, fill=fill)
    q = queries(sum(n_new), Hq, dtype, seed + 1, size)
    out, lse, err = chunk(q, kc, vc, table, lens, n_new, num_ctas, scale)
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, lens, n_new, scale), max(lens))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [(1, 1), (2, 1), (15, 15), (16, 1), (17, 16), (127, 1), (128, 128), (129, 3), (200, 64), (255, 255),
                                 (256, 33), (257, 257), (640, 1), (1000, 129), (1024, 16), (1500, 700)])
def test_one_request(T, n, dtype):
    check([T], [n], 8, 2, dtype, seed=T + n)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("Hkv,n", [(1, 1), (3, 40), (2, 130)])
def test_head_layouts(G, Hkv, n):
    check([n + 37, n, n + 300], [n, n, max(1, n // 2)], G * Hkv, Hkv, DTYPES[G % 2], seed=G * 10 + Hkv)


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 40, 151, 200])
def test_splits_of_the_work(num_ctas):
    check([1, 700, 0, 300, 2049, 16], [1, 650, 0, 1, 31, 16], 10, 2, torch.float16, seed=num_ctas, num_ctas=num_ctas)


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_context_few_rows(dtype):
    check([20000, 33], [1, 2], 8, 2, dtype, seed=5)
    check([9000], [9], 16, 2, dtype, seed=6)


def test_mixture_of_many_requests():
    g = torch.Generator().manual_seed(3)
    n_new = torch.randint(0, 4, (300,), generator=g).tolist()
    n_new[17], n_new[200] = 90, 257
    lens = [n + int(torch.randint(0, 200, (1,), generator=g)) for n in n_new]
    check(lens, n_new, 8, 2, torch.bfloat16, seed=9)


def test_4096_requests():
    lens = [(7 * r) % 40 + 1 for r in range(4096)]
    check(lens, [1] * 4096, 2, 1, torch.float16, seed=11)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_see_nothing(dtype):
    """More new tokens than cached ones: the first rows see no token."""
    kc, vc, table = ref.make_cache([3, 0, 40], 2, dtype, 4, fill=float("nan"))
    n_new = [10, 5, 130]
    q = queries(sum(n_new), 8, dtype, 2)
    out, lse, err = chunk(q, kc, vc, table, [3, 0, 40], n_new)
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, [3, 0, 40], n_new), 40)
    assert torch.all(out[:7] == 0) and torch.all(torch.isneginf(lse[:7])) and torch.all(out[10:15] == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [0.0, 1e-3, 8.0, 60.0])
def test_flat_and_sharp_weights(size, dtype):
    check([700], [200], 4, 1, dtype, seed=21, size=size)


@pytest.mark.parametrize("dtype", DTYPES)
def test_short_contexts_are_as_exact_as_the_output(dtype):
    """Up to 128 tokens the weights have twice the bits: what is left is the output's own
    rounding, the scores' and the sums' in fp32."""
    lens, n_new = [2, 3, 5, 17, 40, 128, 100], [2, 1, 5, 17, 8, 128, 60]
    kc, vc, table = ref.make_cache(lens, 2, dtype, 23, fill=float("nan"))
    q = queries(sum(n_new), 8, dtype, 24)
    out, lse, err = chunk(q, kc, vc, table, lens, n_new)
    assert err == 0
    want, _, mag, size = ref.chunk_attention(q, kc, vc, table, lens, n_new)
    d = 2.0 ** -19 * size + 2.0 ** -20
    tol = ref.half_step(dtype) * want.abs() + (2.0 ** -15 + 2 * d[..., None] + 16 * 2.0 ** -23) * mag + 2.0 ** -24
    assert ((out.double() - want).abs() <= tol).all()


def test_rising_scores():
    """Each token outweighs all before it: the running maximum moves at every step."""
    T, dtype = 600, torch.float16
    kc, vc, table = ref.make_cache([T], 1, dtype, 8)
    q = queries(T, 2, dtype, 9, 0.0)
    q[..., 0] = 30.0
    for t in range(T):
        kc[table[0, t // 16].long(), 0, t % 16] = 0
        kc[table[0, t // 16].long(), 0, t % 16, 0] = 0.5 * t
    out, lse, err = chunk(q, kc, vc, table, [T], [T])
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, [T], [T]), T)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_does_not_enter(bad, dtype):
    """NaN and infinities in tokens that only later rows see, and behind the last token."""
    T, n, G = 400, 300, 4
    kc, vc, table = ref.make_cache([T], 2, dtype, 31, fill=bad)
    for t, x in ((350, kc), (377, vc)):
        x[table[0, t // 16].long(), 1, t % 16, 5] = bad
    q = queries(n, 2 * G, dtype, 32)
    want = ref.chunk_attention(q, kc, vc, table, [T], [n])
    for num_ctas in (0, 1):
        out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
        assert err == 0
        first = 350 - (T - n)  # the first row of head 1 that sees one of them
        ref.check_attention(out[:, :G], lse[:, :G], tuple(x[:, :G] for x in want), T)
        ref.check_attention(out[:first, G:], lse[:first, G:], tuple(x[:first, G:] for x in want), T)
    if math.isnan(bad):
        assert torch.isnan(out[first:, G:]).all()


def test_largest_fp16_values():
    """Weights that round upward must not push an output of 65504 to infinity."""
    T, dtype = 333, torch.float16
    kc, vc, table = ref.make_cache([T], 1, dtype, 41)
    vc.copy_(torch.full_like(vc, 65504.0))
    q = queries(50, 4, dtype, 42)
    out, _, err = chunk(q, kc, vc, table, [T], [50])
    assert err == 0 and torch.all(out >= 65440)


def test_rows_of_no_request_are_left():
    dtype = torch.float16
    lens, n_new = [50, 80], [10, 20]
    kc, vc, table = ref.make_cache(lens, 2, dtype, 51)
    q = queries(40, 4, dtype, 52)
    offsets = torch.tensor([3, 13, 33], dtype=torch.int32, device="cuda")
    out, lse, err = chunk(q, kc, vc, table, lens, n_new, offsets=offsets, fill=7.0)
    assert err == 0
    for rows in (slice(0, 3), slice(33, 40)):
        assert torch.all(out[rows] == 7) and torch.all(lse[rows] == 7)
    ref.check_attention(out[3:33], lse[3:33], ref.chunk_attention(q[3:33], kc, vc, table, lens, n_new), 80)


def test_no_lse_and_a_scale():
    dtype = torch.bfloat16
    kc, vc, table = ref.make_cache([90], 2, dtype, 61)
    q = queries(70, 4, dtype, 62)
    out, _, _ = chunk(q, kc, vc, table, [90], [70], lse=False, scale=0.25)
    want = ref.chunk_attention(q, kc, vc, table, [90], [70], 0.25)
    ref.check_attention(out, None, want, 90)


@pytest.mark.parametrize("layout", ["heads_last", "kv_fused", "padded_rows", "one_head_of_many"])
def test_strides(layout):
    dtype, Hkv, lens, n_new = torch.float16, 2, [77, 300], [30, 140]
    kc, vc, table = ref.make_cache(lens, Hkv, dtype, 71, fill=float("nan"))
    nb = kc.shape[0]
    if layout == "heads_last":  # rows as clo_kv4_gather writes them
        k2, v2 = (x.transpose(1, 2).contiguous().view(-1, Hkv, ref.D) for x in (kc, vc))
        k2, v2 = (x.view(nb, 16, Hkv, ref.D).transpose(1, 2) for x in (k2, v2))
    elif layout == "kv_fused":
        both = torch.stack([kc, vc], 1)
        k2, v2 = both[:, 0], both[:, 1]
    elif layout == "padded_rows":
        both = torch.full((2, nb, Hkv, 16, ref.D + 8), float("nan"), dtype=dtype, device="cuda")
        both[0, ..., :ref.D], both[1, ..., :ref.D] = kc, vc
        k2, v2 = both[0, ..., :ref.D], both[1, ..., :ref.D]
    else:
        both = torch.full((2, nb, 5, 16, ref.D), float("nan"), dtype=dtype, device="cuda")
        both[0, :, 1:4:2], both[1, :, 1:4:2] = kc, vc
        k2, v2 = both[0, :, 1:4:2], both[1, :, 1:4:2]
    wide = torch.full((170, 8 + 2 * Hkv, ref.D), float("nan"), dtype=dtype, device="cuda")
    wide[:, :8] = queries(170, 8, dtype, 72)
    q = wide[:, :8]
    out = torch.empty(170, 8, ref.D, dtype=dtype, device="cuda")
    ws = torch.empty(clo.clo_paged_chunk_workspace_size(8, Hkv), dtype=torch.uint8, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clo.clo_paged_chunk_attn(q, k2, v2, table, ctx, offsets_of(n_new), out, ws)
    torch.cuda.synchronize()
    ref.check_attention(out, None, ref.chunk_attention(q, kc, vc, table, lens, n_new), 300)


def test_bad_lengths_offsets_and_blocks():
    dtype = torch.float16
    lens, n_new = [100, 60, 300, 90, 40], [20, 10, 200, 30, 5]
    kc, vc, table = ref.make_cache(lens, 2, dtype, 81)
    q = queries(sum(n_new), 4, dtype, 82)
    want = ref.chunk_attention(q, kc, vc, table, lens, n_new)
    offs = offsets_of(n_new)
    # a bad length
    for n in (-1, table.shape[1] * 16 + 1):
        out, lse, err = chunk(q, kc, vc, table, lens[:1] + [n] + lens[2:], n_new)
        assert err == clo.FLAG_BAD_CTX
        assert torch.all(out[20:30] == 0) and torch.all(torch.isneginf(lse[20:30]))
        keep = torch.tensor([i for i in range(len(out)) if not 20 <= i < 30], device="cuda")
        ref.check_attention(out[keep], lse[keep], tuple(x[keep] for x in want), 300)
    # bad blocks: those who see it are zeroed, the others of the batch are right
    t2 = table.clone()
    t2[2, 5] = kc.shape[0]
    t2[3, 0] = -1
    out, lse, err = chunk(q, kc, vc, t2, lens, n_new)
    assert err == clo.FLAG_BAD_INDEX
    assert torch.all(out[230:260] == 0) and torch.all(out[30:230] == 0) and torch.all(torch.isneginf(lse[30:260]))
    ref.check_attention(out[:30], lse[:30], tuple(x[:30] for x in want), 300)
    ref.check_attention(out[260:], lse[260:], tuple(x[260:] for x in want), 300)
    # offsets that descend or leave the batch: those requests are passed over
    o2 = offs.clone()
    o2[3], o2[5] = 10, 10000
    out, lse, err = chunk(q, kc, vc, table, lens, n_new, offsets=o2, fill=3.0)
    assert err & clo.FLAG_BAD_CTX
    ref.check_attention(out[:10], lse[:10], tuple(x[:10] for x in want), 300)
    assert torch.all(out[260:] == 3)


@pytest.mark.parametrize("B", [7, 70])  # a request a lane; summed up by all threads
def test_offsets_that_overlap_many_times_are_passed_over(B):
    """Every other request descends, the others have all rows: more than 2 N, so no row is written."""
    dtype = torch.float16
    kc, vc, table = ref.make_cache([64] * B, 2, dtype, 83)
    q = queries(40, 4, dtype, 86)
    offs = torch.tensor([40 * (r % 2) for r in range(B + 1)], dtype=torch.int32, device="cuda")
    out, lse, err = chunk(q, kc, vc, table, [64] * B, [40] * B, offsets=offs, fill=3.0)
    assert err == clo.FLAG_BAD_CTX
    assert torch.all(out == 3)


def test_a_block_that_no_row_sees_may_be_bad():
    """Table entries behind the context are not looked at."""
    dtype = torch.float16
    kc, vc, table = ref.make_cache([100], 2, dtype, 84, max_blocks=40)
    table[0, 7:] = 1 << 30
    q = queries(20, 4, dtype, 85)
    out, lse, err = chunk(q, kc, vc, table, [100], [20])
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, [100], [20]), 100)


def test_same_bits_each_time_on_streams_and_in_graphs():
    dtype = torch.bfloat16
    lens, n_new = [5000, 700, 64, 1200], [200, 700, 1, 1]
    kc, vc, table = ref.make_cache(lens, 2, dtype, 91)
    q = queries(sum(n_new), 10, dtype, 92)
    first, lse0, _ = chunk(q, kc, vc, table, lens, n_new)
    again, lse1, _ = chunk(q, kc, vc, table, lens, n_new)
    assert torch.equal(first, again) and torch.equal(lse0, lse1)
    ctx, offs = torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets_of(n_new)
    sets = []
    for _ in range(2):
        out = torch.zeros_like(q)
        ws = torch.empty(clo.clo_paged_chunk_workspace_size(10, 2), dtype=torch.uint8, device="cuda")
        sets.append((out, clo.prepare_paged_chunk_attn(q, kc, vc, table, ctx, offs, out, ws)))
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for st, (_, call) in zip(streams, sets):
        with torch.cuda.stream(st):
            for _ in range(5):
                call()
    torch.cuda.synchronize()
    assert all(torch.equal(out, first) for out, _ in sets)
    # captured, and replayed with other lengths and queries in the same buffers
    out, call = sets[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    lens2 = [4000, 690, 33, 1190]
    ctx.copy_(torch.tensor(lens2, dtype=torch.int32))
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    ref.check_attention(out, None, ref.chunk_attention(q, kc, vc, table, lens2, n_new), 5000)


def test_events_and_large_offsets():
    """A cache in which the used blocks lie beyond 2^31 elements."""
    dtype, Hkv = torch.float16, 8
    need = 2 * (1 << 31) * 2 + (1 << 28)
    if torch.cuda.mem_get_info()[0] < 3 * need:
        pytest.skip("needs 27 GB of device memory")
    nb = (1 << 31) // (Hkv * 16 * ref.D) + 64
    kc, vc = (torch.zeros(nb, Hkv, 16, ref.D, dtype=dtype, device="cuda") for _ in range(2))
    k0, v0, t0 = ref.make_cache([300], Hkv, dtype, 95)
    n = k0.shape[0]
    kc[-n:], vc[-n:] = k0, v0
    q = queries(40, 16, dtype, 96)
    table = torch.where(t0 >= 0, t0 + (nb - n), t0).to(torch.int32)
    out, lse, err = chunk(q, kc, vc, table, [300], [40])
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, k0, v0, t0, [300], [40]), 300)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    for e in ev:
        e.record()
    ws = torch.empty(clo.clo_paged_chunk_workspace_size(16, Hkv), dtype=torch.uint8, device="cuda")
    clo.clo_paged_chunk_attn(q, kc, vc, table, torch.tensor([300], dtype=torch.int32, device="cuda"), offsets_of([40]), out, ws,
                             events=ev)
    torch.cuda.synchronize()
    assert ev[0].elapsed_time(ev[1]) > 0


def test_against_the_decode_kernel():
    """One token a request: what clo_paged_decode_attn computes."""
    dtype = torch.float16
    lens = [1, 500, 64, 0, 2000]
    kc, vc, table = ref.make_cache(lens, 4, dtype, 101)
    q = queries(5, 16, dtype, 102)
    out, lse, err = chunk(q, kc, vc, table, lens, [1] * 5)
    o2, e2 = torch.empty_like(q), torch.empty(5, 16, device="cuda")
    ws = torch.empty(clo.clo_paged_workspace_size(5, 16, 4), dtype=torch.uint8, device="cuda")
    clo.clo_paged_decode_attn(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), o2, ws, lse=e2)
    torch.cuda.synchronize()
    want = ref.chunk_attention(q, kc, vc, table, lens, [1] * 5)
    ref.check_attention(out, lse, want, 2000)
    ref.check_attention(o2, e2, want, 2000)


def test_over_the_read_back_4_bit_cache():
    """clo_kv4_gather's rows are a cache: a chunk attends to a prefix that is held in 4 bits."""
    dtype, Hkv, T, n = torch.float16, 2, 500, 60
    k, v = (torch.randn(512, Hkv, ref.D, generator=torch.Generator().manual_seed(s)).to(dtype).cuda() for s in (1, 2))
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    slots[T:] = -1
    pool = torch.zeros(32, Hkv, clo.clo_kv4_block_bytes(64), dtype=torch.uint8, device="cuda")
    clo.clo_kv4_append(k, v, slots, pool)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    clo.clo_kv4_gather(pool, slots, kb, vb)
    kc, vc = (x.view(32, 16, Hkv, ref.D).transpose(1, 2) for x in (kb, vb))
    table = torch.arange(32, dtype=torch.int32, device="cuda")[None]
    q = queries(n, 8, dtype, 3)
    out, lse, err = chunk(q, kc, vc, table, [T], [n])
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, kc.contiguous(), vc.contiguous(), table, [T], [n]), T)


# ---------------------------------------------------------------- selected blocks

def sparse(q, kc, vc, table, lens, sel, num_ctas=0):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((clo.clo_paged_chunk_workspace_size(q.shape[1], kc.shape[1], num_ctas=num_ctas),), 0xff, dtype=torch.uint8,
                    device="cuda")
    clo.clo_paged_sparse_decode_attn(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), sel, out, ws,
                                     lse=lse, err_flag=err, num_ctas=num_ctas)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def sparse_ref(q, kc, vc, table, lens, sel):
    B, Hq, _ = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    res = [torch.zeros(B, Hq, ref.D, dtype=torch.float64, device="cuda"), torch.full((B, Hq), -math.inf, dtype=torch.float64,
           device="cuda"), torch.zeros(B, Hq, ref.D, dtype=torch.float64, device="cuda"), torch.zeros(B, Hq, dtype=torch.float64,
           device="cuda")]
    for r, T in enumerate(lens):
        for h in range(Hkv):
            cols = [c for c in sel[r, h, :ref.blocks_of(T)].tolist() if c >= 0]
            tok = [c * 16 + i for c in cols for i in range(16) if c * 16 + i < T]
            if not tok:
                continue
            k, v = (ref.cached(x, table, r, T)[h][tok] for x in (kc, vc))
            got = ref.attend_clean(q[r, h * G:(h + 1) * G].double(), k, v, 1 / math.sqrt(ref.D))
            for x, y in zip(res, got):
                x[r, h * G:(h + 1) * G] = y
    return tuple(res)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,Hkv,n_sel,num_ctas", [(4, 2, 1, 0), (1, 3, 7, 0), (8, 1, 8, 3), (5, 2, 20, 0), (3, 2, 33, 1), (2, 8, 64, 0),
                                                  (4, 1, 300, 200)])
def test_sparse(G, Hkv, n_sel, num_ctas, dtype):
    lens = [1, 0, 900, 16 * n_sel, 16 * n_sel + 5, 33]
    kc, vc, table = ref.make_cache(lens, Hkv, dtype, n_sel, fill=float("nan"))
    g = torch.Generator().manual_seed(n_sel)
    sel = torch.full((6, Hkv, n_sel), -7, dtype=torch.int32)  # what is behind the request's blocks is not read
    for r, T in enumerate(lens):
        for h in range(Hkv):
            cols = torch.randperm(ref.blocks_of(T), generator=g)[:n_sel].to(torch.int32)  # any order
            sel[r, h, :len(cols)] = cols
    sel[2, 0, 0] = -1  # left out
    sel = sel.cuda()
    q = queries(6, G * Hkv, dtype, n_sel + 1)
    out, lse, err = sparse(q, kc, vc, table, lens, sel, num_ctas)
    assert err == 0
    ref.check_attention(out, lse, sparse_ref(q, kc, vc, table, lens, sel), max(lens))


def test_sparse_with_every_block_is_dense():
    dtype, lens = torch.float16, [333, 1000]
    kc, vc, table = ref.make_cache(lens, 2, dtype, 5)
    sel = torch.arange(63, dtype=torch.int32, device="cuda").expand(2, 2, 63).contiguous()
    q = queries(2, 8, dtype, 6)
    out, lse, err = sparse(q, kc, vc, table, lens, sel)
    assert err == 0
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, lens, [1, 1]), 1000)


def test_sparse_twice_the_same_block():
    dtype = torch.float16
    kc, vc, table = ref.make_cache([200], 1, dtype, 5)
    sel = torch.tensor([[[3, 3, 5, 3]]], dtype=torch.int32, device="cuda")
    q = queries(1, 4, dtype, 6)
    out, lse, err = sparse(q, kc, vc, table, [200], sel)
    assert err == 0
    ref.check_attention(out, lse, sparse_ref(q, kc, vc, table, [200], sel), 200)


def test_selected_blocks_in_a_graph():
    """Bounds, selection and attention captured once and replayed with other queries, keys
    and lengths in the same buffers."""
    dtype, Hkv, lens = torch.bfloat16, 2, [700, 33, 1500]
    kc, vc, table = ref.make_cache(lens, Hkv, dtype, 15)
    q = queries(3, 8, dtype, 16)
    last = [table[r, (T - 1) // 16].item() * 16 + (T - 1) % 16 for r, T in enumerate(lens)]
    slots = [t for r, T in enumerate(lens) for p in range(ref.blocks_of(T))
             for t in range(table[r, p].item() * 16, table[r, p].item() * 16 + min(16, T - 16 * p))]
    slots = torch.tensor(slots, dtype=torch.int32, device="cuda")
    assert slots[-1] == last[-1]
    bounds = torch.zeros(kc.shape[0], Hkv, ref.RECORD, dtype=torch.uint8, device="cuda")
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    sel = torch.empty(3, Hkv, 20, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sws = torch.empty(clo.clo_paged_select_workspace_size(3, Hkv, table.shape[1]), dtype=torch.uint8, device="cuda")
    ws = torch.empty(clo.clo_paged_chunk_workspace_size(8, Hkv), dtype=torch.uint8, device="cuda")
    calls = [clo.prepare_paged_block_bounds(kc, slots, bounds, err_flag=err),
             clo.prepare_paged_block_select(q, bounds, table, ctx, sel, sws, 1, 2, err_flag=err),
             clo.prepare_paged_sparse_decode_attn(q, kc, vc, table, ctx, sel, out, ws, lse=lse, err_flag=err)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for step in range(2):
        if step == 1:
            kc.mul_(-0.5)
            q.copy_(queries(3, 8, dtype, 17))
            ctx.copy_(torch.tensor([690, 20, 1499], dtype=torch.int32))
            lens = [690, 20, 1499]
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for r, T in enumerate(lens):
            nb = ref.blocks_of(T)
            for h in range(Hkv):
                assert sel[r, h].tolist() == ref.select(q[r, 4 * h:4 * h + 4].cpu(), bounds[table[r, :nb].long(), h].cpu(), nb, 20, 1, 2)
        ref.check_attention(out, lse, sparse_ref(q, kc, vc, table, lens, sel), 1500)


def test_sparse_bad_entries():
    dtype, lens = torch.bfloat16, [200, 100, 64, 300]
    kc, vc, table = ref.make_cache(lens, 2, dtype, 7)
    sel = torch.arange(4, dtype=torch.int32, device="cuda").expand(4, 2, 4).contiguous()
    q = queries(4, 6, dtype, 8)
    want = sparse_ref(q, kc, vc, table, lens, sel)
    sel[0, 1, 2] = 13          # request 0 has 13 blocks: 0 .. 12
    sel[1, 0, 0] = -2
    t2 = table.clone()
    t2[3, 1] = kc.shape[0]     # both heads of request 3
    out, lse, err = sparse(q, kc, vc, t2, lens, sel)
    assert err == clo.FLAG_BAD_INDEX
    for r, h in ((0, 1), (1, 0), (3, 0), (3, 1)):
        assert torch.all(out[r, 3 * h:3 * h + 3] == 0) and torch.all(torch.isneginf(lse[r, 3 * h:3 * h + 3]))
    for r, h in ((0, 0), (1, 1), (2, 0), (2, 1)):
        s = slice(3 * h, 3 * h + 3)
        ref.check_attention(out[r, s], lse[r, s], tuple(x[r, s] for x in want), 300)
    out, lse, err = sparse(q, kc, vc, table, [-5] + lens[1:], sel)
    assert err & clo.FLAG_BAD_CTX and torch.all(out[0] == 0)
