"""clo_kv4_paged_decode_attn on the GPU against the fp64 reference, element by
element, at the tolerance that kv4_ref.attention derives."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def inputs(ctx, n_q, Hq, Hkv, group, dt, seed, spread=1.0, mb=None):
    """q, a pool of shuffled blocks with bell-shaped codes, its table; the
    parameters behind each request's last token are NaN, as are the blocks
    that nobody has."""
    rng = np.random.Generator(np.random.PCG64(seed))
    ctx = np.asarray(ctx)
    B = len(ctx)
    mb = mb or max(1, int(-(-ctx.max() // 16)))
    nb = B * mb + 2
    R = ref.record_bytes(group)
    table = rng.permutation(nb - 2).reshape(B, mb) + 1 if B * mb <= 20000 else None
    if B * mb > 20000:  # a wide table: only blocks in use are made
        used = int(sum(-(-int(c) // 16) for c in ctx))
        nb, at, wide = used + 2, 1, np.full((B, mb), -7)
        for r in range(B):
            n = -(-int(ctx[r]) // 16)
            wide[r, :n] = np.arange(at, at + n)
            at += n
        table = wide
    pool = rng.integers(0, 256, (nb, Hkv, R), dtype=np.uint8)
    pool[:, :, :2048] = (pool[:, :, :2048] & 0x77) + (rng.integers(0, 256, (nb, Hkv, 2048), dtype=np.uint8) & 0x77)
    scale = rng.uniform(0.05, 0.4, (nb, Hkv, 16, 2, 128 // group))
    scale[:, :, :, 1] *= np.minimum(spread ** rng.standard_normal((nb, Hkv, 16, 1)), 2000.0)  # V; fp16 holds it
    zero = -scale * rng.normal(7.5, 1.0, scale.shape)
    par = np.stack([scale, zero], -1).astype(np.float16)
    live = np.zeros((nb, 16), bool)
    for r in range(B):
        for c in range(-(-int(ctx[r]) // 16)):
            live[table[r, c], :max(0, min(16, int(ctx[r]) - 16 * c))] = True
    par = np.where(live[:, None, :, None, None, None], par, np.float16(np.nan))
    pool[:, :, 2048:] = np.ascontiguousarray(par).view(np.uint8).reshape(nb, Hkv, -1)
    q = torch.from_numpy(rng.standard_normal((B, n_q, Hq, 128))).to(dt)
    return q, pool, table, ctx


def run(q, pool, table, ctx, num_ctas=0, scale=None, ws=None, err=None):
    B, n_q, Hq, _ = q.shape
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=dev())
    lse = torch.full(q.shape[:3], float("nan"), dtype=torch.float32, device=dev())
    if ws is None:
        ws = torch.empty(clo.clo_kv4_paged_workspace_size(B, n_q, Hq, pool.shape[1], 128, num_ctas), dtype=torch.uint8,
                         device=dev())
        ws.fill_(0xFF)  # NaN patterns: nothing in it may be read before it is written
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
    clo.clo_kv4_paged_decode_attn(q.to(dev()), torch.as_tensor(pool).to(dev()), i32(table), i32(ctx), out, ws, lse=lse,
                                  err_flag=err, num_ctas=num_ctas, scale=scale)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), int(err.item())


def assert_matches(got, lse, want, what=""):
    o, l, tol, ltol = want
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - o) - tol
    assert over.max() <= 0, f"{what}: {over.max():.3e} over a tolerance of {tol.flat[over.argmax()]:.3e}"
    seen = np.isfinite(l)
    assert np.array_equal(np.isneginf(lse), ~seen), what
    assert np.all(np.abs(lse[seen] - l[seen]) <= ltol[seen]), what


def check(ctx, n_q, Hq, Hkv, group, dtype, seed, num_ctas=0, **kw):
    dt = DT[dtype]
    q, pool, table, ctx = inputs(ctx, n_q, Hq, Hkv, group, dt, seed, **kw)
    got, lse, err = run(q, pool, table, ctx, num_ctas)
    assert err == 0
    want = ref.attention(q.double().numpy(), pool, table, ctx, group, ref.scale_for(), dt)
    assert_matches(got, lse, want, f"{ctx} {n_q} {Hq}/{Hkv} {group} {dtype}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n_q,Hq,Hkv", [(1, 1, 1), (1, 8, 8), (1, 32, 8), (1, 10, 2), (1, 16, 2), (4, 8, 2), (3, 7, 1),
                                        (2, 32, 2), (1, 24, 1), (8, 4, 1), (32, 1, 1)])
def test_head_layouts(n_q, Hq, Hkv, group, dtype):
    """Both ways: a number of CTAs asks for the one that shares all units out."""
    for num_ctas in (0, 5):
        check([1, 15, 16, 17, 200, 333], n_q, Hq, Hkv, group, dtype, n_q * 100 + Hq + group, num_ctas)


@pytest.mark.parametrize("num_ctas", [0, 1, 2, 7, 64])
@pytest.mark.parametrize("ctx", [[1], [16], [2000], [0, 5, 0, 700, 1, 0], [31, 32, 33, 1, 1, 900, 2, 47]])
def test_lengths_and_splits(ctx, num_ctas):
    check(ctx, 1, 8, 2, 64, "f16", 5, num_ctas)


@pytest.mark.parametrize("n_q,group", [(1, 128), (1, 32), (3, 64), (8, 64)])
def test_short_contexts_in_a_wide_table(n_q, group):
    """The same requests with a table that just holds them and with one for far
    longer contexts: the two take different ways, and both meet the tolerance."""
    ctx = [0, 1, 16, 33, 500, 1023, 700, 2]
    for mb in (None, 5000):
        check(ctx, n_q, 8, 2, group, "f16", 31 + n_q, mb=mb)


@pytest.mark.parametrize("ctx", [[64], [128, 100], [300, 256, 40], [1000, 10], [2048], [4000, 3000, 17]])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 4), (64, 64)])
def test_short_contexts_of_all_sizes(ctx, Hq, Hkv):
    check(ctx, 1, Hq, Hkv, 64, "bf16", Hq + len(ctx))


@pytest.mark.parametrize("num_ctas", [0, 3, 40])
@pytest.mark.parametrize("n_q", [2, 4, 5])
def test_drafts_that_see_nothing_or_part_of_a_block(n_q, num_ctas):
    """Requests shorter than the draft: their first queries see no token."""
    check([0, 1, 2, 3, 4, 5, 15, 16, 17, 18, 19, 20, 300], n_q, 12, 3, 32, "bf16", n_q, num_ctas)


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    rng = np.random.Generator(np.random.PCG64(2000 + seed))
    Hkv = int(rng.choice([1, 2, 4, 8]))
    G = int(rng.integers(1, 9))
    n_q = int(rng.integers(1, 32 // G + 1)) if seed % 2 else 1
    B = int(rng.integers(1, 6))
    ctx = rng.integers(0, int(rng.choice([20, 300, 3000])), B)
    check(ctx, n_q, G * Hkv, Hkv, int(rng.choice([32, 64, 128])), str(rng.choice(["f16", "bf16"])), seed,
          int(rng.choice([0, 0, 1, 3, 17, 200])))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_of_many_sizes(group):
    """Tokens whose V scales are orders of magnitude apart, constant groups
    (scale 0) and the smallest and largest scales."""
    q, pool, table, ctx = inputs([500, 77], 1, 8, 2, group, torch.float16, 3, spread=30.0)
    par = pool[:, :, 2048:].copy().view(np.float16).reshape(*pool.shape[:2], 16, 2, -1, 2)
    par[:, :, 3, 1, :, 0] = 0
    par[:, :, 5, :, 0, 0] = np.float16(2.0 ** -24)
    par[:, :, 6, 1, :, 0] = 2000.0
    par[:, :, 6, 1, :, 1] = -30000.0
    pool[:, :, 2048:] = par.reshape(*pool.shape[:2], -1).view(np.uint8)
    got, lse, err = run(q, pool, table, ctx)
    assert err == 0
    want = ref.attention(q.double().numpy(), pool, table, ctx, group, ref.scale_for(), torch.float16)
    assert_matches(got, lse, want)


def test_one_token_rules_the_softmax_and_its_values_are_tiny():
    """The token with nearly all the weight has V scales far below the others'."""
    q, pool, table, ctx = inputs([400], 1, 4, 1, 64, torch.float16, 9)
    rec = pool[table[0]]
    par = rec[:, :, 2048:].copy().view(np.float16).reshape(len(rec), 1, 16, 2, -1, 2)
    par[2, 0, 7, 0] *= 60          # its key: 60 times as long, so it wins for some heads and loses for others
    par[2, 0, 7, 1] *= np.float16(1e-3)
    rec[:, :, 2048:] = par.reshape(len(rec), 1, -1).view(np.uint8)
    pool[table[0]] = rec
    got, lse, err = run(q, pool, table, ctx)
    want = ref.attention(q.double().numpy(), pool, table, ctx, 64, ref.scale_for(), torch.float16)
    assert err == 0
    assert_matches(got, lse, want)


@pytest.mark.parametrize("mul", [1e-6, 200.0, 60000.0])
def test_large_and_small_queries(mul):
    q, pool, table, ctx = inputs([130, 64], 2, 8, 2, 128, torch.float16, 12)
    q = (q.clamp(-1, 1) * mul).to(torch.float16)
    got, lse, err = run(q, pool, table, ctx)
    want = ref.attention(q.double().numpy(), pool, table, ctx, 128, ref.scale_for(), torch.float16)
    assert err == 0
    assert_matches(got, lse, want)


def test_bfloat16_queries_beyond_half_range():
    for mul in (1e-30, 1e6):
        q, pool, table, ctx = inputs([130], 1, 8, 2, 128, torch.bfloat16, 13)
        q = (q.float() * mul).to(torch.bfloat16)
        scale = ref.scale_for() / (mul if mul > 1 else 1)
        got, lse, err = run(q, pool, table, ctx, scale=scale)
        want = ref.attention(q.double().numpy(), pool, table, ctx, 128, scale, torch.bfloat16)
        assert err == 0
        assert_matches(got, lse, want)


@pytest.mark.parametrize("group", [64, 128])
def test_as_many_requests_as_there_may_be(group):
    """4096 requests, most of them empty, in a wide table and in a narrow one."""
    ctx = np.zeros(4096, int)
    ctx[[0, 1, 7, 2048, 4095]] = [3, 40, 700, 33, 1000]
    for mb in (None, 1100):
        check(ctx, 1, 8, 2, group, "f16", 41, mb=mb)
    with pytest.raises(clo.CloError):
        run(*inputs(np.ones(4097, int), 1, 1, 1, 128, torch.float16, 1))


def test_events_bracket_the_kernel():
    q, pool, table, ctx = inputs([900, 40], 1, 16, 4, 64, torch.float16, 19)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
    q, pool = q.to(dev()), torch.as_tensor(pool).to(dev())
    for num_ctas in (0, 30):
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        for e in ev:
            e.record()  # creates it
        out = torch.empty_like(q)
        ws = torch.empty(clo.clo_kv4_paged_workspace_size(2, 1, 16, 4, 128, num_ctas), dtype=torch.uint8, device=dev())
        clo.clo_kv4_paged_decode_attn(q, pool, i32(table), i32(ctx), out, ws, num_ctas=num_ctas, events=ev)
        torch.cuda.synchronize()
        assert 0 < ev[0].elapsed_time(ev[1]) < 1000


def test_output_in_place_of_the_queries():
    """out may be q."""
    for mb, ctx in ((None, [900, 40, 0, 5]), (1500, [3000, 40, 0, 5])):
        q, pool, table, ctx = inputs(ctx, 2, 16, 4, 64, torch.float16, 23, mb=mb)
        want, _, _ = run(q, pool, table, ctx)
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
        both = q.to(dev())
        ws = torch.empty(clo.clo_kv4_paged_workspace_size(4, 2, 16, 4), dtype=torch.uint8, device=dev())
        clo.clo_kv4_paged_decode_attn(both, torch.as_tensor(pool).to(dev()), i32(table), i32(ctx), both, ws)
        assert np.array_equal(both.double().cpu().numpy(), want)


def test_two_calls_at_once_on_two_streams():
    a, b = (inputs([1500, 700], 1, 16, 4, 64, torch.float16, s, mb=1200) for s in (24, 25))
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
    jobs = []
    for q, pool, table, ctx in (a, b):
        out = torch.empty(q.shape, dtype=q.dtype, device=dev())
        ws = torch.empty(clo.clo_kv4_paged_workspace_size(2, 1, 16, 4), dtype=torch.uint8, device=dev())
        st = torch.cuda.Stream()
        call = clo.prepare_kv4_paged_decode_attn(q.to(dev()), torch.as_tensor(pool).to(dev()), i32(table), i32(ctx),
                                                 out, ws, stream=st)
        jobs.append((call, out, run(q, pool, table, ctx)[0]))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, _, _ in jobs:
            call()
    torch.cuda.synchronize()
    for _, out, want in jobs:
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_a_non_finite_token_is_seen_only_by_queries_that_see_it():
    q, pool, table, ctx = inputs([40, 40], 4, 8, 2, 64, torch.float16, 14)
    rec = pool[table[0, 2]]
    par = rec[:, 2048:].copy().view(np.float16).reshape(2, 16, 2, 2, 2)
    par[0, 6] = np.nan             # token 38 of request 0, KV head 0: queries 2 and 3 of 4 see it
    rec[:, 2048:] = par.reshape(2, -1).view(np.uint8)
    pool[table[0, 2]] = rec
    got, lse, err = run(q, pool, table, ctx)
    assert err == 0
    with np.errstate(invalid="ignore"):
        o, l, tol, ltol = ref.attention(q.double().numpy(), pool, table, ctx, 64, ref.scale_for(), torch.float16)
    sick = np.zeros(got.shape[:3], bool)
    sick[0, 2:, :4] = True
    assert np.isnan(got[sick]).all() and np.isnan(lse[sick]).all()
    assert np.all(np.abs(got - o)[~sick] <= tol[~sick]) and np.all(np.abs(lse - l)[~sick] <= ltol[~sick])


@pytest.mark.parametrize("num_ctas", [0, 1, 9])
def test_bad_blocks_and_lengths(num_ctas):
    """They zero the rows they touch, set their flags and nothing else."""
    q, pool, table, ctx = inputs([300, 200, 100, 64, 50], 2, 8, 2, 64, torch.bfloat16, 15)
    want = ref.attention(q.double().numpy(), pool, table, ctx, 64, ref.scale_for(), torch.bfloat16)
    t, c = table.copy(), ctx.copy()
    t[1, 3], t[1, 9] = pool.shape[0], -1
    t[3, 4] = 1 << 30              # behind its last token: not used
    c[2], c[4] = -5, t.shape[1] * 16 + 1
    got, lse, err = run(q, pool, t, c, num_ctas)
    assert err == clo.FLAG_BAD_INDEX | clo.FLAG_BAD_CTX
    for r in (1, 2, 4):
        assert np.all(got[r] == 0) and np.all(np.isneginf(lse[r]))
    for r in (0, 3):
        assert_matches(got[r], lse[r], [x[r] for x in want])


def test_the_same_block_twice_and_shared_between_requests():
    """A shared prefix: entries of the table may repeat."""
    q, pool, table, ctx = inputs([100, 100, 100], 1, 8, 2, 32, torch.float16, 16)
    table[1, :5] = table[0, :5]
    table[2, 1] = table[2, 2]
    got, lse, err = run(q, pool, table, ctx)
    want = ref.attention(q.double().numpy(), pool, table, ctx, 32, ref.scale_for(), torch.float16)
    assert err == 0
    assert_matches(got, lse, want)


def test_three_dimensional_queries_and_no_lse():
    q, pool, table, ctx = inputs([90, 5], 1, 8, 2, 64, torch.float16, 17)
    full, _, _ = run(q, pool, table, ctx)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
    out = torch.empty(2, 8, 128, dtype=torch.float16, device=dev())
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(2, 1, 8, 2), dtype=torch.uint8, device=dev())
    clo.clo_kv4_paged_decode_attn(q[:, 0].contiguous().to(dev()), torch.as_tensor(pool).to(dev()), i32(table),
                                  i32(ctx), out, ws)
    assert np.array_equal(out.double().cpu().numpy(), full[:, 0])


def test_same_bits_every_time_and_on_any_table_width():
    """Results do not depend on timing."""
    q, pool, table, ctx = inputs([3000, 17, 1200, 0, 640], 1, 32, 8, 64, torch.float16, 18)
    first = run(q, pool, table, ctx)
    for _ in range(5):
        again = run(q, pool, table, ctx)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn, and an eager
    call between them."""
    a, b = (inputs(c, 1, 16, 4, 64, torch.float16, s) for c, s in (([900, 40], 19), ([64, 1500], 20)))
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(2, 1, 16, 4), dtype=torch.uint8, device=dev())
    ws.fill_(0xFF)
    calls, outs, wants = [], [], []
    for q, pool, table, ctx in (a, b):
        out = torch.empty(q.shape, dtype=q.dtype, device=dev())
        calls.append(clo.prepare_kv4_paged_decode_attn(q.to(dev()), torch.as_tensor(pool).to(dev()), i32(table),
                                                       i32(ctx), out, ws))
        outs.append(out)
        wants.append(run(q, pool, table, ctx)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for call in calls:
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0)):
        for o in outs:
            o.zero_()
        for k in order:
            graphs[k].replay()
            calls[1 - k]()
        torch.cuda.synchronize()
        for k in (0, 1):
            assert np.array_equal(outs[k].double().cpu().numpy(), wants[k])


def test_long_context_of_a_large_pool():
    """A pool past 4 GiB and a context of 70001 tokens in blocks all over it,
    checked on one KV head."""
    group, Hkv = 128, 8
    R = ref.record_bytes(group)
    nb = (5 << 30) // (Hkv * R)
    n = 70001
    g = torch.Generator(device=dev()).manual_seed(4)
    pool = torch.randint(0, 256, (nb, Hkv, R), dtype=torch.uint8, device=dev(), generator=g)
    par = torch.stack([torch.rand(nb, Hkv, 32, device=dev(), generator=g) * 0.3 + 0.05,
                       -2 + torch.rand(nb, Hkv, 32, device=dev(), generator=g)], -1).half()
    pool[:, :, 2048:] = par.view(torch.uint8).view(nb, Hkv, -1)
    del par
    table = torch.randperm(nb, device=dev(), generator=g)[:-(-n // 16)].to(torch.int32)[None].contiguous()
    q = torch.randn(1, 1, 32, 128, device=dev(), generator=g).half()
    out, lse = torch.empty_like(q), torch.empty(1, 1, 32, device=dev())
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(1, 1, 32, Hkv), dtype=torch.uint8, device=dev())
    clo.clo_kv4_paged_decode_attn(q, pool, table, torch.tensor([n], dtype=torch.int32, device=dev()), out, ws, lse=lse)
    rec = pool[table[0].long()][:, 5:6].cpu().numpy()
    o, l, tol, ltol = ref.attention(q[:, :, 20:24].double().cpu().numpy(), rec, np.arange(len(rec))[None], [n], group,
                                    ref.scale_for(), torch.float16)
    assert_matches(out[:, :, 20:24].double().cpu().numpy(), lse[:, :, 20:24].double().cpu().numpy(), (o, l, tol, ltol))


def test_refused_tensors():
    q, pool, table, ctx = inputs([30, 5], 1, 8, 2, 64, torch.float16, 21)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev())  # noqa: E731
    q, pool, table, ctx = q.to(dev()), torch.as_tensor(pool).to(dev()), i32(table), i32(ctx)
    out = torch.empty_like(q)
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(2, 1, 8, 2), dtype=torch.uint8, device=dev())
    good = [q, pool, table, ctx, out, ws]
    for at, bad in ((0, q.float()), (0, q.cpu()), (1, pool[:, :, :2303].contiguous()), (2, table.long()),
                    (2, table[:1]), (3, ctx[:1]), (4, out.bfloat16()), (4, out[:1]), (5, ws[:16]), (0, q[:, :, :7])):
        a = list(good)
        a[at] = bad
        with pytest.raises(clo.CloError):
            clo.clo_kv4_paged_decode_attn(*a)
    with pytest.raises(clo.CloError):
        clo.clo_kv4_paged_decode_attn(*good, scale=0.0)
    with pytest.raises(clo.CloError):
        clo.clo_kv4_paged_decode_attn(*good, lse=torch.empty(3, device=dev()))
    with pytest.raises(clo.CloError):
        clo.clo_kv4_paged_decode_attn(*good, num_ctas=-1)
