"""The 16-bit paged cache at the edges of its types and tiles."""
import math

import pytest
import torch

import offloaded_kv_decode_gb300 as clo
import paged_ref as ref
from test_paged16_attention_gpu import chunk, offsets_of, queries, sparse, sparse_ref
from test_paged16_cache_gpu import check_select, rand, random_bounds, select

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


# ---------------------------------------------------------------- selection

@pytest.mark.parametrize("why", ["scale", "score", "block"])
@pytest.mark.parametrize("n_first,n_last,n_sel", [(1, 2, 8), (0, 1, 1), (3, 5, 8), (2, 0, 9)])
def test_first_and_last_blocks_come_before_those_without_a_score(n_first, n_last, n_sel, why):
    """More blocks of keys that are not finite, of scores beyond fp32 and of bad table entries
    than a request selects: its first and last ones, the one being filled among them, stay."""
    nb, Hkv, odd = 40, 2, range(4, 37)
    bounds = random_bounds(nb + 8, Hkv, 12)
    q = rand(2, 4, ref.D, dtype=torch.bfloat16, seed=13)
    table = torch.randperm(nb + 8, generator=torch.Generator().manual_seed(14))[:nb].to(torch.int32).repeat(2, 1)
    ids = table[0, 4:37].long()
    if why == "scale":
        bounds[ids] = ref.pack_records(torch.zeros(len(ids), Hkv, 2, ref.D, dtype=torch.int64), torch.full((len(ids), Hkv), math.inf))
    elif why == "score":  # the largest key where the query's code is positive, the smallest where it is negative
        codes = torch.stack([torch.full((ref.D,), 127), torch.full((ref.D,), -127)]).expand(len(ids), Hkv, 2, ref.D)
        bounds[ids] = ref.pack_records(codes, torch.full((len(ids), Hkv), 1e36))
    else:
        table[0, 4:37] = -1
    sel, err = select(q, bounds.cuda(), table.cuda(), [nb * 16 - 3, 20], n_sel, n_first, n_last)
    assert err == (clo.FLAG_BAD_INDEX if why == "block" else 0)
    keep = list(range(n_first)) + list(range(nb - n_last, nb))
    want = sorted(keep + list(odd)[:n_sel - len(keep)])
    for h in range(Hkv):
        assert sel[0, h].tolist() == want
        assert sel[1, h].tolist() == ([0, 1] + [-1] * n_sel)[:n_sel] if n_sel > 1 else [1]


@pytest.mark.parametrize("Hkv", [1, 8, 9, 32])
def test_select_for_any_number_of_heads(Hkv):
    """Up to eight heads share a CTA's records, and more take several; after calls with fewer."""
    check_select([500, 30, 0, 777], 2, Hkv, 12, 1, 2, torch.bfloat16, Hkv)


# ---------------------------------------------------------------- short contexts

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,Hkv", [(1, 4), (3, 2), (5, 1), (7, 2), (4, 1)])
@pytest.mark.parametrize("T,cached", [(129, 0), (300, 0), (1000, 0), (190, 37)])
def test_first_rows_of_a_prompt_are_as_exact_as_the_output(T, cached, G, Hkv, dtype):
    """The rows of a tile (of as many whole tokens as make 128 rows) whose last one sees at
    most 128 tokens have weights of twice the bits, however long the prompt is.  What is left:
    the output's own rounding; weights of 2^-16 (bf16) or 2^-22 (fp16) of themselves, so
    2^-15 together with their sum; the scores' and the sums' roundings in fp32, as in
    check_attention."""
    n = T - (cached if G > 1 else 0)  # (with one head a tile is 128 tokens)
    kc, vc, table = ref.make_cache([T], Hkv, dtype, T + G, fill=float("nan"))
    q = queries(n, G * Hkv, dtype, T + G + 1)
    out, _, err = chunk(q, kc, vc, table, [T], [n])
    assert err == 0
    want, _, mag, size = ref.chunk_attention(q, kc, vc, table, [T], [n])
    tile = 128 // G
    rows = [i for i in range(n) if T - n + min(n, (i // tile + 1) * tile) <= 128]  # of tiles that end within 128 tokens
    assert rows
    d = 2.0 ** -19 * size + 2.0 ** -20
    tol = ref.half_step(dtype) * want.abs() + (2.0 ** -15 + 2 * d[..., None] + 16 * 2.0 ** -23) * mag + 2.0 ** -24
    err = (out.double() - want).abs()
    assert (err[rows] <= tol[rows]).all()


# ---------------------------------------------------------------- rows that are made anew

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channel", [0, 37, 127])
@pytest.mark.parametrize("T,n,Hq,num_ctas", [(9000, 4, 4, 0), (9000, 9, 4, 0), (700, 200, 4, 0), (700, 200, 4, 1), (2000, 5, 16, 5)])
def test_rows_made_anew_keep_their_lse(T, n, Hq, num_ctas, channel, dtype):
    """A V that is not finite, in one channel of a request's last token, which its other rows do
    not see: those are right, and their lse has the bits that it has beside a finite V, also
    where several blocks put the channels of one row together."""
    kc, vc, table = ref.make_cache([T], 2, dtype, 51, fill=float("nan"))
    q = queries(n, Hq, dtype, 52)
    want = ref.chunk_attention(q, kc, vc, table, [T], [n])
    plain, lse0, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0
    vc[table[0, (T - 1) // 16].long(), :, (T - 1) % 16, channel] = math.nan
    first = None
    for _ in range(3):
        out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
        assert err == 0 and torch.equal(lse, lse0)
        ref.check_attention(out[:-1], lse[:-1], tuple(x[:-1] for x in want), T)
        assert torch.isnan(out[-1, :, channel]).all()
        others = torch.arange(ref.D, device="cuda") != channel
        assert torch.equal(out[-1][:, others], plain[-1][:, others])
        assert first is None or torch.equal(out.nan_to_num(7.0), first.nan_to_num(7.0))
        first = out


# ---------------------------------------------------------------- scores that are not finite

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,num_ctas", [(9000, 3, 0), (9000, 3, 1), (20000, 1, 0), (700, 200, 0)])
def test_queries_of_nan_give_nan(T, n, num_ctas, dtype):
    """However the work is split: a row that sees tokens is not one that sees none."""
    kc, vc, table = ref.make_cache([T], 2, dtype, 61, fill=float("nan"))
    q = queries(n, 8, dtype, 62)
    want = ref.chunk_attention(q, kc, vc, table, [T], [n])
    q[n // 2, 5, 7] = math.nan
    out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0
    assert torch.isnan(out[n // 2, 5]).all() and torch.isnan(lse[n // 2, 5])
    keep = torch.ones(n, 8, dtype=torch.bool, device="cuda")
    keep[n // 2, 5] = False
    ref.check_attention(out[keep], lse[keep], tuple(x[keep] for x in want), T)


@pytest.mark.parametrize("dtype", DTYPES)
def test_keys_of_nan_give_nan(dtype):
    """A long run of keys without a number, which some pieces of the work lie in altogether."""
    T = 40000
    kc, vc, table = ref.make_cache([T], 2, dtype, 63)
    kc[table[0, 500:2000].long(), 1, :, 9] = math.nan
    q = queries(1, 8, dtype, 64)
    out, lse, err = chunk(q, kc, vc, table, [T], [1])
    assert err == 0 and torch.isfinite(out[:, :4]).all() and torch.isnan(out[:, 4:]).all() and torch.isnan(lse[:, 4:]).all()
    sel = torch.arange(500, 2000, dtype=torch.int32, device="cuda").expand(1, 2, 1500).contiguous()
    out, lse, err = sparse(q, kc, vc, table, [T], sel)
    assert err == 0 and torch.isfinite(out[:, :4]).all() and torch.isnan(out[:, 4:]).all() and torch.isnan(lse[:, 4:]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_piece_of_keys_of_nan_behind_what_a_row_sees(dtype):
    """The keys from 384 on are without a number, and so is every row that sees one, though the
    last piece of the work holds nothing else of it than those and tokens that it does not see."""
    T, n = 640, 256
    kc, vc, table = ref.make_cache([T], 1, dtype, 67)
    kc[table[0, 24:].long()] = math.nan
    q = queries(n, 1, dtype, 68)
    for num_ctas in (0, 1, 2, 5):
        out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
        assert err == 0 and torch.isnan(out).all() and torch.isnan(lse).all(), num_ctas


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,num_ctas", [(9000, 4, 0), (300, 200, 0), (300, 200, 1)])
def test_rows_made_anew_leave_out_scores_of_minus_infinity(T, n, num_ctas, dtype):
    """Keys of -infinity, the first one's among them, weigh nothing, whether or not the rows are
    made anew for a V that they do not see."""
    kc, vc, table = ref.make_cache([T], 2, dtype, 65)
    q = queries(n, 8, dtype, 66)
    q[..., 3] = q[..., 3].abs() + 0.5
    for t in (0, 1, 70):
        kc[table[0, t // 16].long(), :, t % 16, 3] = -math.inf
    plain, lse0, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0
    k64, v64 = (ref.cached(x, table, 0, T) for x in (kc, vc))
    left = torch.tensor([t for t in range(T) if t not in (0, 1, 70)], device="cuda")
    sees = torch.stack([(left < T - (n - 1 - i)).sum() for i in range(n)]).repeat_interleave(4)
    vc[table[0, (T - 1) // 16].long(), :, (T - 1) % 16, 50] = math.nan
    out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0 and torch.equal(lse, lse0)
    for h in range(2):
        rows = q[:, 4 * h:4 * h + 4].double().reshape(4 * n, ref.D)
        want = ref.attend(rows, k64[h, left], v64[h, left], sees, 1 / math.sqrt(ref.D))
        want = [x.view(n, 4, *x.shape[1:]) for x in want]
        ref.check_attention(plain[:, 4 * h:4 * h + 4], lse0[:, 4 * h:4 * h + 4], want, T)
        ref.check_attention(out[:-1, 4 * h:4 * h + 4], lse[:-1, 4 * h:4 * h + 4], [x[:-1] for x in want], T)


# ---------------------------------------------------------------- the largest values

@pytest.mark.parametrize("T,n,num_ctas", [(333, 50, 0), (333, 50, 1), (9000, 3, 0), (9000, 3, 1), (5000, 130, 0), (100, 100, 0)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_values_of_65504_stay_finite(sign, T, n, num_ctas):
    """In whole items and in ones that the joining kernel puts together."""
    dtype = torch.float16
    kc, vc, table = ref.make_cache([T], 1, dtype, 41)
    vc.fill_(sign * 65504.0)
    q = queries(n, 4, dtype, 42)
    out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0 and torch.isfinite(out).all() and (out.abs() <= 65504).all()
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, [T], [n]), T)
    vc[..., ::2] *= -1
    out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0 and torch.isfinite(out).all() and (out.abs() <= 65504).all()
    ref.check_attention(out, lse, ref.chunk_attention(q, kc, vc, table, [T], [n]), T)


def wide_values(vc, seed):
    """Random values of one size in each quarter of the channels: 2^125 at most 2^127, 2^100, 1 and 2^-100."""
    v = torch.randn(vc.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    size = torch.tensor([2.0 ** 125, 2.0 ** 100, 1.0, 2.0 ** -100], dtype=torch.float64).repeat_interleave(32)
    top = torch.finfo(torch.bfloat16).max
    vc.copy_((v * size).clamp(-top, top).to(torch.bfloat16))


def check_wide(out, lse, want, tokens):
    """As ref.check_attention (bf16), without a part that does not scale with the values: bf16
    weights as small as 2^-126 count, and 2^-149 times 2^14 is far below 2^-100."""
    o, e, mag, size = want
    u = ref.half_step(out.dtype)
    d = 2.0 ** -19 * size + 2.0 ** -20
    tol = (2 * u + 2 * d[..., None] + tokens / 8 * 2.0 ** -23) * mag + u * o.abs()
    assert torch.isfinite(out).all()
    assert ((out.double() - o).abs() <= tol).all()
    ref.check_attention(torch.zeros_like(out), lse, (torch.zeros_like(o), e, mag, size), tokens)


@pytest.mark.parametrize("T,n,G,num_ctas", [(1, 1, 4, 0), (40, 40, 1, 0), (333, 50, 4, 0), (333, 50, 5, 1), (9000, 3, 4, 0), (9000, 3, 4, 1),
                                            (3000, 100, 8, 0), (700, 700, 3, 3)])
def test_large_bf16_values(T, n, G, num_ctas):
    """bf16 values near its largest, where sums of weights times values pass fp32's: in whole
    items and in ones that the joining kernel puts together."""
    dtype = torch.bfloat16
    kc, vc, table = ref.make_cache([T], 2, dtype, 71)
    q = queries(n, 2 * G, dtype, 72)
    top = torch.finfo(dtype).max
    for values in ("wide", "top", "signs"):
        if values == "wide":
            wide_values(vc, T)
        elif values == "top":
            vc.fill_(top)
        else:
            vc[:, :, ::2] *= -1
        out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
        assert err == 0
        check_wide(out, lse, ref.chunk_attention(q, kc, vc, table, [T], [n]), T)
        if values == "top":
            assert torch.all(out == top)
    # beside an infinity that is seen, and a NaN that is not
    wide_values(vc, T)
    want = ref.chunk_attention(q, kc, vc, table, [T], [n])
    vc[table[0, 0].long(), :, 0, 5] = math.inf
    if T > 1:
        vc[table[0, (T - 1) // 16].long(), 0, (T - 1) % 16, 9] = math.nan
    out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0 and not torch.isfinite(out[..., 5]).any()
    rest = [c for c in range(ref.D) if c not in (5, 9)]
    check_wide(out[..., rest], lse, (want[0][..., rest], want[1], want[2][..., rest], want[3]), T)
    if T > 1 and n > 1:
        assert torch.isnan(out[-1, :G, 9]).all()
        check_wide(out[:-1, :, 9:10], None, (want[0][:-1, :, 9:10], None, want[2][:-1, :, 9:10], want[3][:-1]), T)


@pytest.mark.parametrize("T,n,G,num_ctas", [(40, 40, 1, 0), (333, 50, 4, 1), (9000, 3, 4, 0), (3000, 100, 8, 0)])
def test_large_bf16_values_beside_small_ones(T, n, G, num_ctas):
    """Channels of 2^-100 between channels of 2^125: those keep the bits that they have beside
    values of usual size, also where the rows are made anew."""
    dtype = torch.bfloat16
    kc, vc, table = ref.make_cache([T], 2, dtype, 73)
    q = queries(n, 2 * G, dtype, 74)
    small = [c for c in range(ref.D) if c % 4 != 1]
    vc[..., small] *= 2.0 ** -100
    plain, lse0, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0
    vc[..., 1::4] *= 2.0 ** 125
    out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
    assert err == 0 and torch.equal(out[..., small], plain[..., small]) and torch.equal(lse, lse0)
    want = ref.chunk_attention(q, kc, vc, table, [T], [n])
    check_wide(out[..., 1::4], lse, (want[0][..., 1::4], want[1], want[2][..., 1::4], want[3]), T)
    if T > 1:  # a V that most rows do not see, in a small channel
        vc[table[0, (T - 1) // 16].long(), :, (T - 1) % 16, 2] = math.nan
        out, lse, err = chunk(q, kc, vc, table, [T], [n], num_ctas)
        assert err == 0 and torch.isnan(out[-1, :, 2]).all()
        others = [c for c in small if c != 2]
        assert torch.equal(out[..., others], plain[..., others]) and torch.equal(lse, lse0)
        check_wide(out[:-1], lse[:-1], tuple(x[:-1] for x in want), T)


@pytest.mark.parametrize("num_ctas", [0, 5])
def test_large_bf16_values_of_some_requests(num_ctas):
    """Among many requests, in a cache whose heads lie side by side, captured and replayed: the
    others keep the bits that they have beside values of usual size."""
    g = torch.Generator().manual_seed(75)
    n_new = torch.randint(0, 5, (60,), generator=g).tolist()
    n_new[7], n_new[31], n_new[32] = 300, 40, 1
    lens = [n + int(torch.randint(0, 300, (1,), generator=g)) for n in n_new]
    lens[32] = 6000
    dtype, Hkv, Hq = torch.bfloat16, 2, 10
    kc, vc, table = ref.make_cache(lens, Hkv, dtype, 76)
    q = queries(sum(n_new), Hq, dtype, 77)
    plain, lse0, err = chunk(q, kc, vc, table, lens, n_new, num_ctas)
    assert err == 0
    wide = vc.clone()
    wide_values(wide, 78)
    large = [r for r in range(60) if r % 3 == 1 or r == 32]
    for r in large:
        ids = table[r, :ref.blocks_of(lens[r])].long()
        vc[ids] = wide[ids]
    k2, v2 = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(clo.clo_paged_chunk_workspace_size(Hq, Hkv, num_ctas=num_ctas), dtype=torch.uint8, device="cuda")
    call = clo.prepare_paged_chunk_attn(q, k2, v2, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets_of(n_new), out,
                                        ws, lse=lse, err_flag=err, num_ctas=num_ctas)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    first = out.clone()
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(out, first) and torch.equal(lse, lse0)
    want = ref.chunk_attention(q, kc, vc, table, lens, n_new)
    rows = offsets_of(n_new).tolist()
    for r in range(60):
        s = slice(rows[r], rows[r + 1])
        if r not in large:
            assert torch.equal(out[s], plain[s])
        elif n_new[r]:
            check_wide(out[s], lse[s], tuple(x[s] for x in want), max(lens))


@pytest.mark.parametrize("G,Hkv,n_sel,num_ctas", [(4, 2, 1, 0), (1, 3, 7, 0), (5, 2, 20, 1), (8, 1, 300, 0), (2, 2, 64, 3)])
def test_large_bf16_values_of_selected_blocks(G, Hkv, n_sel, num_ctas):
    dtype, lens = torch.bfloat16, [1, 900, 16 * n_sel, 16 * n_sel + 5, 33]
    kc, vc, table = ref.make_cache(lens, Hkv, dtype, n_sel)
    wide_values(vc, n_sel)
    g = torch.Generator().manual_seed(n_sel)
    sel = torch.full((5, Hkv, n_sel), -1, dtype=torch.int32)
    for r, T in enumerate(lens):
        for h in range(Hkv):
            cols = torch.randperm(ref.blocks_of(T), generator=g)[:n_sel].to(torch.int32)
            sel[r, h, :len(cols)] = cols
    sel = sel.cuda()
    q = queries(5, G * Hkv, dtype, n_sel + 1)
    out, lse, err = sparse(q, kc, vc, table, lens, sel, num_ctas)
    assert err == 0
    check_wide(out, lse, sparse_ref(q, kc, vc, table, lens, sel), max(lens))
    if n_sel > 1:
        sel[1:3] = sel[1:3, :, :1]  # one column as often as there is room
        out, lse, err = sparse(q, kc, vc, table, lens, sel, num_ctas)
        assert err == 0
        check_wide(out, lse, sparse_ref(q, kc, vc, table, lens, sel), max(lens))


# ---------------------------------------------------------------- outputs at any 16-byte boundary

@pytest.mark.parametrize("T,n,num_ctas", [(200, 150, 0), (3000, 2, 0), (700, 700, 0), (700, 700, 3)])
def test_outputs_at_a_16_byte_boundary(T, n, num_ctas):
    dtype = torch.bfloat16
    kc, vc, table = ref.make_cache([T], 2, dtype, 43)
    q = queries(n, 8, dtype, 44)
    want, _, _ = chunk(q, kc, vc, table, [T], [n], num_ctas)
    room = torch.full((q.numel() + 16,), 5.0, dtype=dtype, device="cuda")
    out = room[8:8 + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16
    ws = torch.empty(clo.clo_paged_chunk_workspace_size(8, 2, num_ctas=num_ctas), dtype=torch.uint8, device="cuda")
    clo.clo_paged_chunk_attn(q, kc, vc, table, torch.tensor([T], dtype=torch.int32, device="cuda"), offsets_of([n]), out, ws,
                             num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.all(room[:8] == 5) and torch.all(room[-8:] == 5)
