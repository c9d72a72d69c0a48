"""How far clo_kv4_paged_decode_attn is from the 64-bit result over all its
outputs together: the 2-norm of the error, and its mean, which shows what the
element-wise tolerance of kv4_ref.attention leaves room for.

The model, per output o = sum_t p_t V_t with V = code * s + z, u = U16 of the
type (2^-11, 2^-8) and w = 2^-11:
  * the output's own rounding, uniform within u |o|: u |o| / sqrt(3) at most in
    the root mean square;
  * the weights p s, rounded to fp16, each uniform within w of itself and
    independent.  For fp16 outputs they meet the codes counted from 7.5, for
    bf16 the codes themselves: w / sqrt(3) * sqrt(sum_t (p s (code - c))^2);
  * fp32 sums.  The matrix instructions cut their sums off, toward zero, so that
    what they lose adds up; MASS * 2^-24 of sum_t p s code is allowed for it."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# An addition sums 16 products and the accumulator, each cut off at the last place
# of the largest, 2^-23 of it: 17 / 2 of those on average.  After 32 additions
# what the sums have in common is taken out of the accumulators.  So as much as
# 32 * 17 / 2 * 2^-23 of an accumulator that has its size from the start, as it has
# behind one heavy token; and of one that grows, in the 64 additions at most of the
# kernel for short contexts.
MASS = 544


def make_pool(nb, Hkv, group, g):
    """Bell-shaped codes, V without a mean: zero near -7.5 scales."""
    ng = 128 // group
    pool = torch.randint(0, 256, (nb, Hkv, ref.record_bytes(group)), dtype=torch.uint8, device=dev(), generator=g)
    pool[:, :, :2048] = (pool[:, :, :2048] & 0x77) + (torch.randint(
        0, 256, (nb, Hkv, 2048), dtype=torch.uint8, device=dev(), generator=g) & 0x77)
    scale = torch.rand(nb, Hkv, 32 * ng, device=dev(), generator=g) * 0.35 + 0.05
    zero = -scale * (7.0 + 0.5 * torch.randn(scale.shape, device=dev(), generator=g))  # the codes' mean is 7
    pool[:, :, 2048:] = torch.stack([scale, zero], -1).half().view(torch.uint8).flatten(2)
    return pool


def head_rows(pool, blocks, h, group):
    """fp64 K, and V's codes, scales and zeros, [tokens][128] each, of one KV head."""
    rec = pool[blocks.long(), h]
    n = rec.shape[0]
    sh = torch.from_numpy(ref.SH).to(dev())
    k, v = (((rec[:, torch.from_numpy(at.ravel()).to(dev())].view(n, 16, 128) >> sh) & 15).double().view(-1, 128)
            for at in (ref.KB, ref.VB))
    par = rec[:, 2048:].contiguous().view(torch.float16).double().view(n * 16, 2, 128 // group, 2)
    par = par.repeat_interleave(group, 2)
    return k * par[:, 0, :, 0] + par[:, 0, :, 1], v, par[:, 1, :, 0], par[:, 1, :, 1]


def measure(q, pool, table, n, group, num_ctas=0):
    """The call for one request of n tokens, and how far its outputs are off."""
    _, n_q, Hq, _ = q.shape
    Hkv = pool.shape[1]
    out = torch.empty_like(q)
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(1, n_q, Hq, Hkv, 128, num_ctas), dtype=torch.uint8, device=dev())
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    clo.clo_kv4_paged_decode_attn(q, pool, table, torch.tensor([n], dtype=torch.int32, device=dev()), out, ws,
                                  err_flag=err, num_ctas=num_ctas)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return compare(out[0], q[0], pool, table[0], n, group, range(Hkv))


def compare(out, q, pool, blocks, n, group, heads):
    """The sums of the model over one request's outputs [n_q][Hq][128] of some KV
    heads: dict of the error's, the output's, and the expected errors' mean
    squares, the mean error, and the mean of sum_t p s code; and their number."""
    n_q, Hq, _ = q.shape
    G = Hq // pool.shape[1]
    sums = {x: 0.0 for x in ("err2", "out2", "weights2", "plain2", "mean", "mass")}
    for h in heads:
        K, code, s, z = head_rows(pool, blocks[:-(-n // 16)], h, group)
        for i in range(n_q):
            m = n - (n_q - 1 - i)
            x = q[i, h * G:(h + 1) * G].double() @ K[:m].T * ref.scale_for()
            p = torch.softmax(x, -1)
            sc, cd = s[:m], code[:m]
            o = p @ (cd * sc + z[:m])
            d = out[i, h * G:(h + 1) * G].double() - o
            p2 = p * p
            sums["err2"] += float((d * d).sum())
            sums["out2"] += float((o * o).sum())
            sums["weights2"] += float((p2 @ (sc * (cd - 7.5)) ** 2).sum())
            sums["plain2"] += float((p2 @ (sc * cd) ** 2).sum())
            sums["mean"] += float(d.sum())
            sums["mass"] += float((p @ (sc * cd)).sum())
    N = n_q * G * len(heads) * 128
    return {k: v / N for k, v in sums.items()}, N


def check(m, N, dt):
    """The 2-norm is what the roundings give (a tenth more, for chance), and the
    mean error is that of N independent ones (four times its deviation)."""
    u, w = ref.U16[dt], 2.0 ** -11
    weights2 = m["weights2"] if dt == torch.float16 else m["plain2"]
    lost = MASS * 2.0 ** -24 * m["mass"]
    expected2 = (u * u * m["out2"] + w * w * weights2) / 3
    what = f"2-norm {math.sqrt(m['err2'] / m['out2']):.2e}, mean {m['mean'] / math.sqrt(m['out2']):.2e} of the output's"
    assert math.sqrt(m["err2"]) <= 1.1 * math.sqrt(expected2) + lost, what
    assert abs(m["mean"]) <= 4 * math.sqrt(expected2 / N) + lost, what


def one_request(T, n_q, Hq, Hkv, group, dt, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    nb = -(-T // 16) + 1
    pool = make_pool(nb, Hkv, group, g)
    table = torch.randperm(nb, device=dev(), generator=g)[:nb - 1].to(torch.int32)[None].contiguous()
    q = torch.randn(1, n_q, Hq, 128, device=dev(), generator=g).to(dt)
    return q, pool, table


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,n_q", [(32, 8, 1), (32, 2, 1), (16, 2, 4)])
def test_norm_of_the_error(Hq, Hkv, n_q, group, dtype):
    dt = DT[dtype]
    for T, num_ctas in ((1000, 0), (9000, 0), (9000, 3)):
        q, pool, table = one_request(T, n_q, Hq, Hkv, group, dt, T + group)
        m, N = measure(q, pool, table, T, group, num_ctas)
        check(m, N, dt)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group,Hq,n_q", [(32, 8, 1), (128, 8, 1), (64, 32, 1), (32, 8, 8)])
def test_sums_over_many_tokens_do_not_drift(group, Hq, n_q, dtype):
    """One CTA takes 2 * 200003 tokens: 25000 to 50000 a warp."""
    dt = DT[dtype]
    T = 200003
    q, pool, table = one_request(T, n_q, Hq, 2, group, dt, group)
    m, N = measure(q, pool, table, T, group, 1)
    check(m, N, dt)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nats", [10.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("heavy", [0.2, 2.0])
def test_many_light_tokens_beside_a_heavy_one(heavy, nats, dtype):
    """The first token's score is `nats` above the middle of 131071 others', which
    have 0.2 to 85% of the weight between them.  Its V is 0 (code 7, zero -7
    scales; the scale is like the others' or ten times as large), so what is lost
    of the light weights shows: by the end one warp has them all."""
    dt, T, Hkv, group = DT[dtype], 131072, 16, 128
    q, pool, table = one_request(T, 1, Hkv, Hkv, group, dt, 7)
    par = pool[:, :, 2048:].view(torch.float16).view(pool.shape[0], Hkv, 16, 2, 1, 2)
    first = int(table[0, 0])
    total = q[0, 0].double().sum(-1)
    q[0, 0] *= torch.where(total.abs() < 2, 0.0, 1.0)[:, None].to(dt)  # those would need a large key
    K0 = torch.where(total.abs() < 2, 0.0, nats / ref.scale_for() / total)
    par[first, :, 0, 0, :, 0] = 0
    par[first, :, 0, 0, :, 1] = K0.half()[:, None]
    s = torch.tensor(heavy).half()
    par[first, :, 0, 1, :, 0], par[first, :, 0, 1, :, 1] = s.item(), (-7 * s.float()).item()
    pool[first, :, 1024:1024 + 64] = 0x77
    for num_ctas in (0, 20, 1):
        m, N = measure(q, pool, table, T, group, num_ctas)
        check(m, N, dt)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_long_request_among_many_short_ones(dtype):
    """More than four (request, KV head)s for each place a CTA has, one request of
    131072 tokens among them: its sums are not left to a few warps each."""
    dt, T, Hkv, group = DT[dtype], 131072, 32, 64
    places = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    B = 4 * places // Hkv + 2
    g = torch.Generator(device=dev()).manual_seed(3)
    pool = make_pool(T // 16 + 8, Hkv, group, g)
    table = torch.randint(0, pool.shape[0], (B, T // 16), dtype=torch.int32, device=dev(), generator=g)
    table[B // 2] = torch.randperm(pool.shape[0], device=dev(), generator=g)[:T // 16]
    ctx = torch.randint(1, 200, (B,), dtype=torch.int32, device=dev(), generator=g)
    ctx[B // 2] = T
    q = torch.randn(B, 1, Hkv, 128, device=dev(), generator=g).to(dt)
    out = torch.empty_like(q)
    ws = torch.empty(clo.clo_kv4_paged_workspace_size(B, 1, Hkv, Hkv), dtype=torch.uint8, device=dev())
    clo.clo_kv4_paged_decode_attn(q, pool, table, ctx, out, ws)
    m, N = compare(out[B // 2], q[B // 2], pool, table[B // 2], T, group, range(0, Hkv, 4))
    check(m, N, dt)
    for r in (0, B - 1):
        m, N = compare(out[r], q[r], pool, table[r], int(ctx[r]), group, range(Hkv))
        check(m, N, dt)
