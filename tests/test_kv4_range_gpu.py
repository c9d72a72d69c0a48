"""The ends of the value range of the 4-bit cache on the GPU: groups that reach
fp16's largest values, and scales of either sign."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev
from test_kv4_attention_gpu import inputs, run

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
TOP = 65504.0


def wide_rows(dt):
    """Rows [6][1][128] of finite groups that reach the ends of fp16's range."""
    x = torch.zeros(6, 1, 128)
    x[0, 0, ::32] = TOP                                  # 0 .. the largest
    x[1, 0] = torch.linspace(-TOP, TOP, 128)
    x[2, 0, ::32] = -TOP
    x[3] = TOP                                           # constant
    x[4, 0] = torch.tensor([-TOP, TOP]).repeat(64)       # both ends in every group
    x[5, 0] = TOP - 32 * torch.arange(128)               # close to the top
    return x.to(dt).to(dev())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("written", ["f16", "bf16"])
@pytest.mark.parametrize("read", ["f16", "bf16"])
def test_finite_rows_read_back_finite(written, read, group):
    """Within half a scale and the rounding to the type; bf16 rows count as
    clamped to +-65504.  A scale is fp16's next value up, so code 15 may lie up to
    64 above 65504: fp16 then has its largest value."""
    x = wide_rows(DT[written])
    pool = torch.zeros(1, 1, ref.record_bytes(group), dtype=torch.uint8, device=dev())
    slots = torch.arange(6, dtype=torch.int32, device=dev())
    clo.clo_kv4_append(x, x.clone(), slots, pool)
    dt = DT[read]
    k, v = (torch.empty(6, 1, 128, dtype=dt, device=dev()) for _ in range(2))
    clo.clo_kv4_gather(pool, slots, k, v)
    xd = np.clip(x.double().cpu().numpy(), -TOP, TOP)
    _, s, _, _ = ref.quantise(xd, group)
    half = np.repeat(s.astype(np.float64), group, -1) / 2
    vals = ref.values(pool.cpu().numpy(), group)
    for got, val in zip((k, v), vals):
        g = got.double().cpu().numpy()
        assert np.all(np.isfinite(g))
        assert np.all(np.abs(g - xd) <= half + ref.U16[dt] * (np.abs(xd) + half))
        held = val[0, :, :6].transpose(1, 0, 2)
        want = np.clip(held, -TOP, TOP) if dt == torch.float16 else held
        assert np.all(np.abs(g - want) <= (ref.U16[dt] + 2.0 ** -23) * np.abs(want))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_attention_over_rows_at_the_ends_of_the_range_is_finite(group, dtype):
    """One token at a time: the output is that token's V, and fp16's largest value
    where V lies above it."""
    dt = DT[dtype]
    x = wide_rows(dt)
    small = torch.randn(6, 1, 128, device=dev()).to(dt)
    for num_ctas in (0, 2):
        pool = torch.zeros(6, 1, ref.record_bytes(group), dtype=torch.uint8, device=dev())
        clo.clo_kv4_append(small, x, torch.arange(0, 96, 16, dtype=torch.int32, device=dev()), pool)
        q = torch.randn(6, 1, 4, 128, device=dev()).to(dt)
        out = torch.empty_like(q)
        ws = torch.empty(clo.clo_kv4_paged_workspace_size(6, 1, 4, 1, 128, num_ctas), dtype=torch.uint8, device=dev())
        clo.clo_kv4_paged_decode_attn(q, pool, torch.arange(6, dtype=torch.int32, device=dev())[:, None].contiguous(),
                                      torch.ones(6, dtype=torch.int32, device=dev()), out, ws, num_ctas=num_ctas)
        got = out.double().cpu().numpy()
        val = ref.values(pool.cpu().numpy(), group)[1][:, 0, 0][:, None, None]
        want = np.clip(val, -TOP, TOP) if dt == torch.float16 else val
        assert np.all(np.isfinite(got))
        # The weight's rounding (2^-11 of code * scale) and the output's.
        mag = np.abs(val) + 15 * 8736.0
        assert np.all(np.abs(got - want) <= (2.0 ** -11 + 2.0 ** -20) * mag + ref.U16[dt] * (np.abs(want) + 2.0 ** -11 * mag))


@pytest.mark.parametrize("num_ctas", [0, 7])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_of_either_sign(group, dtype, num_ctas):
    """code * scale + zero is defined for a negative scale too: the same values
    with some groups' codes counted down from the top instead of up."""
    dt = DT[dtype]
    q, pool, table, ctx = inputs([700, 33, 5], 2, 8, 2, group, dt, 77)
    rng = np.random.Generator(np.random.PCG64(78))
    par = pool[:, :, 2048:].copy().view(np.float16).reshape(*pool.shape[:2], 16, 2, -1, 2)
    flip = rng.random(par.shape[:-1]) < 0.5
    flip[table[2]] = True  # all of a request's
    with np.errstate(invalid="ignore"):
        par[..., 1] = np.where(flip, par[..., 1] + np.float16(15) * par[..., 0], par[..., 1])
        par[..., 0] = np.where(flip, -par[..., 0], par[..., 0])
    pool[:, :, 2048:] = par.reshape(*pool.shape[:2], -1).view(np.uint8)
    got, lse, err = run(q, pool, table, ctx, num_ctas)
    assert err == 0
    # The reference's tolerance counts magnitudes as code * scale + |zero|: here
    # those of the pairs turned round again, which are the larger of the two ways.
    o, l, _, _ = ref.attention(q.double().numpy(), pool, table, ctx, group, ref.scale_for(), dt)
    turned = par.copy()
    with np.errstate(invalid="ignore"):
        turned[..., 0] = np.abs(par[..., 0])
        turned[..., 1] = np.abs(par[..., 1]) + np.float16(15) * np.abs(par[..., 0])
    high = pool.copy()
    high[:, :, :2048] = 0xff
    high[:, :, 2048:] = turned.reshape(*pool.shape[:2], -1).view(np.uint8)
    K = ref.values(high, group)
    for r in range(3):
        n = int(ctx[r])
        Kmag, Vmag = (x[table[r, :-(-n // 16)]].transpose(1, 0, 2, 3).reshape(2, -1, 128)[:, :n] for x in K)
        for h in range(2):
            qq = np.abs(q.double().numpy()[r, :, 4 * h:4 * h + 4])
            dx = 20 * 2.0 ** -24 * (qq @ Kmag[h].max(0)) * ref.scale_for() + 2.0 ** -22
            inner = (2.0 ** -11 + 2 * dx[..., None]) * Vmag[h].max(0) + n * 2.0 ** -25 * 15 * 0.4
            g, w = got[r, :, 4 * h:4 * h + 4], o[r, :, 4 * h:4 * h + 4]
            assert np.all(np.isfinite(g)) and np.all(np.abs(g - w) <= inner + ref.U16[dt] * (np.abs(w) + inner) + 2.0 ** -25)
            assert np.all(np.abs(lse - l)[r, :, 4 * h:4 * h + 4] <= dx + 2.0 ** -22 * (1 + np.abs(l[r, :, 4 * h:4 * h + 4])))
