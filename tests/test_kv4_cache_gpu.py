"""clo_kv4_append and clo_kv4_gather on the GPU against the plain reference.

The pairs must be the reference's bit for bit, and so must the codes, but for
elements whose quotient lies within 1e-5 of the border between two codes (the
kernel's fp32 quotient is off by less than 15 * 2^-22 = 4e-6), which may be
either."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import offloaded_kv_decode_gb300 as clo
from gpu_util import dev

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def rows(N, Hkv, dt, seed, fused=False):
    """K and V rows [N][Hkv][128]: keys with offset channels, a constant group,
    tiny values, a large one; taken out of wider rows if fused."""
    g = torch.Generator().manual_seed(seed)
    cols = 3 * Hkv * 128 if fused else 0
    both = torch.randn(N, cols + 2 * Hkv * 128, generator=g)
    k = both[:, cols:cols + Hkv * 128].view(N, Hkv, 128)
    v = both[:, cols + Hkv * 128:].view(N, Hkv, 128)
    k += 4 * torch.randn(1, Hkv, 128, generator=g)
    k[N // 2, 0] = -3.25
    v[N // 3] *= 1e-5
    v[N - 1, Hkv - 1, 77] = 900.0
    both = both.to(dt).to(dev())
    return both[:, cols:cols + Hkv * 128].view(N, Hkv, 128), both[:, cols + Hkv * 128:].view(N, Hkv, 128)


def append(k, v, slots, pool):
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    clo.clo_kv4_append(k, v, slots, pool, err_flag=err)
    torch.cuda.synchronize()
    return int(err.item())


def check_rows(pool, slots, k, v, group):
    """The records' rows at `slots` hold the reference's codes and pairs."""
    rec = pool.cpu().numpy()
    kc, vc, par = ref.unpack(rec, group)
    near = 0
    for i, (x, codes) in enumerate(((k, kc), (v, vc))):
        c, s, z, border = ref.quantise(x.double().cpu().numpy(), group)
        got = codes[slots // 16, :, slots % 16]
        pairs = par[slots // 16, :, slots % 16, i]
        assert np.array_equal(pairs[..., 0], s.astype(np.float64), equal_nan=True)
        assert np.array_equal(pairs[..., 1], z.astype(np.float64), equal_nan=True)
        off = got != c
        assert np.all(border[off] < 1e-5) and np.all(np.abs(got - c)[off] <= 1)
        near += int(off.sum())
    return near


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,Hkv,fused", [(1, 1, False), (17, 3, True), (133, 8, False), (700, 2, True)])
def test_append_matches_reference(N, Hkv, fused, group, dtype):
    k, v = rows(N, Hkv, DT[dtype], N + group, fused)
    nb = N // 16 + 3
    g = torch.Generator().manual_seed(N)
    slots = torch.randperm(nb * 16, generator=g)[:N].to(torch.int32)
    pool = torch.randint(0, 256, (nb, Hkv, ref.record_bytes(group)), dtype=torch.uint8, generator=g)
    before = pool.numpy().copy()
    pool = pool.to(dev())
    assert append(k, v, slots.to(dev()), pool) == 0
    near = check_rows(pool, slots.numpy(), k, v, group)
    assert near <= 2
    # Every byte that belongs to no row of the call is as it was.
    expect = before
    ref.write_rows(expect, slots.numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), group)
    differ = np.argwhere(expect != pool.cpu().numpy())
    assert len(differ) <= near or np.isnan(expect[:, :, 2048:].copy().view(np.float16)).any()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_append_non_finite_groups_and_saturation(group):
    """A NaN or an infinity makes its own group read NaN and no other; bf16
    values beyond fp16's range are taken as its largest."""
    for dt in (torch.float16, torch.bfloat16):
        k, v = rows(4, 2, dt, 5)
        k[0, 0, 3] = float("nan")
        k[1, 1, 127] = float("inf")
        v[2, 0, 64] = -float("inf")
        v[2, 1, 0] = float("nan")
        if dt == torch.bfloat16:
            v[3, 0, 5], v[3, 0, 6] = 3e38, -1e5
        pool = torch.zeros(1, 2, ref.record_bytes(group), dtype=torch.uint8, device=dev())
        slots = torch.tensor([3, 0, 15, 8], dtype=torch.int32, device=dev())
        assert append(k, v, slots, pool) == 0
        assert check_rows(pool, slots.cpu().numpy(), k, v, group) <= 2
        ko, vo = (torch.empty(4, 2, 128, dtype=dt, device=dev()) for _ in range(2))
        clo.clo_kv4_gather(pool, slots, ko, vo)
        for x, y in ((k, ko), (v, vo)):
            hurt = (~torch.isfinite(x)).view(4, 2, -1, group).any(-1, keepdim=True).expand(4, 2, 128 // group, group)
            assert torch.equal(torch.isnan(y), hurt.reshape(4, 2, 128))


def test_append_skips_and_flags():
    k, v = rows(6, 2, torch.float16, 9)
    pool = torch.full((2, 2, ref.record_bytes(64)), 7, dtype=torch.uint8, device=dev())
    before = pool.clone()
    only_padding = torch.full((6,), -1, dtype=torch.int32, device=dev())
    assert append(k, v, only_padding, pool) == 0 and torch.equal(pool, before)
    bad = torch.tensor([32, -2, 1 << 30, -(1 << 31), 2 ** 31 - 1, -1], dtype=torch.int32, device=dev())
    assert append(k, v, bad, pool) == clo.FLAG_BAD_INDEX and torch.equal(pool, before)
    some = torch.tensor([31, -1, 0, 32, 5, -1], dtype=torch.int32, device=dev())
    assert append(k, v, some, pool) == clo.FLAG_BAD_INDEX
    check_rows(pool, np.array([31, 0, 5]), k[[0, 2, 4]], v[[0, 2, 4]], 64)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,Hkv", [(1, 1), (45, 3), (1000, 8)])
def test_gather_matches_reference(N, Hkv, group, dtype):
    """Each element is the fp64 value rounded to the type: off by at most half a
    step of it, and 2^-23 for the fp32 value in between."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(N + group)
    nb = 9
    pool = torch.randint(0, 256, (nb, Hkv, ref.record_bytes(group)), dtype=torch.uint8, generator=g)
    par = torch.randn(nb, Hkv, (ref.record_bytes(group) - 2048) // 2, generator=g).half()
    pool[:, :, 2048:] = par.view(torch.uint8)
    slots = torch.randint(0, nb * 16, (N,), generator=g).to(torch.int32)  # slots repeat
    if N > 10:
        slots[3], slots[N - 1], slots[7] = -1, -1, nb * 16
    k, v = (torch.full((N, Hkv, 128), float("nan"), dtype=dt, device=dev()) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=dev())
    clo.clo_kv4_gather(pool.to(dev()), slots.to(dev()), k, v, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == (clo.FLAG_BAD_INDEX if N > 10 else 0)
    s = slots.numpy()
    live = (s >= 0) & (s < nb * 16)
    at = np.where(live, s, 0)
    for x, val in zip((k, v), ref.values(pool.numpy(), group)):
        want = np.where(live[:, None, None], val[at // 16, :, at % 16], 0.0)
        got = x.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= (ref.U16[dt] + 2.0 ** -23) * np.abs(want) + ref.TINY[dt])


def test_round_trip_on_another_stream_and_in_a_graph():
    """Append and read-back of the same rows, captured on a side stream and
    replayed after the inputs changed in place."""
    N, Hkv, group = 300, 4, 32
    k, v = rows(N, Hkv, torch.bfloat16, 21)
    pool = torch.zeros(20, Hkv, ref.record_bytes(group), dtype=torch.uint8, device=dev())
    slots = torch.randperm(320, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32).to(dev())
    ko, vo = (torch.empty(N, Hkv, 128, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    a = clo.prepare_kv4_append(k, v, slots, pool)
    b = clo.prepare_kv4_gather(pool, slots, ko, vo)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a(), b()
    side.synchronize()
    first = ko.clone(), vo.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a(), b()
    ko.zero_(), vo.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ko, first[0]) and torch.equal(vo, first[1])
    k.neg_(), v.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert check_rows(pool, slots.cpu().numpy(), k, v, group) <= 2
    # The read-back is within half a code's step and its own rounding of the
    # row: the cached value is at most |x| + half, and bf16 rounds by 2^-8 of it.
    for x, y in ((k, ko), (v, vo)):
        _, s, z, _ = ref.quantise(x.double().cpu().numpy(), group)
        half = np.repeat(s.astype(np.float64), group, -1) / 2
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        assert np.all(np.abs(y - x) <= half * (1 + 1e-6) + 2.0 ** -8 * (np.abs(x) + half) + 1e-7)


def test_records_past_4_gib():
    """Blocks whose byte offset does not fit 32 bits."""
    Hkv, group = 64, 32
    R = ref.record_bytes(group)
    nb = (5 << 30) // (Hkv * R)
    pool = torch.empty(nb, Hkv, R, dtype=torch.uint8, device=dev())
    k, v = rows(6, Hkv, torch.float16, 3)
    blocks = [0, 1, nb // 2, nb - 2, nb - 1, (1 << 32) // (Hkv * R)]
    slots = torch.tensor([b * 16 + 3 * i for i, b in enumerate(blocks)], dtype=torch.int32, device=dev())
    assert append(k, v, slots, pool) == 0
    for i, b in enumerate(blocks):
        check_rows(pool[b:b + 1], np.array([3 * i]), k[i:i + 1], v[i:i + 1], group)
    ko, vo = (torch.empty(6, Hkv, 128, dtype=torch.float16, device=dev()) for _ in range(2))
    clo.clo_kv4_gather(pool, slots, ko, vo)
    for i, b in enumerate(blocks):
        val = ref.values(pool[b].cpu().numpy(), group)[0][:, 3 * i]
        assert np.all(np.abs(ko[i].double().cpu().numpy() - val) <= (2.0 ** -11 + 2.0 ** -23) * np.abs(val) + 2.0 ** -25)


def test_refused_tensors():
    k, v = rows(4, 2, torch.float16, 1)
    pool = torch.zeros(2, 2, 2304, dtype=torch.uint8, device=dev())
    s = torch.zeros(4, dtype=torch.int32, device=dev())
    for bad in (lambda: clo.clo_kv4_append(k, v.bfloat16(), s, pool),
                lambda: clo.clo_kv4_append(k, v, s.long(), pool),
                lambda: clo.clo_kv4_append(k, v, s[:3], pool),
                lambda: clo.clo_kv4_append(k, v, s, pool[:, :1].contiguous()),
                lambda: clo.clo_kv4_append(k, v, s, pool[:, :, :2300].contiguous()),
                lambda: clo.clo_kv4_append(k.transpose(0, 1), v.transpose(0, 1), s[:2], pool),
                lambda: clo.clo_kv4_append(k[:, :, :64], v[:, :, :64], s, pool),
                lambda: clo.clo_kv4_gather(pool, s, k[:, ::2], v[:, ::2]),
                lambda: clo.clo_kv4_gather(pool, s, k, v.bfloat16()),
                lambda: clo.prepare_kv4_gather(pool, s[:2], k, v)):
        with pytest.raises(clo.CloError):
            bad()
    misaligned = torch.zeros(4 * 2 * 128 + 1, dtype=torch.float16, device=dev())[1:].view(4, 2, 128)
    with pytest.raises(clo.CloError):
        clo.clo_kv4_append(misaligned, v, s, pool)
    empty = k[:0]
    clo.clo_kv4_append(empty, empty, s[:0], pool)
    clo.clo_kv4_gather(pool, s[:0], empty.clone(), empty.clone())
    torch.cuda.synchronize()


def test_refused_while_another_device_is_current(monkeypatch):
    """The call's kernels would start on the other device."""
    k, v = rows(4, 2, torch.float16, 1)
    pool = torch.zeros(2, 2, 2304, dtype=torch.uint8, device=dev())
    s = torch.arange(4, dtype=torch.int32, device=dev())
    call = clo.prepare_kv4_append(k, v, s, pool)
    call()
    kc, vc = k.contiguous(), v.contiguous()
    clo.prepare_kv4_gather(pool, s, kc, vc)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for again in (call, lambda: clo.clo_kv4_append(k, v, s, pool), lambda: clo.prepare_kv4_gather(pool, s, kc, vc)):
        with pytest.raises(clo.CloError, match="current device"):
            again()
