"""Plain 64-bit references and inputs for the 16-bit paged cache (clo_paged.h), on
any device, and the error bounds that the roundings give."""
import math

import torch

D, BLOCK, RECORD = 128, 16, 272


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def blocks_of(n):
    return -(-n // BLOCK)


def make_cache(lens, Hkv, dtype, seed, device="cuda", extra=2, fill=None, max_blocks=None):
    """(kc, vc, table): requests of lens cached tokens in scattered blocks; rows that
    belong to no token hold `fill` (None: random values)."""
    g = torch.Generator().manual_seed(seed)
    nb = [blocks_of(n) for n in lens]
    total = sum(nb) + extra
    kc, vc = (torch.randn(total, Hkv, BLOCK, D, generator=g).to(dtype) for _ in range(2))
    ids = torch.randperm(total, generator=g)
    mb = max(max_blocks or 1, max(nb, default=0), 1)
    table = torch.full((len(lens), mb), -1, dtype=torch.int32)
    used = torch.zeros(total, BLOCK, dtype=torch.bool)
    at = 0
    for r, n in enumerate(lens):
        table[r, :nb[r]] = ids[at:at + nb[r]].to(torch.int32)
        for p in range(nb[r]):
            used[ids[at + p], :min(BLOCK, n - p * BLOCK)] = True
        at += nb[r]
    if fill is not None:
        for x in (kc, vc):
            x[~used[:, None].expand(-1, Hkv, -1)] = fill
    return kc.to(device), vc.to(device), table.to(device)


def cached(x, table, r, n):
    """[Hkv][n][D] in 64 bits."""
    ids = table[r, :blocks_of(n)].long()
    return x[ids].transpose(0, 1).reshape(x.shape[1], -1, D)[:, :n].double()


def attend(q, k, v, sees, scale):
    """One KV head: q [m][D], k, v [T][D] in 64 bits, sees [m] tokens.  (out, lse,
    sum of |weights * v|, the largest sum of |q * k| * scale); a row that sees nothing:
    zeros and -inf.  Values that a row does not see never enter."""
    m, T = q.shape[0], k.shape[0]
    out, mag = (torch.zeros(m, D, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full((m,), -math.inf, dtype=torch.float64, device=q.device)
    size = torch.zeros(m, dtype=torch.float64, device=q.device)
    clean = bool(torch.isfinite(v).all() and torch.isfinite(k).all())
    if clean and T:
        x = (q @ k.t()) * scale
        x = x.masked_fill(torch.arange(T, device=q.device)[None] >= sees[:, None], -math.inf)
        some = sees > 0
        lse[some] = torch.logsumexp(x[some], 1)
        w = torch.exp(x[some] - lse[some, None])
        out[some], mag[some] = w @ v, w @ v.abs()
        size[some] = ((q[some].abs() @ k.t().abs()) * scale).amax(1)
        return out, lse, mag, size
    for i, t in enumerate(sees.tolist()):  # row by row, over what it sees alone
        if t > 0:
            o, e, a, z = attend_clean(q[i:i + 1], k[:t], v[:t], scale)
            out[i], lse[i], mag[i], size[i] = o[0], e[0], a[0], z[0]
    return out, lse, mag, size


def attend_clean(q, k, v, scale):
    x = (q @ k.t()) * scale
    w = torch.softmax(x, 1)
    return w @ v, torch.logsumexp(x, 1), w @ v.abs(), ((q.abs() @ k.t().abs()) * scale).amax(1)


def chunk_attention(q, kc, vc, table, lens, n_new, scale=None):
    """(out [N][Hq][D], lse [N][Hq], mag, size) in 64 bits for requests of lens[r] tokens whose last n_new[r] are rows of q."""
    N, Hq, _ = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out, mag = (torch.zeros(N, Hq, D, dtype=torch.float64, device=q.device) for _ in range(2))
    lse, size = (torch.zeros(N, Hq, dtype=torch.float64, device=q.device) for _ in range(2))
    at = 0
    for r, (T, n) in enumerate(zip(lens, n_new)):
        if n == 0:
            continue
        k, v = cached(kc, table, r, T), cached(vc, table, r, T)
        sees = (T - (n - 1 - torch.arange(n, device=q.device))).clamp(min=0).repeat_interleave(G)
        for h in range(Hkv):
            qh = q[at:at + n, h * G:(h + 1) * G].double().reshape(n * G, D)
            o, e, m, z = attend(qh, k[h], v[h], sees, scale)
            out[at:at + n, h * G:(h + 1) * G] = o.view(n, G, D)
            mag[at:at + n, h * G:(h + 1) * G] = m.view(n, G, D)
            lse[at:at + n, h * G:(h + 1) * G] = e.view(n, G)
            size[at:at + n, h * G:(h + 1) * G] = z.view(n, G)
        at += n
    return out, lse, mag, size


def check_attention(out, lse, ref, tokens):
    """The kernel's out and lse against (out, lse, mag, size) in 64 bits.  Each weight is
    rounded once (half a step u), the sum of the weights may differ from that of the
    rounded ones by as much, the output is rounded once; scores and sums are fp32
    sums of 128 terms and of `tokens` terms, cut off at 2^-23 an addition of 8 or 16;
    a score that is off by d scales a weight by 1 + d; weights below 2^-31 of the
    largest may be lost, and fp16 has no step finer than 2^-24."""
    want, want_lse, mag, size = ref
    u = half_step(out.dtype)
    d = 2.0 ** -19 * size + 2.0 ** -20
    lost = tokens * 2.0 ** -31 * 8
    tol = (2 * u + 2 * d[..., None] + tokens / 8 * 2.0 ** -23) * mag + u * want.abs() + lost + 2.0 ** -24
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1, f"{worst} of the bound; error {err.max().item():.3e}"
    if lse is not None:
        fin = torch.isfinite(want_lse)
        assert torch.equal(torch.isneginf(lse), ~fin)
        e = (lse.double() - want_lse)[fin].abs()
        t = (d + tokens / 8 * 2.0 ** -23 + want_lse.abs() * 2.0 ** -22)[fin]
        assert (e <= t).all(), f"lse off by {e.max().item():.3e}"
    return worst


# ---------------------------------------------------------------- positions

def rotate(x, pos, inv_freq, axis, inter):
    """x [N][H][D] turned in 64 bits; pos [axes][N]."""
    n = len(inv_freq)
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device=x.device)
    t = torch.stack([pos[a].double() for a in axis], 1) * f if n else pos[0].double()[:, None][:, :0]
    c, s = t.cos()[:, None], t.sin()[:, None]
    y = x.double().clone()
    a, b = (y[..., 0:2 * n:2].clone(), y[..., 1:2 * n:2].clone()) if inter else (y[..., :n].clone(), y[..., n:2 * n].clone())
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size = x.double().abs().clone()
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def check_rotated(got, want, size):
    """One rounding, of a result whose angle is off by at most pi * 2^-25 (the fraction
    of a turn as fp32) + 2^-22 (the sine's and cosine's own error) and whose two
    products and sum are fp32."""
    u = half_step(got.dtype)
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -130
    tol = u * want.abs() + (math.pi * 2.0 ** -25 + 2.0 ** -22 + 2.0 ** -23) * (1 + u) * size + tiny
    err = (got.double() - want).abs()
    assert (err <= tol).all(), f"off by {(err / tol).max().item()} of the bound"


# ---------------------------------------------------------------- bounds and selection

def bounds_record(rows):
    """One record from keys [m][D]: codes [2][D] (largest, smallest) and the scale; the
    fp32 quotients that define them."""
    f = rows.float()
    if not torch.isfinite(f).all():
        return torch.zeros(2, D, dtype=torch.int64), torch.tensor(math.inf)
    hi, lo = f.amax(0), f.amin(0)
    scale = torch.maximum(hi.abs(), lo.abs()).amax() / torch.tensor(127.0)
    div = scale if scale > 0 else torch.tensor(1.0)
    return torch.stack([(hi / div).ceil(), (lo / div).floor()]).clamp(-127, 127).long(), scale


def unpack_record(rec):
    """(codes [2][D], scale) of a record's bytes."""
    codes = rec[:256].view(torch.int8).view(32, 2, 4).long()
    return codes.transpose(0, 1).reshape(2, D), rec[256:260].clone().view(torch.float32)[0]


def pack_records(codes, scale):
    """Records [...][272] of codes [...][2][D] and scales [...]."""
    lead = scale.shape
    rec = torch.zeros(*lead, RECORD, dtype=torch.uint8)
    c = codes.to(torch.int8).view(*lead, 2, 32, 4).transpose(-2, -3).contiguous()
    rec[..., :256] = c.view(torch.uint8).view(*lead, 256)
    rec[..., 256:260] = scale.float()[..., None].contiguous().view(torch.uint8).view(*lead, 4)
    return rec


def query_codes(q):
    """Codes of the summed queries q [G][D]."""
    s = q[0].float()
    for h in range(1, q.shape[0]):
        s = s + q[h].float()
    if not torch.isfinite(s).all() or s.abs().max() == 0:
        return torch.zeros(D, dtype=torch.int64)
    step = s.abs().max() / torch.tensor(127.0)
    return (s / step).round().clamp(-127, 127).long() if step > 0 else torch.zeros(D, dtype=torch.int64)


def select(q, rec, nb, n_sel, n_first, n_last):
    """Columns for one request and KV head: q [G][D], rec [nb][272] in the order of the columns."""
    if nb <= n_sel:
        return list(range(nb)) + [-1] * (n_sel - nb)
    code = query_codes(q)
    score = []
    for p in range(nb):
        c, scale = unpack_record(rec[p])
        s = float(torch.maximum(code * c[0], code * c[1]).sum().float() * scale) + 0.0
        forced = p < n_first or p >= nb - n_last or not math.isfinite(float(scale))
        score.append(math.inf if forced else s)
    order = sorted(range(nb), key=lambda p: (-score[p], p))
    return sorted(order[:n_sel])
