"""Plain reference of the paged 4-bit KV cache, in numpy and 64 bits: the
record's layout, the quantiser, the read-back, the attention and the block
plan, each written from the definitions in include/clo_kv4.h (the plan as a
loop over the requests).  Test code only."""
import math

import numpy as np
import torch

D, BLOCK = 128, 16
U16 = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}       # half the smallest step, absolute


def record_bytes(group):
    return 2048 + 128 * (D // group)


# ---------------------------------------------------------------- layout

def _places():
    """(byte, shift) of channel d of token t, for K and V: arrays [16][128]."""
    kb = np.zeros((BLOCK, D), np.int64)
    vb = np.zeros((BLOCK, D), np.int64)
    sh = np.zeros((BLOCK, D), np.int64)
    for t in range(BLOCK):
        for d in range(D):
            w, i = d // 8, d % 8                      # word of eight channels, place in it
            j, c = w // 4, w % 4                      # channels 32j + 8c ..
            kb[t, d] = t * 64 + 4 * (4 * c + j) + i // 2
            vb[t, d] = 1024 + t * 64 + 16 * ((d // 32) ^ ((t >> 1) & 3)) + 4 * (w % 4) + i // 2
            sh[t, d] = 4 * (i % 2)
    return kb, vb, sh


KB, VB, SH = _places()


def unpack(rec, group):
    """Records [..., R] uint8 -> K codes, V codes [..., 16, 128] (int) and pairs
    [..., 16, 2, NG, 2] (fp64; scale, zero)."""
    rec = np.asarray(rec)
    k = (rec[..., KB] >> SH) & 15
    v = (rec[..., VB] >> SH) & 15
    with np.errstate(invalid="ignore"):  # what nothing has been written to may be a NaN
        par = np.ascontiguousarray(rec[..., 2048:]).view(np.float16).astype(np.float64)
    return k, v, par.reshape(*rec.shape[:-1], BLOCK, 2, D // group, 2)


def values(rec, group):
    """fp64 K and V [..., 16, 128]."""
    k, v, par = unpack(rec, group)
    p = np.repeat(par, group, axis=-2)
    return k * p[..., 0, :, 0] + p[..., 0, :, 1], v * p[..., 1, :, 0] + p[..., 1, :, 1]


# ---------------------------------------------------------------- quantiser

def half_down(x):
    h = np.asarray(x, np.float64).astype(np.float16)
    with np.errstate(over="ignore"):
        return np.where(h.astype(np.float64) > x, np.nextafter(h, np.float16(-np.inf)), h)


def half_up(x):
    h = np.asarray(x, np.float64).astype(np.float16)
    with np.errstate(over="ignore"):
        return np.where(h.astype(np.float64) < x, np.nextafter(h, np.float16(np.inf)), h)


def quantise(x, group):
    """Rows [..., 128] (fp64) -> codes (int), scale, zero (fp16 [..., NG]), and
    how far each quotient is from the border between two codes."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], D // group, group)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], np.clip(np.nan_to_num(g, nan=0.0, posinf=0.0, neginf=0.0), -65504, 65504), 0.0)
    zero = half_down(g.min(-1))
    scale = half_up((g.max(-1) - zero.astype(np.float64)) / 15)
    s = scale.astype(np.float64)[..., None]
    quot = np.where(s > 0, (g - zero.astype(np.float64)[..., None]) / np.where(s > 0, s, 1), 0.0)
    border = np.abs(quot - np.floor(quot) - 0.5)
    nan = np.float16(np.nan)
    return (np.rint(quot).astype(np.int64).reshape(x.shape), np.where(finite, scale, nan),
            np.where(finite, zero, nan), border.reshape(x.shape))


def write_rows(pool, slots, k, v, group):
    """What an append of rows k, v [N][Hkv][128] (fp64) does to pool
    [num_blocks][Hkv][R] (numpy, in place); slots out of range are skipped."""
    ck, sk, zk, _ = quantise(k, group)
    cv, sv, zv, _ = quantise(v, group)
    ng = D // group
    for n, slot in enumerate(np.asarray(slots).tolist()):
        if slot < 0 or slot // BLOCK >= pool.shape[0]:
            continue
        b, t = slot // BLOCK, slot % BLOCK
        for h in range(pool.shape[1]):
            rec = pool[b, h]
            for codes, places in ((ck, KB), (cv, VB)):
                for half in (0, 1):
                    at, c = places[t, half::2], codes[n, h, half::2]
                    rec[at] = (rec[at] & (0xF0 if half == 0 else 0x0F)) | (c << (4 * half))
            par = np.stack([np.stack([sk[n, h], zk[n, h]], -1), np.stack([sv[n, h], zv[n, h]], -1)]).astype(np.float16)
            rec[2048 + t * 8 * ng:2048 + (t + 1) * 8 * ng] = par.reshape(-1).view(np.uint8)


# ---------------------------------------------------------------- attention

def attention(q, rec, table, ctx, group, scale, dtype):
    """fp64 out [B][n_q][Hq][128] and lse [B][n_q][Hq], and how far a kernel
    may be from them, element by element.

    The tolerance follows the arithmetic such a kernel needs: scores in fp32
    (the codes' and the zeros' shares summed apart, up to 20 roundings of
    2^-24 on the sum of magnitudes, and 2^-22 for the exponential), weights
    p * scale_v rounded once to fp16 (2^-11, and half the smallest step where
    they are below 2^-14 of the largest), fp32 sums, and one rounding of the
    output to its type."""
    B, n_q, Hq, _ = q.shape
    Hkv = rec.shape[1]
    G = Hq // Hkv
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    tol = np.zeros(q.shape)
    ltol = np.zeros(q.shape[:3])
    for r in range(B):
        n = int(ctx[r])
        if n == 0:
            continue
        blocks = table[r, :-(-n // BLOCK)]
        ck, cv, par = unpack(rec[blocks], group)
        par = np.repeat(par, group, axis=-2)  # [nb][Hkv][16][2][128][2]
        flat = lambda x: x.transpose(1, 0, *range(2, x.ndim)).reshape(Hkv, -1, *x.shape[3:])[:, :n]  # noqa: E731
        ck, cv, par = flat(ck), flat(cv), flat(par)
        with np.errstate(invalid="ignore"):
            K = ck * par[:, :, 0, :, 0] + par[:, :, 0, :, 1]
            Kmag = ck * par[:, :, 0, :, 0] + np.abs(par[:, :, 0, :, 1])
            sv, zv = par[:, :, 1, :, 0], par[:, :, 1, :, 1]
            for i in range(n_q):
                m = n - (n_q - 1 - i)
                if m <= 0:
                    continue
                for h in range(Hkv):
                    qq = q[r, i, h * G:(h + 1) * G]
                    x = qq @ K[h, :m].T * scale
                    dx = (20 * 2.0 ** -24) * (np.abs(qq) @ Kmag[h, :m].T * scale).max(-1) + 2.0 ** -22
                    top = x.max(-1, keepdims=True)
                    e = np.exp(x - top)
                    total = e.sum(-1, keepdims=True)
                    p = e / total
                    V = cv[h, :m] * sv[h, :m] + zv[h, :m]
                    o = p @ V
                    mag = p @ (cv[h, :m] * sv[h, :m] + np.abs(zv[h, :m]))
                    floor = m * 2.0 ** -25 * 15 * (p[:, :, None] * sv[h, None, :m]).max((1, 2), keepdims=False)[:, None]
                    rows = (r, i, slice(h * G, (h + 1) * G))
                    out[rows] = o
                    lse[rows] = (top + np.log(total))[:, 0]
                    ltol[rows] = dx + 2.0 ** -22 * (1 + np.abs(lse[rows]))
                    inner = (2.0 ** -11 + 2 * dx[:, None]) * mag + floor
                    tol[rows] = inner + U16[dtype] * (np.abs(o) + inner) + TINY[dtype]
    return out, lse, tol, ltol


# ---------------------------------------------------------------- block plan

BAD_INDEX, BAD_CTX, NO_ROOM = 0x1, 0x4, 0x10


def plan(length, keep, add, table, ring, state, max_new):
    """The plan of clo_paged_plan, one request after the other."""
    table, ring = table.copy(), ring.copy()
    B, mb = table.shape
    nb = lambda x: -(-x // BLOCK)  # noqa: E731
    head, count = (int(x) for x in state)
    size = len(ring)
    err = 0
    ok = 0 <= head < size and 0 <= count <= size
    if not ok:
        err |= BAD_INDEX
        head0, count0, head, count = head, count, 0, 0
    free = [int(ring[(head + j) % size]) for j in range(count)]
    back = []
    len_out, start, offsets = np.array(length), np.full(B, -1), np.zeros(B + 1, np.int64)
    slots = np.full(max_new, -1)
    tokens = blocks = 0
    for r in range(B):
        n, k, a = int(length[r]), int(keep[r]), int(add[r])
        good = 0 <= k <= n <= mb * BLOCK and a >= 0 and k + a <= mb * BLOCK
        if not good:
            err |= BAD_CTX
            a = 0
        first = tokens
        tokens += a
        offsets[r + 1] = tokens
        if not good:
            continue
        need = max(nb(k + a) - nb(n), 0)
        blocks += need
        if a > 0 and (tokens > max_new or blocks > count):
            err |= NO_ROOM
            continue
        for c in range(nb(n), nb(k + a)):
            table[r, c] = free.pop(0)
        back += [int(table[r, c]) for c in range(nb(k + a), nb(n))]
        len_out[r], start[r] = k + a, k
        for j in range(a):
            b = int(table[r, (k + j) // BLOCK])
            if 0 <= b < 1 << 27:
                slots[first + j] = b * BLOCK + (k + j) % BLOCK
            else:
                err |= BAD_INDEX
    room = size - count if ok else 0
    if len(back) > room:
        err |= BAD_INDEX
        back = back[:room]
    for j, b in enumerate(back):
        ring[(head + count + j) % size] = b
    taken = count - len(free)
    out = [(head + taken) % size, count - taken + len(back)] if ok else [head0, count0]
    return dict(len_out=len_out, start=start, offsets=offsets, slot_map=slots, block_table=table, free_ring=ring,
                ring_out=np.array(out)), err


def scale_for(d=D):
    return 1.0 / math.sqrt(d)
