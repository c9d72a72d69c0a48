"""Cases of the paged 16-bit KV cache: new tokens rotated and appended, attention of a chunk of new tokens over the
cache, the bounds of each block's keys, and decode attention over the blocks that a score from those bounds selects.

The cache is kc, vc [num_blocks][Hkv][16][128] in fp16 or bf16; token t of request r is row t % 16 of block
table[r][t / 16], and a token's slot is block * 16 + row.  The bounds are uint8 [num_blocks][Hkv][272]: bytes
8w .. 8w + 3 of a record hold the codes of the largest keys of channels 4w .. 4w + 3, the next four those of the
smallest, as signed bytes; the float at byte 256 is their scale.
"""
import math
import random

import torch

own = False

D = 128
BLOCK = 16
RECORD = 272
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # One decode step: the new token of each of 256 requests.
        {"name": "append_decode_b256", "op": "append", "N": 256, "Hq": 32, "Hkv": 8, "rot": 128, "axes": 1, "inter": False, "theta": 10000.0,
         "pos_hi": 4096, "fused": False, "dtype": "f16"},
        # An odd chunk of a prompt with pictures in it (time, height, width), taken out of a fused QKV projection.
        {"name": "append_chunk_5003", "op": "append", "N": 5003, "Hq": 40, "Hkv": 8, "rot": 128, "axes": 3, "inter": False, "theta": 1e6,
         "pos_hi": 65536, "fused": True, "dtype": "bf16"},
        # A whole 64K-token prompt; half the channels are rotated, neighbours in pairs.
        {"name": "append_prompt_64k", "op": "append", "N": 65536, "Hq": 32, "Hkv": 8, "rot": 64, "axes": 1, "inter": True, "theta": 5e5,
         "pos_hi": 1000000, "fused": False, "dtype": "f16"},
        # The smallest call: 16 new tokens of one request after 1008 cached ones.
        {"name": "chunk_b1_16_of_1k", "op": "chunk", "B": 1, "dec": 0, "n_lo": 16, "n_hi": 16, "base_lo": 1008, "base_hi": 1008, "Hq": 32, "Hkv": 8,
         "dtype": "f16"},
        # A whole prompt of 2000 tokens, nothing cached before it.
        {"name": "chunk_b1_prompt_2000", "op": "chunk", "B": 1, "dec": 0, "n_lo": 2000, "n_hi": 2000, "base_lo": 0, "base_hi": 0, "Hq": 40, "Hkv": 8,
         "dtype": "bf16"},
        # A mixed step: 48 requests decode a token each, 16 others bring chunks of their prompts; 5 query heads on a KV head.
        {"name": "chunk_mixed_b64", "op": "chunk", "B": 64, "dec": 48, "n_lo": 100, "n_hi": 512, "base_lo": 0, "base_hi": 16384, "Hq": 40, "Hkv": 8,
         "dtype": "bf16"},
        # One token of one request over 128K cached ones.
        {"name": "chunk_b1_1_of_128k", "op": "chunk", "B": 1, "dec": 1, "n_lo": 1, "n_hi": 1, "base_lo": 131071, "base_hi": 131071, "Hq": 32, "Hkv": 8,
         "dtype": "f16"},
        # A large chunk of a long prompt.
        {"name": "chunk_b1_4096_of_64k", "op": "chunk", "B": 1, "dec": 0, "n_lo": 4096, "n_hi": 4096, "base_lo": 61440, "base_hi": 61440, "Hq": 32,
         "Hkv": 8, "dtype": "f16"},
        # The bounds of the blocks that one decode step of 256 requests wrote to.
        {"name": "bounds_decode_b256", "op": "bounds", "B": 256, "n_lo": 1, "n_hi": 1, "Hkv": 8, "dtype": "f16"},
        # Those of a 64K-token prompt.
        {"name": "bounds_prompt_64k", "op": "bounds", "B": 1, "n_lo": 65531, "n_hi": 65531, "Hkv": 8, "dtype": "bf16"},
        # One request of 128K tokens: 256 of its 8192 blocks are selected for each KV head and attended to.
        {"name": "sparse_b1_128k", "op": "sparse", "B": 1, "Hq": 32, "Hkv": 8, "lo": 131072, "hi": 131072, "n_sel": 256, "first": 1, "last": 2,
         "dtype": "f16"},
        # A batch of long contexts, an eighth of whose blocks is selected; 5 query heads on a KV head.
        {"name": "sparse_b16_64k", "op": "sparse", "B": 16, "Hq": 40, "Hkv": 8, "lo": 50001, "hi": 65536, "n_sel": 512, "first": 4, "last": 8,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "bounds", "sparse"])
    dtype = rng.choice(["f16", "bf16"])
    Hkv, G = rng.choice([1, 2, 4, 8, 32]), rng.randint(1, 8)
    if op == "append":
        axes = rng.choice([1, 1, 3])
        return {"op": op, "N": _log(rng, 1, min(65536, 2000000 // (Hkv * (G + 2)))), "Hq": G * Hkv, "Hkv": Hkv, "rot": rng.choice([32, 64, 96, 128]),
                "axes": axes, "inter": rng.random() < 0.5, "theta": rng.choice([10000.0, 5e5, 1e6]), "pos_hi": _log(rng, 16, 1000000),
                "fused": rng.random() < 0.5, "dtype": dtype}
    if op == "bounds":
        B = _log(rng, 1, 256)
        n_hi = _log(rng, 1, max(1, 524288 // (B * Hkv)))
        return {"op": op, "B": B, "n_lo": max(1, n_hi // 2), "n_hi": n_hi, "Hkv": Hkv, "dtype": dtype}
    if op == "sparse":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131072, max(16, 8000000 // (B * Hkv))))
        first, last = rng.randint(0, 4), rng.randint(1, 8)
        n_sel = max(first + last, min(512, _log(rng, 1, max(2, hi // BLOCK))))
        return {"op": op, "B": B, "Hq": G * Hkv, "Hkv": Hkv, "lo": rng.choice([0, max(0, hi - 5), hi // 2]), "hi": hi, "n_sel": n_sel, "first": first,
                "last": last, "dtype": dtype}
    B = _log(rng, 1, 64)
    n_hi = _log(rng, 1, 4096)
    # As many cached tokens as keep the pass and its cache within the largest listed case.
    base_hi = max(1, min(131072, 16000000 // (B * Hkv), 240000000 // (B * n_hi * G * Hkv // 16 + 1) - n_hi))
    base_hi = _log(rng, 1, base_hi)
    while B > 1 and B * n_hi * (base_hi + n_hi) * G * Hkv > 8e9:
        B //= 2
    while n_hi > 1 and n_hi * (base_hi + n_hi) * G * Hkv > 8e9:
        n_hi //= 2
    return {"op": op, "B": B, "dec": rng.choice([0, 0, B // 2, B]), "n_lo": rng.choice([0, n_hi // 2, n_hi]), "n_hi": n_hi,
            "base_lo": rng.choice([0, base_hi // 2, base_hi]), "base_hi": base_hi, "Hq": G * Hkv, "Hkv": Hkv, "dtype": dtype}


# ---------------------------------------------------------------- inputs

def _cache(num_blocks, Hkv, dt, g):
    """A filled cache; keys have channels of their own offset."""
    kc, vc = (torch.empty(num_blocks, Hkv, BLOCK, D, dtype=dt, device="cuda").normal_(generator=g) for _ in range(2))
    kc += torch.randn(1, Hkv, 1, D, generator=g, device="cuda").to(dt)
    return kc, vc


def _table(ctx, g):
    """A table of scattered blocks, -1 behind a request's last; the number of blocks."""
    nb = (ctx + BLOCK - 1) // BLOCK
    mb = max(1, int(nb.max()))
    col = torch.arange(mb, device="cuda")[None]
    total = int(nb.sum()) + 3
    table = torch.full((ctx.numel(), mb), -1, dtype=torch.int32, device="cuda")
    table[col < nb[:, None]] = torch.randperm(total, generator=g, device="cuda")[:total - 3].to(torch.int32)
    return table, total


def _nan_behind(kc, vc, table, ctx):
    """What lies behind a request's last token is of other use: anything, NaN among it."""
    live = ctx > 0
    last = table[live, ((ctx[live].long() - 1) // BLOCK)].long()
    behind = torch.arange(BLOCK, device="cuda")[None] > (ctx[live, None] - 1) % BLOCK
    for x in (kc, vc):
        x[last] = torch.where(behind[:, None, :, None], torch.full_like(x[last], float("nan")), x[last])


def _lengths(c):
    """New tokens of each request: the same for every seed, so that the batch is."""
    rng = random.Random(c["B"] * 1000003 + c["n_hi"])
    return [1 if r < c.get("dec", 0) else rng.randint(c["n_lo"], c["n_hi"]) for r in range(c["B"])]


def _slots(n, g):
    """The slots of requests with n[r] tokens that follow one another from inside a block on; the number of blocks."""
    slots, used = [], 0
    for c in n:
        first = int(torch.randint(0, BLOCK, (1,), generator=g, device="cuda"))
        t = first + torch.arange(c, device="cuda")
        slots.append(used * BLOCK + t)
        used += (first + c + BLOCK - 1) // BLOCK
    slots = torch.cat(slots)
    num_blocks = sum(c // BLOCK + 2 for c in n)
    shuffled = torch.randperm(num_blocks, generator=g, device="cuda")
    slots = (shuffled[slots // BLOCK] * BLOCK + slots % BLOCK).to(torch.int32)
    return slots, num_blocks


def _per_127(x):
    """The quotient itself, where a division by a plain number would be a product with its reciprocal."""
    return x / torch.full_like(x, 127)


def _code_bounds(rows, there):
    """Codes of the largest and smallest [..., D] and scales [...] of keys [..., 16, D], of the rows that are there [..., 16]."""
    f = rows.float()
    hi = torch.where(there[..., None], f, -math.inf).amax(-2)
    lo = torch.where(there[..., None], f, math.inf).amin(-2)
    scale = _per_127(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    div = torch.where(scale > 0, scale, 1)[..., None]
    return (hi / div).ceil_().clamp_(-127, 127), (lo / div).floor_().clamp_(-127, 127), scale


def _records(hi, lo, scale):
    rec = torch.zeros(*scale.shape, RECORD, dtype=torch.uint8, device="cuda")
    both = torch.stack([hi.unflatten(-1, (32, 4)), lo.unflatten(-1, (32, 4))], -2).to(torch.int8)
    rec[..., :256] = both.flatten(-3).view(torch.uint8)
    rec[..., 256:260] = scale[..., None].contiguous().view(torch.uint8)
    return rec


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, Hkv = DTYPES[c["dtype"]], c["Hkv"]
    randint = lambda lo, hi, n: torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    if c["op"] == "append":
        N, Hq = c["N"], c["Hq"]
        s = {}
        s["slots"], num_blocks = _slots([N], g)
        s["slots"][N - N // 50:] = -1  # the padding of a batch of fixed size
        sizes = [Hq, Hkv, Hkv]
        if c["fused"]:
            qkv = torch.empty(N, sum(sizes), D, dtype=dt, device="cuda").normal_(generator=g)
            s["q"], s["k"], s["v"] = qkv.split(sizes, 1)
        else:
            s["q"], s["k"], s["v"] = (torch.empty(N, h, D, dtype=dt, device="cuda").normal_(generator=g) for h in sizes)
        n = c["rot"] // 2
        s["inv_freq"] = c["theta"] ** (-torch.arange(n, dtype=torch.float64) / n)
        # The slower pairs turn with the time, the others with height and width in turn.
        s["axis"] = torch.zeros(n, dtype=torch.int64) if c["axes"] == 1 else torch.where(torch.arange(n) < n // 4, 0, 1 + torch.arange(n) % 2)
        first = int(torch.randint(0, c["pos_hi"], (1,), generator=g, device="cuda"))
        s["pos"] = torch.stack([first + torch.arange(N, device="cuda") // (1 if a == 0 else 7) + randint(0, 9, N) for a in range(c["axes"])]).to(torch.int32)
        s["q_out"] = torch.empty(N, Hq, D, dtype=dt, device="cuda")
        s["kc"], s["vc"] = (torch.zeros(num_blocks, Hkv, BLOCK, D, dtype=dt, device="cuda") for _ in range(2))
    elif c["op"] == "bounds":
        s = {}
        s["slots"], num_blocks = _slots(_lengths(c), g)
        s["kc"], _ = _cache(num_blocks, Hkv, dt, g)
        s["bounds"] = torch.zeros(num_blocks, Hkv, RECORD, dtype=torch.uint8, device="cuda")
    elif c["op"] == "chunk":
        B = c["B"]
        n = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")[torch.randperm(B, generator=g, device="cuda")]
        ctx = n + randint(c["base_lo"], c["base_hi"], B)
        s = {"n": n.tolist(), "len": ctx.tolist(), "ctx": ctx}
        s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0).to(torch.int32)])
        s["table"], num_blocks = _table(ctx, g)
        s["kc"], s["vc"] = _cache(num_blocks, Hkv, dt, g)
        _nan_behind(s["kc"], s["vc"], s["table"], ctx)
        N = sum(s["n"]) + 2  # two rows of padding behind the last request's
        s["q"] = torch.empty(N, c["Hq"], D, dtype=dt, device="cuda").normal_(generator=g)
        s["out"] = torch.zeros(N, c["Hq"], D, dtype=dt, device="cuda")
        s["lse"] = torch.zeros(N, c["Hq"], device="cuda")
    else:
        B = c["B"]
        ctx = randint(c["lo"], c["hi"], B)
        s = {"ctx": ctx}
        s["table"], num_blocks = _table(ctx, g)
        s["kc"], s["vc"] = _cache(num_blocks, Hkv, dt, g)
        there = torch.ones(num_blocks, Hkv, BLOCK, dtype=torch.bool, device="cuda")
        live = ctx > 0
        last = s["table"][live, ((ctx[live].long() - 1) // BLOCK)].long()
        there[last] = (torch.arange(BLOCK, device="cuda")[None] <= (ctx[live, None] - 1) % BLOCK)[:, None]
        s["bounds"] = torch.cat([_records(*_code_bounds(k, t)) for k, t in zip(s["kc"].split(8192), there.split(8192))])
        _nan_behind(s["kc"], s["vc"], s["table"], ctx)
        s["q"] = torch.empty(B, c["Hq"], D, dtype=dt, device="cuda").normal_(generator=g)
        s["sel"] = torch.empty(B, Hkv, c["n_sel"], dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(B, c["Hq"], D, dtype=dt, device="cuda")
        s["lse"] = torch.empty(B, c["Hq"], device="cuda")
    s["case"] = c
    if own:
        _prepare_calls(s)
    return s


def _prepare_calls(s):
    """The calls of a serving loop on these buffers, checked once, as the package offers them."""
    import offloaded_kv_decode_gb300 as clo

    c = s["case"]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    if c["op"] == "append":
        pairs = clo.clo_rope_pairs(s["inv_freq"], s["axis"]).cuda()
        s["calls"] = [clo.prepare_paged_rope_append(s["q"], s["k"], s["v"], s["pos"], pairs, s["slots"], s["kc"], s["vc"], s["q_out"],
                                                    interleaved=c["inter"], err_flag=err)]
    elif c["op"] == "bounds":
        s["calls"] = [clo.prepare_paged_block_bounds(s["kc"], s["slots"], s["bounds"], err_flag=err)]
    elif c["op"] == "chunk":
        ws = work(clo.clo_paged_chunk_workspace_size(c["Hq"], c["Hkv"]))
        s["calls"] = [clo.prepare_paged_chunk_attn(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["offsets"], s["out"], ws, lse=s["lse"],
                                                   err_flag=err)]
    else:
        sws = work(clo.clo_paged_select_workspace_size(c["B"], c["Hkv"], s["table"].shape[1]))
        ws = work(clo.clo_paged_chunk_workspace_size(c["Hq"], c["Hkv"]))
        s["calls"] = [clo.prepare_paged_block_select(s["q"], s["bounds"], s["table"], s["ctx"], s["sel"], sws, n_first=c["first"], n_last=c["last"],
                                                     err_flag=err),
                      clo.prepare_paged_sparse_decode_attn(s["q"], s["kc"], s["vc"], s["table"], s["ctx"], s["sel"], s["out"], ws, lse=s["lse"],
                                                           err_flag=err)]


# ---------------------------------------------------------------- plain forms

def _plain_append(s):
    c = s["case"]
    n = c["rot"] // 2
    angle = s["pos"].double()[s["axis"].cuda()].t() * s["inv_freq"].cuda()  # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotated(x):
        f = x.float()
        a, b = (f[..., 0:2 * n:2], f[..., 1:2 * n:2]) if c["inter"] else (f[..., :n], f[..., n:2 * n])
        y = [a * cos - b * sin, a * sin + b * cos]
        y = torch.stack(y, -1).flatten(-2) if c["inter"] else torch.cat(y, -1)
        return torch.cat([y, f[..., 2 * n:]], -1).to(x.dtype)

    live = s["slots"] >= 0
    slots = s["slots"][live].long()
    s["q_out"].copy_(rotated(s["q"]))
    s["kc"][slots // BLOCK, :, slots % BLOCK] = rotated(s["k"])[live]
    s["vc"][slots // BLOCK, :, slots % BLOCK] = s["v"][live]


def _plain_bounds(s):
    slots = s["slots"].long()
    follows = torch.cat([slots[1:] == slots[:-1] + 1, slots.new_zeros(1, dtype=torch.bool)])
    last = slots[(slots % BLOCK == BLOCK - 1) | ~follows]  # the last new token in its block
    for at in last.split(8192):
        rows = s["kc"][at // BLOCK]
        there = (torch.arange(BLOCK, device="cuda")[None] <= at[:, None] % BLOCK)[:, None]
        s["bounds"][at // BLOCK] = _records(*_code_bounds(rows, there.expand(-1, rows.shape[1], -1)))


def _bounds_values(bounds):
    """fp32 [num_blocks][Hkv][32][largest, smallest][4]."""
    codes = bounds[..., :256].view(torch.int8).unflatten(-1, (32, 2, 4))
    return codes * bounds[..., 256:260].view(torch.float32)[..., None, None]


def _softmax_products(q, k, v, seen):
    """(softmax(q k^T) v, lse) in fp32 over the tokens that are seen; zeros and -inf for a row that sees none."""
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(D)).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1), (top + torch.log(total))[..., 0]


def _plain_chunk(s):
    c = s["case"]
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    at = 0
    for r, (n, length) in enumerate(zip(s["n"], s["len"])):
        if n == 0:
            continue
        blocks = s["table"][r, :-(-length // BLOCK)].long()
        k, v = (x[blocks].transpose(0, 1).flatten(1, 2)[:, :length].float() for x in (s["kc"], s["vc"]))
        step = max(1, (1 << 29) // (length * c["Hq"]))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            sees = length - n + 1 + torch.arange(lo, hi, device="cuda")
            t = int(length - n + hi)  # the tokens that some row of this part sees
            seen = (torch.arange(t, device="cuda")[None] < sees[:, None]).repeat_interleave(G, 0)
            q = s["q"][at + lo:at + hi].float().view(hi - lo, Hkv, G, D).transpose(0, 1).reshape(Hkv, -1, D)
            o, lse = _softmax_products(q, k[:, :t], v[:, :t], seen)
            s["out"][at + lo:at + hi] = o.view(Hkv, hi - lo, G, D).transpose(0, 1).reshape(hi - lo, c["Hq"], D).to(s["out"].dtype)
            s["lse"][at + lo:at + hi] = lse.view(Hkv, hi - lo, G).transpose(0, 1).reshape(hi - lo, c["Hq"])
        at += n


def _query_codes(q, Hkv):
    """Whole numbers -127 .. 127 [B][Hkv][D] for the sum of each group's queries, added up in the order of the heads."""
    q = q.float().unflatten(1, (Hkv, -1))
    total = q[:, :, 0].clone()
    for h in range(1, q.shape[2]):
        total += q[:, :, h]
    step = _per_127(total.abs().amax(-1, keepdim=True))
    return torch.where(step > 0, total / torch.where(step > 0, step, 1), 0).round_().clamp_(-127, 127)


def _plain_sparse(s):
    c = s["case"]
    B, Hkv, n_sel = c["B"], c["Hkv"], c["n_sel"]
    G = c["Hq"] // Hkv
    ctx = s["ctx"].long()
    nb = (ctx + BLOCK - 1) // BLOCK
    mb = s["table"].shape[1]
    col = torch.arange(mb, device="cuda")
    code = _query_codes(s["q"], Hkv)[..., None]
    rec = s["bounds"][s["table"].long()]  # [B][mb][Hkv][272]
    codes = rec[..., :256].view(torch.int8).unflatten(-1, (32, 2, 4)).float()
    hi, lo = (codes[..., i, :].flatten(-2).transpose(1, 2) for i in (0, 1))  # [B][Hkv][mb][D]
    # whole numbers below 2^24: exact in any order
    score = (torch.matmul(hi, code.clamp(min=0)) + torch.matmul(lo, code.clamp(max=0)))[..., 0]
    score = score * rec[..., 256:260].view(torch.float32)[..., 0].transpose(1, 2) + 0.0
    forced = (col < c["first"])[None] | (col >= nb[:, None] - c["last"])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((col < nb[:, None])[:, None], score, -math.inf)
    sel = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :n_sel]  # ties: the lower block first
    sel = torch.where(sel < nb[:, None, None], sel, mb).sort(-1).values
    if sel.shape[-1] < n_sel:
        sel = torch.cat([sel, sel.new_full((B, Hkv, n_sel - sel.shape[-1]), mb)], -1)
    s["sel"].copy_(torch.where(sel < mb, sel, -1))
    k_tok = (sel[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(2)  # [B][Hkv][n_sel * 16]
    seen = (k_tok < ctx[:, None, None]) & (sel < mb).repeat_interleave(BLOCK, -1)
    block = torch.gather(s["table"].long()[:, None].expand(B, Hkv, mb), 2, sel.clamp(max=mb - 1))
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    k, v = (torch.where(seen[..., None], x[block, head].flatten(2, 3).float(), 0) for x in (s["kc"], s["vc"]))
    o, lse = _softmax_products(s["q"].float().view(B, Hkv, G, D), k, v, seen[:, :, None])
    s["out"].copy_(o.view(B, c["Hq"], D))
    s["lse"].copy_(lse.view(B, c["Hq"]))


PLAIN = {"append": _plain_append, "bounds": _plain_bounds, "chunk": _plain_chunk, "sparse": _plain_sparse}


def run(s):
    op = s["case"]["op"]
    if own:
        for call in s["calls"]:
            call()
    else:
        PLAIN[op](s)
    if op == "bounds":
        return {"bounds": _bounds_values(s["bounds"])}
    return {n: s[n] for n in {"append": ("q_out", "kc", "vc"), "chunk": ("out", "lse"), "sparse": ("sel", "out", "lse")}[op]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    Hkv = c["Hkv"]
    if c["op"] == "append":  # queries in and out, K and V in and out
        return {"bytes": float(c["N"] * (4 * D * (c["Hq"] + 2 * Hkv) + 4 + 4 * c["axes"])), "flops": float(c["N"] * 3 * c["rot"] * (c["Hq"] + Hkv))}
    if c["op"] == "bounds":  # the keys of the new tokens' blocks in, their records out, and the values that these stand for
        tokens = sum(_lengths(c))
        blocks = tokens / BLOCK + c["B"] * (BLOCK - 1) / BLOCK
        return {"bytes": blocks * Hkv * (2 * D * BLOCK + 2 * RECORD + 8 * D) + 4 * tokens, "flops": 2.0 * blocks * Hkv * BLOCK * D}
    if c["op"] == "chunk":
        n, base = _lengths(c), (c["base_lo"] + c["base_hi"]) / 2
        tokens, rows = c["B"] * base + sum(n), sum(n)
        pairs = sum(x * base + x * (x + 1) / 2 for x in n)
        return {"bytes": tokens * Hkv * 4 * D + rows * c["Hq"] * (4 * D + 4) + tokens / 4 + 8 * c["B"], "flops": 4.0 * D * c["Hq"] * pairs}
    tokens = c["B"] * (c["lo"] + c["hi"]) / 2
    read = min(tokens, c["B"] * c["n_sel"] * BLOCK)
    return {"bytes": tokens / BLOCK * (Hkv * 260 + 4) + read * Hkv * 4 * D + c["B"] * (c["Hq"] * (4 * D + 4) + 4 * Hkv * c["n_sel"] + 4),
            "flops": 4.0 * D * tokens / BLOCK * Hkv + 4.0 * D * c["Hq"] * read}


# ---------------------------------------------------------------- in 64 bits

def _exact_attention(q, k, v):
    """q [Hq][D] against k, v [Hkv][T][D], all of them seen."""
    x = torch.einsum("hgd,htd->hgt", q.view(k.shape[0], -1, D), k) / math.sqrt(D)
    return torch.einsum("hgt,htd->hgd", torch.softmax(x, -1), v).reshape(-1, D), torch.logsumexp(x, -1).reshape(-1)


def _exact_append(s, c):
    n = c["rot"] // 2
    turn = torch.stack([s["pos"][a].double() for a in s["axis"].tolist()], 1) * s["inv_freq"].cuda()[None]
    unit = torch.polar(torch.ones_like(turn), turn)[:, None]
    res = {}
    for name in "qk":
        x = s[name].double()
        pair = x[..., :2 * n].unflatten(-1, (n, 2)) if c["inter"] else x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
        x = x.clone()
        x[..., :2 * n] = z.flatten(-2) if c["inter"] else z.transpose(-1, -2).flatten(-2)
        res[name] = x
    out = {"q_out": res["q"], "kc": s["kc"].double(), "vc": s["vc"].double()}
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows].long()
    for name, x in (("kc", res["k"]), ("vc", s["v"].double())):
        by_slot = out[name].transpose(1, 2).contiguous().view(-1, c["Hkv"], D)
        by_slot[at] = x[rows]
        out[name] = by_slot.view(-1, BLOCK, c["Hkv"], D).transpose(1, 2).contiguous()
    return out


def _exact_bounds(s, c):
    """A step is the largest magnitude's 127th part, rounded to fp32; the codes count steps, outward."""
    slots = s["slots"].long().tolist()
    block, rows = [], []
    for i, x in enumerate(slots):
        if x % BLOCK == BLOCK - 1 or i + 1 == len(slots) or slots[i + 1] != x + 1:
            block.append(x // BLOCK)
            rows.append(x % BLOCK + 1)
    value = torch.zeros(*s["bounds"].shape[:2], 32, 2, 4, dtype=torch.float64, device="cuda")
    block, rows = torch.tensor(block, device="cuda"), torch.tensor(rows, device="cuda")
    for count in range(1, BLOCK + 1):
        for at in block[rows == count].split(4096):
            k = s["kc"][at, :, :count].double()
            ends = torch.stack([k.amax(2), k.amin(2)], 2)  # [m][Hkv][2][D]
            step = (ends.abs().amax((2, 3)) / torch.full_like(ends[:, :, 0, 0], 127)).float().double()[..., None, None]
            # fp32 quotients: the codes are defined by them
            steps = torch.where(step > 0, ends / torch.where(step > 0, step, 1), 0).float().double()
            steps = torch.stack([steps[:, :, 0].ceil(), steps[:, :, 1].floor()], 2).clamp(-127, 127)
            value[at] = (steps * step).unflatten(-1, (32, 4)).transpose(2, 3)
    return {"bounds": value}


def _exact_chunk(s, c):
    out, lse = s["out"].double(), s["lse"].double()
    Hkv, G, at = c["Hkv"], c["Hq"] // c["Hkv"], 0
    for r, (n, length) in enumerate(zip(s["n"], s["len"])):
        if n == 0:
            continue
        ids = s["table"][r, :-(-length // BLOCK)].long()
        for h in range(Hkv):
            k, v = (x[ids, h].reshape(-1, D)[:length].double() for x in (s["kc"], s["vc"]))
            for g in range(G):
                head = h * G + g
                for lo in range(0, n, 1024):
                    q = s["q"][at + lo:at + min(n, lo + 1024), head].double()
                    x = q @ k.t() / math.sqrt(D)
                    last = length - n + lo + torch.arange(q.shape[0], device="cuda")
                    x.masked_fill_(torch.arange(length, device="cuda")[None] > last[:, None], -math.inf)
                    lse[at + lo:at + lo + q.shape[0], head] = torch.logsumexp(x, 1)
                    out[at + lo:at + lo + q.shape[0], head] = torch.softmax(x, 1) @ v
        at += n
    return {"out": out, "lse": lse}


def _exact_sparse(s, c):
    B, Hq, Hkv, n_sel = c["B"], c["Hq"], c["Hkv"], c["n_sel"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    G = Hq // Hkv
    for r, length in enumerate(s["ctx"].tolist()):
        nb = -(-length // BLOCK)
        ids = s["table"][r, :nb].long()
        for h in range(Hkv if nb else 0):
            cols = torch.arange(nb, device="cuda")
            if nb > n_sel:
                # fp32 sums in the order of the heads, then whole numbers: the selection is defined by them
                total = torch.zeros(D, device="cuda")
                for g in range(G):
                    total = total + s["q"][r, h * G + g].float()
                step = total.abs().max() / torch.full_like(total[0], 127)
                code = torch.zeros_like(total) if step == 0 else (total / step).round()
                rec = s["bounds"][ids, h]
                ends = rec[:, :256].contiguous().view(torch.int8).view(nb, 32, 2, 4).long()
                top, low = ends[:, :, 0].reshape(nb, D), ends[:, :, 1].reshape(nb, D)
                code = code.long().clamp(-127, 127)
                score = torch.maximum(top * code, low * code).sum(1).float() * rec[:, 256:260].contiguous().view(torch.float32)[:, 0]
                rank = sorted(range(nb), key=lambda i, x=score.tolist(): (not (i < c["first"] or i >= nb - c["last"]), -x[i], i))
                cols = torch.tensor(sorted(rank[:n_sel]), device="cuda")
            tok = (cols[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).view(-1)
            k, v = (x[ids[cols], h].reshape(-1, D)[tok < length].double() for x in (s["kc"], s["vc"]))
            o, e = _exact_attention(s["q"][r, h * G:(h + 1) * G].double(), k[None], v[None])
            out[r, h * G:(h + 1) * G], lse[r, h * G:(h + 1) * G] = o, e
    return {"sel": None, "out": out, "lse": lse}


def exact(case, seed):
    c = dict(case)
    if c["op"] == "chunk" and work(c)["flops"] > 8e12:
        return None
    s = prepare(c, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "chunk": _exact_chunk, "sparse": _exact_sparse}[c["op"]](s, c)
