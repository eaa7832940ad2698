"""The 8-bit paged cache's operators: cases, plain forms, 64-bit values.

Each case names one operator (``op``) and its sizes:

``append``   new tokens' queries rotated, their keys rotated and stored with their values in a paged cache
             held in 8 bits (``kv8_append_paged``), and what the blocks so touched then hold, read
             back (``kv8_read_paged``)
``read``     cached tokens of an 8-bit cache expanded to bf16 (``kv8_read_paged``)
``decode``   one query per sequence over an 8-bit cache (``attn_decode_paged_kv8``)
``prefill``  the last N tokens of each sequence as queries over an 8-bit cache that holds them already:
             prompt chunks, draft tokens (``attn_prefill_paged_kv8``)

An 8-bit cache is [num_blocks, Hkv, record] bytes.  A record holds 16 token slots of one KV head: K codes
(16 rows of d bytes), V codes (the same), then 32 bytes: the scale of K and of V (fp32), a word of flags and
zeros.  A code is an e4m3 number and stands for itself times the scale, a power of two: the smallest under
which no value of the block's tokens is above 448.
"""

import math

import torch

own = False

BLOCK = 16
TAIL = 32
DEV = "cuda"
MOST = 448.0             # the largest e4m3 number
LEAST_EXP = -64          # exponents of a scale
MOST_EXP = 64


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of 64 sequences: one new token each, long contexts among them.
        dict(name="append_decode_step", op="append", S=64, lo=1, hi=1, ctx=32768, pad=0, Hq=12, Hkv=2, d=128,
             rot=128, axes=1, interleaved=False),
        # A prefill batch of ragged chunks, partial rotation, a padded batch.
        dict(name="append_ragged_chunks", op="append", S=7, lo=100, hi=2300, ctx=4096, pad=37, Hq=12, Hkv=2, d=128,
             rot=64, axes=1, interleaved=False),
        # Long prompts of image patches and text: three position axes.
        dict(name="append_three_axes", op="append", S=5, lo=500, hi=5001, ctx=1000, pad=0, Hq=16, Hkv=4, d=128,
             rot=128, axes=3, interleaved=False),
        # A cached prefix brought back to bf16.
        dict(name="read_prefix", op="read", S=3, lo=2000, hi=9000, Hkv=4, d=128),
        # Short prefixes of many sequences.
        dict(name="read_short_d64", op="read", S=33, lo=0, hi=99, Hkv=2, d=64),
        # The smallest decode: one sequence with a short context.
        dict(name="decode_one_short", op="decode", S=1, lo=100, hi=100, Hq=12, Hkv=2, d=128),
        # The paged-decode batch of this repository: 64 sequences of 128 .. 4096 tokens.
        dict(name="decode_batch", op="decode", S=64, lo=128, hi=4096, Hq=12, Hkv=2, d=128),
        # A few long contexts.
        dict(name="decode_long", op="decode", S=8, lo=30000, hi=131072, Hq=16, Hkv=2, d=128),
        # Many short ragged sequences of small heads, empty ones among them; 16 query heads a KV head.
        dict(name="decode_many_d64", op="decode", S=256, lo=0, hi=2048, Hq=64, Hkv=4, d=64),
        # Chunks of 2048 tokens on top of up to 6144 cached ones.
        dict(name="prefill_chunks", op="prefill", S=4, N=2048, lo=2048, hi=8192, Hq=12, Hkv=2, d=128),
        # Four draft tokens of each of 32 sequences, to be verified in one pass.
        dict(name="prefill_draft_tokens", op="prefill", S=32, N=4, lo=500, hi=6000, Hq=12, Hkv=2, d=128),
        # Short chunks of small heads, of sequences shorter than the chunk (left-padded) among them.
        dict(name="prefill_padded_d64", op="prefill", S=24, N=100, lo=0, hi=700, Hq=16, Hkv=4, d=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, most):
    Hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 5, 6, 8, 12, 16])
    while Hkv * g > most:
        g = max(1, g // 2)
    return Hkv * g, Hkv


def draw(rng):
    op = rng.choice(["append", "append", "read", "decode", "decode", "prefill", "prefill"])
    d = rng.choice([64, 128])
    Hq, Hkv = _heads(rng, 32)
    if op == "append":
        axes = rng.choice([1, 1, 2, 3])
        S = _log(rng, 1, 128)
        most = max(1, min(16000, (16384 * 16 * 128) // ((Hq + 2 * Hkv) * d)) // S)
        hi = _log(rng, 1, most)
        return dict(op=op, S=S, lo=max(1, hi // rng.choice([1, 2, 9])), hi=hi, ctx=_log(rng, 1, 8192),
                    pad=rng.choice([0, 0, 3, 64]), Hq=Hq, Hkv=Hkv, d=d,
                    rot=d if axes > 1 else rng.choice([d, d, d // 2, 16]), axes=axes,
                    interleaved=rng.random() < 0.4)
    if op == "read":
        S = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(16000, (16000 * 4 * 128) // (Hkv * d)) // S))
        return dict(op=op, S=S, lo=rng.choice([0, hi // 3, hi]), hi=hi, Hkv=Hkv, d=d)
    if op == "decode":
        S = _log(rng, 1, 256)
        most = (8 * 70000 * 2 * 128) // (Hkv * d)
        hi = max(1, min(100000, _log(rng, 1, max(2, most // S))))
        return dict(op=op, S=S, lo=rng.choice([0, hi // 10, hi]), hi=hi, Hq=Hq, Hkv=Hkv, d=d)
    S = _log(rng, 1, 64)
    N = _log(rng, 1, 2048)
    most = min((4 * 12 * 2048 * 4096 * 128) // (S * Hq * N * d), (2048 * 4096 * 128) // (S * Hkv * d))
    hi = max(1, min(32000, _log(rng, 1, max(2, most))))
    return dict(op=op, S=S, N=N, lo=rng.choice([0, hi // 10, hi]), hi=hi, Hq=Hq, Hkv=Hkv, d=d)


def _spread(S, lo, hi):
    """S lengths spread evenly over lo .. hi (the case fixes them; a seed only orders them)."""
    return [lo + int((hi - lo + 1) * ((b * 0.6180339887498949 + 0.5) % 1.0)) for b in range(S)] if hi > lo else [hi] * S


# -------------------------------------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7 + 5)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).float().to(DEV)


def _pair_axis(rot, axes):
    """Contiguous sections of the pairs (time, height, width); None for one axis."""
    if axes == 1:
        return None
    n = rot // 2
    first = n // 4 if axes == 3 else n // 2
    rest = (n - first) // max(1, axes - 1)
    return [min(axes - 1, 0 if p < first else 1 + (p - first) // max(1, rest)) for p in range(n)]


def _table(lens, g):
    """A pool of exactly the blocks that `lens` need, in random order; table rows padded with -1."""
    nb = torch.tensor([-(-n // BLOCK) for n in lens], dtype=torch.int64, device=DEV)
    most = max(1, int(max(-(-n // BLOCK) for n in lens)))
    used = sum(-(-n // BLOCK) for n in lens)
    perm = torch.randperm(max(1, used), generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(most, device=DEV)[None] < nb[:, None]] = perm[:used]
    return table, max(1, used)


def _random_kv8(blocks, Hkv, d, g):
    """Records of normalised activations: codes around the middle of their range, block scales of 2^-8 .. 2^-5."""
    rec = torch.zeros(blocks, Hkv, 2 * BLOCK * d + TAIL, dtype=torch.uint8, device=DEV)
    e = torch.randint(-8, -4, (blocks, Hkv, 2, 1), generator=g, device=DEV)
    x = torch.empty(blocks, Hkv, 2, BLOCK * d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    x *= torch.exp2(-e.float()).to(torch.bfloat16)
    rec[..., : 2 * BLOCK * d] = x.clamp_(-MOST, MOST).to(torch.float8_e4m3fn).view(torch.uint8).flatten(2)
    rec[..., 2 * BLOCK * d: 2 * BLOCK * d + 8] = torch.exp2(e[..., 0].float()).contiguous().view(torch.uint8)
    return rec


def _order(lens, seed):
    p = torch.randperm(len(lens), generator=torch.Generator().manual_seed(int(seed))).tolist()
    return [lens[i] for i in p]


def _ints(rows):
    return torch.cat(rows).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    op, d, S = case["op"], case["d"], case["S"]
    s = dict(case)
    if op == "append":
        Hq, Hkv, A = case["Hq"], case["Hkv"], case["axes"]
        both = zip(_spread(S, 0, case["ctx"]), _spread(S, case["lo"], case["hi"])[::-1])
        ctx, new = zip(*_order(list(both), seed))
        s["table"], blocks = _table([c + n for c, n in zip(ctx, new)], g)
        T, pad = sum(new), case["pad"]
        s["tokens"] = T
        s["seq_ids"] = _ints([torch.full((n,), b) for b, n in enumerate(new)] + [torch.full((pad,), -1)])
        s["positions"] = _ints([torch.arange(c, c + n) for c, n in zip(ctx, new)] + [torch.zeros(pad)])
        # The tokens of every block that the batch reaches, those that were there among them.
        first = [c - c % BLOCK for c in ctx]
        s["read_ids"] = _ints([torch.full((c + n - f,), b) for b, (c, n, f) in enumerate(zip(ctx, new, first))])
        s["read_pos"] = _ints([torch.arange(f, c + n) for c, n, f in zip(ctx, new, first)])
        s["inv_freq"], s["pair_axis"] = _inv_freq(case["rot"]), _pair_axis(case["rot"], A)
        p = s["positions"]
        s["rope_positions"] = torch.stack([p // 1024, (p // 32) % 32, p % 32][:A]).to(torch.int32) if A > 1 else None
        rows = T + pad
        x = _randn(g, rows, (Hq + 2 * Hkv) * d)
        x *= torch.exp(0.25 * _randn(g, (Hq + 2 * Hkv) * d))
        x = x.to(torch.bfloat16)
        s["q"] = x[:, : Hq * d].view(rows, Hq, d)
        s["k"] = x[:, Hq * d: (Hq + Hkv) * d].view(rows, Hkv, d)
        s["v"] = x[:, (Hq + Hkv) * d:].view(rows, Hkv, d)
        s["q_out"] = torch.zeros(rows, Hq, d, dtype=torch.bfloat16, device=DEV)
        s["kv_cache"] = _random_kv8(blocks, Hkv, d, g)
        return s
    lens = _order(_spread(S, case["lo"], case["hi"]), seed)
    s["table"], blocks = _table(lens, g)
    s["kv_cache"] = _random_kv8(blocks, case["Hkv"], d, g)
    if op == "read":
        s["seq_ids"] = _ints([torch.full((n,), b) for b, n in enumerate(lens)])
        s["positions"] = _ints([torch.arange(n) for n in lens])
        return s
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape = (S, case["Hq"], d) if op == "decode" else (S, case["Hq"], case["N"], d)
    s["q"] = _randn(g, *shape).to(torch.bfloat16)
    # Scratch that a serving loop keeps between steps (a fixed size, whatever the batch).
    s["workspace"] = torch.empty(16 << 20, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ run
def run(s):
    return {"append": _run_append, "read": _run_read, "decode": _run_decode, "prefill": _run_prefill}[s["op"]](s)


def _run_append(s):
    if own:
        import exact_attention_47_gb300 as attn
        attn.kv8_append_paged(s["q"], s["k"], s["v"], s["kv_cache"], s["table"], s["seq_ids"], s["positions"],
                                   inv_freq=s["inv_freq"], rope_positions=s["rope_positions"],
                                   pair_axis=s["pair_axis"], interleaved=s["interleaved"], q_out=s["q_out"])
        k, v = attn.kv8_read_paged(s["kv_cache"], s["table"], s["read_ids"], s["read_pos"], s["d"])
        return {"q": s["q_out"], "k": k, "v": v}
    T, d = s["tokens"], s["d"]
    at = s["positions"][:T] if s["rope_positions"] is None else s["rope_positions"][:, :T]
    c, sn = _cos_sin(at, s["inv_freq"], s["pair_axis"])
    c, sn = c[:, None], sn[:, None]
    s["q_out"][:T] = _rotate(s["q"][:T].float(), c, sn, s["interleaved"]).to(torch.bfloat16)
    kv = torch.stack([_rotate(s["k"][:T].float(), c, sn, s["interleaved"]), s["v"][:T].float()], 2)  # [T, Hkv, 2, d]
    phys, slot = _slots(s["table"], s["seq_ids"][:T], s["positions"][:T])
    blocks, which = torch.unique(phys, return_inverse=True)
    # The scales of the blocks touched: what their new tokens need, or what they had where some tokens stay.
    codes, scales = _parts(s["kv_cache"], d)
    most = torch.zeros(len(blocks), *kv.shape[1:3], device=DEV)
    most.index_reduce_(0, which, kv.abs().amax(-1), "amax")
    new = torch.zeros(len(blocks), dtype=torch.bool, device=DEV)
    new[which[slot == 0]] = True
    had = torch.where(new[:, None, None], 0.0, scales[blocks])
    now = torch.maximum(had, _scale_for(most))
    old = codes[blocks].view(torch.float8_e4m3fn).float() * (had / now)[..., None, None]
    old = torch.where(new[:, None, None, None, None], 0.0, old)
    old[which, :, :, slot] = kv / now[which][..., None]
    codes[blocks] = old.clamp(-MOST, MOST).to(torch.float8_e4m3fn).view(torch.uint8)
    scales[blocks] = now
    k, v = _rows(s["kv_cache"], s["table"], s["read_ids"], s["read_pos"], d)
    return {"q": s["q_out"], "k": k, "v": v}


def _run_read(s):
    if own:
        import exact_attention_47_gb300 as attn
        k, v = attn.kv8_read_paged(s["kv_cache"], s["table"], s["seq_ids"], s["positions"], s["d"])
        return {"k": k, "v": v}
    k, v = _rows(s["kv_cache"], s["table"], s["seq_ids"], s["positions"], s["d"])
    return {"k": k, "v": v}


def _run_decode(s):
    if own:
        import exact_attention_47_gb300 as attn
        o, lse = attn.attn_decode_paged_kv8(s["q"], s["kv_cache"], s["table"], s["seq_lens"], workspace=s["workspace"])
        return {"o": o, "lse": lse}
    o, lse = _attend(s, s["q"][:, :, None])
    return {"o": o[:, :, 0], "lse": lse[:, :, 0]}


def _run_prefill(s):
    if own:
        import exact_attention_47_gb300 as attn
        o, lse = attn.attn_prefill_paged_kv8(s["q"], s["kv_cache"], s["table"], s["seq_lens"],
                                             workspace=s["workspace"])
        return {"o": o, "lse": lse}
    o, lse = _attend(s, s["q"])
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------------------- plain pieces
def _cos_sin(positions, inv_freq, pair_axis):
    """[tokens, pairs]: the angles in 64 bits (far positions lose them in 32)."""
    if pair_axis is None:
        a = positions[..., None].double() * inv_freq.double()
    else:
        a = positions[pair_axis].movedim(0, -1).double() * inv_freq.double()
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, c, s, interleaved):
    rot = 2 * c.shape[-1]
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)
    a, b = head[..., : rot // 2], head[..., rot // 2:]
    return torch.cat([a * c - b * s, b * c + a * s, rest], -1)


def _slots(table, seq_ids, positions):
    pos = positions.long()
    return table[seq_ids.long(), pos // BLOCK].long(), pos % BLOCK


def _scale_for(most):
    """The smallest power of two under which `most` is at most 448 = 1.75 2^8."""
    m, e = torch.frexp(most)             # most = m 2^e, m in [1/2, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(LEAST_EXP, MOST_EXP)
    return torch.exp2(torch.where(most > 0, e, LEAST_EXP).float())


def _parts(rec, d):
    """Views of records: codes [..., 2, 16, d] uint8 and scales [..., 2] fp32."""
    n = 2 * BLOCK * d
    return rec[..., :n].unflatten(-1, (2, BLOCK, d)), rec.view(torch.float32)[..., n // 4: n // 4 + 2]


def _rows(cache, table, seq_ids, positions, d):
    phys, slot = _slots(table, seq_ids, positions)
    codes, scales = _parts(cache, d)
    x = codes[phys, :, :, slot].view(torch.float8_e4m3fn).float() * scales[phys][..., None]
    return x[:, :, 0].to(torch.bfloat16), x[:, :, 1].to(torch.bfloat16)


def _attend(s, q):
    """q [S, Hq, N, d], its rows the last N tokens of each sequence."""
    S, Hq, N, d = q.shape
    Hkv = s["Hkv"]
    codes, scales = _parts(s["kv_cache"][s["table"].clamp(min=0).long()], d)     # [S, nb, Hkv, 2, 16, d]
    L = codes.shape[1] * BLOCK
    kv = codes.contiguous().view(torch.float8_e4m3fn).float() * scales[..., None, None]
    k, v = (kv[:, :, :, i].transpose(1, 2).reshape(S, Hkv, L, d) for i in (0, 1))
    x = q.float().reshape(S, Hkv, (Hq // Hkv) * N, d) @ k.transpose(-1, -2) * d ** -0.5
    last = s["seq_lens"].long()[:, None] - N + torch.arange(N, device=DEV)       # the last key that a row sees
    hidden = torch.arange(L, device=DEV) > last[..., None]                       # [S, N, L]
    x = x.view(S, Hq, N, L).masked_fill_(hidden[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-3e38))
    n = p.sum(-1, keepdim=True)
    live = torch.arange(L, device=DEV) < s["seq_lens"][:, None]                  # what lies behind the end is not read
    v = torch.where(live[:, None, :, None], v, 0.0)
    o = (p.view(S, Hkv, -1, L) @ v).view(S, Hq, N, d) / torch.where(n > 0, n, 1.0)
    return o.to(torch.bfloat16), (m + torch.log(n))[..., 0]


# ----------------------------------------------------------------------------------------------- work
def work(case):
    """Inputs once, outputs once; operations of the products (a rotation: six a pair)."""
    op, d, Hkv = case["op"], case["d"], case["Hkv"]
    if op == "append":
        new = _spread(case["S"], case["lo"], case["hi"])[::-1]
        ctx = _spread(case["S"], 0, case["ctx"])
        T, R = sum(new), sum(c % BLOCK + n for c, n in zip(ctx, new))
        read = T * ((case["Hq"] + 2 * Hkv) * d * 2 + 8)
        wrote = T * (case["Hq"] * d * 2 + 2 * Hkv * d)
        return {"bytes": read + wrote + R * (Hkv * 6 * d + 8),
                "flops": T * (case["Hq"] + Hkv) * case["rot"] * 3 + T * Hkv * d * 4}
    lens = _spread(case["S"], case["lo"], case["hi"])
    if op == "read":
        return {"bytes": max(1, sum(lens) * (Hkv * 6 * d + 8)), "flops": sum(lens) * Hkv * d * 2}
    cache = sum(lens) * 2 * d + 8 * sum(-(-n // BLOCK) for n in lens)
    N = case.get("N", 1)
    pairs = sum(max(0, n - N + i + 1) for n in lens for i in range(N))
    return {"bytes": Hkv * cache + case["S"] * case["Hq"] * N * (d * 4 + 4), "flops": pairs * case["Hq"] * d * 4}


# ---------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs in 64 bits, from the definitions, sequence by sequence."""
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "append":
        return _append64(s)
    if op == "read":
        lens = torch.bincount(s["seq_ids"], minlength=s["S"]).tolist()
        both = [_cached64(s, b, n) for b, n in enumerate(lens) if n]
        return {"k": torch.cat([x[0] for x in both]), "v": torch.cat([x[1] for x in both])} if both else None
    q = s["q"].double() if op == "prefill" else s["q"].double()[:, :, None]
    S, Hq, N = q.shape[:3]
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((S, Hq, N), -math.inf, dtype=torch.float64, device=DEV)
    group = Hq // s["Hkv"]
    for b, n in enumerate(s["seq_lens"].tolist()):
        first = max(0, N - n)                        # rows before it belong to no token
        if first == N:
            continue
        k, v = _cached64(s, b, n)
        see = torch.arange(n, device=DEV)[None] <= torch.arange(n - N + first, n, device=DEV)[:, None]
        for h in range(Hq):
            x = q[b, h, first:] @ k[:, h // group].T / math.sqrt(d)
            x = torch.where(see, x, torch.tensor(-math.inf, dtype=torch.float64, device=DEV))
            lse[b, h, first:] = torch.logsumexp(x, -1)
            o[b, h, first:] = torch.softmax(x, -1) @ v[:, h // group]
    return {"o": o, "lse": lse} if op == "prefill" else {"o": o[:, :, 0], "lse": lse[:, :, 0]}


def _decode64(code):
    """e4m3 codes: sign, 4 bits of exponent (bias 7), 3 of fraction; exponent 0 has no leading one."""
    c = code.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
    return torch.where(c >= 128, -v, v)


def _cached64(s, b, n):
    """Keys and values [n, Hkv, d] of the first n tokens of sequence b."""
    d, Hkv = s["d"], s["Hkv"]
    rec = s["kv_cache"][s["table"][b, : -(-n // BLOCK)].long()]
    size = BLOCK * d
    at = rec[..., 2 * size: 2 * size + 8].contiguous().view(torch.float32).double()
    return tuple((_decode64(rec[..., i * size: (i + 1) * size]).view(-1, Hkv, BLOCK, d) * at[..., i, None, None])
                 .transpose(1, 2).reshape(-1, Hkv, d)[:n] for i in (0, 1))


def _nearest64(x, step):
    """The multiple of the power of two `step` [...] by an e4m3 number that is nearest to x, the even one of two."""
    y = (x / step).clamp(-MOST, MOST)
    unit = torch.exp2((torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))) - 3)
    return torch.round(y / unit) * unit * step


def _turn64(x, pos, s):
    """x [n, H, d] rotated by pos [axes, n], one pair at a time."""
    y = x.clone()
    half = s["rot"] // 2
    f = s["inv_freq"].double()
    for i in range(half):
        p = pos[s["pair_axis"][i] if s["pair_axis"] is not None else 0].double()[:, None]
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.polar(torch.ones_like(p), p * f[i]) * torch.complex(x[..., a], x[..., b])
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _append64(s):
    T, Hkv, d = s["tokens"], s["Hkv"], s["d"]
    pos = (s["positions"][None] if s["rope_positions"] is None else s["rope_positions"])[:, :T]
    q = s["q_out"].double()
    q[:T] = _turn64(s["q"][:T].double(), pos, s)
    new = torch.stack([_turn64(s["k"][:T].double(), pos, s), s["v"][:T].double()])          # [2, T, Hkv, d]
    at, out, t = s["positions"][:T].tolist(), [], 0
    for b, n in enumerate(torch.bincount(s["seq_ids"][:T], minlength=s["S"]).tolist()):
        ctx = at[t]
        keep = ctx % BLOCK
        # All rows from the first block touched on, in whole blocks; those behind the end are zeros.
        rows = -(-(keep + n) // BLOCK) * BLOCK
        x = torch.zeros(2, rows, Hkv, d, dtype=torch.float64, device=DEV)
        step = torch.full((2, rows // BLOCK, Hkv), 2.0 ** LEAST_EXP, dtype=torch.float64, device=DEV)
        if keep:
            x[0, :keep], x[1, :keep] = (y[ctx - keep:] for y in _cached64(s, b, ctx))
            rec = s["kv_cache"][int(s["table"][b, ctx // BLOCK])]
            step[:, 0] = rec[:, 2 * BLOCK * d: 2 * BLOCK * d + 8].contiguous().view(torch.float32).double().T
        x[:, keep: keep + n] = new[:, t: t + n]
        fresh = x.clone()
        fresh[:, :keep] = 0                          # the tokens that stay have fixed the old scale
        most = fresh.abs().view(2, -1, BLOCK, Hkv, d).amax((2, 4))
        need = torch.exp2(torch.ceil(torch.log2(most.clamp(min=1e-300) / MOST)).clamp(LEAST_EXP, MOST_EXP))
        step = torch.maximum(step, need)
        out.append(_nearest64(x, step.repeat_interleave(BLOCK, 1)[..., None])[:, : keep + n])
        t += n
    out = torch.cat(out, 1)
    return {"q": q, "k": out[0], "v": out[1]}
