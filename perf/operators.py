"""The rotary-position, paged-append and 4-bit-cache operators: cases, plain forms, 64-bit values.

Each case names one operator (``op``) and its sizes:

``rope``         rotation of queries and keys by positions with one to three axes, on its way from the
                 projection's token-major layout to the attention's head-major one (``rope_fwd``), or of
                 their gradients on the way back (``rope_bwd``)
``append``       new tokens' queries rotated, their keys rotated and stored with their values in a paged
                 bf16 cache (``rope_append_paged``)
``append_kv4``   the same into a cache held in 4 bits (``rope_append_paged_kv4``), and the stored rows read
                 back, as a chunk that attends to what the cache holds does (``kv4_read_paged``)
``read_kv4``     cached tokens of a 4-bit cache expanded to bf16 (``kv4_read_paged``)
``decode_kv4``   one query per sequence over a 4-bit cache (``attn_decode_paged_kv4``)

A 4-bit cache is [num_blocks, Hkv, record] bytes.  A record holds 16 token slots of one KV head:
K codes (16 rows of d/2 bytes), V codes (the same), K parameters (16 rows of d/group pairs of bf16),
V parameters.  A value is code * scale + min with its group's (min, scale).  Element e of a K row is
nibble i + 4 h of word (d/32) c + w of the row, e = 32 w + 8 i + 2 c + h; of a V row, nibble p of word
(d/64) r + w, e = r + 8 (8 w + p).
"""

import math

import torch

own = False

BLOCK = 16
DEV = "cuda"


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # The Qwen-style layer's prefill: queries and keys of the merged projection of 4 x 4096 tokens.
        dict(name="rope_qwen_prefill_fwd", op="rope", dir="fwd", B=4, N=4096, Hq=12, Hkv=2, d=128, rot=128,
             axes=1, interleaved=False, merged=True, far=0),
        # Gradients of a sequence of image patches: three axes, adjacent pairs, an odd length.
        dict(name="rope_three_axes_bwd", op="rope", dir="bwd", B=1, N=5001, Hq=16, Hkv=16, d=64, rot=64,
             axes=3, interleaved=True, merged=False, far=0),
        # One decode step of 64 sequences: one new token each, far positions among them.
        dict(name="append_decode_step", op="append", S=64, lo=1, hi=1, ctx=32768, pad=0, Hq=12, Hkv=2, d=128,
             rot=128, axes=1, interleaved=False),
        # A prefill batch of ragged chunks, partial rotation, a padded batch.
        dict(name="append_prefill", op="append", S=7, lo=100, hi=2300, ctx=4096, pad=37, Hq=12, Hkv=2, d=128,
             rot=64, axes=1, interleaved=False),
        # A decode step into the 4-bit cache.
        dict(name="append_kv4_decode_step", op="append_kv4", S=48, lo=1, hi=1, ctx=8192, pad=16, Hq=12, Hkv=2,
             d=128, group=32, rot=128, axes=1, interleaved=False),
        # A long prefill into the 4-bit cache, three axes.
        dict(name="append_kv4_prefill", op="append_kv4", S=5, lo=500, hi=5001, ctx=1000, pad=0, Hq=16, Hkv=4,
             d=128, group=64, rot=128, axes=3, interleaved=False),
        # A cached prefix brought back to bf16 for a chunk that attends to it.
        dict(name="read_kv4_prefix", op="read_kv4", S=3, lo=2000, hi=9000, Hkv=4, d=128, group=32),
        # Short prefixes of many sequences.
        dict(name="read_kv4_short", op="read_kv4", S=33, lo=0, hi=99, Hkv=2, d=64, group=32),
        # The smallest decode: one sequence with a short context.
        dict(name="decode_kv4_one_short", op="decode_kv4", S=1, lo=100, hi=100, Hq=12, Hkv=2, d=128, group=32),
        # The paged-decode batch of this repository: 64 sequences of 128 .. 4096 tokens.
        dict(name="decode_kv4_batch", op="decode_kv4", S=64, lo=128, hi=4096, Hq=12, Hkv=2, d=128, group=32),
        # A few long contexts.
        dict(name="decode_kv4_long", op="decode_kv4", S=8, lo=30000, hi=131072, Hq=16, Hkv=2, d=128, group=64),
        # Many short ragged sequences of small heads, empty ones among them; 16 query heads a KV head.
        dict(name="decode_kv4_many_d64", op="decode_kv4", S=256, lo=0, hi=2048, Hq=64, Hkv=4, d=64, group=32),
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
    op = rng.choice(["rope", "append", "append_kv4", "read_kv4", "decode_kv4", "decode_kv4"])
    d = rng.choice([64, 128])
    Hq, Hkv = _heads(rng, 32)
    axes = rng.choice([1, 1, 2, 3])
    rot = d if axes > 1 else rng.choice([d, d, d // 2, 16])
    pairs = rng.random() < 0.4
    if op == "rope":
        tokens = min(_log(rng, 1, 16000), (16384 * 14 * 128) // ((Hq + Hkv) * d))
        B = rng.choice([1, 2, 3]) if tokens > 3 else 1
        return dict(op="rope", dir=rng.choice(["fwd", "bwd"]), B=B, N=max(1, tokens // B), Hq=Hq, Hkv=Hkv, d=d,
                    rot=rot, axes=axes, interleaved=pairs, merged=rng.random() < 0.5,
                    far=rng.choice([0, 0, 1 << 20]))
    if op in ("append", "append_kv4"):
        S = _log(rng, 1, 128)
        most = max(1, min(16000, (16384 * 16 * 128) // ((Hq + 2 * Hkv) * d)) // S)
        hi = _log(rng, 1, most)
        c = dict(op=op, S=S, lo=max(1, hi // rng.choice([1, 2, 9])), hi=hi, ctx=_log(rng, 1, 8192),
                 pad=rng.choice([0, 0, 3, 64]), Hq=Hq, Hkv=Hkv, d=d, rot=rot, axes=axes, interleaved=pairs)
        return c if op == "append" else dict(c, group=rng.choice([32, 64]))
    group = rng.choice([32, 64])
    if op == "read_kv4":
        S = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(16000, (16000 * 4 * 128) // (Hkv * d)) // S))
        return dict(op=op, S=S, lo=rng.choice([0, hi // 3, hi]), hi=hi, Hkv=Hkv, d=d, group=group)
    S = _log(rng, 1, 256)
    most = (8 * 70000 * 2 * 128) // (Hkv * d)
    hi = max(1, min(100000, _log(rng, 1, max(2, most // S))))
    return dict(op=op, S=S, lo=rng.choice([0, hi // 10, hi]), hi=hi, Hq=Hq, Hkv=Hkv, d=d, group=group)


def _spread(S, lo, hi):
    """S lengths spread evenly over lo .. hi (the case fixes them; a seed only orders them)."""
    return [lo + int((hi - lo + 1) * ((b * 0.6180339887498949 + 0.5) % 1.0)) for b in range(S)] if hi > lo else [hi] * S


# -------------------------------------------------------------------------------------------- prepare
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7 + 3)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).float().to(DEV)


def _pair_axis(rot, axes):
    """Three axes: contiguous sections (time, height, width); None for one axis."""
    if axes == 1:
        return None
    n = rot // 2
    first = n // 4 if axes == 3 else n // 2
    rest = (n - first) // max(1, axes - 1)
    return [min(axes - 1, 0 if p < first else 1 + (p - first) // max(1, rest)) for p in range(n)]


def _record(d, group):
    return 2 * BLOCK * (d // 2) + 2 * BLOCK * (d // group) * 4


def _table(lens, g):
    """A pool of exactly the blocks that `lens` need, in random order; table rows padded with -1."""
    nb = torch.tensor([-(-n // BLOCK) for n in lens], dtype=torch.int64, device=DEV)
    most = max(1, int(max(-(-n // BLOCK) for n in lens)))
    total = max(1, sum(-(-n // BLOCK) for n in lens))
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(most, device=DEV)[None]
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device=DEV)
    used = col < nb[:, None]
    table[used] = perm[: int(sum(-(-n // BLOCK) for n in lens))]
    return table, total


def _random_kv4(blocks, Hkv, d, group, g):
    """Records whose codes and parameters look like those of normalised activations."""
    rec = torch.randint(0, 256, (blocks, Hkv, _record(d, group)), generator=g, dtype=torch.uint8, device=DEV)
    n = 2 * BLOCK * (d // group)
    scale = (0.3 * torch.exp(0.4 * _randn(g, blocks, Hkv, n))).to(torch.bfloat16)
    low = (-7.5 * scale.float() * (1 + 0.15 * _randn(g, blocks, Hkv, n))).to(torch.bfloat16)
    rec[..., 2 * BLOCK * (d // 2):] = torch.stack([low, scale], -1).reshape(blocks, Hkv, 2 * n).view(torch.uint8)
    return rec


def _order(lens, seed):
    p = torch.randperm(len(lens), generator=torch.Generator().manual_seed(int(seed))).tolist()
    return [lens[i] for i in p]


def prepare(case, seed):
    g = _gen(seed)
    op, d = case["op"], case["d"]
    s = dict(case)
    if op == "rope":
        B, N, Hq, Hkv, A = case["B"], case["N"], case["Hq"], case["Hkv"], case["axes"]
        s["inv_freq"], s["pair_axis"] = _inv_freq(case["rot"]), _pair_axis(case["rot"], A)
        if A == 1:
            start = torch.randint(0, 1000, (B, 1), generator=g, device=DEV) + case["far"]
            s["positions"] = (start + torch.arange(N, device=DEV)).to(torch.int32)
        else:  # a grid of patches: a frame number, a row and a column
            t = torch.arange(N, device=DEV) + case["far"]
            w = 1 + int(torch.randint(20, 60, (1,), generator=g, device=DEV))
            ax = [t // (w * w), (t // w) % w + case["far"], t % w + case["far"]][:A]
            s["positions"] = torch.stack(ax).to(torch.int32)[:, None].expand(A, B, N).contiguous()
        if case["dir"] == "fwd" and case["merged"]:
            x = _randn(g, B, N, (Hq + 2 * Hkv) * d).to(torch.bfloat16)
            s["q"] = x[..., : Hq * d].view(B, N, Hq, d).transpose(1, 2)
            s["k"] = x[..., Hq * d: (Hq + Hkv) * d].view(B, N, Hkv, d).transpose(1, 2)
        else:
            s["q"] = _randn(g, B, Hq, N, d).to(torch.bfloat16)
            s["k"] = _randn(g, B, Hkv, N, d).to(torch.bfloat16)
            if case["dir"] == "fwd":
                s["q"] = s["q"].transpose(1, 2).contiguous().transpose(1, 2)
                s["k"] = s["k"].transpose(1, 2).contiguous().transpose(1, 2)
        return s
    if op in ("append", "append_kv4"):
        S, Hq, Hkv, A = case["S"], case["Hq"], case["Hkv"], case["axes"]
        both = zip(_spread(S, 0, case["ctx"]), _spread(S, case["lo"], case["hi"])[::-1])
        ctx, new = zip(*_order(list(both), seed))
        s["table"], blocks = _table([c + n for c, n in zip(ctx, new)], g)
        T = sum(new)
        ids = torch.repeat_interleave(torch.arange(S), torch.tensor(new))
        pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
        rows = T + case["pad"]
        s["seq_ids"] = torch.cat([ids, torch.full((case["pad"],), -1)]).to(torch.int32).to(DEV)
        s["positions"] = torch.cat([pos, torch.zeros(case["pad"], dtype=torch.int64)]).to(torch.int32).to(DEV)
        s["tokens"] = T
        s["inv_freq"], s["pair_axis"] = _inv_freq(case["rot"]), _pair_axis(case["rot"], A)
        s["rope_positions"] = None
        if A > 1:
            p = s["positions"]
            s["rope_positions"] = torch.stack([p // 1024, (p // 32) % 32, p % 32][:A]).to(torch.int32)
        x = _randn(g, rows, (Hq + 2 * Hkv) * d)
        x *= torch.exp(0.25 * _randn(g, (Hq + 2 * Hkv) * d))
        x = x.to(torch.bfloat16)
        s["q"] = x[:, : Hq * d].view(rows, Hq, d)
        s["k"] = x[:, Hq * d: (Hq + Hkv) * d].view(rows, Hkv, d)
        s["v"] = x[:, (Hq + Hkv) * d:].view(rows, Hkv, d)
        s["q_out"] = torch.zeros(rows, Hq, d, dtype=torch.bfloat16, device=DEV)
        if op == "append":
            s["k_cache"] = _randn(g, blocks, Hkv, BLOCK, d).to(torch.bfloat16)
            s["v_cache"] = _randn(g, blocks, Hkv, BLOCK, d).to(torch.bfloat16)
        else:
            s["kv_cache"] = _random_kv4(blocks, Hkv, d, case["group"], g)
        return s
    S = case["S"]
    lens = _order(_spread(S, case["lo"], case["hi"]), seed)
    s["table"], blocks = _table(lens, g)
    s["kv_cache"] = _random_kv4(blocks, case["Hkv"], d, case["group"], g)
    if op == "read_kv4":
        s["seq_ids"] = torch.repeat_interleave(torch.arange(S), torch.tensor(lens)).to(torch.int32).to(DEV)
        s["positions"] = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(DEV)
        return s
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["q"] = _randn(g, S, case["Hq"], d).to(torch.bfloat16)
    # Scratch that a serving loop keeps between steps (a fixed size, whatever the batch).
    s["workspace"] = torch.empty(8 << 20, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ run
def run(s):
    return {"rope": _run_rope, "append": _run_append, "append_kv4": _run_append_kv4, "read_kv4": _run_read,
            "decode_kv4": _run_decode}[s["op"]](s)


def _run_rope(s):
    back = s["dir"] == "bwd"
    if own:
        import exact_attention_47_gb300 as attn
        f = attn.rope_bwd if back else attn.rope_fwd
        q, k = f(s["q"], s["k"], s["positions"], s["inv_freq"], pair_axis=s["pair_axis"],
                 interleaved=s["interleaved"])
        return {"q": q, "k": k}
    c, sn = _cos_sin(s["positions"], s["inv_freq"], s["pair_axis"])
    c, sn = c[:, None], (-sn if back else sn)[:, None]
    return {"q": _rotate(s["q"].float(), c, sn, s["interleaved"]).to(torch.bfloat16).contiguous(),
            "k": _rotate(s["k"].float(), c, sn, s["interleaved"]).to(torch.bfloat16).contiguous()}


def _run_append(s):
    if own:
        import exact_attention_47_gb300 as attn
        attn.rope_append_paged(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["seq_ids"],
                               s["positions"], inv_freq=s["inv_freq"], rope_positions=s["rope_positions"],
                               pair_axis=s["pair_axis"], interleaved=s["interleaved"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    q, k, v = _rotated_rows(s)
    phys, slot = _slots(s)
    s["q_out"][: s["tokens"]] = q.to(torch.bfloat16)
    s["k_cache"][phys, :, slot] = k.to(torch.bfloat16)
    s["v_cache"][phys, :, slot] = v.to(torch.bfloat16)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_append_kv4(s):
    T = s["tokens"]
    if own:
        import exact_attention_47_gb300 as attn
        attn.rope_append_paged_kv4(s["q"], s["k"], s["v"], s["kv_cache"], s["table"], s["seq_ids"], s["positions"],
                                   s["group"], inv_freq=s["inv_freq"], rope_positions=s["rope_positions"],
                                   pair_axis=s["pair_axis"], interleaved=s["interleaved"], q_out=s["q_out"])
        k, v = attn.kv4_read_paged(s["kv_cache"], s["table"], s["seq_ids"][:T], s["positions"][:T], s["d"],
                                   s["group"])
        return {"q": s["q_out"], "k": k, "v": v}
    q, k, v = _rotated_rows(s)
    s["q_out"][:T] = q.to(torch.bfloat16)
    d, group = s["d"], s["group"]
    phys, slot = _slots(s)
    kc, kp = _quantise(k, group)
    vc, vp = _quantise(v, group)
    codes, params = _parts(s["kv_cache"], d, group)
    codes[phys, :, 0, slot] = _pack_k(kc)
    codes[phys, :, 1, slot] = _pack_v(vc)
    params[phys, :, 0, slot] = kp
    params[phys, :, 1, slot] = vp
    k, v = _rows_kv4(s, phys, slot)
    return {"q": s["q_out"], "k": k, "v": v}


def _run_read(s):
    if own:
        import exact_attention_47_gb300 as attn
        k, v = attn.kv4_read_paged(s["kv_cache"], s["table"], s["seq_ids"], s["positions"], s["d"], s["group"])
        return {"k": k, "v": v}
    k, v = _rows_kv4(s, *_slots(dict(s, tokens=s["seq_ids"].numel())))
    return {"k": k, "v": v}


def _run_decode(s):
    if own:
        import exact_attention_47_gb300 as attn
        o, lse = attn.attn_decode_paged_kv4(s["q"], s["kv_cache"], s["table"], s["seq_lens"], s["group"],
                                            workspace=s["workspace"])
        return {"o": o, "lse": lse}
    S, Hq, Hkv, d, group = s["S"], s["Hq"], s["Hkv"], s["d"], s["group"]
    codes, params = _parts(s["kv_cache"][s["table"].clamp(min=0).long()], d, group)  # [S, nb, Hkv, 2, 16, ...]
    L = codes.shape[1] * BLOCK
    k = _values(_unpack_k(codes[:, :, :, 0]), params[:, :, :, 0], group).transpose(1, 2).reshape(S, Hkv, L, d)
    v = _values(_unpack_v(codes[:, :, :, 1]), params[:, :, :, 1], group).transpose(1, 2).reshape(S, Hkv, L, d)
    x = s["q"].float().view(S, Hkv, Hq // Hkv, d) @ k.transpose(-1, -2) * d ** -0.5
    x.masked_fill_(torch.arange(L, device=DEV) >= s["seq_lens"][:, None, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-3e38))
    n = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(n > 0, n, 1.0)
    lse = m + torch.log(n)
    return {"o": o.view(S, Hq, d).to(torch.bfloat16), "lse": lse.view(S, Hq)}


# ---------------------------------------------------------------------------------------- plain pieces
def _cos_sin(positions, inv_freq, pair_axis):
    """[..., tokens, pairs]: the angles in 64 bits (far positions lose them in 32)."""
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


def _rotated_rows(s):
    """The batch's token rows (without its padding) in 32 bits: rotated queries and keys, values."""
    T = s["tokens"]
    at = s["positions"][:T] if s["rope_positions"] is None else s["rope_positions"][:, :T]
    c, sn = _cos_sin(at, s["inv_freq"], s["pair_axis"])
    c, sn = c[:, None], sn[:, None]
    return (_rotate(s["q"][:T].float(), c, sn, s["interleaved"]), _rotate(s["k"][:T].float(), c, sn, s["interleaved"]),
            s["v"][:T].float())


def _slots(s):
    T = s["tokens"]
    pos = s["positions"][:T].long()
    return s["table"][s["seq_ids"][:T].long(), pos // BLOCK].long(), pos % BLOCK


def _quantise(x, group):
    """[..., d] fp32 -> codes [..., d] uint8 and (min, scale) [..., d/group, 2] bf16."""
    y = x.unflatten(-1, (-1, group))
    low = y.amin(-1, keepdim=True).to(torch.bfloat16).float()
    top = y.amax(-1, keepdim=True)
    scale = ((top - low) / 15.0).clamp(min=0.0).to(torch.bfloat16).float()
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    codes = torch.where(scale > 0, torch.round((y - low) / scale), 0.0).clamp(0, 15).to(torch.uint8)
    return codes.flatten(-2), torch.cat([low, scale], -1).to(torch.bfloat16)


def _parts(rec, d, group):
    """Views of records: codes [..., 2, 16, d/2] uint8 and parameters [..., 2, 16, d/group, 2] bf16."""
    n = 2 * BLOCK * (d // 2)
    return (rec[..., :n].unflatten(-1, (2, BLOCK, d // 2)),
            rec[..., n:].view(torch.bfloat16).unflatten(-1, (2, BLOCK, d // group, 2)))


def _nibbles_to_bytes(n):
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _bytes_to_nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _pack_k(c):  # (w, i, c, h) -> (c, w, h, i)
    return _nibbles_to_bytes(c.unflatten(-1, (-1, 4, 4, 2)).movedim((-2, -4, -1, -3), (-4, -3, -2, -1)).flatten(-4))


def _unpack_k(b):  # (c, w, h, i) -> (w, i, c, h)
    n = _bytes_to_nibbles(b)
    return n.unflatten(-1, (4, -1, 2, 4)).movedim((-3, -1, -4, -2), (-4, -3, -2, -1)).flatten(-4)


def _pack_v(c):  # (w, p, r) -> (r, w, p)
    return _nibbles_to_bytes(c.unflatten(-1, (-1, 8, 8)).movedim(-1, -3).flatten(-3))


def _unpack_v(b):  # (r, w, p) -> (w, p, r)
    return _bytes_to_nibbles(b).unflatten(-1, (8, -1, 8)).movedim(-3, -1).flatten(-3)


def _values(codes, params, group):
    p = params.float()
    return (codes.unflatten(-1, (-1, group)).float() * p[..., 1:] + p[..., :1]).flatten(-2)


def _rows_kv4(s, phys, slot):
    d, group = s["d"], s["group"]
    codes, params = _parts(s["kv_cache"], d, group)
    k = _values(_unpack_k(codes[phys, :, 0, slot]), params[phys, :, 0, slot], group)
    v = _values(_unpack_v(codes[phys, :, 1, slot]), params[phys, :, 1, slot], group)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


# ----------------------------------------------------------------------------------------------- work
def work(case):
    """Inputs once, outputs once; operations of the products (a rotation: six a pair)."""
    op, d = case["op"], case["d"]
    if op == "rope":
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hkv"])
        return {"bytes": rows * d * 4 + case["B"] * case["N"] * 4 * case["axes"], "flops": rows * case["rot"] * 3}
    if op in ("append", "append_kv4"):
        T = sum(_spread(case["S"], case["lo"], case["hi"]))
        Hq, Hkv = case["Hq"], case["Hkv"]
        read = T * (Hq + 2 * Hkv) * d * 2 + T * 8
        flops = T * (Hq + Hkv) * case["rot"] * 3
        if op == "append":
            return {"bytes": read + T * (Hq + 2 * Hkv) * d * 2, "flops": flops}
        row4 = d + 8 * (d // case["group"])  # both codes and both parameters of a token and head
        return {"bytes": read + T * Hq * d * 2 + 2 * T * Hkv * row4 + T * Hkv * d * 4,
                "flops": flops + T * Hkv * d * 10}
    if op == "read_kv4":
        T = sum(_spread(case["S"], case["lo"], case["hi"]))
        row4 = d + 8 * (d // case["group"])
        return {"bytes": max(1, T * (case["Hkv"] * (row4 + d * 4) + 8)), "flops": T * case["Hkv"] * d * 4}
    lens = _spread(case["S"], case["lo"], case["hi"])
    row4 = d + 8 * (d // case["group"])
    return {"bytes": sum(lens) * case["Hkv"] * row4 + case["S"] * case["Hq"] * (d * 4 + 4),
            "flops": sum(lens) * case["Hq"] * d * 4}


# ---------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The outputs in 64 bits, from the definitions, token by token and pair by pair."""
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    if op == "rope":
        B, N = case["B"], case["N"]
        pos = s["positions"].view(case["axes"], B, N)
        sign = -1.0 if case["dir"] == "bwd" else 1.0
        return {n: torch.stack([_turn64(s[n][b].double(), pos[:, b], s, sign) for b in range(B)]) for n in ("q", "k")}
    if op == "decode_kv4":
        return _decode64(s)
    if op == "read_kv4":
        k, v = _read64(s, s["seq_ids"], s["positions"])
        return {"k": k, "v": v}
    T = s["tokens"]
    pos = (s["positions"][None] if s["rope_positions"] is None else s["rope_positions"])[:, :T]
    q = s["q_out"].double()
    q[:T] = _turn64(s["q"][:T].double().transpose(0, 1), pos, s, 1.0).transpose(0, 1)
    k = _turn64(s["k"][:T].double().transpose(0, 1), pos, s, 1.0).transpose(0, 1)
    v = s["v"][:T].double()
    if op == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        row = s["table"].long().gather(0, s["seq_ids"][:T].long()[:, None].expand(-1, s["table"].shape[1]))
        block = row.gather(1, (s["positions"][:T].long() // BLOCK)[:, None])[:, 0]
        at = block * BLOCK + s["positions"][:T].long() % BLOCK
        for c, x in ((kc, k), (vc, v)):
            flat = c.transpose(1, 2).reshape(-1, case["Hkv"], d)
            flat[at] = x
            c.copy_(flat.view(-1, BLOCK, case["Hkv"], d).transpose(1, 2))
        return {"q": q, "k_cache": kc, "v_cache": vc}
    return {"q": q, "k": _nearest64(k, case["group"]), "v": _nearest64(v, case["group"])}


def _turn64(x, pos, s, sign):
    """x [H, n, d] rotated by pos [axes, n], one pair at a time."""
    y = x.clone()
    half = s["rot"] // 2
    f = s["inv_freq"].double()
    for i in range(half):
        p = pos[s["pair_axis"][i] if s["pair_axis"] is not None else 0].double()
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.polar(torch.ones_like(p), sign * p * f[i]) * torch.complex(x[..., a], x[..., b])
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _nearest64(x, group):
    """What a 4-bit row of x stands for: the nearest of the 16 levels of each group, the even one of two."""
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], group):
        y = x[..., a: a + group]
        low = y.min(-1, keepdim=True).values.to(torch.bfloat16).double()
        step = ((y.max(-1, keepdim=True).values - low) / 15.0).clamp(min=0).to(torch.bfloat16).double()
        n = torch.where(step > 0, torch.round((y - low) / step.clamp(min=1e-300)), 0.0)
        out[..., a: a + group] = low + step * n.clamp(0, 15)
    return out


def _places(d, kind):
    """Byte and shift of each element in a row of K or V codes."""
    e = torch.arange(d, device=DEV)
    if kind == 0:
        w, i, c, h = e // 32, e // 8 % 4, e // 2 % 4, e % 2
        n = ((d // 32) * c + w) * 8 + i + 4 * h
    else:
        n = ((d // 64) * (e % 8) + e // 64) * 8 + e // 8 % 8
    return n // 2, 4 * (n % 2)


def _expand64(rec, slot, kind, d, group):
    """Values of rows `slot` [n] of records rec [n, Hkv, bytes]: [n, Hkv, d]."""
    byte, shift = _places(d, kind)
    n, H = rec.shape[:2]
    base = (kind * BLOCK + slot)[:, None, None] * (d // 2)
    code = (rec.gather(-1, (base + byte).expand(n, H, d)).int() >> shift) & 15
    par = rec[..., BLOCK * d:].contiguous().view(torch.bfloat16).double().view(n, H, 2, BLOCK, d // group, 2)
    par = par[torch.arange(n, device=DEV), :, kind, slot].repeat_interleave(group, 2)
    return code.double() * par[..., 1] + par[..., 0]


def _read64(s, ids, positions):
    rec = s["kv_cache"][s["table"][ids.long(), positions.long() // BLOCK].long()]
    return tuple(_expand64(rec, positions.long() % BLOCK, kind, s["d"], s["group"]) for kind in (0, 1))


def _decode64(s):
    S, Hq, Hkv, d = s["S"], s["Hq"], s["Hkv"], s["d"]
    o = torch.zeros(S, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((S, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n:
            pos = torch.arange(n, device=DEV)
            k, v = _read64(s, torch.full_like(pos, b), pos)
            x = torch.einsum("gqd,ngd->gqn", s["q"][b].double().view(Hkv, Hq // Hkv, d), k) / math.sqrt(d)
            lse[b] = torch.logsumexp(x, -1).view(-1)
            o[b] = torch.einsum("gqn,ngd->gqd", torch.softmax(x, -1), v).reshape(Hq, d)
    return {"o": o, "lse": lse}
