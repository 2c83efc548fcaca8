"""The attention side of a decode step, measured: norms of queries and keys
with the position rotation, the append to a paged int8 cache, attention over
that cache, and cached tokens read back.

With ``own`` false every operator runs in its plain form (elementary torch
operations in 32 bits, angles in 64); with ``own`` true the framework's calls
run on the same tensors.

The cache, as include/tern.h defines it: a block holds 64 tokens of one
sequence; codes int8 [blocks][kv heads][2][64*D] (K, then V) and one fp32
scale for each block, head and side, scales [blocks][kv heads][2].  Inside a
block the codes lie in the order in which the matrix cores read them:
  K: token 16t + r, dim 64s + 16g + b  at  [t][s][g][r][b]
  V: token 16t + 4g + i, dim 16u + r   at  [u][g][r][t][i]
A step's sequences: tokens cu[i] .. cu[i+1] belong to sequence i, whose length
with them is lens[i]; table[i] lists its blocks.
"""
import math
import random

import torch

own = False

BLOCK = 64
EPS = 1e-6


# ---- cases ----------------------------------------------------------------

def spread(text):
    """Whole numbers of a text: "5,7" -> 5, 7; "10..1000x3" -> 10, 100, 1000 (evenly over the logarithm)."""
    out = []
    for part in text.split(","):
        if ".." in part:
            lo, rest = part.split("..")
            hi, count = rest.split("x")
            lo, hi, count = int(lo), int(hi), int(count)
            out += [round(lo * (hi / lo) ** (i / max(1, count - 1))) for i in range(count)]
        elif "x" in part:
            value, count = part.split("x")
            out += [int(value)] * int(count)
        else:
            out.append(int(part))
    return out


def listed():
    return [
        # one decoded token of the larger model's heads: the smallest launch of the step
        {"name": "norm-rope-token", "op": "norm", "hq": 32, "hkv": 8, "d": 128, "tokens": 1, "far": 40000,
         "interleaved": False, "dtype": "float32"},
        # a prompt's queries and keys, from the prefill's fp32 rows q|k|v
        {"name": "norm-rope-prompt", "op": "norm", "hq": 32, "hkv": 8, "d": 128, "tokens": 4096, "far": 0,
         "interleaved": False, "dtype": "float32"},
        # one token of a single stream joins a half-filled block (smaller model's heads)
        {"name": "append-token", "op": "append", "hq": 16, "hkv": 8, "d": 128, "new": "1", "prev": "4133",
         "interleaved": False, "dtype": "float32"},
        # a batch of streams, one token each, at ragged lengths
        {"name": "append-batch", "op": "append", "hq": 32, "hkv": 8, "d": 128, "new": "1x48", "prev": "40..30000x48",
         "interleaved": False, "dtype": "float32"},
        # a prompt into an empty cache beside a chunk that continues another sequence
        {"name": "append-prompt", "op": "append", "hq": 32, "hkv": 8, "d": 128, "new": "4001,130", "prev": "0,1000",
         "interleaved": False, "dtype": "float32"},
        # a shared prefix read back for a look or a move
        {"name": "read-prefix", "op": "read", "hkv": 8, "d": 128, "new": "777", "prev": "51"},
        # a batch's whole contexts moved to another program's cache
        {"name": "read-contexts", "op": "read", "hkv": 8, "d": 128, "new": "2500..9000x8", "prev": "0x8"},
        # one token early in a conversation (smaller model): latency
        {"name": "attend-short", "op": "attend", "hq": 16, "hkv": 8, "d": 128, "new": "1", "prev": "512", "window": 0},
        # one token of a single stream at the models' context limit
        {"name": "attend-long", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "new": "1", "prev": "40959",
         "window": 0},
        # a batch of streams, one token each, ragged
        {"name": "attend-batch", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "new": "1x64",
         "prev": "200..16000x64", "window": 0},
        # seven drafted positions verified at once
        {"name": "attend-verify", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "new": "7", "prev": "12338",
         "window": 0},
        # a prompt from nothing beside a chunk of a long one
        {"name": "attend-prompt", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "new": "4096,1024",
         "prev": "0,15000", "window": 0},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["norm", "append", "read", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8] if hkv < 8 else [1, 2, 4])
    if op == "norm":
        return {"op": op, "hq": hq, "hkv": hkv, "d": d, "tokens": log(1, 4096), "far": rng.randrange(0, 200000),
                "interleaved": rng.random() < 0.3, "dtype": rng.choice(["float32", "bfloat16"])}
    if op == "append":
        if rng.random() < 0.5:      # streams of one to eight tokens each
            seqs, most = log(1, 64), rng.choice([1, 1, 8])
            new = ",".join(str(rng.randint(1, most)) for _ in range(seqs))
        else:                       # prompts and chunks
            seqs = rng.randint(1, 3)
            new = ",".join(str(log(17, 1300)) for _ in range(seqs))
        prev = ",".join(str(rng.choice([0, log(1, 30000)])) for _ in range(seqs))
        return {"op": op, "hq": hq, "hkv": hkv, "d": d, "new": new, "prev": prev,
                "interleaved": rng.random() < 0.3, "dtype": rng.choice(["float32", "bfloat16"])}
    if op == "read":
        seqs = log(1, 8)
        return {"op": op, "hkv": hkv, "d": d, "new": ",".join(str(log(1, 5000)) for _ in range(seqs)),
                "prev": ",".join(str(rng.choice([0, log(1, 3000)])) for _ in range(seqs))}
    kind = rng.random()
    if kind < 0.4:                  # decoding streams
        seqs = log(1, 64)
        new, prev = [1] * seqs, [log(1, 150000 // (seqs + 3)) for _ in range(seqs)]
    elif kind < 0.7:                # verified drafts
        seqs = log(1, 8)
        new, prev = [rng.randint(2, 16) for _ in range(seqs)], [log(1, 12000) for _ in range(seqs)]
    else:                           # prompts and chunks
        seqs = rng.randint(1, 2)
        new = [log(17, 2000) for _ in range(seqs)]
        prev = [rng.choice([0, log(1, 8000)]) for _ in range(seqs)]
    return {"op": op, "hq": hq, "hkv": hkv, "d": d, "new": ",".join(map(str, new)),
            "prev": ",".join(map(str, prev)), "window": rng.choice([0, 0, 0, log(16, 8000)])}


def visible(new, prev, window):
    """(query, key) pairs of one sequence: the query at position p sees min(p + 1, window) keys."""
    full = sum(range(prev + 1, prev + new + 1))
    if window:
        full = sum(min(p, window) for p in range(prev + 1, prev + new + 1))
    return full


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": n * ((4 if case["dtype"] == "float32" else 2) + 2), "flops": 8 * n}
    new, prev = spread(case["new"]), spread(case["prev"])
    kv = 2 * case["hkv"] * case["d"]
    if case["op"] == "append":
        tokens = sum(new)
        back = sum(n + p % BLOCK for n, p in zip(new, prev))    # the tokens of the touched blocks, returned
        e = 4 if case["dtype"] == "float32" else 2
        q = tokens * case["hq"] * case["d"]
        return {"bytes": tokens * kv * (e + 1) + q * (e + 2) + back * kv * 2, "flops": 10 * (tokens * kv + q)}
    if case["op"] == "read":
        return {"bytes": sum(new) * kv * 3, "flops": sum(new) * kv}
    seen = [min(p + n, case["window"] + n - 1) if case["window"] else p + n for n, p in zip(new, prev)]
    pairs = sum(visible(n, p, case["window"]) for n, p in zip(new, prev))
    return {"bytes": sum(seen) * kv + sum(new) * case["hq"] * case["d"] * 4,
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ---- inputs ---------------------------------------------------------------

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def to_codes(k, v):
    """K and V [blocks, heads, 64, D] whole numbers -> codes in the cache's order."""
    n, h, _, d = k.shape
    kc = k.view(n, h, 4, 16, d // 64, 4, 16).permute(0, 1, 2, 4, 5, 3, 6).reshape(n, h, 1, BLOCK * d)
    vc = v.view(n, h, 4, 4, 4, d // 16, 16).permute(0, 1, 5, 3, 6, 2, 4).reshape(n, h, 1, BLOCK * d)
    return torch.cat([kc, vc], 2)


def from_codes(codes, d):
    """codes [..., heads, 2, 64*D] -> K and V [..., heads, 64, D]."""
    lead = codes.shape[:-2]
    m = len(lead)
    ax = tuple(range(m))
    k = codes[..., 0, :].reshape(*lead, 4, d // 64, 4, 16, 16).permute(*ax, m, m + 3, m + 1, m + 2, m + 4)
    v = codes[..., 1, :].reshape(*lead, d // 16, 4, 16, 4, 4).permute(*ax, m + 3, m + 1, m + 4, m, m + 2)
    return k.reshape(*lead, BLOCK, d), v.reshape(*lead, BLOCK, d)


def prepare(case, seed):
    g = generator(seed)
    d, hkv = case["d"], case["hkv"]
    state = {"case": case}
    if case["op"] in ("norm", "append"):
        hq = case["hq"]
        tokens = case["tokens"] if case["op"] == "norm" else sum(spread(case["new"]))
        # the fused q|k|v linear's rows; heads and values of unequal size, as models have them
        rows = torch.randn(tokens, hq + 2 * hkv, d, generator=g, device="cuda")
        rows *= torch.exp(0.7 * torch.randn(1, hq + 2 * hkv, 1, generator=g, device="cuda"))
        rows *= torch.exp(0.4 * torch.randn(tokens, hq + 2 * hkv, 1, generator=g, device="cuda"))
        rows = rows.to(getattr(torch, case["dtype"]))
        state["q"], state["k"], state["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        state["q_gain"] = torch.rand(d, generator=g, device="cuda") * 1.5 + 0.5
        state["k_gain"] = torch.rand(d, generator=g, device="cuda") * 1.5 + 0.5
        state["inv_freq"] = 1e6 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    if case["op"] == "norm":
        state["pos"] = torch.arange(case["far"], case["far"] + tokens, dtype=torch.int32, device="cuda")
    else:
        new, prev = spread(case["new"]), spread(case["prev"])
        total = [n + p for n, p in zip(new, prev)]
        count = [-(-t // BLOCK) for t in total]
        blocks = sum(count) + 3
        order = torch.randperm(blocks, generator=g, device="cuda")[:sum(count)].to(torch.int32)
        table = torch.zeros(len(new), max(count), dtype=torch.int32, device="cuda")
        at = 0
        for i, c in enumerate(count):
            table[i, :c] = order[at:at + c]
            at += c
        state["table"] = table
        state["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
        state["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        # cached tokens: normed keys, values whose size differs from token to token
        codes = torch.empty(blocks, hkv, 2, BLOCK * d, dtype=torch.int8, device="cuda")
        scales = torch.empty(blocks, hkv, 2, device="cuda")
        for lo in range(0, blocks, 256):
            n = min(256, blocks - lo)
            k = torch.randn(n, hkv, BLOCK, d, generator=g, device="cuda")
            v = torch.randn(n, hkv, BLOCK, d, generator=g, device="cuda")
            v *= torch.exp(0.4 * torch.randn(n, hkv, BLOCK, 1, generator=g, device="cuda"))
            s = torch.stack([k.abs().amax((2, 3)), v.abs().amax((2, 3))], 2) / 127
            scales[lo:lo + n] = s
            codes[lo:lo + n] = to_codes(torch.round(k / s[:, :, 0, None, None]),
                                        torch.round(v / s[:, :, 1, None, None])).to(torch.int8)
        state["codes"], state["scales"] = codes, scales
        if case["op"] == "attend":
            # normed queries with a gain: scores spread over a few units, as trained heads have them
            q = torch.randn(sum(new), case["hq"], d, generator=g, device="cuda")
            q *= 0.5 + 2.5 * torch.rand(1, case["hq"], 1, generator=g, device="cuda")
            state["q"] = q.to(torch.bfloat16)
        if case["op"] == "append":
            # the whole of the blocks that the new tokens go to, read back
            back = [n + p % BLOCK for n, p in zip(new, prev)]
            state["back"] = sum(back)
            state["back_cu"] = torch.tensor([sum(back[:i]) for i in range(len(back) + 1)], dtype=torch.int32,
                                            device="cuda")
    if own:
        import ternary_weight_decode_amd as tw
        state["tw"] = tw
        if case["op"] in ("norm", "append"):
            state["transform"] = tw.QkTransform(d, q_gain=state["q_gain"], k_gain=state["k_gain"], eps=EPS,
                                                inv_freq=state["inv_freq"], interleaved=case["interleaved"])
        if case["op"] != "norm":
            state["cache"] = tw.I8KvCache(codes=state["codes"], scales=state["scales"])
            state["batch"] = tw.I8KvBatch(state["cu"], state["lens"], state["table"])
        if case["op"] == "append":
            state["back_batch"] = tw.I8KvBatch(state["back_cu"], state["lens"], state["table"])
    return state


# ---- plain forms ----------------------------------------------------------

def plain_rotate(x, pos, inv_freq, interleaved):
    """x [T, heads, D] fp32, pos [T]."""
    angle = pos.to(torch.float64)[:, None] * inv_freq
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def plain_norm_rope(x, gain, pos, inv_freq, interleaved):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    return plain_rotate(x, pos, inv_freq, interleaved)


def plain_norm(st):
    il = st["case"]["interleaved"]
    return (plain_norm_rope(st["q"], st["q_gain"], st["pos"], st["inv_freq"], il).to(torch.bfloat16),
            plain_norm_rope(st["k"], st["k_gain"], st["pos"], st["inv_freq"], il).to(torch.bfloat16))


def owners(cu, lens, tokens):
    """Sequence and position of every token."""
    t = torch.arange(tokens, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    return seq, t + (lens - cu[1:])[seq]


def plain_read(codes, scales, table, cu, lens, tokens):
    d = codes.shape[-1] // BLOCK
    seq, pos = owners(cu, lens, tokens)
    block, slot = table[seq, pos // BLOCK].long(), pos % BLOCK
    k, v = from_codes(codes, d)
    return ((k[block, :, slot].float() * scales[block, :, 0, None]).to(torch.bfloat16),
            (v[block, :, slot].float() * scales[block, :, 1, None]).to(torch.bfloat16))


def plain_append(st):
    cu, lens, table, codes, scales = st["cu"], st["lens"], st["table"], st["codes"], st["scales"]
    d, tokens = st["case"]["d"], st["q"].shape[0]
    seq, pos = owners(cu, lens, tokens)
    il = st["case"]["interleaved"]
    q = plain_norm_rope(st["q"], st["q_gain"], pos, st["inv_freq"], il).to(torch.bfloat16)
    k = plain_norm_rope(st["k"], st["k_gain"], pos, st["inv_freq"], il)
    block, slot = table[seq, pos // BLOCK].long(), pos % BLOCK
    touched, place = torch.unique(block, return_inverse=True)
    first = torch.full((touched.numel(),), BLOCK, device=cu.device, dtype=slot.dtype)
    first = first.scatter_reduce(0, place, slot, "amin")
    sides = []
    for side, (new, old) in enumerate(zip((k, st["v"].float()), from_codes(codes[touched], d))):
        top = torch.zeros(touched.numel(), new.shape[1], device=cu.device)
        top = top.scatter_reduce(0, place[:, None].expand(-1, new.shape[1]), new.abs().amax(-1), "amax")
        before = torch.where(first[:, None] > 0, scales[touched][:, :, side], torch.zeros_like(top))
        room = 127 * before
        _, e = torch.frexp(top / room)
        grow = torch.clamp(e, min=0).to(torch.float32)          # top / room in [2^(e-1), 2^e)
        grow = torch.where(room * torch.exp2(grow - 1) >= top, grow - 1, grow).clamp(min=0)
        fresh = before == 0
        scale = torch.where(fresh, top / 127, before * torch.exp2(grow))
        grow = torch.where(fresh, torch.zeros_like(grow), grow)
        whole = torch.round(old.float() * torch.exp2(-grow)[:, :, None, None])
        mine = torch.where(scale[place][..., None] > 0, new / scale[place][..., None], torch.zeros_like(new))
        whole[place, :, slot] = torch.round(mine).clamp(-127, 127)
        scales[touched, :, side] = scale
        sides.append(whole)
    codes[touched] = to_codes(*sides).to(torch.int8)
    return (q, *plain_read(codes, scales, table, st["back_cu"], lens, st["back"]))


def plain_attend(st):
    case, codes, scales, table, q = st["case"], st["codes"], st["scales"], st["table"], st["q"].float()
    new, prev = spread(case["new"]), spread(case["prev"])
    d, hkv, group = case["d"], case["hkv"], case["hq"] // case["hkv"]
    out = torch.empty_like(q)

    def some(ids, rows, width, query):
        """Sequences ids: query [ids, rows, hq, d], keys padded to width blocks."""
        k, v = from_codes(codes[table[ids, :width].long()], d)              # [ids, width, hkv, 64, d]
        sc = scales[table[ids, :width].long()]
        k = (k.float() * sc[..., 0, None, None]).transpose(1, 2).reshape(len(ids), hkv, width * BLOCK, d)
        v = (v.float() * sc[..., 1, None, None]).transpose(1, 2).reshape(len(ids), hkv, width * BLOCK, d)
        query = query.view(len(ids), rows, hkv, group, d).transpose(1, 2).reshape(len(ids), hkv, rows * group, d)
        p = torch.matmul(query, k.transpose(2, 3).contiguous()) * d ** -0.5
        n, total = st["cu"][1:][ids] - st["cu"][:-1][ids], st["lens"][ids]
        at = (total - n)[:, None] + torch.arange(rows, device=q.device)     # positions [ids, rows]
        at = at[:, None, :, None].expand(-1, -1, -1, group).reshape(len(ids), 1, rows * group, 1)
        t = torch.arange(width * BLOCK, device=q.device)
        hide = (t > at) | (t >= total[:, None, None, None])
        if case["window"]:
            hide |= t <= at - case["window"]
        p.masked_fill_(hide, float("-inf"))
        p -= p.amax(-1, keepdim=True)
        p = p.exp_()
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        return o.view(len(ids), hkv, rows, group, d).transpose(1, 2).reshape(len(ids), rows, hkv * group, d)

    if max(new) <= 16:      # a batch, padded
        rows = max(new)
        ids = torch.arange(len(new), device=q.device)
        take = (st["cu"][:-1, None] + torch.arange(rows, device=q.device)).clamp(max=q.shape[0] - 1)
        o = some(ids, rows, table.shape[1], q[take])
        keep = torch.arange(rows, device=q.device) < (st["cu"][1:] - st["cu"][:-1])[:, None]
        out = o[keep]
    else:                   # one sequence after another, its queries in parts
        at = 0
        for i, (n, p) in enumerate(zip(new, prev)):
            ids = torch.tensor([i], device=q.device)
            out[at:at + n] = some(ids, n, -(-(n + p) // BLOCK), q[None, at:at + n])[0]
            at += n
    return out.to(torch.bfloat16)


# ---- one pass -------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "norm":
            return plain_norm(state)
        if op == "append":
            return plain_append(state)
        if op == "read":
            return plain_read(state["codes"], state["scales"], state["table"], state["cu"], state["lens"],
                              sum(spread(state["case"]["new"])))
        return plain_attend(state)
    tw = state["tw"]
    if op == "norm":
        return tw.qk_norm_rope(state["transform"], state["q"], state["k"], state["pos"])
    if op == "append":
        q = tw.i8_kv_append(state["cache"], state["batch"], state["transform"], state["k"], state["v"],
                            q=state["q"])
        return (q, *tw.i8_kv_read(state["cache"], state["back_batch"], state["back"]))
    if op == "read":
        return tw.i8_kv_read(state["cache"], state["batch"], sum(spread(state["case"]["new"])))
    return tw.i8_kv_attend(state["cache"], state["batch"], state["q"], window=state["case"]["window"])


# ---- the definitions in 64 bits -------------------------------------------

def exact_turn(x, gain, pos, inv_freq, interleaved):
    """x [T, heads, D]: norm, gain, then each pair turned as a complex number."""
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gain.double()
    half = x.shape[-1] // 2
    pairs = x.unflatten(-1, (half, 2)) if interleaved else x.unflatten(-1, (2, half)).transpose(-1, -2)
    angle = pos.double().view(-1, 1, 1) * inv_freq
    z = torch.complex(pairs[..., 0], pairs[..., 1]) * torch.polar(torch.ones_like(angle), angle)
    y = torch.stack([z.real, z.imag], -1)
    return (y if interleaved else y.transpose(-1, -2)).flatten(-2)


def exact_block(state, number, head, side):
    """Codes [64, D] of one block, head and side, taken from their places one by one."""
    d = state["case"]["d"]
    t = torch.arange(BLOCK, device="cuda")[:, None]
    c = torch.arange(d, device="cuda")[None, :]
    if side == 0:
        place = (((t // 16) * (d // 64) + c // 64) * 4 + c % 64 // 16) * 256 + t % 16 * 16 + c % 16
    else:
        place = (((c // 16) * 4 + t % 16 // 4) * 16 + c % 16) * 16 + t // 16 * 4 + t % 4
    return state["codes"][number][..., head, side, :][..., place].double()


def exact_sequence(state, i, length):
    """K and V [length, hkv, D] of sequence i."""
    blocks = state["table"][i, :-(-length // BLOCK)].long()
    sides = []
    for side in (0, 1):
        heads = [(exact_block(state, blocks, h, side) * state["scales"][blocks, h, side].double()[:, None, None])
                 .flatten(0, 1)[:length] for h in range(state["case"]["hkv"])]
        sides.append(torch.stack(heads, 1))
    return sides


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return tuple(exact_turn(st[n], st[n + "_gain"], st["pos"], st["inv_freq"], case["interleaved"])
                     for n in ("q", "k"))
    new, prev = spread(case["new"]), spread(case["prev"])
    if case["op"] == "read":
        parts = [exact_sequence(st, i, n + p) for i, (n, p) in enumerate(zip(new, prev))]
        return tuple(torch.cat([part[side][p:] for part, p in zip(parts, prev)]) for side in (0, 1))
    if case["op"] == "append":
        pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, prev)]).cuda()
        q = exact_turn(st["q"], st["q_gain"], pos, st["inv_freq"], case["interleaved"])
        fresh = [exact_turn(st["k"], st["k_gain"], pos, st["inv_freq"], case["interleaved"]), st["v"].double()]
        back = [[], []]
        at = 0
        for i, (n, p) in enumerate(zip(new, prev)):
            for side in (0, 1):
                left, done = p, 0
                while done < n:
                    slot, m = left % BLOCK, min(n - done, BLOCK - left % BLOCK)
                    mine = fresh[side][at + done:at + done + m].transpose(0, 1)     # [hkv, m, d]
                    top = mine.abs().amax((1, 2))
                    if slot == 0:
                        scale = top / 127
                        kept = mine[:, :0]
                    else:
                        number = int(st["table"][i, left // BLOCK])
                        old = torch.stack([exact_block(st, number, h, side)[:slot] for h in range(case["hkv"])])
                        scale = st["scales"][number, :, side].double()
                        grow = torch.ceil(torch.log2(top / (127 * scale))).clamp(min=0)
                        scale = scale * 2 ** grow
                        kept = torch.round(old / (2 ** grow)[:, None, None]) * scale[:, None, None]
                    put = torch.round(mine / scale[:, None, None]).clamp(-127, 127) * scale[:, None, None]
                    back[side].append(torch.cat([kept, put], 1).transpose(0, 1))
                    left, done = left + m, done + m
            at += n
        return (q, torch.cat(back[0]), torch.cat(back[1]))
    out, at = [], 0
    group = case["hq"] // case["hkv"]
    for i, (n, p) in enumerate(zip(new, prev)):
        k, v = exact_sequence(st, i, n + p)
        rows = []
        for lo in range(0, n, 1024):
            hi = min(n, lo + 1024)
            pos = torch.arange(p + lo, p + hi, device="cuda")[:, None]
            t = torch.arange(n + p, device="cuda")[None, :]
            seen = t <= pos
            if case["window"]:
                seen = seen & (pos - t < case["window"])
            heads = []
            for h in range(case["hq"]):
                s = st["q"][at + lo:at + hi, h].double() @ k[:, h // group].T / math.sqrt(case["d"])
                heads.append(torch.softmax(s.masked_fill(~seen, -math.inf), -1) @ v[:, h // group])
            rows.append(torch.stack(heads, 1))
        out.append(torch.cat(rows))
        at += n
    return torch.cat(out)
