"""The step of a drafted tree, measured: matrix-vector products with 4-bit
weights and group scales, the trees' masks and positions, attention of a tree's
rows over the paged int8 cache, and the accepted branch left alone in the cache.

With ``own`` false every operator runs in its plain form (elementary torch
operations in 32 bits); with ``own`` true the framework's calls run on the same
tensors.

4-bit weights: W[n][k] = t[n][k] * scale[n][k / group], t in [-8, 7], fp16
scales.

A tree: rows 0 .. n-1 of a sequence are its newest tokens, at positions
(slots) p0 .. p0 + n - 1 of its cache; parent[j] < j is the row that row j
continues, -1 what continues the cached context itself.  mask[j] has the bits
of j and of the rows that it descends from (64 to a word).  The cache is that of
include/tern.h: a block holds 64 tokens of one sequence, codes int8 [blocks][kv
heads][2][64*D] (K, then V), one fp32 scale for each block, head and side, the
codes of a block in the order
  K: token 16t + r, dim 64s + 16g + b  at  [t][s][g][r][b]
  V: token 16t + 4g + i, dim 16u + r   at  [u][g][r][t][i]
"""
import math
import random

import torch

own = False

BLOCK = 64
VOCAB = 151936


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
        else:
            out.append(int(part))
    return out


def listed():
    return [
        # one token through the smaller model's fused q|k|v: the smallest launch, latency counts
        {"name": "q4-token-small", "op": "gemv", "n": 4096, "k": 1024, "group": 32, "m": 1, "act": "bf16"},
        # one token through the larger model's fused gate|up: the weights' bytes count
        {"name": "q4-token-gateup", "op": "gemv", "n": 24576, "k": 4096, "group": 128, "m": 1, "act": "bf16"},
        # seven drafted positions through the larger model's down, int8 activations
        {"name": "q4-verify-down", "op": "gemv", "n": 4096, "k": 12288, "group": 64, "m": 7, "act": "int8"},
        # an odd matrix with a tree level of thirteen rows
        {"name": "q4-ragged", "op": "gemv", "n": 5003, "k": 1152, "group": 32, "m": 13, "act": "bf16"},
        # one tree of a single stream
        {"name": "mask-tree", "op": "mask", "nodes": "64", "prev": "12338", "fan": 12},
        # a batch of trees, from a lone root to the widest
        {"name": "mask-batch", "op": "mask", "nodes": "1..512x48", "prev": "200..16000x48", "fan": 40},
        # a small tree early in a conversation (smaller model): latency
        {"name": "attend-tree-small", "op": "attend", "hq": 16, "hkv": 8, "d": 128, "nodes": "8", "prev": "512",
         "fan": 3},
        # one tree of a single stream in a long context
        {"name": "attend-tree", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "nodes": "64", "prev": "12338",
         "fan": 12},
        # a batch of streams with trees of their own, ragged
        {"name": "attend-tree-batch", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "nodes": "9..33x32",
         "prev": "200..8000x32", "fan": 5},
        # trees of many rows, several words of mask each
        {"name": "attend-tree-wide", "op": "attend", "hq": 32, "hkv": 8, "d": 128, "nodes": "500,130",
         "prev": "4001,900", "fan": 50},
        # the accepted branch of a single stream's tree (smaller model's layer)
        {"name": "keep-tree", "op": "keep", "hkv": 8, "d": 128, "nodes": "64", "prev": "12338", "fan": 12},
        # a batch of streams
        {"name": "keep-batch", "op": "keep", "hkv": 8, "d": 128, "nodes": "9..64x48", "prev": "40..16000x48", "fan": 9},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["gemv", "gemv", "mask", "attend", "attend", "keep"])
    if op == "gemv":
        k = 128 * log(1, 128)
        return {"op": op, "n": log(1, min(30000, 90000000 // k)), "k": k, "group": rng.choice([32, 64, 128]),
                "m": rng.choice([1, 1, rng.randint(2, 16)]), "act": rng.choice(["bf16", "bf16", "int8"])}
    seqs = log(1, 32)
    top = 512 if op == "mask" else 64 if seqs > 4 else 400
    nodes = [log(1, top) for _ in range(seqs)]
    prev = [rng.choice([0, log(1, 6000), log(1, 200000 // (seqs * 5 + 10))]) for _ in range(seqs)]
    case = {"op": op, "nodes": ",".join(map(str, nodes)), "prev": ",".join(map(str, prev)),
            "fan": rng.choice([1, rng.randint(2, 12), rng.randint(8, 60)])}
    if op == "mask":        # branching trees: another seed is another tree
        nodes[0], case["fan"] = max(nodes[0], 24), rng.randint(2, 60)
        case["nodes"] = ",".join(map(str, nodes))
    if op != "mask":
        hkv = rng.choice([1, 2, 4, 8])
        case.update({"hkv": hkv, "d": rng.choice([64, 128, 128])})
        if op == "attend":
            case["hq"] = hkv * rng.choice([1, 2, 3, 4, 8] if hkv < 8 else [1, 2, 4])
    return case


def work(case):
    if case["op"] == "gemv":
        n, k, m = case["n"], case["k"], case["m"]
        e = 2 if case["act"] == "bf16" else 1
        return {"bytes": n * k / 2 + 2 * n * k / case["group"] + m * k * e + 4 * m * n, "flops": 2 * m * n * k}
    nodes, prev = spread(case["nodes"]), spread(case["prev"])
    rows = sum(nodes)
    if case["op"] == "mask":
        return {"bytes": rows * (4 + 4 + 8 * words_of(nodes)), "flops": 0}
    kv = 2 * case["hkv"] * case["d"]
    if case["op"] == "keep":
        # at least the root of each tree is kept: its block's tokens are returned
        back = sum(1 + p % BLOCK for p in prev)
        return {"bytes": rows * 12 + back * kv * 3, "flops": back * kv}
    # every row sees its context and itself
    return {"bytes": sum(n + p for n, p in zip(nodes, prev)) * kv + rows * case["hq"] * case["d"] * 4,
            "flops": 4 * sum(n * (p + 1) for n, p in zip(nodes, prev)) * case["hq"] * case["d"]}


def words_of(nodes):
    return -(-max(nodes) // 64)


# ---- inputs ---------------------------------------------------------------

def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def make_tree(rng, n, fan):
    """Parents of a drafter's candidates, level by level, up to `fan` in a level (1: a chain)."""
    parent, level = [-1], [0]
    while len(parent) < n:
        width = min(n - len(parent), rng.randint(1 + fan // 2, fan) if fan > 1 else 1)
        at = len(parent)
        parent += sorted(rng.choice(level) for _ in range(width))
        level = list(range(at, at + width))
    return parent


def branch(parent, row):
    """Rows from the root to `row`."""
    out = []
    while row >= 0:
        out.append(row)
        row = parent[row]
    return out[::-1]


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
    state = {"case": case}
    if case["op"] == "gemv":
        n, k, group, m = case["n"], case["k"], case["group"], case["m"]
        # rounded weights of a bell curve, its tails clipped
        t = torch.randn(n, k, generator=g, device="cuda").mul_(2.9).round_().clamp_(-8, 7).to(torch.int8)
        scale = (torch.rand(n, k // group, generator=g, device="cuda") * 0.02 + 0.002).to(torch.float16)
        # channels of unequal size, as activations have them
        x = torch.randn(m, k, generator=g, device="cuda")
        x *= torch.exp(0.8 * torch.randn(1, k, generator=g, device="cuda"))
        state["t"], state["scale"] = t, scale
        if case["act"] == "int8":
            state["s_x"] = x.abs().amax(1) / 127
            state["q"] = torch.round(x / state["s_x"][:, None]).clamp_(-127, 127).to(torch.int8)
        else:
            state["x"] = x.to(torch.bfloat16)
        if own:
            import ternary_weight_decode_amd as tw
            state["tw"], state["packed"] = tw, tw.q4_pack(t, scale)
        return state

    rng = random.Random(seed * 104729 + 5)
    nodes, prev = spread(case["nodes"]), spread(case["prev"])
    # how many tokens are kept, so how many come back, goes by the trees alone: these are the case's own there
    shape = random.Random(case["nodes"]) if case["op"] == "keep" else rng
    trees = [make_tree(shape, n, case["fan"]) for n in nodes]
    total = [n + p for n, p in zip(nodes, prev)]
    rows = sum(nodes)

    def whole(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device="cuda")

    state["cu"] = whole([sum(nodes[:i]) for i in range(len(nodes) + 1)])
    state["lens"] = whole(total)
    state["parent"] = whole([p for tree in trees for p in tree])
    words = state["words"] = words_of(nodes)
    hkv, d = case.get("hkv", 1), case.get("d", 64)
    count = [-(-t // BLOCK) for t in total]
    blocks = sum(count) + 3
    order = torch.randperm(blocks, generator=g, device="cuda")[:sum(count)].to(torch.int32)
    table = torch.zeros(len(nodes), max(count), dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(count):
        table[i, :c] = order[at:at + c]
        at += c
    state["table"] = table
    if case["op"] != "mask":
        # cached tokens: normed keys, values whose size differs from token to token and block to block
        codes = torch.empty(blocks, hkv, 2, BLOCK * d, dtype=torch.int8, device="cuda")
        scales = torch.empty(blocks, hkv, 2, device="cuda")
        for lo in range(0, blocks, 256):
            n = min(256, blocks - lo)
            k = torch.randn(n, hkv, BLOCK, d, generator=g, device="cuda")
            v = torch.randn(n, hkv, BLOCK, d, generator=g, device="cuda")
            v *= torch.exp(0.4 * torch.randn(n, hkv, BLOCK, 1, generator=g, device="cuda"))
            v *= torch.exp(0.4 * torch.randn(n, hkv, 1, 1, generator=g, device="cuda"))
            s = torch.stack([k.abs().amax((2, 3)), v.abs().amax((2, 3))], 2) / 127
            scales[lo:lo + n] = s
            codes[lo:lo + n] = to_codes(torch.round(k / s[:, :, 0, None, None]),
                                        torch.round(v / s[:, :, 1, None, None])).to(torch.int8)
        state["codes"], state["scales"] = codes, scales
    if case["op"] == "attend":
        # the step's masks, made once for all layers
        bits = []
        for tree in trees:
            mask = []
            for j, p in enumerate(tree):
                mask.append((mask[p] if p >= 0 else 0) | 1 << j)
            bits += [[(m >> 64 * w & (1 << 64) - 1) for w in range(words)] for m in mask]
        state["mask"] = whole([[b - (1 << 64) if b >> 63 else b for b in row] for row in bits], torch.int64)
        # normed queries with a gain: scores spread over a few units, as trained heads have them
        q = torch.randn(rows, case["hq"], d, generator=g, device="cuda")
        q *= 0.5 + 2.5 * torch.rand(1, case["hq"], 1, generator=g, device="cuda")
        state["q"] = q.to(torch.bfloat16)
    if case["op"] == "keep":
        token, target, kept = [], [], []
        for tree in trees:
            mine = rng.sample(range(VOCAB), 2 * len(tree))      # all unlike
            choice, answer = mine[:len(tree)], mine[len(tree):]
            # a branch whose tokens come from where none of them goes, so that a pass can be repeated
            rowsof = [branch(tree, r) for r in shape.sample(range(len(tree)), min(len(tree), 40))] + [[0]]
            best = max((b for b in rowsof if all(r == k or r >= len(b) for k, r in enumerate(b))), key=len)
            for a, b in zip(best, best[1:]):
                answer[a] = choice[b]
            token += choice
            target += answer
            kept.append(len(best))
        state["token"], state["target"] = whole(token), whole(target)
        state["width"] = 20
        # the whole of the blocks that the kept tokens stand in, read back
        back = [min(c, 20) + p % BLOCK for c, p in zip(kept, prev)]
        state["back"] = sum(back)
        state["back_cu"] = whole([sum(back[:i]) for i in range(len(back) + 1)])
        state["lens_out"] = torch.empty(len(nodes), dtype=torch.int32, device="cuda")
    if own:
        import ternary_weight_decode_amd as tw
        state["tw"] = tw
        state["batch"] = tw.I8KvBatch(state["cu"], state["lens"], table)
        if case["op"] != "mask":
            state["cache"] = tw.I8KvCache(codes=state["codes"], scales=state["scales"])
        if case["op"] == "keep":
            state["back_batch"] = tw.I8KvBatch(state["back_cu"], state["lens_out"], table)
    return state


# ---- plain forms ----------------------------------------------------------

def plain_gemv(st):
    t, scale = st["t"], st["scale"]
    n, k = t.shape
    w = (t.view(n, -1, st["case"]["group"]).float() * scale.float()[:, :, None]).view(n, k)
    x = st["q"].float() * st["s_x"][:, None] if "q" in st else st["x"].float()
    return torch.matmul(x, w.t())


def owners(cu, lens, tokens):
    """Sequence of every token, its row there and its position."""
    t = torch.arange(tokens, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t.to(torch.int32), right=True)
    return seq, t - cu[seq], t + (lens - cu[1:])[seq]


def ancestors(st):
    """[sequences, rows, rows]: 1 where the column is the row itself or one that it descends from."""
    nodes = spread(st["case"]["nodes"])
    n, rows, parent = len(nodes), max(nodes), st["parent"].long()
    seq, j, _ = owners(st["cu"], st["lens"], sum(nodes))
    near = torch.zeros(n, rows, rows + 1, device=parent.device)     # the last column: no parent
    near[seq, j, torch.where(parent < 0, rows, parent)] = 1
    near = near[:, :, :rows] + torch.eye(rows, device=parent.device)
    for _ in range((rows - 1).bit_length()):                         # twice as far back each time
        near = torch.clamp(torch.matmul(near, near), max=1)
    return near


def plain_mask(st):
    nodes, words = spread(st["case"]["nodes"]), st["words"]
    near = ancestors(st)
    n, rows, _ = near.shape
    seq, j, _ = owners(st["cu"], st["lens"], sum(nodes))
    mine = near[seq, j]                                              # [T, rows]
    bit = torch.zeros(mine.shape[0], words * 64, dtype=torch.int64, device=mine.device)
    bit[:, :rows] = mine.to(torch.int64)
    mask = (bit.view(-1, words, 64) << torch.arange(64, device=mine.device)).sum(-1)
    pos = (st["lens"] - st["cu"][1:] + st["cu"][:-1])[seq] + mine.sum(-1).to(torch.int32) - 1
    return mask, pos.to(torch.int32)


def plain_read(codes, scales, table, cu, lens, tokens):
    d = codes.shape[-1] // BLOCK
    seq, _, pos = owners(cu, lens, tokens)
    block, slot = table[seq, pos // BLOCK].long(), pos % BLOCK
    some, place = torch.unique(block, return_inverse=True)
    k, v = from_codes(codes[some], d)
    return ((k[place, :, slot].float() * scales[block, :, 0, None]).to(torch.bfloat16),
            (v[place, :, slot].float() * scales[block, :, 1, None]).to(torch.bfloat16))


def plain_attend(st):
    case, codes, scales, table, q = st["case"], st["codes"], st["scales"], st["table"], st["q"].float()
    nodes = spread(case["nodes"])
    d, hkv, group = case["d"], case["hkv"], case["hq"] // case["hkv"]
    n, rows, width = len(nodes), max(nodes), table.shape[1]
    take = (st["cu"][:-1, None] + torch.arange(rows, device=q.device)).clamp(max=q.shape[0] - 1)
    k, v = from_codes(codes[table.long()], d)                           # [n, width, hkv, 64, d]
    sc = scales[table.long()]
    k = (k.float() * sc[..., 0, None, None]).transpose(1, 2).reshape(n, hkv, width * BLOCK, d)
    v = (v.float() * sc[..., 1, None, None]).transpose(1, 2).reshape(n, hkv, width * BLOCK, d)
    query = q[take].view(n, rows, hkv, group, d).transpose(1, 2).reshape(n, hkv, rows * group, d)
    p = torch.matmul(query, k.transpose(2, 3).contiguous()) * d ** -0.5
    # token p of the context, or row p - p0 of the tree where its bit is set
    first = (st["lens"] - st["cu"][1:] + st["cu"][:-1]).long()
    t = torch.arange(width * BLOCK, device=q.device)
    row = t - first[:, None]                                             # [n, keys]
    at = row.clamp(0, 64 * st["words"] - 1)
    word = st["mask"][take].gather(2, (at // 64)[:, None].expand(-1, rows, -1))
    seen = (row < 0)[:, None] | ((word >> (at % 64)[:, None]) & 1 == 1) & \
        (row < (st["cu"][1:] - st["cu"][:-1])[:, None])[:, None]         # [n, rows, keys]
    seen = seen[:, :, None].expand(-1, -1, group, -1).reshape(n, 1, rows * group, -1)
    p.masked_fill_(~seen, float("-inf"))
    p -= p.amax(-1, keepdim=True)
    p = p.exp_()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    o = o.view(n, hkv, rows, group, d).transpose(1, 2).reshape(n, rows, hkv * group, d)
    return o[torch.arange(rows, device=q.device) < (st["cu"][1:] - st["cu"][:-1])[:, None]].to(torch.bfloat16)


def plain_keep(st):
    nodes, width = spread(st["case"]["nodes"]), st["width"]
    codes, scales, table, cu, lens = st["codes"], st["scales"], st["table"], st["cu"], st["lens"]
    near = ancestors(st)
    n, rows, _ = near.shape
    seq, j, _ = owners(cu, lens, sum(nodes))
    start = cu[:-1].long()[seq]
    parent = st["parent"].long()
    # a row is accepted where it and all that it descends from carry the token that the target answers
    # their parents with (siblings are unlike)
    agrees = (parent < 0) & (j == 0) | (parent >= 0) & (st["token"] == st["target"][start + parent.clamp(min=0)])
    wrong = torch.ones(n, rows, device=codes.device)
    wrong[seq, j] = 1 - agrees.float()
    taken = torch.matmul(near, wrong[:, :, None])[:, :, 0] == 0          # [n, rows], a chain of rows
    rank = taken.cumsum(1) - 1
    taken &= rank < width
    path = torch.full((n, width + 1), -1, dtype=torch.int64, device=codes.device)
    path.scatter_(1, torch.where(taken, rank, width), torch.where(
        taken, torch.arange(rows, device=codes.device), torch.full_like(rank, -1)))
    path = path[:, :width]
    count = (path >= 0).sum(1)
    last = path.gather(1, count[:, None] - 1)[:, 0]
    following = st["target"][cu[:-1] + last]
    # the kept rows' tokens, from slot p0 + path[k] to slot p0 + k
    p0 = lens - (cu[1:] - cu[:-1])
    lens_out = (p0 + count).to(torch.int32)
    i, k = torch.nonzero(path >= 0, as_tuple=True)
    to, of = p0[i] + k, p0[i] + path[i, k]
    to_block, of_block = table[i, to // BLOCK].long(), table[i, of // BLOCK].long()
    touched, place = torch.unique(to_block, return_inverse=True)
    source, origin = torch.unique(of_block, return_inverse=True)
    d = st["case"]["d"]
    moves = (to_block != of_block)[:, None]
    sides = []
    given, kept = from_codes(codes[source], d), from_codes(codes[touched], d)
    for side in (0, 1):
        code = given[side][origin, :, of % BLOCK].float()               # [moved, heads, d]
        value = code * scales[of_block][:, :, side, None]
        most = torch.where(moves, value.abs().amax(-1), torch.zeros_like(value[..., 0]))
        top = torch.zeros(touched.numel(), value.shape[1], device=codes.device)
        top = top.scatter_reduce(0, place[:, None].expand(-1, value.shape[1]), most, "amax")
        before = scales[touched][:, :, side]
        room = 127 * before
        _, e = torch.frexp(top / room)
        grow = torch.clamp(e, min=0).to(torch.float32)                   # top / room in [2^(e-1), 2^e)
        grow = torch.where(room * torch.exp2(grow - 1) >= top, grow - 1, grow).clamp(min=0)
        scale = before * torch.exp2(grow)
        old = torch.round(kept[side].float() * torch.exp2(-grow)[:, :, None, None])
        same = torch.round(code * torch.exp2(-grow)[place][..., None])
        other = torch.round(value / scale[place][..., None]).clamp(-127, 127)
        old[place, :, to % BLOCK] = torch.where(moves[..., None], other, same)
        sides.append((old, scale))
    codes[touched] = to_codes(sides[0][0], sides[1][0]).to(torch.int8)
    scales[touched] = torch.stack([sides[0][1], sides[1][1]], 2)
    st["lens_out"].copy_(lens_out)
    return (path.to(torch.int32), count.to(torch.int32), following, lens_out,
            *plain_read(codes, scales, table, st["back_cu"], lens_out, st["back"]))


# ---- one pass -------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if not own:
        return {"gemv": plain_gemv, "mask": plain_mask, "attend": plain_attend, "keep": plain_keep}[op](state)
    tw = state["tw"]
    if op == "gemv":
        n, k, group = state["case"]["n"], state["case"]["k"], state["case"]["group"]
        if "q" in state:
            return tw.q4_gemv_i8(state["packed"], n, k, group, state["q"], state["s_x"])
        return tw.q4_gemv(state["packed"], n, k, group, state["x"])
    if op == "mask":
        return tw.draft_tree_mask(state["batch"], state["parent"], state["words"])
    if op == "attend":
        return tw.i8_kv_attend_tree(state["cache"], state["batch"], state["q"], state["mask"])
    path, count, following = tw.draft_tree_accept(state["batch"], state["parent"], state["token"], state["target"],
                                                  state["width"])
    lens = tw.i8_kv_keep(state["cache"], state["batch"], state["parent"].shape[0], path, lens_out=state["lens_out"])
    return (path, count, following, lens, *tw.i8_kv_read(state["cache"], state["back_batch"], state["back"]))


# ---- the definitions in 64 bits -------------------------------------------

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


def exact_sequence(state, i, length, head):
    """K and V [length, D] of one head of sequence i."""
    blocks = state["table"][i, :-(-length // BLOCK)].long()
    return [(exact_block(state, blocks, head, side) * state["scales"][blocks, head, side].double()[:, None, None])
            .flatten(0, 1)[:length] for side in (0, 1)]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "mask":
        return None
    if case["op"] == "gemv":
        x = st["x"].double() if "x" in st else st["q"].double() * st["s_x"].double()[:, None]
        out = []
        for lo in range(0, case["n"], 4096):
            w = st["t"][lo:lo + 4096].double() * st["scale"][lo:lo + 4096].double().repeat_interleave(case["group"], 1)
            out.append((w @ x.t()).t())
        return torch.cat(out, 1)
    nodes, prev = spread(case["nodes"]), spread(case["prev"])
    parent = st["parent"].tolist()
    if case["op"] == "attend":
        group = case["hq"] // case["hkv"]
        out, at = [], 0
        for i, (n, p) in enumerate(zip(nodes, prev)):
            tree = parent[at:at + n]
            seen = torch.zeros(n, p + n, dtype=torch.bool)
            seen[:, :p] = True
            for j in range(n):
                seen[j, [p + r for r in branch(tree, j)]] = True
            seen = seen.cuda()
            heads = []
            for h in range(case["hkv"]):
                k, v = exact_sequence(st, i, n + p, h)
                for s in range(h * group, (h + 1) * group):
                    score = st["q"][at:at + n, s].double() @ k.T / math.sqrt(case["d"])
                    heads.append(torch.softmax(score.masked_fill(~seen, -math.inf), -1) @ v)
            out.append(torch.stack(heads, 1))
            at += n
        return torch.cat(out)
    # keep: one sequence, head and side after another
    token, target = st["token"].tolist(), st["target"].tolist()
    sides, at = ([], []), 0
    for i, (n, p) in enumerate(zip(nodes, prev)):
        tree, path = parent[at:at + n], [0]
        while len(path) < st["width"]:
            child = [c for c in range(n) if tree[c] == path[-1] and token[at + c] == target[at + path[-1]]]
            if not child:
                break
            path.append(child[0])
        at += n
        for side in (0, 1):
            heads = []
            for h in range(case["hkv"]):
                rows = []
                for block in range(p // BLOCK, (p + len(path) - 1) // BLOCK + 1):
                    number = int(st["table"][i, block])
                    scale = float(st["scales"][number, h, side])
                    code = exact_block(st, number, h, side)
                    mine = [(k, r) for k, r in enumerate(path) if (p + k) // BLOCK == block]
                    far = {}
                    for k, r in mine:
                        if (p + r) // BLOCK != block:
                            other = int(st["table"][i, (p + r) // BLOCK])
                            far[k] = exact_block(st, other, h, side)[(p + r) % BLOCK] * float(st["scales"][other, h, side])
                    top = max([float(f.abs().max()) for f in far.values()], default=0.0)
                    grow = 0
                    while top > 127 * scale * 2 ** grow:
                        grow += 1
                    scale *= 2 ** grow
                    new = torch.round(code / 2 ** grow)
                    for k, r in mine:
                        new[(p + k) % BLOCK] = (torch.round(far[k] / scale).clamp(-127, 127) if k in far
                                                else torch.round(code[(p + r) % BLOCK] / 2 ** grow))
                    rows.append(new * scale)
                rows = torch.cat(rows)[:p % BLOCK + len(path)]
                heads.append(rows)
            sides[side].append(torch.stack(heads, 1))
    return (None, None, None, None, torch.cat(sides[0]), torch.cat(sides[1]))
