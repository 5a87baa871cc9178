"""Cases of the operators for drafted tokens: what a serving step with a tree of drafts does around the model's
products, over the 8-bit key/value cache, and the pass in front of the cache that training shares with it.

Queries and keys are normed for each head and rotated to their positions (`norm`; `norm_grad` is its backward pass).
The requests' drafts form trees, whose places and visibility follow from their parents (`trees`); their queries attend
over the cache and over their ancestors (`attention`); the target's probabilities decide which drafts stay (`verify`);
and their keys and values move together in the cache (`compact`).

`run` computes them with elementary torch operations where `own` is false and through the
package's entry points where it is true.  `exact` is the definition in 64 bits.
"""
import math
import zlib

import numpy as np
import torch

own = False

CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a batch's trees before a step: all latency
        {"name": "trees_64x32", "op": "trees", "requests": 64, "nodes": 32, "ragged": False, "context": 4096, "window": 0, "pad": 0},
        # the trees of a large server's step
        {"name": "trees_2000x200", "op": "trees", "requests": 2000, "nodes": 200, "ragged": True, "context": 32768, "window": 64,
         "pad": 37},
        # single tokens of 64 running requests, slices of one projection
        {"name": "norm_decode_64", "op": "norm", "tokens": 64, "heads": 32, "kv_heads": 8, "head": 128, "rotate": 128,
         "interleaved": False, "type": "bf16", "weight": "bf16", "fused": True, "positions": 8192, "pad": 3},
        # prompts' tokens
        {"name": "norm_prefill_16k", "op": "norm", "tokens": 16384, "heads": 32, "kv_heads": 8, "head": 128, "rotate": 128,
         "interleaved": False, "type": "bf16", "weight": "bf16", "fused": True, "positions": 32768, "pad": 0},
        # a training step's backward pass: short heads, neighbours rotated in pairs, half of each head, the other type
        {"name": "norm_grad_8k_f16", "op": "norm_grad", "tokens": 8191, "heads": 32, "kv_heads": 16, "head": 64, "rotate": 32,
         "interleaved": True, "type": "f16", "weight": "f32", "fused": False, "positions": 8192, "pad": 0},
        # a small tree of one request over a short context: latency
        {"name": "attention_1x8", "op": "attention", "requests": 1, "nodes": 8, "ragged": False, "context": 777, "heads": 32,
         "kv_heads": 8, "head": 128, "block_tokens": 64, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 0},
        # a batch of trees
        {"name": "attention_32x32", "op": "attention", "requests": 32, "nodes": 32, "ragged": True, "context": 4096, "heads": 32,
         "kv_heads": 8, "head": 128, "block_tokens": 64, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 2},
        # large trees over long contexts, short heads, blocks of 16, the other types, a window
        {"name": "attention_9x61_f16", "op": "attention", "requests": 9, "nodes": 61, "ragged": True, "context": 32768, "heads": 48,
         "kv_heads": 16, "head": 64, "block_tokens": 16, "window": 20000, "type": "f16", "codes": "e5m2", "pad": 0},
        # a small tree of the likeliest tokens, one request
        {"name": "verify_1x26", "op": "verify", "requests": 1, "nodes": 26, "chain": False, "vocab": 32000, "certain": True},
        # a batch's chains of tokens drawn from a draft model's probabilities
        {"name": "verify_64x5", "op": "verify", "requests": 64, "nodes": 5, "chain": True, "vocab": 128256, "certain": False},
        # the accepted drafts of a batch
        {"name": "compact_64x32", "op": "compact", "requests": 64, "nodes": 32, "context": 4096, "kv_heads": 8, "head": 128,
         "block_tokens": 64, "codes": "e4m3"},
        # and of a large one with long paths, blocks of 16, the other 8-bit type
        {"name": "compact_500x100", "op": "compact", "requests": 500, "nodes": 100, "context": 1000, "kv_heads": 16, "head": 64,
         "block_tokens": 16, "codes": "e5m2"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["trees", "norm", "norm", "norm_grad", "norm_grad", "attention", "attention", "attention", "verify",
                     "verify", "compact"])
    if op == "trees":
        return {"op": op, "requests": _spread(rng, 1, 2000), "nodes": _spread(rng, 12, 200), "ragged": rng.random() < 0.7,
                "context": _spread(rng, 200, 100000), "window": rng.choice([0, 0, 3, 64]), "pad": rng.choice([0, 1, 40])}
    if op in ("norm", "norm_grad"):
        heads, kv_heads, d = rng.choice([(32, 8, 128), (64, 8, 128), (16, 16, 64), (16, 2, 64), (5, 1, 128), (8, 4, 256),
                                         (12, 12, 96), (3, 1, 80)])
        return {"op": op, "tokens": _spread(rng, 1, 160_000_000 // (2 * (heads + kv_heads) * d) // (1 if op == "norm" else 2)),
                "heads": heads, "kv_heads": kv_heads, "head": d, "rotate": rng.choice([d, d, 32, 0]),
                "interleaved": rng.random() < 0.4, "type": rng.choice(["bf16", "bf16", "f16"]),
                "weight": rng.choice(["same", "f32"]), "fused": rng.random() < 0.5, "positions": _spread(rng, 1, 100000),
                "pad": rng.choice([0, 0, 5])}
    if op == "verify":
        vocab, certain = _spread(rng, 1000, 150000), rng.random() < 0.5
        nodes = _spread(rng, 2, 64)
        requests = _spread(rng, 1, max(1, min(128, 60_000_000 // (vocab * nodes))))
        return {"op": op, "requests": requests, "nodes": nodes, "chain": rng.random() < 0.4, "vocab": vocab, "certain": certain}
    kv_heads, d = rng.choice([(8, 128), (4, 128), (1, 128), (2, 64), (16, 64), (8, 64), (3, 128)])
    kind = {"kv_heads": kv_heads, "head": d, "block_tokens": rng.choice([16, 32, 64, 128]),
            "codes": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "compact":
        requests, nodes = _spread(rng, 1, 500), _spread(rng, 1, 128)
        return {"op": op, "requests": requests, "nodes": nodes,
                "context": _spread(rng, nodes, max(nodes, min(20000, 500_000_000 // (kv_heads * d * requests)))), **kind}
    heads = kv_heads * rng.choice([1, 2, 4, 4, 5, 8])
    nodes = _spread(rng, 1, 80)
    requests = _spread(rng, 1, 64)
    # the plain form's scores and values stay below a few GB
    most = min(65536, 300_000_000 // (kv_heads * d * requests), 600_000_000 // (heads * nodes * requests))
    return {"op": op, "requests": requests, "nodes": nodes, "ragged": rng.random() < 0.7,
            "context": _spread(rng, nodes, max(nodes, most)), "heads": heads, **kind,
            "window": rng.choice([0, 0, 0, 200, 3000]), "type": rng.choice(["bf16", "bf16", "f16"]), "pad": rng.choice([0, 0, 2])}


def _host(case):
    """A generator for the case's lengths, the same for every seed, so that shapes are."""
    return np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()) % (1 << 31))


def _parents(r, n, chain):
    """Parents of n nodes, level by level as a drafter makes them; -1 is the root's."""
    i = np.arange(n)
    if chain:
        return i - 1
    low, high = (i - 1) // 3, np.maximum((2 * i) // 3, (i - 1) // 3 + 1)
    return np.where(i == 0, -1, np.minimum(low + (r.rand(n) * (high - low)).astype(np.int64), i - 1))


def _batch(case):
    """Nodes and lengths (the nodes among them) of the case's requests, and behind them the empty places of a captured batch."""
    r, n = _host(case), case["requests"]
    nodes, length = np.full(n, case["nodes"]), np.full(n, max(case["context"], case["nodes"]))
    if case.get("ragged"):
        nodes = r.randint(max(1, case["nodes"] // 2), case["nodes"] + 1, n)
        length = np.maximum(r.randint(max(1, case["context"] // 4), case["context"] + 1, n), nodes)
        nodes[0], length[0] = case["nodes"], max(case["context"], case["nodes"])
    return nodes, length


def _blocks(n, p):
    return -(-n // p)


# ------------------------------------------------------------------ inputs
def _cuda(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _starts(nodes):
    return np.concatenate([[0], np.cumsum(nodes)])


def _scale(amax, largest):
    """2^k with the smallest k in [-48, 48] such that largest * 2^k >= amax; 1 where amax is 0."""
    m, e = torch.frexp(amax / largest)
    k = (e - (m == 0.5).to(e.dtype)).clamp(-48, 48)
    return torch.where(amax > 0, ((k.int() + 127) << 23).view(torch.float32), 1.0)


def _cache(gen, blocks, case, spread):
    """A cache that is in use: codes [blocks][kv heads][block tokens][head] and scales [blocks][kv heads]; a few
    channels are large, blocks are of unlike size."""
    codes, scale = [], []
    for at in range(0, blocks, 4096):
        n = min(4096, blocks - at)
        x = torch.randn((n, case["kv_heads"], case["block_tokens"], case["head"]), generator=gen, device="cuda")
        x *= 1 + 6 * (torch.rand(case["head"], generator=gen, device="cuda") < 0.03)
        x *= torch.exp(spread * torch.randn((n, case["kv_heads"], 1, 1), generator=gen, device="cuda"))
        s = _scale(x.abs().amax((2, 3)), LARGEST[case["codes"]])
        codes.append((x / s[:, :, None, None]).to(CODES[case["codes"]]).view(torch.uint8))
        scale.append(s)
    return torch.cat(codes), torch.cat(scale)


def _pages(r, state, case, gen, length):
    p = case["block_tokens"]
    held = _blocks(length, p)
    blocks = int(held.sum()) + 7
    order, at = r.permutation(blocks), _starts(held)
    tables = np.full((len(held), int(held.max()) + 1), -1, np.int32)
    for i, h in enumerate(held):
        tables[i, :h] = order[at[i]:at[i] + h]
    state["tables"] = _cuda(tables, torch.int32)
    state["k_codes"], state["k_scale"] = _cache(gen, blocks, case, 0.2)
    state["v_codes"], state["v_scale"] = _cache(gen, blocks, case, 0.7)


def _masks(nodes, parents, words):
    """Visibility of each node as int64 words: bits of itself and its ancestors; and its depth.  On the host."""
    bits, depth = np.zeros((len(parents), words), np.uint64), np.zeros(len(parents), np.int64)
    at = 0
    for n in nodes.tolist():
        for i in range(n):
            up = parents[at + i]
            if up >= 0:
                bits[at + i], depth[at + i] = bits[at + up], depth[at + up] + 1
            bits[at + i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
        at += n
    return bits.view(np.int64), depth


def _table(positions, rotate):
    """cos, then sin, of every position's angles, as a model keeps them: from angles in 64 bits."""
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(rotate // 2) * 2.0 / rotate)[None]
    return _cuda(np.concatenate([np.cos(angle), np.sin(angle)], 1), torch.float32)


def prepare(case, seed):
    r = np.random.RandomState((seed * 7 + 1) % (1 << 31))
    gen = torch.Generator("cuda").manual_seed(seed)
    state, op = {"case": case}, case["op"]
    if op in ("norm", "norm_grad"):
        t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["head"]
        kind = TYPES[case["type"]]
        weight = kind if case["weight"] == "same" else TYPES[case["weight"]]

        def heads(spread):  # of one projection, or of two
            x = torch.randn((t + case["pad"], h + g, d), generator=gen, device="cuda")
            x *= torch.exp(spread * torch.randn((t + case["pad"], h + g, 1), generator=gen, device="cuda"))
            x = x.to(kind)
            return (x[:, :h], x[:, h:]) if case["fused"] else (x[:, :h].contiguous(), x[:, h:].contiguous())
        state["q"], state["k"] = heads(0.7)
        state["q_weight"], state["k_weight"] = ((1 + 0.3 * torch.randn(d, generator=gen, device="cuda")).to(weight) for _ in range(2))
        position = r.randint(0, case["positions"], t)
        if t > case["positions"] // 2:  # prompts
            position = (r.randint(0, case["positions"]) + np.arange(t)) % case["positions"]
        state["positions"] = _cuda(np.concatenate([position, np.full(case["pad"], -1)]), torch.int32)
        state["table"] = _table(case["positions"], case["rotate"]) if case["rotate"] else None
        if op == "norm_grad":
            state["dq"], state["dk"] = heads(1.0)
        return state
    if op == "verify":
        n, m, v = case["requests"], case["nodes"], case["vocab"]
        parents = np.concatenate([_parents(r, m, case["chain"]) for _ in range(n)])
        # peaked distributions, as a model's; the draft model's are near them
        logits = 2.5 * torch.randn((n * m, v), generator=gen, device="cuda")
        state["target"] = torch.softmax(logits * 1.6, 1)
        if not case["certain"]:
            logits += 0.8 * torch.randn((n * m, v), generator=gen, device="cuda")
        draft = torch.softmax(logits * 1.6, 1)
        del logits
        # children of a node: its likeliest tokens in order, or tokens drawn from its draft distribution
        rank = np.zeros(n * m, np.int64)
        for i in range(n):
            p = parents[i * m:(i + 1) * m]
            for j in range(1, m):
                rank[i * m + j] = (p[:j] == p[j]).sum()
        most = int(rank.max()) + 1
        pick = draft.topk(most, 1).indices if case["certain"] else torch.multinomial(draft, most, replacement=True, generator=gen)
        at = np.maximum(parents, 0) + np.repeat(np.arange(n) * m, m)
        state["drafts"] = pick[_cuda(at, torch.int64), _cuda(rank, torch.int64)].int()
        state["draft"] = None if case["certain"] else draft
        state["parents"] = _cuda(parents, torch.int32)
        state["q_start"] = _cuda(np.arange(n + 1) * m, torch.int32)
        state["accept_random"] = torch.rand(n * m, generator=gen, device="cuda")
        state["sample_random"] = torch.rand(n, generator=gen, device="cuda")
        return state
    nodes, length = _batch(case)
    pad = case.get("pad", 0)
    state["most"] = int(nodes.max())
    state["most_k"] = int(length.max())
    parents = np.concatenate([_parents(r, int(n), False) for n in nodes])
    if op == "trees":
        state["parents"] = _cuda(np.concatenate([parents, np.full(pad, -1)]), torch.int32)
    elif op == "attention":
        bits, depth = _masks(nodes, parents, _blocks(state["most"], 64))
        state["positions"] = _cuda(np.concatenate([np.repeat(length - nodes, nodes) + depth, np.full(pad, -1)]), torch.int32)
        state["mask"] = _cuda(np.concatenate([bits, np.zeros((pad, bits.shape[1]), np.int64)]), torch.int64)
        state["q"] = (1.5 * torch.randn((int(nodes.sum()) + pad, case["heads"], case["head"]), generator=gen,
                                        device="cuda")).to(TYPES[case["type"]])
    else:
        # what verification gives: the way from the root to some node, and how many nodes it has
        path, counts, at = np.full(len(parents), -1), [], 0
        for n in nodes.tolist():
            way, i = [], int(r.randint(0, n))
            while i >= 0:
                way, i = [i] + way, int(parents[at + i])
            path[at:at + len(way)] = way
            counts.append(len(way))
            at += n
        state["path"], state["counts"] = _cuda(path, torch.int32), _cuda(np.array(counts), torch.int32)
        state["most_path"] = max(counts)
    if op != "trees":
        _pages(r, state, case, gen, length)
    state["lengths"], state["q_start"] = _cuda(length, torch.int32), _cuda(_starts(nodes), torch.int32)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    return globals()[("_own_" if own else "_plain_") + case["op"]](state, case)


def _own_trees(s, case):
    import block_scaled_precision_mx_gb300 as mx
    mask, positions = mx.kv_draft_trees(s["parents"], s["lengths"], s["q_start"], s["most"], window=case["window"])
    return {"mask": mask, "positions": positions}


def _own_norm(s, case):
    import block_scaled_precision_mx_gb300 as mx
    q, k = mx.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"], s["positions"], eps=EPS,
                           interleaved=case["interleaved"])
    return {"q": q[:case["tokens"]], "k": k[:case["tokens"]]}


def _own_norm_grad(s, case):
    import block_scaled_precision_mx_gb300 as mx
    dq, dk, dqw, dkw = mx.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"],
                                                s["positions"], eps=EPS, interleaved=case["interleaved"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _own_attention(s, case):
    import block_scaled_precision_mx_gb300 as mx
    out, lse = mx.kv_tree_attention(s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["tables"], s["lengths"],
                                    s["q_start"], s["most"], s["mask"], s["positions"],
                                    elem={"e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["codes"]], window=case["window"])
    return {"out": out, "lse": lse}


def _own_verify(s, case):
    import block_scaled_precision_mx_gb300 as mx
    path, tokens, counts = mx.kv_verify_drafts(s["target"], s["drafts"], s["parents"], s["q_start"], s["accept_random"],
                                               s["sample_random"], draft_probs=s["draft"])
    return {"path": path, "tokens": tokens, "counts": counts}


def _own_compact(s, case):
    import block_scaled_precision_mx_gb300 as mx
    # The operator works in place, and the same path on a cache that it has been through once is another task: the blocks
    # that a pass writes to are put back in front of the next one.
    names = ("k_codes", "v_codes", "k_scale", "v_scale")
    if "before" not in s:
        p, length = case["block_tokens"], s["lengths"].long()
        first = (length - s["q_start"].long().diff()) // p
        page = first[:, None] + torch.arange(_blocks(s["most_path"], p) + 1, device="cuda")[None]
        s["blocks"] = s["tables"].long().gather(1, torch.minimum(page, (length - 1)[:, None] // p)).reshape(-1)
        s["before"] = [s[name][s["blocks"]] for name in names]
    else:
        for name, was in zip(names, s["before"]):
            s[name].index_copy_(0, s["blocks"], was)
    kept = mx.kv_cache_compact(s["path"], s["counts"], s["lengths"], s["q_start"], s["tables"], s["k_codes"], s["v_codes"],
                               s["k_scale"], s["v_scale"], elem={"e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["codes"]])
    kind = CODES[case["codes"]]
    return {"lengths": kept, "k": s["k_codes"].view(kind), "k_scale": s["k_scale"], "v": s["v_codes"].view(kind),
            "v_scale": s["v_scale"]}


def _plain_trees(s, case):
    start, most, t = s["q_start"].long(), s["most"], s["parents"].numel()
    words = _blocks(most, 64)
    row = torch.arange(t, device="cuda")
    request = torch.searchsorted(start[1:], row, right=True)
    live = row < start[-1]
    first = start[request.clamp(max=len(start) - 2)]
    node, parent = row - first, s["parents"].long()
    mask = torch.zeros((t, words), dtype=torch.int64, device="cuda")
    depth = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    at, seen = torch.where(live, node, -1), torch.arange(words, device="cuda")[None]
    for step in range(most):  # a node further up each time
        on = at >= 0
        if not case["window"] or step < case["window"]:
            bit = torch.ones_like(at) << (at.clamp(min=0) % 64)
            mask += torch.where(on[:, None] & (seen == (at // 64)[:, None]), bit[:, None], 0)
        depth += on
        at = torch.where(on, parent[(first + at).clamp(0, t - 1)], -1)
    length = s["lengths"].long()[request.clamp(max=len(start) - 2)]
    base = length - (start[1:] - start[:-1])[request.clamp(max=len(start) - 2)]
    return {"mask": mask, "positions": torch.where(live, base + depth, -1).int()}


def _turn(x, table, positions, interleaved, back=False):
    """x [tokens][heads][head] with its first values turned by the positions' angles (or back)."""
    if table is None:
        return x
    n = table.shape[1]
    cos, sin = table.to(x.dtype)[positions].split(n // 2, 1)
    cos, sin = cos[:, None], (-sin if back else sin)[:, None]
    head, rest = x[..., :n], x[..., n:]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else head.split(n // 2, 2)
    u, v = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([u, v], 3).flatten(2) if interleaved else torch.cat([u, v], 2)
    return torch.cat([head, rest], 2)


def _plain_norm(s, case):
    out, t = {}, case["tokens"]
    for name in ("q", "k"):
        x = s[name][:t].float()
        y = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * s[name + "_weight"].float()
        out[name] = _turn(y, s["table"], s["positions"][:t].long(), case["interleaved"]).to(s[name].dtype)
    return out


def _plain_norm_grad(s, case):
    out, t = {}, case["tokens"]
    for name in ("q", "k"):
        x, w = s[name][:t].float(), s[name + "_weight"].float()
        g = _turn(s["d" + name][:t].float(), s["table"], s["positions"][:t].long(), case["interleaved"], back=True)
        r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
        y, gw = x * r, g * w
        dx = r * (gw - y * (gw * y).mean(2, keepdim=True))
        out["d" + name] = torch.cat([dx, dx.new_zeros((case["pad"],) + dx.shape[1:])]).to(s[name].dtype)
        out["d" + name + "_weight"] = (g * y).sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_attention(s, case):
    q, p, h, w = s["q"], case["block_tokens"], case["kv_heads"], case["window"]
    t, heads, d = q.shape
    n, lk, lq = s["lengths"].numel(), s["most_k"], s["most"]
    start, length = s["q_start"].long(), s["lengths"].long()
    query = start[1:] - start[:-1]
    key = torch.arange(lk, device="cuda")
    there = key[None] < length[:, None]
    block = torch.where(there, s["tables"].long()[:, key // p], 0)
    kind = CODES[case["codes"]]

    def gather(codes, scale):  # [n][kv heads][lk][head]
        x = codes[block, :, key % p].view(kind).float() * scale[block][..., None]
        return torch.where(there[:, :, None, None], x, 0.0).transpose(1, 2)

    row = torch.arange(lq, device="cuda")
    live = row[None] < query[:, None]
    token = (start[:-1, None] + row[None]).clamp(max=t - 1)
    qs = q.float()[token].reshape(n, lq, h, heads // h, d).permute(0, 2, 3, 1, 4).reshape(n, h, -1, d)
    score = (qs @ gather(s["k_codes"], s["k_scale"]).transpose(2, 3)).reshape(n, h, heads // h, lq, lk)
    score *= 1.0 / math.sqrt(d)
    # the context, within the window; of the nodes those whose bits are set
    node = key[None] - (length - query)[:, None]
    mask = s["mask"][token]
    bit = mask.gather(2, (node // 64).clamp(0, mask.shape[2] - 1)[:, None].expand(-1, lq, -1)) >> (node % 64)[:, None] & 1
    seen = torch.where(node[:, None] < 0, key[None, None] > s["positions"].long()[token][:, :, None] - w if w else True, bit == 1)
    score = score.masked_fill_(~(seen & there[:, None])[:, None, None], -math.inf)
    most = score.amax(4, keepdim=True)
    score -= torch.where(most > -math.inf, most, 0.0)
    weight = score.exp_()
    total = weight.sum(4)
    out = (weight.reshape(n, h, -1, lk) @ gather(s["v_codes"], s["v_scale"])).reshape(n, h, -1, lq, d)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = total.log() + most[..., 0]
    at = torch.where(live, token, t).reshape(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(-1, heads, d)
    lse = lse.permute(0, 3, 1, 2).reshape(-1, heads)
    out = out.new_zeros((t + 1, heads, d)).index_copy(0, at, out)[:t]
    lse = lse.new_full((t + 1, heads), -math.inf).index_copy(0, at, lse)[:t]
    return {"out": out.to(q.dtype), "lse": lse}


def _plain_verify(s, case):
    n, m, v = case["requests"], case["nodes"], case["vocab"]
    target, draft = s["target"].view(n, m, v), None if s["draft"] is None else s["draft"].view(n, m, v)
    drafts, parents = s["drafts"].long().view(n, m), s["parents"].long().view(n, m)
    random = s["accept_random"].double().view(n, m)
    each = torch.arange(n, device="cuda")
    node = torch.zeros(n, dtype=torch.int64, device="cuda")      # the last one accepted
    count = torch.ones(n, dtype=torch.int64, device="cuda")
    path = torch.full((n, m + 1), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    left = torch.ones(n, dtype=torch.float64, device="cuda")     # what the rejected children leave of its probabilities
    taken = torch.zeros(n, dtype=torch.float64, device="cuda")   # how often the draft's have been taken off them

    def rest():
        return (target[each, node].double() - taken[:, None] * draft[each, node]).clamp_(min=0)
    for i in range(1, m):
        child, token = parents[:, i] == node, drafts[:, i]
        p = target[each, node, token].double()
        if draft is None:
            p = torch.where(((parents[:, 1:i] == node[:, None]) & (drafts[:, 1:i] == token[:, None])).any(1), 0.0, p)
            yes = child & (random[:, i] * left < p)
            left = torch.where(child & ~yes, left - p, left)
        else:
            q = draft[each, node, token].double()
            yes = child & (random[:, i] * q * left < (p - taken * q).clamp(min=0))
            no = child & ~yes
            taken = torch.where(no, taken + left, taken)
            left = torch.where(no, rest().sum(1), left)
        path.scatter_(1, torch.where(yes, count, m)[:, None], i)
        path[:, m] = -1
        count += yes
        node, left, taken = torch.where(yes, i, node), torch.where(yes, 1.0, left), torch.where(yes, 0.0, taken)
    if draft is None:  # every child of the last node has been rejected
        last = torch.cat([target[each, node].double(), torch.zeros((n, 1), dtype=torch.float64, device="cuda")], 1)
        last = last.scatter(1, torch.where(parents[:, 1:] == node[:, None], drafts[:, 1:], v), 0.0)[:, :v]
    else:
        last = rest()
    last = torch.where(last.sum(1, keepdim=True) > 0, last, target[each, node].double())
    upto = last.cumsum(1)
    next_token = (upto <= s["sample_random"].double()[:, None] * upto[:, -1:]).sum(1).clamp(max=v - 1)
    at = torch.arange(m, device="cuda")[None]
    path = path[:, :m]
    following = drafts.gather(1, torch.cat([path[:, 1:], path[:, :1]], 1).clamp(min=0))
    tokens = torch.where(at < count[:, None] - 1, following, torch.where(at == count[:, None] - 1, next_token[:, None], -1))
    return {"path": path.reshape(-1).int(), "tokens": tokens.reshape(-1).int(), "counts": count.int()}


def _plain_compact(s, case):
    p, kind, largest = case["block_tokens"], CODES[case["codes"]], LARGEST[case["codes"]]
    start, length, counts = s["q_start"].long(), s["lengths"].long(), s["counts"].long()
    context = length - start[1:] + start[:-1]
    i = torch.arange(s["most_path"], device="cuda")[None]
    node = s["path"].long()[(start[:-1, None] + i).clamp(max=s["path"].numel() - 1)]
    request, step = torch.nonzero((i < counts[:, None]) & (node != i), as_tuple=True)  # the nodes that move
    source, to = (context[:, None] + node)[request, step], (context[:, None] + i)[request, step]
    tables = s["tables"].long()
    from_block, to_block = tables[request, source // p], tables[request, to // p]
    out = {"lengths": (context + counts).int()}
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        x = codes[from_block, :, source % p].view(kind).float() * scale[from_block][..., None]
        # a block keeps its scale or grows it, and the codes in front of what moves into it follow
        amax = torch.zeros_like(scale).index_reduce(0, to_block, x.abs().amax(2), "amax")
        first = torch.full((codes.shape[0],), 0, device="cuda").index_reduce(0, to_block, to % p, "amin", include_self=False)
        grown = torch.where(amax > 0, torch.maximum(scale, _scale(amax, largest)), scale)
        front = torch.arange(p, device="cuda")[None] < first[:, None]
        values = codes.view(kind).float()
        values = torch.where(front[:, None, :, None], values * (scale / grown)[:, :, None, None], values)
        values[to_block, :, to % p] = (x / grown[to_block][..., None]).clamp(-largest, largest)
        out[name], out[name + "_scale"] = values.to(kind), grown
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        size = TYPES[case["type"]].itemsize
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head"]
        rows = min(case["tokens"], case["positions"])
        return {"bytes": values * size * (2 if op == "norm" else 3) + 4 * rows * case["rotate"] + 4 * case["tokens"]
                + 4 * 2 * case["head"] * (1 if op == "norm" else 2), "flops": 0}
    if op == "verify":
        n, m = case["requests"], case["nodes"]
        # the last node's probabilities of each request; parents, drafts, random numbers, two probabilities, path and tokens of each node
        return {"bytes": n * case["vocab"] * (4 if case["certain"] else 8) + n * m * 28, "flops": 0}
    nodes, length = _batch(case)
    words = _blocks(int(nodes.max()), 64)
    if op == "trees":
        return {"bytes": int(nodes.sum() + case["pad"]) * (8 + 8 * words) + 8 * len(nodes), "flops": 0}
    row, p = case["kv_heads"] * case["head"], case["block_tokens"]
    if op == "compact":
        # a path has about as many nodes as the tree is deep; most of them move, codes read and written
        depth = int(np.log2(np.maximum(nodes, 1)).sum())
        return {"bytes": 2 * 2 * depth * row + 8 * depth + 16 * len(nodes), "flops": 0}
    w, pairs, keys = case["window"], 0, 0
    for n, m in zip(length.tolist(), nodes.tolist()):
        context = n - m
        pairs += m * ((min(context, w) if w else context) + max(1, int(math.log2(m))))
        keys += (min(context, w) if w else context) + m
    tokens = int(nodes.sum())
    return {"bytes": 2 * keys * row + 8 * keys // p * case["kv_heads"] + tokens * (case["heads"] * (4 * case["head"] + 4) + 8 * words),
            "flops": 4 * pairs * case["heads"] * case["head"]}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_turn(x, table, positions, interleaved, sign):
    x = x.clone()
    if table is None:
        return x
    half = table.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = table[positions, i].double()[:, None], sign * table[positions, half + i].double()[:, None]
        x[..., a], x[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return x


def _exact_norm(s, case):
    t, out = case["tokens"], {}
    at = s["positions"][:t].long()
    for name in ("q", "k"):
        x, w = s[name][:t].double(), s[name + "_weight"].double()
        length = (x.pow(2).sum(2, keepdim=True) / case["head"] + EPS).sqrt()
        if case["op"] == "norm":
            out[name] = _exact_turn(x / length * w, s["table"], at, case["interleaved"], 1.0)
            continue
        g = _exact_turn(s["d" + name][:t].double(), s["table"], at, case["interleaved"], -1.0)
        gw = g * w
        dx = gw / length - x * (gw * x).sum(2, keepdim=True) / (case["head"] * length.pow(3))
        out["d" + name] = torch.cat([dx, dx.new_zeros((case["pad"],) + dx.shape[1:])])
        out["d" + name + "_weight"] = (g * x / length).sum((0, 1))
    return out


def _exact_attention(s, case):
    t, heads, d = s["q"].shape
    group, p, w = heads // case["kv_heads"], case["block_tokens"], case["window"]
    out = torch.zeros((t, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((t, heads), -math.inf, dtype=torch.float64, device="cuda")
    start, kind = s["q_start"].tolist(), CODES[case["codes"]]
    masks = s["mask"].cpu().numpy().view(np.uint64)
    for i, n in enumerate(s["lengths"].tolist()):
        a, b = start[i], start[i + 1]
        blocks = s["tables"][i, :_blocks(n, p)].long()
        context = n - (b - a)
        seen = np.ones((b - a, n), bool)
        for j in range(b - a):
            seen[:, context + j] = masks[a:b, j // 64] >> np.uint64(j % 64) & np.uint64(1) == 1
        seen = torch.from_numpy(seen).cuda()
        if w:
            j = torch.arange(n, device="cuda")
            seen &= (j[None] >= context) | (j[None] > s["positions"][a:b].long()[:, None] - w)
        for g in range(case["kv_heads"]):
            k = (s["k_codes"][blocks, g].view(kind).double() * s["k_scale"][blocks, g].double()[:, None, None]).reshape(-1, d)[:n]
            v = (s["v_codes"][blocks, g].view(kind).double() * s["v_scale"][blocks, g].double()[:, None, None]).reshape(-1, d)[:n]
            z = torch.einsum("thd,ld->thl", s["q"][a:b, g * group:(g + 1) * group].double(), k) / math.sqrt(d)
            z.masked_fill_(~seen[:, None], -math.inf)
            total = torch.logsumexp(z, 2)
            lse[a:b, g * group:(g + 1) * group] = total
            out[a:b, g * group:(g + 1) * group] = torch.einsum("thl,ld->thd", torch.exp(z - total[:, :, None]), v)
    return {"out": out, "lse": lse}


def _power64(k):
    """2^k in 64 bits, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _code64(x, codes):
    """The nearest value of the 8-bit type (ties to even, the largest where x is beyond it), in 64 bits."""
    mantissa, lowest = {"e4m3": (3, -6), "e5m2": (2, -14)}[codes]
    _, e = torch.frexp(x)
    step = _power64((e - 1).clamp(min=lowest) - mantissa)
    return (torch.round(x / step) * step).clamp(-LARGEST[codes], LARGEST[codes])


def _exact_compact(s, case):
    p, largest, out = case["block_tokens"], LARGEST[case["codes"]], {"lengths": None}
    start, length, counts = s["q_start"].tolist(), s["lengths"].tolist(), s["counts"].tolist()
    path, tables = s["path"].tolist(), s["tables"].tolist()
    runs = []  # (block, its first offset, blocks and offsets that its new tokens come from)
    for r in range(len(length)):
        context, at = length[r] - (start[r + 1] - start[r]), None
        for i in range(counts[r]):
            node = path[start[r] + i]
            if node == i:
                continue
            block, offset = divmod(context + i, p)
            if at != block:
                runs.append((tables[r][block], offset, [], []))
                at = block
            runs[-1][2].append(tables[r][(context + node) // p])
            runs[-1][3].append((context + node) % p)
    if len(runs) > 8000:
        return None
    for name in ("k", "v"):
        old, old_scale = s[name + "_codes"].view(CODES[case["codes"]]).double(), s[name + "_scale"].double()
        value, scale = old.clone(), old_scale.clone()
        for block, offset, from_block, from_offset in runs:
            x = old[from_block, :, from_offset] * old_scale[from_block][:, :, None]
            amax = x.abs().amax((0, 2))
            k = torch.ceil(torch.log2(amax.clamp(min=1e-300) / largest)).clamp(-48, 48)
            k = torch.where(largest * _power64(k - 1) >= amax, k - 1, k).clamp(-48, 48)
            k = torch.where((largest * _power64(k) < amax) & (k < 48), k + 1, k)
            new = torch.where(amax > 0, torch.maximum(_power64(k), old_scale[block]), old_scale[block])
            value[block, :, :offset] = _code64(old[block, :, :offset] * (old_scale[block] / new)[:, None, None], case["codes"])
            value[block, :, offset:offset + len(x)] = _code64(x / new[None, :, None], case["codes"]).transpose(0, 1)
            scale[block] = new
        out[name], out[name + "_scale"] = value, scale
    return out


def exact(case, seed):
    if case["op"] in ("trees", "verify"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s, case)
    return _exact_compact(s, case) if case["op"] == "compact" else _exact_norm(s, case)
