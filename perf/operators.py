"""Cases of the 8-bit key/value cache operators: what a serving step does around the model's products.

A step gives every request its cache blocks and its new tokens' places (`tables`), writes the new
keys and values into the cache as 8-bit codes with one power-of-two scale for each block of tokens
and head (`append`), and lets the step's queries attend over the cache (`attention`).

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
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token for each of 64 running requests: the smallest table update, all latency
        {"name": "tables_decode_64", "op": "tables", "requests": 64, "block_tokens": 64, "longest": 8192,
         "mixed": False, "chunk": 1, "pad": 0},
        # a large server's step: requests that start, go on, are rewound and finish, blocks of 16
        {"name": "tables_mixed_2000", "op": "tables", "requests": 2000, "block_tokens": 16, "longest": 32768,
         "mixed": True, "chunk": 1024, "pad": 37},
        # one token a request into partly filled blocks
        {"name": "append_decode_64", "op": "append", "requests": 64, "tokens": 1, "kv_heads": 8, "head": 128,
         "block_tokens": 64, "type": "bf16", "codes": "e4m3", "fused": True},
        # chunks of prompts, ragged, ending and starting inside blocks
        {"name": "append_prefill_8k", "op": "append", "requests": 7, "tokens": 1300, "kv_heads": 8, "head": 128,
         "block_tokens": 64, "type": "bf16", "codes": "e4m3", "fused": True},
        # many prompts of short heads in the other 16-bit and the other 8-bit type, blocks of 16
        {"name": "append_prefill_64k_f16", "op": "append", "requests": 33, "tokens": 2500, "kv_heads": 16, "head": 64,
         "block_tokens": 16, "type": "f16", "codes": "e5m2", "fused": False},
        # one request's next token over a short context: latency
        {"name": "decode_1x777", "op": "attention", "requests": 1, "tokens": 1, "context": 777, "ragged": False,
         "heads": 32, "kv_heads": 8, "head": 128, "block_tokens": 64, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 0},
        # a full batch's next tokens over ragged contexts, with places of a captured batch left empty
        {"name": "decode_64x4k", "op": "attention", "requests": 64, "tokens": 1, "context": 4096, "ragged": True,
         "heads": 32, "kv_heads": 8, "head": 128, "block_tokens": 64, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 3},
        # few requests with long contexts
        {"name": "decode_8x64k", "op": "attention", "requests": 8, "tokens": 1, "context": 65536, "ragged": True,
         "heads": 64, "kv_heads": 8, "head": 128, "block_tokens": 128, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 0},
        # a key/value head for every query head, short heads, blocks of 16, the other types
        {"name": "decode_33x3000_f16", "op": "attention", "requests": 33, "tokens": 1, "context": 3000, "ragged": True,
         "heads": 16, "kv_heads": 16, "head": 64, "block_tokens": 16, "window": 0, "type": "f16", "codes": "e5m2", "pad": 0},
        # four drafted tokens a request to be judged at once, within a window
        {"name": "draft_24x4_window", "op": "attention", "requests": 24, "tokens": 4, "context": 6000, "ragged": True,
         "heads": 64, "kv_heads": 8, "head": 128, "block_tokens": 64, "window": 2048, "type": "bf16", "codes": "e4m3", "pad": 0},
        # ragged prompts, some behind a cached prefix
        {"name": "prefill_6x1500", "op": "attention", "requests": 6, "tokens": 1500, "context": 2100, "ragged": True,
         "heads": 32, "kv_heads": 8, "head": 128, "block_tokens": 16, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 0},
        # a long prompt's last chunk
        {"name": "prefill_4096_of_32k", "op": "attention", "requests": 1, "tokens": 4096, "context": 32768, "ragged": False,
         "heads": 32, "kv_heads": 8, "head": 128, "block_tokens": 64, "window": 0, "type": "bf16", "codes": "e4m3", "pad": 0},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over the logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    n = min(high, max(low, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["tables", "append", "append", "attention", "attention", "attention", "attention"])
    if op == "tables":
        mixed = rng.random() < 0.6
        return {"op": op, "requests": _spread(rng, 1, 2000), "block_tokens": rng.choice([16, 32, 64, 128]),
                "longest": _spread(rng, 1, 32768), "mixed": mixed, "chunk": _spread(rng, 1, 1024) if mixed else 1,
                "pad": rng.choice([0, 0, 1, 40])}
    heads = rng.choice([(8, 128), (4, 128), (1, 128), (2, 64), (16, 64), (8, 64), (3, 128)])
    kind = {"kv_heads": heads[0], "head": heads[1], "block_tokens": rng.choice([16, 32, 64, 128]),
            "type": rng.choice(["bf16", "bf16", "f16"]), "codes": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "append":
        requests = _spread(rng, 1, 256)
        tokens = 1 if rng.random() < 0.4 else _spread(rng, 2, max(2, min(4096, 60000 // requests)))
        return {"op": op, "requests": requests, "tokens": tokens, **kind, "fused": rng.random() < 0.5}
    group = rng.choice([1, 2, 4, 4, 5, 8])
    heads = kind["kv_heads"] * group
    if heads * kind["head"] == 3072:
        group, heads = 1, kind["kv_heads"]
    row = kind["kv_heads"] * kind["head"]
    how = rng.random()
    if how < 0.6:  # single tokens and drafts
        tokens = 1 if how < 0.4 else rng.randint(2, 9)
        requests = _spread(rng, 1, 128)
        context = _spread(rng, tokens, max(tokens, min(65536, 500_000_000 // (row * requests))))
    else:
        tokens = _spread(rng, 16, 4096)
        requests = rng.randint(1, 8) if tokens < 1000 else rng.randint(1, 3)
        most = 4_000_000_000 // (heads * requests * tokens)
        context = _spread(rng, tokens, max(tokens, min(32768, most)))
    return {"op": op, "requests": requests, "tokens": tokens, "context": context, "ragged": rng.random() < 0.7,
            "heads": heads, **kind, "window": rng.choice([0, 0, 0, 128, 1000]), "pad": rng.choice([0, 0, 2])}


def _lengths(case):
    """The case's lengths, on the host: a dict of numpy arrays, the same ones for every seed, so that shapes are."""
    r = np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()) % (1 << 31))
    n = case["requests"]
    if case["op"] == "tables":
        longest = case["longest"]
        before = r.randint(1, longest + 1, n)
        after = before + 1
        if case["mixed"]:
            what = r.rand(n)
            # a tenth start, a tenth read a prompt's next chunk, a tenth finish, a tenth are rewound
            chunk = r.randint(1, case["chunk"] + 1, n)
            before = np.where(what < 0.1, 0, before)
            after = np.where(what < 0.2, before + chunk, before + 1)
            after = np.where((what >= 0.2) & (what < 0.3), 0, after)
            after = np.where((what >= 0.3) & (what < 0.4), np.maximum(before - r.randint(0, 9, n), 0), after)
        return {"before": before, "after": after}
    if case["op"] == "append":
        t = case["tokens"]
        new = np.full(n, 1) if t == 1 else r.randint(max(1, t // 2), t + 1, n)
        before = r.randint(0, 4 * case["block_tokens"], n)
        before = np.where(r.rand(n) < (0.05 if t == 1 else 0.6), 0, before)  # prompts mostly start fresh
        return {"before": before, "after": before + new}
    t, c = case["tokens"], case["context"]
    length, query = np.full(n, c), np.full(n, t)
    if case["ragged"]:
        length = r.randint(max(t, c // 4), c + 1, n)
        if t > 16:
            query = r.randint(max(1, t // 4), t + 1, n)
        length[0], query[0] = c, t
    # places of a captured batch that no request has: one query token each, nothing to attend to
    length, query = (np.concatenate([x, np.full(case["pad"], v)]) for x, v in ((length, 0), (query, 1)))
    return {"before": length - query, "after": length, "query": query}


def _blocks(n, p):
    return -(-n // p)


# ------------------------------------------------------------------ inputs
def _tables(r, held, width, blocks):
    """Block tables [requests][width]: distinct blocks in no order for what each request holds, -1 elsewhere; and the rest."""
    order = r.permutation(blocks)
    tables = np.full((len(held), width), -1, np.int32)
    at = np.concatenate([[0], np.cumsum(held)])
    for i, h in enumerate(held):
        tables[i, :h] = order[at[i]:at[i] + h]
    return tables, order[at[-1]:].astype(np.int32)


def _values(gen, shape, spread):
    """Values as keys and values have them: normal, a few channels large, blocks of unlike size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    channel = 1 + 6 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.03)
    x *= channel
    x *= torch.exp(spread * torch.randn(shape[:2] + (1,) * (len(shape) - 2), generator=gen, device="cuda"))
    return x


def _scale(amax, largest):
    """2^k with the smallest k in [-48, 48] such that largest * 2^k >= amax; 1 where amax is 0."""
    m, e = torch.frexp(amax / largest)
    k = (e - (m == 0.5).to(e.dtype)).clamp(-48, 48)
    return torch.where(amax > 0, ((k.int() + 127) << 23).view(torch.float32), 1.0)


def _cache(gen, blocks, case, spread):
    """A cache that is in use: codes [blocks][kv heads][block tokens][head] and scales [blocks][kv heads]."""
    codes, scale = [], []
    for at in range(0, blocks, 4096):
        n = min(4096, blocks - at)
        x = _values(gen, (n, case["kv_heads"], case["block_tokens"], case["head"]), spread)
        s = _scale(x.abs().amax((2, 3)), LARGEST[case["codes"]])
        codes.append((x / s[:, :, None, None]).to(CODES[case["codes"]]).view(torch.uint8))
        scale.append(s)
    return torch.cat(codes), torch.cat(scale)


def _cuda(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def prepare(case, seed):
    length = _lengths(case)
    r = np.random.RandomState((seed * 7 + 1) % (1 << 31))
    gen = torch.Generator("cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "tables":
        p = case["block_tokens"]
        held, want = _blocks(length["before"], p), _blocks(length["after"], p)
        width = int(max(held.max(), want.max())) + 2
        blocks = int(np.maximum(held, want).sum()) + 100
        tables, spare = _tables(r, held, width, blocks)
        free = np.full(blocks, -1, np.int32)
        free[:len(spare)] = spare
        state |= {"tables": _cuda(tables, torch.int32), "before": _cuda(length["before"], torch.int32),
                  "after": _cuda(length["after"], torch.int32), "free": _cuda(free, torch.int32),
                  "free_count": torch.tensor([len(spare)], dtype=torch.int32, device="cuda"),
                  "tokens": int(np.maximum(length["after"] - length["before"], 0).sum()) + case["pad"]}
        return state
    p, d, h = case["block_tokens"], case["head"], case["kv_heads"]
    held = _blocks(length["after"], p)
    blocks = int(held.sum()) + 7
    tables, _ = _tables(r, held, int(held.max()) + 1, blocks)
    state["k_codes"], state["k_scale"] = _cache(gen, blocks, case, 0.2)
    state["v_codes"], state["v_scale"] = _cache(gen, blocks, case, 0.7)
    if case["op"] == "append":
        new = length["after"] - length["before"]
        first = np.concatenate([[0], np.cumsum(new)])[:-1]
        request = np.repeat(np.arange(len(new)), new)
        position = np.arange(int(new.sum())) - first[request] + length["before"][request]
        state["slots"] = _cuda(tables[request, position // p].astype(np.int64) * p + position % p, torch.int64)
        t = len(position)
        kv = _values(gen, (t, 2 * h, d), 0.3).clamp(-60000, 60000).to(TYPES[case["type"]])
        if not case["fused"]:  # keys and values of a product of their own each
            kv = torch.stack([kv[:, :h], kv[:, h:]])
            state["k"], state["v"] = kv[0], kv[1]
        else:  # slices of one product's result
            state["k"], state["v"] = kv[:, :h], kv[:, h:]
        return state
    query = length["query"]
    state["q"] = (1.5 * torch.randn((int(query.sum()), case["heads"], d), generator=gen, device="cuda")).to(TYPES[case["type"]])
    state["tables"] = _cuda(tables, torch.int32)
    state["lengths"] = _cuda(length["after"], torch.int32)
    state["q_start"] = _cuda(np.concatenate([[0], np.cumsum(query)]), torch.int32)
    state["most_q"], state["most_k"] = int(query.max()), int(length["after"].max())
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attention": _own_attention}[case["op"]](state, case)
    return {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention}[case["op"]](state, case)


def _own_tables(s, case):
    import block_scaled_precision_mx_gb300 as mx
    q_start, slots, positions, info = mx.kv_block_tables(
        s["tables"], s["before"], s["after"], s["free"], s["free_count"], s["tokens"], case["block_tokens"])
    return {"tables": s["tables"], "free": s["free"], "q_start": q_start, "slots": slots, "positions": positions, "info": info}


def _own_append(s, case):
    import block_scaled_precision_mx_gb300 as mx
    mx.kv_cache_append(s["k"], s["v"], s["slots"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                       elem={"e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["codes"]])
    kind = CODES[case["codes"]]
    return {"k": s["k_codes"].view(kind), "k_scale": s["k_scale"], "v": s["v_codes"].view(kind), "v_scale": s["v_scale"]}


def _own_attention(s, case):
    import block_scaled_precision_mx_gb300 as mx
    out, lse = mx.kv_attention(s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["tables"], s["lengths"],
                               s["q_start"], s["most_q"], elem={"e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["codes"]],
                               causal=True, window=case["window"])
    return {"out": out, "lse": lse}


def _plain_tables(s, case):
    p, tables, free = case["block_tokens"], s["tables"].long(), s["free"].long()
    before, after, count = s["before"].long(), s["after"].long(), s["free_count"].long()
    held, want, new = (before + p - 1) // p, (after + p - 1) // p, (after - before).clamp(min=0)
    need, gone = (want - held).clamp(min=0), (held - want).clamp(min=0)
    need_at, gone_at = need.cumsum(0) - need, gone.cumsum(0) - gone
    q_start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    left = count + gone.sum() - need.sum()
    column = torch.arange(tables.shape[1], device="cuda")[None]
    # the released blocks on top of the free ones, then the wanted ones off the top
    out = (column >= want[:, None]) & (column < held[:, None])
    place = torch.where(out, count + gone_at[:, None] + column - want[:, None], free.numel())
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, place.reshape(-1), tables.reshape(-1))[:-1]
    into = (column >= held[:, None]) & (column < want[:, None])
    place = count + gone.sum() - 1 - need_at[:, None] - column + held[:, None]
    fits = left >= 0
    tables = torch.where(into & fits, stack[place.clamp(0, free.numel() - 1)], tables)
    kept = torch.arange(free.numel(), device="cuda") < left
    free = torch.where(kept & fits, stack, free)
    token = torch.arange(s["tokens"], device="cuda")
    request = torch.searchsorted(q_start[1:], token, right=True).clamp(max=len(before) - 1)
    position = before[request] + token - q_start[request]
    slot = tables[request, (position // p).clamp(0, tables.shape[1] - 1)] * p + position % p
    used = (token < q_start[-1]) & fits
    info = torch.cat([torch.where(fits, left, count), (-left).clamp(min=0)])
    return {"tables": tables.int(), "free": free.int(), "q_start": q_start.int(), "slots": torch.where(used, slot, -1),
            "positions": torch.where(used, position, -1).int(), "info": info.int()}


def _plain_append_one(x, slots, codes, scale, kind, largest):
    p = codes.shape[2]
    block, offset, x = slots // p, slots % p, x.float()
    amax = torch.zeros_like(scale).index_reduce(0, block, x.abs().amax(2), "amax")
    first = torch.full((codes.shape[0],), p, device="cuda").index_reduce(0, block, offset, "amin")
    # a block that had tokens keeps its scale or grows it, and its codes follow
    kept, fresh = (first > 0) & (first < p), first == 0
    of_new = _scale(amax, largest)
    grown = torch.where(kept[:, None] & (amax > 0), torch.maximum(scale, of_new), torch.where(fresh[:, None], of_new, scale))
    old = torch.arange(p, device="cuda")[None] < torch.where(kept, first, 0)[:, None]
    again = codes.view(kind).float() * (scale / grown)[:, :, None, None]
    values = torch.where(old[:, None, :, None], again, codes.view(kind).float())
    values[block, :, offset] = (x / grown[block][:, :, None]).clamp(-largest, largest)
    return values.to(kind), grown


def _plain_append(s, case):
    kind, largest = CODES[case["codes"]], LARGEST[case["codes"]]
    k, k_scale = _plain_append_one(s["k"], s["slots"], s["k_codes"], s["k_scale"], kind, largest)
    v, v_scale = _plain_append_one(s["v"], s["slots"], s["v_codes"], s["v_scale"], kind, largest)
    return {"k": k, "k_scale": k_scale, "v": v, "v_scale": v_scale}


def _plain_attention(s, case):
    q, p, h = s["q"], case["block_tokens"], case["kv_heads"]
    t, heads, d = q.shape
    n, lk, lq = s["lengths"].numel(), max(1, s["most_k"]), s["most_q"]
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
    position = (length - query)[:, None] + row[None]
    seen = there[:, None, :] & (key[None, None] <= position[:, :, None])
    if case["window"]:
        seen &= key[None, None] > position[:, :, None] - case["window"]
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    most = score.amax(4, keepdim=True)
    score -= torch.where(most > -math.inf, most, 0.0)
    weight = score.exp_()
    total = weight.sum(4)
    out = (weight.reshape(n, h, -1, lk) @ gather(s["v_codes"], s["v_scale"])).reshape(n, h, -1, lq, d)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = total.log() + most[..., 0]
    # back to one row for each token
    at = torch.where(live, token, t).reshape(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(-1, heads, d)
    lse = lse.permute(0, 3, 1, 2).reshape(-1, heads)
    out = out.new_zeros((t + 1, heads, d)).index_copy(0, at, out)[:t]
    lse = lse.new_zeros((t + 1, heads)).index_copy(0, at, lse)[:t]
    return {"out": out.to(q.dtype), "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    length = _lengths(case)
    before, after = length["before"], length["after"]
    p = case["block_tokens"]
    if case["op"] == "tables":
        new = int(np.maximum(after - before, 0).sum())
        moved = int(np.abs(_blocks(after, p) - _blocks(before, p)).sum())
        # lengths in, starts out, moved blocks in and out, a slot and a position for each token
        return {"bytes": 12 * len(before) + 8 * moved + 12 * (new + case["pad"]), "flops": 0}
    row = case["kv_heads"] * case["head"]
    if case["op"] == "append":
        new = int((after - before).sum())
        touched = int((_blocks(after, p) - before // p).sum())
        return {"bytes": 2 * new * row * (2 + 1) + 8 * new + 2 * 8 * touched * case["kv_heads"], "flops": 0}
    query, w = length["query"], case["window"]
    pairs = keys = 0
    for n, m in zip(after.tolist(), query.tolist()):
        if not n:
            continue
        seen = np.arange(n - m + 1, n + 1)
        pairs += int((np.minimum(seen, w) if w else seen).sum())
        keys += min(n, w + m - 1) if w else n
    tokens = int(query.sum())
    return {"bytes": 2 * keys * row + 8 * keys // p * case["kv_heads"] + tokens * case["heads"] * (4 * case["head"] + 4),
            "flops": 4 * pairs * case["heads"] * case["head"]}


# ------------------------------------------------------------------ the definition, in 64 bits
def _power64(k):
    """2^k in 64 bits, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _code64(x, codes):
    """The nearest value of the 8-bit type (ties to even, the largest where x is beyond it), in 64 bits."""
    mantissa, lowest = {"e4m3": (3, -6), "e5m2": (2, -14)}[codes]
    _, e = torch.frexp(x)
    step = _power64((e - 1).clamp(min=lowest) - mantissa)
    return (torch.round(x / step) * step).clamp(-LARGEST[codes], LARGEST[codes])


def _exact_append_one(x, slots, codes, scale, case):
    p, largest = case["block_tokens"], LARGEST[case["codes"]]
    value, scale, x = codes.view(CODES[case["codes"]]).double(), scale.double(), x.double()
    block = (slots // p).tolist()
    edges = [i for i in range(len(block)) if i == 0 or block[i] != block[i - 1]] + [len(block)]
    for a, b in zip(edges, edges[1:]):
        first, to = int(slots[a]) % p, block[a]
        amax = x[a:b].abs().amax((0, 2))
        k = torch.ceil(torch.log2(amax.clamp(min=1e-300) / largest)).clamp(-48, 48)
        k = torch.where(largest * _power64(k - 1) >= amax, k - 1, k).clamp(-48, 48)
        k = torch.where((largest * _power64(k) < amax) & (k < 48), k + 1, k)
        new = torch.where(amax > 0, _power64(k), 1.0)
        if first:
            new = torch.where(amax > 0, torch.maximum(new, scale[to]), scale[to])
            value[to, :, :first] = _code64(value[to, :, :first] * (scale[to] / new)[:, None, None], case["codes"])
        scale[to] = new
        value[to, :, first:first + b - a] = _code64(x[a:b] / new[None, :, None], case["codes"]).transpose(0, 1)
    return value, scale


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        k, k_scale = _exact_append_one(s["k"], s["slots"], s["k_codes"], s["k_scale"], case)
        v, v_scale = _exact_append_one(s["v"], s["slots"], s["v_codes"], s["v_scale"], case)
        return {"k": k, "k_scale": k_scale, "v": v, "v_scale": v_scale}
    t, heads, d = s["q"].shape
    group, p, w = heads // case["kv_heads"], case["block_tokens"], case["window"]
    out = torch.zeros((t, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((t, heads), -math.inf, dtype=torch.float64, device="cuda")
    start, kind = s["q_start"].tolist(), CODES[case["codes"]]
    for i, n in enumerate(s["lengths"].tolist()):
        a, b = start[i], start[i + 1]
        if n == 0 or a == b:
            continue
        blocks = s["tables"][i, :_blocks(n, p)].long()
        for g in range(case["kv_heads"]):
            k = (s["k_codes"][blocks, g].view(kind).double() * s["k_scale"][blocks, g].double()[:, None, None]).reshape(-1, d)[:n]
            v = (s["v_codes"][blocks, g].view(kind).double() * s["v_scale"][blocks, g].double()[:, None, None]).reshape(-1, d)[:n]
            for c in range(a, b, 1024):
                e = min(b, c + 1024)
                q = s["q"][c:e, g * group:(g + 1) * group].double()
                z = torch.einsum("thd,ld->thl", q, k) / math.sqrt(d)
                at = torch.arange(c, e, device="cuda") - b + n
                j = torch.arange(n, device="cuda")
                hide = j[None] > at[:, None]
                if w:
                    hide |= j[None] <= at[:, None] - w
                z.masked_fill_(hide[:, None], -math.inf)
                m = torch.logsumexp(z, 2)
                lse[c:e, g * group:(g + 1) * group] = m
                out[c:e, g * group:(g + 1) * group] = torch.einsum("thl,ld->thd", torch.exp(z - m[:, :, None]), v)
    return {"out": out, "lse": lse}
