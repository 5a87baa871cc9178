"""The 8-bit key/value cache on the GPU against its 64-bit reference: block tables and slot maps and the
cache's codes and scales exactly, attention within the tolerance that kv_reference derives."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


# ------------------------------------------------------------------ block tables
def state(rng, before, after, p, spare, width):
    """Tables of distinct blocks for `before`, a free stack of `spare` others."""
    held = -(-before // p)
    blocks = rng.permutation(int(held.sum()) + spare)
    tables = np.full((len(before), width), -1, np.int32)
    at = 0
    for r, h in enumerate(held):
        tables[r, :h] = blocks[at:at + h]
        at += h
    free = np.full(len(blocks) + 3, -7, np.int32)
    free[:spare] = blocks[at:]
    return tables, free


def check_tables(before, after, p, spare, width, pad=0, seed=0, twice=True):
    rng = np.random.RandomState(seed)
    before, after = np.asarray(before, np.int32), np.asarray(after, np.int32)
    tables, free = state(rng, before, after, p, spare, width)
    tokens = int(np.maximum(after.astype(np.int64) - before, 0).sum()) + pad
    want = ref.tables(tables, before, after, free, spare, tokens, p)
    t, f = gpu(tables), gpu(free)
    count = torch.tensor([spare], dtype=torch.int32, device="cuda")
    for _ in range(2 if twice else 1):  # the same call again changes nothing
        got = mx.kv_block_tables(t, gpu(before), gpu(after), f, count, tokens, p)
        assert mx.mx_check() == mx.MX_OK
        for g, w in zip((t, f, *got), want):
            assert np.array_equal(g.cpu().numpy(), w)
    assert int(count) == spare
    return want


@pytest.mark.parametrize("p", [16, 32, 64, 128])
@pytest.mark.parametrize("requests", [1, 2, 31, 511, 513, 1500])
def test_tables_mixed(p, requests):
    rng = np.random.RandomState(p + requests)
    before = rng.randint(0, 700, requests)
    what = rng.rand(requests)
    after = np.where(what < 0.3, before + 1, np.where(what < 0.5, 0, np.where(what < 0.7, before // 2, before + rng.randint(0, 300, requests))))
    check_tables(before, after, p, spare=30 * requests, width=70, pad=5, seed=requests)


def test_tables_edges():
    check_tables([0], [0], 16, 1, 1)                                # nothing to do
    check_tables([0], [0], 16, 0, 1, pad=3)
    check_tables([0, 16, 15, 17], [1, 17, 16, 17], 16, 4, 3)        # exactly at blocks' ends
    check_tables([64, 0, 128], [0, 192, 0], 64, 0, 3)               # all popped blocks were pushed in this call
    check_tables([64, 0, 128], [0, 64, 0], 64, 5, 3)                # more pushed than popped
    check_tables([0] * 16384, [1] * 16384, 16, 16384, 1)            # the most requests


def test_tables_too_few_blocks_moves_nothing():
    want = check_tables([10, 70, 5], [0, 200, 90], 16, 3, 20, pad=2)
    assert want[5].tolist()[1] > 0 and (want[3] == -1).all()


@pytest.mark.parametrize("before,after,tokens,count", [
    ([-1, 3], [1, 4], 8, 4), ([0, 3], [1, 1000], 1000, 4), ([0, 3], [1, -4], 8, 4), ([0, 3], [9, 9], 5, 4),
    ([0, 3], [1, 4], 8, -1), ([0, 3], [1, 4], 8, 9)])
def test_tables_broken_contract_is_reported_and_moves_nothing(before, after, tokens, count):
    tables, free = np.full((2, 4), 1, np.int32), np.arange(8, dtype=np.int32)
    t, f = gpu(tables), gpu(free)
    c = torch.tensor([count], dtype=torch.int32, device="cuda")
    q_start, slots, positions, info = mx.kv_block_tables(t, gpu(np.int32(before)), gpu(np.int32(after)), f, c, tokens, 16)
    assert mx.mx_check() == mx.MX_ERR_INVALID_ARG
    assert mx.mx_check() == mx.MX_OK
    assert np.array_equal(t.cpu(), tables) and np.array_equal(f.cpu(), free)
    assert (slots == -1).all() and (positions == -1).all() and (q_start == 0).all() and int(info[1]) == 0


# ------------------------------------------------------------------ append
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def values(rng, shape, kind, spread=2.0):
    x = rng.randn(*shape) * np.exp(spread * rng.randn(*shape[:-1], 1))
    return torch.from_numpy(x.clip(-6e4, 6e4)).to(kind)


def a_cache(rng, blocks, kv_heads, p, d, elem):
    x = rng.randn(blocks, kv_heads, p, d) * np.exp(1.5 * rng.randn(blocks, kv_heads, 1, 1))
    scale = np.array([[ref.scale_for(x[b, h], elem) for h in range(kv_heads)] for b in range(blocks)])
    return ref.encode(x / scale[:, :, None, None], elem), scale.astype(np.float32)


def slots_for(rng, before, after, p, blocks):
    order, at, out = rng.permutation(blocks), 0, []
    for a, b in zip(before, after):
        own = order[at:at + -(-b // p)]
        at += len(own)
        out += [int(own[i // p]) * p + i % p for i in range(a, b)]
    assert at <= blocks
    return np.array(out, np.int64)


@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("p,d,kv_heads", [(16, 64, 3), (16, 128, 1), (32, 128, 2), (64, 64, 5), (64, 128, 8), (128, 128, 2),
                                          (128, 64, 1)])
def test_append(p, d, kv_heads, kind, elem):
    rng = np.random.RandomState(p * d + elem)
    before = np.array([0, 0, 1, p - 1, p, 5, 3, 2 * p + 7, 0])
    after = before + np.array([1, p, 1, 1, 1, 3 * p, 0, 2, 2 * p + 3])
    blocks = int((-(-after // p)).sum()) + 2
    slots = slots_for(rng, before, after, p, blocks)
    slots = np.concatenate([slots[:1], [-1], slots[1:], [-1, -1]])  # places left out
    t = len(slots)
    fused = values(rng, (t, 2 * kv_heads + 1, d), TYPES[kind]).cuda()
    k, v = fused[:, :kv_heads], fused[:, kv_heads + 1:]             # slices of one projection
    want, codes, scales = [], [], []
    for x in (k, v):
        c, s = a_cache(rng, blocks, kv_heads, p, d, elem)
        codes.append(gpu(c))
        scales.append(gpu(s))
        want.append(ref.append(x.double().cpu().numpy(), slots, c, s, elem))
    for _ in range(2):  # the same tokens again change nothing
        mx.kv_cache_append(k, v, gpu(slots), codes[0], codes[1], scales[0], scales[1], elem=elem)
        assert mx.mx_check() == mx.MX_OK
        for c, s, w in zip(codes, scales, want):
            assert np.array_equal(s.cpu().numpy(), w[1])
            table = ref.decode_table(elem)
            assert np.array_equal(table[c.cpu().numpy()], table[w[0]], equal_nan=True)


@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
def test_append_zeros_nan_inf_and_limits(elem):
    d, p = 64, 16
    x = np.zeros((8, 1, d), np.float32)
    x[1] = np.nan
    x[2, 0, :3] = [np.inf, -np.inf, 1.0]
    x[3, 0, 0] = 3e38
    x[4, 0, 0] = 2.0 ** -126
    x[5, 0, 5] = -448 * 2.0 ** 10
    x[6, 0, 5] = 450 * 2.0 ** 10
    k = torch.from_numpy(x).bfloat16().cuda()
    slots = np.arange(8, dtype=np.int64) * p
    codes, scale = np.zeros((8, 1, p, d), np.uint8), np.full((8, 1), np.nan, np.float32)
    want_c, want_s = ref.append(k.double().cpu().numpy(), slots, codes, scale, elem)
    kc, vc, ks, vs = gpu(codes), gpu(codes), gpu(scale), gpu(scale)
    mx.kv_cache_append(k, k, gpu(slots), kc, vc, ks, vs, elem=elem)
    assert mx.mx_check() == mx.MX_OK
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(c.cpu().numpy(), want_c)


def test_append_token_by_token_matches_the_reference():
    """A block filled one token a call, its scale growing: codes and scales after every step."""
    rng = np.random.RandomState(5)
    p, d, h, elem = 16, 64, 2, mx.E4M3
    codes, scale = np.zeros((2, h, p, d), np.uint8), np.ones((2, h), np.float32)
    kc, ks, vc, vs = gpu(codes), gpu(scale), gpu(codes), gpu(scale)
    for i in range(p):
        x = values(rng, (1, h, d), torch.bfloat16, spread=3.0).cuda()
        slots = np.array([p + i], np.int64)
        mx.kv_cache_append(x, x, gpu(slots), kc, vc, ks, vs, elem=elem)
        codes, scale = ref.append(x.double().cpu().numpy(), slots, codes, scale, elem)
        assert np.array_equal(ks.cpu().numpy(), scale) and np.array_equal(kc.cpu().numpy(), codes)
        assert np.array_equal(vs.cpu().numpy(), scale) and np.array_equal(vc.cpu().numpy(), codes)


def test_append_slots_out_of_range_are_left_out_and_reported():
    codes, scale = torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device="cuda"), torch.ones(2, 1, device="cuda")
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16, device="cuda")
    mx.kv_cache_append(x, x, gpu(np.array([32, -5, 1 << 40], np.int64)), codes, codes.clone(), scale, scale.clone())
    assert mx.mx_check() == mx.MX_ERR_INVALID_ARG
    assert mx.mx_check() == mx.MX_OK
    assert not codes.any() and (scale == 1).all()


# ------------------------------------------------------------------ attention
def attention_case(rng, lens, queries, heads, kv_heads, d, p, kind, elem, q_pad=0, block_shift=0):
    """Numpy cache, tables (-1 past the length), codes that no token owns set to NaN, and queries in a
    strided slice."""
    lens, queries = np.asarray(lens, np.int32), np.asarray(queries, np.int32)
    held = -(-lens // p)
    blocks = int(held.sum()) + 3
    kc, ks = a_cache(rng, blocks, kv_heads, p, d, elem)
    vc, vs = a_cache(rng, blocks, kv_heads, p, d, elem)
    order = rng.permutation(blocks)
    tables, at = np.full((len(lens), max(1, int(held.max()) + 1)), -1, np.int32), 0
    for r, h in enumerate(held):
        tables[r, :h] = order[at:at + h]
        if h and lens[r] % p:
            for c in (kc, vc):
                c[order[at + h - 1], :, lens[r] % p:] = 0x7F   # places no token has yet
        at += h
    ks[order[at:]] = vs[order[at:]] = np.nan
    kc[order[at:]] = vc[order[at:]] = 0x7F
    q_start = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
    q = values(rng, (int(q_start[-1]) + q_pad, heads + 2, d), TYPES[kind], spread=0.5).cuda()[:, 1:-1]
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, tables=tables, lens=lens, q_start=q_start)


def run_attention(c, elem, causal=True, window=0, scale=None, **kw):
    args = [gpu(c[n]) for n in ("kc", "vc", "ks", "vs", "tables", "lens", "q_start")]
    most = int(np.diff(c["q_start"]).max(initial=0))
    return mx.kv_attention(c["q"], *args, max_q_len=most, elem=elem, causal=causal, window=window, softmax_scale=scale, **kw)


def check_attention(c, elem, causal=True, window=0, scale=None):
    d = c["q"].shape[2]
    used = int(c["q_start"][-1])
    out, lse = run_attention(c, elem, causal, window, scale)
    again = run_attention(c, elem, causal, window, scale)
    assert mx.mx_check() == mx.MX_OK
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), again[1].view(torch.int32))
    want, want_lse, tol, lse_tol = ref.attention(
        c["q"].double().cpu().numpy()[:used], c["kc"], c["vc"], c["ks"], c["vs"], c["tables"], c["lens"], c["q_start"],
        elem, d ** -0.5 if scale is None else scale, causal, window)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (got[used:] == 0).all() and (got_lse[used:] == -np.inf).all()
    got, got_lse = got[:used], got_lse[:used]
    empty = want_lse == -np.inf
    assert (got_lse[empty] == -np.inf).all() and (got[empty] == 0).all()
    half_ulp = 2.0 ** -9 if out.dtype == torch.bfloat16 else 2.0 ** -12
    off = np.abs(got - want)
    bound = tol + half_ulp * 2 * (np.abs(want) + tol) + 2.0 ** -25
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    assert (off[fine] <= bound[fine]).all(), (off[fine] / bound[fine]).max()
    fine = ~empty & ~np.isnan(want_lse)
    assert np.array_equal(np.isnan(got_lse), np.isnan(want_lse))
    assert (np.abs(got_lse - want_lse)[fine] <= lse_tol[fine]).all(), (np.abs(got_lse - want_lse)[fine] / lse_tol[fine]).max()
    return out, lse


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 0, 511, 777]


@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("d,p", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64), (128, 128)])
def test_single_tokens(d, p, kind, elem):
    rng = np.random.RandomState(d + p + elem)
    check_attention(attention_case(rng, LENS, [1] * len(LENS), 8, 2, d, p, kind, elem), elem)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (5, 1), (8, 1), (18, 2), (16, 1), (32, 2), (33, 1), (64, 1), (130, 1)])
def test_head_layouts(heads, kv_heads):
    rng = np.random.RandomState(heads)
    check_attention(attention_case(rng, [1, 70, 300], [1, 1, 1], heads, kv_heads, 128, 64, "bf16", mx.E4M3), mx.E4M3)
    check_attention(attention_case(rng, [9, 70, 150], [2, 7, 3], heads, kv_heads, 64, 16, "f16", mx.E5M2), mx.E5M2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 5, 64, 100])
def test_masks(causal, window):
    rng = np.random.RandomState(window)
    lens = [1, 5, 40, 64, 130, 257, 0, 7, 3, 300]
    queries = [1, 5, 3, 2, 4, 6, 2, 0, 8, 1]       # more queries than tokens (the first rows see nothing), none at all
    for p, d in ((16, 128), (128, 64)):
        check_attention(attention_case(rng, lens, queries, 4, 2, d, p, "bf16", mx.E4M3, q_pad=3), mx.E4M3, causal, window)


@pytest.mark.parametrize("window", [0, 1, 77, 200])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,p,kind,elem", [(128, 64, "bf16", 0), (64, 16, "f16", 1), (128, 16, "f16", 0), (64, 128, "bf16", 0)])
def test_prompts(d, p, kind, elem, causal, window):
    rng = np.random.RandomState(window + p)
    lens, queries = [300, 129, 1, 512, 65, 0, 200, 90], [300, 100, 1, 33, 65, 3, 0, 130]
    check_attention(attention_case(rng, lens, queries, 4, 2, d, p, kind, elem, q_pad=2), elem, causal, window)


@pytest.mark.parametrize("group", [1, 3, 8])
def test_prompt_head_groups(group):
    rng = np.random.RandomState(group)
    check_attention(attention_case(rng, [700, 64, 257], [150, 64, 200], 2 * group, 2, 128, 64, "bf16", 0), 0)


@pytest.mark.parametrize("queries", [1, 4, 20, 90])
def test_one_long_context(queries):
    """Few rows over a long context: the work is split over it and joined."""
    rng = np.random.RandomState(queries)
    check_attention(attention_case(rng, [20000], [queries], 8, 2, 128, 64, "bf16", 0), 0)
    check_attention(attention_case(rng, [9999, 30, 4000], [queries, min(30, queries), 2], 4, 4, 64, 16, "f16", 0), 0)


@pytest.mark.parametrize("queries", [1, 6, 30, 100])
def test_scores_of_every_size(queries):
    """A large softmax scale (one weight near 1), a tiny one (all alike), and blocks of very unlike scales."""
    rng = np.random.RandomState(queries)
    c = attention_case(rng, [400, 150], [queries, min(150, queries)], 4, 2, 128, 32, "bf16", 0)
    check_attention(c, 0, scale=3.0)
    check_attention(c, 0, scale=1e-4)
    c["ks"] *= 2.0 ** rng.randint(-3, 3, c["ks"].shape)
    c["vs"] *= 2.0 ** rng.randint(-30, 30, c["vs"].shape)
    check_attention(c, 0)


@pytest.mark.parametrize("queries", [1, 5, 30, 60, 120])
def test_nan_reaches_only_rows_that_see_it(queries):
    rng = np.random.RandomState(3)
    c = attention_case(rng, [260, 130], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    blocks = c["tables"][0]
    at = 260 - queries // 2 - 1                                  # seen by the last rows only (by all, if there is one)
    c["vc"][blocks[at // 64], 0, at % 64, 7] = 0xFF
    c["vc"][blocks[at // 64], 0, at % 64, 90] = 0x7F
    c["kc"][c["tables"][1][(130 - queries // 3 - 1) // 64], 1, (130 - queries // 3 - 1) % 64, 3] = 0x7F
    check_attention(c, 0)
    c = attention_case(rng, [260, 130], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    c["vc"][c["tables"][0][0], :, 3] = 0x7F                      # before every row's window
    c["kc"][c["tables"][0][0], :, 3] = 0x7F
    check_attention(c, 0, window=30)
    c = attention_case(rng, [260, 130], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    c["q"] = c["q"].clone()
    c["q"][-1, 1, 5] = float("nan")                              # one row's own
    check_attention(c, 0)


def test_cache_past_32_bits():
    """Codes whose offsets pass 2^32, in blocks at the end of a large cache."""
    rng = np.random.RandomState(9)
    p, d, h, blocks = 128, 128, 8, 36000                         # 4.7 GB of codes each
    c = attention_case(rng, [500, 129], [1, 40], 8, h, d, p, "bf16", 0)
    n = len(c["ks"])
    kc, vc = (torch.zeros(blocks, h, p, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = torch.ones(blocks, h, device="cuda"), torch.ones(blocks, h, device="cuda")
    for big, small in ((kc, "kc"), (vc, "vc"), (ks, "ks"), (vs, "vs")):
        big[-n:] = gpu(c[small])
    tables = np.where(c["tables"] >= 0, c["tables"] + blocks - n, -1).astype(np.int32)
    small = run_attention(c, 0)
    big = mx.kv_attention(c["q"], kc, vc, ks, vs, gpu(tables), gpu(c["lens"]), gpu(c["q_start"]), 40)
    assert torch.equal(small[0], big[0]) and torch.equal(small[1], big[1])
    k = values(rng, (3, h, d), torch.bfloat16).cuda()
    slots = np.array([(blocks - 1) * p + p - 2, (blocks - 1) * p + p - 1, (blocks - 2) * p], np.int64)
    before = kc[-2:].cpu().numpy(), ks[-2:].cpu().numpy()
    mx.kv_cache_append(k, k, gpu(slots), kc, vc, ks, vs)
    want = ref.append(k.double().cpu().numpy(), slots - (blocks - 2) * p, *before, 0)
    table = ref.decode_table(0)
    assert np.array_equal(table[kc[-2:].cpu().numpy()], table[want[0]], equal_nan=True)
    assert np.array_equal(ks[-2:].cpu().numpy(), want[1])
    assert mx.mx_check() == mx.MX_OK


@pytest.mark.parametrize("requests,queries,tokens", [(1100, 1, 16384), (2100, 20, 16384), (3000, 3, 200), (16384, 1, 64)])
def test_many_requests(requests, queries, tokens):
    """More tiles in all than the ranges' 32-bit arithmetic takes, and as many requests as there may be: every
    request's table names one block over and over, so it sees that block's tokens, weighted alike."""
    rng = np.random.RandomState(requests)
    p, d, h, heads = 64, 64, 8, 16
    c = attention_case(rng, [p], [queries], heads, h, d, p, "bf16", 0)
    c["q"] = c["q"].repeat(requests, 1, 1)
    c["tables"] = np.full((requests, -(-tokens // p)), c["tables"][0, 0], np.int32)
    c["lens"] = np.full(requests, tokens, np.int32)
    c["q_start"] = np.arange(requests + 1, dtype=np.int32) * queries
    out, lse = run_attention(c, 0, causal=False)
    assert mx.mx_check() == mx.MX_OK
    assert (out.view(requests, -1) == out.view(requests, -1)[:1]).float().mean() > 0.9  # (splits differ: last bits may)
    small = dict(c, q=c["q"][:queries], tables=c["tables"][:1], lens=np.array([p]), q_start=np.array([0, queries]))
    full, rest = divmod(tokens, p)
    want, want_lse, tol, lse_tol = ref.attention(
        small["q"].double().cpu().numpy(), c["kc"], c["vc"], c["ks"], c["vs"], small["tables"], small["lens"],
        small["q_start"], 0, d ** -0.5, False, 0)
    if rest:  # the last block is seen in part: the reference over all of the tokens
        want, want_lse, tol, lse_tol = ref.attention(
            small["q"].double().cpu().numpy(), c["kc"], c["vc"], c["ks"], c["vs"], small["tables"], np.array([tokens]),
            small["q_start"], 0, d ** -0.5, False, 0)
    else:
        want_lse, lse_tol = want_lse + np.log(full), lse_tol + tokens * 2.0 ** -23
        tol = tol * 2 + tokens * 2.0 ** -23 * np.abs(want).max()
    out = out.double().cpu().numpy().reshape(requests, queries, heads, d)
    lse = lse.double().cpu().numpy().reshape(requests, queries, heads)
    assert (np.abs(out - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -25).all()
    assert (np.abs(lse - want_lse) <= lse_tol).all()


@pytest.mark.parametrize("queries", [1, 70])
def test_blocks_out_of_range_are_not_read_and_reported(queries):
    rng = np.random.RandomState(1)
    c = attention_case(rng, [200], [queries], 4, 2, 128, 64, "bf16", 0)
    c["tables"][0, 1] = len(c["ks"])
    run_attention(c, 0)
    assert mx.mx_check() == mx.MX_ERR_INVALID_ARG
    assert mx.mx_check() == mx.MX_OK


@pytest.mark.parametrize("queries", [1, 50])
def test_side_stream_own_buffers_and_graph(queries):
    """On a stream of the caller's, into the caller's buffers, captured and replayed with new inputs."""
    rng = np.random.RandomState(queries)
    c = attention_case(rng, [300, 75], [queries, 1], 8, 2, 128, 64, "bf16", 0)
    tensors = [gpu(c[n]) for n in ("kc", "vc", "ks", "vs", "tables", "lens", "q_start")]
    t, heads, d = c["q"].shape
    q = c["q"].clone()
    out, lse = torch.empty(t, heads, d, dtype=q.dtype, device="cuda"), torch.empty(t, heads, device="cuda")
    ws = torch.zeros(mx.kv_attention_workspace_bytes(t, 2, queries, heads, 2, d), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def call():
        mx.kv_attention(q, *tensors, max_q_len=queries, out=out, lse=lse, workspace=ws)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    q.copy_(q.flip(0))
    tensors[5].sub_(1)
    out.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    want = mx.kv_attention(q, *tensors, max_q_len=queries)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert mx.mx_check() == mx.MX_OK


def test_a_workspace_serves_call_after_call():
    """One workspace, cleared once, for calls of unlike sizes in turn: its counters are zero after each, and what
    else earlier calls left in it does not matter."""
    rng = np.random.RandomState(21)
    ws = torch.full((mx.kv_attention_workspace_bytes(1, 4, 1000, 8, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    for lens, queries in (([5000, 70], [1, 1]), ([3], [1]), ([900, 40, 2000], [100, 40, 3]), ([20000], [2]), ([5000, 70], [1, 1])):
        c = attention_case(rng, lens, queries, 8, 2, 128, 64, "bf16", 0)
        for _ in range(2):
            out, lse = run_attention(c, 0, workspace=ws)
            want = run_attention(c, 0)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            assert not ws[:4096].any()
    assert mx.mx_check() == mx.MX_OK


# ------------------------------------------------------------------ together
def test_serving_steps():
    """Prompts, single tokens, a rewind and a finish through tables, append and attention, each step
    against the reference's own cache."""
    rng = np.random.RandomState(11)
    p, d, kv_heads, heads, blocks, elem = 16, 64, 2, 6, 40, mx.E4M3
    tables = torch.full((4, 20), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(blocks, dtype=torch.int32, device="cuda")
    count = torch.tensor([blocks], dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((blocks, kv_heads, p, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((blocks, kv_heads), float("nan"), device="cuda") for _ in range(2))
    host = [kc.cpu().numpy(), ks.cpu().numpy(), vc.cpu().numpy(), vs.cpu().numpy()]
    before = np.zeros(4, np.int32)
    for after in ([40, 17, 0, 90], [41, 18, 33, 91], [41, 19, 34, 92], [36, 0, 35, 93], [37, 70, 36, 94], [0, 71, 37, 95]):
        after = np.array(after, np.int32)
        tokens = int(np.maximum(after - before, 0).sum())
        q_start, slots, positions, info = mx.kv_block_tables(tables, gpu(before), gpu(after), free, count, tokens, p)
        count = info[:1]
        x = values(rng, (tokens, heads + 2 * kv_heads, d), torch.bfloat16, spread=0.7).cuda()
        q, k, v = x.split([heads, kv_heads, kv_heads], dim=1)
        mx.kv_cache_append(k, v, slots, kc, vc, ks, vs)
        at = slots.cpu().numpy()
        host[0], host[1] = ref.append(k.double().cpu().numpy(), at, host[0], host[1], elem)
        host[2], host[3] = ref.append(v.double().cpu().numpy(), at, host[2], host[3], elem)
        assert np.array_equal(kc.cpu().numpy(), host[0]) and np.array_equal(vc.cpu().numpy(), host[2])
        c = dict(q=q, kc=host[0], vc=host[2], ks=host[1], vs=host[3], tables=tables.cpu().numpy(), lens=after,
                 q_start=q_start.cpu().numpy())
        check_attention(c, elem)
        held = sum(-(-int(n) // p) for n in after)
        assert info.tolist() == [blocks - held, 0]
        before = after
    assert mx.mx_check() == mx.MX_OK
