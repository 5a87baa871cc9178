"""Attention of a tree's queries over the 8-bit key/value cache on the GPU, against the formula in 64 bits within the
tolerance that the reference derives."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import drafts_reference as ref
from tests import kv_reference as kv
from tests.test_gpu_drafts import gpu, ok, reported, starts

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 0.0), "f16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def caches(rng, tables_blocks, kv_heads, p, d, elem):
    codes, scales = [], []
    for spread in (0.5, 1.5):
        x = rng.randn(tables_blocks, kv_heads, p, d) * np.exp(spread * rng.randn(tables_blocks, kv_heads, 1, 1))
        s = np.array([[kv.scale_for(x[b, h], elem) for h in range(kv_heads)] for b in range(tables_blocks)])
        codes.append(kv.encode(x / s[:, :, None, None], elem))
        scales.append(s.astype(np.float32))
    return codes, scales


def inputs(context, nodes, p, kv_heads, group, d, elem, kind="bf16", seed=0, pad=0, mask=None, words=None, window=0, reach=None):
    rng = np.random.RandomState(seed)
    context, nodes = np.asarray(context), np.asarray(nodes)
    lengths = (context + nodes).astype(np.int32)
    held = -(-lengths // p)
    blocks = int(held.sum()) + 2
    order, at = rng.permutation(blocks), starts(held)
    tables = np.full((len(nodes), int(held.max()) + 1), -1, np.int32)
    for r, n in enumerate(held):
        tables[r, :n] = order[at[r]:at[r] + n]
    codes, scales = caches(rng, blocks, kv_heads, p, d, elem)
    t = int(nodes.sum()) + pad
    parents = np.concatenate([ref.random_parents(rng, n, reach) for n in nodes] + [np.full(pad, -1)]).astype(np.int32)
    words = words or max(1, -(-int(nodes.max()) // 64))
    tree, positions = ref.trees(parents, lengths, starts(nodes), words, window, t)
    if mask == "random":
        tree = rng.randint(0, 1 << 32, (t, words)).astype(np.uint64) << np.uint64(32) | rng.randint(0, 1 << 32, (t, words)).astype(np.uint64)
    q = torch.from_numpy(rng.randn(t, kv_heads * group, d) * np.exp(0.3 * rng.randn(t, 1, 1))).to(TYPES[kind][0])
    return dict(q=q, codes=codes, scales=scales, tables=tables, lengths=lengths, q_start=starts(nodes), most=int(nodes.max()),
                mask=tree, positions=positions, elem=elem, window=window, kind=kind, d=d)


def call(a, **kw):
    return mx.kv_tree_attention(a["q"].cuda(), *(gpu(c) for c in a["codes"]), *(gpu(s) for s in a["scales"]), gpu(a["tables"]),
                                gpu(a["lengths"]), gpu(a["q_start"]), a["most"], gpu(a["mask"].view(np.int64)),
                                gpu(a["positions"]) if a["window"] else None, elem=a["elem"], window=a["window"], **kw)


def check(a, got=None, rows=None):
    got = got or call(a)
    ok()
    seen = ref.sees(a["mask"], a["positions"], a["lengths"], a["q_start"], a["window"])
    out, lse, tol, lse_tol = ref.tree_attention(a["q"].double().numpy(), *a["codes"], *a["scales"], a["tables"], a["lengths"],
                                                a["q_start"], seen, a["elem"], a["d"] ** -0.5)
    _, half_step, smallest = TYPES[a["kind"]]
    mine, mine_lse = (x.detach().cpu().double().numpy() for x in got)
    nan = np.isnan(out)
    assert np.array_equal(np.isnan(mine), nan)
    tol = tol + (np.abs(out) + tol) * half_step + smallest
    assert (np.abs(mine - out)[~nan] <= tol[~nan]).all(), (np.abs(mine - out)[~nan] / tol[~nan]).max()
    some = np.isfinite(lse)
    assert np.array_equal(np.isneginf(mine_lse), np.isneginf(lse))
    assert (np.abs(mine_lse - lse, where=some, out=np.zeros_like(lse)) <= lse_tol + (~some)).all()
    return got


# nodes x group rows a kv head: up to 16 and more, in one unit of 128 or 256 rows and in several
@pytest.mark.parametrize("kind,elem", [("bf16", mx.E4M3), ("f16", mx.E5M2)])
@pytest.mark.parametrize("p,d,kv_heads,group", [(16, 64, 3, 1), (32, 128, 2, 4), (64, 128, 1, 8), (128, 64, 2, 5), (64, 64, 1, 16)])
def test_tree_attention(p, d, kv_heads, group, kind, elem):
    context = [0, 1, 63, 64, 130, p - 1, 300, 127, 500]
    for nodes in ([1, 2, 1, 2, 1, 1, 2, 0, 2], [2, 3, 4, 1, 2, 4, 3, 4, 0], [33, 16, 12, 7, 1, 0, 9, 30, 20]):
        check(inputs(context, nodes, p, kv_heads, group, d, elem, kind, seed=p + group, pad=3))


@pytest.mark.parametrize("window", [1, 5, 64, 100, 1000])
@pytest.mark.parametrize("nodes", [[4, 3, 0, 1, 2], [30, 64, 17, 40, 9]])
def test_tree_attention_windows(nodes, window):
    check(inputs([0, 40, 7, 257, 500], nodes, 64, 2, 4, 128, mx.E4M3, seed=window, window=window))
    check(inputs([0, 40, 7, 257, 500], nodes, 16, 1, 2, 64, mx.E5M2, "f16", seed=window, window=window, reach=2))


@pytest.mark.parametrize("words", [None, 3, 16])
def test_tree_attention_any_mask(words):
    """Bits at random: nodes that a row sees behind it, rows that do not see themselves, bits behind the last node."""
    check(inputs([0, 100, 64, 1], [1, 4, 3, 2], 64, 2, 4, 128, mx.E4M3, mask="random", words=words))
    check(inputs([0, 100, 64, 1, 3], [60, 64, 33, 17, 1], 64, 1, 4, 128, mx.E4M3, mask="random", words=words))
    if words != 1:
        check(inputs([0, 100, 70], [130, 190, 65], 16, 1, 1, 64, mx.E5M2, "f16", mask="random", words=words))


def test_tree_attention_large_trees():
    check(inputs([100, 0], [300, 1024], 32, 1, 1, 64, mx.E4M3))
    check(inputs([777], [257], 64, 1, 2, 128, mx.E4M3, reach=3))


@pytest.mark.parametrize("nodes", [[3, 4, 2], [40, 17, 64]])
def test_rows_that_see_nothing(nodes):
    a = inputs([0, 0, 100], nodes, 64, 2, 4, 128, mx.E4M3)
    a["mask"][::2] = 0
    out, lse = check(a)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()
    a = inputs([0, 0, 100], nodes, 64, 2, 4, 128, mx.E4M3, window=1)
    a["mask"][:] = 0  # with a window of 1 that ends in front of the nodes
    out, lse = check(a)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("nodes", [[3, 4, 2], [40, 17, 60]])
@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
def test_nan_reaches_the_rows_that_see_it(nodes, elem):
    a = inputs([50, 64, 0], nodes, 16, 2, 4, 128, elem, seed=3)
    for r, c in ((0, 51), (1, 64), (2, 1), (0, 7)):  # nodes, and a token in front of them
        block, off = a["tables"][r, c // 16], c % 16
        a["codes"][1][block, 0, off, 5] = 0x7F
        if c == 51:
            a["codes"][0][block, 1, off, 9] = 0x7F   # a key: all of the rows that see it
    out, _ = call(a)
    ok()
    out = out.float().cpu().numpy()
    seen = ref.sees(a["mask"], a["positions"], a["lengths"], a["q_start"], 0)
    want = np.zeros(out.shape, bool)
    for r, c in ((0, 51), (1, 64), (2, 1), (0, 7)):
        rows = np.arange(a["q_start"][r], a["q_start"][r + 1])[seen[r][:, c]]
        want[rows, :4, 5] = True
        if c == 51:
            want[rows, 4:] = True
    assert np.array_equal(np.isnan(out), want)


@pytest.mark.parametrize("nodes", [[3, 4, 2, 1], [40, 17, 64, 5], [130, 1, 0, 200]])
@pytest.mark.parametrize("window", [0, 70])
def test_a_chain_is_a_draft(nodes, window):
    """What kv_attention gives for the same tokens in a row: bit by bit where the same kernel does both (up to 16 rows a
    kv head), else both within the formula's tolerance."""
    a = inputs([50, 64, 0, 300], nodes, 64, 2, 4, 128, mx.E4M3, reach=1, window=window, pad=2)
    got = call(a)
    want = mx.kv_attention(a["q"].cuda(), *(gpu(c) for c in a["codes"]), *(gpu(s) for s in a["scales"]), gpu(a["tables"]),
                           gpu(a["lengths"]), gpu(a["q_start"]), a["most"], window=window)
    ok()
    if max(nodes) <= 4:
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    check(a, got)
    check(a, want)


@pytest.mark.parametrize("nodes", [[3, 4, 2], [40, 17, 64]])
def test_broken_contracts(nodes):
    a = inputs([50, 64, 10], nodes, 64, 2, 4, 128, mx.E4M3, window=60)
    whole = call(a)
    ok()
    s = a["q_start"]
    for key, r, value in (("lengths", 1, nodes[1] - 1), ("lengths", 1, -3), ("lengths", 1, 1 << 29)):
        b = dict(a, **{key: a[key].copy()})
        b[key][r] = value
        out = [torch.full_like(whole[0], 7.0), torch.full_like(whole[1], 7.0)]
        call(b, out=out[0], lse=out[1])
        reported()
        for x, w in zip(out, whole):
            assert torch.equal(x[:s[1]], w[:s[1]]) and torch.equal(x[s[2]:], w[s[2]:]) and (x[s[1]:s[2]] == 7).all()
    b = dict(a, positions=a["positions"].copy())
    b["positions"][1], b["positions"][2] = 49, 2147483647  # in front of the nodes, behind them: taken as the nearest
    got = call(b)
    reported()
    b["positions"][1], b["positions"][2] = 50, 50 + nodes[0] - 1
    want = call(b)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_graph_streams_and_strides():
    a = inputs([500, 64, 0, 130], [40, 17, 64, 3], 64, 2, 4, 128, mx.E4M3, pad=2)
    want = call(a)
    ok()
    args = (*(gpu(c) for c in a["codes"]), *(gpu(s) for s in a["scales"]), gpu(a["tables"]), gpu(a["lengths"]),
            gpu(a["q_start"]), a["most"], gpu(a["mask"].view(np.int64)))
    wide = torch.full((len(a["q"]), 14, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:11] = a["q"].cuda()
    q = wide[:, 3:11]
    got = mx.kv_tree_attention(q, *args)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = mx.kv_tree_attention(q, *args)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = mx.kv_tree_attention(q, *args)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            out[0].fill_(7)
            g.replay()
        assert all(torch.equal(x, y) for _, out in graphs for x, y in zip(out, want))
    ok()
