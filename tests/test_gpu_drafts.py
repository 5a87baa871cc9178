"""Drafted tokens beside the 8-bit key/value cache on the GPU against the 64-bit reference: masks, positions, paths,
tokens, codes and scales exactly; the norm and rotation and their gradients within the tolerances derived there."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import drafts_reference as ref
from tests import kv_reference as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def starts(nodes):
    return np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)


def ok():
    assert mx.mx_check() == mx.MX_OK


def reported():
    assert mx.mx_check() == mx.MX_ERR_INVALID_ARG
    assert mx.mx_check() == mx.MX_OK


# ------------------------------------------------------------------ norm and rotation
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 0.0), "f16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}


def rows(rng, shape, kind, spread=1.0):
    x = rng.randn(*shape) * np.exp(spread * rng.randn(*shape[:-1], 1))
    return torch.from_numpy(x.clip(-6e4, 6e4)).to(kind)


def rotation(positions, rot):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)[None]
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, want, tol):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max()


CASES = [  # tokens, heads, kv heads, head_dim, rot, interleaved, weights, slices
    (1, 1, 1, 64, 64, False, "same", False), (7, 5, 1, 128, 128, False, "same", True), (33, 32, 8, 128, 128, True, "f32", True),
    (130, 3, 2, 80, 32, False, "f32", True), (19, 4, 4, 96, 96, False, "same", False), (5, 6, 0, 96, 96, True, "same", True),
    (64, 8, 4, 256, 256, False, "same", True), (12, 2, 1, 256, 16, True, "f32", False), (9, 3, 3, 8, 0, False, "same", True),
    (257, 2, 2, 64, 32, True, "f32", True), (40, 17, 9, 72, 64, False, "same", True), (3, 64, 8, 128, 64, False, "same", False)]


def norm_inputs(case, kind, seed=0):
    t, h, g, d, rot, _, weights, slices = case
    rng = np.random.RandomState(seed + t * d)
    x = rows(rng, (t, h + g + 1, d), kind).cuda()
    q, k = x[:, :h], x[:, h + 1:]
    if not slices:
        q, k = q.contiguous(), k.contiguous()
    wk = torch.float32 if weights == "f32" else kind
    qw, kw = (torch.from_numpy(1 + 0.5 * rng.randn(d)).to(wk).cuda() for _ in range(2))
    table = gpu(rotation(500, rot)) if rot else None
    return rng, q, k if g else None, qw, kw, table, gpu(rng.randint(0, 500, t), torch.int32)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_norm(case, kind):
    dtype, half_step, smallest = TYPES[kind]
    interleaved = case[5]
    _, q, k, qw, kw, table, positions = norm_inputs(case, dtype)
    got = mx.qk_norm_rope(q, k, qw, kw, table, positions, eps=1e-5, interleaved=interleaved)
    ok()
    for x, w, y in zip((q, k), (qw, kw), got):
        if x is None:
            assert y is None
            continue
        want, tol = ref.norm(f64(x), f64(w), None if table is None else table.cpu().numpy(), positions.cpu().numpy(), 1e-5,
                             interleaved, half_step, smallest)
        close(y, want, tol)
    # in place, in the slices: the same bits, and nothing beside them
    if k is not None:
        base = q._base if q._base is not None else None
        beside = base[:, case[1]].clone() if base is not None and base.dim() == 3 else None
        mx.qk_norm_rope(q, k, qw, kw, table, positions, eps=1e-5, interleaved=interleaved, q_out=q, k_out=k)
        ok()
        assert torch.equal(q, got[0]) and torch.equal(k, got[1])
        assert beside is None or torch.equal(base[:, case[1]], beside)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES)
def test_norm_backward(case, kind):
    dtype, half_step, smallest = TYPES[kind]
    interleaved = case[5]
    rng, q, k, qw, kw, table, positions = norm_inputs(case, dtype)
    dy = rows(rng, (case[0], case[1] + case[2], case[3]), dtype).cuda()
    dq, dk = dy[:, :case[1]], dy[:, case[1]:] if case[2] else None
    got = mx.qk_norm_rope_backward(dq, dk, q, k, qw, kw, table, positions, eps=1e-5, interleaved=interleaved)
    ok()
    for x, g, w, dx, dw in zip((q, k), (dq, dk), (qw, kw), got[:2], got[2:]):
        if x is None:
            assert dx is None and (dw == 0).all()
            continue
        want, want_w, tol, tol_w = ref.norm_backward(f64(g), f64(x), f64(w), None if table is None else table.cpu().numpy(),
                                                     positions.cpu().numpy(), 1e-5, interleaved, half_step, smallest)
        close(dx, want, tol)
        close(dw, want_w, tol_w)
    again = mx.qk_norm_rope_backward(dq, dk, q, k, qw, kw, table, positions, eps=1e-5, interleaved=interleaved)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    # over the results' gradients themselves
    mx.qk_norm_rope_backward(dq, dk, q, k, qw, kw, table, positions, eps=1e-5, interleaved=interleaved, dq=dq, dk=dk)
    ok()
    assert torch.equal(dq, got[0]) and (dk is None or torch.equal(dk, got[1]))


def test_norm_backward_is_the_slope_of_the_forward():
    """dx and dw against differences of the formula in 64 bits, along random directions."""
    rng = np.random.RandomState(5)
    t, h, d = 6, 3, 64
    x, w, dy, table = rng.randn(t, h, d), 1 + 0.3 * rng.randn(d), rng.randn(t, h, d), rotation(50, 32)
    positions = rng.randint(0, 50, t)

    def value(x, w):
        n = x / np.sqrt((x * x).mean(2, keepdims=True) + 1e-5) * w
        return (ref.turn(n, table, positions, False)[0] * dy).sum()
    q = torch.from_numpy(x).to(torch.float16).cuda()
    g = torch.from_numpy(dy).to(torch.float16).cuda()
    x, dy = f64(q), f64(g)
    got = mx.qk_norm_rope_backward(g, None, q, None, gpu(w, torch.float32), None, gpu(table), gpu(positions, torch.int32), eps=1e-5)
    ok()
    w = f64(gpu(w, torch.float32))
    _, _, tol, tol_w = ref.norm_backward(dy, x, w, table, positions, 1e-5, False, 2.0 ** -11, 2.0 ** -25)
    for _ in range(5):
        ex, ew = rng.randn(*x.shape), rng.randn(d)
        step = 1e-5
        slope = (value(x + step * ex, w + step * ew) - value(x - step * ex, w - step * ew)) / (2 * step)
        mine = (f64(got[0]) * ex).sum() + (f64(got[2]) * ew).sum()
        # what the gradients may be off by; the differences themselves by step^2 / 6 of a third derivative of at most
        # about 18 rows x 6 x 8 x 8 (each row's |e|, |x|, |y| and |dy| are 8): 1e-7
        assert abs(slope - mine) <= (tol * np.abs(ex)).sum() + (tol_w * np.abs(ew)).sum() + 1e-6


def test_norm_positions_left_out_and_out_of_range():
    rng = np.random.RandomState(1)
    q, k = rows(rng, (6, 4, 128), torch.bfloat16).cuda(), rows(rng, (6, 2, 128), torch.bfloat16).cuda()
    w = torch.ones(128, device="cuda", dtype=torch.bfloat16)
    table = gpu(rotation(10, 128))
    for positions, broken in (([3, -1, 0, 9, -1, 2], False), ([3, -2, 0, 9, 10, 2], True), ([0, -2147483648, 1, 1, 2147483647, 1], True)):
        out = [torch.full_like(x, 7.0) for x in (q, k)]
        mx.qk_norm_rope(q, k, w, w, table, gpu(np.int32(positions)), q_out=out[0], k_out=out[1])
        (reported if broken else ok)()
        good = [0, 2, 3, 5]
        whole = mx.qk_norm_rope(q[good], k[good], w, w, table, gpu(np.int32(positions)[good]))
        for a, b in zip(out, whole):
            assert torch.equal(a[good], b) and (a[[1, 4]] == 7).all()
        grads = mx.qk_norm_rope_backward(q, k, q * 0.5, k, w, w, table, gpu(np.int32(positions)))
        (reported if broken else ok)()
        some = mx.qk_norm_rope_backward(q[good], k[good], q[good] * 0.5, k[good], w, w, table, gpu(np.int32(positions)[good]))
        for a, b in zip(grads[:2], some[:2]):
            assert torch.equal(a[good], b) and (a[[1, 4]] == 0).all()
        for a, b in zip(grads[2:], some[2:]):  # (the same terms, perhaps in another order)
            assert torch.allclose(a, b, rtol=0, atol=float(24 * 2.0 ** -24 * 50))


def test_norm_of_no_tokens_and_of_zeros():
    w = torch.ones(64, device="cuda", dtype=torch.float16)
    none = torch.empty(0, 3, 64, device="cuda", dtype=torch.float16)
    p0 = torch.empty(0, device="cuda", dtype=torch.int32)
    out = mx.qk_norm_rope(none, none, w, w, None, p0)
    assert out[0].shape == (0, 3, 64)
    grads = mx.qk_norm_rope_backward(none, none, none, none, w, w, None, None)
    assert (grads[2] == 0).all() and (grads[3] == 0).all()
    zero = torch.zeros(2, 3, 64, device="cuda", dtype=torch.float16)
    out = mx.qk_norm_rope(zero, zero, w, w, None, None)
    ok()
    assert (out[0] == 0).all()


def test_norm_far_strides():
    """Rows whose offsets pass 32 bits (of elements and of bytes)."""
    base = torch.empty(3 << 30, device="cuda", dtype=torch.bfloat16)
    q = base.as_strided((3, 2, 64), (1 << 30, 1 << 29, 1))
    rng = np.random.RandomState(2)
    x = rows(rng, (3, 2, 64), torch.bfloat16).cuda()
    q.copy_(x)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    positions, table = gpu(np.int32([1, 2, 3])), gpu(rotation(10, 64))
    want = mx.qk_norm_rope(x, x, w, w, table, positions)
    got = mx.qk_norm_rope(q, q, w, w, table, positions)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    grads, far = mx.qk_norm_rope_backward(x, x, x, x, w, w, table, positions), mx.qk_norm_rope_backward(q, q, q, q, w, w, table, positions)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(grads, far))
    mx.qk_norm_rope(x, None, w, None, table, positions, q_out=q)
    assert torch.equal(q.contiguous(), want[0])


# ------------------------------------------------------------------ trees
def check_trees(nodes, most, window, pad=0, words=None, seed=0, reach=None):
    rng = np.random.RandomState(seed)
    parents = np.concatenate([ref.random_parents(rng, n, reach) for n in nodes] + [np.full(pad, 5)]).astype(np.int32)
    lengths = np.array([n + rng.randint(0, 1000) for n in nodes], np.int32)
    words = words or max(1, -(-most // 64))
    want = ref.trees(parents, lengths, starts(nodes), words, window, len(parents))
    out = torch.full((len(parents), words), 77, dtype=torch.int64, device="cuda")
    mask, positions = mx.kv_draft_trees(gpu(parents), gpu(lengths), gpu(starts(nodes)), most, window=window, tree_mask=out)
    ok()
    assert np.array_equal(mask.cpu().numpy().view(np.uint64), want[0]) and np.array_equal(positions.cpu().numpy(), want[1])


@pytest.mark.parametrize("window", [0, 1, 3, 64, 1000000])
def test_trees(window):
    check_trees([1], 1, window)
    check_trees([5, 0, 64, 63, 65, 1], 65, window, pad=3)
    check_trees([32] * 40, 32, window, words=3)
    check_trees([200, 129, 1, 0], 200, window, reach=2)
    check_trees([1024, 7, 1000], 1024, window, reach=1)    # chains
    check_trees([1024], 1024, window, pad=200)


def test_trees_forests_and_broken_contracts():
    parents, q_start = np.int32([-1, -1, 1, -1, 3, 0, 1]), np.int32([0, 5, 7])
    mask, positions = mx.kv_draft_trees(gpu(parents), gpu(np.int32([9, 2])), gpu(q_start), 5)
    reported()  # the second request's first node has a parent
    assert mask[:, 0].tolist() == [1, 2, 6, 8, 24, 0, 0] and positions.tolist() == [4, 4, 5, 4, 5, -1, -1]
    for q, lengths in (([0, 5, 8], [9, 2]), ([0, 6, 7], [9, 2]), ([0, 5, 4], [9, 2]), ([-1, 5, 7], [9, 2]),
                       ([0, -2147483648, 2147483647], [9, 2]), ([0, 5, 7], [4, 2]), ([0, 5, 7], [-5, 2]), ([0, 5, 7], [9, (1 << 30) + 1])):
        out = torch.full((7, 1), 77, dtype=torch.int64, device="cuda")
        mx.kv_draft_trees(gpu(np.int32([-1, 0, 1, 2, 3, -1, 0])), gpu(np.int32(lengths)), gpu(np.int32(q)), 5, tree_mask=out)
        reported()
        rows = out[:, 0].tolist()
        # written as a request's or as rows behind the last one, or not at all; requests that are whole, as ever
        assert all(x in (77, 0, full) for x, full in zip(rows, [1, 3, 7, 15, 31, 1, 3]))
        if q == [0, 5, 7]:
            assert rows == ([1, 3, 7, 15, 31] if lengths[0] == 9 else [77] * 5) + ([1, 3] if lengths[1] == 2 else [77] * 2)


# ------------------------------------------------------------------ verification
def probs(rng, n, vocab, peak=3.0):
    z = peak * rng.randn(n, vocab)
    p = np.exp(z - z.max(1, keepdims=True))
    return (p / p.sum(1, keepdims=True)).astype(np.float32)


def check_verify(nodes, vocab, certain, seed=0, pad=0, reach=None, offset=0, stride=0, target=None, draft=None, accept=None,
                 sample=None, drafts=None, parents=None):
    rng = np.random.RandomState(seed)
    t = int(sum(nodes)) + pad
    if parents is None:
        parents = np.concatenate([ref.random_parents(rng, n, reach) for n in nodes] + [np.zeros(pad)]).astype(np.int32)
    if target is None:
        target = probs(rng, t, vocab)
        draft = None if certain else probs(rng, t, vocab) * 0.4 + 0.6 * target[:t]
        draft = None if certain else (draft / draft.sum(1, keepdims=True)).astype(np.float32)
    if drafts is None:
        drafts, at = np.full(t, -5, np.int32), 0
        for n in nodes:
            for i in range(1, n):
                row = target[at + parents[at + i]] if certain else draft[at + parents[at + i]]
                drafts[at + i] = rng.choice(vocab, p=row.astype(np.float64) / row.astype(np.float64).sum())
            at += n
    accept = rng.rand(t).astype(np.float32) if accept is None else accept
    sample = rng.rand(len(nodes)).astype(np.float32) if sample is None else sample
    want = ref.verify(target, draft, drafts, parents, starts(nodes), accept, sample)

    def strided(x):  # rows apart, beginning anywhere
        if x is None or not (offset or stride):
            return None if x is None else gpu(x)
        base = torch.full((t * (vocab + stride) + offset,), float("nan"), device="cuda")
        y = base[offset:].as_strided((t, vocab), (vocab + stride, 1))
        y.copy_(gpu(x))
        return y
    got = mx.kv_verify_drafts(strided(target), gpu(drafts), gpu(parents), gpu(starts(nodes)), gpu(accept), gpu(sample),
                              draft_probs=strided(draft))
    ok()
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    return want


@pytest.mark.parametrize("certain", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 127, 512, 513, 1021, 32000, 50257, 131075])
def test_verify(vocab, certain):
    check_verify([1, 5, 0, 9, 17], vocab, certain, seed=vocab, pad=2)
    check_verify([26], vocab, certain, seed=vocab + 1, reach=3)


@pytest.mark.parametrize("certain", [True, False])
@pytest.mark.parametrize("requests", [1, 20, 39, 77, 153, 400])
def test_verify_many_requests(requests, certain):
    rng = np.random.RandomState(requests)
    want = check_verify(list(rng.randint(1, 7, requests)), 2003, certain, seed=requests)
    assert requests < 39 or len(set(want[2].tolist())) > 1  # paths of several lengths (a word on the inputs)


@pytest.mark.parametrize("certain", [True, False])
@pytest.mark.parametrize("offset,stride", [(0, 1), (1, 3), (2, 4), (3, 5)])
def test_verify_rows_anywhere(offset, stride, certain):
    check_verify([4, 7, 3], 4099, certain, seed=offset, offset=offset, stride=stride)


@pytest.mark.parametrize("certain", [True, False])
def test_verify_large_trees_and_many_siblings(certain):
    check_verify([300, 1024, 65], 700, certain, seed=1)
    t = 64  # every node a child of the root, most of them rejected, tokens that come again
    rng = np.random.RandomState(3)
    parents = np.concatenate([[-1], np.zeros(t - 1)]).astype(np.int32)
    target, draft = probs(rng, t, 40, 1.0), probs(rng, t, 40, 1.0)
    drafts = rng.randint(0, 40, t).astype(np.int32)
    for seed in range(6):
        accept = np.float32(1) - np.float32(2.0 ** -20) * rng.rand(t).astype(np.float32)
        check_verify([t], 40, certain, target=target, draft=None if certain else draft, drafts=drafts, parents=parents,
                     accept=np.minimum(accept, np.float32(1 - 2.0 ** -24)), sample=rng.rand(1).astype(np.float32))


def dyadic(rng, n, vocab, bits):
    """Rows of multiples of 2^-bits that sum to 1: every sum and product below is exact in 64 bits."""
    out = np.zeros((n, vocab))
    for i in range(n):
        cuts = np.sort(rng.randint(0, (1 << bits) + 1, vocab - 1))
        out[i] = np.diff(np.concatenate([[0], cuts, [1 << bits]])) / float(1 << bits)
    return out.astype(np.float32)


@pytest.mark.parametrize("certain", [True, False])
def test_verify_at_exact_borders(certain):
    """Random numbers that lie on the borders: a draft is accepted strictly below, a token begins at its running sum."""
    rng = np.random.RandomState(9)
    for trial in range(40):
        n, vocab = 6, 16
        target, draft = dyadic(rng, n, vocab, 10), None if certain else dyadic(rng, n, vocab, 10)
        drafts = rng.randint(0, vocab, n).astype(np.int32)
        accept = (rng.randint(0, 1 << 10, n) / 1024.0).astype(np.float32)
        parents = np.int32([-1, 0, 0, 1, 1, 2])
        for i in range(1, n):  # the first children's borders exactly
            p, q = target[parents[i], drafts[i]], 1.0 if certain else draft[parents[i], drafts[i]]
            if q > 0 and p < q and rng.rand() < 0.7 and (p / q) * 1024 == int((p / q) * 1024):
                accept[i] = p / q
        row = np.cumsum(target[rng.randint(0, n)])
        sample = np.float32([min(row[rng.randint(0, vocab)], 1 - 2.0 ** -24)])
        check_verify([n], vocab, certain, target=target, draft=draft, drafts=drafts, parents=parents, accept=accept, sample=sample)
    one_hot = np.eye(16, dtype=np.float32)[[3, 5, 7, 9, 11, 13]]  # nothing is left: the target's own
    for s in (0.0, 0.5, 1 - 2.0 ** -24):
        check_verify([6], 16, certain, target=one_hot, draft=None if certain else one_hot, parents=np.int32([-1, 0, 1, 2, 3, 4]),
                     drafts=np.int32([0, 3, 5, 7, 9, 2]), accept=np.full(6, 0.999, np.float32), sample=np.float32([s]))


def test_verify_follows_the_target():
    """What comes out as the first token is distributed as the target says, whatever is drafted: 20000 requests of one
    root and three children; each token's share is within 5 standard deviations, sqrt(p (1 - p) / 20000)."""
    rng = np.random.RandomState(11)
    n, vocab = 16000, 12
    p, q = probs(rng, 1, vocab, 1.0), probs(rng, 1, vocab, 1.0)
    parents = np.tile(np.int32([-1, 0, 0, 0]), n)
    for certain in (False, True):
        drafts = rng.choice(vocab, 4 * n, p=q[0] / q[0].sum()).astype(np.int32)
        if certain:
            drafts = np.tile(np.int32([0, 4, 7, 1]), n)
        target = np.broadcast_to(p, (4 * n, vocab)).copy()
        draft = None if certain else gpu(np.broadcast_to(q, (4 * n, vocab)).copy())
        _, tokens, counts = mx.kv_verify_drafts(gpu(target), gpu(drafts), gpu(parents), gpu(np.arange(n + 1, dtype=np.int32) * 4),
                                                gpu(rng.rand(4 * n).astype(np.float32)), gpu(rng.rand(n).astype(np.float32)),
                                                draft_probs=draft)
        ok()
        share = np.bincount(tokens.view(n, 4)[:, 0].cpu().numpy(), minlength=vocab) / n
        assert (np.abs(share - p[0]) <= 5 * np.sqrt(p[0] * (1 - p[0]) / n)).all()
        assert 0.2 < float((counts > 1).float().mean()) < 1


def test_verify_broken_contracts():
    rng = np.random.RandomState(4)
    target = probs(rng, 8, 50)
    good = dict(drafts=[0, 3, 4, 5, 0, 3, 4, 5], parents=[-1, 0, 1, 2, -1, 0, 1, 2], q_start=[0, 4, 8])

    def call(target=target, **kw):
        a = dict(good, **kw)
        out = mx.kv_verify_drafts(gpu(target), gpu(np.int32(a["drafts"])), gpu(np.int32(a["parents"])), gpu(np.int32(a["q_start"])),
                                  gpu(np.full(8, 0.5, np.float32)), gpu(np.full(2, 0.5, np.float32)))
        return [x.cpu().numpy() for x in out]
    whole = call()
    ok()
    for kw in (dict(drafts=[0, 50, 4, 5, 0, 3, 4, 5]), dict(drafts=[0, 3, -1, 5, 0, 3, 4, 5]), dict(parents=[0, 0, 1, 2, -1, 0, 1, 2]),
               dict(parents=[-1, 0, 2, 2, -1, 0, 1, 2]), dict(parents=[-1, -2, 1, 2, -1, 0, 1, 2]),
               dict(parents=[-1, 2147483647, 1, 2, -1, 0, 1, 2])):
        path, tokens, counts = call(**kw)
        reported()
        assert counts.tolist() == [0, whole[2][1]] and (path[:4] == -1).all() and (tokens[:4] == -1).all()
        assert np.array_equal(path[4:], whole[0][4:]) and np.array_equal(tokens[4:], whole[1][4:])
    for q_start in ([0, 4, 9], [0, -1, 8], [5, 4, 8], [-3, 4, 8], [0, 2147483647, -2147483648]):
        _, _, counts = call(q_start=q_start)
        reported()
        assert counts[0] in (0, whole[2][0]) and counts[1] in (0, whole[2][1])
    for odd in (np.nan, np.inf, -0.5, 2.5):
        bad = target.copy()
        bad[:, 49] = odd
        path, tokens, counts = call(target=bad)
        reported()
        bad[:, 49] = 0
        same = call(target=bad)
        ok()
        assert np.array_equal(path, same[0]) and np.array_equal(tokens, same[1])
    path, tokens, counts = call(target=np.zeros_like(target))
    reported()
    assert counts.tolist() == [1, 1] and (tokens == -1).all() and path[0] == path[4] == 0


@pytest.mark.parametrize("vocab", [1000, 1 << 20])
def test_verify_rows_that_are_no_distributions(vocab):
    """Entries that are probabilities each, but whose sums are not near 1: a token of the vocabulary, or none."""
    for value in (1.9, 1.0, 1e-3):
        target = torch.full((3, vocab), value, device="cuda")
        draft = torch.full((3, vocab), 1e-6, device="cuda")
        for q in (None, draft):
            tokens = torch.full((3,), 77777777, dtype=torch.int32, device="cuda")
            _, _, counts = mx.kv_verify_drafts(target, gpu(np.int32([0, 5, 6])), gpu(np.int32([-1, 0, 1])), gpu(np.int32([0, 3])),
                                               gpu(np.full(3, 0.5, np.float32)), gpu(np.float32([0.7])), draft_probs=q, tokens=tokens)
            mx.mx_check()
            n = int(counts)
            assert 1 <= n <= 3 and all(-1 <= t < vocab for t in tokens.tolist()) and all(t == -1 for t in tokens.tolist()[n:])


# ------------------------------------------------------------------ compaction
def check_compact(context, nodes, paths, p, kv_heads, d, elem, seed=0, spread=1.5, pad=0, scales=None):
    rng = np.random.RandomState(seed)
    context, nodes = np.asarray(context), np.asarray(nodes)
    lengths = (context + nodes).astype(np.int32)
    held = -(-lengths // p)
    blocks = int(held.sum()) + 3
    order, at = rng.permutation(blocks), starts(held)
    tables = np.full((len(nodes), int(held.max()) + 2), -1, np.int32)
    for r, n in enumerate(held):
        tables[r, :n] = order[at[r]:at[r] + n]
    path = np.full(int(nodes.sum()) + pad, -1, np.int32)
    for r, way in enumerate(paths):
        path[starts(nodes)[r]:starts(nodes)[r] + len(way)] = way
    counts = np.array([len(w) for w in paths], np.int32)
    caches, want = [], []
    for _ in range(2):
        x = rng.randn(blocks, kv_heads, p, d) * np.exp(spread * rng.randn(blocks, kv_heads, 1, 1))
        scale = np.array([[kv.scale_for(x[b, h], elem) for h in range(kv_heads)] for b in range(blocks)]).astype(np.float32)
        codes = kv.encode(x / scale[:, :, None, None].astype(np.float64), elem)
        if scales is not None:
            scales(rng, scale, codes)
        caches.append((codes, scale))
        want.append(ref.compact(path, counts, lengths, starts(nodes), tables, codes, scale, elem))
    codes, scale = [gpu(c) for c, _ in caches], [gpu(s) for _, s in caches]
    kept = mx.kv_cache_compact(gpu(path), gpu(counts), gpu(lengths), gpu(starts(nodes)), gpu(tables), *codes, *scale, elem=elem)
    ok()
    assert np.array_equal(kept.cpu().numpy(), want[0][2])
    for c, s, (wc, ws, _) in zip(codes, scale, want):
        assert np.array_equal(s.cpu().numpy(), ws)
        assert np.array_equal(c.cpu().numpy(), wc)


def random_paths(rng, nodes, keep=0.3):
    return [sorted(set([0] * (n > 0) + [i for i in range(n) if rng.rand() < keep])) for n in nodes]


@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("p,d,kv_heads", [(16, 64, 3), (16, 128, 1), (32, 128, 2), (64, 64, 5), (64, 128, 8), (128, 128, 2), (128, 64, 1)])
def test_compact(p, d, kv_heads, elem):
    rng = np.random.RandomState(p + d + elem)
    nodes = [1, 7, 0, 32, 33, 64, p, p + 1, 3 * p, 20]
    context = [0, p - 3, 5, p, 2 * p - 1, 3, p - 1, 2 * p + 5, p - 2, 0]
    check_compact(context, nodes, random_paths(rng, nodes), p, kv_heads, d, elem, seed=p)
    check_compact(context, nodes, random_paths(rng, nodes, 0.9), p, kv_heads, d, elem, seed=p + 1, pad=4)
    check_compact(context, nodes, [list(range(n)) for n in nodes], p, kv_heads, d, elem)     # all stay in place
    check_compact(context, nodes, [[n - 1] if n else [] for n in nodes], p, kv_heads, d, elem, spread=4.0)  # the last moves to the front
    check_compact(context, nodes, [[] for n in nodes], p, kv_heads, d, elem)                 # none is kept


def test_compact_most_nodes():
    rng = np.random.RandomState(1)
    check_compact([100, 7], [1024, 1024], random_paths(rng, [1024, 1024], 0.5), 16, 2, 64, mx.E4M3)


@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
def test_compact_odd_scales_and_codes(elem):
    def zeros(rng, scale, codes):  # blocks of scale 0, whatever their codes; NaN codes among the rest
        scale[rng.rand(*scale.shape) < 0.4] = 0
        codes[rng.rand(*codes.shape) < 0.05] = 0x7F

    def ends(rng, scale, codes):
        scale[:] = np.where(rng.rand(*scale.shape) < 0.5, 2.0 ** -48, 2.0 ** 48)
    rng = np.random.RandomState(3)
    nodes, context = [40, 33, 64], [10, 31, 16]
    for scales in (zeros, ends):
        check_compact(context, nodes, random_paths(rng, nodes), 16, 2, 64, elem, scales=scales)
        check_compact(context, nodes, random_paths(rng, nodes, 0.1), 16, 2, 128, elem, seed=2, scales=scales)


def test_compact_broken_contracts():
    rng = np.random.RandomState(2)
    codes = [gpu(rng.randint(0, 120, (8, 2, 16, 64)).astype(np.uint8)) for _ in range(2)]
    scale = [torch.full((8, 2), 0.5, device="cuda") for _ in range(2)]
    good = dict(path=[0, 2, 5, -1, -1, -1, -1, -1, 0, 3, -1, -1], counts=[3, 2], lengths=[20, 30], q_start=[0, 8, 12],
                tables=[[4, 1, -1], [0, 6, -1]])

    def call(which=0, bad=None, **kw):
        a = {k: gpu(np.int32(v)) for k, v in dict(good, **kw).items()}
        before, scales = [c.clone() for c in codes], [s.clone() for s in scale]
        if bad is not None:
            scales[0][bad[0], 1] = bad[1]
        kept = mx.kv_cache_compact(a["path"], a["counts"], a["lengths"], a["q_start"], a["tables"], *before, *scales)
        return kept.tolist(), before, scales
    kept, whole, _ = call()
    ok()
    assert kept == [15, 28]
    for kw in (dict(counts=[9, 2]), dict(counts=[-1, 2]), dict(counts=[4, 2]), dict(path=[0, 2, 2] + good["path"][3:]),
               dict(path=[0, 5, 2] + good["path"][3:]), dict(path=[0, 2, 8] + good["path"][3:]), dict(path=[-1, 2, 5] + good["path"][3:]),
               dict(path=[0, 2, 2147483647] + good["path"][3:]), dict(lengths=[7, 30]), dict(lengths=[49, 30]), dict(lengths=[-1, 30]),
               dict(tables=[[-1, 1, -1], [0, 6, -1]]), dict(tables=[[4, 8, -1], [0, 6, -1]]), dict(q_start=[-1, 8, 12])):
        kept, after, scales = call(**kw)
        reported()
        assert kept[1] == 28 and kept[0] == kw.get("lengths", [20])[0], kw
        for a, b, w in zip(after, codes, whole):
            assert torch.equal(a[[4, 1]], b[[4, 1]]) and torch.equal(a[[0, 6]], w[[0, 6]])
        assert all((s == 0.5).all() for s in scales)
    for q_start in ([0, 8, 13], [0, 13, 12], [0, 8, 7], [2147483647, -2147483648, 12]):
        kept, after, _ = call(q_start=q_start)
        reported()
        assert set(kept) <= {15, 28, 20, 30}
    # a scale out of range: what comes from its block is NaN, what goes into it is left out
    for odd in (float("nan"), float("inf"), -0.5, 2.0 ** 49, 2.0 ** -49):
        _, after, scales = call(bad=(1, odd))      # node 5 of the first request, place 17
        reported()
        assert (after[0][4, 1, 14] == 0x7F).all() and torch.equal(after[0][4, 0], whole[0][4, 0]) and torch.equal(after[1], whole[1])
        _, after, scales = call(bad=(4, odd))
        reported()
        assert torch.equal(after[0][4, 1], codes[0][4, 1]) and torch.equal(after[0][4, 0], whole[0][4, 0])


def test_compact_codes_past_32_bits():
    """A cache of more than 4 GB: the moved tokens' codes are behind 2^32."""
    blocks, p, d, heads = 9000, 64, 128, 64
    codes = [torch.zeros((blocks, heads, p, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.ones((blocks, heads), device="cuda") for _ in range(2)]
    assert codes[0].numel() > 1 << 32
    tables = gpu(np.int32([[blocks - 1, blocks - 2]]))
    for c in codes:
        c[blocks - 2, :, 3] = 0x31
    mx.kv_cache_compact(gpu(np.int32([0, 5] + [-1] * 8)), gpu(np.int32([2])), gpu(np.int32([72])), gpu(np.int32([0, 10])), tables,
                        *codes, *scale)
    ok()
    for c in codes:
        assert (c[blocks - 1, :, 63] == 0x31).all() and int((c == 0x31).sum()) == 2 * heads * d
        assert (c[blocks - 1, :, :63] == 0).all()
