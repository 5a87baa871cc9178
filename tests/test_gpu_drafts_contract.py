"""Drafted tokens at the ends of what their entry points document, on the GPU against the 64-bit reference."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import drafts_reference as ref
from tests import kv_reference as kv
from tests.test_gpu_drafts import check_verify, gpu, ok, probs, reported, rotation, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("tokens,heads,kv_heads", [(1, 4, 2), (5, 1, 1), (37, 8, 1), (130, 3, 3)])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_norm_in_place_and_between_each_other(order, tokens, heads, kv_heads):
    """Queries, keys and others in one buffer, by tokens or by heads first: over themselves, over the place of others, and
    over the results' gradients, which all give what separate tensors do; anything else that shares bytes is refused."""
    rng = np.random.RandomState(tokens)
    d, all_heads = 64, 2 * (heads + kv_heads) + 1
    buf = rows(rng, (tokens, all_heads, d) if order == "tokens" else (all_heads, tokens, d), torch.bfloat16).cuda()

    def split(b):
        return (b if order == "tokens" else b.transpose(0, 1)).split([heads, kv_heads, heads, kv_heads, 1], dim=1)
    q, k, q2, k2, _ = split(buf)
    w, table, positions = torch.ones(d, device="cuda"), gpu(rotation(50, d)), gpu(rng.randint(0, 50, tokens), torch.int32)
    want = mx.qk_norm_rope(q.contiguous(), k.contiguous(), w, w, table, positions)
    back = mx.qk_norm_rope_backward(q2.contiguous(), k2.contiguous(), q.contiguous(), k.contiguous(), w, w, table, positions)

    def same(got, expected):
        ok()
        assert all(torch.equal(a, b) for a, b in zip(got, expected))
    for places in ((0, 1), (2, 3), (0, 3), (2, 1)):  # (what the results may lie over: queries on queries, keys on keys)
        parts = split(buf.clone())
        same(mx.qk_norm_rope(parts[0], parts[1], w, w, table, positions, q_out=parts[places[0]], k_out=parts[places[1]]), want)
        assert torch.equal(parts[4], split(buf)[4])
        parts = split(buf.clone())
        same(mx.qk_norm_rope_backward(parts[2], parts[3], parts[0], parts[1], w, w, table, positions, dq=parts[places[0]], dk=parts[places[1]]), back)
        assert torch.equal(parts[4], split(buf)[4])
    narrow = q[:, :1], k[:, :1]
    with pytest.raises(mx.MxError):
        mx.qk_norm_rope(*narrow, w, w, table, positions, q_out=narrow[1], k_out=narrow[0])
    with pytest.raises(mx.MxError):
        mx.qk_norm_rope(*narrow, w, w, table, positions, q_out=narrow[0], k_out=narrow[0])
    with pytest.raises(mx.MxError):
        mx.qk_norm_rope(*narrow, w, w, table, positions, q_out=torch.empty(1, 1, d, dtype=q.dtype, device="cuda").expand(tokens, 1, d)
                        if tokens > 1 else narrow[1])
    with pytest.raises(mx.MxError):
        mx.qk_norm_rope_backward(q, k, q, k, w, w, table, positions, dq_weight=w)
    ok()
    assert torch.equal(mx.qk_norm_rope(q, k, w, w, table, positions)[0], want[0])  # (nothing was written)


# ------------------------------------------------------------------ verification
STARS = {  # the root's target and draft rows, and tokens that its children take in turn
    "half": ([1 / 2, 1 / 2], [1, 0], [0]), "quarter": ([1 / 4, 3 / 4], [1, 0], [0]), "sixteenth": ([1 / 16, 15 / 16], [1, 0], [0]),
    "two": ([1 / 4, 1 / 4, 1 / 2], [1 / 2, 1 / 2, 0], [0, 1, 1]), "apart": ([1 / 4, 1 / 4, 1 / 2, 0, 0], [1 / 2, 0, 0, 1 / 4, 1 / 4], [3, 0, 4]),
    "most": ([1 / 8, 1 / 8, 3 / 4], [3 / 4, 1 / 4, 0], [0, 1, 0, 0])}


@pytest.mark.parametrize("below", [0, 1])
@pytest.mark.parametrize("children", [17, 18, 22, 31, 32, 33, 63, 64, 65, 200, 1022])
@pytest.mark.parametrize("star", list(STARS))
def test_verify_siblings_of_a_narrow_draft(star, children, below):
    """One node's many children, drawn from few tokens, so that W q passes 16, 32 and more: what is used up stays so.  Rows and
    random numbers are dyadic, so that the reference's sums and products are exact, and it is exact what the next token is."""
    p, q, turns = STARS[star]
    n = 1 + below + children  # (below: the parent is a child of the root, which is accepted)
    parents = np.int32([-1] + [0] * below + [below] * children)
    drafts = np.int32([-7] + [len(p) - 1] * below + [turns[i % len(turns)] for i in range(children)])
    target, draft = np.tile(np.float32(p), (n, 1)), np.tile(np.float32(q), (n, 1))
    if below:
        target[0] = draft[0] = np.eye(len(p))[len(p) - 1]
    rng = np.random.RandomState(children)
    for trial in range(4):
        accept = (rng.randint(1 << 9, 1 << 10, n) / 1024).astype(np.float32)  # 1/2 and above: rejected by all of the rows
        if trial:  # behind the first few, which use their tokens up, any number
            accept[below + 5:] = (rng.randint(0, 1 << 10, n - below - 5) / (1024 << 4 * trial)).astype(np.float32)
        if star == "half":
            accept[1 + below] = 0.5 if trial else accept[1 + below]
        if below:
            accept[1] = 0.25
        for sample in (0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
            want = check_verify([n], len(p), False, target=target, draft=draft, drafts=drafts, parents=parents, accept=accept,
                                sample=np.float32([sample]))
            if trial == 0:
                assert int(want[2][0]) == 1 + below  # (a word on the inputs: all of them are rejected)


@pytest.mark.parametrize("share", [0.6, 0.9, 1.4, 2.6])  # of 2^-44, the unit of the sums
@pytest.mark.parametrize("rejected", [0, 1, 2, 5])
def test_verify_sums_of_many_tiny_probabilities(rejected, share):
    """2^20 - 2 entries that are alike stand in front of the two large ones, one of which the draft has.  Each is
    rounded by 2^-45 at most, and what is left of p - q, below 2^-23, by 2^-48 before: 1.2 * 2^-45 an entry."""
    vocab, n = 1 << 20, 1 + rejected
    target, draft = np.full((n, vocab), share * 2.0 ** -44, np.float32), np.zeros((n, vocab), np.float32)
    target[:, -2:], draft[:, -1] = 0.5, 1
    tiny = float(target[0, 0])
    for sample in np.float32([0, 5e-9, 1e-8, 2e-8, 3e-8]):
        path, tokens, counts = mx.kv_verify_drafts(gpu(target), gpu(np.full(n, vocab - 1, np.int32)), gpu(np.int32([-1] + [0] * rejected)),
                                                   gpu(np.int32([0, n])), gpu(np.full(n, 0.75, np.float32)), gpu(np.array([sample])),
                                                   draft_probs=gpu(draft))
        ok()
        assert counts.tolist() == [1] and path.tolist() == [0] + [-1] * rejected
        token = int(tokens[0])
        # what the running sum has to pass, and what it is before and behind the token, each within its bound; the second
        # large entry is gone with the first rejection
        mark = float(sample) * (tiny * (vocab - 2) + (0.5 if rejected else 1.0))
        off = (token + 2 + float(sample) * vocab) * 1.2 * 2.0 ** -45
        assert token * tiny <= mark + off
        assert (token + 1) * tiny + (0.5 if token >= vocab - 2 else 0) > mark - off


@pytest.mark.parametrize("certain", [True, False])
@pytest.mark.parametrize("power", [-30, -70, -100, -130])
def test_verify_tokens_that_are_next_to_impossible(power, certain):
    """Probabilities of a few times 2^power beside one large: the test is of their ratio, however small both are, and exactly
    so (of certain drafts: of the random number and the probability)."""
    rng = np.random.RandomState(-power)
    vocab, n, kept = 6, 9, []
    for trial in range(200):
        target, draft = (rng.randint(0, 64, (n, vocab)) * 2.0 ** power for _ in range(2))
        target[:, -1], draft[:, -1] = 1, 0.5
        drafts = rng.randint(0, vocab, n).astype(np.int32)
        if not certain and trial % 2:
            drafts[1] = vocab - 2  # rejected: its W leaves p - W q of the others
            target[0, vocab - 2] = 0
        accept = rng.randint(0, 64, n) * 2.0 ** (power if certain else -6)
        accept[rng.rand(n) < 0.1] = 0
        parents = np.array([-1] + [min(i - 1, rng.randint(0, 3)) for i in range(1, n)], np.int32)
        want = check_verify([n], vocab, certain, target=target.astype(np.float32), draft=None if certain else draft.astype(np.float32), drafts=drafts,
                            parents=parents, accept=accept.astype(np.float32), sample=np.float32([rng.randint(8, 64) / 64]))
        kept.append(int(want[2][0]))
    assert len(set(kept)) > 2  # (a word on the inputs)


def one_request(target, drafts, accept, sample, draft=None):
    """(path, tokens, count) of one root whose other nodes are its children."""
    n = len(drafts)
    out = mx.kv_verify_drafts(gpu(np.float32(target)), gpu(np.int32(drafts)), gpu(np.int32([-1] + [0] * (n - 1))), gpu(np.int32([0, n])),
                              gpu(np.float32(accept)), gpu(np.float32([sample])), draft_probs=None if draft is None else gpu(np.float32(draft)))
    return out[0].tolist(), out[1].tolist(), int(out[2])


@pytest.mark.parametrize("value,vocab,drawn", [(1.0, 1000, True), (1.0, 2, True), (1.0, 3, True), (1.9, 2, True), (1.0, 4095, True), (1.0, 4096, False),
                                               (1.5, 4000, False), (2.0 ** -10, 1 << 20, True), (1.0, 1 << 20, False), (1.9, 1 << 20, False)])
def test_verify_reports_sums_of_two_and_above(value, vocab, drawn):
    """The next token is still drawn as the formula says, up to a sum of 4096."""
    for sample in (0.0, 0.5, 0.75):
        path, tokens, count = one_request(np.full((1, vocab), value), [0], [0], sample)
        reported()
        assert (path, count) == ([0], 1)
        assert tokens == [int(sample * vocab) if drawn else -1]


@pytest.mark.parametrize("requests", [39, 77, 153, 400])
def test_verify_far_sums_of_many_requests(requests):
    """(With fewer CTAs a request each sums more of a row.)"""
    for vocab, value in ((1 << 20, 1.9375), (1 << 20, 2.0 ** -9), (2048, 1.9375)):
        target = torch.full((requests, vocab), value, device="cuda")
        none = gpu(np.full(requests, -1, np.int32))
        path, tokens, counts = mx.kv_verify_drafts(target, none, none, gpu(np.arange(requests + 1, dtype=np.int32)),
                                                   torch.zeros(requests, device="cuda"), torch.full((requests,), 0.5, device="cuda"))
        reported()
        assert (counts == 1).all() and (path == 0).all()
        assert (tokens == (vocab // 2 if value * vocab < 4096 else -1)).all()


def test_verify_does_not_report_sums_below_two():
    for row in ([1.9375], [1.0, 0.96875], [2.0 ** -10] * 2047, [2.0 ** -19] * ((1 << 20) - 1)):
        for rejected in (0, 3):  # (sums of the whole row, and of what is behind its first token's whole draft)
            n, draft = 1 + rejected, np.zeros((1 + rejected, len(row)))
            draft[:, 0] = 1.96875
            one_request(np.tile(row, (n, 1)), [0] * n, [1 - 2.0 ** -24] * n, 0.5, draft if rejected else None)
            ok()


@pytest.mark.parametrize("heavy", [2, 9, 500, 60000])
def test_verify_z_stays_below_two(heavy):
    """Target 1/4, 1/2 and many of 1.9, draft 3/4 and 1/4: behind the first child's rejection Z is as good as 2, and the second
    child is accepted below 1/4 / (1/4 2) = 1/2."""
    target, draft = np.full((3, 2 + heavy), 1.9), np.zeros((3, 2 + heavy))
    target[:, :2], draft[:, :2] = [0.25, 0.5], [0.75, 0.25]
    for second in (0.0, 0.2, 0.4, 0.4999, 0.5001, 0.6, 0.9):
        path, _, _ = one_request(target, [0, 0, 1], [0, 0.5, second], 0.5, draft)
        reported()
        assert path == ([0, 2, -1] if second < 0.5 else [0, -1, -1])


def test_verify_random_numbers_of_one_and_above_accept_nothing_more():
    """(Out of contract; with q above 1 as well they passed 64 bits and accepted what a smaller number rejects.)"""
    for number in (1.0, 1.25, 1.5, 1.9375):
        path, _, _ = one_request([[0.5, 0.25]] * 2, [0, 0], [0, number], 0.25, [[1.9375, 0]] * 2)
        assert path == [0, -1]
    mx.mx_check()


@pytest.mark.parametrize("certain", [True, False])
def test_verify_outputs_between_rows_of_probabilities(certain):
    """Rows apart leave room, which is no input: outputs there are no overlap, and those a row further are."""
    rng = np.random.RandomState(7)
    t, vocab, pad = 9, 601, 200
    base = [torch.zeros(t, vocab + pad, device="cuda") for _ in range(2)]
    for b in base:
        b[:, :vocab] = gpu(probs(rng, t, vocab))
    target, draft = (b[:, :vocab] for b in base)
    rest = (gpu(rng.randint(0, vocab, t), torch.int32), gpu(np.int32([-1, 0, 0, 1, 2, 0, 1, 5, 3])), gpu(np.int32([0, t])),
            gpu(rng.rand(t).astype(np.float32)), gpu(rng.rand(1).astype(np.float32)))
    draft = None if certain else draft
    want = mx.kv_verify_drafts(target, *rest, draft_probs=draft)
    words = [b.view(torch.int32) for b in base]
    got = mx.kv_verify_drafts(target, *rest, draft_probs=draft, path=words[0][3, vocab:vocab + t], tokens=words[1][0, vocab + pad - t:],
                              counts=words[0][3, vocab + t:vocab + t + 1])
    ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for place in (words[0][3, vocab - 1:vocab - 1 + t], words[0].view(-1)[vocab + pad - 1:vocab + pad - 1 + t]):
        with pytest.raises(mx.MxError):
            mx.kv_verify_drafts(target, *rest, draft_probs=draft, tokens=place)
    with pytest.raises(mx.MxError):
        mx.kv_verify_drafts(target, *rest, draft_probs=draft, path=got[0], tokens=got[0])
    ok()


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf"), -0.5, 2.0 ** 49, 2.0 ** -49])
@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("p,d,context,way", [(16, 64, 10, [0, 3, 25, 28, 29]), (16, 128, 16, [0, 17, 33]), (32, 64, 40, [2, 26, 30, 33])])
def test_compact_keeps_what_is_beside_a_block_out_of_range(p, d, context, way, elem, odd):
    """The last block's scale is no scale (for half of the heads): its tokens become NaN, and the codes, scales and moved
    tokens of the blocks that they come to are what they are with any NaN in their place."""
    rng = np.random.RandomState(p + context)
    nodes, heads = 34, 4
    held = -(-(context + nodes) // p)
    tables = rng.permutation(held + 1)[None, :held].astype(np.int32)
    path = np.int32([way + [-1] * (nodes - len(way))])[0]
    counts, lengths, q_start = np.int32([len(way)]), np.int32([context + nodes]), np.int32([0, nodes])
    assert (context + way[-1]) // p == held - 1 > (context + len(way) - 1) // p  # (moved from, not into)
    caches, want = [], []
    for _ in range(2):
        codes = rng.randint(0, 120, (held + 1, heads, p, d)).astype(np.uint8)
        scale = 2.0 ** rng.randint(-3, 4, (held + 1, heads)).astype(np.float32)
        scale[tables[0, 0], 1] = 0  # (a block of zeros among those that are moved into)
        scale[tables[0, -1], ::2] = np.nan
        want.append(ref.compact(path, counts, lengths, q_start, tables, codes, scale, elem))
        scale[tables[0, -1], ::2] = odd
        want[-1][1][tables[0, -1], ::2] = odd
        caches.append((codes, scale))
    codes, scale = [gpu(c) for c, _ in caches], [gpu(s) for _, s in caches]
    kept = mx.kv_cache_compact(gpu(path), gpu(counts), gpu(lengths), gpu(q_start), gpu(tables), *codes, *scale, elem=elem)
    reported()
    assert kept.tolist() == [context + len(way)]
    for c, s, (wc, ws, _) in zip(codes, scale, want):
        assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
        assert np.array_equal(c.cpu().numpy(), wc)
