"""What the key/value cache's operators do with device inputs that break their contract, on the GPU: nothing is
read or written out of range, mx_check reports it, and what does not depend on the broken input is right; and
inputs that look broken but are not."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import kv_reference as ref
from tests.test_gpu_kv import attention_case, built, check_attention, gpu, run_attention, values  # noqa: F401

pytestmark = pytest.mark.gpu
MOST, LEAST = 2 ** 31 - 1, -2 ** 31


def reported():
    assert mx.mx_check() == mx.MX_ERR_INVALID_ARG
    assert mx.mx_check() == mx.MX_OK


# ------------------------------------------------------------------ attention
BROKEN = [{"q_start": {1: -1}}, {"q_start": {1: LEAST}}, {"q_start": {1: MOST}}, {"q_start": {1: MOST, 2: LEAST}},
          {"q_start": {1: LEAST, 2: MOST}}, {"q_start": {1: MOST, 2: LEAST + 3}}, {"q_start": {1: "past"}},
          {"q_start": {1: "fewer"}}, {"q_start": {3: MOST}}, {"q_start": {3: LEAST}}, {"q_start": {0: -5}},
          {"lens": {1: -1}}, {"lens": {1: "past"}}, {"lens": {0: MOST, 2: LEAST}}]


@pytest.mark.parametrize("broken", BROKEN, ids=str)
@pytest.mark.parametrize("queries,more", [(4, 0), (40, 0), (40, 600)])
def test_broken_lengths_and_query_starts(queries, more, broken):
    """A request whose rows or length are out of range is left out; the others' rows are right, and no other row
    of the output is touched.  (`more` empty requests: the ranges are planned by a kernel of their own.)"""
    rng = np.random.RandomState(queries)
    c = attention_case(rng, [100, 90, 80] + [0] * more, [queries] * 3 + [0] * more, 4, 2, 128, 16, "bf16", 0, q_pad=3)
    tokens, most = len(c["q"]), c["tables"].shape[1] * 16
    for name, places in broken.items():
        for i, v in places.items():
            v = {"past": tokens + 1 if name == "q_start" else most + 1, "fewer": queries - 1}.get(v, v)
            c[name][i] = v
    starts = c["q_start"].astype(np.int64)
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    args = [gpu(c[n]) for n in ("kc", "vc", "ks", "vs", "tables", "lens", "q_start")]
    mx.kv_attention(c["q"], *args, max_q_len=queries, out=out, lse=lse)
    reported()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    touched = np.zeros(tokens, bool)
    if 0 <= starts[-1] <= tokens:                                  # rows that no request has
        touched[starts[-1]:] = True
        assert (got[starts[-1]:] == 0).all() and (got_lse[starts[-1]:] == -np.inf).all()
    for r in range(3):
        a, b, n = starts[r], starts[r + 1], int(c["lens"][r])
        if not (0 <= a < b <= tokens and b - a <= queries and 0 <= n <= most):
            continue
        touched[a:b] = True
        want, want_lse, tol, lse_tol = ref.attention(
            c["q"][a:b].double().cpu().numpy(), c["kc"], c["vc"], c["ks"], c["vs"], c["tables"][r:r + 1], [n],
            [0, b - a], 0, 128 ** -0.5, True, 0)
        assert (np.abs(got[a:b] - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -25).all()
        assert (np.abs(got_lse[a:b] - want_lse) <= lse_tol).all()
    assert (got[~touched] == 7).all() and (got_lse[~touched] == 7).all()


@pytest.mark.parametrize("queries", [1, 4, 40, 100])
@pytest.mark.parametrize("p", [16, 64])
def test_table_entries_in_front_of_the_window_are_not_read(p, queries):
    """A caller with a sliding window gives back the blocks that it has left behind."""
    rng = np.random.RandomState(queries + p)
    lens = [400, 257, 20]
    for window in (1, 30, 100):
        c = attention_case(rng, lens, [min(n, queries) for n in lens], 4, 2, 128, p, "bf16", 0)
        for r, n in enumerate(lens):
            first = max(0, n - min(n, queries) - window + 1)
            c["tables"][r, :first // p] = rng.choice([-1, -5], first // p)
        check_attention(c, 0, window=window)


@pytest.mark.parametrize("bad", [-1, "past"])
@pytest.mark.parametrize("queries", [1, 4, 40, 100])
def test_a_block_out_of_range_gives_nan_where_it_is_seen(queries, bad):
    rng = np.random.RandomState(queries)
    c = attention_case(rng, [200, 130], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    want = run_attention(c, 0)
    c["tables"][0, 0] = len(c["ks"]) if bad == "past" else bad
    out, lse = run_attention(c, 0)
    reported()
    assert torch.isnan(out[:queries]).all() and torch.isnan(lse[:queries]).all()
    assert torch.equal(out[queries:], want[0][queries:]) and torch.equal(lse[queries:], want[1][queries:])


# ------------------------------------------------------------------ block tables
def test_tables_negative_blocks_are_reported():
    """A table's entry or a free block below 0 gives its tokens no place, not even the last of its block."""
    p = 16
    tables = gpu(np.array([[-1, -1], [3, -1], [-1, -1]], np.int32))
    free = gpu(np.array([5, -2, 6, 0], np.int32))
    count = torch.tensor([3], dtype=torch.int32, device="cuda")
    # request 0 goes on in an entry that was never assigned; 1 goes on in its own; 2 takes 6, then the bad one
    before, after = np.array([10, 10, 0], np.int32), np.array([16, 16, 20], np.int32)
    q_start, slots, positions, info = mx.kv_block_tables(tables, gpu(before), gpu(after), free, count, 32, p)
    reported()
    want = [-1] * 6 + list(range(3 * p + 10, 3 * p + 16)) + list(range(6 * p, 7 * p)) + [-1] * 4
    assert slots.cpu().tolist() == want
    assert q_start.cpu().tolist() == [0, 6, 12, 32] and info.cpu().tolist() == [1, 0]


def test_tables_negative_blocks_given_back_are_reported():
    tables = gpu(np.array([[2, -3]], np.int32))
    free = gpu(np.array([0, 1, -9, -9], np.int32))
    count = torch.tensor([2], dtype=torch.int32, device="cuda")
    mx.kv_block_tables(tables, gpu(np.array([20], np.int32)), gpu(np.array([0], np.int32)), free, count, 0, 16)
    reported()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("elem", [mx.E4M3, mx.E5M2])
def test_append_to_a_block_of_scale_zero(elem):
    """Its tokens are zeros, whatever their codes; zeros that follow leave it a block of zeros."""
    p, d, h = 16, 64, 2
    rng = np.random.RandomState(elem)
    codes = rng.randint(0, 100, (2, h, p, d)).astype(np.uint8)
    codes[:, :, :, 7] = 0x7F                                        # (NaN codes are zeros too)
    scale = np.zeros((2, h), np.float32)
    x = values(rng, (2, h, d), torch.bfloat16)
    x[0, 0] = 0                                                    # block 0, head 0: a token of zeros
    slots = np.array([5, p + 3], np.int64)
    kc, vc, ks, vs = gpu(codes), gpu(codes), gpu(scale), gpu(scale)
    mx.kv_cache_append(x.cuda(), x.cuda(), gpu(slots), kc, vc, ks, vs, elem=elem)
    assert mx.mx_check() == mx.MX_OK
    table = ref.decode_table(elem)
    for c, s in ((kc, ks), (vc, vs)):
        c, s = c.cpu().numpy(), s.cpu().numpy()
        for t, (block, off) in enumerate(((0, 5), (1, 3))):
            for head in range(h):
                want = ref.scale_for(x[t, head].double().numpy(), elem)
                assert s[block, head] == want
                got = table[c[block, head]] * s[block, head]
                assert (got[:off] == 0).all()
                assert np.array_equal(got[off], table[ref.encode(x[t, head].double().numpy() / want, elem)] * want)
                assert np.array_equal(c[block, head, off + 1:], codes[block, head, off + 1:])


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -1.0, 2.0 ** -60, 2.0 ** 60])
def test_append_to_a_block_of_an_unusable_scale_is_left_out_and_reported(scale):
    p, d, h = 16, 64, 2
    rng = np.random.RandomState(7)
    codes = rng.randint(0, 100, (2, h, p, d)).astype(np.uint8)
    scales = np.ones((2, h), np.float32)
    scales[0, 1] = scale
    x = values(rng, (2, h, d), torch.bfloat16).cuda()
    slots = np.array([5, p + 3], np.int64)
    want = ref.append(x.double().cpu().numpy(), slots[1:], codes, np.ones((2, h), np.float32), 0)
    kc, vc, ks, vs = gpu(codes), gpu(codes), gpu(scales), gpu(np.ones((2, h), np.float32))
    mx.kv_cache_append(x, x, gpu(slots), kc, vc, ks, vs)
    reported()
    kc, ks = kc.cpu().numpy(), ks.cpu().numpy()
    assert np.array_equal(kc[0, 1], codes[0, 1]) and np.array_equal(ks[0, 1], scales[0, 1], equal_nan=True)
    both = ref.append(x.double().cpu().numpy(), slots, codes, np.ones((2, h), np.float32), 0)
    assert np.array_equal(vc.cpu().numpy(), both[0]) and np.array_equal(vs.cpu().numpy(), both[1])
    assert np.array_equal(kc[0, 0], both[0][0, 0]) and np.array_equal(kc[1], both[0][1]) and ks[0, 0] == both[1][0, 0]


# ------------------------------------------------------------------ strides
@pytest.mark.parametrize("tokens,heads", [(1, 1), (3, 1), (1, 4)])
def test_axes_of_one_with_odd_strides(tokens, heads):
    """A tensor's axis of one may have any stride, one that is no multiple of 8 among them."""
    rng = np.random.RandomState(tokens + heads)
    c = attention_case(rng, [70], [tokens], heads, 1, 64, 16, "bf16", 0)
    c["q"] = c["q"].clone()
    check_attention(c, 0)
    st = 3 if tokens == 1 else heads * 64, 5 if heads == 1 else 64
    want = run_attention(c, 0)
    got = run_attention(dict(c, q=c["q"].as_strided(c["q"].shape, (*st, 1))), 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k = c["q"][:, :1].clone()
    slots = gpu(np.arange(tokens, dtype=np.int64))
    caches = []
    for x in (k, k.as_strided(k.shape, (3 if tokens == 1 else 64, 5, 1))):
        cache = [torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.ones(1, 1, device="cuda") for _ in range(2)]
        mx.kv_cache_append(x, x, slots, *cache)
        caches.append(cache)
    assert mx.mx_check() == mx.MX_OK
    assert all(torch.equal(a, b) for a, b in zip(*caches))
