"""The scales of a key/value cache that kv_cache_append did not write, on the GPU: blocks of scale 0, blocks that
a row does not see with any scale at all, the ends of the range, and products of a row's and a block's scale
that leave FP32.  Few rows (1, 4) and prompts (40, 100 queries), against the 64-bit reference and its tolerances."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests.test_gpu_kv import attention_case, built, check_attention, gpu, run_attention  # noqa: F401

pytestmark = pytest.mark.gpu

QUERIES = [1, 4, 40, 100]


@pytest.mark.parametrize("queries", QUERIES)
@pytest.mark.parametrize("d,p,elem", [(128, 64, 0), (64, 16, 1), (128, 128, 0)])
def test_a_scale_of_zero_is_a_block_of_zeros(d, p, elem, queries):
    """Whatever its codes are; of the keys, of the values, of both, and of every block."""
    rng = np.random.RandomState(queries + p)
    lens = [300, 150, 129]
    for which in (("ks",), ("vs",), ("ks", "vs")):
        c = attention_case(rng, lens, [min(queries, n) for n in lens], 4, 2, d, p, "bf16", elem)
        for n in which:
            c[n][c["tables"][0, 1], 0] = 0                       # one head of a block
            c[n][c["tables"][0, 0]] = 0
            c[n][c["tables"][1][c["tables"][1] >= 0]] = 0         # a whole request
        out, _ = check_attention(c, elem)
        if "vs" in which:
            a, b = c["q_start"][1:3]
            assert (out[a:b] == 0).all()


@pytest.mark.parametrize("scale", [float("nan"), 0.0, float("inf"), -1.0, 1e-40, 1e30])
@pytest.mark.parametrize("queries", QUERIES)
def test_scales_that_no_row_sees_do_not_matter(queries, scale):
    """Blocks of 16 in front of the window, in the tile that it begins in."""
    rng = np.random.RandomState(queries)
    lens, q = [300, 177], [queries, queries]
    c = attention_case(rng, lens, q, 4, 2, 128, 16, "bf16", 0)
    for r, n in enumerate(lens):
        first = max(0, n - queries - 30 + 1)                      # the first token that some row sees
        hidden = c["tables"][r, :first // 16]
        for n in ("ks", "vs"):
            c[n][hidden] = scale
    check_attention(c, 0, window=30)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -1.0, 2.0 ** -60, 2.0 ** 60])
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("queries", QUERIES)
def test_unusable_scales_are_reported_and_reach_only_rows_that_see_them(queries, which, scale):
    rng = np.random.RandomState(queries + 1)
    c = attention_case(rng, [300, 177], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    want = run_attention(c, 0)
    c[which][c["tables"][0, 1], 1] = scale                        # heads 2 and 3 of request 0
    out, lse = run_attention(c, 0)
    assert mx.mx_check() == mx.MX_ERR_INVALID_ARG
    assert mx.mx_check() == mx.MX_OK
    assert torch.isnan(out[:queries, 2:]).all()
    if which == "ks":
        assert torch.isnan(lse[:queries, 2:]).all()
    for got, w in zip((out, lse), want):
        assert torch.equal(got[:queries, :2], w[:queries, :2]) and torch.equal(got[queries:], w[queries:])


@pytest.mark.parametrize("queries", QUERIES)
def test_the_ends_of_the_scales_range(queries):
    """Value blocks of 2^-48 and 2^48 in one row, near-equal weights: the sum of weights keeps both."""
    rng = np.random.RandomState(queries + 2)
    c = attention_case(rng, [256, 256], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    for n, r in (("vs", 0), ("ks", 1)):
        c[n][c["tables"][r, :2]] = 2.0 ** -48
    c["vs"][c["tables"][0, 2:4]] = 2.0 ** 48
    check_attention(c, 0, scale=1e-3)


@pytest.mark.parametrize("queries", QUERIES)
def test_products_of_scales_below_the_smallest_number(queries):
    """A tiny softmax scale, tiny queries and key blocks of 2^-48: every visible token weighs the same, and
    masked ones nothing."""
    rng = np.random.RandomState(queries + 3)
    c = attention_case(rng, [200, 120], [queries, queries], 4, 2, 128, 64, "bf16", 0)
    c["ks"][c["tables"][0, 1]] = 2.0 ** -48
    check_attention(c, 0, scale=1e-37)
    check_attention(c, 0, scale=1e-37, window=20)
    c["q"] = (c["q"].double() * 2.0 ** -110).to(torch.bfloat16)
    check_attention(c, 0)
    check_attention(c, 0, scale=1e-30, window=20)


@pytest.mark.parametrize("queries", [1, 4, 17])
@pytest.mark.parametrize("elem", [0, 1])
def test_lse_beside_value_scales_of_zero(elem, queries):
    """Short requests, whose lse is small, over value blocks of scale 0, alone and beside others."""
    for seed in range(6):
        rng = np.random.RandomState(100 * queries + seed)
        lens = [*range(1, 40), 70, 100]
        c = attention_case(rng, lens, [min(queries, n) for n in lens], 6, 2, 64, 32, "f16", elem)
        c["vs"][c["tables"][:, 0]] = 0
        check_attention(c, elem)
        check_attention(c, elem, window=1)
