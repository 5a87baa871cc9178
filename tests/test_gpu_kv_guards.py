"""What the key/value cache's entry points write, on the GPU: every element that they owe, in both types and with
rows that are whole, cut, empty and NaN; and no byte outside their outputs and the workspace they asked for."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests.test_gpu_kv import attention_case, built, check_attention, gpu, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,elem", [("bf16", 0), ("f16", 0), ("f16", 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries", [3, 9, 30, 100, 300])
def test_whole_cut_empty_and_nan_rows_in_both_types(queries, d, kind, elem):
    """Long contexts whose work several CTAs share, short ones that one has, queries without tokens, and NaN in a
    value that half of the rows see."""
    rng = np.random.RandomState(queries + d)
    lens, q = [6000, 40, 0, 2500, 129], [queries, min(queries, 50), 2, queries, 129]
    c = attention_case(rng, lens, q, 4, 2, d, 64, kind, elem, q_pad=5)
    for r in (0, 3):
        at = lens[r] - queries // 2 - 1
        c["vc"][c["tables"][r, at // 64], 1, at % 64, 5] = 0x7F
        c["vc"][c["tables"][r, 1], 0, 3, d - 1] = 0x7F
    check_attention(c, elem)
