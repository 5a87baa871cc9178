"""examples/kv_serving.py when the cache runs out of blocks, on the GPU: the step raises, nothing has changed, and the
requests go on once one of them has left."""
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests.test_gpu_kv_example import example  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_step_without_blocks_stops(example):  # noqa: F811
    layer = example.Layer(256, 4, 2, 64, 6, 16, 3, 150)
    gen = torch.Generator("cuda").manual_seed(3)

    def step(after, tokens, most):
        x = torch.randn(tokens, 256, generator=gen, device="cuda").to(torch.bfloat16)
        return layer.step(x, torch.tensor(after, dtype=torch.int32, device="cuda"), most)
    step([40, 16, 1], 57, 40)                                     # 3 + 1 + 1 of 6 blocks
    before = [t.clone() for t in (*layer.codes, *layer.scale, layer.tables, layer.free, layer.free_count, layer.lengths)]
    with pytest.raises(RuntimeError, match="1 cache blocks are missing"):
        step([49, 17, 2], 11, 9)                                  # two more, one is left
    now = (*layer.codes, *layer.scale, layer.tables, layer.free, layer.free_count, layer.lengths)
    assert all(torch.equal(a, b) for a, b in zip(before, now))
    out = step([49, 17, 0], 10, 9)[3]                             # the third leaves
    assert torch.isfinite(out).all() and layer.free_count.item() == 0
    assert mx.mx_check() == mx.MX_OK
