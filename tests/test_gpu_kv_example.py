"""examples/kv_serving.py on the GPU: its steps' attention against the 64-bit reference over the cache
that they wrote, and the whole command."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from tests import kv_reference as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("kv_serving", os.path.join(ROOT, "examples", "kv_serving.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_attend_over_what_they_wrote(example):
    layer = example.Layer(256, 4, 2, 64, 30, 16, 3, 150)
    gen = torch.Generator("cuda").manual_seed(2)
    before = np.zeros(3, np.int64)
    for after in ([100, 1, 17], [101, 2, 18], [102, 40, 0], [103, 41, 60]):
        new = np.maximum(np.array(after) - before, 0)
        x = torch.randn(int(new.sum()), 256, generator=gen, device="cuda").to(torch.bfloat16)
        q, out, lse, y = layer.step(x, torch.tensor(after, dtype=torch.int32, device="cuda"), int(new.max()))
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        want, want_lse, tol, lse_tol = ref.attention(
            q.double().cpu().numpy(), *[c.cpu().numpy() for c in (*layer.codes, *layer.scale)], layer.tables.cpu().numpy(),
            np.array(after), q_start, mx.E4M3, 64 ** -0.5, True, 0)
        off = np.abs(out.double().cpu().numpy() - want)
        assert (off <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -25).all()
        assert (np.abs(lse.double().cpu().numpy() - want_lse) <= lse_tol).all()
        assert y.shape == x.shape and torch.isfinite(y).all()
        before = np.array(after)
    assert mx.mx_check() == mx.MX_OK


def test_the_command_runs(example, capsys):
    example.main(["--requests", "3", "--prompt", "70", "--steps", "4"])
    assert "blocks held" in capsys.readouterr().out
