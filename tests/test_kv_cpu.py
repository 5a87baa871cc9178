"""CPU checks of the 8-bit key/value cache's entry points: every invalid argument is refused on the
host, before any launch; and of the 64-bit reference that the GPU tests compare with."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from block_scaled_precision_mx_gb300 import build as mxbuild
from tests import kv_reference as ref

FAKE = 1 << 20  # non-null, 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    mxbuild.build()
    return mx.load()


def refuses(call, ok, cases, unsupported=()):
    for kw in cases:
        assert call(**dict(ok, **kw)) == mx.MX_ERR_INVALID_ARG, kw
    for kw in unsupported:
        assert call(**dict(ok, **kw)) == mx.MX_ERR_UNSUPPORTED, kw


def test_block_tables_refuses_bad_arguments(lib):
    ok = dict(tables=FAKE, requests=4, max_blocks=8, before=FAKE, after=FAKE, free=FAKE, capacity=64, count=FAKE, p=64,
              tokens=16, q_start=FAKE, slots=FAKE, positions=FAKE, info=FAKE)

    def call(**a):
        return lib.kv_block_tables(a["tables"], a["requests"], a["max_blocks"], a["before"], a["after"], a["free"],
                                   a["capacity"], a["count"], a["p"], a["tokens"], a["q_start"], a["slots"],
                                   a["positions"], a["info"], None)
    refuses(call, ok, [{k: None} for k in ("tables", "before", "after", "free", "count", "q_start", "slots", "positions",
                                           "info")]
            + [{"tables": FAKE + 2}, {"slots": FAKE + 4}, {"requests": 0}, {"requests": 16385}, {"max_blocks": 0},
               {"max_blocks": 1 << 25}, {"capacity": 0}, {"capacity": 1 << 31}, {"p": 48}, {"p": 8}, {"p": 256},
               {"tokens": -1}, {"tokens": 1 << 31}])


def test_append_refuses_bad_arguments(lib):
    ok = dict(k=FAKE, v=FAKE, type=0, tokens=4, kst=1024, ksh=128, vst=1024, vsh=128, slots=FAKE, kc=FAKE, vc=FAKE,
              ks=FAKE, vs=FAKE, elem=0, blocks=16, kv_heads=8, p=64, d=128)

    def call(**a):
        return lib.kv_cache_append(a["k"], a["v"], a["type"], a["tokens"], a["kst"], a["ksh"], a["vst"], a["vsh"],
                                   a["slots"], a["kc"], a["vc"], a["ks"], a["vs"], a["elem"], a["blocks"], a["kv_heads"],
                                   a["p"], a["d"], None)
    refuses(call, ok, [{k: None} for k in ("k", "v", "slots", "kc", "vc", "ks", "vs")]
            + [{"k": FAKE + 8}, {"vc": FAKE + 4}, {"ks": FAKE + 2}, {"type": 2}, {"elem": 3}, {"tokens": -1},
               {"kst": 1020}, {"vsh": 4}, {"blocks": 0}, {"kv_heads": 0}, {"kv_heads": 1025}, {"p": 24}, {"d": 96},
               {"d": 256}, {"blocks": 1 << 22, "kv_heads": 8}], [{"elem": 2}])
    assert call(**dict(ok, tokens=0, k=None, v=None, slots=None)) == mx.MX_OK  # nothing to do, nothing launched


def test_attention_refuses_bad_arguments(lib):
    ok = dict(q=FAKE, type=0, tokens=4, heads=32, qst=4096, qsh=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, elem=0,
              blocks=16, kv_heads=8, p=64, d=128, tables=FAKE, max_blocks=4, lengths=FAKE, q_start=FAKE, requests=4,
              max_q=1, scale=0.1, causal=1, window=0, out=FAKE, lse=FAKE, ws=FAKE)

    def call(**a):
        return lib.kv_attention(a["q"], a["type"], a["tokens"], a["heads"], a["qst"], a["qsh"], a["kc"], a["vc"], a["ks"],
                                a["vs"], a["elem"], a["blocks"], a["kv_heads"], a["p"], a["d"], a["tables"],
                                a["max_blocks"], a["lengths"], a["q_start"], a["requests"], a["max_q"], a["scale"],
                                a["causal"], a["window"], a["out"], a["lse"], a["ws"], None)
    refuses(call, ok, [{k: None} for k in ("q", "kc", "vc", "ks", "vs", "tables", "lengths", "q_start", "out", "lse",
                                           "ws")]
            + [{"q": FAKE + 8}, {"out": FAKE + 8}, {"ws": FAKE + 8}, {"lengths": FAKE + 2}, {"type": 5}, {"elem": 3},
               {"tokens": -1}, {"heads": 0}, {"heads": 30}, {"heads": 65536}, {"qst": 4100}, {"qsh": 4}, {"blocks": 0},
               {"kv_heads": 0}, {"p": 100}, {"d": 80}, {"max_blocks": 0}, {"max_blocks": 1 << 25}, {"requests": 0},
               {"requests": 16385}, {"max_q": -1}, {"max_q": 5}, {"scale": 0.0}, {"scale": -1.0},
               {"scale": float("nan")}, {"scale": float("inf")}, {"causal": 2}, {"window": -1}, {"window": 1 << 31}],
            [{"elem": 2}])
    assert call(**dict(ok, tokens=0, max_q=0, q=None, out=None, lse=None)) == mx.MX_OK


def test_python_entry_points_check_their_tensors():
    q = torch.zeros(2, 4, 64, dtype=torch.float32)
    codes, scale = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2)
    tables, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.kv_attention(q, codes, codes, scale, scale, tables, lens, lens, 1)
    with pytest.raises(ValueError):
        mx.kv_cache_append(q, q, lens, codes, codes, scale, scale)
    with pytest.raises(ValueError):
        mx.kv_block_tables(tables.long(), lens, lens, lens, lens, 1, 16)
    with pytest.raises(ValueError):
        mx.kv_block_tables(tables, lens[:1], lens, lens, lens, 1, 16)


# ------------------------------------------------------------------ the reference itself
@pytest.mark.parametrize("elem,kind", [(0, torch.float8_e4m3fn), (1, torch.float8_e5m2)])
def test_reference_codes_are_the_formats(elem, kind):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    values = codes.view(kind).float().numpy()
    assert np.array_equal(ref.decode_table(elem), values.astype(np.float64), equal_nan=True)
    rng = np.random.RandomState(elem)
    x = (rng.randn(20000) * 2.0 ** rng.randint(-14, 9, 20000)).clip(-ref.MAX[elem], ref.MAX[elem]).astype(np.float32)
    finite = values[np.isfinite(values)]
    x = np.concatenate([x, finite, (np.sort(finite)[1:] + np.sort(finite)[:-1]) / 2]).astype(np.float32)  # and all ties
    want = torch.from_numpy(x).to(kind).view(torch.uint8).numpy()
    got = ref.encode(x, elem)
    assert np.array_equal(ref.decode_table(elem)[got], ref.decode_table(elem)[want])
    assert ref.encode(np.array([np.inf, -1e30, np.nan]), elem)[2] == 0x7F
    assert list(ref.decode_table(elem)[ref.encode(np.array([np.inf, -1e30]), elem)]) == [ref.MAX[elem], -ref.MAX[elem]]


def test_reference_tables_small():
    t = np.array([[5, 7, -1], [3, -1, -1], [-1, -1, -1]], np.int32)
    free = np.array([0, 1, 2, -1, -1, -1, -1, -1], np.int32)
    # request 0 shrinks from two blocks to one, 1 grows within its block, 2 starts with two
    out = ref.tables(t, [20, 3, 0], [4, 5, 17], free, 3, 20, 16)
    assert out[0].tolist() == [[5, 7, -1], [3, -1, -1], [7, 2, -1]]
    assert out[1][:2].tolist() == [0, 1] and out[5].tolist() == [2, 0]
    assert out[2].tolist() == [0, 0, 2, 19]
    assert out[3].tolist() == [51, 52] + list(range(112, 128)) + [32, -1]
    assert out[4].tolist() == [3, 4] + list(range(17)) + [-1]
