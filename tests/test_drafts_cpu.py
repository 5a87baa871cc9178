"""CPU checks of the entry points for drafted tokens and of the norm and rotation: every invalid argument is refused on
the host, before any launch; and of the 64-bit reference that the GPU tests compare with."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from block_scaled_precision_mx_gb300 import build as mxbuild
from tests import drafts_reference as ref
from tests.test_kv_cpu import FAKE, refuses


@pytest.fixture(scope="module")
def lib():
    mxbuild.build()
    return mx.load()


NORM = dict(q=FAKE, k=FAKE, type=0, tokens=4, heads=32, kv_heads=8, d=128, qst=4096, qsh=128, kst=1024, ksh=128, qw=FAKE,
            kw=FAKE, wf32=0, table=FAKE, places=100, rot=128, pos=FAKE, eps=1e-6, inter=0, qo=FAKE, ko=FAKE, qost=4096,
            qosh=128, kost=1024, kosh=128)
NORM_BAD = ([{k: None} for k in ("q", "k", "qw", "kw", "table", "pos", "qo", "ko")]
            + [{"q": FAKE + 8}, {"ko": FAKE + 4}, {"table": FAKE + 8}, {"pos": FAKE + 2}, {"qw": FAKE + 1},
               {"wf32": 1, "kw": FAKE + 2}, {"wf32": 2}, {"type": 2}, {"tokens": -1}, {"tokens": 1 << 31}, {"heads": 0},
               {"heads": 65536}, {"kv_heads": -1}, {"d": 0}, {"d": 4}, {"d": 100}, {"d": 264}, {"qst": 4100}, {"ksh": 4},
               {"kosh": 12}, {"places": 0}, {"places": 1 << 31}, {"rot": 8}, {"rot": 24}, {"rot": 144}, {"rot": -16},
               {"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")}, {"inter": 2}])


def test_norm_refuses_bad_arguments(lib):
    def call(**a):
        return lib.qk_norm_rope(a["q"], a["k"], a["type"], a["tokens"], a["heads"], a["kv_heads"], a["d"], a["qst"], a["qsh"],
                                a["kst"], a["ksh"], a["qw"], a["kw"], a["wf32"], a["table"], a["places"], a["rot"], a["pos"],
                                a["eps"], a["inter"], a["qo"], a["ko"], a["qost"], a["qosh"], a["kost"], a["kosh"], None)
    refuses(call, NORM, NORM_BAD)
    assert call(**dict(NORM, tokens=0, q=None, k=None, qo=None, ko=None)) == mx.MX_OK  # nothing to do, nothing launched


def test_norm_backward_refuses_bad_arguments(lib):
    ok = dict(NORM, dq=FAKE, dk=FAKE, dqst=4096, dqsh=128, dkst=1024, dksh=128, dqw=FAKE, dkw=FAKE, ws=FAKE)

    def call(**a):
        return lib.qk_norm_rope_backward(a["qo"], a["ko"], a["q"], a["k"], a["type"], a["tokens"], a["heads"], a["kv_heads"],
                                         a["d"], a["qost"], a["qosh"], a["kost"], a["kosh"], a["qst"], a["qsh"], a["kst"],
                                         a["ksh"], a["qw"], a["kw"], a["wf32"], a["table"], a["places"], a["rot"], a["pos"],
                                         a["eps"], a["inter"], a["dq"], a["dk"], a["dqst"], a["dqsh"], a["dkst"], a["dksh"],
                                         a["dqw"], a["dkw"], a["ws"], None)
    refuses(call, ok, NORM_BAD + [{k: None} for k in ("dq", "dk", "dqw", "dkw", "ws")]
            + [{"dq": FAKE + 8}, {"dkst": 4}, {"dqw": FAKE + 2}, {"ws": FAKE + 8}])
    assert mx.load().qk_norm_rope_workspace_bytes(100) == 0 and mx.load().qk_norm_rope_workspace_bytes(128) > 0


def test_trees_refuse_bad_arguments(lib):
    far = 1 << 24
    ok = dict(parents=FAKE, tokens=40, lengths=FAKE, q_start=FAKE, requests=4, most=16, window=0, mask=far, words=1, pos=far + 4096)

    def call(**a):
        return lib.kv_draft_trees(a["parents"], a["tokens"], a["lengths"], a["q_start"], a["requests"], a["most"], a["window"],
                                  a["mask"], a["words"], a["pos"], None)
    refuses(call, ok, [{k: None} for k in ("parents", "lengths", "q_start", "mask", "pos")]
            + [{"parents": FAKE + 2}, {"mask": FAKE + 4}, {"tokens": -1}, {"tokens": 1 << 31}, {"requests": 0},
               {"requests": 16385}, {"most": 41}, {"most": -1}, {"tokens": 4000, "most": 1025, "words": 17}, {"words": 0},
               {"words": 17}, {"tokens": 400, "most": 65}, {"window": -1}, {"window": 1 << 31}, {"pos": FAKE}, {"pos": FAKE + 156},
               {"mask": FAKE - 312}, {"lengths": far + 8}, {"q_start": far + 4096 + 156}])
    assert call(**dict(ok, tokens=0, most=0, parents=None, mask=None, pos=None)) == mx.MX_OK


def test_tree_attention_refuses_bad_arguments(lib):
    ok = dict(q=FAKE, type=0, tokens=40, heads=32, qst=4096, qsh=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, elem=0,
              blocks=16, kv_heads=8, p=64, d=128, tables=FAKE, max_blocks=4, lengths=FAKE, q_start=FAKE, requests=4,
              max_q=16, mask=FAKE, words=1, pos=FAKE, scale=0.1, window=5, out=FAKE, lse=FAKE, ws=FAKE)

    def call(**a):
        return lib.kv_tree_attention(a["q"], a["type"], a["tokens"], a["heads"], a["qst"], a["qsh"], a["kc"], a["vc"], a["ks"],
                                     a["vs"], a["elem"], a["blocks"], a["kv_heads"], a["p"], a["d"], a["tables"],
                                     a["max_blocks"], a["lengths"], a["q_start"], a["requests"], a["max_q"], a["mask"],
                                     a["words"], a["pos"], a["scale"], a["window"], a["out"], a["lse"], a["ws"], None)
    refuses(call, ok, [{k: None} for k in ("q", "kc", "vc", "ks", "vs", "tables", "lengths", "q_start", "mask", "pos", "out",
                                           "lse", "ws")]
            + [{"mask": FAKE + 4}, {"pos": FAKE + 2}, {"words": 0}, {"words": 17}, {"tokens": 400, "max_q": 65},
               {"tokens": 4000, "max_q": 1025, "words": 16}, {"max_q": 41}, {"heads": 30}, {"window": -1}, {"scale": 0.0},
               {"type": 5}, {"ws": FAKE + 8}], [{"elem": 2}])
    assert call(**dict(ok, tokens=0, max_q=0, q=None, out=None, lse=None, mask=None, pos=None)) == mx.MX_OK


def test_verify_refuses_bad_arguments(lib):
    ok = dict(target=FAKE, tst=1000, draft=FAKE, dst=1000, vocab=1000, drafts=FAKE, parents=FAKE, tokens=40, q_start=FAKE,
              requests=4, most=16, accept=FAKE, sample=FAKE, path=1 << 24, out=(1 << 24) + 4096, counts=(1 << 24) + 8192)

    def call(**a):
        return lib.kv_verify_drafts(a["target"], a["tst"], a["draft"], a["dst"], a["vocab"], a["drafts"], a["parents"],
                                    a["tokens"], a["q_start"], a["requests"], a["most"], a["accept"], a["sample"], a["path"],
                                    a["out"], a["counts"], None)
    refuses(call, ok, [{k: None} for k in ("target", "drafts", "parents", "q_start", "accept", "sample", "path", "out", "counts")]
            + [{"target": FAKE + 2}, {"draft": FAKE + 1}, {"path": FAKE + 2}, {"vocab": 0}, {"vocab": (1 << 20) + 1, "tst": 1 << 21, "dst": 1 << 21},
               {"tst": 999}, {"dst": 999}, {"tokens": -1}, {"requests": 0}, {"requests": 16385}, {"most": 41}, {"most": -1},
               {"tokens": 4000, "most": 1025}, {"path": FAKE}, {"out": FAKE + 156}, {"counts": FAKE - 12},
               {"drafts": (1 << 24) + 156}, {"sample": (1 << 24) + 8192 + 12}])


def test_compact_refuses_bad_arguments(lib):
    far = 1 << 24
    ok = dict(path=FAKE, counts=FAKE, tokens=40, lengths=FAKE + 64, q_start=FAKE, requests=4, tables=FAKE, max_blocks=8, kc=FAKE,
              vc=FAKE, ks=FAKE, vs=FAKE, elem=0, blocks=16, kv_heads=8, p=64, d=128, kept=far)

    def call(**a):
        return lib.kv_cache_compact(a["path"], a["counts"], a["tokens"], a["lengths"], a["q_start"], a["requests"], a["tables"],
                                    a["max_blocks"], a["kc"], a["vc"], a["ks"], a["vs"], a["elem"], a["blocks"], a["kv_heads"],
                                    a["p"], a["d"], a["kept"], None)
    refuses(call, ok, [{k: None} for k in ("path", "counts", "lengths", "q_start", "tables", "kc", "vc", "ks", "vs", "kept")]
            + [{"kept": FAKE}, {"kept": FAKE + 12}, {"kept": FAKE + 64}, {"kept": FAKE + 52}, {"kept": FAKE + 124}, {"kept": FAKE - 12}, {"kc": FAKE + 8}, {"vs": FAKE + 2},
               {"tokens": -1}, {"requests": 0}, {"requests": 16385}, {"max_blocks": 0}, {"max_blocks": 1 << 25}, {"elem": 3},
               {"blocks": 0}, {"kv_heads": 0}, {"p": 24}, {"d": 96}], [{"elem": 2}])


def test_python_entry_points_check_their_tensors():
    x, w, i32 = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.ones(64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.qk_norm_rope(x, x, w, w, None, None)                      # not CUDA tensors
    with pytest.raises(ValueError):
        mx.qk_norm_rope(x.float(), x.float(), w, w, None, None)
    with pytest.raises(ValueError):
        mx.kv_draft_trees(i32, i32, i32, 2)                          # q_start
    with pytest.raises(ValueError):
        mx.kv_draft_trees(i32.long(), i32, torch.zeros(3, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        mx.kv_verify_drafts(torch.zeros(2, 9), i32, i32, torch.zeros(3, dtype=torch.int32), torch.zeros(2), torch.zeros(2))
    codes, scale = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2)
    with pytest.raises(ValueError):
        mx.kv_cache_compact(i32, i32, i32, i32, torch.zeros(2, 1, dtype=torch.int32), codes, codes, scale, scale)


# ------------------------------------------------------------------ the reference itself
def test_reference_trees_small():
    mask, positions = ref.trees(np.array([-1, 0, 0, 2, 1]), [9], [0, 5], 1, 0, 6)
    assert mask[:, 0].tolist() == [1, 3, 5, 13, 19, 0] and positions.tolist() == [4, 5, 5, 6, 6, -1]
    assert ref.trees(np.array([-1, 0, 0, 2, 1]), [9], [0, 5], 1, 2, 5)[0][:, 0].tolist() == [1, 3, 5, 12, 18]


def test_reference_verify_small():
    target = np.array([[0.5, 0.25, 0.25], [0.0, 0.0, 1.0], [0.5, 0.5, 0.0]])
    # the first child's token has 1/2: accepted below it; behind it only token 2 is left
    path, tokens, counts = ref.verify(target, None, [0, 0, 1], [-1, 0, 0], [0, 3], [0, 0.49, 0], [0.3])
    assert path.tolist() == [0, 1, -1] and tokens.tolist() == [0, 2, -1] and counts.tolist() == [2]
    # not at it; then the second's 1/4 of the 1/2 that is left: accepted below 1/2, its own next token at 0.6 is 1
    path, tokens, counts = ref.verify(target, None, [0, 0, 1], [-1, 0, 0], [0, 3], [0, 0.5, 0.49], [0.6])
    assert path.tolist() == [0, 2, -1] and tokens.tolist() == [1, 1, -1]
    # both rejected: token 2 is all that is left
    path, tokens, counts = ref.verify(target, None, [0, 0, 1], [-1, 0, 0], [0, 3], [0, 0.5, 0.5], [0.0])
    assert path.tolist() == [0, -1, -1] and tokens.tolist() == [2, -1, -1] and counts.tolist() == [1]
    # drawn drafts: 1/2 against 3/4, rejected from 2/3 on; what is left of the target is (0, 1/8, 1/8)
    draft = np.array([[0.75, 0.125, 0.125]] * 3)
    path, tokens, counts = ref.verify(target, draft, [0, 0, 1], [-1, 0, 1], [0, 3], [0, 0.67, 0], [0.5])
    assert path.tolist() == [0, -1, -1] and tokens.tolist() == [2, -1, -1]
    path, tokens, counts = ref.verify(target, draft, [0, 0, 1], [-1, 0, 1], [0, 3], [0, 0.66, 0], [0.5])
    assert path.tolist() == [0, 1, -1] and tokens.tolist() == [0, 2, -1]  # token 1 has no chance behind node 1


def test_reference_turn_is_a_rotation():
    rng = np.random.RandomState(0)
    x, table = rng.randn(4, 2, 32), np.concatenate([np.cos(np.arange(40.)).reshape(5, 8), np.sin(np.arange(40.)).reshape(5, 8)], 1)
    for interleaved in (False, True):
        y = ref.turn(x, table, np.array([0, 4, 2, 2]), interleaved)[0]
        assert np.allclose((y ** 2).sum(2), (x ** 2).sum(2)) and np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(ref.turn(y, table, np.array([0, 4, 2, 2]), interleaved, back=True)[0], x)
