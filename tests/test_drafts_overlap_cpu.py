"""CPU checks of the entry points for drafted tokens: outputs that share bytes with an input, or with each other, are
refused on the host, before any launch."""
import pytest

import block_scaled_precision_mx_gb300 as mx
from block_scaled_precision_mx_gb300 import build as mxbuild

GAP = 1 << 24  # every tensor of a call by itself, unless a case says otherwise


@pytest.fixture(scope="module")
def lib():
    mxbuild.build()
    return mx.load()


def apart(names):
    return {n: GAP * (i + 1) for i, n in enumerate(names)}


def refused(call, ok, cases):
    """(The call without a case would be launched; no GPU is here to do so, nor may one read these addresses.)"""
    for kw in cases:
        assert call(**dict(ok, **kw)) == mx.MX_ERR_INVALID_ARG, kw


def test_verify(lib):
    ok = dict(apart(["target", "draft", "drafts", "parents", "q_start", "accept", "sample", "path", "out", "counts"]), tokens=40, tst=1000,
              dst=1024)

    def call(**a):
        return lib.kv_verify_drafts(a["target"], a["tst"], a["draft"], a["dst"], 1000, a["drafts"], a["parents"], a["tokens"],
                                    a["q_start"], 4, 16, a["accept"], a["sample"], a["path"], a["out"], a["counts"], None)
    last = 4 * (39 * 1000 + 999)
    refused(call, ok, [{o: ok[i]} for o in ("path", "out", "counts") for i in ("target", "draft", "drafts", "parents", "q_start", "accept", "sample")]
            + [{"path": ok["target"] + last}, {"out": ok["target"] - 156}, {"counts": ok["draft"] + 4 * (39 * 1024 + 999)},
               {"counts": ok["draft"] + 4 * (5 * 1024 + 997)}, {"path": ok["out"]}, {"path": ok["out"] + 156}, {"counts": ok["path"] + 156},
               {"out": ok["counts"] - 156}])


def test_trees(lib):
    ok = apart(["parents", "lengths", "q_start", "mask", "pos"])

    def call(**a):
        return lib.kv_draft_trees(a["parents"], 40, a["lengths"], a["q_start"], 4, 16, 0, a["mask"], 2, a["pos"], None)
    refused(call, ok, [{"pos": ok["mask"]}, {"pos": ok["mask"] + 636}, {"mask": ok["pos"] - 632}, {"mask": ok["pos"] + 152},
                       {"pos": ok["parents"] + 156}, {"mask": ok["q_start"] + 16}])


# tokens 4, 32 + 8 heads of 128, contiguous: 32768 and 8192 bytes; 100 positions of 128 angles
NORM = dict(tokens=4, heads=32, kv_heads=8, d=128, wf32=0, qst=4096, kst=1024, qost=4096, kost=1024)


def test_norm(lib):
    ok = dict(NORM, **apart(["q", "k", "qw", "kw", "table", "pos", "qo", "ko"]))

    def call(**a):
        return lib.qk_norm_rope(a["q"], a["k"], 0, a["tokens"], a["heads"], a["kv_heads"], a["d"], a["qst"], 128, a["kst"], 128, a["qw"],
                                a["kw"], a["wf32"], a["table"], 100, 128, a["pos"], 1e-6, 0, a["qo"], a["ko"], a["qost"], 128,
                                a["kost"], 128, None)
    refused(call, ok, [{"qo": ok[i]} for i in ("k", "qw", "kw", "table", "pos", "ko")] + [{"ko": ok[i]} for i in ("q", "qw", "kw", "table", "pos")]
            + [{"qo": ok["q"] + 16}, {"qo": ok["q"] - 16}, {"qo": ok["q"] + 32768 - 16}, {"qo": ok["q"], "qost": 5120},
               {"qst": 5120, "qo": ok["q"] + 256}, {"ko": ok["k"], "kost": 2048}, {"qo": ok["table"] + 4 * 100 * 128 - 16},
               {"qo": ok["qw"] + 240}, {"wf32": 1, "qo": ok["qw"] + 496}, {"k": ok["q"], "qo": ok["q"]},
               {"qo": ok["ko"] - 32768 + 16}, {"qost": 4088}, {"qost": 0}, {"kost": 8}])


def test_norm_backward(lib):
    ok = dict(NORM, **apart(["gq", "gk", "q", "k", "qw", "kw", "table", "pos", "qo", "ko", "dqw", "dkw", "ws"]))

    def call(**a):
        return lib.qk_norm_rope_backward(a["gq"], a["gk"], a["q"], a["k"], 0, a["tokens"], a["heads"], a["kv_heads"], a["d"], 4096, 128,
                                         1024, 128, a["qst"], 128, a["kst"], 128, a["qw"], a["kw"], a["wf32"], a["table"], 100, 128,
                                         a["pos"], 1e-6, 0, a["qo"], a["ko"], a["qost"], 128, a["kost"], 128, a["dqw"], a["dkw"], a["ws"],
                                         None)
    inputs = ("gq", "gk", "q", "k", "qw", "kw", "table", "pos")
    refused(call, ok, [{o: ok[i]} for o in ("dqw", "dkw", "ws") for i in inputs + ("qo", "ko")]
            + [{"qo": ok[i]} for i in ("gk", "k", "qw", "kw", "table", "pos", "ko")] + [{"ko": ok[i]} for i in ("gq", "q", "qw", "table", "pos")]
            + [{"qo": ok["gq"] + 16}, {"qo": ok["q"] - 16}, {"qo": ok["gq"], "qost": 5120}, {"ko": ok["gk"], "kost": 2048},
               {"dqw": ok["dkw"]}, {"dqw": ok["dkw"] - 508}, {"dqw": ok["ws"] + 64}, {"dkw": ok["ws"] + mx.load().qk_norm_rope_workspace_bytes(128) - 4},
               {"gk": ok["gq"], "qo": ok["gq"]}, {"qost": 0}, {"kost": 8}, {"tokens": 0, "dqw": ok["dkw"]}])


def test_compact(lib):
    inputs, outputs = ("path", "counts", "lengths", "q_start", "tables"), ("kc", "vc", "ks", "vs", "kept")
    ok = apart(inputs + outputs)
    codes, scales = 16 * 8 * 64 * 128, 4 * 16 * 8

    def call(**a):
        return lib.kv_cache_compact(a["path"], a["counts"], 40, a["lengths"], a["q_start"], 4, a["tables"], 8, a["kc"], a["vc"], a["ks"],
                                    a["vs"], 0, 16, 8, 64, 128, a["kept"], None)
    refused(call, ok, [{o: ok[i]} for o in outputs for i in inputs] + [{a: ok[b]} for a in outputs for b in outputs if a != b]
            + [{"kc": ok["vc"] + codes - 16}, {"kc": ok["vc"] - codes + 16}, {"ks": ok["vs"] + scales - 4}, {"ks": ok["vc"] + codes - 4},
               {"kept": ok["vs"] + scales - 4}, {"kept": ok["kc"] - 12}])
