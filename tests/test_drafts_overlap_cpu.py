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
