"""The ends of kv_attention's loading warps, on the CPU: the phase that each slot's barrier is waited for is the
one that the slot's last copy completes, wherever the loader stopped.  (csrc/kv_ring.cuh compiled by g++, against
a model of the barriers.)"""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_precision_mx_gb300", "csrc")


@pytest.fixture(scope="module")
def last_parity(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cc").write_text('#include "kv_ring.cuh"\nextern "C" unsigned last_parity(unsigned issued, unsigned slot, '
                               "unsigned slots) { return mxgb::kv_ring_last_parity(issued, slot, slots); }\n")
    lib = str(d / "ring.so")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", CSRC, str(d / "ring.cc"), "-o", lib])
    fn = ctypes.CDLL(lib).last_parity
    fn.restype, fn.argtypes = ctypes.c_uint, [ctypes.c_uint] * 3
    return fn


@pytest.mark.parametrize("slots", [3, 4, 5])
def test_every_copy_in_flight_is_waited_for(last_parity, slots):
    for issued in range(1, 40):
        for slot in range(min(slots, issued)):
            last = max(i for i in range(issued) if i % slots == slot)
            in_phase = last // slots                # the barrier's phase while that copy is in flight
            # a wait for a parity returns at once unless it is that of the phase in progress
            assert last_parity(issued, slot, slots) == in_phase % 2


def test_the_loaders_count_what_they_issue():
    """One count in each loader, at the copies themselves, behind the wait that may give up."""
    for name in ("kv_attention.cuh", "kv_prefill.cuh"):
        text = open(os.path.join(CSRC, name)).read()
        assert len(re.findall(r"\+\+issued;", text)) == 1
        assert len(re.findall(r"kv_ring_last_parity\(issued, i, ", text)) == 1
    text = open(os.path.join(CSRC, "kv_prefill.cuh")).read()
    gave_up, counted = text.index("!kv_wait(&raw_empty[slot]"), text.index("++issued;")
    assert gave_up < counted < text.index("mbar_arrive_expect_tx(&raw_full[slot], bytes)")


def test_whole_warps_wait_by_one_vote():
    """The kernels' roles wait through kv_wait, whose lanes agree; a wait of single lanes would let some of a warp
    give up in front of the next operation of the whole warp."""
    for name in ("kv_attention.cuh", "kv_prefill.cuh"):
        text = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"\bmbar_(?:try_)?wait\(", text):
            assert "__all_sync(0xFFFFFFFFu, " in text[m.start() - 40:m.start()], text[m.start() - 60:m.end()]
