"""The workspaces that the binding keeps for kv_attention, on the CPU: made once whichever threads ask, never
dropped, asked for and cleared on the stream that the call goes to, and few."""
import threading
import time

import pytest
import torch

import block_scaled_precision_mx_gb300 as mx

CPU = torch.device("cpu")


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    monkeypatch.setattr(mx, "_workspaces", {})
    monkeypatch.setattr(mx, "_workspaces_old", [])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def test_threads_that_ask_at_once_get_one_buffer(monkeypatch):
    made, zeros = [], torch.zeros

    def slow_zeros(*a, **k):
        time.sleep(0.05)
        made.append(zeros(*a, **k))
        return made[-1]
    monkeypatch.setattr(torch, "zeros", slow_zeros)
    start, got = threading.Barrier(4), []

    def work():
        start.wait()
        got.append(mx._kv_workspace(5000, CPU, 7, None))
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and all(g is made[0] for g in got)


def test_only_outgrown_buffers_are_put_aside():
    a = mx._kv_workspace(5000, CPU, 7, None)
    assert mx._workspaces_old == []
    b = mx._kv_workspace(6000, CPU, 7, None)
    assert len(mx._workspaces_old) == 1 and mx._workspaces_old[0] is a and mx._workspaces[(None, 7)] is b
