"""The workspaces that the binding keeps for kv_attention, on the CPU: made once whichever threads ask, never
dropped, asked for and cleared on the stream that the call goes to, and few."""
import threading
import time

import pytest
import torch

import block_scaled_precision_mx_gb300 as mx
from block_scaled_precision_mx_gb300 import build as mxbuild

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


class Streams:
    """torch's current stream, as the binding asks for it and changes it; `capturing` names the streams that are captured."""

    def __init__(self, monkeypatch, current, capturing=()):
        self.current, self.cleared_on, zeros, zero_ = current, [], torch.zeros, torch.Tensor.zero_
        monkeypatch.setattr(mx, "_stream", lambda s: self.current if s is None else int(s))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.current in capturing)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: pytest.fail("waits for a stream"))

        class Within:
            def __init__(inner, handle):
                inner.handle = handle

            def __enter__(inner):
                inner.before, self.current = self.current, inner.handle

            def __exit__(inner, *exc):
                self.current = inner.before
        monkeypatch.setattr(torch.cuda, "stream", Within)

        def noted(fn):
            def call(*a, **k):
                self.cleared_on.append(self.current)
                return fn(*a, **k)
            return call
        monkeypatch.setattr(torch, "zeros", noted(zeros))
        monkeypatch.setattr(torch.Tensor, "zero_", noted(zero_))


def test_a_given_streams_buffer_is_made_on_it(monkeypatch):
    s = Streams(monkeypatch, current=3)
    a = mx._kv_workspace(5000, CPU, 9, 9)
    assert s.cleared_on == [9] and s.current == 3
    assert mx._kv_workspace(5000, CPU, 9, 9) is a and mx._kv_workspace(5000, CPU, 3, None) is not a
    assert s.cleared_on == [9, 3]


def test_a_given_stream_under_capture_gets_its_own(monkeypatch):
    s = Streams(monkeypatch, current=3, capturing=(9,))
    a, b = (mx._kv_workspace(5000, CPU, 9, 9) for _ in range(2))
    assert a is not b and not mx._workspaces and s.cleared_on == [9, 9]


def test_a_capture_elsewhere_does_not_clear_a_given_streams_buffer(monkeypatch):
    s = Streams(monkeypatch, current=3, capturing=(3,))
    a = mx._kv_workspace(5000, CPU, 9, 9)
    assert s.cleared_on == [9] and mx._workspaces[(None, 9)] is a


@pytest.fixture
def calls(monkeypatch):
    """kv_attention on CPU tensors up to the library's entry, which only notes (workspace, its bytes, stream)."""
    mxbuild.build()
    real, noted = mx.load(), []

    class Library:
        kv_attention_workspace_bytes = staticmethod(lambda *a: real.kv_attention_workspace_bytes(*a))

        @staticmethod
        def kv_attention(*a):
            noted.append((a[-2], a[-1]))
            return mx.MX_OK
    monkeypatch.setattr(mx, "load", lambda: Library)
    monkeypatch.setattr(mx, "_stream", lambda s: 0 if s is None else int(s))
    monkeypatch.setattr(mx, "_at", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(mx, "_rows_of_heads", lambda x, name: (x.shape, x.data_ptr(), 0, *x.stride()[:2]))
    mx.kv_attention_workspace_bytes.cache_clear()

    def call(requests, queries, heads=8, kv_heads=2, d=128, **kw):
        q = torch.zeros(requests * queries, heads, d, dtype=torch.bfloat16)
        codes, scale = torch.zeros(1, kv_heads, 16, d, dtype=torch.uint8), torch.ones(1, kv_heads)
        ints = torch.zeros(requests + 1, dtype=torch.int32)
        mx.kv_attention(q, codes, codes, scale, scale, ints[:requests, None], ints[:requests], ints, queries, **kw)
        return noted[-1]
    yield call
    mx.kv_attention_workspace_bytes.cache_clear()


def test_handles_of_default_streams(monkeypatch, calls):
    """2 is another stream in every thread: nothing is kept for it, and a call on it brings its workspace.  1 is 0."""
    Streams(monkeypatch, current=0)
    with pytest.raises(ValueError, match="per-thread"):
        calls(2, 1, stream=2)
    assert not mx._workspaces
    ws = torch.zeros(1 << 24, dtype=torch.uint8)
    assert calls(2, 1, stream=2, workspace=ws) == (ws.data_ptr(), 2)
    shared, _ = calls(2, 1)
    assert calls(2, 1, stream=1) == (shared, 1) and len(mx._workspaces) == 1


def test_buffers_are_few_whatever_the_requests(calls):
    """One buffer a kernel and head size, however many requests calls have: prompts of 1 to 256 requests, and as
    many as there may be, then every kernel at both head sizes."""
    prompts = {calls(n, 17)[0] for n in (*range(1, 257, 5), 16384)}
    assert len(prompts) == 1 and not mx._workspaces_old
    for d in (64, 128):
        for queries in (1, 2, 4, 17, 40):
            for n in (1, 3, 300):
                calls(n, queries, heads=8, kv_heads=2, d=d)
    assert not mx._workspaces_old                                 # (the largest came first)
    mx._workspaces.clear()
    for n in (1, 300):
        for queries, d in ((1, 64), (1, 128), (4, 64), (4, 128), (40, 64), (40, 128)):
            calls(n, queries, d=d)
    kept = sum(w.numel() for w in (*mx._workspaces.values(), *mx._workspaces_old))
    assert len(mx._workspaces_old) <= 5 and kept <= 100e6          # (44 MB the largest, smaller ones together as much)


def test_strides_of_axes_of_one_do_not_matter():
    """Strides go to the library, which takes multiples of 8; torch gives an axis of one any stride."""
    class Cuda:
        is_cuda, dtype = True, torch.bfloat16

        def __init__(self, x):
            self.shape, self.dim, self.stride, self.data_ptr = x.shape, x.dim, x.stride, x.data_ptr
    x = torch.zeros(5, 64, 1, dtype=torch.bfloat16).transpose(1, 2)            # one head, stride 1
    assert x.shape == (5, 1, 64) and x.stride() == (64, 1, 1)
    assert mx._rows_of_heads(Cuda(x), "k")[3:] == (64, 0)
    x = torch.zeros(3, 3, 100, dtype=torch.bfloat16)[1:2, :1, :64]             # one token of one head
    assert mx._rows_of_heads(Cuda(x), "k")[3:] == (0, 0)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    assert mx._rows_of_heads(Cuda(x), "k")[3:] == (128, 64)
