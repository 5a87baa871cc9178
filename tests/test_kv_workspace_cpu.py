"""What the binding keeps for kv_attention calls without a workspace, on the CPU: one buffer for each
stream, grown when needed, given up after a timeout and never freed under work in flight."""
import torch

import block_scaled_precision_mx_gb300 as mx


def test_workspaces_are_kept_by_stream_and_grow(monkeypatch):
    monkeypatch.setattr(mx, "_workspaces", {})
    monkeypatch.setattr(mx, "_workspaces_old", [])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    dev = torch.device("cpu")
    a = mx._kv_workspace(5000, dev, 1, None)
    assert a.numel() == 5000 and not a.any()
    assert mx._kv_workspace(4000, dev, 1, None) is a
    assert mx._kv_workspace(4000, dev, 2, None) is not a
    b = mx._kv_workspace(6000, dev, 1, None)
    assert b.numel() == 6000 and any(x is a for x in mx._workspaces_old)
    monkeypatch.setattr(mx, "load", lambda: type("L", (), {"mx_check": staticmethod(lambda s: mx.MX_ERR_TIMEOUT)}))
    assert mx.mx_check(0) == mx.MX_ERR_TIMEOUT
    assert not mx._workspaces and any(x is b for x in mx._workspaces_old)


def test_a_capture_gets_its_own(monkeypatch):
    monkeypatch.setattr(mx, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    a, b = (mx._kv_workspace(5000, torch.device("cpu"), 1, None) for _ in range(2))
    assert a is not b and not a[:4096].any() and not mx._workspaces
