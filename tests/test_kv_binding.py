"""The binding of the cache and its attention on the host: what it refuses before the library is called (stand-ins for device
tensors and for the library, so no GPU is needed)."""
import pytest

from mxfp8_activation_quant_gb300 import kv


def test_no_workspace_is_kept_for_the_per_thread_stream(monkeypatch):
    """Its handle, 2, names another stream in each thread, and launches of two threads would share the memory."""
    monkeypatch.setattr(kv, "_workspaces", {})
    monkeypatch.setattr(kv, "_capturing", lambda: False)
    with pytest.raises(ValueError, match="workspace"):
        kv._workspace(0, 2, 4096, None)
    assert not kv._workspaces
