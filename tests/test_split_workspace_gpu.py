"""The split workspace that the binding keeps for a stream: whose memory it is, and that the stream finds it zero."""
import pytest
import torch

from test_attention_workspace_gpu import owner_of
from test_paged_attention_gpu import mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_it_is_the_streams(mxq, handle, monkeypatch):  # noqa: F811
    """Made while another stream is the current one and busy: zeros are written in the order of the stream that uses them."""
    from mxfp8_activation_quant_gb300 import _lib

    monkeypatch.setattr(_lib, "_workspaces", {})
    named, busy = torch.cuda.Stream(), torch.cuda.Stream()
    work = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        for _ in range(50):
            work.random_()
        ws = _lib.workspace_for(named.cuda_stream if handle else named)
    with torch.cuda.stream(named):
        ones = int(ws.any())
    torch.cuda.synchronize()
    assert ones == 0 and owner_of(ws.data_ptr()) == named.cuda_stream


def test_the_default_streams_handle(mxq, monkeypatch):  # noqa: F811
    from mxfp8_activation_quant_gb300 import _lib

    monkeypatch.setattr(_lib, "_workspaces", {})
    with torch.cuda.stream(torch.cuda.Stream()):
        ws = _lib.workspace_for(0)
    torch.cuda.synchronize()
    assert owner_of(ws.data_ptr()) == 0 and not bool(ws.any())
