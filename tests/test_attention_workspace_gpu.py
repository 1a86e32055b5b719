"""The workspace that the binding keeps for a stream: whose memory it is."""
import pytest
import torch

from test_paged_attention_gpu import Case, mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


def owner_of(address):
    """The stream that torch's allocator takes for the owner of an address."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= address < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("current", ["default", "side"])
def test_kept_memory_belongs_to_the_stream_it_is_used_on(mxq, current):  # noqa: F811
    """What is freed when a workspace grows goes back to the stream that its launches were on; the default stream's handle is 0."""
    from mxfp8_activation_quant_gb300 import kv

    c = Case(mxq, [40], 1, 8, 128, True, seed=62)
    k, v = c.caches()
    side, named = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.default_stream(), named, named.cuda_stream):
        raw = stream if isinstance(stream, int) else stream.cuda_stream
        kv._workspaces.pop((torch.cuda.current_device(), raw), None)
        with torch.cuda.stream(side if current == "side" else torch.cuda.default_stream()):
            mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=torch.empty_like(c.q), stream=stream)
        torch.cuda.synchronize()
        assert owner_of(kv._workspaces[torch.cuda.current_device(), raw][0]) == raw
