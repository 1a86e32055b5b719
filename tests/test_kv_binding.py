"""The binding of the cache and its attention on the host: what it refuses before the library is called (stand-ins for device
tensors and for the library, so no GPU is needed)."""
import pytest
import torch

from mxfp8_activation_quant_gb300 import kv


class Device:
    """A tensor as if it were on a device."""

    def __init__(self, t, device=0):
        self.t, self.device_index, self.is_cuda = t, device, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 0x7F0000000000


class Library:
    """Counts calls, and accepts all of them."""
    calls = 0

    def mxq_paged_attention_workspace_bytes(self, *_):
        return 4096

    def call(self, *_):
        self.calls += 1
        return 0

    kv_write_mxfp8 = kv_read_bf16 = paged_attention_mxfp8 = call


@pytest.fixture
def lib(monkeypatch):
    library = Library()
    monkeypatch.setattr(kv, "_fns", lambda: library)
    monkeypatch.setattr(kv, "_device", lambda: 0)
    monkeypatch.setattr(kv, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(kv, "_capturing", lambda: False)
    return library


def arguments():
    """Of each call: every tensor that it takes, by name."""
    cache = lambda: kv.MXFP8Cache(Device(torch.zeros(4, 16, 2, 128, dtype=torch.uint8)),  # noqa: E731
                                  Device(torch.zeros(4, 16, 2, 4, dtype=torch.uint8)))
    rows = lambda: Device(torch.zeros(3, 2, 128, dtype=torch.bfloat16))  # noqa: E731
    ints = lambda *shape: Device(torch.zeros(shape, dtype=torch.int32))  # noqa: E731
    u8 = lambda *shape: Device(torch.zeros(shape, dtype=torch.uint8))  # noqa: E731
    q = lambda: Device(torch.zeros(3, 16, 128, dtype=torch.bfloat16))  # noqa: E731
    return {
        "kv_write_mxfp8": dict(k=rows(), slots=ints(3), k_cache=cache(), v=rows(), v_cache=cache()),
        "kv_read_bf16": dict(k_cache=cache(), block_table=ints(3, 4), cu_rows=ints(4), k_out=rows(), v_cache=cache(), v_out=rows(),
                             starts=ints(3)),
        "paged_attention_mxfp8": dict(q=q(), k_cache=cache(), block_table=ints(3, 4), seq_lens=ints(3), scale=0.1, v_cache=cache(),
                                      out=q(), out_q=u8(3, 2048), sf_packed=u8(4 * 64), sf_rowmajor=u8(3 * 64),
                                      sf_128x4=u8(128 * 64), lse=Device(torch.zeros(3, 16)), status=ints(4),
                                      workspace=u8(4096)),
    }


@pytest.mark.parametrize("call", list(arguments()))
def test_tensors_of_another_device_are_refused(lib, call):
    """Each of them alone, and the caches' data and scales: the launch would be on the current one."""
    getattr(kv, call)(**arguments()[call])
    assert lib.calls == 1
    for name, value in arguments()[call].items():
        for part in ((None,) if isinstance(value, Device) else ("data", "sf") if isinstance(value, kv.MXFP8Cache) else ()):
            args = arguments()[call]
            (args[name] if part is None else getattr(args[name], part)).device_index = 1
            with pytest.raises(ValueError, match="another device"):
                getattr(kv, call)(**args)
    assert lib.calls == 1


@pytest.mark.parametrize("name", ["sf_packed", "sf_rowmajor", "sf_128x4", "workspace", "status"])
def test_buffers_that_are_not_dense_are_refused(lib, name):
    """Their bytes are counted, and a view repeats or skips some: an expanded one has memory for a single element."""
    full = arguments()["paged_attention_mxfp8"][name].t
    views = [full[:1].expand(full.shape), full.repeat(2)[::2]]
    if name == "workspace":
        views.append(torch.zeros(1024))  # (not bytes)
    if name == "status":
        views.append(torch.zeros(0, dtype=torch.int32))
    for view in views:
        args = arguments()["paged_attention_mxfp8"]
        args[name] = Device(view)
        with pytest.raises(AssertionError):
            kv.paged_attention_mxfp8(**args)
    assert lib.calls == 0


def test_no_workspace_is_kept_for_the_per_thread_stream(monkeypatch):
    """Its handle, 2, names another stream in each thread, and launches of two threads would share the memory."""
    monkeypatch.setattr(kv, "_workspaces", {})
    monkeypatch.setattr(kv, "_capturing", lambda: False)
    with pytest.raises(ValueError, match="workspace"):
        kv._workspace(0, 2, 4096, None)
    assert not kv._workspaces
