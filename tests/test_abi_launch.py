"""The binding's choice of device and stream (CPU only: devices are stood in for)."""
import pytest
import torch

lx = pytest.importorskip("cross_entropy_tv_amd", reason="HIP library not built")


class Devices:
    """torch.cuda's current device, changed and restored by torch.cuda.device as a context."""

    def __init__(self, monkeypatch, current=0):
        self.current = current
        devices = self

        class Guard:
            def __init__(self, index):
                self.index = index

            def __enter__(self):
                self.before, devices.current = devices.current, self.index

            def __exit__(self, *exc):
                devices.current = self.before

        monkeypatch.setattr(lx, "_current_device", lambda: self.current)
        monkeypatch.setattr(lx, "_current_raw_stream", lambda index: 1000 + index)
        monkeypatch.setattr(torch.cuda, "device", Guard)


class Stream:
    def __init__(self, index, handle):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


def test_the_tensors_device_is_current_for_the_call(monkeypatch):
    devices = Devices(monkeypatch)
    for stream, ptr in ((None, 1001), (Stream(1, 77), 77), (78, 78)):
        with lx._Launch(torch.device("cuda:1"), stream) as at:
            assert devices.current == 1 and at.ptr == ptr
        assert devices.current == 0
    with pytest.raises(RuntimeError, match="inside"):
        with lx._Launch(torch.device("cuda:1"), None):
            raise RuntimeError("inside")
    assert devices.current == 0


def test_a_stream_that_is_none_leaves_the_device_as_it_was(monkeypatch):
    devices = Devices(monkeypatch)
    with pytest.raises((TypeError, ValueError)):
        with lx._Launch(torch.device("cuda:1"), "no stream"):
            pass
    assert devices.current == 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Its kernels would run on that device, on this one's memory."""
    devices = Devices(monkeypatch)
    with pytest.raises(ValueError, match="stream must be one of cuda:1"):
        with lx._Launch(torch.device("cuda:1"), Stream(0, 77)):
            pass
    assert devices.current == 0
