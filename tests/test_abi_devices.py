"""Calls on tensors of a device that is not the current one, on the CPU with
stand-ins for the tensors and the library."""

import pytest
import torch

from uniform_noise_diffusion_amd import binding as B


class Tensor:
    def __init__(self, dtype, device, n=1):
        self.dtype, self.index, self.shape, self.n = dtype, device, torch.Size([n]), n
        self.is_cuda, self.device = device >= 0, torch.device("cuda", max(device, 0))

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def data_ptr(self):
        return 4096


@pytest.fixture
def seen(monkeypatch):
    """The devices that were current when the library was entered."""
    seen, now = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.was

    class Stream:
        cuda_stream = 0

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, now[0], args[-1])) or B.MDLM_OK

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(B, "load", Library)
    return seen


def test_token_check_runs_on_its_tensors_device(seen):
    for dev in (0, 1):
        B.mdlm_check_tokens(Tensor(torch.int32, dev, 5), 8, Tensor(torch.int32, dev))
    assert seen == [("mdlm_check_tokens", 0, 1000), ("mdlm_check_tokens", 1, 1001)]


def test_token_check_takes_tensors_of_one_device(seen):
    with pytest.raises(ValueError, match="device"):
        B.mdlm_check_tokens(Tensor(torch.int32, 1, 5), 8, Tensor(torch.int32, 0))
    with pytest.raises(ValueError, match="device"):
        B.mdlm_check_tokens(Tensor(torch.int32, -1, 5), 8, Tensor(torch.int32, 0))
    with pytest.raises(TypeError):
        B.mdlm_check_tokens(Tensor(torch.int64, 0, 5), 8, Tensor(torch.int32, 0))
    with pytest.raises(ValueError, match="status"):
        B.mdlm_check_tokens(Tensor(torch.int32, 0, 5), 8, Tensor(torch.int32, 0, 0))
    assert not seen
