"""The binding's host side, with fakes in the place of the device."""
import types

import torch

from token_dispatch_fp32_b200 import _binding as b


def test_current_stream_without_torchs_short_way(monkeypatch):
    """A torch without the unlisted function: the public one gives the handle."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda dev: types.SimpleNamespace(cuda_stream=1000 + dev))
    assert b._raw_stream_of()(3) == 1003


def test_a_call_takes_the_current_streams_handle(monkeypatch):
    got = []
    monkeypatch.setattr(b, "_raw_stream", lambda index: 70 + index)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(b, "_lib", types.SimpleNamespace(f=lambda *a: got.append(a) or b.MR_OK))
    dev = torch.device("cuda", 1)
    b._call("f", dev, None, 5, None)
    b._call("f", dev, types.SimpleNamespace(device=dev, cuda_stream=9), 6)
    assert got == [(5, None, 71), (6, 9)]
