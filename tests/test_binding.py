"""The binding where torch lacks the entry points that it does not promise: the
public ones serve instead."""
import pytest

import post_weight_quantization_04_amd as P

torch = pytest.importorskip("torch")


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def bare_torch(monkeypatch):
    """The binding loaded anew with a torch that has public entry points alone."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.delattr(torch.autograd.forward_ad, "_current_level", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: FakeStream(100 + index))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for name in ("_TORCH", "_FORWARD_AD", "_RAW_STREAM", "_CURRENT_DEVICE"):
        monkeypatch.setattr(P, name, None)
    P._torch()


def test_current_stream_and_device(bare_torch):
    stream, where = P._place(torch.device("cuda", 1), "A", None)
    assert stream == 101 and where is P._HERE
    stream, where = P._place(torch.device("cuda", 2), "A", None)
    assert stream == 102 and isinstance(where, torch.cuda.device)


def test_tangents_are_looked_for(bare_torch, monkeypatch):
    x = torch.zeros(3)
    monkeypatch.setattr(torch.autograd.forward_ad, "unpack_dual",
                        lambda t: torch.autograd.forward_ad.UnpackedDualTensor(t, torch.ones(3) if t is x else None))
    P._no_grad(torch.zeros(3), None)
    with pytest.raises(ValueError, match="tangents"):
        P._no_grad(x)
