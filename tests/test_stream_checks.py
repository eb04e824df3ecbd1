"""A stream of another device than the tensors' is refused, and the current device
stays what it was (no GPU: the devices and the stream are stand-ins)."""
import pytest
import torch

from dynamic_block_sparse_stats_b200 import api


class _Stream:
    cuda_stream = 5

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def entered(monkeypatch):
    now = []

    class device:  # a class: a generator that nobody leaves would be left by its deletion
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            now.append(self.d)

        def __exit__(self, *_):
            now.remove(self.d)

    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", device)
    monkeypatch.setattr(api, "_check_devices", lambda named: torch.device("cuda", 0))
    return now


def test_another_devices_stream(entered):
    t = torch.zeros(4, 8, dtype=torch.bfloat16)
    other = _Stream(1)
    for call in (lambda: api.ckpt8_pack(t, stream=other), lambda: api.linear_fwd(t, torch.zeros_like(t), stream=other),
                 lambda: api.linear_bwd(t, t, torch.zeros(8, 8, dtype=torch.bfloat16), stream=other),
                 lambda: api.a2v_norm(t, stream=other)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
        assert entered == []


def test_the_calls_own_device_and_stream(entered):
    s = _Stream(0)
    with api._on(s.device, s):
        assert entered == [s.device, s]
    assert entered == []
