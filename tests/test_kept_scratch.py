"""Scratch that the binding keeps for the backward calls: whose it is, when none
is kept, and how far it grows (host only: stand-ins for the device's side)."""
import threading

import pytest
import torch

import fp8_quantized_gemm_gb300 as F


class Operand:
    def __init__(self, index):
        self.device = torch.device("cuda", index) if index is not None else torch.device("cpu")


class Block:
    count = 0

    def __init__(self, size, dtype, device):
        Block.count += 1
        self.size, self.device, self.at = size, device, Block.count << 32
        assert dtype == torch.uint8

    def data_ptr(self):
        return self.at


@pytest.fixture
def device(monkeypatch):
    """current device 0, current stream `device.sid`, nothing captured."""
    class State:
        dev, sid, capturing = 0, 0, False

    monkeypatch.setattr(F, "_get_device", lambda: State.dev)
    monkeypatch.setattr(F, "_stream_id", lambda dev: State.sid, raising=False)
    monkeypatch.setattr(F, "_raw_stream", lambda dev: 4096 + State.sid)
    monkeypatch.setattr(F, "_capturing", lambda: State.capturing)
    monkeypatch.setattr(F, "_kept", threading.local())
    monkeypatch.setattr(torch, "empty", Block)
    return State


def get(nbytes, index=0):
    return F._scratch(nbytes, None, Operand(index), None)


@pytest.mark.parametrize("index", [1, None])
def test_operands_of_another_device_are_refused_and_leave_nothing(device, index):
    with pytest.raises(ValueError):
        get(1000, index)
    p, n, owner = get(1000)
    assert owner.device.index == 0 and n >= 1000


def test_one_buffer_per_stream(device):
    seen = {}
    for sid in (0, 3, 35, 0, 3, 35):
        device.sid = sid
        p, n, _ = get(1000)
        assert seen.setdefault(sid, p) == p
    assert len(set(seen.values())) == 3


def test_handles_of_other_streams_keep_nothing(device):
    """An id that is a handle may come back as another stream's."""
    device.sid = 0x55aa10
    assert get(1000)[0] != get(1000)[0]


def test_captures_and_large_calls_keep_nothing(device):
    first = get(1000)[0]
    device.capturing = True
    assert get(1000)[0] != get(1000)[0]
    device.capturing = False
    assert get(F._KEPT + 1)[0] != get(F._KEPT + 1)[0]
    assert get(1000)[0] == first


def test_growth(device):
    """As large as the calls need, not the most that is kept."""
    p, n, t = get(100)
    assert n == t.size <= 1 << 16
    q, big, t = get(3 << 20)
    assert q != p and 3 << 20 <= big <= 4 << 20 and t.size == big
    assert get(100)[0] == q and get(big)[0] == q
    assert get(F._KEPT)[1] == F._KEPT


def test_threads_have_their_own(device):
    got = []
    t = threading.Thread(target=lambda: got.append(get(1000)[0]))
    t.start()
    t.join()
    assert got[0] != get(1000)[0]


def test_explicit_streams_need_a_workspace(device):
    with pytest.raises(ValueError):
        F._scratch(10, None, Operand(0), 12345)
