"""Evictions in a row, without a GPU: the lengths that one returns may be handed to the next."""
import pytest
from test_kv4_cpu import recorded, some  # noqa: F401 (a fixture)
from test_kv_cpu import Rows, fake_cuda, zg  # noqa: F401 (fixtures)


class Placed(Rows):
    """A stand-in with an address of its own."""
    made = 0

    def __init__(self, *a):
        super().__init__(*a)
        Placed.made += 1
        self.at = 4096 * Placed.made

    def data_ptr(self):
        return self.at


@pytest.fixture
def evictions(recorded, monkeypatch):  # noqa: F811
    import torch
    dev, _ = recorded
    calls = []
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Placed(shape, dtype, 0))
    monkeypatch.setattr(dev.Z, "zg_kv_evict", lambda *a: calls.append((a[3], a[8], a[9])))
    return dev, calls


def test_returned_lengths_are_taken_again(evictions):
    dev, calls = evictions
    s = some(dev)
    e = dev.CacheEviction(s["c"], 2, 5, 30, 3)
    length = s["length"]
    for _ in range(4):
        new, kept = e(s["w"], s["table"], length)
        assert calls[-1][0] is length and calls[-1][1] is new and calls[-1][2] is kept
        assert new.data_ptr() != length.data_ptr() and e.length is new and kept is e.kept
        length = new
    assert len({new.data_ptr() for _, new, _ in calls}) == 2


def test_other_lengths_always_go_to_the_same_buffer(evictions):
    import torch
    dev, calls = evictions
    s = some(dev)
    e = dev.CacheEviction(s["c"], 2, 5, 30, 3)
    for _ in range(3):
        assert e(s["w"], s["table"], Placed((2,), torch.int32))[0] is calls[0][1]
    # another view of the returned lengths is theirs too
    again = Placed((2,), torch.int32)
    again.at = calls[0][1].at
    assert e(s["w"], s["table"], again)[0].data_ptr() != again.at
