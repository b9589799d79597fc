"""A page table's constructor returns when everything that it has filled is there, so that a step on another stream
need not wait for the constructing one: no fill is enqueued behind its synchronisation.  Without a GPU: the
constructor runs over stand-ins that write down what it enqueues, in order."""
import types

import pytest

from deepseek_v4_compressed_wkv_gb300 import layer


class Array:
    """A stand-in of a CUDA tensor."""

    def __init__(self, *shape):
        self.shape, self.dtype, self.device, self.is_cuda = shape, layer._I32, "cuda:0", True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.fixture
def events(monkeypatch):
    seen = []

    def filled(name):
        def make(*size, **kw):
            seen.append(name)
            return Array(*size)
        return make

    stream = types.SimpleNamespace(synchronize=lambda: seen.append("synchronize"))
    cuda = types.SimpleNamespace(is_current_stream_capturing=lambda: False, current_stream=lambda device=None: stream)
    fake = types.SimpleNamespace(cuda=cuda, empty=lambda *size, **kw: Array(*size),
                                 **{n: filled(n) for n in ("zeros", "full", "ones", "tensor")})
    monkeypatch.setattr(layer, "torch", fake)
    monkeypatch.setattr(layer, "_split", lambda t, sizes: [Array(n) for n in sizes])
    monkeypatch.setattr(layer, "load_library", lambda: types.SimpleNamespace(csa_pages_workspace=lambda *a: 100))
    return seen


def test_nothing_is_filled_behind_the_synchronisation(events):
    layer.PageTable(Array(40), Array(3, 5), Array(3), 16)
    assert events.count("synchronize") == 1
    assert events[-1] == "synchronize" and "zeros" in events


@pytest.mark.gpu
def test_steps_on_another_stream_while_the_constructing_one_is_busy():
    """The constructing stream has work before and behind the constructor; a fork, an extension and a packing on
    another stream, which waits for nothing, keep their lists."""
    import torch
    import deepseek_v4_compressed_wkv_gb300 as csa

    def dev(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    a = torch.randn(4096, 4096, device="cuda")
    more, parent = dev([5, 0, 3]), dev([0, 0, -1])
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        busy = a
        for _ in range(20):
            busy = busy @ a
        t = csa.PageTable.allocate(8, 3, 4, 2)
        for _ in range(20):
            busy = busy @ a
        first = t.extend(more, stream=other)
        src, dst, count = t.fork(parent, stream=other)
        with torch.cuda.stream(other):
            forked = torch.cat((first, count, src[:1], dst[:1])).clone()
            moved = torch.cat(t.compact(stream=other)[::2]).clone()
        torch.cuda.synchronize()
        # pages 0-2 and 3-4; the third sequence ends, page 2 is copied to page 3: nothing is behind the four in use
        assert forked.tolist() == [0, 0, 0, 1, 2, 3]
        assert moved[-1] == 0 and t.refs.tolist() == [2, 2, 1, 1, 0, 0, 0, 0]
        t.status()
