"""The cache's status word when the appends run on another stream than the current one."""
import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_layer_ops import DEV, entries

pytestmark = pytest.mark.gpu


def busy():
    """Some milliseconds of work for the current stream."""
    a = torch.ones(4096, 4096, device=DEV)
    for _ in range(30):
        a = a @ a * 1e-4
    return a


def test_status_on_the_stream_of_the_append():
    """The append is still to come when status is asked for: reading the word on the current stream, which
    has nothing to wait for, would miss it."""
    c = csa.PagedCache.allocate(3, 4, 64)
    e = entries(1, 2, 64, 0, 1)
    table, far = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.full((1,), 50, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            busy()
        c.append(e, table, far, stream=s)
        with pytest.raises(csa.CSAError, match="beyond the page table"):
            c.status(stream=s)
        c.status(stream=s)
    assert not c.latent.any()


def test_a_word_is_not_cleared_behind_an_append():
    """The stream that makes the cache is busy; the first append, on another one, is not ordered behind it
    for the status word's sake."""
    table, far = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.full((1,), 50, dtype=torch.int32, device=DEV)
    e, pool, s = entries(1, 2, 64, 0, 1), torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy()
        c = csa.PagedCache(pool)
        c.append(e, table, far, stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        with pytest.raises(csa.CSAError, match="beyond the page table"):
            c.status(stream=s)


def test_bits_of_an_append_behind_status_stay_for_the_next():
    c = csa.PagedCache.allocate(3, 4, 64)
    e = entries(1, 2, 64, 0, 1)
    table = torch.zeros(1, 2, dtype=torch.int32, device=DEV)
    for first, what in ((50, "beyond"), (-9, "negative"), (50, "beyond")):
        c.append(e, table, torch.full((1,), first, dtype=torch.int32, device=DEV))
        with pytest.raises(csa.CSAError, match=what) as x:
            c.status()
        assert ("negative" in str(x.value)) == (first < 0)
    c.status()


def test_made_and_used_in_a_capture():
    """Making a cache over arrays that exist does not break a capture."""
    pool, e = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV), entries(1, 2, 64, 0, 1)
    table, first = torch.tensor([[2, 1]], dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    csa.PagedCache(pool).append(e, table, first)
    pool.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = csa.PagedCache(pool)
        c.append(e, table, first)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool[2, 1:3], e["latent"][0])
    c.status()
