"""Groups most of whose sequences have ended or are too short for the shared entries: they cost what they cost without groups,
and the others' results are those of their entries."""
import math

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import check, gen, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def batch(B, live, H, D, shared, own, short, width, page=16, seed=0):
    """B sequences of one group, those of `live` with `shared` common and `own` further entries, the others with `short`
    of their own."""
    g = gen(seed)
    lens = torch.full((B,), short, dtype=torch.int32)
    lens[live] = shared + own
    need = (lens + page - 1) // page
    whole = shared // page
    mine = torch.zeros(B, dtype=torch.int64)
    mine[live] = whole
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = whole
    for b in range(B):
        k = int(need[b])
        table[b, :int(mine[b])] = torch.arange(int(mine[b]), dtype=torch.int32)
        n = k - int(mine[b])
        table[b, int(mine[b]):k] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    pool = torch.randn(at + 1, page, D, generator=g, device=DEV).bfloat16()
    q = torch.randn(B, H, D, generator=g, device=DEV).bfloat16()
    args = q, csa.PagedCache(pool), table.to(DEV), lens.to(DEV)
    kw = dict(groups=torch.tensor([0, B], dtype=torch.int32, device=DEV), shared=torch.tensor([shared], dtype=torch.int32, device=DEV))
    values = lambda b: pool[table[b, :int(need[b])].long().to(DEV)].flatten(0, 1)[:int(lens[b])]  # noqa: E731
    return args, kw, values


@pytest.mark.parametrize("H", [1, 3, 16, 60])
@pytest.mark.parametrize("short", [0, 5, 47])
@pytest.mark.parametrize("live", [[299], [0], [1, 2, 63, 64, 65, 130, 298], [150]])
def test_results(H, short, live):
    B, D, shared, own = 300, 64, 48, 21
    args, kw, values = batch(B, live, H, D, shared, own, short, width=6000)
    a = csa.Attention(H, D)
    out, lse = a.decode(*args, **kw)
    assert a.device_status() == 0
    assert a.kernel_launches() >= 3  # the shared rows have items of their own
    for b in sorted({0, 1, 2, 100, 297, 298, 299, *live}):
        check((out[b], lse[b]), reference(args[0][b], values(b)), f"sequence {b}")
    if short == 0:
        ended = torch.ones(B, dtype=torch.bool, device=DEV)
        ended[live] = False
        assert (out[ended] == 0).all() and (lse[ended] == -math.inf).all()


def test_the_time_is_not_that_of_a_look_at_all_sequences_for_each():
    """20000 sequences, the last 20 alive: within ten times of the call without groups (a look at the whole group for each
    of its items: more than a hundred times)."""
    B = 20000
    args, kw, values = batch(B, list(range(B - 20, B)), 16, 64, 256, 30, 0, width=400)
    a = csa.Attention(16, 64)

    def time(**kw):
        ts = []
        for _ in range(5):
            x, y = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            x.record()
            a.decode(*args, **kw)
            y.record()
            torch.cuda.synchronize()
            ts.append(x.elapsed_time(y))
        return sorted(ts)[2]

    time(), time(**kw)
    without = time()
    assert time(**kw) < 10 * without
    out, lse = a.decode(*args, **kw)
    for b in (B - 20, B - 7, B - 1):
        check((out[b], lse[b]), reference(args[0][b], values(b)), f"sequence {b}")
    assert a.device_status() == 0
