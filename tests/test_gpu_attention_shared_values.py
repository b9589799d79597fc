"""Infinities and scores at the ends of f32 in attention over shared entries: they show, or do not, as in the call
without groups.  References and tolerances are those of test_gpu_attention."""
import math

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import check, reference
from test_gpu_attention_shared import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(params=[False, True])
def items(request, monkeypatch):
    """Page tables as long as the sequences, and so long that the shared rows get items of their own."""
    monkeypatch.setattr(Batch, "long", request.param)


def entries(b, i, lo, hi):
    """Places in the cache of sequence i's entries lo .. hi - 1."""
    j, page = torch.arange(lo, hi, device=DEV), b.cache.page_size
    return b.table[i].long()[j // page] * page + j % page


@pytest.mark.parametrize("H,D,shared,own", [(16, 128, 64, 30), (8, 64, 130, 70), (16, 512, 3000, 90), (33, 256, 500, 700), (64, 128, 128, 64)])
@pytest.mark.parametrize("where", ["shared", "own"])
def test_an_infinity_of_weight_0_shows(items, where, H, D, shared, own):
    """All shared rows, or all of one sequence's own ones, hold -inf in a feature where every query is positive: their
    scores are -inf, their weights 0, and 0 times infinity is NaN in that feature of whoever sees them, and nothing else is."""
    lens, at = [shared + own, shared + own + 1, shared + own - 1], 7
    b = Batch([3], [shared], lens, H, D, 16, "latent")
    b.q[:, :, at] = 1.0
    rows, sees = (entries(b, 0, 0, shared), (0, 1, 2)) if where == "shared" else (entries(b, 1, shared, lens[1]), (1,))
    if where == "shared":  # (pages in part are each sequence's own)
        rows = torch.cat([entries(b, i, 0, shared) for i in range(3)])
    b.cache.latent.view(-1, D)[rows, at] = -math.inf
    a = csa.Attention(H, D)
    got, want = a.decode(*b.args, **b.kw), a.decode(*b.args)
    for i in range(3):
        for out, lse in (got, want):
            if i not in sees:
                check((out[i], lse[i]), reference(b.q[i], b.values[i]), f"sequence {i}")
                continue
            seen = b.values[i][shared:] if where == "shared" else b.values[i][:shared]
            ref = reference(b.q[i], seen)
            ref[0][:, at] = 0
            assert out[i][:, at].isnan().all(), i
            out = out[i].clone()
            out[:, at] = 0
            check((out, lse[i]), ref, f"sequence {i}")
    assert a.device_status() == 0


@pytest.mark.parametrize("H,D", [(16, 128), (64, 256)])
def test_scores_past_the_largest_show_as_nan_to_their_group_only(items, H, D):
    """One shared row whose scores pass f32's range upwards: NaN for the sequences that have it, not for the one
    that is shorter than its group's, nor for the other group."""
    b = Batch([3, 2], [100, 64], [150, 120, 99, 90, 64], H, D, 16, "latent")
    b.q[:, :, 3] = 2.0 ** 66
    b.cache.latent[:, :, 3] = b.cache.latent[:, :, 3] * 0  # (unused slots stay NaN)
    for i, v in enumerate(b.values):
        v[:, 3] = 0
    a = csa.Attention(H, D)
    for out, lse in (a.decode(*b.args, **b.kw), a.decode(*b.args)):
        for i in range(5):
            check((out[i], lse[i]), reference(b.q[i], b.values[i]), f"sequence {i}")
    b.cache.latent.view(-1, D)[torch.cat([entries(b, i, 70, 71) for i in (0, 1)]), 3] = 2.0 ** 66
    for out, lse in (a.decode(*b.args, **b.kw), a.decode(*b.args)):
        assert out[:2].isnan().all() and lse[:2].isnan().all()
        for i in (2, 3, 4):
            check((out[i], lse[i]), reference(b.q[i], b.values[i]), f"sequence {i}")
    assert a.device_status() == 0
