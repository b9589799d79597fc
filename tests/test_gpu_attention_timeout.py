"""The time-out path of the attention kernel, exercised without any fault: in the bounds-checked build
of the library (CSA_LIBRARY_VARIANT=bounds) the environment variable CSA_TEST_STALL_LAST_STAGE makes
every CTA's row warps leave out their first tile and shortens every device-side wait to 0.2 s.  The
score warp's wait for that tile runs out: the CTAs give up, the copies and products in flight complete,
the TMEM is freed, csa_attention_status reports CSA_ERR_TIMEOUT, and the next call on the same handle
gives what the call before gave, bit for bit.  Forms: items drawn (a prompt), one long sequence cut
over the GPU and joined, many cut sequences (whose join then finds records of the larger call before
in the workspace), codes.  The product build has no such hook, so this file only runs inside the
bounds-checked run (tests/test_gpu_attention_bounds.py)."""
import os

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import DEV, Pages, gen

pytestmark = pytest.mark.gpu

CSA_ERR_TIMEOUT = -4


@pytest.mark.parametrize("kind,lens", [("latent", [1500]), ("latent", [700] * 40), ("fp4", [900] * 3), ("fp4", [500] * 30)])
def test_a_decode_that_gives_up_is_reported_and_the_handle_recovers(monkeypatch, kind, lens):
    if os.environ.get("CSA_LIBRARY_VARIANT") != "bounds":
        pytest.skip("the stall hook exists only in the bounds-checked build")
    H, D = 64, 256
    a = csa.Attention(H, D)
    large = Pages([400] * 200, 64, D, kind, 1)
    qb = torch.randn(200, H, D, generator=gen(3), device=DEV).bfloat16()
    P = Pages(lens, 64, D, kind, 2)
    q = qb[:len(lens)].contiguous()
    want = a.decode(q, P.cache, P.table, P.dev_lens)
    a.decode(qb, large.cache, large.table, large.dev_lens)  # leaves its records and pieces in the workspace
    assert a.device_status() == 0
    monkeypatch.setenv("CSA_TEST_STALL_LAST_STAGE", "1")
    a.decode(q, P.cache, P.table, P.dev_lens)
    with pytest.raises(csa.CSAError, match="wait budget exhausted"):
        a.device_status()
    monkeypatch.delenv("CSA_TEST_STALL_LAST_STAGE")
    got = a.decode(q, P.cache, P.table, P.dev_lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert a.device_status() == 0


@pytest.mark.parametrize("H,D,N,window", [(64, 512, 300, 128), (16, 128, 900, 0)])
def test_a_prefill_that_gives_up_is_reported_and_the_handle_recovers(monkeypatch, H, D, N, window):
    if os.environ.get("CSA_LIBRARY_VARIANT") != "bounds":
        pytest.skip("the stall hook exists only in the bounds-checked build")
    a = csa.Attention(H, D, window)
    q = torch.randn(2, N, H, D, generator=gen(4), device=DEV).bfloat16()
    kv = torch.randn(2, N, D, generator=gen(5), device=DEV).bfloat16()
    want = a.prefill(q, kv)
    assert a.device_status() == 0
    monkeypatch.setenv("CSA_TEST_STALL_LAST_STAGE", "1")
    a.prefill(q, kv)
    assert csa.load_library().csa_attention_status(a._h, None) == CSA_ERR_TIMEOUT
    monkeypatch.delenv("CSA_TEST_STALL_LAST_STAGE")
    got = a.prefill(q, kv)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert a.device_status() == 0
