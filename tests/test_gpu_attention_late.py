"""A segment that is published while the warps that wait for it give up: in the bounds-checked build
(CSA_LIBRARY_VARIANT=bounds) the environment variable CSA_TEST_LATE_SEGMENT shortens every device-side
wait to 0.2 s and makes each CTA's scheduling warp publish its first segment at the moment when the first
of those waits has run out.  Some warps of the softmax and of the epilogue then have left, others find the
segment there; the named barriers between them have no time limit, so they must go on or leave together.
The call ends, csa_attention_status reports CSA_ERR_TIMEOUT, and the next call on the handle gives what the
call before gave.  Runs inside tests/test_gpu_layer_bounds.py."""
import os

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import DEV, Pages, gen

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(os.environ.get("CSA_LIBRARY_VARIANT") != "bounds",
                                                  reason="the hook exists only in the bounds-checked build")]


def late(monkeypatch, a, call):
    want = call()
    assert a.device_status() == 0
    for _ in range(2):
        monkeypatch.setenv("CSA_TEST_LATE_SEGMENT", "1")
        call()
        with pytest.raises(csa.CSAError, match="wait budget exhausted"):
            a.device_status()
        monkeypatch.delenv("CSA_TEST_LATE_SEGMENT")
        got = call()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert a.device_status() == 0


@pytest.mark.parametrize("kind,lens", [("latent", [1500]), ("latent", [700] * 40), ("latent", [90] * 400), ("fp4", [900] * 3),
                                       ("fp4", [500] * 30)])
def test_a_decode_gives_up_as_one(monkeypatch, kind, lens):
    a, P = csa.Attention(64, 256), Pages(lens, 64, 256, kind, 2)
    q = torch.randn(len(lens), 64, 256, generator=gen(3), device=DEV).bfloat16()
    late(monkeypatch, a, lambda: a.decode(q, P.cache, P.table, P.dev_lens))


@pytest.mark.parametrize("H,D,N,window", [(64, 512, 300, 128), (16, 128, 900, 0), (3, 64, 500, 40)])
def test_a_prefill_gives_up_as_one(monkeypatch, H, D, N, window):
    a = csa.Attention(H, D, window)
    q = torch.randn(2, N, H, D, generator=gen(4), device=DEV).bfloat16()
    kv = torch.randn(2, N, D, generator=gen(5), device=DEV).bfloat16()
    late(monkeypatch, a, lambda: a.prefill(q, kv))
