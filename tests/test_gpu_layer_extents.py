"""The bounds-checked build's own checks (CSA_LIBRARY_VARIANT=bounds): with the environment variable
CSA_TEST_SHORT_EXTENTS the library takes the outputs for one row shorter than they are ("rows"), or an
attention handle's workspace for one piece long ("slots").  Nothing is out of bounds; the stores that the
checks then take for it are left out and reported.  Runs inside tests/test_gpu_layer_bounds.py."""
import os

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import DEV, Pages, gen
from test_gpu_layer_ops import entries, norm_inputs

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(os.environ.get("CSA_LIBRARY_VARIANT") != "bounds",
                                                  reason="the checks exist only in the bounds-checked build")]
WHAT = "out of bounds|outside the cache .bounds-checked"


@pytest.mark.parametrize("lens", [[300] * 200, [5000], [700] * 40])
@pytest.mark.parametrize("which", ["rows", "slots"])
def test_attention_outputs_and_pieces(monkeypatch, lens, which):
    """Items that are whole, joined where they are few, and joined where they are many."""
    H, D, B = 64, 128, len(lens)
    a, P = csa.Attention(H, D), Pages(lens, 64, D, "latent", 1)
    q = torch.randn(B, H, D, generator=gen(2), device=DEV).bfloat16()
    want = a.decode(q, P.cache, P.table, P.dev_lens)
    assert a.device_status() == 0
    whole = a.kernel_launches() == 1
    monkeypatch.setenv("CSA_TEST_SHORT_EXTENTS", which)
    out, lse = torch.full_like(want[0], 3.0), torch.full_like(want[1], 3.0)
    a.decode(q, P.cache, P.table, P.dev_lens, out=out, lse=lse)
    if which == "rows":
        assert (out[-1, -1] == 3).all() and lse[-1, -1] == 3
        assert torch.equal(out.view(B * H, D)[:-1], want[0].view(B * H, D)[:-1])
    if which == "rows" or not whole:
        with pytest.raises(csa.CSAError, match=WHAT):
            a.device_status()
    monkeypatch.delenv("CSA_TEST_SHORT_EXTENTS")
    got = a.decode(q, P.cache, P.table, P.dev_lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and a.device_status() == 0


@pytest.mark.parametrize("fp4", [0, 1, 2])
def test_cache_write(monkeypatch, fp4):
    c, e = csa.PagedCache.allocate(3, 4, 64, fp4), entries(1, 2, 64, fp4, 1)
    table, first = torch.tensor([[1, 2]], dtype=torch.int32, device=DEV), torch.tensor([6], dtype=torch.int32, device=DEV)
    monkeypatch.setenv("CSA_TEST_SHORT_EXTENTS", "rows")
    c.append(e, table, first)
    with pytest.raises(csa.CSAError, match=WHAT):
        c.status()
    pool, new = (c.codes, e["codes"]) if fp4 else (c.latent, e["latent"])
    assert torch.equal(pool[2, 2], new[0, 0]) and not pool[2, 3].any()


@pytest.mark.parametrize("block", [0, 32, 128])
@pytest.mark.parametrize("dim", [128, 4096])
def test_norm(monkeypatch, dim, block):
    x, r, gain = norm_inputs(5, dim)
    want = csa.rmsnorm_residual_q8(x, r, gain, scale_block=block)
    monkeypatch.setenv("CSA_TEST_SHORT_EXTENTS", "rows")
    rr = r.clone()
    with pytest.raises(csa.CSAError, match=WHAT):
        csa.rmsnorm_residual_q8(x, rr, gain, scale_block=block, inplace=True)
    assert torch.equal(rr[:4], want["residual"][:4]) and torch.equal(rr[4], r[4])
    monkeypatch.delenv("CSA_TEST_SHORT_EXTENTS")
    got = csa.rmsnorm_residual_q8(x, r, gain, scale_block=block)
    assert torch.equal(got["y"], want["y"])
