"""Special values in attention: scales of fp4 entries that are not numbers, and scores at the ends of
f32.  References and tolerances are those of test_gpu_attention."""
import math

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import DEV, Pages, check, fp4_values, gen, reference, visible

pytestmark = pytest.mark.gpu


def test_every_scale_byte():
    """256 sequences of one entry, each with another scale byte: the weight is 1, the output the entry's
    values; 0x7F and 0xFF are NaN."""
    D = 64
    codes = torch.randint(0, 256, (256, 1, D // 2), generator=gen(1), device=DEV, dtype=torch.uint8)
    scales = torch.arange(256, device=DEV, dtype=torch.int32).to(torch.uint8)[:, None, None].expand(256, 1, D // 16).contiguous()
    want = fp4_values(codes, scales)[:, 0]
    nan = (torch.arange(256, device=DEV) & 127) == 127
    assert torch.equal(want.isnan().all(-1), nan) and want[~nan].isfinite().all()
    a = csa.Attention(64, D)
    q = torch.randn(256, 64, D, generator=gen(2), device=DEV).bfloat16()
    out, lse = a.decode(q, csa.PagedCache(None, codes, scales), torch.arange(256, device=DEV, dtype=torch.int32)[:, None],
                        torch.ones(256, dtype=torch.int32, device=DEV))
    assert out[nan].isnan().all() and lse[nan].isnan().all()
    assert torch.equal(out[~nan].double(), want[~nan][:, None].expand(-1, 64, -1))
    assert lse[~nan].isfinite().all()


@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("D,at,block", [(64, 0, 0), (192, 63, 5), (256, 64, 7), (512, 299, 31), (512, 150, 16)])
def test_a_scale_that_is_not_a_number_shows(D, at, block, byte):
    """In one visible entry's block: the sequence's scores with that entry are NaN, the others' are not;
    behind the length it is not read."""
    P = Pages([300, 300, 150], 16, D, "fp4", D)
    a = csa.Attention(64, D)
    q = torch.randn(3, 64, D, generator=gen(3), device=DEV).bfloat16()
    want = a.decode(q, P.cache, P.table, P.dev_lens)
    for b in range(3):
        check((want[0][b], want[1][b]), reference(q[b], P.values[b]))
    P.cache.scales[int(P.table[0, at // 16]), at % 16, block] = byte
    out, lse = a.decode(q, P.cache, P.table, P.dev_lens)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert torch.equal(out[1:], want[0][1:]) and torch.equal(lse[1:], want[1][1:])
    if at:
        short = torch.tensor([at, 300, 150], dtype=torch.int32, device=DEV)
        out, lse = a.decode(q, P.cache, P.table, short)
        check((out[0], lse[0]), reference(q[0], P.values[0][:at]))


@pytest.mark.parametrize("H,D,window,sinks", [(64, 512, 40, 3), (8, 128, 40, 3), (16, 64, 0, 0), (33, 64, 70, 0), (1, 64, 20, 1)])
def test_scores_below_f32_are_weight_0_in_every_tile(H, D, window, sinks):
    """Rows of finite values whose scores pass f32's range downwards: exp(-inf) = 0, wherever in an item's
    rows they lie (some of its tokens see them, or all)."""
    N, g = 200, gen(H)
    q, kv = torch.randn(1, N, H, D, generator=g, device=DEV).bfloat16(), torch.randn(1, N, D, generator=g, device=DEV).bfloat16()
    q[..., 0], kv[..., 0] = 2.0 ** 66, 0
    low = torch.tensor([1, 30, 31, 77, 120, 121, 199], device=DEV)
    kv[0, low, 0] = -2.0 ** 66  # -2^132: f32 ends at 2^128
    finite = torch.ones(N, dtype=torch.bool, device=DEV)
    finite[low] = False
    out, lse = csa.Attention(H, D, window, sinks).prefill(q, kv)
    for t in range(N):
        rows = visible(t, window, sinks).to(DEV)
        check((out[0, t], lse[0, t]), reference(q[0, t], kv[0][rows[finite[rows]]]), f"token {t}")
    cache, table = csa.PagedCache(kv.view(10, 20, D)), torch.arange(10, dtype=torch.int32, device=DEV)[None]
    out, lse = csa.Attention(H, D).decode(q[:, 9], cache, table, torch.tensor([199], dtype=torch.int32, device=DEV))
    check((out[0], lse[0]), reference(q[0, 9], kv[0, :199][finite[:199]]))


@pytest.mark.parametrize("H", [8, 64])
def test_an_infinity_in_a_row_does_not_pass_for_a_number(H):
    """Its score is -inf for half of the heads: tokens that see the row get NaN in its feature at least, the
    others do not."""
    g = gen(H)
    q, kv = torch.randn(1, 200, H, 64, generator=g, device=DEV).bfloat16(), torch.randn(1, 200, 64, generator=g, device=DEV).bfloat16()
    a = csa.Attention(H, 64, 20, 3)
    clean = a.prefill(q, kv)[0]
    for at in (1, 50, 63, 64, 120, 199):
        x = kv.clone()
        x[0, at, 7] = -math.inf
        out = a.prefill(q, x)[0]
        see = torch.tensor([at in visible(t, 20, 3).tolist() for t in range(200)], device=DEV)
        assert torch.equal(out[0][~see], clean[0][~see])
        assert out[0][see][..., 7].isnan().all()
