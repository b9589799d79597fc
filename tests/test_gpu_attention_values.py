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


def sized(n, D, scores, seed):
    """q [D], c [n, D] whose products are the given powers of two (times 1, 0 or -1 in c's bf16 values):
    one feature holds them, the others of q are 0, of c random."""
    c = torch.randn(n, D, generator=gen(seed), device=DEV).bfloat16()
    q = torch.zeros(D, dtype=torch.bfloat16, device=DEV)
    q[1] = 2.0 ** 14 if abs(scores).max() < 2 ** 60 else 2.0 ** 64
    c[:, 1] = (scores / q[1].double()).bfloat16()
    assert torch.equal(c[:, 1].double() * q[1].double(), scores)
    return q, c


def best(q, c, scale):
    """The output, lse and sum of weighted magnitudes.  The scores are exact in f32, and of two that differ
    by more than a few the smaller has the weight 0."""
    s = c.double() @ q.double() * scale
    p = torch.softmax(s, 0)
    return p @ c.double(), torch.logsumexp(s, 0), p @ c.double().abs()


def agrees(out, lse, ref):
    mean, z, size = ref  # (a rounding of the weights, one of the output; the sums' f32 steps)
    assert ((out.double() - mean).abs() <= 2.0 ** -8 * (size + mean.abs()) + 2.0 ** -12 * size).all()
    assert ((lse.double() - z).abs() <= 2.0 ** -22 * z.abs() + 2.0 ** -12).all()


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 30, 2.0 ** 32, -2.0 ** 24, -2.0 ** 32])
@pytest.mark.parametrize("n", [40, 300, 5000])
def test_large_scores(n, size):
    """Base-2 scores of up to 0.7 * 2^30: all equal; the larger ones first, last, and in one tile only."""
    D, H = 64, 8
    a, step = csa.Attention(H, D), abs(size) * 2.0 ** -7
    near = torch.arange(n, device=DEV)
    for k, up in enumerate((near < 0, near < n // 3, near >= n - 5, near == n // 2)):
        q, c = sized(n, D, torch.where(up, size + step, size).double(), n + k)
        qq, rows = q.expand(1, H, D).contiguous(), torch.zeros(-(-n // 64) * 64, D, dtype=torch.bfloat16, device=DEV)
        rows[:n] = c
        out, lse = a.decode(qq, csa.PagedCache(rows.view(-1, 64, D)), torch.arange(-(-n // 64), dtype=torch.int32, device=DEV)[None],
                            torch.tensor([n], dtype=torch.int32, device=DEV))
        ref = best(q, c, D ** -0.5)
        agrees(out[0], lse[0], ref)
        if n <= 300:
            out, lse = a.prefill(q.expand(1, n, H, D).contiguous(), c[None])
            for t in (0, 1, n // 3, n // 2, n - 5, n - 1):
                agrees(out[0, t], lse[0, t], best(q, c[:t + 1], D ** -0.5))


@pytest.mark.parametrize("size", [2.0 ** 34, 2.0 ** 60, -2.0 ** 34, -2.0 ** 60, -2.0 ** 127, 2.0 ** 127])
def test_scores_without_digits_give_nan(size):
    """Base-2 scores of 2^30 and more: never a finite result that is wrong."""
    D, H, n = 64, 8, 200
    q, c = sized(n, D, torch.full((n,), size, device=DEV, dtype=torch.float64), 1)
    a = csa.Attention(H, D)
    out, lse = a.prefill(q.expand(1, n, H, D).contiguous(), c[None])
    assert out.isnan().all() and lse.isnan().all()
    out, lse = a.decode(q.expand(1, H, D).contiguous(), csa.PagedCache(c[:192].view(3, 64, D).contiguous()),
                        torch.arange(3, dtype=torch.int32, device=DEV)[None], torch.tensor([150], dtype=torch.int32, device=DEV))
    assert out.isnan().all() and lse.isnan().all()


def test_products_near_f32s_end_under_a_small_scale():
    D, H, n = 64, 8, 300
    for size in (-2.0 ** 127, 2.0 ** 127):
        q, c = sized(n, D, torch.full((n,), size, device=DEV, dtype=torch.float64), 2)
        a = csa.Attention(H, D, scale=1e-36)
        out, lse = a.prefill(q.expand(1, n, H, D).contiguous(), c[None])
        for t in (0, 1, 63, 64, 299):
            mean, z, mag = best(q, c[:t + 1], float(torch.tensor(1e-36)))
            agrees(out[0, t], lse[0, t], (mean, z, mag))
