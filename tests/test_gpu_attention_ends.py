"""The ends of attention's ranges: no sequences or tokens at all, and lengths past the page table's end.
References and tolerances are those of test_gpu_attention."""
import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_attention import DEV, Pages, check, gen, reference

pytestmark = pytest.mark.gpu


def test_no_sequences_and_no_tokens():
    """An empty batch is an answer of no rows, as it is for the cache write and the norm."""
    a, c = csa.Attention(8, 128), csa.PagedCache.allocate(2, 8, 128)

    def z(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device=DEV)

    i32 = torch.int32
    for B, N, rows in ((0, 5, 5), (2, 0, 5), (0, 0, 0), (3, 0, 0)):
        out, lse = a.prefill(z(B, N, 8, 128), z(B, rows, 128))
        assert out.shape == (B, N, 8, 128) and lse.shape == (B, N, 8)
        out, lse = a.prefill(z(B, N, 8, 128), z(B, rows, 128), lens=z(B, dtype=i32), out=z(B, N, 8, 128))
        assert out.shape == (B, N, 8, 128) and lse.shape == (B, N, 8)
    for width in (0, 3):
        out, lse = a.decode(z(0, 8, 128), c, z(0, width, dtype=i32), z(0, dtype=i32))
        assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    for f in (lambda: a.decode(z(0, 8, 64), c, z(0, 1, dtype=i32), z(0, dtype=i32)),
              lambda: a.decode(z(0, 8, 128), c, z(1, 1, dtype=i32), z(0, dtype=i32)),
              lambda: a.prefill(z(0, 5, 8, 128), z(0, 4, 128)), lambda: a.prefill(z(0, 5, 8, 128), z(1, 5, 128))):
        with pytest.raises(csa.CSAError):
            f()
    assert a.kernel_launches() == 0 and a.device_status() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (300, 0)])
@pytest.mark.parametrize("page,pages", [(16, 9), (7, 30), (64, 40)])
def test_a_length_past_the_page_table_is_its_end(window, sinks, page, pages):
    """Every page of the table is there: the results are those of the largest length, and the flag is raised."""
    H, D, top = 64, 128, page * pages
    P = Pages([top, top, 50], page, D, "latent", page, window, sinks, extra=0)
    q = torch.randn(3, H, D, generator=gen(2), device=DEV).bfloat16()
    a = csa.Attention(H, D, window, sinks)
    want = a.decode(q, P.cache, P.table, P.dev_lens)
    for b in range(3):
        check((want[0][b], want[1][b]), reference(q[b], P.values[b]))
    assert a.device_status() == 0
    for past in (top + 1, top + page, 2 ** 31 - 1):
        got = a.decode(q, P.cache, P.table, torch.tensor([top, past, 50], dtype=torch.int32, device=DEV))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        with pytest.raises(csa.CSAError, match="a length out of range"):
            a.device_status()
