"""Attention calls as programs make them: between other work of their stream that writes their inputs
and overwrites them again, in graphs beside copies and branches, on two streams in turn, with batches
whose shares of the GPU begin and end inside, at and between sequences; and the calls that are refused
by their handle.  References and tolerances are those of test_gpu_attention."""
import ctypes
import math

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from deepseek_v4_compressed_wkv_gb300.layer import _Cache
from test_gpu_attention import DEV, Pages, check, gen, reference, run_decode, run_prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [
    [1] * 500 + [4000], [4000] + [1] * 500, [0] * 300 + [700] * 3 + [0] * 300, [449] * 152, [448, 449] * 60,
    [64] * 400 + [385], [65, 0, 1000, 64, 63, 0, 2000] * 9, [385] * 19, [385] * 20, [2500] * 19 + [1]])
def test_batches_whose_shares_end_anywhere(lens):
    run_decode(16, 64, 32, lens, "latent", seed=len(lens))
    run_decode(100, 64, 32, lens[:60], "fp4", seed=len(lens))  # two items a sequence


@pytest.mark.parametrize("H", [3, 21, 48, 63, 100])
def test_windows_with_heads_that_straddle_items(H):
    run_prefill(2, 220, H, 64, 385, 9, 300, seed=H)
    run_prefill(1, 5, H, 64, 385, 9, 700, seed=H)


def test_no_pages_at_all():
    q = torch.randn(3, 64, 128, generator=gen(1), device=DEV).bfloat16()
    a, c = csa.Attention(64, 128), csa.PagedCache.allocate(1, 8, 128)
    out, lse = a.decode(q, c, torch.zeros(3, 0, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV))
    assert (out == 0).all() and (lse == -math.inf).all() and a.device_status() == 0


def test_between_work_that_writes_and_overwrites_its_inputs():
    """A call's kernels are set up while the work before ends: they must not read or write early."""
    B, H, D = 24, 64, 256
    P = Pages([900] * B, 64, D, "latent", 7)
    a = csa.Attention(H, D)
    pool, qs = P.cache.latent.clone(), [torch.randn(B, H, D, generator=gen(i), device=DEV).bfloat16() for i in range(6)]
    want = [a.decode(x, P.cache, P.table, P.dev_lens) for x in qs]
    for b in (0, B - 1):
        check((want[0][0][b], want[0][1][b]), reference(qs[0][b], P.values[b]))
    q, lens = torch.empty_like(qs[0]), torch.empty_like(P.dev_lens)
    out, lse, kept = torch.empty_like(q), torch.empty(B, H, device=DEV), []
    torch.cuda.synchronize()
    for i in range(60):
        P.cache.latent.copy_(pool)
        lens.copy_(P.dev_lens)
        q.copy_(qs[i % 6])
        a.decode(q, P.cache, P.table, lens, out=out, lse=lse)
        q.fill_(math.nan)
        lens.zero_()
        P.cache.latent.fill_(math.nan)
        kept.append((out.clone(), lse.clone()))
        out.zero_()
    for i, (o, l) in enumerate(kept):
        assert torch.equal(o, want[i % 6][0]) and torch.equal(l, want[i % 6][1])
    assert a.device_status() == 0


def test_prefills_back_to_back_over_one_buffer():
    a = csa.Attention(16, 128, 64, 2)
    g = gen(9)
    data = [(torch.randn(2, 300, 16, 128, generator=g, device=DEV).bfloat16(),
             torch.randn(2, 300, 128, generator=g, device=DEV).bfloat16()) for _ in range(4)]
    want = [a.prefill(q, kv)[0] for q, kv in data]
    q, kv, got = torch.empty_like(data[0][0]), torch.empty_like(data[0][1]), []
    for i in range(40):
        q.copy_(data[i % 4][0])
        kv.copy_(data[i % 4][1])
        got.append(a.prefill(q, kv)[0])
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 4])


def test_in_a_graph_with_copies_and_a_branch():
    """The nodes before a call in a graph: a copy, a memset, and another stream's branch."""
    a, P, q, want = run_decode(64, 256, 16, [1500, 30, 0, 700], "latent", seed=5)
    b = csa.Attention(64, 256)
    src, qq, out = q.clone(), torch.zeros_like(q), torch.zeros_like(q)
    lens, zero = P.dev_lens.clone(), torch.ones(4, 64, 256, device=DEV, dtype=torch.bfloat16)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        qq.copy_(src)
        with torch.cuda.stream(side):
            zero.zero_()
            other = b.decode(src, P.cache, P.table, lens, stream=side)
        main.wait_stream(side)
        a.decode(qq, P.cache, P.table, lens, out=out)
        twice = a.decode(qq, P.cache, P.table, lens)
        qq.zero_()
    for _ in range(5):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x in (out, other[0], twice[0]):
            assert torch.equal(x, want[0])
        assert not zero.any() and not qq.any()


def test_one_handle_on_two_streams_in_turn():
    a, P, q, want = run_decode(64, 512, 16, [3000, 5, 800], "latent", seed=11)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(20):
        got.append(a.decode(q, P.cache, P.table, P.dev_lens, stream=s[i % 2]))
        s[(i + 1) % 2].wait_event(s[i % 2].record_event())
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], want[0]) and torch.equal(x[1], want[1]) for x in got)


def test_queries_that_are_not_numbers_stay_in_their_rows():
    a, P, q, want = run_decode(64, 128, 16, [700, 90], "latent", seed=12)
    bad = q.clone()
    bad[0, 3, 5], bad[1, 60, 0] = math.nan, math.inf
    out, lse = a.decode(bad, P.cache, P.table, P.dev_lens)
    same = torch.ones(2, 64, dtype=torch.bool, device=DEV)
    same[0, 3] = same[1, 60] = False
    assert torch.equal(out[same], want[0][same]) and torch.equal(lse[same], want[1][same])
    assert not torch.isfinite(out[~same]).any()


@pytest.mark.parametrize("kind", ["latent", "fp4"])
def test_a_single_visible_row_is_the_result(kind):
    """Its weight is 1: the output is the row, without a rounding (an fp4 row's values are bf16 numbers)."""
    a, P, q, (out, lse) = run_decode(64, 512, 16, [1, 1, 0, 1], kind, seed=21)
    for b in (0, 1, 3):
        assert torch.equal(out[b].double(), P.values[b][:1].expand(64, -1))
    a, q, kv, (out, lse) = run_prefill(2, 50, 16, 128, 1, 0)
    assert torch.equal(out, kv[:, :50, None].expand(-1, -1, 16, -1))
    a, q, kv, (out, lse) = run_prefill(2, 60, 64, 256, 0, 0)
    assert torch.equal(out[:, 0], kv[:, :1].expand(-1, 64, -1))


def test_calls_that_are_too_large_are_refused():
    """Sizes that the kernels' 31-bit numbers do not hold; the addresses are never read."""
    lib, A = csa.load_library(), 4096
    a = csa.Attention(64, 512)

    def decode(B=1, width=1, **kw):
        d = dict(latent=A, codes=None, scales=None, pages=4, page_size=16, head_dim=512, fp4=1)
        d.update(kw)
        c = _Cache(*(d[k] for k in ("latent", "codes", "scales", "pages", "page_size", "head_dim", "fp4")))
        rc = lib.csa_attention_decode(a._h, A, ctypes.addressof(c), A, width, A, B, A, None, None)
        return rc, lib.csa_last_error().decode()

    def prefill(B, N, start, rows):
        rc = lib.csa_attention_prefill(a._h, A, A, B, N, start, rows, None, A, None, None)
        return rc, lib.csa_last_error().decode()

    for (rc, msg), frag in (
            (decode(pages=2 ** 30, page_size=2), "2^31 - 1"),
            (decode(pages=2 ** 30, page_size=2, latent=None, codes=A, scales=A), "2^31 - 1"),
            (decode(width=2 ** 26), "2^30"), (decode(B=2 ** 25), "B ("), (decode(B=2 ** 20, width=2 ** 18), "tiles"),
            (prefill(2 ** 10, 2 ** 15, 0, 2 ** 15), "2^31"), (prefill(1, 1, 2 ** 30, 2 ** 30 + 1), "2^30"),
            (prefill(4, 1, 2 ** 29, 2 ** 29 + 1), "B * kv_rows"), (prefill(1, 2, 5, 6), "kv_rows"),
            (prefill(1, 600, 2 ** 29, 2 ** 30 - 1), "tiles")):
        assert rc == -1 and frag in msg, (rc, msg, frag)
    assert a.kernel_launches() == 0
