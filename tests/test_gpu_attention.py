"""Attention over one shared key/value row per position against its definition in 64 bits: a prompt
with a window and sinks, and one new token over a paged cache of latents or fp4 codes.

Tolerance of an output element, from the arithmetic: the weights exp(S - max) are rounded to bf16
(2^-8 of sum p|c|), the output is rounded to bf16 (2^-8 of itself), and the f32 scores are off by at
most ds = (D + 4) 2^-23 scale sum|q c| (one f32 step a product and addition, doubled for the tensor
core's alignment), which moves every weight by the relative amount ds, as n f32 additions of the sum
do by n 2^-23.  lse is off by ds, the sum's n 2^-23 and its own f32 steps."""
import math

import numpy as np
import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa

pytestmark = pytest.mark.gpu
DEV = "cuda"
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def visible(t, window, sinks):
    j = torch.arange(t + 1)
    return j if window == 0 else j[(j < sinks) | (j > t - window)]


def reference(q, c, scale=None):
    """q [H, D], c [n, D] (the visible rows) in 64 bits -> out, lse, and their tolerances."""
    q, c = q.double(), c.double()
    D, n = q.shape[1], len(c)
    scale = scale or D ** -0.5
    if n == 0:
        z = torch.zeros_like(q)
        return z, torch.full((len(q),), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros_like(z[:, 0])
    s = q @ c.T * scale
    ds = ((D + 4) * 2.0 ** -23 * scale * (q.abs() @ c.abs().T)).amax(1)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out = p @ c
    size = p @ c.abs()
    tol = 2.0 ** -8 * (size + out.abs()) + (2 * ds + (n + 16) * 2.0 ** -22)[:, None] * size
    return out, lse, tol, ds + (n + 16) * 2.0 ** -23 + 2.0 ** -22 * (lse.abs() + s.abs().amax(1))


def check(got, ref, what=""):
    out, lse, tol, ltol = ref
    d = (got[0].double() - out).abs()
    assert torch.isfinite(got[0]).all(), what
    assert (d <= tol).all(), f"{what}: off by {(d / tol.clamp(min=1e-30)).max():.3g} tolerances"
    if len(out) and torch.isinf(lse[0]):
        assert torch.equal(got[1].double(), lse), what
    else:
        e = (got[1].double() - lse).abs()
        assert (e <= ltol).all(), f"{what}: lse off by {(e / ltol).max():.3g} tolerances"


def fp4_values(codes, scales):
    c = codes.long().cpu()
    v = torch.stack((E2M1[c & 15], E2M1[c >> 4]), -1).flatten(-2)
    a = scales.view(torch.float8_e4m3fn).float().double().cpu()
    return (v.unflatten(-1, (-1, 16)) * a[..., None]).flatten(-2).to(DEV)


class Pages:
    """A shuffled paged cache for sequences of the given lengths; unused slots hold NaN (latent)."""

    def __init__(self, lens, page, D, kind, seed=0, window=0, sinks=0, extra=2, spread=1.0):
        g = gen(seed)
        B, width = len(lens), max(1, max(-(-n // page) for n in lens) + extra)
        pages = B * width + 3
        self.lens, self.page = lens, page
        perm = torch.randperm(pages, generator=g, device=DEV)[: B * width].to(torch.int32).view(B, width)
        self.table = torch.full((B, width), -7, dtype=torch.int32, device=DEV)  # ids past the end are not looked at
        self.values = []
        if kind == "latent":
            pool = torch.full((pages, page, D), math.nan, dtype=torch.bfloat16, device=DEV)
        else:
            codes = torch.randint(0, 256, (pages, page, D // 2), generator=g, device=DEV, dtype=torch.uint8)
            scales = torch.full((pages, page, D // 16), 0x7F, dtype=torch.uint8, device=DEV)  # NaN
        for b, n in enumerate(lens):
            need = -(-n // page)
            self.table[b, :need] = perm[b, :need]
            j = torch.arange(n, device=DEV)
            rows = perm[b].long()[j // page] * page + j % page
            keep = visible(n - 1, window, sinks).to(DEV) if n else j
            at = rows[keep]  # entries that the window hides stay NaN
            if kind == "latent":
                v = (torch.randn(len(at), D, generator=g, device=DEV) * spread).bfloat16()
                pool.view(-1, D)[at] = v
                self.values.append(v.double())
            else:
                s = (torch.rand(len(at), D // 16, generator=g, device=DEV) * 0.4 + 0.1).to(torch.float8_e4m3fn)
                scales.view(-1, D // 16)[at] = s.view(torch.uint8)
                self.values.append(fp4_values(codes.view(-1, D // 2)[at], s.view(torch.uint8)))
        self.cache = csa.PagedCache(pool) if kind == "latent" else csa.PagedCache(None, codes, scales)
        self.dev_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)


def run_decode(H, D, page, lens, kind, window=0, sinks=0, seed=0, spread=1.0, scale=0.0):
    P = Pages(lens, page, D, kind, seed, window, sinks, spread=spread)
    q = torch.randn(len(lens), H, D, generator=gen(seed + 1), device=DEV).bfloat16()
    a = csa.Attention(H, D, window, sinks, scale)
    out = torch.full((len(lens) + 1, H, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(lens) + 1, H), 3.0, device=DEV)
    got = a.decode(q, P.cache, P.table, P.dev_lens, out=out[:-1], lse=lse[:-1])
    for b in range(len(lens)):
        check((got[0][b], got[1][b]), reference(q[b], P.values[b], scale or None), f"sequence {b} of {lens[b]}")
    assert (out[-1] == 3).all() and (lse[-1] == 3).all()
    assert a.device_status() == 0
    again = a.decode(q, P.cache, P.table, P.dev_lens)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    return a, P, q, got


EDGES = [0, 1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 300]


@pytest.mark.parametrize("kind", ["latent", "fp4"])
@pytest.mark.parametrize("D", [64, 128, 192, 256, 320, 448, 512])
def test_decode_lengths_around_tiles(kind, D):
    run_decode(64, D, 16, EDGES, kind, seed=D)


@pytest.mark.parametrize("H", [1, 7, 16, 33, 64, 65, 128, 200])
def test_decode_head_counts(H):
    run_decode(H, 128, 32, [70, 1, 0, 333], "latent", seed=H)
    run_decode(H, 512, 32, [130, 5], "fp4", seed=H)


@pytest.mark.parametrize("page", [1, 3, 7, 64, 100, 1000])
def test_decode_page_sizes(page):
    run_decode(64, 512, page, [5, 64, 200, 999], "latent", seed=page)
    run_decode(16, 64, page, [5, 64, 200, 999], "fp4", seed=page)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (128, 4), (100, 70), (128, 128), (500, 0)])
@pytest.mark.parametrize("kind", ["latent", "fp4"])
def test_decode_window_and_sinks(window, sinks, kind):
    run_decode(64, 512 if kind == "latent" else 128, 16, [0, 1, 4, 127, 128, 129, 132, 133, 200, 700], kind, window, sinks)


@pytest.mark.parametrize("B,longest", [(1, 20000), (2, 9000), (3, 4097), (40, 700), (160, 130), (300, 70), (1000, 5)])
def test_decode_splits_and_joins(B, longest):
    rng = np.random.RandomState(B)
    lens = [longest] + [int(x) for x in rng.randint(0, longest + 1, B - 1)]
    run_decode(64, 128, 64, lens, "latent", seed=B)
    if B < 50:
        run_decode(64, 512, 64, lens, "latent" if B % 2 else "fp4", seed=B + 1)


@pytest.mark.parametrize("spread", [1e-3, 8.0, 40.0])
def test_decode_flat_and_peaked_scores(spread):
    """The running maximum hardly moves, or moves by hundreds from tile to tile."""
    run_decode(64, 512, 16, [1, 65, 700, 5000], "latent", seed=5, spread=spread)
    run_decode(16, 64, 16, [1, 65, 700, 5000], "latent", seed=6, spread=spread, scale=0.5)


def test_decode_scores_that_grow_along_the_cache():
    """Every tile raises the running maximum: what was summed has to be scaled down each time."""
    D, n = 512, 700
    pool = torch.randn(11, 64, D, generator=gen(3), device=DEV).bfloat16()
    q = torch.randn(1, 64, D, generator=gen(4), device=DEV).bfloat16()
    up = torch.linspace(0, 12, 704, device=DEV).view(11, 64, 1)
    pool = (pool.float() + up * q[0, :1].float() / 4).bfloat16()
    a = csa.Attention(64, D)
    got = a.decode(q, csa.PagedCache(pool), torch.arange(11, dtype=torch.int32, device=DEV).view(1, 11),
                   torch.tensor([n], dtype=torch.int32, device=DEV))
    check((got[0][0], got[1][0]), reference(q[0], pool.view(-1, D)[:n]))


def test_decode_codes_and_latents_agree():
    """Codes and scales hold the latent exactly, and every sum is made in the same order."""
    a, P, q, got = run_decode(64, 512, 16, [0, 1, 77, 400, 3000], "fp4", seed=9)
    lat = torch.zeros(P.cache.pages, P.page, 512, dtype=torch.float64, device=DEV)
    for b, n in enumerate(P.lens):
        j = torch.arange(n, device=DEV)
        lat.view(-1, 512)[P.table[b].long()[j // P.page] * P.page + j % P.page] = P.values[b]
    same = a.decode(q, csa.PagedCache(lat.bfloat16()), P.table, P.dev_lens)
    assert torch.equal(same[0], got[0]) and torch.equal(same[1], got[1])


def test_decode_flags_lengths_and_pages():
    P = Pages([100, 50, 20], 16, 128, "latent")
    q = torch.randn(3, 8, 128, generator=gen(2), device=DEV).bfloat16()
    a = csa.Attention(8, 128)
    top = P.table.shape[1] * 16
    for bad in ([-1, 50, 20], [100, -2 ** 31, 20]):
        got = a.decode(q, P.cache, P.table, torch.tensor(bad, dtype=torch.int32, device=DEV))
        with pytest.raises(csa.CSAError, match="a length out of range"):
            a.device_status()
        assert a.device_status() == 0
        b = 0 if bad[0] < 0 else 1
        assert (got[0][b] == 0).all() and torch.isinf(got[1][b]).all()
        check((got[0][2], got[1][2]), reference(q[2], P.values[2]))
    a.decode(q, P.cache, P.table, torch.tensor([2 ** 31 - 1, 50, 20], dtype=torch.int32, device=DEV))
    with pytest.raises(csa.CSAError, match="a length out of range"):  # clamped to the table, whose end is unset
        a.device_status()
    for page in (-1, P.cache.pages, 2 ** 31 - 1):
        t = P.table.clone()
        t[1, 2] = page
        got = a.decode(q, P.cache, t, P.dev_lens)
        with pytest.raises(csa.CSAError, match="a page outside the cache"):
            a.device_status()
        for b in (0, 2):
            check((got[0][b], got[1][b]), reference(q[b], P.values[b]))
    assert top > 100


def test_decode_beyond_32_bit_offsets():
    """A cache of more than 2^31 values (4.7 GB), its pages read at both ends."""
    pages, page, D = 36000, 128, 512
    pool = torch.empty(pages, page, D, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[pages - 1, 0, pages - 2, 1, pages - 3]], dtype=torch.int32, device=DEV)
    for p in table[0].tolist():
        pool[p] = torch.randn(page, D, generator=gen(p), device=DEV).bfloat16()
    q = torch.randn(1, 64, D, generator=gen(1), device=DEV).bfloat16()
    a = csa.Attention(64, D)
    got = a.decode(q, csa.PagedCache(pool), table, torch.tensor([600], dtype=torch.int32, device=DEV))
    check((got[0][0], got[1][0]), reference(q[0], pool[table[0].long()].view(-1, D)[:600]))


# ---- prompts


def run_prefill(B, N, H, D, window, sinks, start=0, lens=None, seed=0, tail=3):
    g = gen(seed)
    q = torch.randn(B, N, H, D, generator=g, device=DEV).bfloat16()
    kv = torch.randn(B, start + N + tail, D, generator=g, device=DEV).bfloat16()
    kv[:, start + N:] = math.nan  # rows past the call are nobody's
    if lens is not None:
        for b, n in enumerate(lens):
            kv[b, start + n:] = math.nan
    a = csa.Attention(H, D, window, sinks)
    out = torch.full((B + 1, N, H, D), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B + 1, N, H), 3.0, device=DEV)
    got = a.prefill(q, kv, start, None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV),
                    out=out[:-1], lse=lse[:-1])
    for b in range(B):
        n = N if lens is None else lens[b]
        step = max(1, n // 40)
        for i in sorted({*range(0, n, step), *range(min(n, 3)), *range(max(0, n - 3), n)}):
            keep = visible(start + i, window, sinks).to(DEV)
            check((got[0][b, i], got[1][b, i]), reference(q[b, i], kv[b][keep]), f"token {i} of sequence {b}")
        assert (out[b, n:] == 3).all() and (lse[b, n:] == 3).all()
    assert (out[-1] == 3).all() and (lse[-1] == 3).all()
    assert a.device_status() == 0
    again = a.prefill(q, kv, start, None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV),
                      out=out[:-1].clone(), lse=lse[:-1].clone())
    assert torch.equal(again[0], out[:-1]) and torch.equal(again[1], lse[:-1])
    return a, q, kv, got


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 130, 333])
def test_prefill_lengths(N):
    run_prefill(1, N, 64, 512, 128, 0, seed=N)
    run_prefill(2, N, 64, 128, 0, 0, seed=N + 1)


@pytest.mark.parametrize("H,D", [(1, 64), (8, 128), (16, 192), (40, 256), (64, 320), (65, 384), (128, 512), (130, 64)])
def test_prefill_heads_and_widths(H, D):
    run_prefill(2, 150, H, D, 64, 5, seed=H)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (3, 0), (63, 1), (64, 64), (65, 0), (127, 1), (128, 4), (128, 16),
                                          (129, 0), (200, 100), (0, 0), (10000, 3)])
def test_prefill_windows_and_sinks(window, sinks):
    run_prefill(1, 300, 64, 512, window, sinks, seed=window)


@pytest.mark.parametrize("start", [1, 60, 127, 128, 129, 1000])
def test_prefill_chunks_of_a_prompt(start):
    run_prefill(2, 70, 64, 512, 128, 4, start, seed=start)
    run_prefill(1, 1, 64, 256, 0, 0, start, seed=start)


def test_prefill_padded_batches():
    run_prefill(5, 140, 64, 512, 128, 4, 10, lens=[140, 0, 1, 77, 139])
    run_prefill(3, 200, 16, 128, 0, 0, 0, lens=[0, 200, 100])
    run_prefill(2, 9, 64, 64, 4, 0, 0, lens=[0, 0])


def test_prefill_of_a_few_tokens_over_many_rows():
    """Few queries, long visible ranges: their rows are split over the GPU."""
    run_prefill(1, 2, 64, 512, 0, 0, 6000, seed=1)
    run_prefill(3, 1, 64, 128, 3000, 10, 9000, seed=2)


def test_prefill_agrees_with_one_token_at_a_time():
    a, q, kv, got = run_prefill(1, 140, 64, 512, 128, 4)
    for i in (0, 77, 139):
        one = a.prefill(q[:, i:i + 1].contiguous(), kv, i)
        ref = reference(q[0, i], kv[0][visible(i, 128, 4).to(DEV)])
        check((one[0][0, 0], one[1][0, 0]), ref)
        cache = csa.PagedCache(kv[:, :140].reshape(14, 10, 512).contiguous())
        dec = a.decode(q[:, i].contiguous(), cache, torch.arange(14, dtype=torch.int32, device=DEV)[None],
                       torch.tensor([i + 1], dtype=torch.int32, device=DEV))
        check((dec[0][0], dec[1][0]), ref)


def test_rows_reach_only_the_tokens_that_see_them():
    """A NaN or an infinity in one row shows in the tokens that see it and in no other."""
    for H, D in ((64, 512), (8, 128), (33, 64)):
        g = gen(H)
        q = torch.randn(1, 200, H, D, generator=g, device=DEV).bfloat16()
        kv = torch.randn(1, 200, D, generator=g, device=DEV).bfloat16()
        a = csa.Attention(H, D, 20, 3)
        clean = a.prefill(q, kv)
        for bad in (math.nan, math.inf):
            for at in (1, 50, 120, 199):
                x = kv.clone()
                x[0, at, D // 2] = bad
                out, _ = a.prefill(q, x)
                see = torch.tensor([at in visible(t, 20, 3).tolist() for t in range(200)], device=DEV)
                assert torch.equal(out[0][~see], clean[0][0][~see])
                assert not torch.isfinite(out[0][see]).all(-1).all(-1).any()


def test_prefill_flags_lengths():
    a = csa.Attention(8, 128, 16)
    q, kv = torch.zeros(2, 5, 8, 128, dtype=torch.bfloat16, device=DEV), torch.ones(2, 5, 128, dtype=torch.bfloat16, device=DEV)
    for lens, rows in (([-3, 5], (0, 5)), ([9, 2], (5, 2))):
        out = torch.full_like(q, 3)
        a.prefill(q, kv, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), out=out)
        with pytest.raises(csa.CSAError, match="a length out of range"):
            a.device_status()
        for b, n in enumerate(rows):
            assert (out[b, :n] == 1).all() and (out[b, n:] == 3).all()


# ---- streams, graphs, refusals


def test_other_streams_and_handles_at_once():
    a1, P1, q1, g1 = run_decode(64, 512, 16, [3000, 5, 800], "latent", seed=1)
    a2, P2, q2, g2 = run_decode(64, 512, 16, [700, 4000], "fp4", seed=2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append((a1.decode(q1, P1.cache, P1.table, P1.dev_lens, stream=s1), g1))
        got.append((a2.decode(q2, P2.cache, P2.table, P2.dev_lens, stream=s2), g2))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_captured_and_replayed_with_new_lengths():
    a, P, q, _ = run_decode(64, 512, 16, [3000, 0, 800, 17], "latent", seed=3)
    out, lse = torch.zeros_like(q), torch.zeros(4, 64, device=DEV)
    lens = P.dev_lens.clone()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g1, stream=side):
        a.decode(q, P.cache, P.table, lens, out=out, lse=lse)
    out2, lse2 = torch.zeros_like(q), torch.zeros(4, 64, device=DEV)
    with torch.cuda.graph(g2, stream=side):
        a.decode(q, P.cache, P.table, lens, out=out2, lse=lse2)
    for now in ([3000, 0, 800, 17], [2999, 0, 1, 16], [64, 0, 799, 0]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(now):
            check((out[b], lse[b]), reference(q[b], P.values[b][:n]))
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    pre, q4, kv, want = run_prefill(2, 100, 64, 512, 32, 4)
    out3 = torch.zeros_like(q4)
    g3 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g3, stream=side):
        pre.prefill(q4, kv, out=out3)
    g3.replay()
    torch.cuda.synchronize()
    assert torch.equal(out3, want[0])


def test_binding_refusals():
    a = csa.Attention(8, 128)
    q, kv = torch.zeros(1, 4, 8, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 4, 128, dtype=torch.bfloat16, device=DEV)
    bad = [lambda: a.prefill(q.float(), kv), lambda: a.prefill(q.cpu(), kv), lambda: a.prefill(q[0], kv),
           lambda: a.prefill(q, kv[:, :3]), lambda: a.prefill(q, kv, 1), lambda: a.prefill(q, kv, -1),
           lambda: a.prefill(q, kv, 2 ** 31), lambda: a.prefill(q.transpose(1, 2), kv),
           lambda: a.prefill(q[:, :, :4].contiguous(), kv), lambda: a.prefill(q, kv, out=q[:, :3]),
           lambda: a.prefill(q, kv, lse=torch.zeros(1, 4, 7, device=DEV)),
           lambda: a.prefill(q, kv, lens=torch.zeros(1, dtype=torch.int64, device=DEV)),
           lambda: a.prefill(q, torch.zeros(1, 9, 64, dtype=torch.bfloat16, device=DEV))]
    c = csa.PagedCache.allocate(4, 8, 128)
    t, n = torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    one = q[:, 0].contiguous()
    bad += [lambda: a.decode(q, c, t, n), lambda: a.decode(one, c, t[0], n), lambda: a.decode(one, c, t.long(), n),
            lambda: a.decode(one, c, t, n.cpu()), lambda: a.decode(one, csa.PagedCache.allocate(4, 8, 64), t, n),
            lambda: a.decode(one, csa.PagedCache.allocate(4, 8, 128, fp4=2), t, n),
            lambda: a.decode(one, c, t.repeat(1, 2)[:, ::2], n), lambda: a.decode(one, c, t.repeat(2, 1), n),
            lambda: csa.Attention(8, 2 ** 32 + 128), lambda: csa.Attention(8, 128, window=2 ** 32),
            lambda: csa.PagedCache(), lambda: csa.PagedCache(torch.zeros(2, 2, 64, device=DEV)),
            lambda: csa.PagedCache(codes=torch.zeros(2, 2, 64, dtype=torch.uint8, device=DEV))]
    # an odd start inside a tensor: the rows are no longer on 16-byte boundaries
    odd = torch.zeros(4 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(1, 4, 128)
    bad += [lambda: a.prefill(q, odd)]
    for f in bad:
        with pytest.raises(csa.CSAError):
            f()
    assert a.kernel_launches() == 0
