"""The residual RMSNorm with an 8-bit output and the paged cache's write, each against its
definition in 64 bits (or byte for byte), and the layer's serving steps run together.

Tolerances: the sum s is one f32 addition; n has the relative error of the mean's f32 sum
(dim 2^-24 at most, all terms positive, half of it after the root) and five f32 steps; bf16 outputs
add 2^-8 of themselves, f32 scales one step of the division; a quantised value is off by half an e4m3 step
(2^-4 of itself, 2^-10 below the smallest normal number, 2^-6) and by n's and the scale's errors."""
import math

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
import synthetic

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def norm_inputs(rows, dim, seed=0, size=1.0):
    g = gen(seed)
    x = (torch.randn(rows, dim, generator=g, device=DEV) * size).bfloat16()
    r = (torch.randn(rows, dim, generator=g, device=DEV) * 2 * size).bfloat16()
    return x, r, 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)


def check_norm(got, x, r, gain, block, eps=1e-6):
    dim = x.shape[-1]
    s = x.double() + (0 if r is None else r.double())
    n = s / (s.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()
    dn = (dim / 2 + 6) * 2.0 ** -24
    if r is not None:
        assert torch.equal(got["residual"], (x.float() + r.float()).bfloat16())
    assert ((got["y"].double() - n).abs() <= (2.0 ** -8 + 2 * dn) * n.abs() + 1e-40).all()
    b = n.unflatten(-1, (-1, block or dim))
    a = b.abs().amax(-1).clamp(min=448 * 2.0 ** -126) / 448
    if block == 32:
        scale = got["scales"].double()
        assert torch.equal(torch.exp2(torch.round(torch.log2(scale))), scale)
        # the next power of two up, or its neighbour where amax is within its error of a power of two
        assert (scale >= a * (1 - 2 * dn - 2.0 ** -23)).all() and (scale < 2 * a * (1 + 2 * dn + 2.0 ** -23)).all()
    else:
        scale = got["scales"].double()
        assert ((scale - a).abs() <= (dn + 2.0 ** -22) * a).all()
    q = got["q"].double().unflatten(-1, (-1, block or dim)) * scale[..., None]
    tol = b.abs() * (2.0 ** -4 + 2 * dn + 2.0 ** -22) + scale[..., None] * 2.0 ** -10
    assert ((q - b).abs() <= tol).all()


@pytest.mark.parametrize("block", [0, 32, 128])
@pytest.mark.parametrize("rows,dim", [(1, 128), (3, 256), (1, 384), (7, 512), (2, 640), (33, 4096), (5, 4224), (1, 8192),
                                      (2, 16384), (1000, 128), (129, 7040)])
def test_norm_shapes(rows, dim, block):
    x, r, gain = norm_inputs(rows, dim, rows + dim)
    check_norm(csa.rmsnorm_residual_q8(x, r, gain, scale_block=block), x, r, gain, block)


@pytest.mark.parametrize("dim", [32, 64, 96, 160, 288, 2016])
def test_norm_odd_widths(dim):
    x, r, gain = norm_inputs(19, dim, dim)
    for block in (0, 32):
        check_norm(csa.rmsnorm_residual_q8(x, r, gain, scale_block=block), x, r, gain, block)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e17])
def test_norm_magnitudes(size):
    x, r, gain = norm_inputs(9, 512, 3, size)
    for block in (0, 32, 128):
        check_norm(csa.rmsnorm_residual_q8(x, r, gain, eps=0.0 if size == 1e-6 else 1e-6, scale_block=block), x, r, gain,
                   block, 0.0 if size == 1e-6 else 1e-6)


def test_norm_without_residual_in_place_and_leading_dimensions():
    x, r, gain = norm_inputs(24, 256, 4)
    got = csa.rmsnorm_residual_q8(x, None, gain)
    assert got["residual"] is x
    check_norm(got, x, None, gain, 128)
    full = csa.rmsnorm_residual_q8(x, r, gain)
    rr = r.clone()
    same = csa.rmsnorm_residual_q8(x.view(2, 3, 4, 256), rr.view(2, 3, 4, 256), gain, inplace=True)
    assert torch.equal(rr, full["residual"]) and torch.equal(same["y"].view(24, 256), full["y"])
    assert same["residual"].data_ptr() == rr.data_ptr() and same["scales"].shape == (2, 3, 4, 2)
    assert torch.equal(same["q"].view(24, 256).view(torch.uint8), full["q"].view(torch.uint8))
    assert csa.rmsnorm_residual_q8(x, r, gain, y=False)["y"] is None
    empty = csa.rmsnorm_residual_q8(x[:0], r[:0], gain)
    assert empty["q"].shape == (0, 256)


def test_norm_zero_rows_and_values_that_are_not_numbers():
    x, r, gain = norm_inputs(6, 256, 5)
    r[:] = 0
    x[0] = 0
    x[1, 3] = math.nan
    x[2, 200] = math.inf
    x[3, 7] = -math.inf
    for block in (0, 32, 128):
        got = csa.rmsnorm_residual_q8(x, r, gain, scale_block=block)
        y, q, a = got["y"].float(), got["q"].float(), got["scales"].float()
        assert (y[0] == 0).all() and (q[0] == 0).all() and torch.isfinite(a[0]).all() and (a[0] > 0).all()
        assert torch.isnan(y[1]).all() and torch.isnan(q[1]).all() and torch.isnan(a[1]).all()
        for row, at in ((2, 200), (3, 7)):  # inf times the factor 0 is NaN, the others are 0
            assert torch.isnan(y[row, at]) and (y[row].isnan().sum() == 1) and (y[row].nan_to_num() == 0).all()
            assert torch.isnan(a[row, at // (block or 256)]) and a[row].isnan().sum() == 1
        check_norm({k: v[4:] for k, v in got.items()}, x[4:], r[4:], gain, block)


def test_norm_on_another_stream_and_in_a_graph():
    x, r, gain = norm_inputs(64, 4096, 6)
    want = csa.rmsnorm_residual_q8(x, r, gain)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = csa.rmsnorm_residual_q8(x, r, gain, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cap = csa.rmsnorm_residual_q8(x, r, gain)
    g.replay()
    torch.cuda.synchronize()
    for o in (got, cap):
        assert torch.equal(o["y"], want["y"]) and torch.equal(o["scales"], want["scales"])
        assert torch.equal(o["q"].view(torch.uint8), want["q"].view(torch.uint8))


def test_norm_refusals():
    x, r, gain = norm_inputs(2, 256)
    for f in (lambda: csa.rmsnorm_residual_q8(x.float(), r, gain), lambda: csa.rmsnorm_residual_q8(x, r[:1], gain),
              lambda: csa.rmsnorm_residual_q8(x, r, gain.bfloat16()), lambda: csa.rmsnorm_residual_q8(x, r, gain[:128]),
              lambda: csa.rmsnorm_residual_q8(x, r, gain, scale_block=64), lambda: csa.rmsnorm_residual_q8(x, None, gain, inplace=True),
              lambda: csa.rmsnorm_residual_q8(x[:, ::2], r[:, ::2], gain[::2]), lambda: csa.rmsnorm_residual_q8(x.cpu(), r, gain),
              lambda: csa.rmsnorm_residual_q8(x[:, :100].contiguous(), None, gain[:100].contiguous())):
        with pytest.raises(csa.CSAError):
            f()


# ---- the paged cache's write


def entries(B, G, D, fp4, seed):
    g = gen(seed)
    e = {"latent": torch.randn(B, G, D, generator=g, device=DEV).bfloat16()}
    if fp4:
        e["codes"] = torch.randint(0, 256, (B, G, D // 2), generator=g, device=DEV, dtype=torch.uint8)
        e["scales"] = torch.randint(0, 256, (B, G, D // (32 if fp4 == 2 else 16)), generator=g, device=DEV, dtype=torch.uint8)
    return e


@pytest.mark.parametrize("fp4", [0, 1, 2])
@pytest.mark.parametrize("B,G,D,page", [(1, 1, 512, 16), (128, 1, 512, 64), (5, 37, 64, 7), (3, 200, 128, 64), (2, 9, 96, 1),
                                        (4, 3, 32, 1000)])
def test_append_writes_the_slots_and_nothing_else(B, G, D, page, fp4):
    width = 3 + -(-G // page)
    pages = B * width + 2
    table = torch.randperm(pages, generator=gen(1), device=DEV)[: B * width].to(torch.int32).view(B, width)
    first = torch.randint(0, 3 * page, (B,), generator=gen(2), device=DEV, dtype=torch.int32)
    mask = (torch.rand(B, generator=gen(3), device=DEV) < 0.6).to(torch.uint8)
    cache = csa.PagedCache.allocate(pages, page, D, fp4)
    e = entries(B, G, D, fp4, 4)
    want = {}
    for n, pool in (("latent", cache.latent), ("codes", cache.codes), ("scales", cache.scales)):
        if pool is not None:
            pool.view(torch.uint8).fill_(0x5A)
            want[n] = pool.clone()
    for b in range(B):
        if mask[b]:
            j = int(first[b]) + torch.arange(G, device=DEV)
            rows = table[b].long()[j // page] * page + j % page
            for n, w in want.items():
                w.flatten(0, 1)[rows] = e[n][b]
    cache.append(e, table, first, mask=mask)
    for n, w in want.items():
        assert torch.equal(getattr(cache, n).view(torch.uint8), w.view(torch.uint8)), n
    cache.status()


def test_append_to_both_forms_and_odd_addresses():
    lat = torch.zeros(4, 8, 32, dtype=torch.bfloat16, device=DEV)
    codes, scales = torch.zeros(4, 8, 16, dtype=torch.uint8, device=DEV), torch.zeros(4, 8, 2, dtype=torch.uint8, device=DEV)
    c = csa.PagedCache(lat, codes, scales)
    e = entries(1, 5, 32, 1, 7)
    for k in ("latent", "codes", "scales"):  # entries that begin one element into an allocation
        buf = torch.zeros(e[k].numel() + 1, dtype=e[k].dtype, device=DEV)
        buf[1:] = e[k].flatten()
        e[k] = buf[1:].view(e[k].shape)
    c.append(e, torch.tensor([[2, 1]], dtype=torch.int32, device=DEV), torch.tensor([6], dtype=torch.int32, device=DEV))
    for k, pool in (("latent", lat), ("codes", codes), ("scales", scales)):
        assert torch.equal(pool[2, 6:], e[k][0, :2]) and torch.equal(pool[1, :3], e[k][0, 2:])


def test_append_leaves_out_what_does_not_fit():
    c = csa.PagedCache.allocate(3, 4, 64)
    e = entries(4, 2, 64, 0, 8)
    table = torch.tensor([[0, 1], [2, -1], [2, 3], [0, 1]], dtype=torch.int32, device=DEV)
    c.append(e, table, torch.tensor([0, 3, 4, -1], dtype=torch.int32, device=DEV))
    with pytest.raises(csa.CSAError, match="a negative index, a page outside the cache"):
        c.status()
    c.status()
    # the last sequence's second entry is index 0 of page 0, the slot of the first one's first: not
    # looked at; what the others wrote is
    assert torch.equal(c.latent[0, 1], e["latent"][0, 1]) and torch.equal(c.latent[2, 3], e["latent"][1, 0])
    assert (c.latent[1] == 0).all() and (c.latent[2, :3] == 0).all()
    c.append(e, table, torch.tensor([7, 8, 2 ** 31 - 1, 20], dtype=torch.int32, device=DEV))
    with pytest.raises(csa.CSAError, match="an index beyond the page table"):
        c.status()
    assert torch.equal(c.latent[1, 3], e["latent"][0, 0])


def test_append_of_nothing():
    """A prefill of fewer tokens than a group has no entries: appending them does nothing; a cache that an
    append on another stream is the first to use reports what that left out."""
    c = csa.PagedCache.allocate(3, 4, 64)
    none, table = torch.zeros(2, 0, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    c.append({"latent": none}, table, torch.zeros(2, dtype=torch.int32, device=DEV))
    c.append({"latent": none[:0]}, table[:0], torch.zeros(0, dtype=torch.int32, device=DEV))
    with pytest.raises(csa.CSAError, match="must be"):
        c.append({"latent": none[:1]}, table, torch.zeros(2, dtype=torch.int32, device=DEV))
    c.status()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    one = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    c.append({"latent": one}, table[:1], torch.full((1,), 9, dtype=torch.int32, device=DEV), stream=s)
    torch.cuda.synchronize()
    with pytest.raises(csa.CSAError, match="beyond the page table"):
        c.status()
    assert not c.latent.any()


def test_append_beyond_32_bit_offsets():
    """More than 2^32 bytes of entries in one call, to pages in reverse order, an index that the page size
    does not divide first; and an index near 2^31 into a table that ends long before."""
    G, page, D = 2 ** 22 + 77, 48, 512
    n = -(-(G + 5) // page)
    new = torch.empty(1, G, D, dtype=torch.bfloat16, device=DEV)
    new.view(torch.int16)[0] = torch.arange(G, device=DEV, dtype=torch.int32).to(torch.int16)[:, None]
    pool = torch.zeros(n, page, D, dtype=torch.bfloat16, device=DEV)
    table = torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV)[None]
    cache = csa.PagedCache(pool)
    cache.append({"latent": new}, table, torch.tensor([5], dtype=torch.int32, device=DEV))
    got = pool.flip(0).view(-1, D).view(torch.int16)
    assert torch.equal(got[5:5 + G], new[0].view(torch.int16)) and not got[:5].any() and not got[5 + G:].any()
    before = got.sum(dtype=torch.int64)
    cache.append({"latent": new[:, :100].contiguous()}, table, torch.tensor([2 ** 31 - 50], dtype=torch.int32, device=DEV))
    assert pool.view(torch.int16).sum(dtype=torch.int64) == before


def test_append_refusals():
    c = csa.PagedCache.allocate(3, 4, 64)
    e, t, f = entries(2, 2, 64, 0, 9), torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    for g in (lambda: c.append({}, t, f), lambda: c.append(e, t.long(), f), lambda: c.append(e, t[:1], f),
              lambda: c.append(e, t, f.long()), lambda: c.append(e, t, f[:1]), lambda: c.append(e, t, f, mask=f),
              lambda: c.append({"latent": e["latent"][..., :32].contiguous()}, t, f),
              lambda: c.append({"latent": e["latent"].float()}, t, f), lambda: c.append({"latent": e["latent"].cpu()}, t, f)):
        with pytest.raises(csa.CSAError):
            g()
    assert (c.latent == 0).all()


# ---- together


def make_compressor(dim, H, ratio, overlap, B):
    layer = synthetic.Layer(dim, H, ratio, overlap, 1 / math.sqrt(dim), rope_dim=64, fp4=1)
    w = [torch.from_numpy(a).to(DEV) for a in synthetic.weights(3, layer)]
    c = csa.Compressor(dim, H, ratio, overlap, max_batch=B, rope_dim=64, fp4=1, max_pos=4096)
    c.set_weights(*w)
    return c


def dense(q, rows):
    s = q.double() @ rows.double().T / math.sqrt(q.shape[-1])
    return torch.softmax(s, -1) @ rows.double()


@pytest.mark.parametrize("fp4", [0, 1])
@pytest.mark.parametrize("ratio,overlap", [(4, 1), (8, 0)])
def test_a_layers_serving_steps_together(fp4, ratio, overlap):
    """norm -> compressor prefill -> pages, then decode steps: norm -> compressor -> pages ->
    attention over everything compressed so far; against the entries kept in a plain list."""
    B, dim, D, H, N, page = 3, 256, 128, 64, 37, 4
    comp, attn = make_compressor(dim, D, ratio, overlap, B), csa.Attention(H, D)
    g = gen(11)
    gain = 1 + 0.1 * torch.randn(dim, generator=g, device=DEV)
    width = 16
    table = torch.randperm(B * width, generator=g, device=DEV).to(torch.int32).view(B, width)
    cache = csa.PagedCache.allocate(B * width, page, D, fp4)
    x = torch.randn(B, N, dim, generator=g, device=DEV).bfloat16()
    res = torch.randn(B, N, dim, generator=g, device=DEV).bfloat16()
    e = comp.prefill(csa.rmsnorm_residual_q8(x, res, gain)["y"])
    kept = [list(e["latent"][b]) for b in range(B)]
    cache.append(e, table, torch.zeros(B, dtype=torch.int32, device=DEV))
    pos = torch.full((B,), N, dtype=torch.int32, device=DEV)
    for step in range(2 * ratio + 1):
        h = csa.rmsnorm_residual_q8(torch.randn(B, dim, generator=g, device=DEV).bfloat16(),
                                    torch.randn(B, dim, generator=g, device=DEV).bfloat16(), gain, scale_block=32)
        d = comp.decode(h["y"], pos)
        cache.append(d, table, torch.div(pos, ratio, rounding_mode="floor").to(torch.int32), mask=d["emitted"])
        pos += 1
        lens = torch.div(pos, ratio, rounding_mode="floor").to(torch.int32)
        q = torch.randn(B, H, D, generator=g, device=DEV).bfloat16()
        out, lse = attn.decode(q, cache, table, lens)
        for b in range(B):
            if d["emitted"][b]:
                kept[b].append(d["latent"][b].clone())
            assert len(kept[b]) == int(lens[b])
            rows = torch.stack(kept[b])
            ref = dense(q[b], rows)
            size = torch.softmax(q[b].double() @ rows.double().T / math.sqrt(D), -1) @ rows.double().abs()
            assert ((out[b].double() - ref).abs() <= 2.0 ** -8 * (size + ref.abs()) + 2e-3 * size).all()
    cache.status()
    assert attn.device_status() == 0 and comp.device_status() == 0


def test_a_prefills_cache_rows_are_pages():
    """csa_compress_prefill_into's cache [B, rows, D] is a paged cache with one page a sequence."""
    B, dim, D, N = 2, 256, 128, 50
    comp = make_compressor(dim, D, 4, 1, B)
    x = torch.randn(B, N, dim, generator=gen(1), device=DEV).bfloat16()
    lat = torch.zeros(B, 20, D, dtype=torch.bfloat16, device=DEV)
    n = comp.prefill_into(x, {"latent": lat})
    attn = csa.Attention(8, D)
    q = torch.randn(B, 8, D, generator=gen(2), device=DEV).bfloat16()
    out, _ = attn.decode(q, csa.PagedCache(lat), torch.arange(B, dtype=torch.int32, device=DEV)[:, None],
                         torch.full((B,), n, dtype=torch.int32, device=DEV))
    for b in range(B):
        ref, size = dense(q[b], lat[b, :n]), torch.softmax(q[b].double() @ lat[b, :n].double().T / math.sqrt(D), -1) @ lat[b, :n].double().abs()
        assert ((out[b].double() - ref).abs() <= 2.0 ** -8 * (size + ref.abs()) + 2e-3 * size).all()


def test_a_decode_step_in_a_graph():
    """The step's four calls captured once and replayed while positions advance on the device."""
    B, dim, D, H, page, ratio = 2, 256, 128, 16, 8, 4
    comp, attn = make_compressor(dim, D, ratio, 1, B), csa.Attention(H, D)
    twin, gain = make_compressor(dim, D, ratio, 1, B), torch.ones(dim, device=DEV)
    table = torch.arange(B * 4, dtype=torch.int32, device=DEV).view(B, 4)
    caches = [csa.PagedCache.allocate(B * 4, page, D, 1) for _ in range(2)]
    x, res = torch.zeros(B, dim, dtype=torch.bfloat16, device=DEV), torch.zeros(B, dim, dtype=torch.bfloat16, device=DEV)
    q, pos = torch.randn(B, H, D, generator=gen(5), device=DEV).bfloat16(), torch.zeros(B, dtype=torch.int32, device=DEV)

    def step(c, cache, out=None, lse=None):
        h = csa.rmsnorm_residual_q8(x, res, gain)
        d = c.decode(h["y"], pos)
        cache.append(d, table, torch.div(pos, ratio, rounding_mode="floor").to(torch.int32), mask=d["emitted"])
        return attn.decode(q, cache, table, torch.div(pos + 1, ratio, rounding_mode="floor").to(torch.int32), out, lse)

    out, lse = torch.zeros_like(q), torch.zeros(B, H, device=DEV)
    step(comp, caches[0], out, lse)  # first calls on the device before the capture
    comp.state_reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(comp, caches[0], out, lse)
    for i in range(13):
        x.copy_(torch.randn(B, dim, generator=gen(100 + i), device=DEV))
        pos.fill_(i)
        g.replay()
        want = step(twin, caches[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i


def test_a_run_without_pauses_gives_what_it_gives_with_pauses():
    """Norm, cache write and attention in a row, each set up while the one before ends, over buffers that
    the next step overwrites: 40 steps enqueued at once against the same steps with a pause after each call."""
    B, H, D, page, n = 12, 64, 512, 16, 300
    g = gen(31)
    start = torch.randn(B * 20, page, D, generator=g, device=DEV).bfloat16()
    table = torch.randperm(B * 20, generator=g, device=DEV).to(torch.int32).view(B, 20)
    xs = [torch.randn(B, D, generator=g, device=DEV).bfloat16() for _ in range(40)]
    gain = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
    runs = []
    for pause in (True, False):
        cache, a = csa.PagedCache(start.clone()), csa.Attention(H, D, 200, 4)
        x, res, pos = torch.empty_like(xs[0]), torch.zeros_like(xs[0]), torch.arange(B, dtype=torch.int32, device=DEV) + n - 60
        kept = []

        def wait():
            if pause:
                torch.cuda.synchronize()

        for i in range(40):
            x.copy_(xs[i])
            wait()
            o = csa.rmsnorm_residual_q8(x, res, gain, inplace=True)
            wait()
            cache.append({"latent": o["y"]}, table, pos)
            wait()
            pos += 1
            q = o["y"][:, None].expand(B, H, D) * 1
            x.fill_(math.nan)
            out, lse = a.decode(q, cache, table, pos)
            wait()
            o["y"].fill_(math.nan)
            kept.append((out, lse, o["q"].view(torch.uint8), res.clone()))
            q.fill_(math.nan)
        torch.cuda.synchronize()
        cache.status()
        assert a.device_status() == 0
        runs.append((kept, cache.latent.clone()))
    for p, q in zip(runs[0][0], runs[1][0]):
        assert all(torch.equal(x, y) for x, y in zip(p, q))
    assert torch.isfinite(runs[0][0][-1][0]).all() and torch.equal(runs[0][1], runs[1][1])
