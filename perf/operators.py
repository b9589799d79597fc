"""Workloads of the attention-layer operators: attention over a paged cache for one new token,
sliding-window attention with sinks for prompts, the cache's write, and the residual RMSNorm with an
8-bit output.

`listed()` gives fixed cases, `draw(rng)` more of the same ranges.  `run` computes them in plain
torch operations in 32 bits, or with the library's operators when `own` is set; `exact` from the
definitions in 64 bits.  Heads share one key/value row per position (key = value = latent).
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _decode(name, batch, longest, heads=64, dim=512, page=64, kind="latent", window=0, sinks=0, same=False):
    return {"name": name, "op": "decode", "batch": batch, "longest": longest, "heads": heads, "dim": dim, "page": page,
            "kind": kind, "window": window, "sinks": sinks, "same": same}


def _prefill(name, batch, tokens, heads=64, dim=512, window=128, sinks=0, start=0, ragged=False):
    return {"name": name, "op": "prefill", "batch": batch, "tokens": tokens, "heads": heads, "dim": dim,
            "window": window, "sinks": sinks, "start": start, "ragged": ragged}


def _append(name, batch, entries, dim=512, page=64, kind="latent"):
    return {"name": name, "op": "append", "batch": batch, "entries": entries, "dim": dim, "page": page, "kind": kind}


def _norm(name, rows, dim=4096, block=128):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "block": block}


def listed():
    return [
        # one conversation's first answer tokens: 33 entries of a ratio-128 layer, where latency counts
        _decode("decode 1x33", 1, 33, page=16, same=True),
        # a serving batch at positions up to 8191 of a ratio-4 layer: ragged, 0 to 2048 entries each
        _decode("decode 128x2048 latent", 128, 2048),
        # the same with the entries kept as the compressor's e2m1 codes and e4m3 scales
        _decode("decode 128x2048 fp4", 128, 2048, kind="fp4"),
        # one 131072-token document in a ratio-4 layer: the cache's length has to be split
        _decode("decode 1x32768 latent", 1, 32768, page=128, same=True),
        # the exact recent tokens of the same batch: window 128, four first tokens kept
        _decode("decode window 128+4", 128, 8191, page=32, window=128, sinks=4),
        # the exact-window attention of one layer over a 4096-token prompt
        _prefill("prefill 4096 w128", 1, 4096),
        # a padded batch of odd prompts continuing at position 300, four first tokens kept
        _prefill("prefill 4x333 w128+4", 4, 333, sinks=4, start=300, ragged=True),
        # narrow heads (the indexer's width) with a longer window
        _prefill("prefill 2x1777 d128 w512", 2, 1777, heads=16, dim=128, window=512, sinks=16),
        # a decode step writes the entries of the sequences whose group completed
        _append("append 128x1 fp4", 128, 1, kind="fp4"),
        # a prefill of 8 x 8192 tokens writes its 2048 entries a sequence
        _append("append 8x2048 latent", 8, 2048),
        # the norm in front of a decode step's layer, scales per 32 as powers of two
        _norm("norm 128 rows b32", 128, block=32),
        # the norm in front of a prompt's layer, f32 scales per 128
        _norm("norm 16461 rows b128", 16461),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prefill", "prefill", "append", "norm"))
    dim = 64 * rng.choice((1, 2, 2, 3, 4, 5, 8, 8, 8))
    heads = rng.choice((64, 64, 64, _log(rng, 1, 128)))
    page = rng.choice((16, 64, 128, _log(rng, 1, 200)))
    kind = rng.choice(("latent", "fp4"))
    window, sinks = rng.choice((0, 128, _log(rng, 1, 1024))), rng.choice((0, 4, rng.randint(0, 70)))
    if op == "decode":
        batch = _log(rng, 1, 128)
        longest = _log(rng, 1, min(32768, 262144 // batch))
        c = _decode("", batch, longest, heads, dim, page, kind, window, sinks, rng.random() < 0.3)
    elif op == "prefill":
        batch = _log(rng, 1, 8)
        window = max(1, min(window or 128, 512))
        most = min(4096 * 64 // max(heads, 64), 4096 * 132 * 512 // ((window + sinks) * dim))
        tokens = _log(rng, 1, max(1, min(4096, most // batch)))
        c = _prefill("", batch, tokens, heads, dim, window, sinks, rng.choice((0, _log(rng, 1, 2000))), rng.random() < 0.5)
    elif op == "append":
        batch = _log(rng, 1, 128)
        c = _append("", batch, _log(rng, 1, 16384 // batch), dim, page, kind)
    else:
        block = rng.choice((32, 128, 0))
        dim = (block or 32) * _log(rng, 1, 8192 // (block or 32))
        c = _norm("", _log(rng, 1, min(16461, 16461 * 4096 // dim)), dim, block)
    del c["name"]
    return c


def _lens(case, gen):
    """Entries of each sequence: the longest for all, or spread from 0 to it with both ends present."""
    b, longest = case["batch"], case["longest"]
    if case["same"]:
        return torch.full((b,), longest, dtype=torch.int32, device=DEV)
    n = torch.randint(0, longest + 1, (b,), generator=gen, device=DEV, dtype=torch.int32)
    n[0] = longest
    if b > 2:
        n[2] = 0
    return n


def _entries(shape, dim, kind, gen):
    """Normalised latents as the compressor emits them, or their e2m1 codes and e4m3 scales."""
    if kind == "latent":
        return {"latent": torch.randn(*shape, dim, generator=gen, device=DEV).bfloat16()}
    codes = torch.randint(0, 256, (*shape, dim // 2), generator=gen, device=DEV, dtype=torch.uint8)
    scales = (torch.rand(*shape, dim // 16, generator=gen, device=DEV) * 0.4 + 0.1).to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": scales.view(torch.uint8)}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    op, s = case["op"], {"case": case}
    if op in ("decode", "append"):
        b, page = case["batch"], case["page"]
        if op == "decode":
            first = _lens(case, gen)
            width = -(-case["longest"] // page)
        else:  # earlier entries of each sequence, then the new ones
            first = torch.randint(0, 2 * page, (b,), generator=gen, device=DEV, dtype=torch.int32)
            width = -(-(2 * page + case["entries"]) // page)
        pages = b * width
        s["table"] = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).view(b, width)
        s["first"] = first
        s["pool"] = _entries((pages, page), case["dim"], case["kind"], gen)
        if op == "append":
            s["new"] = _entries((b, case["entries"]), case["dim"], case["kind"], gen)
            s["mask"] = (torch.rand(b, generator=gen, device=DEV) < (0.25 if case["entries"] == 1 else 1.0)).to(torch.uint8)
            s["mask"][0] = 1
    if op == "decode":
        s["q"] = randn(case["batch"], case["heads"], case["dim"]).bfloat16()
    elif op == "prefill":
        b, n = case["batch"], case["tokens"]
        s["q"] = randn(b, n, case["heads"], case["dim"]).bfloat16()
        s["kv"] = randn(b, case["start"] + n, case["dim"]).bfloat16()
        s["lens"] = None
        if case["ragged"]:
            s["lens"] = torch.randint(0, n + 1, (b,), generator=gen, device=DEV, dtype=torch.int32)
            s["lens"][0] = n
        # rows behind a sequence's last token keep what they hold
        s["out"] = torch.zeros(b, n, case["heads"], case["dim"], dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros(b, n, case["heads"], dtype=torch.float32, device=DEV)
    elif op == "norm":
        s["x"] = randn(case["rows"], case["dim"]).bfloat16()
        s["residual"] = (2 * randn(case["rows"], case["dim"])).bfloat16()
        s["gain"] = 1 + 0.02 * randn(case["dim"])
    if own:
        import deepseek_v4_compressed_wkv_gb300 as csa
        if op in ("decode", "prefill"):
            s["attention"] = csa.Attention(case["heads"], case["dim"], window=case["window"], sinks=case["sinks"])
        if op in ("decode", "append"):
            s["cache"] = csa.PagedCache(**s["pool"])
    return s


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import deepseek_v4_compressed_wkv_gb300 as csa
    op = s["case"]["op"]
    if op == "decode":
        o, lse = s["attention"].decode(s["q"], s["cache"], s["table"], s["first"])
        return {"out": o, "lse": lse}
    if op == "prefill":
        o, lse = s["attention"].prefill(s["q"], s["kv"], start_pos=s["case"]["start"], lens=s["lens"], out=s["out"], lse=s["lse"])
        return {"out": o, "lse": lse}
    if op == "append":
        s["cache"].append(s["new"], s["table"], s["first"], mask=s["mask"])
        return s["pool"]
    return csa.rmsnorm_residual_q8(s["x"], s["residual"], s["gain"], scale_block=s["case"]["block"])


def _rows(table, index, page):
    """Pool rows of entries `index` [B, n] of each sequence."""
    p = torch.gather(table.long(), 1, (index // page).clamp(max=table.shape[1] - 1))
    return p * page + index % page


def _values(pool, rows):
    """The entries' values in 32 bits, [..., D]."""
    if "latent" in pool:
        return pool["latent"].flatten(0, 1)[rows].float()
    c = pool["codes"].flatten(0, 1)[rows].int()
    v = torch.tensor(E2M1, device=DEV)[torch.stack((c & 15, c >> 4), -1)].flatten(-2)
    a = pool["scales"].view(torch.float8_e4m3fn).flatten(0, 1)[rows].float()
    return (v.unflatten(-1, (-1, 16)) * a.unsqueeze(-1)).flatten(-2)


def _attend(q, kv, keep):
    """q [n, H, D], kv [n, K, D], keep [n, K], in 32 bits: attention and the scores' log-sum."""
    x = (q @ kv.transpose(1, 2)) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~keep.unsqueeze(1), -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = (e @ kv) / total.clamp(min=1e-38)
    return o, (torch.log(total) + top).squeeze(-1)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "decode":
        n = s["first"].long().unsqueeze(1)
        k = torch.arange(case["longest"], device=DEV).unsqueeze(0)
        if case["window"] and case["longest"] > case["window"] + case["sinks"]:
            # the first tokens, then the window's, which begins behind them
            k = k[:, : case["window"] + case["sinks"]]
            k = torch.where(k < case["sinks"], k, k - case["sinks"] + (n - case["window"]).clamp(min=case["sinks"]))
        k = k.expand(case["batch"], -1)
        o, lse = _attend(s["q"].float(), _values(s["pool"], _rows(s["table"], k, case["page"])), k < n)
        return {"out": o.bfloat16(), "lse": lse}
    if op == "prefill":
        b, n, start, w, f = case["batch"], case["tokens"], case["start"], case["window"], case["sinks"]
        t = torch.arange(start, start + n, device=DEV).unsqueeze(1)
        i = torch.arange(f + w, device=DEV).unsqueeze(0)
        j = torch.where(i < f, i, t - w + 1 + i - f)  # the first tokens, then the window, which may reach into them
        keep = (j >= 0) & (j <= t) & ((i < f) | (j >= f))
        kv = s["kv"][:, j.clamp(0, start + n - 1)].float().flatten(0, 1)
        o, lse = _attend(s["q"].float().flatten(0, 1), kv, keep.repeat(b, 1))
        o, lse = o.view(b, n, case["heads"], -1).bfloat16(), lse.view(b, n, -1)
        if s["lens"] is None:
            return {"out": o, "lse": lse}
        there = torch.arange(n, device=DEV) < s["lens"].unsqueeze(1)
        return {"out": torch.where(there[..., None, None], o, s["out"]), "lse": torch.where(there[..., None], lse, s["lse"])}
    if op == "append":
        at = s["first"].long().unsqueeze(1) + torch.arange(case["entries"], device=DEV)
        rows, there = _rows(s["table"], at, case["page"]), s["mask"].bool()
        for name, pool in s["pool"].items():
            pool.flatten(0, 1)[rows[there].flatten()] = s["new"][name][there].flatten(0, 1)
        return s["pool"]
    x = s["x"].float() + s["residual"].float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["gain"]
    block = case["block"] or case["dim"]
    b = y.unflatten(-1, (-1, block))
    a = b.abs().amax(-1).clamp(min=448 * 2.0**-126) / 448
    if block == 32:
        m, e = torch.frexp(a)
        a = torch.ldexp(torch.ones_like(a), torch.where(m == 0.5, e - 1, e))
    q = (b / a.unsqueeze(-1)).clamp(-448, 448).flatten(-2).to(torch.float8_e4m3fn)
    return {"residual": x.bfloat16(), "y": y.bfloat16(), "q": q, "scales": a.to(torch.float8_e8m0fnu) if block == 32 else a}


def work(case):
    op = case["op"]
    if op == "append":
        row = case["dim"] * 2 if case["kind"] == "latent" else case["dim"] // 2 + case["dim"] // 16
        share = 0.25 if case["entries"] == 1 else 1.0
        return {"bytes": 2 * row * max(1, share * case["batch"]) * case["entries"], "flops": 0}
    if op == "norm":
        n, block = case["rows"] * case["dim"], case["block"] or case["dim"]
        return {"bytes": n * 9 + n // block * (1 if block == 32 else 4) + case["dim"] * 4, "flops": 8 * n}
    h, d, w, f = case["heads"], case["dim"], case["window"], case["sinks"]
    if op == "decode":
        # lengths are spread evenly from 0 to the longest unless all are the same
        top, b = case["longest"], case["batch"]
        seen = lambda n: min(n, w + f) if w else n  # noqa: E731
        keys = b * seen(top) if case["same"] else seen(top) + (b - 1) * sum(seen(top * (2 * i + 1) // 64) for i in range(32)) / 32
        row = 2 * d if case["kind"] == "latent" else d // 2 + d // 16
        return {"bytes": keys * row + b * h * (4 * d + 4), "flops": 4 * h * d * keys}
    b, n, start = case["batch"], case["tokens"], case["start"]
    share = (1 + (b - 1) / 2) / b if case["ragged"] else 1.0
    keys = share * b * sum(min(t + 1, w + f) for t in range(start, start + n))
    rows = n + (min(start, w - 1 + f))
    return {"bytes": share * b * (n * h * (4 * d + 4) + rows * 2 * d), "flops": 4 * h * d * keys}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "append":
        return None  # bytes are moved, nothing is computed
    if op == "norm":
        x = s["x"].double() + s["residual"].double()
        y = x / (x.pow(2).sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * s["gain"].double()
        out = {"residual": x, "y": y, "q": torch.empty_like(y), "scales": []}
        block = case["block"] or case["dim"]
        for at in range(0, case["dim"], block):
            part = y[:, at:at + block]
            a = part.abs().max(1).values / 448
            if block == 32:
                a = torch.exp2(torch.ceil(torch.log2(a)))
            out["q"][:, at:at + block] = part / a[:, None]
            out["scales"].append(a)
        out["scales"] = torch.stack(out["scales"], 1)
        return out
    h, d, w, f = case["heads"], case["dim"], case["window"], case["sinks"]

    def attention(q, c, t):
        """Queries q [m, H, D] at positions t [m] over rows c [K, D] that begin at position 0."""
        j = torch.arange(len(c), device=DEV)
        see = (j <= t[:, None]) & ((j < f) | (j > t[:, None] - w)) if w else j <= t[:, None]
        x = torch.einsum("mhd,kd->mhk", q.double(), c) * d**-0.5
        x = torch.where(see[:, None], x, -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.where(see[:, None], torch.exp(x - lse[..., None]), 0.0)
        return torch.einsum("mhk,kd->mhd", p, c), lse

    if op == "decode":
        out = torch.zeros(case["batch"], h, d, dtype=torch.float64, device=DEV)
        lse = torch.full((case["batch"], h), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["first"].tolist()):
            if n:
                pages = s["table"][b, : -(-n // case["page"])].long()
                if "latent" in s["pool"]:
                    c = s["pool"]["latent"][pages].flatten(0, 1)[:n].double()
                else:
                    codes = s["pool"]["codes"][pages].flatten(0, 1)[:n].long()
                    c = torch.empty(n, d, dtype=torch.float64, device=DEV)
                    value = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
                    c[:, 0::2], c[:, 1::2] = value[codes % 16], value[codes // 16]
                    a = s["pool"]["scales"][pages].flatten(0, 1)[:n].view(torch.float8_e4m3fn).double()
                    c *= a.repeat_interleave(16, 1)
                o, m = attention(s["q"][b][None], c, torch.tensor([n - 1], device=DEV))
                out[b], lse[b] = o[0], m[0]
        return {"out": out, "lse": lse}
    b, n, start = case["batch"], case["tokens"], case["start"]
    out = torch.zeros(b, n, h, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(b, n, h, dtype=torch.float64, device=DEV)
    lens = [n] * b if s["lens"] is None else s["lens"].tolist()
    for i in range(b):
        for at in range(0, lens[i], 256):
            end = min(lens[i], at + 256)
            # rows before the block's oldest window stay only where they are first tokens
            low = max(0, start + at - w + 1)
            first = min(f, low)
            c = torch.cat((s["kv"][i, :first], s["kv"][i, low:start + end])).double()
            j = torch.cat((torch.arange(first, device=DEV), torch.arange(low, start + end, device=DEV)))
            t = torch.arange(start + at, start + end, device=DEV)
            see = (j <= t[:, None]) & ((j < f) | (j > t[:, None] - w))
            x = torch.einsum("mhd,kd->mhk", s["q"][i, at:end].double(), c) * d**-0.5
            x = torch.where(see[:, None], x, -math.inf)
            z = torch.logsumexp(x, -1)
            out[i, at:end] = torch.einsum("mhk,kd->mhd", torch.exp(x - z[..., None]), c)
            lse[i, at:end] = z
    return {"out": out, "lse": lse}
