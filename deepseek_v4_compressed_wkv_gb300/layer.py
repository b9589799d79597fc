"""Binding of the operators around the compressor: the residual RMSNorm with an 8-bit output, the matrix
product that takes it, the paged cache of entries with its page table, and attention over it or over a
prompt's own rows.

    y = rmsnorm_residual_q8(x, residual, gain)["y"]         # the compressor's x
    step = compressor.decode(y, positions)                  # entries of the groups that complete
    cache = PagedCache.allocate(pages, 64, 512)             # latent rows; fp4=1: codes and scales
    cache.append(step, page_table, index, mask=step["emitted"])
    attn = Attention(heads=64, head_dim=512)
    out, lse = attn.decode(q, cache, page_table, lens)      # one new token a sequence
    recent = Attention(64, 512, window=128, sinks=4)
    out, lse = recent.prefill(q, kv)                        # a prompt over its exact rows

and for several answers of a prompt:

    q = linear_q8(n["q"], n["scales"], weight, weight_scales)   # n: the norm with scale_block=128
    pages = PageTable.allocate(4096, 128, 256, page_size=64)
    cache.append(step, pages.table, pages.extend(more))
    cache.copy_pages(*pages.fork(parent))                   # sequence i becomes what parent[i] was
    out, lse = attn.decode(q, cache, pages.table, pages.lens, groups=groups, shared=shared)

As in the rest of the package the functions only marshal arguments; shapes and layouts are those of
``include/csa.h``.  Work runs on the current stream or on ``stream``; tensors that the call makes
belong to that stream, and those passed in are kept for it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import CSAError, Out, _check, load_library

__all__ = ["Attention", "PagedCache", "PageTable", "linear_q8", "linear_q8_status", "rmsnorm_residual_q8"]

_empty, _empty_like, _split = torch.empty, torch.empty_like, torch.split_with_sizes
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_current_device = torch.cuda.current_device
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


class _Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("refs", "table", "lens", "workspace", "status")] + [
        (n, ctypes.c_int) for n in ("pages", "sequences", "max_pages", "page_size")]


class _Cache(ctypes.Structure):
    _fields_ = [("latent", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("fp4", ctypes.c_int)]


def _want(name, t, dtype, shape, device):
    """The data pointer of a contiguous CUDA tensor of the given type and shape on the current
    device (a pointer into another GPU's memory would fault)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():  # (-1 on the CPU)
        return t.data_ptr()
    if t.dtype != dtype:
        raise CSAError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise CSAError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise CSAError(f"{name} must be a contiguous CUDA tensor")
    raise CSAError(f"{name} is on {t.device}, but the current CUDA device is cuda:{device}")


# The current stream's handle of a device: the call behind torch.cuda.current_stream(), without the
# object that it makes (3 of the 15 us that a small call takes on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


class _Here:
    """Tensors made by a call belong to its stream: a stream that is not the current one must own
    what the call makes, and keep what it reads and writes until it is done with it."""
    __slots__ = ("made",)

    def __init__(self, stream, tensors):
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
        self.made = torch.cuda.stream(stream)

    def __call__(self, make, *args, **kw):
        with self.made:
            return make(*args, **kw)


class PagedCache:
    """A paged cache of entries over the caller's arrays: latent bf16 [pages, page_size, D] and / or
    codes u8 [.., D/2] with scales u8 [.., D/16] (fp4 = 1; [.., D/32] for fp4 = 2)."""

    def __init__(self, latent=None, codes=None, scales=None, fp4: int = 1):
        if latent is None and codes is None:
            raise CSAError("a cache needs latent, or codes and scales")
        if (codes is None) != (scales is None):
            raise CSAError("codes and scales go together")
        if fp4 not in (1, 2):
            raise CSAError(f"fp4 must be 1 or 2, got {fp4}")
        base = latent if latent is not None else codes
        if base.dim() != 3 or not base.is_cuda:
            raise CSAError("a cache's arrays are CUDA tensors [pages, page_size, features]")
        self.pages, self.page_size = base.shape[0], base.shape[1]
        self.head_dim = D = latent.shape[2] if latent is not None else 2 * codes.shape[2]
        self.latent, self.codes, self.scales, self.fp4 = latent, codes, scales, fp4
        self.device = base.get_device()
        ptr = [0, 0, 0]
        at = (self.pages, self.page_size)
        if latent is not None:
            ptr[0] = _want("latent", latent, _BF16, (*at, D), self.device)
        if codes is not None:
            ptr[1] = _want("codes", codes, _U8, (*at, D // 2), self.device)
            ptr[2] = _want("scales", scales, _U8, (*at, D // (32 if fp4 == 2 else 16)), self.device)
        self._struct = _Cache(*ptr, self.pages, self.page_size, D, fp4)
        self._ref = ctypes.addressof(self._struct)
        self._arrays = [t for t in (latent, codes, scales) if t is not None]
        # Cleared here, and done when this returns: an append on another stream, or in a captured graph, must
        # not have to do it, nor its bits be cleared afterwards.
        self._flag = torch.zeros(1, dtype=_I32, device=base.device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(base.device).synchronize()
        self._append, self._copy = load_library().csa_cache_append, load_library().csa_cache_copy_pages

    @classmethod
    def allocate(cls, pages: int, page_size: int, head_dim: int, fp4: int = 0, device="cuda"):
        """A cache of latent rows (fp4 = 0), or of codes and scales (1 or 2, as the compressor's)."""
        if not fp4:
            return cls(torch.zeros(pages, page_size, head_dim, dtype=_BF16, device=device))
        block = 32 if fp4 == 2 else 16
        return cls(None, torch.zeros(pages, page_size, head_dim // 2, dtype=_U8, device=device),
                   torch.zeros(pages, page_size, head_dim // block, dtype=_U8, device=device), fp4)

    def append(self, entries: dict, page_table, first, mask=None, stream=None):
        """Writes entries (a compressor call's outputs, [B, G, ..], or [B, ..] for one each) of
        sequence b to indices first[b] .. of its pages, where mask[b] is not 0.  page_table int32
        [B, max_pages], first int32 [B], mask u8 [B] or None.  No entries: nothing is done."""
        dev = _current_device()
        if self.device != dev:
            raise CSAError(f"the cache is on cuda:{self.device}, but the current CUDA device is cuda:{dev}")
        B = first.shape[0]
        src, G = [None, None, None], None
        for i, (name, pool) in enumerate((("latent", self.latent), ("codes", self.codes), ("scales", self.scales))):
            if pool is None:
                continue
            t = entries.get(name)
            if t is None:
                raise CSAError(f"the entries lack {name}, which the cache has")
            if G is None:
                G = t.shape[1] if t.dim() == 3 else 1
            if t.shape[-1] != pool.shape[2] or t.shape[0] != B or t.numel() != B * G * pool.shape[2]:
                raise CSAError(f"{name} must be [{B}, {G}, {pool.shape[2]}], got {tuple(t.shape)}")
            src[i] = _want(name, t, pool.dtype, t.shape, dev)
        if B == 0 or G == 0:  # (a prefill of fewer tokens than a group has emits nothing)
            return
        pt = _want("page_table", page_table, _I32, (B, page_table.shape[-1]), dev)
        fi = _want("first", first, _I32, (B,), dev)
        mk = None if mask is None else _want("mask", mask, _U8, (B,), dev)
        if stream is None:
            s = _raw_stream(dev)
        else:
            _Here(stream, (*self._arrays, *(entries.get(n) for n in ("latent", "codes", "scales")), page_table, first, mask,
                           self._flag))
            s = stream.cuda_stream
        out = Out(*src, None)
        rc = self._append(self._ref, ctypes.addressof(out), B, G, pt, page_table.shape[1], fi, mk, self._flag.data_ptr(), s)
        if rc < 0:
            _check(rc, "csa_cache_append")

    def copy_pages(self, src, dst, count=None, stream=None):
        """Copies page src[i] to page dst[i] (int32 [n] each) of every array, for i < n, or i < count (int32 [1] on
        the device): the lists of PageTable.fork and .compact.  No page may be written twice, or read and written,
        in one call."""
        dev = _current_device()
        if self.device != dev:
            raise CSAError(f"the cache is on cuda:{self.device}, but the current CUDA device is cuda:{dev}")
        if src.dim() != 1 or src.shape[0] >= 2 ** 31:
            raise CSAError(f"src must be [n], n below 2^31, got {tuple(src.shape)}")
        sp, dp = _want("src", src, _I32, src.shape, dev), _want("dst", dst, _I32, src.shape, dev)
        cp = None if count is None else _want("count", count, _I32, (1,), dev)
        if stream is None:
            s = _raw_stream(dev)
        else:
            _Here(stream, (*self._arrays, src, dst, count, self._flag))
            s = stream.cuda_stream
        rc = self._copy(self._ref, sp, dp, src.shape[0], cp, self._flag.data_ptr(), s)
        if rc < 0:
            _check(rc, "csa_cache_copy_pages")

    def status(self, stream=None):
        """Raises CSAError if an append since the last call left an entry out (a negative index, an
        index beyond the page table, or a page outside the cache), or copy_pages a page.  Reads and clears the cache's status
        word on the current stream or on ``stream``, and waits for it: appends on other streams have to
        be ordered before it (events, wait_stream), like all work on one cache."""
        with torch.cuda.stream(stream):
            seen = self._flag.clone()
            self._flag.zero_()
            bits = int(seen.item())
        if bits:
            what = [w for b, w in ((1, "a negative index"), (2, "an index beyond the page table"),
                                   (4, "a page outside the cache"),
                                   (8, "a store outside the cache (bounds-checked build)")) if bits & b]
            raise CSAError("append left entries out, or copy_pages pages: " + ", ".join(what))


class PageTable:
    """The page table of paged caches over the caller's arrays, all int32: refs [pages] (sequences that have a page;
    0: free), table [sequences, max_pages] (also the page_table of PagedCache.append and Attention.decode) and lens
    [sequences].  One table serves the caches of all layers.  Its steps run on the device, one after the other (one
    stream, or events between streams).  What a step returns are arrays of the table's own, which its next step of
    the same kind writes again: the caches take them before that, or a copy is made of them."""

    def __init__(self, refs, table, lens, page_size: int):
        if refs.dim() != 1 or table.dim() != 2 or lens.dim() != 1 or not refs.is_cuda:
            raise CSAError("a page table's arrays are CUDA tensors refs [pages], table [sequences, max_pages] and lens [sequences]")
        self.refs, self.table, self.lens, self.page_size = refs, table, lens, page_size
        self.pages, (self.sequences, self.max_pages), self.device = refs.shape[0], table.shape, refs.get_device()
        ptr = [_want("refs", refs, _I32, refs.shape, self.device), _want("table", table, _I32, table.shape, self.device),
               _want("lens", lens, _I32, (self.sequences,), self.device)]
        self._lib = load_library()
        if max(self.pages, self.sequences, self.max_pages, page_size) >= 2 ** 31:
            raise CSAError("pages, sequences, max_pages and page_size must be below 2^31")
        n = _check(self._lib.csa_pages_workspace(self.pages, self.sequences, self.max_pages), "csa_pages_workspace")
        self._work = torch.empty(n, dtype=_I32, device=refs.device)
        ints = functools.partial(torch.zeros, dtype=_I32, device=refs.device)
        n, most = self.sequences, max(1, self.pages // 2)
        self._flag = ints(1)
        self._rows, self._first = (n,), ints(n)
        self._forks = _split(ints(2 * n + 1), (n, n, 1))
        self._moves = _split(ints(2 * most + 1), (most, most, 1))
        # All of them are there when this returns (as a cache's word): a step on another stream must not find a fill
        # behind it, which would take its count and lists back.
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(refs.device).synchronize()
        self._at = [t.data_ptr() for t in (self._first, *self._forks, *self._moves)]
        self._struct = _Pages(*ptr, self._work.data_ptr(), self._flag.data_ptr(), self.pages, self.sequences, self.max_pages,
                              page_size)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def allocate(cls, pages: int, sequences: int, max_pages: int, page_size: int, device="cuda"):
        """A table of `sequences` sequences without entries over `pages` free pages."""
        return cls(torch.zeros(pages, dtype=_I32, device=device),
                   torch.full((sequences, max_pages), -1, dtype=_I32, device=device),
                   torch.zeros(sequences, dtype=_I32, device=device), page_size)

    def _step(self, stream, *used):
        """The stream handle of a call."""
        dev = _current_device()
        if self.device != dev:
            raise CSAError(f"the page table is on cuda:{self.device}, but the current CUDA device is cuda:{dev}")
        if stream is None:
            return _raw_stream(dev)
        _Here(stream, (self.refs, self.table, self.lens, self._work, self._flag, self._first, *self._forks, *self._moves, *used))
        return stream.cuda_stream

    def extend(self, more, stream=None):
        """Every sequence gets pages for more[b] >= 0 new entries (int32 [sequences]) and is as much longer.
        Returns where they begin, int32 [sequences]: append's `first` (-1 where the pages have run out or the
        row is full; status tells)."""
        s = _raw_stream(self.device) if stream is None and _current_device() == self.device else self._step(stream, more)
        mp = _want("more", more, _I32, self._rows, self.device)
        rc = self._lib.csa_pages_extend(self._ref, mp, self._at[0], s)
        if rc < 0:
            _check(rc, "csa_pages_extend")
        return self._first

    def fork(self, parent, stream=None):
        """Sequence i becomes what sequence parent[i] was (int32 [sequences]; negative: it ends, its pages are free).  Full
        pages are shared, each page that is not full stays with one heir.  Returns (src, dst, count), the copies
        that every cache then has to make: cache.copy_pages(*table.fork(parent))."""
        s = _raw_stream(self.device) if stream is None and _current_device() == self.device else self._step(stream, parent)
        pp = _want("parent", parent, _I32, self._rows, self.device)
        at = self._at
        rc = self._lib.csa_pages_fork(self._ref, pp, at[1], at[2], at[3], s)
        if rc < 0:
            _check(rc, "csa_pages_fork")
        return self._forks

    def compact(self, stream=None):
        """Moves the pages in use to the front of the pool.  Returns (src, dst, count) for copy_pages, as fork."""
        s = _raw_stream(self.device) if stream is None and _current_device() == self.device else self._step(stream)
        at = self._at
        rc = self._lib.csa_pages_compact(self._ref, at[4], at[5], at[6], s)
        if rc < 0:
            _check(rc, "csa_pages_compact")
        return self._moves

    def status(self, stream=None):
        """Raises CSAError if a step since the last call could not be done in full.  Reads and clears the table's
        status word on the current stream or on ``stream``, and waits for it."""
        with torch.cuda.stream(stream):
            seen = self._flag.clone()
            self._flag.zero_()
            bits = int(seen.item())
        if bits:
            what = [w for b, w in ((1, "the pages ran out"), (2, "an argument or a length out of range"),
                                   (4, "a page outside the pool in the table"),
                                   (8, "a store out of bounds (bounds-checked build)")) if bits & b]
            raise CSAError("page table: " + ", ".join(what))


class Attention:
    """Attention of `heads` query heads over one shared key/value row of head_dim features per
    position: all earlier positions, or the last `window` and the first `sinks`."""

    def __init__(self, heads: int, head_dim: int, window: int = 0, sinks: int = 0, scale: float = 0.0):
        self._lib = load_library()
        if max(heads, head_dim, window, sinks) >= 2 ** 31 or min(heads, head_dim, window, sinks) < 0:
            raise CSAError("heads, head_dim, window and sinks must be in [0, 2^31)")
        self.heads, self.head_dim, self.window, self.sinks = heads, head_dim, window, sinks
        h = ctypes.c_void_p()
        _check(self._lib.csa_attention_create(heads, head_dim, window, sinks, scale or 0.0, ctypes.byref(h)),
               "csa_attention_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            self._lib.csa_attention_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def prefill(self, q, kv, start_pos: int = 0, lens=None, out=None, lse=None, stream=None):
        """q bf16 [B, N, heads, head_dim]: tokens start_pos .. of each sequence; kv bf16 [B, rows,
        head_dim], rows >= start_pos + N; lens int32 [B]: tokens of each sequence in a padded batch
        (outputs of the others are left as they were).  Returns (out bf16 like q, lse f32 [B, N, heads]).
        No sequences or no tokens: nothing is done."""
        if q.dim() != 4 or kv.dim() != 3:
            raise CSAError("q must be [B, N, heads, head_dim] and kv [B, rows, head_dim]")
        B, N = q.shape[0], q.shape[1]
        if start_pos < 0 or start_pos + N > kv.shape[1]:
            raise CSAError(f"start_pos {start_pos} must be >= 0 and start_pos + {N} at most kv's {kv.shape[1]} rows")
        dev = _current_device()
        shape, lshape = (B, N, self.heads, self.head_dim), (B, N, self.heads)
        qp = _want("q", q, _BF16, shape, dev)
        kp = _want("kv", kv, _BF16, (B, kv.shape[1], self.head_dim), dev)
        lp = None if lens is None else _want("lens", lens, _I32, (B,), dev)
        op, out, zp, lse, s = self._outputs(q, out, lse, shape, lshape, dev, stream, (q, kv, lens, out, lse))
        if B == 0 or N == 0:
            return out, lse
        rc = self._lib.csa_attention_prefill(self._h, qp, kp, B, N, start_pos, kv.shape[1], lp, op, zp, s)
        if rc < 0:
            _check(rc, "csa_attention_prefill")
        return out, lse

    def _outputs(self, q, out, lse, shape, lshape, dev, stream, used):
        """(pointer, out, pointer, lse, stream handle) of a call."""
        if stream is None:
            s = _raw_stream(dev)
            if out is None and lse is None:  # (nothing of the caller's to check)
                out, lse = _empty_like(q), _empty(lshape, dtype=_F32, device=q.device)
                return out.data_ptr(), out, lse.data_ptr(), lse, s
            out = _empty_like(q) if out is None else out
            lse = _empty(lshape, dtype=_F32, device=q.device) if lse is None else lse
        else:
            make, s = _Here(stream, used), stream.cuda_stream
            out = make(_empty_like, q) if out is None else out
            lse = make(_empty, lshape, dtype=_F32, device=q.device) if lse is None else lse
        return _want("out", out, _BF16, shape, dev), out, _want("lse", lse, _F32, lshape, dev), lse, s

    def decode(self, q, cache: PagedCache, page_table, lens, out=None, lse=None, stream=None, groups=None, shared=None):
        """q bf16 [B, heads, head_dim]: one new token a sequence, at position lens[b] - 1 (lens int32
        [B] on the device) of its entries in the cache; page_table int32 [B, max_pages].  Returns
        (out bf16 like q, lse f32 [B, heads]).  No sequences: nothing is done.

        groups int32 [G + 1] with shared int32 [G], 1 <= G <= B: sequences groups[g] .. groups[g + 1] - 1 have their
        first shared[g] entries in common (the full pages that PageTable.fork shares), which are then read with all
        of the group's queries together where the number of heads and the table's width promise that it pays.  The
        sequences' lengths are not known here: few shared entries in a wide table can take longer than without groups
        (figures in include/csa.h).  Only without a window."""
        if q.dim() != 3 or page_table.dim() != 2 or page_table.shape[1] >= 2 ** 31:
            raise CSAError("q must be [B, heads, head_dim] and page_table [B, max_pages], max_pages below 2^31")
        B = q.shape[0]
        dev = _current_device()
        if cache.device != dev:
            raise CSAError(f"the cache is on cuda:{cache.device}, but the current CUDA device is cuda:{dev}")
        shape, lshape = (B, self.heads, self.head_dim), (B, self.heads)
        qp = _want("q", q, _BF16, shape, dev)
        width = page_table.shape[1]
        pp = _want("page_table", page_table, _I32, (B, width), dev)
        lp = _want("lens", lens, _I32, (B,), dev)
        op, out, zp, lse, s = self._outputs(q, out, lse, shape, lshape, dev, stream,
                                            (q, page_table, lens, out, lse, *cache._arrays))
        if groups is not None or shared is not None:
            self._decode_shared(qp, cache, pp, width, lp, B, groups, shared, op, zp, s, dev, stream, q.device)
            return out, lse
        if B == 0:
            return out, lse
        rc = self._lib.csa_attention_decode(self._h, qp, cache._ref, pp, width, lp, B, op, zp, s)
        if rc < 0:
            _check(rc, "csa_attention_decode")
        return out, lse

    def _decode_shared(self, qp, cache, pp, width, lp, B, groups, shared, op, zp, s, dev, stream, device):
        if groups is None or shared is None or shared.dim() != 1:
            raise CSAError("groups [G + 1] and shared [G] go together")
        G = shared.shape[0]
        gp, hp = _want("groups", groups, _I32, (G + 1,), dev), _want("shared", shared, _I32, (G,), dev)
        if G > B or (G < 1 and B > 0):
            raise CSAError(f"there must be 1 to {B} groups, got {G}")
        if B == 0:
            return
        n = self._lib.csa_attention_shared_workspace(self._h, B, G, width, cache.page_size)
        if n < 0:
            _check(n, "csa_attention_shared_workspace")
        work = None
        if n and stream is None:
            work = _empty(n, dtype=_U8, device=device)
        elif stream is not None:
            here = _Here(stream, (groups, shared))
            work = here(_empty, n, dtype=_U8, device=device) if n else None
        rc = self._lib.csa_attention_decode_shared(self._h, qp, cache._ref, pp, width, lp, B, gp, hp, G,
                                                   None if work is None else work.data_ptr(), op, zp, s)
        if rc < 0:
            _check(rc, "csa_attention_decode_shared")

    def kernel_launches(self) -> int:
        return _check(self._lib.csa_attention_launches(self._h), "csa_attention_launches")

    def device_status(self, stream=None):
        s = _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream
        return _check(self._lib.csa_attention_status(self._h, s), "csa_attention_status")


def rmsnorm_residual_q8(x, residual, gain, eps: float = 1e-6, scale_block: int = 128, y: bool = True, inplace: bool = False,
                        stream=None) -> dict:
    """x bf16 [.., dim] plus residual (or None), normalised by its root mean square with gain f32 [dim].
    Returns residual (the sum, bf16, written over the one passed in with inplace; x itself without a
    residual), y (bf16, None without y), q (float8_e4m3fn) and its scales: f32 [.., dim / 128] (scale_block 128), f32 [.., 1]
    (0: one per row) or float8_e8m0fnu [.., dim / 32] (32)."""
    shape = x.shape
    dim = shape[-1]
    if scale_block not in (0, 32, 128):
        raise CSAError(f"scale_block must be 0, 32 or 128, got {scale_block}")
    if dim == 0 or dim % (128 if scale_block == 128 else 32) or dim >= 2 ** 31:
        raise CSAError(f"the last dimension must be a multiple of {128 if scale_block == 128 else 32} below 2^31, got {dim}")
    if inplace and residual is None:
        raise CSAError("inplace writes over a residual: none was given")
    dev = _current_device()
    xp = _want("x", x, _BF16, shape, dev)
    rp = None if residual is None else _want("residual", residual, _BF16, shape, dev)
    gp = _want("gain", gain, _F32, (dim,), dev)
    if stream is None:
        empty, like, s = _empty, _empty_like, _raw_stream(dev)
    else:
        make, s = _Here(stream, (x, residual, gain)), stream.cuda_stream
        empty, like = functools.partial(make, _empty), functools.partial(make, _empty_like)
    total = x if residual is None else residual if inplace else like(x)
    yt = like(x) if y else None
    q = like(x, dtype=_E4M3)
    scales = empty(shape[:-1] + (dim // (scale_block or dim),), dtype=_E8M0 if scale_block == 32 else _F32, device=x.device)
    rc = load_library().csa_rmsnorm_residual_q8(xp, rp, gp, x.numel() // dim, dim, eps, scale_block,
                                                None if residual is None else total.data_ptr(),
                                                None if yt is None else yt.data_ptr(), q.data_ptr(), scales.data_ptr(), s)
    if rc < 0:
        _check(rc, "csa_rmsnorm_residual_q8")
    return {"residual": total, "y": yt, "q": q, "scales": scales}


def linear_q8(q, scales, weight, weight_scales, dtype=_BF16, out=None, stream=None):
    """q float8_e4m3fn [.., K] with scales f32 [.., K / 128] (as rmsnorm_residual_q8 leaves them with scale_block
    128) times weight float8_e4m3fn [N, K] with weight_scales f32 [ceil(N / 128), K / 128]: dtype bf16 or f32
    [.., N].  A row's last bits may depend on the number of rows.  No rows or no columns: nothing is done."""
    if weight.dim() != 2 or q.dim() < 1:
        raise CSAError("q must be [.., K] and weight [N, K]")
    N, K = weight.shape
    if K == 0 or K % 128 or K >= 2 ** 31:
        raise CSAError(f"the last dimension must be a positive multiple of 128 below 2^31, got {K}")
    if dtype is not _BF16 and dtype is not _F32:
        raise CSAError(f"dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    blocks = K // 128
    lead = (q.shape[0],) if q.dim() == 2 else tuple(q.shape[:-1])
    dev = _current_device()
    qp = _want("q", q, _E4M3, (*lead, K), dev)
    ap = _want("scales", scales, _F32, (*lead, blocks), dev)
    wp = _want("weight", weight, _E4M3, (N, K), dev)
    bp = _want("weight_scales", weight_scales, _F32, ((N + 127) // 128, blocks), dev)
    if stream is None:
        s = _raw_stream(dev)
        if out is None:
            out = _empty((*lead, N), dtype=dtype, device=q.device)
            op = out.data_ptr()
        else:
            op = _want("out", out, dtype, (*lead, N), dev)
    else:
        make, s = _Here(stream, (q, scales, weight, weight_scales, out)), stream.cuda_stream
        if out is None:
            out = make(_empty, (*lead, N), dtype=dtype, device=q.device)
        op = _want("out", out, dtype, (*lead, N), dev)
    T = q.numel() // K
    if T == 0 or N == 0:
        return out
    rc = load_library().csa_linear_q8(qp, ap, wp, bp, T, N, K, op, dtype is _F32, s)
    if rc < 0:
        _check(rc, "csa_linear_q8")
    return out


def linear_q8_status(stream=None):
    """Raises CSAError if a linear_q8 on the current device, from any thread or stream, since the last call ran out of
    a wait's time.  Reads and clears the device's flag on the current stream or on ``stream``, and waits for it: calls
    still running on other streams are the next look's."""
    s = _raw_stream(_current_device()) if stream is None else stream.cuda_stream
    _check(load_library().csa_linear_q8_status(s), "csa_linear_q8_status")
