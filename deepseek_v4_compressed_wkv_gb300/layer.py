"""Binding of the operators around the compressor: the residual RMSNorm with an 8-bit output, the
paged cache of entries, and attention over it or over a prompt's own rows.

    y = rmsnorm_residual_q8(x, residual, gain)["y"]         # the compressor's x
    step = compressor.decode(y, positions)                  # entries of the groups that complete
    cache = PagedCache.allocate(pages, 64, 512)             # latent rows; fp4=1: codes and scales
    cache.append(step, page_table, index, mask=step["emitted"])
    attn = Attention(heads=64, head_dim=512)
    out, lse = attn.decode(q, cache, page_table, lens)      # one new token a sequence
    recent = Attention(64, 512, window=128, sinks=4)
    out, lse = recent.prefill(q, kv)                        # a prompt over its exact rows

As in the rest of the package the functions only marshal arguments; shapes and layouts are those of
``include/csa.h``.  Work runs on the current stream or on ``stream``; tensors that the call makes
belong to that stream, and those passed in are kept for it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import CSAError, Out, _check, load_library

__all__ = ["Attention", "PagedCache", "rmsnorm_residual_q8"]

_empty, _empty_like = torch.empty, torch.empty_like
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_current_device = torch.cuda.current_device
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


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
        self._append = load_library().csa_cache_append

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

    def status(self, stream=None):
        """Raises CSAError if an append since the last call left an entry out (a negative index, an
        index beyond the page table, or a page outside the cache).  Reads and clears the cache's status
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
            raise CSAError("append left entries out: " + ", ".join(what))


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

    def decode(self, q, cache: PagedCache, page_table, lens, out=None, lse=None, stream=None):
        """q bf16 [B, heads, head_dim]: one new token a sequence, at position lens[b] - 1 (lens int32
        [B] on the device) of its entries in the cache; page_table int32 [B, max_pages].  Returns
        (out bf16 like q, lse f32 [B, heads]).  No sequences: nothing is done."""
        if q.dim() != 3 or page_table.dim() != 2:
            raise CSAError("q must be [B, heads, head_dim] and page_table [B, max_pages]")
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
        if B == 0:
            return out, lse
        rc = self._lib.csa_attention_decode(self._h, qp, cache._ref, pp, width, lp, B, op, zp, s)
        if rc < 0:
            _check(rc, "csa_attention_decode")
        return out, lse

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
    if dim == 0 or dim % (128 if scale_block == 128 else 32):
        raise CSAError(f"the last dimension must be a multiple of {128 if scale_block == 128 else 32}, got {dim}")
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
