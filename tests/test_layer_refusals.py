"""Refusals of the operators around the compressor that need no GPU: the C entry points check their
arguments before they touch a device, report a status and a message, and enqueue nothing."""
import ctypes
import math

import pytest

import deepseek_v4_compressed_wkv_gb300 as csa
from deepseek_v4_compressed_wkv_gb300.layer import _Cache

A = 4096  # an address that is never read: every call here is refused


def err():
    return csa.load_library().csa_last_error().decode()


def cache(**kw):
    d = dict(latent=A, codes=None, scales=None, pages=4, page_size=16, head_dim=512, fp4=1)
    d.update(kw)
    return _Cache(*(d[k] for k in ("latent", "codes", "scales", "pages", "page_size", "head_dim", "fp4")))


@pytest.mark.parametrize("args,frag", [
    ((0, 512, 0, 0, 0.0), "heads"), ((1025, 512, 0, 0, 0.0), "heads"), ((64, 0, 0, 0, 0.0), "head_dim"),
    ((64, 100, 0, 0, 0.0), "head_dim"), ((64, 576, 0, 0, 0.0), "head_dim"), ((64, 512, -1, 0, 0.0), "window"),
    ((64, 512, 128, -1, 0.0), "sinks"), ((64, 512, 0, 0, math.nan), "scale"), ((64, 512, 0, 0, math.inf), "scale"),
    ((64, 512, 0, 0, -1.0), "scale")])
def test_attention_create_refuses(args, frag):
    h = ctypes.c_void_p()
    assert csa.load_library().csa_attention_create(*args, ctypes.byref(h)) == -1 and not h.value
    assert frag in err()


def test_null_handles_and_pointers_are_refused():
    lib = csa.load_library()
    assert lib.csa_attention_create(64, 512, 0, 0, 0.0, None) == -1
    assert lib.csa_attention_prefill(None, A, A, 1, 1, 0, 1, None, A, None, None) == -1
    assert lib.csa_attention_decode(None, A, None, A, 1, A, 1, A, None, None) == -1
    assert lib.csa_attention_status(None, None) == -1
    assert lib.csa_attention_launches(None) == -1
    lib.csa_attention_destroy(None)


@pytest.mark.parametrize("kw,frag", [
    (dict(latent=None), "neither"), (dict(codes=A), "together"), (dict(codes=A, scales=A, fp4=3), "fp4"),
    (dict(pages=0), "pages"), (dict(pages=2 ** 31), "pages"), (dict(page_size=0), "page_size"), (dict(head_dim=24), "head_dim"),
    (dict(head_dim=528), "head_dim"), (dict(codes=A, scales=A, fp4=2, head_dim=48), "head_dim")])
def test_append_refuses_caches(kw, frag):
    c, o = cache(**kw), csa.Out(A, A, A, None)
    rc = csa.load_library().csa_cache_append(ctypes.addressof(c), ctypes.addressof(o), 1, 1, A, 1, A, None, None, None)
    assert rc == -1 and frag in err()


@pytest.mark.parametrize("out,B,G,table,width,first,frag", [
    ((A, None, None), 0, 1, A, 1, A, "B"), ((A, None, None), 1, 0, A, 1, A, "G"), ((A, None, None), 65536, 65536, A, 1, A, "2^31"),
    ((None, A, A), 1, 1, A, 1, A, "lack"), ((A, None, None), 1, 1, None, 1, A, "page_table"),
    ((A, None, None), 1, 1, A, 0, A, "page_table"), ((A, None, None), 1, 1, A, 1, None, "first")])
def test_append_refuses_calls(out, B, G, table, width, first, frag):
    c, o = cache(), csa.Out(*out, None)
    rc = csa.load_library().csa_cache_append(ctypes.addressof(c), ctypes.addressof(o), B, G, table, width, first, None, None, None)
    assert rc == -1 and frag in err()


@pytest.mark.parametrize("kw,frag", [
    (dict(block=64), "scale_block"), (dict(dim=100), "dim"), (dict(dim=0), "dim"), (dict(dim=16384 + 128), "dim"),
    (dict(dim=160), "dim"), (dict(rows=-1), "rows"), (dict(rows=2 ** 31), "rows"), (dict(eps=-1.0), "eps"),
    (dict(eps=math.nan), "eps"), (dict(x=None), "required"), (dict(x=A + 8), "aligned"), (dict(res=A + 2), "aligned"),
    (dict(y=A + 4), "aligned"), (dict(scales=A + 2), "aligned"), (dict(scales=None), "required")])
def test_norm_refuses(kw, frag):
    d = dict(x=A, res=A, gain=A, rows=1, dim=4096, eps=1e-6, block=128, total=A, y=A, q=A, scales=A)
    d.update(kw)
    rc = csa.load_library().csa_rmsnorm_residual_q8(d["x"], d["res"], d["gain"], d["rows"], d["dim"], d["eps"], d["block"],
                                                    d["total"], d["y"], d["q"], d["scales"], None)
    assert rc == -1 and frag in err()


def test_norm_of_no_rows_enqueues_nothing():
    assert csa.load_library().csa_rmsnorm_residual_q8(None, None, None, 0, 4096, 1e-6, 128, None, None, None, None, None) == 0
