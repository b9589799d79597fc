"""Further refusals of the serving layer's operators that need no GPU (see test_serving_refusals)."""
import ctypes

import pytest

import deepseek_v4_compressed_wkv_gb300 as csa
from test_serving_refusals import A, err, pages

MOST = 2 ** 31 - 1024  # the steps' loops look up to 256 places past the last, in 32-bit arithmetic


@pytest.mark.parametrize("kw", [dict(pages=MOST + 1), dict(pages=2 ** 31 - 1), dict(sequences=MOST + 1, max_pages=1, page_size=1),
                                dict(sequences=2 ** 31 - 1, max_pages=1), dict(sequences=1, max_pages=2 ** 31 - 1, page_size=1),
                                dict(sequences=1, max_pages=MOST + 1, page_size=1), dict(sequences=2 ** 16, max_pages=2 ** 15 - 1, page_size=1, pages=2 ** 31 - 100)])
def test_page_tables_whose_last_index_leaves_no_room(kw):
    lib, t = csa.load_library(), pages(**kw)
    at = ctypes.addressof(t)
    for rc in (lib.csa_pages_extend(at, A, A, None), lib.csa_pages_fork(at, A, A, A, A, None), lib.csa_pages_compact(at, A, A, A, None)):
        assert rc == -1 and "2^31 - 1024" in err()
    assert lib.csa_pages_workspace(t.pages, t.sequences, t.max_pages) == -1 and "2^31 - 1024" in err()


def test_the_largest_page_tables_have_a_workspace():
    lib = csa.load_library()
    assert lib.csa_pages_workspace(MOST, 1, 1) > MOST
    assert lib.csa_pages_workspace(1, 1, MOST) > MOST and lib.csa_pages_workspace(1, MOST, 1) > MOST


def meta(*shape, dtype):
    import torch
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_sizes_that_the_library_would_take_for_smaller_ones(monkeypatch):
    """The library's counts are 32-bit: 2^32 + 128 features passed on as they are would be 128."""
    import torch
    from deepseek_v4_compressed_wkv_gb300 import layer
    e4m3, i32, far = torch.float8_e4m3fn, torch.int32, 2 ** 32 + 128
    monkeypatch.setattr(layer, "_current_device", lambda: 0)
    cache = layer.PagedCache.__new__(layer.PagedCache)
    cache.device = 0
    attention = layer.Attention.__new__(layer.Attention)
    attention.heads, attention.head_dim, attention._h = 16, 64, None
    list_ = meta(far, dtype=i32)
    q, row, lens = meta(1, 16, 64, dtype=torch.bfloat16), meta(1, far, dtype=i32), meta(1, dtype=i32)
    for f in (lambda: csa.linear_q8(meta(1, far, dtype=e4m3), meta(1, far // 128, dtype=torch.float32), meta(1, far, dtype=e4m3),
                                    meta(1, far // 128, dtype=torch.float32)),
              lambda: cache.copy_pages(list_, list_), lambda: attention.decode(q, cache, row, lens),
              lambda: attention.decode(q, cache, row, lens, groups=meta(2, dtype=i32), shared=meta(1, dtype=i32)),
              lambda: csa.rmsnorm_residual_q8(meta(1, far, dtype=torch.bfloat16), None, meta(far, dtype=torch.float32))):
        with pytest.raises(csa.CSAError, match="2.31"):
            f()
