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
