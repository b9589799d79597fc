"""What pages' steps and copies say of their arguments.  A fork's parents at the ends of their range: a negative one ends the
sequence and is no error, one past the last sequence ends it too and is one."""
import pytest

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_pages import dev, listed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sequences", [3, 100])  # one CTA, a cluster
@pytest.mark.parametrize("parent,told", [(-1, False), (-2, False), (-7, False), (-2 ** 31, False), (None, True), (2 ** 31 - 1, True)])
def test_a_sequence_ends(sequences, parent, told):
    t = csa.PageTable.allocate(3 * sequences, sequences, 4, 2)
    t.extend(dev([5] + [0] * (sequences - 2) + [3]))
    parents = list(range(sequences))
    parents[-1] = sequences if parent is None else parent
    assert listed(t.fork(dev(parents))) == []
    assert t.lens.tolist() == [5] + [0] * (sequences - 1) and t.refs.tolist() == [1, 1, 1] + [0] * (3 * sequences - 3)
    assert t.table[-1].tolist() == [-1] * 4
    if told:
        with pytest.raises(csa.CSAError, match="argument"):
            t.status()
    t.status()


def test_the_cache_names_the_call_that_left_a_page_out():
    c = csa.PagedCache.allocate(4, 2, 64)
    c.copy_pages(dev([1, 9]), dev([2, 3]))
    with pytest.raises(csa.CSAError, match="copy_pages .*outside"):
        c.status()
    c.status()


@pytest.mark.parametrize("sequences", [2, 100])
@pytest.mark.parametrize("page", [10 ** 9, -1, 400])
def test_a_page_outside_the_pool_that_is_only_copied_is_told(sequences, page):
    """The parent keeps its row, which nobody looks at; the heir's copy of the last page is of none."""
    t = csa.PageTable.allocate(4 * sequences, sequences, 4, 2)
    t.extend(dev([3] + [0] * (sequences - 1)))
    t.table[0, 1] = page
    assert listed(t.fork(dev([0, 0] + list(range(2, sequences))))) == [(page, 2)]
    assert t.table[1].tolist() == [0, 2, -1, -1] and t.lens.tolist()[:2] == [3, 3]
    with pytest.raises(csa.CSAError, match="outside"):
        t.status()
