"""Positions are 32-bit numbers: a page table whose columns hold more than 2^31 - 128 of them is
refused (lengths, and their sums in key tiles, would wrap)."""
import ctypes

import pytest

from tree_speculative_decoding_gated_gb300 import build, tgdn

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build.build()
    return tgdn.lib()


@pytest.mark.parametrize("page_size,most", [(16, (1 << 24)), (128, (1 << 24) - 1), (256, (1 << 23) - 1)])
def test_columns(L, page_size, most):
    def pages(cols):
        return ctypes.byref(tgdn.CPages(2, 8, page_size, cols, *[FAKE] * 5))
    pool = ctypes.byref(tgdn.CPool(1, 1, 64, FAKE))
    tree = ctypes.byref(tgdn.CTree(2, 2, 1, 4, 1, *[FAKE] * 7))
    assert L.tgdn_pages_workspace_bytes(pages(most)) > 0
    for cols in (most + 1, 2 * most):
        p = pages(cols)
        assert L.tgdn_pages_workspace_bytes(p) == 0
        assert L.tgdn_pages_reserve(p, FAKE, FAKE, None) == tgdn.ETOOBIG
        assert L.tgdn_pages_append(p, pool, 0, FAKE, None, 0, None, FAKE, 0, 64, FAKE, 0, 64, 1,
                                   None) == tgdn.ETOOBIG
        assert L.tgdn_pages_fork(p, pool, 1, FAKE, FAKE, FAKE, FAKE, None) == tgdn.ETOOBIG
        assert L.tgdn_pages_free(p, 1, FAKE, None) == tgdn.ETOOBIG
        assert L.tgdn_pages_compact(p, pool, FAKE, FAKE, None) == tgdn.ETOOBIG
        assert L.tgdn_paged_tree_attention(tree, p, 1, 1, 64, tgdn.BF16, FAKE, 64, FAKE, 64, FAKE, 64,
                                           FAKE, FAKE, 0.1, FAKE, 64, None, 0, None) == tgdn.ETOOBIG
