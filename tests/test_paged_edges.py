"""The paged cache's entry points at the edge of what they accept, checked without a GPU."""
import ctypes

import pytest

from gated_delta_rule_100_b200 import build as kbuild
from gated_delta_rule_100_b200 import kda

A = ctypes.c_void_p(0x10000)     # stand-in device address: only validated, never dereferenced
INV = kda.KDA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def copy(lib, pool=A, outer=2, os=1 << 20, ps=4096, nb=4096, pages=9, src=A, dst=A, n=3):
    return lib.kda_pages_copy(pool, outer, os, ps, nb, pages, src, dst, n, None)


def test_a_pool_of_no_layers_needs_no_memory(lib):
    assert copy(lib, pool=None, outer=0) == kda.KDA_OK
    assert copy(lib, pool=None) == INV
    nbytes = lib.kda_pages_compact_workspace_bytes(9)
    assert lib.kda_pages_compact_pool(None, 0, 1 << 20, 4096, 4096, 9, A, nbytes, None) == kda.KDA_OK
    assert lib.kda_pages_compact_pool(None, 1, 1 << 20, 4096, 4096, 9, A, nbytes, None) == INV


def attn(lib, strides=None, append=True, Hkv=2, ps=16, pages=9, total=5, ws=None):
    st = None if strides is None else (ctypes.c_longlong * 6)(*strides)
    new = A if append else None
    return lib.kda_paged_attn(A, new, new, A, A, A, A, A, None, 0.125, A, None, 2, total, 4, 4 * Hkv, Hkv, 64, ps, pages, 40, 2,
                              256 * Hkv, 64 * Hkv, 64 * Hkv, st, 0, ws, 0, None)


@pytest.mark.parametrize("strides,ok", [
    ((2048, 128, 64), True),                  # dense
    ((2048, 64, 1024), True),                 # heads outside a page's tokens
    ((4096, 256, 64), True),                  # keys and values of a token side by side
    ((4096, 128, 2048 + 64), True),
    ((2048, 64, 64), False),                  # a token's second head is the next token's first
    ((2048, 128, 128), False),
    ((2048, 120, 64), False),
    ((1024, 128, 64), False),                 # a page's second half is the next page
    ((2040, 128, 64), False),
    ((128, 128 * 9, 64), True),               # pages inside tokens
    ((128, 128 * 8, 64), False),
    ((64, 128 * 9, 64 * 8), False),
])
@pytest.mark.parametrize("pool", ["keys", "values"])
def test_places_that_overlap_are_refused_where_they_are_written(lib, strides, ok, pool):
    """A call without tokens ends after the checks of its arguments."""
    both = (2048, 128, 64) + strides if pool == "values" else strides + (2048, 128, 64)
    assert attn(lib, both, total=0) == (kda.KDA_OK if ok else INV)
    assert attn(lib, both, total=0, append=False) == kda.KDA_OK
    assert ok or attn(lib, both) == INV


def test_strides_along_one_place_say_nothing(lib):
    assert attn(lib, (64, 64, 64) * 2, total=0, Hkv=1, ps=1, pages=1) == kda.KDA_OK
    assert attn(lib, (64, 64, 64) * 2, total=0, Hkv=1, ps=1, pages=2) == kda.KDA_OK
    assert attn(lib, (64, 64, 64) * 2, total=0, Hkv=1, ps=2, pages=2) == INV
    assert attn(lib, (1 << 38, 1 << 38, 64) * 2, total=0, Hkv=1, ps=1, pages=1 << 30) == kda.KDA_OK
    assert attn(lib, (1 << 38, 1 << 37, 64) * 2, total=0, Hkv=1, ps=2, pages=1 << 30) == kda.KDA_OK


@pytest.mark.parametrize("os,ps,ok", [
    (9 * 4096, 4096, True), (4096, 2 * 4096, True), (17 * 4096, 2 * 4096, True),
    (4096, 4096, False), (8 * 4096, 4096, False), (16 * 4096, 2 * 4096, False), (2 * 4096, 2 * 4096, False), (0, 4096, False),
    (9 * 4096, 4080, False),
])
def test_pools_whose_pages_overlap_are_refused(lib, os, ps, ok):
    """Two layers of nine pages; a list without pairs ends after the checks."""
    nbytes = lib.kda_pages_compact_workspace_bytes(9)
    assert copy(lib, os=os, ps=ps, n=0) == (kda.KDA_OK if ok else INV)
    assert ok or lib.kda_pages_compact_pool(A, 2, os, ps, 4096, 9, A, nbytes, None) == INV
    # one layer's step, or one page's, says nothing
    assert copy(lib, os=os, ps=4096, outer=1, n=0) == kda.KDA_OK
    assert copy(lib, os=9 * 4096, ps=ps, pages=1, n=0) == kda.KDA_OK


def test_copies_have_a_longest_list(lib):
    assert copy(lib, n=(1 << 21) + 1) == kda.KDA_ERR_UNSUPPORTED
    assert copy(lib, n=(1 << 31) - 1) == kda.KDA_ERR_UNSUPPORTED
