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
