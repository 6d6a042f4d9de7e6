"""The pages of a cache: pools, lists and lengths at the edge of what is documented."""
import pytest
import torch

from gated_delta_rule_100_b200 import kda
from paged_testlib import Cache

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def used():
    c = Cache(4, 4, 10, 8)
    c.reserve([0, 1, 2], [30, 9, 4])
    c.free([0])
    return c


def test_a_pool_of_no_layers_moves_nothing():
    """It has no memory to point at; the pools beside it are forked and packed."""
    c = used()
    t, ln, ref = c.cuda()
    none, real = torch.zeros((0, 10, 8), device="cuda"), torch.randn((2, 10, 8), device="cuda")
    want = real.clone()
    pairs = kda.pages_fork(t, ln, ref, ints(1), ints(3), 8, pools=[none, real])
    _, a, b = c.fork([1], [3])
    want[:, b] = want[:, a]
    assert pairs.tolist() == [a, b] and torch.equal(real, want)
    kda.pages_compact(t, ln, ref, 8, pools=[none, real])
    f, to = torch.tensor(c.compact()).T
    want[:, to] = want[:, f]
    kda.pages_copy(none, ints(0), ints(1))
    c.same(t, ln, ref)
    assert torch.equal(real, want) and kda.stream_status() == kda.KDA_OK


def test_pages_of_no_bytes_are_refused_before_the_table_changes():
    c = used()
    t, ln, ref = c.cuda()
    for bad in (torch.zeros((2, 10, 0), device="cuda"), torch.zeros((0, 10, 0), device="cuda")):
        with pytest.raises(kda.KdaError):
            kda.pages_fork(t, ln, ref, ints(1), ints(3), 8, pools=[bad])
        with pytest.raises(kda.KdaError):
            kda.pages_compact(t, ln, ref, 8, pools=[bad])
    c.same(t, ln, ref)


def test_pools_whose_pages_overlap_are_refused_before_the_table_changes():
    c = used()
    t, ln, ref = c.cuda()
    flat = torch.zeros(400, device="cuda")
    for strides in ((8, 8, 1), (72, 8, 1), (16, 16, 1), (8, 12, 1)):
        bad = flat.as_strided((2, 10, 8), strides)
        with pytest.raises(kda.KdaError):
            kda.pages_fork(t, ln, ref, ints(1), ints(3), 8, pools=[bad])
        with pytest.raises(kda.KdaError):
            kda.pages_compact(t, ln, ref, 8, pools=[bad])
        with pytest.raises(kda.KdaError):
            kda.pages_copy(bad, ints(0), ints(1))
    c.same(t, ln, ref)


@pytest.mark.parametrize("layout", ["dense", "pages first", "every other page", "every other layer"])
def test_pools_that_are_views(layout):
    x = torch.randint(0, 1 << 20, (6, 19, 8), dtype=torch.int32, device="cuda")
    pool = {"dense": x, "pages first": x.view(19, 6, 8).transpose(0, 1), "every other page": x[:, ::2],
            "every other layer": x[1::2]}[layout]
    want = pool.clone()
    want[:, [1, 4]] = want[:, [7, 0]]
    kda.pages_copy(pool, ints(7, 0), ints(1, 4))
    assert torch.equal(pool, want) and kda.stream_status() == kda.KDA_OK
