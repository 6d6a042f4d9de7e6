"""The pages of a cache: pools, lists and lengths at the edge of what is documented."""
import numpy as np
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


@pytest.mark.parametrize("n,outer", [(700, 1), (2600, 1), (5000, 3), (40_000, 1), (300_000, 1), (1_300_000, 1)])
def test_long_copies_leave_out_what_is_named_twice(n, outer):
    """Lists by which a block copies one pair, some, many, and more than it looks up at once: destinations named twice near each other
    and at the list's two ends, or read elsewhere, pages out of range, pairs skipped and onto themselves."""
    gen = torch.Generator().manual_seed(n)
    pages = 2 * n + 50
    ids = torch.randperm(pages, generator=gen).int()
    src, dst = ids[:n].clone(), ids[n: 2 * n].clone()
    src[torch.randint(n, (n // 7,), generator=gen)] = int(src[0])  # a source may be read often
    dst[n - 1] = dst[1]                                       # written by the first block and by the last
    dst[n // 2 + 1] = dst[n // 2]
    src[n // 3] = dst[n // 5]
    dst[5] = src[5]
    src[7] = dst[5 + n // 2]                                  # read by one, written by another
    src[11], dst[11] = -1, -1
    src[n - 20], dst[n - 20] = -1, -1
    dst[13], src[17], dst[19] = pages, -1, -1
    pool = torch.randint(0, 1 << 30, (outer, pages, 4), dtype=torch.int32, generator=gen)
    want = pool.clone()
    s, d = src.long(), dst.long()
    fine = (s >= 0) & (s < pages) & (d >= 0) & (d < pages)
    times = torch.zeros(pages, dtype=torch.long)
    times.index_add_(0, d[(d >= 0) & (d < pages)], torch.ones_like(d[(d >= 0) & (d < pages)]))
    times.index_add_(0, s[(s >= 0) & (s < pages)], torch.ones_like(s[(s >= 0) & (s < pages)]))
    keep = fine & (s != d) & (times[d.clamp(0, pages - 1)] == 1)
    assert 0 < int(keep.sum()) < n - 8
    want[:, d[keep]] = pool[:, s[keep]]
    x = pool.cuda()
    kda.pages_copy(x, src.cuda(), dst.cuda())
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(x.cpu(), want)
    good = keep.nonzero()[:, 0]
    x = pool.cuda()
    kda.pages_copy(x, src[good].cuda(), dst[good].cuda())
    assert kda.stream_status() == kda.KDA_OK and torch.equal(x.cpu(), want)


@pytest.mark.parametrize("bad", [-1, -(1 << 31), 33, (1 << 31) - 1])
def test_lengths_that_cannot_be_are_reported(bad):
    """By the calls that end or renumber rows too; what the table holds within its bounds is still done."""
    c = Cache(4, 4, 10, 8)
    c.reserve([0, 1], [32, 9])
    t, ln, ref = c.cuda()
    ln[0] = bad
    kda.pages_free(t, ln, ref, ints(0), 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    assert int(ln[0]) == 0 and int((ref == 0).sum()) == (8 if bad > 0 else 4) and torch.equal(t[1].cpu(), torch.from_numpy(c.table[1]))
    t, ln, ref = c.cuda()
    ln[3] = bad
    t[3] = t[0]  # four live pages, so that the length alone is what is wrong
    kda.pages_compact(t, ln, ref, 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    c.compact()
    assert torch.equal(t[:2].cpu(), torch.from_numpy(c.table[:2])) and torch.equal(ref.cpu(), torch.from_numpy(c.ref))


def test_lengths_of_whole_tables_are_fine():
    c = Cache(4, 4, 10, 8)
    c.reserve([0, 1], [32, 25])
    t, ln, ref = c.cuda()
    kda.pages_compact(t, ln, ref, 8)
    c.compact()
    c.same(t, ln, ref)
    kda.pages_free(t, ln, ref, ints(0, 1, 2), 8)
    c.free([0, 1, 2])
    c.same(t, ln, ref)
    assert kda.stream_status() == kda.KDA_OK


@pytest.mark.parametrize("page", [-1, 10, 1 << 30, -(1 << 31)])
def test_a_fork_reports_a_last_page_that_is_none(page):
    c = Cache(4, 4, 10, 8)
    c.reserve([0], [12])
    t, ln, ref = c.cuda()
    t[0, 1] = page
    pairs = kda.pages_fork(t, ln, ref, ints(0), ints(2), 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    assert pairs.tolist() == [[page], [2]]


def test_pools_of_more_pages_than_the_flags_that_are_kept():
    """300,001 pages are past the first eight steps of a warp, so that the second pass reads counts again; nearly all of
    them in use, the free ones in runs all over the pool."""
    c = Cache(1024, 300, 300_001, 2)
    r = np.random.default_rng(4)
    t, ln, ref = c.cuda()
    info = ints(0)

    def reserve(rows, new):
        kda.pages_reserve(t, ln, ref, ints(*rows), ints(*new), 2, info=info)
        assert info.item() == c.reserve(rows, new)
        c.same(t, ln, ref)

    reserve(list(range(1000)), [600 - int(x) for x in r.integers(0, 2, 1000)])
    for _ in range(2):
        gone = r.permutation(1000)[:100].tolist()
        kda.pages_free(t, ln, ref, ints(*gone), 2)
        c.free(gone)
        c.same(t, ln, ref)
        reserve(gone[:60], [int(x) for x in r.integers(0, 601, 60)])
        src, dst = [k for k in range(1000) if c.length[k]][-40:], gone[60:]
        pairs = kda.pages_fork(t, ln, ref, ints(*src), ints(*dst), 2, info=info)
        left, a, b = c.fork(src, dst)
        assert (info.item(), pairs.tolist()) == (left, [a, b])
        c.same(t, ln, ref)
    kda.pages_compact(t, ln, ref, 2, info=info)
    c.compact()
    c.same(t, ln, ref)
    assert kda.stream_status() == kda.KDA_OK
