"""The pages of a cache against the same lists on the host, and a run of a hybrid stack's step on them."""
import numpy as np
import pytest
import torch

from gated_delta_rule_100_b200 import kda
from paged_testlib import Cache

pytestmark = pytest.mark.gpu


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fill(R, P, pages, ps, seed, share=True):
    """A cache in use: reservations, forks and frees in random order."""
    r = np.random.default_rng(seed)
    c = Cache(R, P, pages, ps)
    for _ in range(3 * R):
        row = int(r.integers(R))
        if c.length[row]:
            if r.random() < 0.5:
                c.free([row])
            continue
        busy = [k for k in range(R) if c.length[k]]
        if share and busy and r.random() < 0.3:
            c.fork([busy[int(r.integers(len(busy)))]], [row])
        else:
            c.reserve([row], [int(r.integers(0, P * ps + 1))])
    return c, r


SHAPES = [(1, 1, 1, 1), (3, 5, 11, 16), (8, 4, 20, 7), (40, 16, 300, 16), (200, 33, 5001, 64), (70, 128, 9000, 3)]


@pytest.mark.parametrize("R,P,pages,ps", SHAPES)
@pytest.mark.parametrize("seed", range(3))
def test_lists_follow_the_host(R, P, pages, ps, seed):
    """Long runs of calls on one cache, each compared whole."""
    c, r = fill(R, P, pages, ps, seed)
    t, ln, ref = c.cuda()
    info = ints(-77)
    for step in range(12):
        rows = r.permutation(R)[: int(r.integers(1, R + 1))]
        kind = ["reserve", "fork", "free", "compact"][step % 4]
        if kind == "free":
            rows = rows[: max(1, len(rows) // 3)]
            kda.pages_free(t, ln, ref, ints(*rows.tolist()), ps)
            c.free(rows)
        elif kind == "reserve":
            new = [int(r.integers(c.length[k], P * ps + 1)) for k in rows]
            kda.pages_reserve(t, ln, ref, ints(*rows.tolist()), ints(*new), ps, info=info)
            assert c.reserve(rows, new) == info.item()
        elif kind == "fork":
            dst = [k for k in rows if c.length[k] == 0]
            src = [k for k in range(R) if k not in dst]
            if not dst or not src:
                continue
            src = [src[int(r.integers(len(src)))] for _ in dst]
            a, b = kda.pages_fork(t, ln, ref, ints(*src), ints(*[int(k) for k in dst]), ps, info=info)
            left, x, y = c.fork(src, dst)
            assert (info.item(), a.tolist(), b.tolist()) == (left, x, y)
        else:
            kda.pages_compact(t, ln, ref, ps, info=info)
            c.compact()
            assert info.item() == int((c.ref == 0).sum())
        assert kda.stream_status() == kda.KDA_OK
        c.same(t, ln, ref)


@pytest.mark.parametrize("seed", range(2))
def test_large_pool(seed):
    """Page numbers past every slice of the cluster's CTAs, a list of thousands."""
    c = Cache(4096, 40, 150001, 16)
    r = np.random.default_rng(seed)
    t, ln, ref = c.cuda()
    info = ints(0)
    for _ in range(2):
        rows = r.permutation(4096)[:3001]
        rows = np.array([k for k in rows if c.length[k] == 0])
        new = r.integers(0, 641, len(rows))
        kda.pages_reserve(t, ln, ref, ints(*rows.tolist()), ints(*new.tolist()), 16, info=info)
        assert info.item() == c.reserve(rows, new)
        c.same(t, ln, ref)
        gone = r.permutation(4096)[:1500]
        kda.pages_free(t, ln, ref, ints(*gone.tolist()), 16)
        c.free(gone)
        c.same(t, ln, ref)
    src = [k for k in range(4096) if c.length[k]][:50]
    dst = [k for k in range(4096) if not c.length[k]][:1000]
    src = [src[i % 50] for i in range(1000)]
    a, b = kda.pages_fork(t, ln, ref, ints(*src), ints(*dst), 16, info=info)
    assert (info.item(), a.tolist(), b.tolist()) == c.fork(src, dst)
    c.same(t, ln, ref)
    kda.pages_compact(t, ln, ref, 16, info=info)
    c.compact()
    c.same(t, ln, ref)
    assert kda.stream_status() == kda.KDA_OK


def test_ref_that_is_not_16_byte_aligned():
    c, _ = fill(20, 8, 100, 4, 3)
    t, ln, ref = c.cuda()
    buf = torch.zeros(101, dtype=torch.int32, device="cuda")
    odd = buf[1:]
    odd.copy_(ref)
    rows = [k for k in range(20) if c.length[k] == 0][:2]
    kda.pages_reserve(t, ln, odd, ints(*rows), ints(5, 6)[: len(rows)], 4)
    c.reserve(rows, [5, 6])
    kda.pages_compact(t, ln, odd, 4)
    c.compact()
    c.same(t, ln, odd)


@pytest.mark.parametrize("bad", ["twice", "range", "negative", "shrinks", "long"])
def test_reserve_refuses_a_bad_list_whole(bad):
    c, _ = fill(12, 4, 40, 8, 1)
    c.free(range(12))
    c.reserve([3], [9])
    t, ln, ref = c.cuda()
    rows, new = [1, 2, 3], [4, 5, 10]
    if bad == "twice":
        rows[1] = 1
    elif bad == "range":
        rows[1] = 12
    elif bad == "negative":
        rows[1] = -1
    elif bad == "shrinks":
        new[2] = 8
    else:
        new[1] = 33
    kda.pages_reserve(t, ln, ref, ints(*rows), ints(*new), 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    c.same(t, ln, ref)


@pytest.mark.parametrize("bad", ["dst twice", "dst range", "src range", "dst in use", "src is dst"])
def test_fork_refuses_a_bad_list_whole(bad):
    c = Cache(8, 4, 40, 8)
    c.reserve([0, 1], [9, 20])
    t, ln, ref = c.cuda()
    src, dst = [0, 1, 0], [4, 5, 6]
    if bad == "dst twice":
        dst[1] = 4
    elif bad == "dst range":
        dst[1] = 8
    elif bad == "src range":
        src[1] = -3
    elif bad == "dst in use":
        dst[1] = 1
    else:
        src[1] = 6
    a, b = kda.pages_fork(t, ln, ref, ints(*src), ints(*dst), 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    c.same(t, ln, ref)
    assert a.tolist() == b.tolist() == [-1] * 3


def test_free_refuses_a_bad_list_whole():
    c = Cache(8, 4, 40, 8)
    c.reserve([0, 1], [9, 20])
    t, ln, ref = c.cuda()
    for rows in ([0, 0], [0, 8], [-1, 1]):
        kda.pages_free(t, ln, ref, ints(*rows), 8)
        assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
        c.same(t, ln, ref)


def test_too_few_pages_change_nothing():
    c = Cache(8, 8, 10, 8)
    c.reserve([0], [50])
    t, ln, ref = c.cuda()
    info = ints(0)
    kda.pages_reserve(t, ln, ref, ints(1, 2), ints(8, 25), 8, info=info)
    assert info.item() == 3 - 5
    c.same(t, ln, ref)
    a, b = kda.pages_fork(t, ln, ref, ints(0, 0, 0, 0), ints(1, 2, 3, 4), 8, info=info)
    assert info.item() == 3 - 4 and a.tolist() == b.tolist() == [-1] * 4
    c.same(t, ln, ref)
    kda.pages_reserve(t, ln, ref, ints(1, 2), ints(8, 16), 8, info=info)
    assert info.item() == 0 == c.reserve([1, 2], [8, 16])
    c.same(t, ln, ref)
    assert kda.stream_status() == kda.KDA_OK


def test_empty_lists():
    c, _ = fill(5, 4, 20, 8, 2)
    t, ln, ref = c.cuda()
    none, info = ints(), ints(-7)
    kda.pages_free(t, ln, ref, none, 8)
    kda.pages_reserve(t, ln, ref, none, none, 8, info=info)
    assert info.item() == int((c.ref == 0).sum())
    kda.pages_fork(t, ln, ref, none, none, 8, info=info)
    assert info.item() == int((c.ref == 0).sum())
    kda.pages_copy(torch.zeros((1, 3, 8), device="cuda"), none, none)
    c.same(t, ln, ref)


def test_corrupt_cache_is_reported_in_bounds():
    c = Cache(4, 4, 10, 8)
    c.reserve([0, 1], [30, 9])
    for what in ("table", "count"):
        t, ln, ref = c.cuda()
        if what == "table":
            t[0, 1] = 10
        else:
            ref[int(t[0, 1])] = 0
        kda.pages_free(t, ln, ref, ints(0), 8)
        assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
        assert (ref >= 0).all() and int(ln[0]) == 0
    t, ln, ref = c.cuda()
    t[0, 1] = -4
    kda.pages_fork(t, ln, ref, ints(0), ints(3), 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    t, ln, ref = c.cuda()
    t[0, 1] = 1 << 30
    kda.pages_compact(t, ln, ref, 8)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG


# ------------------------------------------------------------------- copy ----
POOLS = [(1, 4, 16), (3, 9, 48), (2, 40, 16384), (2, 40, 16400), (5, 12, 70000 // 16 * 16), (1, 300, 262144), (33, 20, 1040)]


@pytest.mark.parametrize("outer,pages,nb", POOLS)
@pytest.mark.parametrize("spread", [False, True])
def test_copy(outer, pages, nb, spread):
    r = np.random.default_rng(nb)
    x = torch.randint(0, 256, (outer, pages, nb + (64 if spread else 0)), dtype=torch.uint8, device="cuda")
    pool = x[:, :, 16:16 + nb] if spread else x
    n = max(1, pages // 3)
    ids = r.permutation(pages)
    src, dst = ids[:n].copy(), ids[n: 2 * n]
    src[n // 2] = src[0]  # a source may be read twice
    want = x.clone()
    w = want[:, :, 16:16 + nb] if spread else want
    w[:, dst] = pool[:, src]
    kda.pages_copy(pool, ints(*src.tolist()), ints(*dst.tolist()))
    assert torch.equal(x, want)
    assert kda.stream_status() == kda.KDA_OK


def test_copy_leaves_out_what_is_named_twice():
    pool = torch.arange(10 * 8, dtype=torch.float32, device="cuda").view(1, 10, 8)
    want = pool.clone()
    # 3 is written twice; 5 is written and read; 9 is out of range; 7 -> 7 is nothing; -1 is skipped
    kda.pages_copy(pool, ints(0, 1, 2, 5, 9, 7, -1), ints(3, 3, 5, 6, 10, 7, -1))
    want[:, 6] = want[:, 5]
    assert torch.equal(pool, want)
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    kda.pages_copy(pool, ints(-1, 4), ints(-1, 1))
    want[:, 1] = want[:, 4]
    assert torch.equal(pool, want) and kda.stream_status() == kda.KDA_OK


def test_copy_refusals():
    pool = torch.zeros((2, 4, 8), device="cuda")
    for bad in (pool[0], pool.transpose(0, 2), pool[:, :, ::2], pool.cpu()):
        with pytest.raises(ValueError):
            kda.pages_copy(bad, ints(0), ints(1))
    with pytest.raises(ValueError):
        kda.pages_copy(pool, ints(0), ints(1, 2))
    with pytest.raises(kda.KdaError):
        kda.pages_copy(torch.zeros((1, 4, 3), device="cuda"), ints(0), ints(1))


@pytest.mark.parametrize("R,P,pages,ps", SHAPES[2:])
def test_compact_moves_the_pools(R, P, pages, ps):
    c, _ = fill(R, P, pages, ps, 5)
    t, ln, ref = c.cuda()
    a = torch.randn((3, pages, 5, 8), device="cuda")
    b = torch.randint(0, 99, (1, pages, 32), device="cuda", dtype=torch.int16)
    wa, wb = a.clone(), b.clone()
    t0, ref0 = t.clone(), ref.clone()
    t2, ref2 = kda.pages_compact(t, ln, ref, ps, table_out=torch.zeros_like(t), ref_out=torch.zeros_like(ref), pools=[a, b])
    assert torch.equal(t, t0) and torch.equal(ref, ref0)
    moves = c.compact()
    if moves:
        f, to = torch.tensor(moves, device="cuda").T
        wa[:, to], wb[:, to] = wa[:, f], wb[:, f]
    c.same(t2, ln, ref2)
    assert torch.equal(a, wa) and torch.equal(b, wb)


def test_compact_moves_the_pools_of_a_large_cache():
    """More pages than one launch compacts."""
    c = Cache(700, 100, 70001, 4)
    r = np.random.default_rng(3)
    t, ln, ref = c.cuda()
    rows, new = np.arange(700), r.integers(300, 401, 700)
    kda.pages_reserve(t, ln, ref, ints(*rows.tolist()), ints(*new.tolist()), 4)
    c.reserve(rows, new)
    gone = r.permutation(700)[:350]
    kda.pages_free(t, ln, ref, ints(*gone.tolist()), 4)
    c.free(gone)
    a = torch.randint(0, 1 << 20, (2, 70001, 8), device="cuda", dtype=torch.int32)
    want = a.clone()
    kda.pages_compact(t, ln, ref, 4, pools=[a])
    f, to = torch.tensor(c.compact(), device="cuda").T
    want[:, to] = want[:, f]
    c.same(t, ln, ref)
    assert torch.equal(a, want) and kda.stream_status() == kda.KDA_OK


@pytest.mark.parametrize("bad", ["bytes", "pointer", "overlap"])
def test_bad_pools_are_refused_before_the_table_changes(bad):
    c = Cache(4, 4, 10, 8)
    c.reserve([0, 1, 2], [30, 9, 4])
    c.free([0])
    good = torch.zeros((1, 10, 8), device="cuda")
    pool = {"bytes": lambda: torch.zeros((2, 10, 3), device="cuda"), "pointer": lambda: torch.zeros(90, device="cuda")[1:81].view(1, 10, 8),
            "overlap": lambda: good.expand(3, 10, 8)}[bad]()
    t, ln, ref = c.cuda()
    with pytest.raises(kda.KdaError):
        kda.pages_fork(t, ln, ref, ints(1), ints(3), 8, pools=[good, pool])
    with pytest.raises(kda.KdaError):
        kda.pages_compact(t, ln, ref, 8, pools=[good, pool])
    c.same(t, ln, ref)
    assert kda.stream_status() == kda.KDA_OK


def test_captured_page_calls():
    """reserve, fork with copies, free and compact in one graph, replayed on changed lists."""
    R, P, pages, ps = 16, 8, 120, 4
    c = Cache(R, P, pages, ps)
    t, ln, ref = c.cuda()
    pool = torch.randn((2, pages, 16), device="cuda")
    rows, new, src, dst, gone, info = ints(0, 1, 2), ints(9, 31, 4), ints(0, 1), ints(5, 6), ints(1), ints(0)

    def step():
        kda.pages_reserve(t, ln, ref, rows, new, ps, info=info)
        kda.pages_fork(t, ln, ref, src, dst, ps, pools=[pool])
        kda.pages_free(t, ln, ref, gone, ps)
        kda.pages_compact(t, ln, ref, ps, pools=[pool])

    def host(rows, new, src, dst, gone):
        left = c.reserve(rows, new)
        _, a, b = c.fork(src, dst)
        for x, y in zip(a, b):
            if x >= 0:
                host.pool[:, y] = host.pool[:, x]
        c.free(gone)
        for x, y in c.compact():
            host.pool[:, y] = host.pool[:, x]
        return left

    host.pool = pool.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    assert info.item() == host([0, 1, 2], [9, 31, 4], [0, 1], [5, 6], [1])
    c.same(t, ln, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for lists in (([1, 2, 3], [5, 17, 32], [2, 3], [7, 8], [0]), ([0, 4, 9], [3, 3, 30], [9, 0], [10, 11], [5])):
        for x, y in zip((rows, new, src, dst, gone), lists):
            x.copy_(ints(*y))
        g.replay()
        torch.cuda.synchronize()
        assert info.item() == host(*lists)
        c.same(t, ln, ref)
        assert torch.equal(pool, host.pool)
    assert kda.stream_status() == kda.KDA_OK
