"""The paged cache in libkda_debug.so: rows of queries and outputs, partial sums, entries, table places and lists whose
bounds rest on the plan's arithmetic are checked before use.  No check may fail, and results are the release build's."""
import numpy as np
import pytest
import torch

from gated_delta_rule_100_b200 import kda
from paged_testlib import Cache, appended, attention64, make

pytestmark = pytest.mark.gpu

LONG = 1 << 18


@pytest.fixture(autouse=True)
def debug_library():
    kda.use_debug_library(True)
    yield
    kda.use_debug_library(False)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps,span", [
    ([1], [257], 4, 4, 64, 16, 0),
    ([1, 0, 3, 5], [5, 9, 9001, 2], 12, 2, 128, 7, LONG),
    ([1] * 130, list(range(1, 131)), 6, 2, 64, 16, LONG),
    ([300, 1, 129], [5000, 70, 120], 8, 2, 128, 64, LONG),
    ([40] * 20, [50 + 61 * i for i in range(20)], 8, 2, 64, 16, LONG),
    ([700, 300, 1200], [2500, 300, 1600], 32, 8, 64, 32, LONG),
], ids=["whole", "few", "tokens", "chunk", "many", "more items than SMs"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_attention(nq, ln, Hq, Hkv, d, ps, span, dtype):
    c = make(nq, ln, Hq, Hkv, d, ps, dtype=dtype, seed=31, span=span, permute=True, extra_rows=1)
    o, z, tol, ltol = attention64(c, *appended(c))
    lse = torch.full((c["total"], Hq), 7.0, device="cuda")
    out = kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"], max_q=c["max_q"],
                         rows=c["rows"], k_new=c["kn"], v_new=c["vn"], lse=lse)
    assert kda.stream_status() == kda.KDA_OK
    some = ~torch.isinf(z)
    assert ((out.double() - o).abs() <= tol).all() and ((lse.double() - z).abs() <= ltol)[some].all()


@pytest.mark.parametrize("R,P,pages,ps", [(3, 5, 11, 16), (40, 16, 300, 16), (300, 100, 20_001, 4)])
def test_pages(R, P, pages, ps):
    c = Cache(R, P, pages, ps)
    r = np.random.default_rng(R)
    t, ln, ref = c.cuda()
    pool = torch.randn((2, pages, 8), device="cuda")
    want = pool.clone()
    for _ in range(4):
        rows = [k for k in r.permutation(R).tolist() if c.length[k] == 0][: max(1, R // 2)]
        new = r.integers(0, P * ps + 1, len(rows)).tolist()
        kda.pages_reserve(t, ln, ref, ints(*rows), ints(*new), ps)
        c.reserve(rows, new)
        dst = [k for k in range(R) if c.length[k] == 0][: R // 8]
        src = [k for k in range(R) if c.length[k]][: len(dst)]
        dst = dst[: len(src)]
        kda.pages_fork(t, ln, ref, ints(*src), ints(*dst), ps, pools=[pool])
        _, a, b = c.fork(src, dst)
        pairs = [(x, y) for x, y in zip(a, b) if x >= 0]
        if pairs:
            x, y = map(list, zip(*pairs))
            want[:, y] = want[:, x]
        gone = [k for k in r.permutation(R).tolist() if c.length[k]][: max(1, R // 3)]
        kda.pages_free(t, ln, ref, ints(*gone), ps)
        c.free(gone)
        kda.pages_compact(t, ln, ref, ps, pools=[pool])
        moves = c.compact()
        if moves:
            x, y = map(list, zip(*moves))
            want[:, y] = want[:, x]
        c.same(t, ln, ref)
        assert torch.equal(pool, want) and kda.stream_status() == kda.KDA_OK
