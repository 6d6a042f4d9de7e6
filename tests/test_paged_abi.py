"""The paged cache's entry points reject bad arguments before touching a GPU."""
import ctypes

import pytest
import torch

from gated_delta_rule_100_b200 import build as kbuild
from gated_delta_rule_100_b200 import kda

A = ctypes.c_void_p(0x10000)     # stand-in device addresses: only validated, never dereferenced
MIS = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)
INV, UNS, ALI = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def attn(lib, q=A, k_new=A, v_new=A, kp=A, vp=A, cu=A, table=A, length=A, rows=None, scale=0.125, out=A, lse=None, N=2,
         total=5, max_q=4, Hq=8, Hkv=2, d=64, ps=16, pages=9, P=40, R=2, qs=None, ks=None, vs=None, strides=None,
         dtype=0, ws=A, nbytes=1 << 40):
    st = None if strides is None else (ctypes.c_longlong * 6)(*strides)
    return lib.kda_paged_attn(q, k_new, v_new, kp, vp, cu, table, length, rows, scale, out, lse, N, total, max_q, Hq, Hkv,
                              d, ps, pages, P, R, Hq * d if qs is None else qs, Hkv * d if ks is None else ks,
                              Hkv * d if vs is None else vs, st, dtype, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(kp=None), INV), (dict(vp=None), INV), (dict(cu=None), INV), (dict(table=None), INV),
    (dict(length=None), INV), (dict(out=None), INV), (dict(ws=None), INV), (dict(nbytes=16), INV),
    (dict(k_new=None), INV), (dict(v_new=None), INV), (dict(N=0), INV), (dict(total=-1), INV), (dict(max_q=0), INV),
    (dict(Hq=9), INV), (dict(Hkv=0), INV), (dict(ps=0), INV), (dict(pages=0), INV), (dict(P=0), INV), (dict(R=1), INV),
    (dict(R=0, rows=A), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV),
    (dict(scale=float("inf")), INV), (dict(qs=8 * 64 - 8), INV), (dict(ks=64), INV), (dict(strides=[-8, 128, 64] * 2), INV),
    (dict(d=96), UNS), (dict(d=256), UNS), (dict(dtype=2), UNS), (dict(P=1 << 20, ps=1 << 12), UNS),
    (dict(q=MIS), ALI), (dict(k_new=MIS), ALI), (dict(vp=MIS), ALI), (dict(out=MIS), ALI), (dict(lse=ODD), ALI),
    (dict(cu=ODD), ALI), (dict(rows=ODD), ALI), (dict(ws=MIS), ALI), (dict(qs=8 * 64 + 4), ALI),
    (dict(strides=[2048, 132, 64] * 2), ALI),
])
def test_paged_attn_rejects(lib, kw, code):
    assert attn(lib, **kw) == code


def test_no_tokens_need_nothing(lib):
    assert attn(lib, total=0, max_q=0, q=None, out=None, k_new=None, v_new=None, ws=None, nbytes=0) == kda.KDA_OK
    assert kda.paged_attn_workspace_bytes(2, 0, 0, 8, 2, 64, 16, 4) == 0
    assert kda.paged_attn_workspace_bytes(2, 5, 4, 8, 2, 96, 16, 4) == 0
    assert kda.paged_attn_workspace_bytes(2, 5, 4, 8, 2, 64, 16, 40) > 0
    assert kda.paged_attn_workspace_bytes(2, 50, 48, 8, 2, 64, 16, 4000) > 0
    assert kda.paged_attn_workspace_bytes(2, 50, 48, 8, 2, 64, 16, 4) == 0  # short caches are not split


def reserve(lib, table=A, length=A, ref=A, rows=A, new=A, n=2, info=None, R=4, P=4, pages=9, ps=16):
    return lib.kda_pages_reserve(table, length, ref, rows, new, n, info, R, P, pages, ps, None)


def fork(lib, table=A, length=A, ref=A, src=A, dst=A, n=2, cs=A, cd=A, info=None, R=4, P=4, pages=9, ps=16):
    return lib.kda_pages_fork(table, length, ref, src, dst, n, cs, cd, info, R, P, pages, ps, None)


def free(lib, table=A, length=A, ref=A, rows=A, n=2, R=4, P=4, pages=9, ps=16):
    return lib.kda_pages_free(table, length, ref, rows, n, R, P, pages, ps, None)


def compact(lib, table=A, length=A, ref=A, to=A, ro=A, info=None, R=4, P=4, pages=9, ps=16, ws=A, nbytes=1 << 40):
    return lib.kda_pages_compact(table, length, ref, to, ro, info, R, P, pages, ps, ws, nbytes, None)


SIZES = [(dict(R=0), INV), (dict(P=0), INV), (dict(pages=0), INV), (dict(ps=0), INV), (dict(R=65537), UNS),
         (dict(R=65536, P=32768), UNS), (dict(P=1 << 20, ps=1 << 12), UNS), (dict(pages=(1 << 30) + 1), UNS),
         (dict(table=None), INV), (dict(length=None), INV), (dict(ref=None), INV), (dict(table=ODD), ALI),
         (dict(length=ODD), ALI), (dict(ref=ODD), ALI)]


@pytest.mark.parametrize("call,extra", [
    (reserve, [(dict(rows=None), INV), (dict(new=None), INV), (dict(n=-1), INV), (dict(n=5), INV), (dict(info=ODD), ALI),
               (dict(n=8193, R=9000), UNS), (dict(rows=ODD), ALI)]),
    (fork, [(dict(src=None), INV), (dict(dst=None), INV), (dict(cs=None), INV), (dict(cd=None), INV), (dict(n=5), INV),
            (dict(src=ODD), ALI), (dict(cd=ODD), ALI), (dict(n=8193, R=9000), UNS)]),
    (free, [(dict(rows=None), INV), (dict(n=5), INV), (dict(n=-1), INV), (dict(rows=ODD), ALI)]),
    (compact, [(dict(to=None), INV), (dict(ro=None), INV), (dict(ws=None), INV), (dict(nbytes=64), INV), (dict(ro=ODD), ALI),
               (dict(ws=MIS), ALI)]),
], ids=["reserve", "fork", "free", "compact"])
def test_pages_reject(lib, call, extra):
    for kw, code in SIZES + extra:
        assert call(lib, **kw) == code, kw


def copy(lib, pool=A, outer=2, os=1 << 20, ps=4096, nb=4096, pages=9, src=A, dst=A, n=3):
    return lib.kda_pages_copy(pool, outer, os, ps, nb, pages, src, dst, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(pool=None), INV), (dict(outer=-1), INV), (dict(nb=0), INV), (dict(pages=0), INV), (dict(n=-1), INV),
    (dict(src=None), INV), (dict(dst=None), INV), (dict(ps=2048), INV), (dict(os=1024), INV), (dict(os=-16), INV),
    (dict(pool=MIS), ALI), (dict(nb=4088), ALI), (dict(ps=4104), ALI), (dict(src=ODD), ALI),
    (dict(n=0), kda.KDA_OK), (dict(outer=0), kda.KDA_OK),
])
def test_pages_copy_rejects(lib, kw, code):
    assert copy(lib, **kw) == code


def test_compact_pool_rejects(lib):
    def call(pool=A, pages=9, ws=A, nbytes=1 << 40, page=4096):
        return lib.kda_pages_compact_pool(pool, 2, 1 << 20, page, page, pages, ws, nbytes, None)
    assert call(pool=None) == INV and call(ws=None) == INV and call(nbytes=64) == INV and call(page=4104) == ALI
    assert call(ws=MIS) == ALI
    assert kda.load().kda_pages_compact_workspace_bytes(0) == 0
    assert kda.load().kda_pages_compact_workspace_bytes(9) > 0


def test_binding_wants_cuda_tensors():
    x = torch.zeros(4, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.pages_free(x, x[0], x[0], x[0], 16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.pages_copy(torch.zeros(1, 4, 8), x[0], x[0])
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        kda.paged_attn(torch.zeros(1, 1, 64), torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 1, 64), x[0], x, x[0], 1.0,
                       max_q=1)
    with pytest.raises(ValueError, match="must be"):
        kda.paged_attn(torch.zeros(1, 64), torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, 1, 64), x[0], x, x[0], 1.0, max_q=1)
