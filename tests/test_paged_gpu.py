"""Attention over a paged cache against 64 bits, where it can go wrong."""
import numpy as np
import pytest
import torch

from gated_delta_rule_100_b200 import kda
from paged_testlib import appended, attention64, make

pytestmark = pytest.mark.gpu


def call(c, **kw):
    lse = torch.full((c["total"], c["q"].shape[1]), 7.0, device="cuda")
    out = torch.full_like(c["q"], 5.0, memory_format=torch.contiguous_format)
    new = dict(k_new=c["kn"], v_new=c["vn"]) if kw.pop("append", True) else {}
    kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"], max_q=c["max_q"],
                   rows=c["rows"], out=out, lse=lse, **new, **kw)
    return out, lse


def bits(t):
    return t.contiguous().view(torch.int16)


def check(c, out, lse, kp, vp):
    o, z, tol, ltol = attention64(c, kp, vp)
    real = sum(c["nq"])
    off = (out.double() - o).abs()[:real]
    bad = ~(off <= tol[:real])
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs, worst {float((off / tol[:real].clamp(min=1e-30)).max())} of its bound"
    empty = torch.isinf(z[:real])
    assert torch.equal(empty, torch.isinf(lse[:real]) & (lse[:real] < 0))
    assert not (out[:real][empty] != 0).any()
    err = torch.where(empty, 0.0, (lse[:real].double() - torch.where(empty, 0.0, z[:real])).abs())
    assert (err <= ltol[:real]).all(), float((err / ltol[:real].clamp(min=1e-30)).max())
    # rows behind the last sequence are left
    assert (out[real:] == 5.0).all() and (lse[real:] == 7.0).all()


def run(c, append=True):
    kp, vp = appended(c)
    if not append:
        c["kp"].copy_(kp)
        c["vp"].copy_(vp)
    out, lse = call(c, append=append)
    assert kda.stream_status() == kda.KDA_OK
    assert torch.equal(bits(c["kp"]), bits(kp)) and torch.equal(bits(c["vp"]), bits(vp))
    check(c, out, lse, kp, vp)
    return out, lse


TOKENS = [
    # nq, ln, Hq, Hkv, d, ps
    ([1], [1], 1, 1, 64, 16),
    ([1], [2], 4, 4, 128, 1),
    ([1], [257], 4, 4, 64, 16),
    ([1, 1, 1], [64, 65, 63], 8, 2, 128, 64),
    ([1, 0, 1], [5, 9, 1000], 16, 1, 64, 7),
    ([1] * 5, [1, 16, 17, 4097, 300], 32, 8, 128, 32),
    ([1] * 130, list(range(1, 131)), 6, 2, 64, 16),
    ([1, 1], [0, 3], 4, 2, 128, 16),          # no place for the token: an empty row
    ([1] * 3, [9001, 2, 777], 48, 3, 128, 128),
]
FEW = [
    ([3], [3], 4, 4, 64, 16),
    ([4, 2, 1], [4, 2, 100], 4, 1, 128, 16),
    ([5], [2], 2, 2, 64, 16),                 # three tokens before the first place
    ([7, 8], [70, 1031], 10, 2, 128, 5),
    ([2, 0, 0, 6], [2, 0, 40, 333], 7, 7, 64, 48),
]
CHUNKS = [
    ([17], [17], 1, 1, 64, 16),
    ([64, 1], [64, 129], 8, 2, 128, 64),
    ([100, 33], [164, 33], 6, 2, 64, 16),
    ([129], [640], 4, 4, 128, 32),
    ([255, 257, 1], [255, 300, 500], 3, 1, 128, 128),
    ([300], [120], 2, 1, 64, 16),             # more new tokens than places
    ([70, 70, 70], [1000, 70, 71], 24, 8, 64, 16),
    ([520], [1500], 16, 2, 128, 64),
    ([40, 1, 90], [1040, 2000, 91], 12, 4, 128, 24),  # a page size that is no power of two
    ([50], [50], 5, 1, 64, 9),
    ([1000], [1000], 7, 1, 128, 256),
    ([90], [1000], 2, 1, 128, 8),
    ([200, 1], [777, 800], 4, 2, 64, 384),
]


LONG = 1 << 18  # keys that a table has room for: past 32 rows the chunk kernel runs


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", TOKENS + FEW + CHUNKS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("span", [0, LONG], ids=["short", "long"])
def test_against_64_bits(nq, ln, Hq, Hkv, d, ps, dtype, span):
    run(make(nq, ln, Hq, Hkv, d, ps, dtype=dtype, seed=len(nq) + d, span=span))


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", [TOKENS[5], FEW[1], CHUNKS[2], CHUNKS[7]])
@pytest.mark.parametrize("layout", ["heads", "pair"])
def test_layouts_slices_and_rows(nq, ln, Hq, Hkv, d, ps, layout):
    c = make(nq, ln, Hq, Hkv, d, ps, layout=layout, wide=True, permute=True, extra_rows=3, pad_q=5, seed=9, span=LONG)
    run(c)


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", [TOKENS[5], FEW[3], CHUNKS[1], CHUNKS[8]])
def test_cache_that_holds_the_new_tokens(nq, ln, Hq, Hkv, d, ps):
    run(make(nq, ln, Hq, Hkv, d, ps, seed=4, span=LONG), append=False)


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", [TOKENS[5], CHUNKS[2], CHUNKS[7]])
def test_large_scores(nq, ln, Hq, Hkv, d, ps):
    # scores with a standard deviation of 12: the running maximum moves far and often
    run(make(nq, ln, Hq, Hkv, d, ps, q_scale=12.0, seed=5, span=LONG))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("nq,ln", [([1, 1], [9000, 300]), ([100], [9000])], ids=["few", "chunk"])
@pytest.mark.parametrize("gap", [12.0, 20.0])
def test_sink(nq, ln, dtype, gap):
    """One key outweighs every other by 2^17 (2^29): what thousands of the others add up to is kept, though each is far
    below fp16's smallest normal number."""
    c = make(nq, ln, 2, 1, 64, 16, dtype=dtype, seed=3, span=LONG, poison=False)
    for t in (c["q"], c["kp"], c["kn"]):
        t.zero_()
    c["q"][..., 0] = 8.0
    for n in range(len(nq)):
        c["kp"][int(c["table"][c["row_of"][n], 0]), 0, :, 0] = gap  # scale 1/8: a score of `gap`
    c["vp"].abs_().add_(1.0)
    c["vn"].abs_().add_(1.0)
    for n in range(len(nq)):
        c["vp"][int(c["table"][c["row_of"][n], 0]), 0] = 0.0  # the sink's own value
    kp, vp = appended(c)
    out, lse = call(c)
    check(c, out, lse, kp, vp)


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", [TOKENS[5], FEW[3], CHUNKS[5], CHUNKS[7]])
def test_same_bits_again(nq, ln, Hq, Hkv, d, ps):
    c = make(nq, ln, Hq, Hkv, d, ps, seed=6, span=LONG)
    a = call(c)
    for _ in range(3):
        b = call(c)
        assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", [TOKENS[8], CHUNKS[7]])
def test_padded_batch(nq, ln, Hq, Hkv, d, ps):
    """Sequences of no tokens, as a captured graph pads its batch with, change nothing."""
    c = make(nq, ln, Hq, Hkv, d, ps, seed=7, span=LONG)
    a = call(c)
    e = dict(c)
    e["cu"] = torch.cat([c["cu"], c["cu"][-1:].repeat(9)])
    e["table"] = torch.cat([c["table"], c["table"][:1].repeat(9, 1) * 0 - 1])
    e["length"] = torch.cat([c["length"], torch.zeros(9, dtype=torch.int32, device="cuda")])
    b = call(e)
    assert kda.stream_status() == kda.KDA_OK
    o, z, tol, ltol = attention64(c, *appended(c))
    assert ((b[0].double() - o).abs() <= tol).all() and ((b[1].double() - z).abs() <= ltol).all()
    assert ((a[0].double() - o).abs() <= tol).all()


@pytest.mark.parametrize("nq,ln,Hq,Hkv,d,ps", [([1] * 4, [9, 70, 300, 33], 8, 2, 128, 16), ([60, 2], [200, 90], 8, 2, 64, 16)])
def test_captured_and_replayed(nq, ln, Hq, Hkv, d, ps):
    """One graph, replayed for other lengths, tables and contents; two graphs in flight at once."""
    big = make(nq, [x + 500 for x in ln], Hq, Hkv, d, ps, seed=1, span=LONG)
    keys = ("q", "kn", "vn", "kp", "vp", "cu", "table", "length")

    def load_into(h, c):
        P = h["table"].shape[1]
        for k in keys:
            if k == "table":
                h[k].fill_(-1)
                h[k][:, : min(P, c[k].shape[1])].copy_(c[k][:, :P])
            elif k in ("kp", "vp"):
                h[k].fill_(float("nan"))
                h[k][: c[k].shape[0]].copy_(c[k])
            else:
                h[k].copy_(c[k])

    graphs = []
    for j in range(2):
        h = {k: big[k].clone() for k in keys}
        h["out"] = torch.zeros_like(big["q"])
        h["lse"] = torch.zeros((big["total"], Hq), device="cuda")
        h["go"] = lambda h=h: kda.paged_attn(h["q"], h["kp"], h["vp"], h["cu"], h["table"], h["length"], big["scale"],
                                             max_q=big["max_q"], k_new=h["kn"], v_new=h["vn"], out=h["out"], lse=h["lse"])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            h["go"]()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            h["go"]()
        graphs.append((g, s, h))
    for by in (0, 3, 400):
        cs = [make(nq, [x + by + j for x in ln], Hq, Hkv, d, ps, seed=100 + by + j) for j in range(2)]
        want = [appended(c) for c in cs]
        for (g, s, h), c in zip(graphs, cs):
            load_into(h, c)
        torch.cuda.synchronize()
        for g, s, h in graphs:
            with torch.cuda.stream(s):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        assert kda.stream_status() == kda.KDA_OK
        for (g, s, h), c, (kp, vp) in zip(graphs, cs, want):
            check(c, h["out"], h["lse"], kp, vp)


def test_calls_on_two_streams_at_once():
    cs = [make([1] * 6, [3000 + 100 * j, 9, 400, 1, 64, 65], 16, 4, 128, 16, seed=j) for j in range(2)]
    want = [appended(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            lse = torch.full((c["total"], 16), 7.0, device="cuda")
            torch.cuda.synchronize()
            got.append((kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"],
                                       max_q=c["max_q"], k_new=c["kn"], v_new=c["vn"], lse=lse, stream=s), lse))
        torch.cuda.synchronize()
        for c, (kp, vp), (out, lse) in zip(cs, want, got):
            check(c, out, lse, kp, vp)


BAD = ["page", "negative page", "length", "negative length", "row", "cu order", "cu end", "max_q"]


@pytest.mark.parametrize("what", BAD)
@pytest.mark.parametrize("nq,ln", [([1, 1, 2], [100, 40, 7]), ([40, 3, 90], [100, 40, 200])], ids=["few", "chunk"])
def test_bad_numbers_are_reported(what, nq, ln):
    """Nothing outside the buffers is touched: the pages' and outputs' neighbours keep their bits."""
    c = make(nq, ln, 8, 2, 64, 16, seed=8, permute=True, poison=False, span=LONG)
    kb = torch.full((c["kp"].shape[0] + 2, *c["kp"].shape[1:]), 3.0, dtype=c["q"].dtype, device="cuda")
    vb = kb.clone()
    kb[1:-1], vb[1:-1] = c["kp"], c["vp"]
    row = c["row_of"][1]
    if what == "page":
        c["table"][row, 0] = kb.shape[0] - 2
    elif what == "negative page":
        c["table"][row, 0] = -1
    elif what == "length":
        c["length"][row] = c["table"].shape[1] * 16 + 1
        c["table"][row] = 0
    elif what == "negative length":
        c["length"][row] = -5
    elif what == "row":
        c["rows"][1] = 99
    elif what == "cu order":
        c["cu"][1] = int(c["cu"][2]) + 1
    elif what == "cu end":
        c["cu"][-1] += 1
    max_q = c["max_q"] - 1 if what == "max_q" else c["max_q"]
    ob = torch.full((c["total"] + 2, 8, 64), 5.0, dtype=c["q"].dtype, device="cuda")
    kda.paged_attn(c["q"], kb[1:-1], vb[1:-1], c["cu"], c["table"], c["length"], c["scale"], max_q=max_q, k_new=c["kn"],
                   v_new=c["vn"], rows=c["rows"], out=ob[1:-1])
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    assert kda.stream_status() == kda.KDA_OK
    for t, v in ((kb, 3.0), (vb, 3.0), (ob, 5.0)):
        assert (t[0] == v).all() and (t[-1] == v).all()


@pytest.mark.parametrize("nq,ln", [([1, 2], [700, 40]), ([200, 70], [1500, 300])], ids=["few", "chunk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_nan_in_a_key_is_not_lost(nq, ln, dtype):
    """A NaN in a key that every row sees is in all of their results, wherever in a tile the key lies."""
    for pos in (0, 1, 9, 17, 33, 63, 65, 66, 127, 129, 400, 537):
        c = make(nq, ln, 4, 2, 64, 16, dtype=dtype, seed=pos, span=LONG)
        kp, vp = appended(c)
        page = int(c["table"][c["row_of"][0], pos // 16])
        c["kp"][page, pos % 16, 1, 5] = float("nan")
        out, lse = call(c)
        assert kda.stream_status() == kda.KDA_OK
        assert torch.isnan(out[: nq[0], 2:].float()).all() and torch.isnan(lse[: nq[0], 2:]).all()
        out[: nq[0], 2:], lse[: nq[0], 2:] = 0.0, 0.0
        o, z, tol, ltol = attention64(c, kp, vp)
        o[: nq[0], 2:], z[: nq[0], 2:] = 0.0, 0.0
        assert ((out.double() - o).abs() <= tol).all() and ((lse.double() - z).abs() <= ltol).all()


@pytest.mark.parametrize("nq", [1, 100], ids=["few", "chunk"])
def test_sequences_that_overlap_are_reported(nq):
    """Offsets that go back and name the same tokens again: far more work than total_q allows for, refused or done in bounds."""
    N = 400
    c = make([nq] + [0] * (N - 1), [300] * N, 8, 2, 64, 16, seed=1, poison=False, span=LONG)
    c["cu"].copy_(torch.tensor([0, nq] * (N // 2) + [0], dtype=torch.int32))
    ob = torch.full((nq + 2, 8, 64), 5.0, dtype=c["q"].dtype, device="cuda")
    kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"], max_q=nq, k_new=c["kn"],
                   v_new=c["vn"], out=ob[1:-1])
    assert kda.stream_status() == kda.KDA_ERR_INVALID_ARG
    assert (ob[0] == 5.0).all() and (ob[-1] == 5.0).all()


@pytest.mark.parametrize("nq,ln", [([300, 2], [900, 70]), ([1, 1], [9000, 70])], ids=["chunk", "few"])
def test_waits_that_give_up_are_reported(nq, ln):
    """With no patience at all the chunk kernel's waits run out; the call ends, says so, and the next one works."""
    c = make(nq, ln, 8, 2, 128, 64, seed=2, span=LONG)
    kp, vp = appended(c)
    try:
        kda.set_wait_limit(1)
        call(c)
        status = kda.stream_status()
    finally:
        kda.set_wait_limit(0)
    assert status == (kda.KDA_ERR_TIMEOUT if max(nq) > 1 else kda.KDA_OK)
    out, lse = call(c)
    assert kda.stream_status() == kda.KDA_OK
    check(c, out, lse, kp, vp)


def test_refusals():
    c = make([1], [9], 4, 2, 64, 16)
    ok = lambda **kw: kda.paged_attn(*[kw.get(k, c[k]) for k in ("q", "kp", "vp", "cu", "table", "length")], 0.125,  # noqa: E731
                                     max_q=1, k_new=c["kn"], v_new=kw.get("vn", c["vn"]))
    ok()
    for kw in (dict(q=c["q"].float()), dict(kp=c["kp"].half()), dict(cu=c["cu"].long()), dict(table=c["table"][0]),
               dict(length=c["length"].float()), dict(vp=c["vp"][:-1]), dict(vn=None), dict(vn=c["vn"][:, :1]),
               dict(kp=c["kp"].transpose(2, 3).contiguous().transpose(2, 3)), dict(q=c["q"].cpu())):
        with pytest.raises(ValueError):
            ok(**kw)
    with pytest.raises(kda.KdaError):
        kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], 0.0, max_q=1)
    assert np.isfinite(ok().float().cpu().numpy()).all()


def test_pages_beyond_32_bit_offsets():
    """Pages whose elements lie more than 2^31 apart (a pool of 4.3 billion elements of one byte pair each would be
    8.6 GB; the strides alone reach past it)."""
    c = make([1, 3], [40, 20], 4, 2, 64, 16, seed=3, poison=False)
    n = c["kp"].shape[0]
    step = (1 << 31) // (n - 1) // 8 * 8 + 64
    flat = torch.empty((n - 1) * step + 16 * 2 * 64, dtype=torch.bfloat16, device="cuda")
    far = flat.as_strided(c["kp"].shape, (step, 128, 64, 1))
    far.copy_(c["kp"])
    kp, vp = appended(c)
    near = c["kp"]
    c["kp"] = far
    out, lse = call(c)
    c["kp"] = near
    assert torch.equal(bits(far), bits(kp))
    check(c, out, lse, kp, vp)
