"""Attention over a paged cache: what other tests' ordinary values, single calls and small batches do not show."""
import pytest
import torch

from gated_delta_rule_100_b200 import kda
from paged_testlib import appended, attention64, make

pytestmark = pytest.mark.gpu

LONG = 1 << 18  # keys that a table has room for: past 32 rows the chunk kernel runs


def call(c, **kw):
    lse = torch.full((c["total"], c["q"].shape[1]), 7.0, device="cuda")
    out = kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"], max_q=c["max_q"],
                         rows=c["rows"], k_new=c["kn"], v_new=c["vn"], lse=lse, **kw)
    return out, lse


def near(c, out, lse, want, skip=None):
    """Against 64 bits, but for the rows of `skip` (a mask [total, heads])."""
    o, z, tol, ltol = want
    keep = torch.ones_like(z, dtype=torch.bool) if skip is None else ~skip
    assert ((out.double() - o).abs() <= tol)[keep].all()
    none = torch.isinf(z)
    assert torch.equal((lse == -torch.inf)[keep], none[keep]) and (out[keep & none] == 0).all()
    assert ((lse.double() - z).abs() <= ltol)[keep & ~none].all()


NAN = [([1], [40], 0), ([1], [1], LONG), ([1], [9000], LONG), ([100, 1], [9000, 30], LONG), ([300] * 3, [300] * 3, LONG)]


@pytest.mark.parametrize("nq,ln,span", NAN, ids=["whole", "one key", "split", "chunk split", "chunk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_a_row_of_nan_scores_is_no_empty_row(nq, ln, span, dtype):
    """A NaN in a query, or in the only key that a row sees: out and lse are NaN, not 0 and -inf."""
    c = make(nq, ln, 4, 2, 64, 16, dtype=dtype, seed=11, span=span)
    want = attention64(c, *appended(c))
    hit = torch.zeros((c["total"], 4), dtype=torch.bool, device="cuda")
    c["q"][0, 1, 3] = float("nan")
    hit[0, 1] = True
    if ln[0] == nq[0]:  # the first token sees its own key only; key head 1 is read by heads 2 and 3 of every token
        c["kn"][0, 1, 5] = float("nan")
        hit[: nq[0], 2:] = True
    out, lse = call(c)
    assert kda.stream_status() == kda.KDA_OK
    assert torch.isnan(out[hit].float()).all() and torch.isnan(lse[hit]).all()
    near(c, out, lse, want, hit)


@pytest.mark.parametrize("nq,ln,d", [([300, 2], [900, 70], 128), ([40], [5001], 64), ([129] * 9, [1000 + 37 * i for i in range(9)], 128)])
def test_calls_that_give_up_anywhere_end_in_order(nq, ln, d):
    """Waits cut to a few tries run out at different places: before the first product, at a tail's values, at the last
    products.  Every call ends, says so or is right, leaves the memory beside its buffers alone, and the next is right."""
    c = make(nq, ln, 8, 2, d, 64, seed=12, span=LONG, q_scale=4.0)
    kp, vp = appended(c)
    want = attention64(c, kp, vp)
    ob = torch.full((c["total"] + 2, 8, d), 5.0, dtype=c["q"].dtype, device="cuda")
    gave_up = 0
    for tries in (1, 1, 2, 2, 3, 4, 5, 6, 8, 12):
        try:
            kda.set_wait_limit(tries)
            lse = call(c, out=ob[1:-1])[1]
            status = kda.stream_status()
        finally:
            kda.set_wait_limit(0)
        assert status in (kda.KDA_OK, kda.KDA_ERR_TIMEOUT)
        gave_up += status != kda.KDA_OK
        if status == kda.KDA_OK:
            near(c, ob[1:-1], lse, want)
        assert (ob[0] == 5.0).all() and (ob[-1] == 5.0).all()
        out, lse = call(c)
        assert kda.stream_status() == kda.KDA_OK
        near(c, out, lse, want)
        for x, y in ((c["kp"], kp), (c["vp"], vp)):
            assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    assert gave_up


def test_a_tile_without_rows_outlasts_a_long_piece():
    """40 rows an item leave half of a CTA's rows idle for as long as its piece takes: that wait ends by what is being
    loaded, not by the limit of a step's waits.  As many items as SMs, so that no item is cut: 1500 steps of keys each,
    at a limit of about 64 x 4 us."""
    N = torch.cuda.get_device_properties(0).multi_processor_count // 2
    c = make([10], [200_000], 8, 2, 64, 64, seed=13, poison=False)
    kp, vp = appended(c)
    o, z, tol, ltol = attention64(c, kp, vp)
    lse = torch.zeros((10 * N, 8), device="cuda")
    try:
        kda.set_wait_limit(64)
        out = kda.paged_attn(c["q"].repeat(N, 1, 1), kp, vp, torch.arange(0, 10 * N + 1, 10, device="cuda", dtype=torch.int32),
                             c["table"].repeat(N, 1), c["length"].repeat(N), c["scale"], max_q=10, lse=lse)
        assert kda.stream_status() == kda.KDA_OK
    finally:
        kda.set_wait_limit(0)
    assert ((out.view(N, 10, 8, 64).double() - o).abs() <= tol).all() and ((lse.view(N, 10, 8).double() - z).abs() <= ltol).all()


def test_the_binding_refuses_places_that_overlap():
    c = make([1, 3], [40, 20], 4, 2, 64, 16, seed=3, poison=False)
    shape, good = c["kp"].shape, c["kp"]
    flat = torch.zeros(shape[0] * 16 * 2 * 64 + 64, dtype=torch.bfloat16, device="cuda")
    for strides in ((2048, 64, 64, 1), (1024, 128, 64, 1), (2048, 128, 128, 1)):
        for name in ("kp", "vp"):
            with pytest.raises(kda.KdaError):
                call({**c, name: flat.as_strided(shape, strides)})
    assert (flat == 0).all()
    out, lse = call({**c, "kp": good.clone()})
    near(c, out, lse, attention64(c, *appended(c)))


@pytest.mark.parametrize("N", [17, 40, 200])
@pytest.mark.parametrize("append", [True, False])
def test_chunk_batches_of_many_sequences(N, append):
    """More sequences than the plan has warps, or a third of its threads; some without tokens, some without a place."""
    gen = torch.Generator().manual_seed(N)
    nq = torch.randint(0, 70, (N,), generator=gen).tolist()
    ln = [t + int(x) for t, x in zip(nq, torch.randint(0, 1500, (N,), generator=gen))]
    nq[3], ln[3], nq[N // 2], ln[5], nq[N - 1] = 0, 0, 1, max(0, nq[5] - 4), 90
    ln[N - 1] = 2000
    c = make(nq, ln, 8, 2, 64, 16, seed=N, span=LONG, permute=True, extra_rows=2)
    kp, vp = appended(c)
    if not append:
        c["kp"].copy_(kp)
        c["vp"].copy_(vp)
    lse = torch.full((c["total"], 8), 7.0, device="cuda")
    new = dict(k_new=c["kn"], v_new=c["vn"]) if append else {}
    out = kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"], max_q=c["max_q"],
                         rows=c["rows"], lse=lse, **new)
    assert kda.stream_status() == kda.KDA_OK
    near(c, out, lse, attention64(c, kp, vp))
    assert torch.equal(c["kp"].view(torch.int16), kp.view(torch.int16))


@pytest.mark.parametrize("nq,ln", [([1500], [3100]), ([700, 300, 1200], [2500, 300, 1600]), ([513] * 12, [513 + 97 * i for i in range(12)])])
@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_sms(nq, ln, d):
    """Items that stay whole first, then those that are cut: more of them than SMs, and more partial rows than there is
    room for in most of the plans that are compared."""
    c = make(nq, ln, 32, 8, d, 64, seed=sum(nq), span=LONG)
    tiles = sum(-(-t * 4 // 256) for t in nq)
    assert tiles * 8 > torch.cuda.get_device_properties(0).multi_processor_count
    want = attention64(c, *appended(c))
    out, lse = call(c)
    assert kda.stream_status() == kda.KDA_OK
    near(c, out, lse, want)
    again = call(c)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])


@pytest.mark.parametrize("nq,ln", [([1] * 6, [9000, 9, 400, 1, 64, 65]), ([300, 1, 40], [5000, 3000, 41]), ([1], [200])],
                         ids=["few", "chunk", "whole"])
def test_calls_in_flight_on_two_streams(nq, ln):
    """Many calls a stream without a wait between them: workspaces, plans and tickets are each call's own."""
    span = 0 if ln == [200] else LONG
    cs = [make(nq, [x + 13 * j * (x > 100) for x in ln], 16, 4, 128, 16, seed=20 + j, span=span) for j in range(2)]
    want = [attention64(c, *appended(c)) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    calls = 12
    lses = [[torch.full((c["total"], 16), 7.0, device="cuda") for _ in range(calls)] for c in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(calls):
        for j, (c, s) in enumerate(zip(cs, streams)):
            got[j].append(kda.paged_attn(c["q"], c["kp"], c["vp"], c["cu"], c["table"], c["length"], c["scale"],
                                         max_q=c["max_q"], k_new=c["kn"], v_new=c["vn"], lse=lses[j][i], stream=s))
    torch.cuda.synchronize()
    assert kda.stream_status() == kda.KDA_OK
    for c, outs, ls, w in zip(cs, got, lses, want):
        for out, lse in zip(outs, ls):
            near(c, out, lse, w)
