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
