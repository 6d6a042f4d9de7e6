"""The paged cache and its attention, as they are measured.

Each case is one pass through an operator of ``gated_delta_rule_100_b200.kda``:

* ``attn``: ``paged_attn``, new tokens of a packed batch written into a paged
  key/value cache and attending causally over it (single tokens, chunks, both);
* ``copy``: ``pages_copy``, pages of one pool copied onto others;
* ``fork``: ``pages_free`` of earlier branches and ``pages_fork`` of their parents;
* ``turnover``: ``pages_free`` of finished sequences and ``pages_reserve`` for
  those that take their place;
* ``compact``: ``pages_compact``, live pages moved to the front of the pool.

``run`` is the operator's plain form while ``own`` is false, the library's
calls while it is true.
"""
import math

import numpy as np
import torch

own = False

MAX_SCORES = 1 << 32  # scores that the plain form holds at once, padded to the longest sequence


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one request's next token, a short context, the small head size: latency of a serving step
        dict(name="attn_token_one", op="attn", N=1, q_min=1, q_max=1, len_min=257, len_max=257, Hq=4, Hkv=4, d=64,
             ps=16, dtype="bf16", heads_first=False, lse=False),
        # a decode batch of 256 requests with a serving mix of context lengths
        dict(name="attn_token_batch", op="attn", N=256, q_min=1, q_max=1, len_min=128, len_max=16384, Hq=32, Hkv=8,
             d=128, ps=64, dtype="bf16", heads_first=False, lse=False),
        # a long prompt's next chunk of 2048 tokens over the 63,488 before it
        dict(name="attn_chunk_long", op="attn", N=1, q_min=2048, q_max=2048, len_min=65536, len_max=65536, Hq=32,
             Hkv=8, d=128, ps=64, dtype="bf16", heads_first=False, lse=True),
        # single tokens and prompt chunks in one packed batch; heads outside the page's tokens, three queries a key head
        dict(name="attn_mixed", op="attn", N=12, q_min=1, q_max=509, len_min=33, len_max=8191, Hq=24, Hkv=8, d=64,
             ps=16, dtype="fp16", heads_first=True, lse=True),
        # one request's recurrent state (4 heads, fp32 128 x 128) forked to another slot
        dict(name="copy_state_one", op="copy", outer=1, pages=64, page_bytes=4 * 128 * 128 * 4, n=1),
        # 128 key/value pages (64 tokens, 8 heads of 128) of 16 layers copied, as for 128 requests that part
        dict(name="copy_kv", op="copy", outer=32, pages=512, page_bytes=64 * 8 * 128 * 2, n=128),
        # one sequence forked once
        dict(name="fork_one", op="fork", R=8, P=32, pages=256, ps=16, parents=1, branches=1, len_min=301, len_max=301,
             outer=2, page_bytes=16 * 4 * 64 * 2),
        # eight parents forked into eight branches each, long shared prefixes
        dict(name="fork_beam", op="fork", R=128, P=512, pages=32768, ps=64, parents=8, branches=8, len_min=513,
             len_max=16383, outer=8, page_bytes=64 * 8 * 64 * 2),
        # a small server's step: two requests end, two begin
        dict(name="turnover_small", op="turnover", R=16, P=64, pages=1024, ps=16, n=2, len_min=17, len_max=1000),
        # a large one's: 200 of 1024 rows turn over in a pool of 262,144 pages
        dict(name="turnover_large", op="turnover", R=1024, P=1024, pages=262144, ps=16, n=200, len_min=128,
             len_max=12000),
        # a small pool packed
        dict(name="compact_small", op="compact", R=24, P=40, pages=300, ps=16, len_min=1, len_max=200, fill=0.5,
             outer=2, page_bytes=16 * 4 * 64 * 2),
        # a pool of 4 GB packed, three fifths of it live
        dict(name="compact_large", op="compact", R=384, P=256, pages=16384, ps=64, len_min=65, len_max=4095, fill=0.6,
             outer=2, page_bytes=64 * 8 * 128 * 2),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "copy", "fork", "turnover", "compact"])
    if op == "attn":
        while True:
            kind = rng.choice(["token", "few", "chunk"])
            d, Hkv, G = rng.choice([64, 128]), rng.randint(1, 16), rng.randint(1, 8)
            ps = rng.choice([16, 32, 64, 128])
            if kind == "token":
                N, q_min, q_max = _log(rng, 1, 256), 1, 1
            elif kind == "few":
                N, q_min, q_max = _log(rng, 1, 64), 1, rng.randint(2, 8)
            else:
                N, q_min, q_max = _log(rng, 1, 16), 1, _log(rng, 9, 2048)
            len_max = _log(rng, max(64, q_max), 65536)
            len_min = _log(rng, max(1, min(q_max, len_max // 2)), len_max)
            if N * Hkv * G * q_max * len_max <= MAX_SCORES and N * len_max * Hkv * d * 8 <= 35e9:
                break
        return dict(op="attn", N=N, q_min=q_min, q_max=q_max, len_min=len_min, len_max=len_max, Hq=Hkv * G, Hkv=Hkv,
                    d=d, ps=ps, dtype=rng.choice(["bf16", "bf16", "fp16"]), heads_first=rng.random() < 0.3,
                    lse=rng.random() < 0.5)
    row = 2 * rng.choice([64, 128]) * rng.choice([1, 2, 3, 4, 8])  # one token's heads
    ps = rng.choice([16, 32, 64])
    if op == "copy":
        while True:
            outer, pages, n = _log(rng, 1, 64), _log(rng, 4, 4096), _log(rng, 1, 512)
            if 2 * n <= pages and outer * n * row * ps <= 537e6 and outer * pages * row * ps <= 4.3e9:
                break
        return dict(op="copy", outer=outer, pages=pages, page_bytes=row * ps, n=n)
    if op == "fork":
        while True:
            parents, branches, len_max = _log(rng, 1, 16), _log(rng, 1, 12), _log(rng, 20, 16000)
            outer, P = _log(rng, 1, 8), (len_max + ps - 1) // ps + rng.randint(0, 9)
            pages = parents * P + parents * branches + _log(rng, 10, 4000)
            if pages * outer * row * ps <= 4.3e9:
                break
        return dict(op="fork", R=parents * (branches + 1) + rng.randint(0, 20), P=P, pages=pages, ps=ps, parents=parents,
                    branches=branches, len_min=_log(rng, 1, len_max), len_max=len_max, outer=outer, page_bytes=row * ps)
    len_max = _log(rng, 40, 12000)
    P = (len_max + ps - 1) // ps + rng.randint(0, 9)
    R = _log(rng, 4, 1024)
    len_min = _log(rng, 1, len_max)
    if op == "turnover":
        # the pool holds every row at its longest
        len_max = min(len_max, 262144 // R * ps)
        return dict(op="turnover", R=R, P=P, pages=min(262144, R * P + rng.randint(0, 999)), ps=ps,
                    n=rng.randint(1, max(1, R // 4)), len_min=min(len_min, len_max), len_max=len_max)
    outer = rng.choice([1, 2, 3, 4])
    R = max(1, min(R, int(3.0e9 / (P * outer * row * ps))))
    return dict(op="compact", R=R, P=P, pages=R * P + rng.randint(1, 200), ps=ps, len_min=len_min, len_max=len_max,
                fill=rng.uniform(0.3, 0.9), outer=outer, page_bytes=row * ps)


# ----------------------------------------------------------------- inputs ----
def _lengths(case):
    """New tokens and cache lengths (with them) of every sequence of an attention case: the same for every seed, as
    they set the outputs' shapes; what the pages hold and where they lie goes by the seed."""
    r = np.random.default_rng([1, case["N"], case["q_max"], case["len_min"], case["len_max"], case["Hq"]])
    N, lo, hi = case["N"], case["q_min"], case["q_max"]
    nq = np.exp(r.uniform(math.log(lo), math.log(hi + 1), N)).astype(np.int64).clip(lo, hi)
    nq[r.integers(N)] = hi
    ln = np.exp(r.uniform(math.log(case["len_min"]), math.log(case["len_max"] + 1), N)).astype(np.int64)
    ln = ln.clip(case["len_min"], case["len_max"])
    ln[r.integers(N)] = case["len_max"]
    return nq, np.maximum(ln, nq)


def _rows(case, seed):
    """Row lengths of a page case, before the pass."""
    r = np.random.default_rng([seed, 2])
    ln = np.exp(r.uniform(math.log(case["len_min"]), math.log(case["len_max"] + 1), case["R"])).astype(np.int64)
    return r, ln.clip(case["len_min"], case["len_max"])


def _assign(case, ln, r):
    """A page table of rows of `ln` tokens on pages in random places, and the pages' counts."""
    held = (ln + case["ps"] - 1) // case["ps"]
    table = np.full((case["R"], case["P"]), -1, np.int32)
    ids = r.permutation(case["pages"])[: int(held.sum())].astype(np.int32)
    table[np.arange(case["P"])[None, :] < held[:, None]] = ids
    ref = np.zeros(case["pages"], np.int32)
    ref[ids] = 1
    return table, ref


def _pool(case, gen):
    # 16-bit elements, whole pages of them; random bits of a normal draw
    x = torch.empty((case["outer"], case["pages"], case["page_bytes"] // 2), dtype=torch.bfloat16, device="cuda")
    return x.normal_(generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    st = dict(case=case)
    if case["op"] == "attn":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
        nq, ln = _lengths(case)
        N, ps, Hq, Hkv, d = case["N"], case["ps"], case["Hq"], case["Hkv"], case["d"]
        held = (ln + ps - 1) // ps
        r = np.random.default_rng([seed, 3])
        pages = int(held.sum()) + N
        table = np.full((N, int(held.max())), -1, np.int32)
        table[np.arange(table.shape[1])[None, :] < held[:, None]] = r.permutation(pages)[: int(held.sum())]
        total = int(nq.sum())
        shape = (pages, Hkv, ps, d) if case["heads_first"] else (pages, ps, Hkv, d)
        new = lambda *s: torch.empty(s, dtype=dt, device="cuda").normal_(generator=gen)  # noqa: E731
        kp, vp = new(*shape), new(*shape)
        if case["heads_first"]:
            kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
        st |= dict(q=1.5 * new(total, Hq, d), k=new(total, Hkv, d), v=new(total, Hkv, d), kp=kp, vp=vp,
                   cu=dev(np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)), table=dev(table),
                   length=dev(ln.astype(np.int32)), max_q=int(nq.max()), scale=d ** -0.5)
        if case["lse"]:
            st["lse"] = torch.empty((total, Hq), dtype=torch.float32, device="cuda")
        return st
    if case["op"] == "copy":
        r = np.random.default_rng([seed, 4])
        ids = r.permutation(case["pages"])[: 2 * case["n"]].astype(np.int32)
        return st | dict(pool=_pool(case, gen), src=dev(ids[: case["n"]]), dst=dev(ids[case["n"]:]))
    r, ln = _rows(case, seed)
    if case["op"] == "fork":
        place = r.permutation(case["R"])
        parents = place[: case["parents"]]
        branches = place[case["parents"]: case["parents"] * (1 + case["branches"])]
        keep = np.zeros(case["R"], np.int64)
        keep[parents] = ln[parents]
        table, ref = _assign(case, keep, r)
        st |= dict(src=dev(np.tile(parents, case["branches"]).astype(np.int32)), dst=dev(branches.astype(np.int32)),
                   length=dev(keep.astype(np.int32)), pool=_pool(case, gen))
    elif case["op"] == "turnover":
        rows = r.permutation(case["R"])[: case["n"]]
        new = np.minimum(r.permutation(ln)[: case["n"]], ln[rows])  # they fit where the old ones were
        table, ref = _assign(case, ln, r)
        st |= dict(rows=dev(rows.astype(np.int32)), new=dev(new.astype(np.int32)), length=dev(ln.astype(np.int32)))
    else:
        ln = np.where(r.random(case["R"]) < case["fill"], ln, 0)
        table, ref = _assign(case, ln, r)
        st |= dict(length=dev(ln.astype(np.int32)), pool=_pool(case, gen), table_out=dev(table.copy()),
                   ref_out=dev(ref.copy()))
    return st | dict(table=dev(table), ref=dev(ref), info=torch.zeros(1, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------- one pass ----
def run(st):
    if own:
        return _run_own(st)
    return {"attn": _attn, "copy": _copy, "fork": _fork, "turnover": _turnover, "compact": _compact}[st["case"]["op"]](st)


def _run_own(st):
    from gated_delta_rule_100_b200 import kda
    c = st["case"]
    if c["op"] == "attn":
        out = kda.paged_attn(st["q"], st["kp"], st["vp"], st["cu"], st["table"], st["length"], st["scale"],
                             max_q=st["max_q"], k_new=st["k"], v_new=st["v"], lse=st.get("lse"))
        return (out, st["kp"], st["vp"]) + ((st["lse"],) if c["lse"] else ())
    if c["op"] == "copy":
        kda.pages_copy(st["pool"], st["src"], st["dst"])
        return (st["pool"],)
    if c["op"] == "fork":
        kda.pages_free(st["table"], st["length"], st["ref"], st["dst"], c["ps"])
        kda.pages_fork(st["table"], st["length"], st["ref"], st["src"], st["dst"], c["ps"], pools=[st["pool"]],
                       info=st["info"])
        return st["table"], st["length"], st["ref"], st["info"], st["pool"]
    if c["op"] == "turnover":
        kda.pages_free(st["table"], st["length"], st["ref"], st["rows"], c["ps"])
        kda.pages_reserve(st["table"], st["length"], st["ref"], st["rows"], st["new"], c["ps"], info=st["info"])
        return st["table"], st["length"], st["ref"], st["info"]
    kda.pages_compact(st["table"], st["length"], st["ref"], c["ps"], table_out=st["table_out"], ref_out=st["ref_out"],
                      pools=[st["pool"]], info=st["info"])
    return st["table_out"], st["ref_out"], st["info"], st["pool"]


# ------------------------------------------------------------ plain forms ----
def _attn(st):
    q, kp, vp, table, length, c = st["q"], st["kp"], st["vp"], st["table"], st["length"].long(), st["case"]
    N, ps, Hq, Hkv, d, mq = c["N"], c["ps"], c["Hq"], c["Hkv"], c["d"], st["max_q"]
    total, G = q.shape[0], Hq // Hkv
    cu = st["cu"].long()
    nq = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(N, device=q.device), nq, output_size=total)
    i = torch.arange(total, device=q.device) - cu[seq]
    pos = length[seq] - nq[seq] + i
    page = table[seq, pos // ps].long()
    kp[page, pos % ps] = st["k"]
    vp[page, pos % ps] = st["v"]
    at = table.clamp(min=0).long()
    L = table.shape[1] * ps
    K = kp[at].float().reshape(N, L, Hkv, d).permute(0, 2, 3, 1)
    Q = torch.zeros((N, mq, Hq, d), device=q.device)
    Q[seq, i] = q.float()
    Q = Q.view(N, mq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * mq, d)
    s = torch.matmul(Q, K).view(N, Hkv, G, mq, L).mul_(st["scale"])
    del K
    last = length[:, None] - nq[:, None] + torch.arange(mq, device=q.device)  # the last key that a query sees
    hidden = torch.arange(L, device=q.device) > last[:, :, None]
    s.masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    V = vp[at].float().reshape(N, L, Hkv, d).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(N, Hkv, G * mq, L), V).view(N, Hkv, G, mq, d) / l
    out = o.permute(0, 3, 1, 2, 4).reshape(N, mq, Hq, d)[seq, i].to(q.dtype)
    if not c["lse"]:
        return out, kp, vp
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(N, mq, Hq)[seq, i]
    return out, kp, vp, lse


def _copy(st):
    st["pool"][:, st["dst"].long()] = st["pool"][:, st["src"].long()]
    return (st["pool"],)


def _held(table, length, rows, ps):
    return torch.arange(table.shape[1], device=table.device) < ((length[rows] + ps - 1) // ps)[:, None]


def _free(st, rows):
    table, length, ref = st["table"], st["length"], st["ref"]
    mask = _held(table, length, rows, st["case"]["ps"])
    gone = table[rows][mask].long()
    ref.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[rows] = table[rows].masked_fill(mask, -1)
    length[rows] = 0


def _fork(st):
    table, length, ref, ps = st["table"], st["length"], st["ref"], st["case"]["ps"]
    src, dst = st["src"].long(), st["dst"].long()
    _free(st, dst)
    ln = length[src]
    full, rest = ln // ps, ln % ps > 0
    cols = torch.arange(table.shape[1], device=table.device)
    shared = cols < full[:, None]
    old = table[src]
    share = old[shared].long()
    ref.index_add_(0, share, torch.ones_like(share, dtype=torch.int32))
    fresh = torch.nonzero(ref == 0)[: int(rest.sum()), 0]
    ref[fresh] = 1
    new = torch.where(shared, old, table[dst])
    last = torch.nonzero(rest)[:, 0]
    came = old[last, full[last].long()].long()
    new[last, full[last].long()] = fresh.int()
    table[dst] = new
    length[dst] = ln
    st["pool"][:, fresh] = st["pool"][:, came]
    st["info"].copy_((ref == 0).sum())
    return table, length, ref, st["info"], st["pool"]


def _turnover(st):
    table, length, ref, ps = st["table"], st["length"], st["ref"], st["case"]["ps"]
    rows = st["rows"].long()
    _free(st, rows)
    have, want = (length[rows] + ps - 1) // ps, (st["new"] + ps - 1) // ps
    cols = torch.arange(table.shape[1], device=table.device)
    mask = (cols >= have[:, None]) & (cols < want[:, None])
    fresh = torch.nonzero(ref == 0)[: int(mask.sum()), 0]
    mine = table[rows]
    mine[mask] = fresh.int()
    table[rows] = mine
    ref[fresh] = 1
    length[rows] = st["new"]
    st["info"].copy_((ref == 0).sum())
    return table, length, ref, st["info"]


def _compact(st):
    table, ref, ps = st["table"], st["ref"], st["case"]["ps"]
    live = ref > 0
    n = int(live.sum())
    holes = torch.nonzero(~live[:n])[:, 0]
    moved = torch.nonzero(live[n:])[:, 0] + n
    to = torch.arange(ref.numel(), device=ref.device, dtype=torch.int32)
    to[moved] = holes.int()
    rows = torch.arange(table.shape[0], device=ref.device)
    mask = _held(table, st["length"], rows, ps)
    st["table_out"].copy_(torch.where(mask, to[table.clamp(min=0).long()], table))
    new = torch.zeros_like(ref)
    new[:n] = ref[:n]
    new[holes] = ref[moved]
    st["ref_out"].copy_(new)
    st["info"].copy_((~live).sum())
    st["pool"][:, holes] = st["pool"][:, moved]
    return st["table_out"], st["ref_out"], st["info"], st["pool"]


# ------------------------------------------------------------------- work ----
def work(case):
    """Bytes and operations that one pass cannot do without, for the lengths of seed 0."""
    ps = case.get("ps", 0)
    if case["op"] == "attn":
        nq, ln = _lengths(case)
        tok = int(nq.sum())
        keys = int(ln.sum() - nq.sum())
        pairs = float((nq * (ln - nq) + nq * (nq + 1) // 2).sum())
        b = 2 * (keys * 2 * case["Hkv"] * case["d"]           # keys and values before the new ones, read
                 + tok * 4 * case["Hkv"] * case["d"]          # the new ones, read and written
                 + tok * 2 * case["Hq"] * case["d"])          # queries read, outputs written
        b += 4 * (int(((ln + ps - 1) // ps).sum()) + 2 * case["N"] + 1) + (4 * tok * case["Hq"] if case["lse"] else 0)
        return {"bytes": b, "flops": 4.0 * case["Hq"] * case["d"] * pairs}
    if case["op"] == "copy":
        return {"bytes": 2 * case["n"] * case["outer"] * case["page_bytes"] + 8 * case["n"], "flops": 0}
    r, ln = _rows(case, 0)
    if case["op"] == "fork":
        parents = r.permutation(case["R"])[: case["parents"]]
        held = int(((ln[parents] + ps - 1) // ps).sum()) * case["branches"]
        part = int((ln[parents] % ps > 0).sum()) * case["branches"]
        # the old branches' entries read and cleared, their counts; the parents' read, the new ones written, their
        # counts; the free pages sought; the copies
        return {"bytes": 4 * (8 * held + case["pages"]) + 2 * part * case["outer"] * case["page_bytes"], "flops": 0}
    if case["op"] == "turnover":
        rows = r.permutation(case["R"])[: case["n"]]
        new = np.minimum(r.permutation(ln)[: case["n"]], ln[rows])
        held = int(((new + ps - 1) // ps).sum())
        return {"bytes": 4 * (6 * held + case["pages"] + 5 * case["n"]), "flops": 0}
    ln = np.where(r.random(case["R"]) < case["fill"], ln, 0)
    _, ref = _assign(case, ln, r)
    moved = int((ref[int((ref > 0).sum()):] > 0).sum())
    return {"bytes": 4 * (2 * case["R"] * case["P"] + case["R"] + 2 * case["pages"])
            + 2 * moved * case["outer"] * case["page_bytes"], "flops": 0}


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    """Attention in 64 bits, sequence by sequence; the page operators move and count, they compute nothing."""
    if case["op"] != "attn":
        return None
    st = prepare(case, seed)
    nq, ln = _lengths(case)
    G, ps = case["Hq"] // case["Hkv"], case["ps"]
    if float((nq * ln).sum()) * case["Hq"] * case["d"] > 1.5e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    first = 0
    for n in range(case["N"]):
        t, L = int(nq[n]), int(ln[n])
        pages = st["table"][n, : (L + ps - 1) // ps].long()
        for h in range(case["Hkv"]):
            K = st["kp"][pages, :, h].reshape(-1, case["d"])[:L].double()
            V = st["vp"][pages, :, h].reshape(-1, case["d"])[:L].double()
            K[L - t:], V[L - t:] = st["k"][first:first + t, h].double(), st["v"][first:first + t, h].double()
            for a in range(0, t, 256):
                b = min(t, a + 256)
                see = L - t + b
                x = torch.einsum("tgd,kd->gtk", st["q"][first + a:first + b, h * G:(h + 1) * G].double(), K[:see]) * st["scale"]
                ok = torch.arange(see, device="cuda")[None] <= torch.arange(L - t + a, L - t + b, device="cuda")[:, None]
                x = torch.where(ok, x, -math.inf)
                z = torch.logsumexp(x, -1)
                out[first + a:first + b, h * G:(h + 1) * G] = torch.einsum("gtk,kd->tgd", torch.exp(x - z[..., None]), V[:see])
                lse[first + a:first + b, h * G:(h + 1) * G] = z.T
        first += t
    return (out, None, None) + ((lse,) if case["lse"] else ())
