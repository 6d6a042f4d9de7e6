"""A paged cache made for a test, its attention in 64 bits with a bound on the
kernels' rounding, and the page operators on host arrays."""
from __future__ import annotations

import numpy as np
import torch

NAN16 = float("nan")


def make(nq, ln, Hq, Hkv, d, ps, *, dtype=torch.bfloat16, layout="tokens", seed=0, spare=3, extra_rows=0, pad_q=0,
         wide=False, permute=False, poison=True, q_scale=1.0, span=0):
    """A batch of len(nq) sequences.  Every place of the pages that no token holds is NaN when
    `poison`; the new tokens' places hold NaN too until the call writes them.  The table has room for
    `span` keys a row at least: the sizes are what the choice of kernel goes by."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    N, R = len(nq), len(nq) + extra_rows
    held = [-(-n // ps) for n in ln]
    P = max(1, max(held), -(-span // ps)) + int(r.integers(0, 3))
    pages = sum(held) + spare
    ids = r.permutation(pages)
    rows = r.permutation(R)[:N] if permute else np.arange(N)
    table = np.full((R, P), -1, np.int32)
    length = np.zeros(R, np.int32)
    at = 0
    for n in range(N):
        table[rows[n], : held[n]] = ids[at: at + held[n]]
        length[rows[n]] = ln[n]
        at += held[n]
    total = int(sum(nq)) + pad_q

    def rnd(*s):
        return torch.randn(s, device="cuda", generator=gen).to(dtype)

    def heads(h, scale=1.0):
        if not wide:
            return rnd(total, h, d) * scale
        return (rnd(total, h * d + 40) * scale)[:, 8:8 + h * d].view(total, h, d)

    q, kn, vn = heads(Hq, q_scale), heads(Hkv), heads(Hkv)
    shape = (pages, ps, Hkv, d)
    if layout == "heads":  # [pages, heads, tokens, d]
        kp, vp = rnd(pages, Hkv, ps, d).transpose(1, 2), rnd(pages, Hkv, ps, d).transpose(1, 2)
    elif layout == "pair":  # keys and values of a token side by side
        both = rnd(pages, ps, 2, Hkv, d)
        kp, vp = both[:, :, 0], both[:, :, 1]
    else:
        kp, vp = rnd(*shape), rnd(*shape)
    if poison:
        hold = torch.zeros((pages, ps), dtype=torch.bool)
        for n in range(N):
            for pos in range(max(0, ln[n] - nq[n])):
                hold[table[rows[n], pos // ps], pos % ps] = True
        bad = ~hold.cuda()
        kp[bad] = NAN16
        vp[bad] = NAN16
    cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dict(q=q, kn=kn, vn=vn, kp=kp, vp=vp, cu=dev(cu), table=dev(table), length=dev(length),
                rows=dev(rows.astype(np.int32)) if permute or extra_rows else None, nq=list(nq), ln=list(ln),
                row_of=[int(x) for x in rows], ps=ps, scale=float(d) ** -0.5, max_q=max(1, max(nq)), total=total)


def appended(c):
    """The pages as the call has to leave them."""
    kp, vp = c["kp"].clone(), c["vp"].clone()
    table = c["table"].cpu().numpy()
    at = 0
    for n, (t, L) in enumerate(zip(c["nq"], c["ln"])):
        for i in range(t):
            pos = L - t + i
            if pos >= 0:
                page = int(table[c["row_of"][n], pos // c["ps"]])
                kp[page, pos % c["ps"]] = c["kn"][at + i]
                vp[page, pos % c["ps"]] = c["vn"][at + i]
        at += t
    return kp, vp


def attention64(c, kp, vp):
    """out, lse in 64 bits from the pages kp, vp (new tokens in place), and bounds on the error
    of each.

    u = half a step of the 16-bit type.  The weights p_j are rounded once (at most u each:
    u sum p_j |v_j| after the division), the result once more (u |o|).  A score's products are
    exact in 32 bits, their d sums lose at most 2^-23 of sum |q||k| each (tensor cores may
    truncate), scaling and the exponential a few 2^-23 of the score and of the weight; the sums
    over keys lose at most 2^-23 a key.

    fp16's steps stop shrinking at 2^-14, where half of one is 2^-25.  Weights are rounded as
    2^8 times their ratio to a reference that is no larger than the row's largest, so a
    ratio below 2^-22 is off by at most 2^-25 / 2^8 = 2^-33: sum |v_j| times that, over the
    sum of the ratios, e^(z - max), joins the bound."""
    u = torch.finfo(c["q"].dtype).eps / 2
    tiny = 2.0 ** -33 if c["q"].dtype == torch.float16 else 0.0
    q = c["q"].double()
    total, Hq, d = q.shape
    Hkv = kp.shape[2]
    G = Hq // Hkv
    out = torch.zeros_like(q)
    lse = torch.full((total, Hq), -np.inf, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(q)
    ltol = torch.zeros_like(lse)
    at = 0
    for n, (t, L) in enumerate(zip(c["nq"], c["ln"])):
        if t and L:
            pages = c["table"][c["row_of"][n], : -(-L // c["ps"])].long()
            K = kp[pages].reshape(-1, Hkv, d)[:L].double().repeat_interleave(G, 1)
            V = vp[pages].reshape(-1, Hkv, d)[:L].double().repeat_interleave(G, 1)
            Q = q[at: at + t]
            s = torch.einsum("thd,khd->htk", Q, K) * c["scale"]
            mag = torch.einsum("thd,khd->htk", Q.abs(), K.abs()) * c["scale"]
            see = torch.arange(L, device="cuda")[None] <= (L - t + torch.arange(t, device="cuda"))[:, None]
            s = torch.where(see, s, -np.inf)
            z = torch.logsumexp(s, -1)
            some = see.any(-1)
            p = torch.where(see, torch.exp(s - torch.where(some, z, 0.0)[..., None]), 0.0)
            o = torch.einsum("htk,khd->thd", p, V)
            a = torch.einsum("htk,khd->thd", p, V.abs())
            top = torch.where(some, torch.exp(s.amax(-1) - z), 0.0)
            low = tiny * top.T[..., None] * torch.einsum("htk,khd->thd", see.double().expand(Hq, t, L), V.abs())
            ds = 2.0 ** -23 * (d + 4) * torch.where(see, mag, 0.0).amax(-1) + 2.0 ** -21  # of the scores, [h, t]
            rest = 2 * ds + 2.0 ** -23 * (L + 64)
            out[at: at + t] = o
            tol[at: at + t] = u * a + low + u * (o.abs() + u * a) + rest.T[..., None] * a + 2.0 ** -25
            lse[at: at + t] = z.T
            ltol[at: at + t] = (ds + 2.0 ** -23 * (L + 64)).T + 2.0 ** -22 * torch.where(some, z.abs(), 0.0).T
        at += t
    return out, lse, tol, ltol


# ------------------------------------------------------------- page lists ----
class Cache:
    """The page operators on host arrays, as they are documented."""

    def __init__(self, R, P, pages, ps):
        self.table = np.full((R, P), -1, np.int32)
        self.length = np.zeros(R, np.int32)
        self.ref = np.zeros(pages, np.int32)
        self.ps = ps

    def held(self, r):
        return -(-int(self.length[r]) // self.ps)

    def reserve(self, rows, new):
        """Free pages left, or minus those missing."""
        need = [-(-int(n) // self.ps) - self.held(r) for r, n in zip(rows, new)]
        free = np.nonzero(self.ref == 0)[0]
        if sum(need) > len(free):
            return len(free) - sum(need)
        at = 0
        for r, n, k in zip(rows, new, need):
            self.table[r, self.held(r): self.held(r) + k] = free[at: at + k]
            self.ref[free[at: at + k]] = 1
            self.length[r] = n
            at += k
        return len(free) - at

    def fork(self, src, dst):
        free = np.nonzero(self.ref == 0)[0]
        need = [int(self.length[s]) % self.ps != 0 for s in src]
        if sum(need) > len(free):
            return len(free) - sum(need), [-1] * len(src), [-1] * len(src)
        at, a, b = 0, [], []
        for s, d, k in zip(src, dst, need):
            full = int(self.length[s]) // self.ps
            self.table[d, :full] = self.table[s, :full]
            for page in self.table[s, :full]:
                self.ref[page] += 1
            if k:
                a.append(int(self.table[s, full]))
                b.append(int(free[at]))
                self.table[d, full] = free[at]
                self.ref[free[at]] = 1
                at += 1
            else:
                a.append(-1)
                b.append(-1)
            self.length[d] = self.length[s]
        return len(free) - at, a, b

    def free(self, rows):
        for r in rows:
            for j in range(self.held(r)):
                self.ref[self.table[r, j]] -= 1
                self.table[r, j] = -1
            self.length[r] = 0

    def compact(self):
        """The moves made, (from, to)."""
        n = int((self.ref > 0).sum())
        holes = [q for q in range(n) if self.ref[q] == 0]
        moved = [q for q in range(n, len(self.ref)) if self.ref[q] > 0]
        to = np.arange(len(self.ref))
        to[moved] = holes
        for r in range(len(self.length)):
            k = self.held(r)
            self.table[r, :k] = to[self.table[r, :k]]
        self.ref[holes] = self.ref[moved]
        self.ref[n:] = 0
        return list(zip(moved, holes))

    def cuda(self):
        return tuple(torch.from_numpy(x.copy()).cuda() for x in (self.table, self.length, self.ref))

    def same(self, table, length, ref):
        assert np.array_equal(table.cpu().numpy(), self.table)
        assert np.array_equal(length.cpu().numpy(), self.length)
        assert np.array_equal(ref.cpu().numpy(), self.ref)
