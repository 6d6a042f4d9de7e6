"""The paged cache as a server of a hybrid stack uses it: one recurrent layer and one layer of full attention, slots
that share their sequences' pages, and both layers' outputs against 64 bits at every step."""
import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_100_b200 import kda
from kda_testlib import assert_close, f64
from paged_testlib import Cache, attention64

pytestmark = pytest.mark.gpu

R, P, PAGES, PS, HQ, HKV, D, LAYERS = 12, 24, 110, 16, 8, 2, 64, 2


def ints(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")


class Server:
    """Slots on the device, and beside them what each slot's sequence is, token by token."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.r = np.random.default_rng(seed)
        self.host = Cache(R, P, PAGES, PS)
        self.table, self.length, self.ref = self.host.cuda()
        self.kv = torch.full((2 * LAYERS, PAGES, PS, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.state = torch.zeros((R, HKV, D, D), device="cuda")       # the recurrent layer's slots
        self.seen = [[[None, None] for _ in range(LAYERS)] for _ in range(R)]  # keys and values of each layer
        self.state64 = np.zeros((R, HKV, D, D))
        self.info = ints([0])

    def rand(self, *s):
        return torch.randn(s, device="cuda", generator=self.gen).to(torch.bfloat16)

    def feed(self, rows, new):
        """`new` tokens for each of `rows`, through every full-attention layer."""
        self.host.reserve(rows, [self.host.length[k] + t for k, t in zip(rows, new)])
        kda.pages_reserve(self.table, self.length, self.ref, ints(rows), ints([self.host.length[k] for k in rows]), PS,
                          info=self.info)
        self.host.same(self.table, self.length, self.ref)
        cu = ints(np.concatenate([[0], np.cumsum(new)]))
        total = int(sum(new))
        for layer in range(LAYERS):
            # queries, keys and values are slices of one projection, as a model makes them
            qkv = self.rand(total, (HQ + 2 * HKV) * D)
            q = qkv[:, : HQ * D].view(total, HQ, D)
            k, v = (qkv[:, (HQ + i * HKV) * D: (HQ + (i + 1) * HKV) * D].view(total, HKV, D) for i in range(2))
            lse = torch.empty((total, HQ), device="cuda")
            out = kda.paged_attn(q, self.kv[2 * layer], self.kv[2 * layer + 1], cu, self.table, self.length, D ** -0.5,
                                 max_q=max(new), k_new=k, v_new=v, rows=ints(rows), lse=lse)
            at = 0
            for row, t in zip(rows, new):
                s = self.seen[row][layer]
                for i, x in enumerate((k, v)):
                    y = x[at: at + t].clone()
                    s[i] = y if s[i] is None else torch.cat([s[i], y])
                # the same attention over the sequence's own keys in one long page
                n = s[0].shape[0]
                c = dict(q=q[at: at + t], table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"), nq=[t], ln=[n], row_of=[0],
                         ps=n, scale=D ** -0.5)
                o, z, tol, ltol = attention64(c, s[0][None], s[1][None])
                assert ((out[at: at + t].double() - o).abs() <= tol).all()
                assert ((lse[at: at + t].double() - z).abs() <= ltol).all()
                at += t

    def recur(self):
        """One token of every slot through the recurrent layer."""
        q, k = (torch.nn.functional.normalize(self.rand(R, HKV, D).float(), dim=-1).to(torch.bfloat16) for _ in range(2))
        v = self.rand(R, HKV, D)
        g = -0.05 * torch.nn.functional.softplus(torch.randn((R, HKV, D), device="cuda", generator=self.gen))
        beta = torch.rand((R, HKV), device="cuda", generator=self.gen)
        o = kda.decode_step(q, k, v, g, beta, D ** -0.5, self.state)
        want, self.state64 = oracle.kda_decode_step(*(f64(x) for x in (q, k, v, g, beta)), D ** -0.5, self.state64)
        assert_close(f64(o), want, "hybrid recurrent out")
        assert_close(f64(self.state), self.state64, "hybrid recurrent state")

    def fork(self, src, dst):
        pairs = kda.pages_fork(self.table, self.length, self.ref, ints(src), ints(dst), PS, pools=[self.kv], info=self.info)
        left, a, b = self.host.fork(src, dst)
        assert (self.info.item(), pairs.tolist()) == (left, [a, b])
        kda.pages_copy(self.state.view(1, R, HKV, D, D), ints(src), ints(dst))
        for s, d in zip(src, dst):
            self.seen[d] = [[x.clone() for x in layer] for layer in self.seen[s]]
            self.state64[d] = self.state64[s]
        self.host.same(self.table, self.length, self.ref)
        assert torch.equal(self.state[dst], self.state[src])

    def end(self, rows):
        kda.pages_free(self.table, self.length, self.ref, ints(rows), PS)
        self.host.free(rows)
        for k in rows:
            self.seen[k] = [[None, None] for _ in range(LAYERS)]
        self.host.same(self.table, self.length, self.ref)

    def compact(self):
        kda.pages_compact(self.table, self.length, self.ref, PS, pools=[self.kv], info=self.info)
        self.host.compact()
        self.host.same(self.table, self.length, self.ref)


@pytest.mark.parametrize("seed", range(2))
def test_prompts_tokens_branches_and_compaction(seed):
    s = Server(seed)
    s.feed([0, 3, 5], [70, 16, 129])            # prompts
    s.recur()
    for _ in range(3):                           # tokens, one with a prompt's next chunk beside them
        s.feed([5, 0, 3], [1, 1, 1])
        s.recur()
    s.fork([0, 0, 5], [1, 2, 7])                 # branches that share their prompts
    s.feed([0, 1, 2, 3, 7, 5], [1, 4, 1, 40, 2, 1])
    s.recur()
    s.end([0, 3])                                # the parent ends, its branches go on
    s.compact()
    s.feed([1, 2, 7, 5, 8], [1, 1, 33, 1, 20])
    s.fork([7, 8], [0, 3])
    s.compact()
    s.feed([0, 1, 2, 3, 5, 7, 8], [1, 1, 17, 1, 1, 5, 1])
    s.recur()
    s.end([1, 2, 5, 7, 8, 0, 3])
    assert (s.ref == 0).all() and (s.table == -1).all() and (s.length == 0).all()
    assert kda.stream_status() == kda.KDA_OK
