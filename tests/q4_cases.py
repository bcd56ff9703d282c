"""Batches over a 4-bit cache and their attention restated in 64 bits, over the values
that the cache stands for, taken from its pools' bytes.

Tolerance of an output value, with size = sum p (|m| + s n):
 - p is rounded to fp16 and p s again, 2^-11 of each at most: 2^-10 size.  Both are kept
   at 2^11 times their size at the largest score or more (less where s is above 1, and then
   p s is as large); below fp16's normal numbers they are off by 2^-25, so by 2^-36 of
   the largest weight each: 2^-35 n max(1, s_max) (15 + |m|)_max over n tokens.
 - the result is rounded to bf16: 2^-8 of itself.
 - fp32 sums, the approximate exponential (2^-22): 2^-12 size.
 - the scores: exact products, summed in fp32 in four groups: mag = sum |q| (|m| + s n) is
   off by 2^-20 of itself at most, which moves every weight by as much: 2 size times that.
lse: the scores' error, and 2^-18 for sum and logarithm.
"""

import math

import numpy as np
import torch

import q4_reference as ref
from top_sparse_attention_pks_gb300.decoder import Q4Attention, Q4Cache, Q4SparseAttention


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Batch:
    """Requests of ``lens`` tokens on pages dealt at random; what no token holds is the byte
    255 (s and m are NaN there)."""

    def __init__(self, lens, page=16, Hkv=2, G=4, D=64, Nq=1, seed=0, q_scale=1.0, v_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.P, self.Hkv, self.G, self.D, self.Nq = list(lens), page, Hkv, G, D, Nq
        B = len(self.lens)
        pages = [-(-n // page) for n in self.lens]
        N = sum(pages) + 2
        deal = rng.permutation(N)
        self.tab = np.full((B, max(pages + [1]) + 1), -7, np.int64)
        at = 0
        for b, n in enumerate(pages):
            self.tab[b, :n] = deal[at:at + n]
            at += n
        self.cache = Q4Cache(N, page, Hkv, D)
        self.cache.k.fill_(255)
        self.cache.v.fill_(255)
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = sum(self.lens)
        shape = (n, Hkv, D)
        self.k = torch.randn(shape, generator=g, device="cuda") + \
            torch.randn((Hkv, D), generator=g, device="cuda")
        self.v = torch.randn(shape, generator=g, device="cuda") * v_scale
        self.table, self.len_d = i32(self.tab), i32(self.lens)
        self.starts = np.concatenate([[0], np.cumsum(self.lens)]).tolist()
        self.q = (torch.randn((B, Nq, Hkv * G, D), generator=g, device="cuda") * q_scale
                  ).to(torch.bfloat16)
        self.write()

    def write(self):
        self.cache.write(self.k, self.v, self.len_d, self.table, i32(self.starts))
        assert self.cache.device_error() == 0

    def stored(self, kind):
        """The rows' (value, |m| + s n, |m|, s) from the pool, packed [tokens, Hkv, D]."""
        pool = {"k": self.cache.k, "v": self.cache.v}[kind].cpu().numpy()
        n, s, m = ref.unpack(pool, self.Hkv, self.D, kind)
        where = ref.places(self.lens, self.tab, self.starts, self.P)
        if not where:
            e = torch.zeros((0, self.Hkv, self.D), dtype=torch.float64, device="cuda")
            return e, e, 0.0, 0.0
        _, pg, sl = (np.array(c) for c in zip(*where))
        n, s, m = n[pg, sl], s[pg, sl], m[pg, sl]
        x, size = ref.values(n, s, m), ref.values(n, s, np.abs(m))
        return (torch.from_numpy(x).cuda(), torch.from_numpy(size).cuda(),
                float(np.nanmax(np.abs(m))), float(np.nanmax(s)))

    def check(self, out, lse, lists=None, causal=False, sm_scale=0.0, rows=None):
        scale = sm_scale or 1.0 / math.sqrt(self.D)
        k, k_size, _, _ = self.stored("k")
        v, v_size, m_max, s_max = self.stored("v")
        for b in (range(len(self.lens)) if rows is None else rows):
            n = self.lens[b]
            for i in range(self.Nq):
                got, got_lse = out[b, i].double(), lse[b, i].double()
                if lists is None:
                    t = np.arange(max(0, n - self.Nq + i + 1) if causal else n)
                else:
                    t = lists[b][i]
                    t = t[(t >= 0) & (t < n)]
                if len(t) == 0:
                    assert not got.any() and bool((got_lse == -math.inf).all()), (b, i)
                    continue
                at = torch.from_numpy(t + self.starts[b]).cuda()
                q = self.q[b, i].double().view(self.Hkv, self.G, self.D)
                x = torch.einsum("hgd,thd->hgt", q, k[at]) * scale
                mag = torch.einsum("hgd,thd->hgt", q.abs(), k_size[at]).amax(-1) * scale
                z = torch.logsumexp(x, -1)
                p = (x - z[..., None]).exp()
                want = torch.einsum("hgt,thd->hgd", p, v[at])
                size = torch.einsum("hgt,thd->hgd", p, v_size[at])
                tol = (2.0 ** -10 + 2.0 ** -12) * size + 2.0 ** -8 * want.abs()
                tol = tol + 2.0 ** -35 * len(t) * max(1.0, s_max) * (15.0 + m_max)
                tol = tol + (2.0 ** -20 * mag)[..., None] * 2 * size
                got = got.view_as(want)
                none = want.isnan()  # (of values that have a group which is not finite)
                assert bool((got.isnan() == none).all()), f"b={b} i={i}: NaN"
                off = torch.where(none, 0.0, (got - want).abs() / tol)
                assert bool((off <= 1).all()), f"b={b} i={i}: {float(off.max())} of tolerance"
                ltol = 2.0 ** -18 * (1 + z.abs()) + 2.0 ** -20 * mag
                assert bool(((got_lse.view_as(z) - z).abs() <= ltol).all()), f"lse b={b} i={i}"

    def dense(self, causal=False, sm_scale=0.0, q=None, **kw):
        att = Q4Attention(self.len_d, self.table, self.q, self.cache, causal=causal,
                          sm_scale=sm_scale, lse=True)
        att.out.fill_(float("nan"))
        att.lse.fill_(float("nan"))
        out = att()
        assert att.device_error() == 0
        self.check(out, att.lse, causal=causal, sm_scale=sm_scale, **kw)
        return att

    def lists(self, k, seed=0, holes=False):
        """Selected positions [B, Nq, k]: ascending with -1 behind, or in any order."""
        rng = np.random.default_rng(seed)
        out = np.full((len(self.lens), self.Nq, k), -1, np.int64)
        for b, n in enumerate(self.lens):
            for i in range(self.Nq):
                pick = np.sort(rng.permutation(n)[:k])
                if holes:
                    at = rng.permutation(k)[:len(pick)]
                    out[b, i, at] = rng.permutation(pick)
                    out[b, i, rng.random(k) < 0.2] = -1
                else:
                    out[b, i, :len(pick)] = pick
        return out

    def sparse(self, k, holes=False, seed=0, sm_scale=0.0, **kw):
        lists = self.lists(k, seed, holes)
        att = Q4SparseAttention(self.len_d, self.table, i32(lists), self.q, self.cache,
                                trim=not holes, sm_scale=sm_scale, lse=True)
        att.out.fill_(float("nan"))
        att.lse.fill_(float("nan"))
        out = att()
        assert att.device_error() == 0
        self.check(out, att.lse, lists=lists, sm_scale=sm_scale, **kw)
        return att
