"""Attention over a 4-bit cache where the sizes of V or of the weights lie far apart, against 64
bits over the stored values.

Tolerance of an output value, with size = sum p (|m| + s n), and the stages of the kernel: at
most 32 tokens that follow one another, 12 times 256 in a round of its ring, scales that are
looked at once in two rounds.
 - p is rounded to fp16 and p s again: 2^-11 of each, so 2^-10 size.  p is at least 2^11 at the
   largest score, so what is lost below fp16's normal numbers is 2^-36 of the largest weight, which
   is 1 at most: 2^-36 (|m| + 15 s) a token.
 - p s likewise, in the unit of its stage: 2^-36 15 units a token.  The unit is 8 times the
   largest s at most of where they were last looked at, which is within 6144 tokens before the
   stage's end; or it is 1, and then some s there is 2^-7 or more, 2^-11 where the
   request has up to 65536 tokens; or it is 2^-15.
 - s in that unit, when it is 2 or more: 2^-25 of it, times 15 and the stage's weight.
 - the result is rounded to bf16: 2^-8 of itself; fp32 sums and exponentials: 2^-12 size.
 - scores off by 2^-20 of mag = sum |q| (|m| + s n) move every weight by as much: 2 size times that.
"""

import math

import numpy as np
import pytest
import torch

import q4_reference as ref
from q4_cases import Batch, i32
from top_sparse_attention_pks_gb300 import build
from top_sparse_attention_pks_gb300.decoder import Q4Attention, Q4SparseAttention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def groups(b, kind):
    """(value, |m| + s n [tokens, Hkv, D], |m|, s [tokens, Hkv, D / 32]) of the stored rows."""
    pool = {"k": b.cache.k, "v": b.cache.v}[kind].cpu().numpy()
    n, s, m = ref.unpack(pool, b.Hkv, b.D, kind)
    _, pg, sl = (np.array(c) for c in zip(*ref.places(b.lens, b.tab, b.starts, b.P)))
    n, s, m = n[pg, sl], s[pg, sl], m[pg, sl]
    return [torch.from_numpy(x).cuda()
            for x in (ref.values(n, s, m), ref.values(n, s, np.abs(m)), np.abs(m), s)]


def largest(s, block):
    """The largest s [tokens, Hkv, NB] of each block."""
    top = torch.zeros((int(block[-1]) + 1,) + s.shape[1:], dtype=torch.float64, device="cuda")
    return top.scatter_reduce(0, block[:, None, None].expand(s.shape), s, "amax")


def check(b, out, lse, lists=None, causal=False, sm_scale=0.0):
    scale = sm_scale or 1.0 / math.sqrt(b.D)
    k, k_size, _, _ = groups(b, "k")
    v, v_size, m, s = groups(b, "v")
    for r, n in enumerate(b.lens):
        for i in range(b.Nq):
            if lists is None:
                t = np.arange(max(0, n - b.Nq + i + 1) if causal else n)
                index = t
            else:
                keep = np.flatnonzero(lists[r][i] >= 0)
                t, index = lists[r][i][keep], keep
            at = torch.from_numpy(t + b.starts[r]).cuda()
            index = torch.from_numpy(index).cuda()
            q = b.q[r, i].double().view(b.Hkv, b.G, b.D)
            x = torch.einsum("hgd,thd->hgt", q, k[at]) * scale
            mag = torch.einsum("hgd,thd->hgt", q.abs(), k_size[at]).amax(-1) * scale
            z = torch.logsumexp(x, -1)
            p = (x - z[..., None]).exp()
            want = torch.einsum("hgt,thd->hgd", p, v[at])
            size = torch.einsum("hgt,thd->hgd", p, v_size[at])
            # (of all tokens there, also those that this query does not see)
            all_s = s[b.starts[r]:b.starts[r] + n] if lists is None else s[at]
            all_i = torch.arange(n, device="cuda") if lists is None else index
            near = largest(all_s, all_i // 6144)
            near[1:] = torch.maximum(near[1:], near[:-1].clone())
            near = near[index // 6144]
            small = 2.0 ** (7 if (n if lists is None else len(lists[r][i])) > 65536 else 11)
            unit = torch.maximum(8 * near, (small * near).clamp(2.0 ** -15, 1.0))
            w = torch.einsum("hgt,thb->hgb", p, unit * (unit > 1)) * (15 * 2.0 ** -25)
            lost = ((m[at] + 15 * s[at] + 15 * unit) * 2.0 ** -36).sum(0)
            tol = (2.0 ** -10 + 2.0 ** -12 + 2 * 2.0 ** -20 * mag[..., None]) * size
            tol = tol + 2.0 ** -8 * want.abs()
            tol = tol + (w + lost[:, None]).repeat_interleave(32, -1)
            got = out[r, i].double().view_as(want)
            bad = ~((got - want).abs() <= tol)  # (nothing may be a NaN)
            assert not bad.any(), f"{float(((got - want).abs() / tol)[bad].max())} of tolerance"
            # (of a lane's sum of the weights: n / 8 additions, each off by 2^-24)
            ltol = 2.0 ** -18 * (1 + z.abs()) + 2.0 ** -20 * mag + n * 2.0 ** -27
            assert bool(((lse[r, i].double().view_as(z) - z).abs() <= ltol).all())


def dominated(n, share, v_scale, Hkv=1, G=2, D=128, Nq=1, page=64, at=10, seed=0):
    """A request in which token ``at`` has ``share`` of the weight and the others, whose V has a
    mean, about as much each of the rest; v_scale: a number, or one a group of 32 values."""
    b = Batch([n], page, Hkv, G, D, Nq, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    base = torch.randn((Hkv, D), generator=g, device="cuda")
    base = base * (8.0 / base.norm(dim=-1, keepdim=True))
    noise = torch.randn(b.q.shape, generator=g, device="cuda") * 0.01
    b.q = (base.repeat_interleave(G, 0) + noise).to(torch.bfloat16)
    b.k = 0.05 * torch.randn(b.k.shape, generator=g, device="cuda")
    score = math.log(share / (1 - share) * n)
    b.k[at] = base * (score * math.sqrt(D) / 64.0)
    size = torch.as_tensor(v_scale, device="cuda", dtype=torch.float32)
    if size.dim():
        size = size.repeat_interleave(32)
    mean = torch.randn((Hkv, D), generator=g, device="cuda").sign()
    b.v = (torch.randn(b.v.shape, generator=g, device="cuda") * 0.5 + mean) * size
    b.write()
    return b


def run(b, lists=None, causal=False, copies=None):
    """Attention over a request for every SM, all over the same pages, so that a CTA has it whole
    and what comes behind the dominant token is weighed against it; or over ``copies``."""
    n = copies or torch.cuda.get_device_properties(0).multi_processor_count
    lens, table, q = (x.repeat_interleave(n, 0) for x in (b.len_d, b.table, b.q))
    if lists is None:
        att = Q4Attention(lens, table, q, b.cache, causal=causal, lse=True)
    else:
        lists_d = i32(lists).repeat_interleave(n, 0)
        att = Q4SparseAttention(lens, table, lists_d, q, b.cache, lse=True)
    out = att()
    assert att.device_error() == 0
    assert torch.equal(out, out[:1].expand(out.shape))
    check(b, out[:1], att.lse[:1], lists=lists, causal=causal)
    return out[:1]


@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
@pytest.mark.parametrize("v_scale", [1.0, 1e-2, 1e-3, 3e-4, 1e-4, 3e-5, 1e-6, 3e2, 1e4])
def test_a_dominant_token_beside_many(v_scale, share):
    run(dominated(131072, share, v_scale))


@pytest.mark.parametrize("Hkv,G,D,page,Nq", [
    (8, 1, 128, 64, 1), (8, 4, 128, 16, 4), (2, 4, 64, 5, 1), (1, 16, 64, 16, 1),
    (5, 12, 128, 16, 1), (16, 1, 64, 16, 1), (8, 16, 128, 64, 1)])
@pytest.mark.parametrize("v_scale", [1e-4, 1e-6])
def test_small_values_by_every_way_of_copying(Hkv, G, D, page, Nq, v_scale):
    b = dominated(20000, 0.9, v_scale, Hkv, G, D, Nq, page, seed=1)
    run(b, causal=True)
    rng = np.random.default_rng(2)
    lists = np.stack([np.sort(rng.permutation(20000)[:4000])] * Nq)[None]
    lists[..., 7] = 10
    lists[..., 100:140] = -1
    run(b, lists=lists)


@pytest.mark.parametrize("sizes", [(1.0, 1e-4, 1e-2, 1e-6), (1e4, 1.0, 1e-3, 1e-5),
                                   (1e-5, 1e-5, 1e4, 0.0), (2.0 ** -24, 1e-6, 1.0, 100.0)])
def test_groups_of_different_sizes(sizes):
    b = dominated(131072, 0.9, sizes, seed=3)
    run(b)
    run(b, copies=1)  # (every CTA a part of it, in units of its own)
    b = dominated(9000, 0.5, sizes, G=16, at=5000, seed=3)
    run(b, copies=1)


@pytest.mark.parametrize("small,large", [(1e-4, 1.0), (1.0, 1e4), (1e-5, 1e4), (0.0, 1.0)])
def test_sizes_that_change_along_a_request(small, large):
    """Single large tokens, and stretches of small and large ones in turn."""
    b = dominated(60000, 0.9, 1.0, seed=4)
    size = torch.full((60000, 1, 1), small, device="cuda")
    size[[5, 333, 20000, 59999]] = large
    size[30000:30100] = large
    size[40000:50000] = large
    size[41000:42000] = small
    b.v *= size
    b.write()
    run(b)


def test_few_tokens_without_scales_before_many_small_ones():
    """Lists whose first stage has few tokens, and these no scales."""
    b = dominated(20000, 0.9, 1e-6, seed=8)
    b.v[:40] = 1e-6
    b.write()
    lists = np.full((1, 1, 19000), -1)
    lists[0, 0, [3, 40, 77, 100, 130, 170, 200, 230]] = np.arange(5, 13)
    lists[0, 0, 256:] = np.arange(1000, 1000 + 19000 - 256)
    run(b, lists=lists)


def test_values_without_any_scale():
    """All values of a group alike: s is 0 and everything is in m."""
    b = dominated(5000, 0.9, 1.0, seed=5)
    b.v[:] = b.v[:, :, :1]
    b.v[2500:] *= 1e-4
    b.write()
    run(b)


def test_more_than_a_million_tokens():
    n = (1 << 20) + 77
    for v_scale in (0.02, 1.0):
        run(dominated(n, 0.9, v_scale, D=64, G=1, seed=6))


@pytest.mark.parametrize("large", [100.0, 6e4])
def test_a_large_draft_is_without_influence_on_those_before_it(large):
    """The last of four drafted tokens has large values."""
    b = dominated(1000, 0.9, 1.0, 2, 4, 128, 4, seed=7)
    first = run(b, causal=True).clone()
    b.v[-1] *= large / b.v[-1].abs().amax()
    b.write()
    out = run(b, causal=True)
    # the first three queries see the tokens that they saw: 2^-22 15 of the large scale, 2 / 15 of
    # the value, and two roundings
    lim = 2.0 ** -7 * first[:, :3].float().abs() + 15 * 2.0 ** -22 * large * 2 / 15
    assert bool(((out[:, :3].float() - first[:, :3].float()).abs() <= lim).all())
