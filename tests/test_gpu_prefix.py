"""Attention over a batch with shared prefixes against a 64-bit restatement, a
request at a time through its own table row.

Tolerance of an output value: the weights p are rounded to bf16 for the second
product (each by at most 2^-8 of itself, so the sum by 2^-8 sum p |V|), and the
result is rounded to bf16 (2^-8 of itself).  What else there is (fp32 sums of up
to 2^17 terms in a tree of short runs, the approximate exponential's few ulp, the
scores' fp32 products: |score| 2^-24 D in the exponent) is held to 2^-12 sum p |V|.
lse: the scores' error, 2^-24 D sum |q k|, and 2^-18 for the sum and logarithm.
"""

import math

import numpy as np
import pytest
import torch

from top_sparse_attention_pks_gb300 import build, pks
from top_sparse_attention_pks_gb300.decoder import PageTable, PrefixAttention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def dev(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Batch:
    """Rows of `lens` tokens; row b aliases the first `shared[b]` tokens' whole
    pages of its group's store, pages dealt at random.  What no row holds is NaN."""

    def __init__(self, lens, group, shared, page=16, Hkv=2, G=4, D=64, Nq=1, seed=0, spare=2,
                 q_scale=1.0, groups_passed=True):
        rng = np.random.default_rng(seed)
        self.lens, self.P, self.Hkv, self.G, self.D, self.Nq = list(lens), page, Hkv, G, D, Nq
        B = len(lens)
        pages = [-(-n // page) for n in lens]
        width = max(pages + [1]) + 1
        table = np.full((B, width), -7, np.int64)
        store, at = {}, 0
        for b in range(B):
            w = min(shared[b] // page, pages[b]) if group[b] >= 0 else 0
            have = store.setdefault(group[b], [])
            while len(have) < w:
                have.append(at)
                at += 1
            table[b, :w] = have[:w]
            table[b, w:pages[b]] = np.arange(at, at + pages[b] - w)
            at += pages[b] - w
        N = at + spare
        deal = rng.permutation(N)
        held = np.arange(width)[None, :] < np.array(pages)[:, None]
        table = np.where(held, deal[np.where(held, table, 0)], -7)
        g = torch.Generator(device="cuda").manual_seed(seed)
        shape = (N, page, Hkv, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        self.v = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        used = np.zeros((N, page), bool)
        for b in range(B):
            t = np.arange(self.lens[b])
            used[table[b, t // page], t % page] = True
        unused = torch.from_numpy(~used).cuda()
        self.k[unused] = float("nan")
        self.v[unused] = float("nan")
        self.q = (torch.randn((B, Nq, Hkv * G, D), generator=g, device="cuda") * q_scale
                  ).to(torch.bfloat16)
        self.table, self.len_d = dev(table), dev(lens)
        self.group = dev(group) if groups_passed else None

    def attention(self, **kw):
        kw.setdefault("lse", True)
        return PrefixAttention(self.len_d, self.table, self.q, self.k, self.v,
                               prefix_group=self.group, **kw)

    def check(self, out, lse, causal=False, sm_scale=0.0, rows=None, what=""):
        scale = sm_scale or 1.0 / math.sqrt(self.D)
        for b in (range(len(self.lens)) if rows is None else rows):
            n = self.lens[b]
            t = torch.arange(n, device="cuda")
            at = self.table[b].long()[t // self.P] * self.P + t % self.P
            k = self.k.view(-1, self.Hkv, self.D)[at].double()
            v = self.v.view(-1, self.Hkv, self.D)[at].double()
            for i in range(self.Nq):
                lim = max(0, n - self.Nq + i + 1) if causal else n
                got, got_lse = out[b, i].double(), lse[b, i].double()
                if lim == 0:
                    assert not got.any() and bool((got_lse == -math.inf).all()), f"{what} b={b}"
                    continue
                q = self.q[b, i].double().view(self.Hkv, self.G, self.D)
                x = torch.einsum("hgd,thd->hgt", q, k[:lim]) * scale
                mag = torch.einsum("hgd,thd->hgt", q.abs(), k[:lim].abs()).amax(-1) * scale
                z = torch.logsumexp(x, -1)
                p = (x - z[..., None]).exp()
                want = torch.einsum("hgt,thd->hgd", p, v[:lim]).reshape(-1, self.D)
                size = torch.einsum("hgt,thd->hgd", p, v[:lim].abs()).reshape(-1, self.D)
                tol = (2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -8 * want.abs()
                # the scores' own error moves every weight
                tol = tol + (2.0 ** -23 * self.D * mag).reshape(-1, 1) * 2 * size
                bad = (got - want).abs() > tol
                assert not bad.any() and bool(torch.isfinite(got).all()), \
                    f"{what} b={b} i={i}: {float(((got - want).abs() / tol).max())} of tolerance"
                ltol = 2.0 ** -18 * (1 + z.abs()) + 2.0 ** -24 * self.D * mag
                assert bool(((got_lse.view_as(z) - z).abs() <= ltol).all()), f"{what} lse b={b}"

    def run(self, causal=False, sm_scale=0.0, what="", rows=None):
        att = self.attention(causal=causal, sm_scale=sm_scale)
        att.out.fill_(float("nan"))
        att.lse.fill_(float("nan"))
        out = att()
        torch.cuda.synchronize()
        assert att.device_error() == 0, what
        self.check(out, att.lse, causal, sm_scale, rows, what)
        return att


def test_worked_example():
    b = Batch([403, 96, 241, 30, 176], [0, 0, 0, -1, -1], [64, 64, 64, 0, 0])
    b.run()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 4), (8, 8), (3, 5), (4, 16), (6, 7)])
@pytest.mark.parametrize("Nq,causal", [(1, False), (3, True)])
def test_heads(D, Hkv, G, Nq, causal):
    """Up to 48 rows a request: both kernels for the own tokens."""
    Batch([700, 513, 640, 300, 1, 0, 257], [0, 0, 0, -1, 0, 0, 1], [512] * 7, Hkv=Hkv, G=G, D=D,
          Nq=Nq, seed=Hkv * 100 + G).run(causal)


@pytest.mark.parametrize("page", [1, 5, 16, 48, 64, 100, 128, 512])
def test_page_sizes(page):
    Batch([1500, 1333, 1024, 1023, 1025, 7], [4, 4, 4, 4, 4, 4], [1024] * 6, page=page, D=128,
          Hkv=1, G=8, seed=page).run()


@pytest.mark.parametrize("pre", [1, 127, 128, 129, 255, 256, 384, 1000, 2049])
@pytest.mark.parametrize("own", [0, 1, 130])
def test_prefix_lengths(pre, own):
    """Whole and ragged tiles of the prefix, one-token pages so that every
    length is shared to the token; own parts of no token and of some."""
    lens = [pre + own, pre + own // 2, pre]
    Batch(lens, [0, 0, 0], [pre] * 3, page=1, D=64, Hkv=2, G=4, seed=pre + own).run()


@pytest.mark.parametrize("members,G", [(2, 1), (15, 8), (16, 8), (17, 8), (31, 8), (32, 8), (33, 8),
                                       (70, 8), (129, 2)])
def test_rows_of_the_shared_part(members, G):
    """From two rows to more than two items of 256 rows."""
    rng = np.random.default_rng(members)
    lens = (640 + rng.integers(0, 90, members)).tolist()
    Batch(lens, [7] * members, [640] * members, D=128, Hkv=2, G=G, seed=members).run()


@pytest.mark.parametrize("Nq", [2, 8, 17, 64])
@pytest.mark.parametrize("causal", [False, True])
def test_query_tokens(Nq, causal):
    """Drafted tokens, more of them than some requests have tokens."""
    Batch([900, 800, 5, 64, 0, 1300], [0, 0, 0, 0, 0, 0], [768] * 6, D=128, Hkv=2, G=4, Nq=Nq,
          seed=Nq).run(causal)


def test_members_that_share_less():
    """A member that shares little stays on its own; the others take the least
    common prefix; a group id that aliases nothing changes nothing."""
    Batch([2000, 1900, 1500, 400, 300, 2000], [0] * 6, [1600, 1600, 1200, 352, 0, 1600], D=128,
          Hkv=2, G=8, seed=3).run()
    Batch([500, 500, 500], [0, 0, 0], [0, 0, 0], seed=4).run()
    Batch([500] * 9, [2, 0, 1, 2, 0, 1, 2, 0, 1], [320] * 9, seed=5, D=128).run()  # interleaved
    Batch([500] * 4, [10 ** 6, 10 ** 6, 3, 3], [320] * 4, seed=6).run()  # any ids


def test_no_groups():
    for Nq in (1, 6):
        Batch([700, 3, 0, 129], [-1] * 4, [0] * 4, G=4, Nq=Nq, seed=8, groups_passed=False).run()
        Batch([700, 3, 0, 129], [-1] * 4, [0] * 4, G=4, Nq=Nq, seed=8).run()
    one = Batch([1], [-1], [0], Hkv=1, G=1, seed=9)
    one.run()


def test_scales_that_move_the_maximum():
    """Scores of some hundreds: the running maximum moves often and far."""
    for Nq, D in ((1, 128), (5, 64)):
        b = Batch([3000, 2800, 2600], [0] * 3, [2048] * 3, D=D, Hkv=1, G=8, Nq=Nq, q_scale=30.0,
                  seed=D)
        b.run(causal=True)
        b.run(sm_scale=2.0)
        b.run(sm_scale=1e-3)


def test_long_prefix_many_requests():
    rng = np.random.default_rng(1)
    lens = (20000 + rng.integers(0, 700, 64)).tolist()
    Batch(lens, [0] * 64, [20000] * 64, page=64, D=128, Hkv=4, G=8, seed=11).run(rows=[0, 13, 63])


def test_many_requests():
    """4096 requests: the plan's largest batch, every group of 64."""
    rng = np.random.default_rng(2)
    B = 4096
    lens = (128 + rng.integers(0, 60, B)).tolist()
    lens[5] = lens[4000] = 0
    Batch(lens, (np.arange(B) // 64).tolist(), [128] * B, D=64, Hkv=1, G=2, seed=12).run(
        rows=[0, 1, 5, 63, 64, 2000, 4000, 4095])


def test_offsets_past_32_bits():
    """Pools of 4.6 GB each, the requests' pages at their far end: element offsets
    beyond 2^31 on every path (whole boxes, odd starts, drafts)."""
    P, Hkv, D, N = 16, 8, 128, 140_000
    k = torch.empty((N, P, Hkv, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty((N, P, Hkv, D), dtype=torch.bfloat16, device="cuda")
    for Nq, lens in ((1, [700, 650, 90]), (5, [700, 650, 90])):
        b = Batch(lens, [0, 0, -1], [512, 512, 0], page=P, Hkv=Hkv, G=4, D=D, Nq=Nq, seed=20 + Nq)
        n = b.k.shape[0]
        k[N - n:], v[N - n:] = b.k, b.v
        b.k, b.v = k, v
        b.table = torch.where(b.table >= 0, b.table + (N - n), b.table)
        b.run(causal=True)


def test_batches_without_tokens():
    for lens, group in (([0, 0, 0], [0, 0, -1]), ([0], [-1])):
        for Nq in (1, 7):
            b = Batch(lens, group, [0] * len(lens), Hkv=2, G=8, D=128, Nq=Nq, seed=23)
            b.run(causal=True)
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    pool = torch.empty((1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    att = PrefixAttention(dev(np.zeros(0)), dev(np.zeros((0, 1))), q, pool, pool)
    assert att().shape == (0, 8, 64)
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        PrefixAttention(torch.zeros(1, dtype=torch.int32), dev([[0]]),
                        torch.empty((1, 8, 64), dtype=torch.bfloat16, device="cuda"), pool, pool)


def test_results_do_not_depend_on_who_computes_them():
    """Both kernels side by side with pieces claimed by whichever CTA is free: every
    run gives the same bits."""
    rng = np.random.default_rng(24)
    lens = (4000 + rng.integers(1, 900, 32)).tolist()
    b = Batch(lens, (np.arange(32) // 8).tolist(), [4000] * 32, page=16, Hkv=8, G=4, D=128, Nq=4,
              seed=24)
    att = b.run(causal=True, rows=[0, 9, 31])
    want = att.out.clone(), att.lse.clone()
    for _ in range(30):
        att.out.fill_(float("nan"))
        att.attend()
        assert torch.equal(att.out, want[0]) and torch.equal(att.lse, want[1])


def test_infinite_values_in_rows_of_others():
    """A request's own infinities and NaN stay its own, also beside a prefix."""
    b = Batch([600, 610, 620], [0] * 3, [512] * 3, page=16, D=128, Hkv=1, G=8, seed=13)
    page = int(b.table[1, 33])
    b.k[page] = float("nan")
    b.v[page] = float("inf")
    att = b.attention()
    out = att()
    torch.cuda.synchronize()
    b.check(out, att.lse, rows=[0, 2])
    assert bool(torch.isnan(out[1]).all())


def test_bad_pages_and_lengths_are_flagged():
    b = Batch([600, 610, 50], [0, 0, -1], [512, 512, 0], D=128, Hkv=1, G=8, seed=14)
    b.table[2, 1] = 10 ** 6
    att = b.attention()
    out = att()
    torch.cuda.synchronize()
    assert att.device_error() == 1 and att.device_error() == 0
    b.check(out, att.lse, rows=[0, 1])
    assert bool(torch.isfinite(out).all())
    b.table[0, 3] = b.table[1, 3] = -1  # in the shared part
    att()
    torch.cuda.synchronize()
    assert att.device_error() == 1
    b = Batch([600, 610, 50], [0, 0, -1], [512, 512, 0], D=128, Hkv=1, G=8, seed=14)
    b.len_d[1] = 10 ** 6
    b.len_d[2] = -4
    att = b.attention()
    out = att()
    torch.cuda.synchronize()
    assert att.device_error() == 3
    assert not out[1:].any()
    b.check(out, att.lse, rows=[0])


def test_waits_that_run_out():
    """The mbarrier waits of the wide kernel with a limit of one cycle give up
    with code 5, and the same buffers work again afterwards."""
    b = Batch([4000, 4100], [0, 0], [3968] * 2, D=128, Hkv=2, G=8, seed=15)
    att = b.attention(wait_limit=1)
    att()
    torch.cuda.synchronize()
    assert att.device_error() == 5
    att.args.wait_limit = 0
    for _ in range(2):
        out = att()
    torch.cuda.synchronize()
    assert att.device_error() == 0
    b.check(out, att.lse)


def test_repeats_are_equal_and_capture_follows_the_lengths():
    b = Batch([900, 1200, 1300, 40], [0, 0, 0, 1], [768] * 4, D=128, Hkv=2, G=8, Nq=2, seed=16)
    att = b.attention(causal=True)
    first = att().clone(), att.lse.clone()
    for _ in range(3):
        out = att()
        assert torch.equal(out, first[0]) and torch.equal(att.lse, first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        att()
    lens = list(b.lens)
    for drop in (0, 1, 100, 500):
        b.lens = [max(0, n - drop) for n in lens]
        b.len_d.copy_(dev(b.lens))
        att.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert att.device_error() == 0
        b.check(att.out, att.lse, causal=True, what=f"drop {drop}")


def test_one_plan_for_several_layers_and_streams():
    b = Batch([900, 1200, 1300, 40], [0, 0, 0, 1], [768] * 4, D=64, Hkv=2, G=8, seed=17)
    att = b.attention()
    att.plan()
    for layer in range(3):
        out = att.attend(b.q, b.k, b.v)
        torch.cuda.synchronize()
        b.check(out, att.lse)
        b.q = (b.q.float() * 0.7).to(torch.bfloat16)
        b.k, b.v = b.v.clone(), b.k.clone()
    with pytest.raises(ValueError):
        att.attend(b.q[:, :, :8].contiguous())
    with pytest.raises(TypeError):
        att.attend(b.q.float())
    # two objects on two streams at once
    other = Batch([5000, 5100], [0, 0], [4096] * 2, D=128, Hkv=4, G=4, seed=18)
    att2, att3 = b.attention(), other.attention()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        att2(stream=s1)
        att3(stream=s2)
    torch.cuda.synchronize()
    b.check(att2.out, att2.lse)
    other.check(att3.out, att3.lse)


def test_fork_extend_attend_free_compact():
    """The calls together, as a sampling loop makes them: a prompt is forked,
    every fork grows a token at a time (its K/V written by the caller), the batch
    attends with the forks as one group, half of them are dropped, the pages are
    compacted, and the rest goes on."""
    P, Hkv, G, D, N = 16, 2, 8, 128, 400
    rows, prompt, forks = 10, 1000, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn((N, P, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((N, P, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    pool = pks.Pool(N, P, np.random.default_rng(0).permutation(N))
    bt, _ = pool.build_block_table([prompt, 70] + [0] * (rows - 2), 80)
    lens, table = dev([prompt, 70] + [0] * (rows - 2)), dev(bt)
    pages = PageTable(lens, table, N, P, pools=[k, v])
    pages.fork(dev([0] * (forks - 1)), dev(range(2, 2 + forks - 1)))
    group = dev([0, -1] + [0] * (rows - 2))
    q = torch.randn((rows, 1, Hkv * G, D), generator=g, device="cuda").to(torch.bfloat16)
    att = PrefixAttention(lens, table, q, k, v, prefix_group=group, lse=True)
    add = torch.ones(rows, dtype=torch.int32, device="cuda")
    add[rows - 1] = 0
    ref = Batch.__new__(Batch)
    ref.P, ref.Hkv, ref.G, ref.D, ref.Nq = P, Hkv, G, D, 1

    def steps(n):
        for _ in range(n):
            pages.extend(add)
            t = lens.long() - 1  # the new token's row
            for b in range(rows):
                if int(add[b]):
                    page = int(table[b, int(t[b]) // P])
                    new = torch.randn((2, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
                    k[page, int(t[b]) % P], v[page, int(t[b]) % P] = new[0], new[1]
            att()
        torch.cuda.synchronize()
        assert pages.device_error() == 0 and att.device_error() == 0
        ref.lens, ref.table, ref.k, ref.v, ref.q = lens.tolist(), table, k, v, q
        ref.check(att.out, att.lse)

    steps(1)
    assert len({int(table[b, 62]) for b in (0, 2, 3, 4, 5, 6, 7, 8)}) == 8, "a page each"
    assert len({int(table[b, 61]) for b in (0, 2, 3, 4, 5, 6, 7, 8)}) == 1
    steps(20)
    pages.free(dev([0, 3, 5, 7]))
    add[[0, 3, 5, 7]] = 0
    held = int((pages.refs > 0).sum())
    pages.compact()
    assert int(table[[1, 2, 4, 6, 8]].max()) == held - 1
    steps(3)


@pytest.mark.parametrize("page", [8, 24, 32, 40, 192])
@pytest.mark.parametrize("D,G", [(64, 8), (128, 16)])
def test_boxes(page, D, G):
    """Boxes of 8, 16, 32 and 64 rows, whole tiles and ends, one block of rows and
    two; several pieces a CTA."""
    members = 20 if page < 40 else 6
    pre = -(-1000 // page) * page
    lens = [pre + 7 * i for i in range(members)] + [3 * page + 5]
    Batch(lens, [1] * members + [-1], [pre] * members + [0], page=page, D=D, Hkv=2, G=G,
          seed=page + D).run()
    Batch(lens, [1] * members + [-1], [pre] * members + [0], page=page, D=D, Hkv=2, G=G, Nq=3,
          seed=page + D + 1).run(causal=True, rows=[0, 5, members])


@pytest.mark.parametrize("Hkv", [1, 2, 4, 8])
@pytest.mark.parametrize("page", [1, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_own_tokens_row_by_row(Hkv, page, D):
    """Pages without whole boxes: every number of heads that a CTA takes."""
    Batch([100, 33, 16, 15, 1], [-1] * 5, [0] * 5, page=page, D=D, Hkv=Hkv, G=2, Nq=3,
          seed=Hkv + page + D).run(causal=True)


@pytest.mark.parametrize("B,Hkv,G,Nq", [
    (1, 1, 4, 2),      # hundreds of parts a row
    (3, 8, 8, 1),
    (40, 8, 16, 1),    # a warp a row
    (6, 8, 8, 17),     # the most rows of that kind (152 SMs: 6,080), and one more
    (190, 8, 4, 1),    # request
    (191, 8, 4, 1),
    (16, 8, 16, 8),    # eight lanes a row, some rows of many parts
])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_and_parts(B, Hkv, G, Nq, D):
    """Few and many rows to merge, the first request's of many parts, some of none."""
    lens = [9000] + [0, 70, 300, 17][: B - 1] * (B // 4 + 1)
    lens = lens[:B]
    Batch(lens, [-1] * B, [0] * B, D=D, Hkv=Hkv, G=G, Nq=Nq, seed=B).run(
        rows=sorted({0, min(1, B - 1), min(3, B - 1), B - 1}))


def test_little_own_work_beside_the_prefix():
    """Pieces of a few tiles, and of twelve."""
    for own in (20, 200, 900):
        Batch([320 + own] * 13, [0] * 8 + [1] * 5, [320] * 13, page=5, D=128, Hkv=8, G=4,
              seed=own).run(rows=[0, 7, 8, 12])


def test_later_calls_keep_to_a_layers_tensors():
    b = Batch([900, 1200], [0, 0], [768] * 2, seed=21)
    att = b.attention()
    q = (b.q.float() * 0.5).to(torch.bfloat16)
    b.q = q.clone()
    att.plan()
    att.attend(q)
    del q
    trash = [torch.full_like(b.q, float("nan")) for _ in range(8)]
    out = att()
    torch.cuda.synchronize()
    b.check(out, att.lse)
    del trash


def test_another_current_device_is_refused(monkeypatch):
    b = Batch([900, 1200], [0, 0], [768] * 2, seed=22)
    att = b.attention()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (att, att.plan, att.attend, b.attention):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("Nq,groups", [(1, True), (1, False), (5, True)])
def test_attention_needs_a_plan_of_its_shapes(Nq, groups):
    b = Batch([900, 1200], [0, 0], [768] * 2, Nq=Nq, seed=23, groups_passed=groups)
    att = b.attention()
    att.out.fill_(3.0)
    att.attend()
    torch.cuda.synchronize()
    assert att.device_error() == 4 and bool((att.out == 3.0).all())
    att.plan()
    # a plan of the same buffers for other shapes
    other = b.attention(causal=True)
    other.args.workspace, other.args.workspace_bytes = (att.args.workspace,
                                                        att.args.workspace_bytes)
    other.out.fill_(3.0)
    other.attend()
    assert other.device_error() == 4 and bool((other.out == 3.0).all())
    out = att.attend()
    torch.cuda.synchronize()
    assert att.device_error() == 0
    b.check(out, att.lse)


def test_a_refused_layer_leaves_the_one_before_in_place(monkeypatch):
    b = Batch([900, 1200], [0, 0], [768] * 2, seed=25)
    att = b.attention()
    out = att().clone()
    q, k, v = (torch.randn_like(x) for x in (b.q, b.k, b.v))
    odd = torch.empty(v.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view(v.shape)
    refused = [((q, k, v[1:]), ValueError), ((q, k[:, :, :1].contiguous(), v), ValueError),
               ((q, k, v.float()), TypeError), ((q, k, odd), pks.PksError),
               ((q, k, v.cpu()), ValueError)]
    for tensors, error in refused:
        with pytest.raises(error):
            att.attend(*tensors)
        att.out.fill_(float("nan"))
        assert torch.equal(att.attend(), out) and torch.equal(att(), out)
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        with pytest.raises(ValueError):
            att.attend(q, k, v)
    assert torch.equal(att.attend(), out)
    b.q, b.k, b.v = q, k, v
    b.check(att.attend(q, k, v), att.lse)
