"""Attention over a 4-bit cache, dense and over selected tokens, against the 64-bit
restatement of q4_cases (which derives the tolerances)."""

import os
import subprocess
import sys
import threading
from pathlib import Path

import numpy as np
import pytest
import torch

from q4_cases import Batch, i32
from top_sparse_attention_pks_gb300 import build
from top_sparse_attention_pks_gb300.decoder import Q4Attention, Q4Cache, Q4SparseAttention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("Hkv,G,D,page", [
    (2, 4, 64, 16), (8, 4, 128, 64), (8, 8, 128, 16), (1, 1, 64, 1), (1, 8, 128, 5), (3, 7, 64, 17),
    (4, 2, 128, 48), (5, 5, 128, 16), (6, 1, 64, 8), (7, 3, 128, 32), (16, 8, 128, 16),
    (16, 2, 64, 64), (9, 4, 64, 3), (15, 1, 128, 16), (32, 4, 128, 16), (18, 2, 64, 16),
    (8, 4, 128, 5), (3, 4, 64, 8), (2, 8, 128, 128), (13, 2, 64, 1), (17, 4, 64, 16), (27, 1, 64, 5)])
def test_dense_one_query(Hkv, G, D, page):
    Batch(LENS, page, Hkv, G, D, seed=Hkv).dense()


@pytest.mark.parametrize("Hkv,G,D,page,Nq", [
    (2, 4, 64, 16, 4), (8, 4, 128, 64, 4), (8, 16, 128, 16, 1), (1, 12, 64, 1, 1),
    (1, 16, 128, 5, 3), (4, 8, 128, 16, 5), (8, 8, 128, 64, 8), (2, 1, 64, 16, 64),
    (16, 16, 128, 16, 1), (12, 3, 128, 17, 3), (9, 16, 64, 16, 2), (3, 5, 64, 16, 2),
    (5, 2, 128, 8, 7), (10, 9, 64, 16, 1), (11, 12, 64, 16, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_dense_several_queries(Hkv, G, D, page, Nq, causal):
    Batch(LENS, page, Hkv, G, D, Nq, seed=Nq).dense(causal=causal)


@pytest.mark.parametrize("Hkv,G,D,page,k", [
    (2, 4, 64, 16, 64), (8, 8, 128, 64, 100), (1, 8, 128, 1, 7), (3, 16, 64, 17, 300),
    (16, 4, 128, 16, 33), (8, 1, 64, 5, 1), (32, 2, 128, 16, 16), (7, 12, 128, 16, 50)])
@pytest.mark.parametrize("holes", [False, True])
@pytest.mark.parametrize("Nq", [1, 3])
def test_selected_tokens(Hkv, G, D, page, k, holes, Nq):
    Batch(LENS, page, Hkv, G, D, Nq, seed=k).sparse(k, holes)


@pytest.mark.parametrize("page", list(range(1, 20)) + [24, 40, 100])
def test_pages_of_every_small_size(page):
    """A stage of one head is 256 tokens: pages of 7 are 38 of them, more than a warp's lanes."""
    lens = [255, 256, 257, 300, 511, 800]
    Batch(lens, page, 1, 2, 128, seed=page).dense()
    Batch(lens, page, 2, 2, 64, seed=page).dense()
    Batch(lens, page, 4, 9, 128, 2, seed=page).dense(causal=True)


@pytest.mark.parametrize("B,Hkv,longest", [(76, 16, 400), (77, 16, 400), (152, 8, 420), (153, 8, 90),
                                           (8, 8, 128), (8, 8, 160), (8, 8, 190), (1, 2, 700)])
def test_few_short_segments(B, Hkv, longest):
    """On both sides of the limits up to which a CTA has a segment to itself, some of them empty."""
    lens = np.random.default_rng(B).integers(0, longest + 1, B)
    lens[::7] = 0
    lens[-1] = longest
    Batch(lens, 16, Hkv, 2, 128, seed=B).dense()
    Batch(lens, 16, Hkv, 2, 128, 3, seed=B).sparse(70, holes=True)


def test_long_requests_split_over_all_sms():
    Batch([20000, 3, 0, 45011, 700], 64, 8, 8, 128, seed=1).dense()
    Batch([70001], 16, 1, 4, 128, seed=2).dense()
    Batch([50000, 9], 16, 2, 6, 64, 3, seed=3).dense(causal=True)
    Batch([30000, 40000], 16, 8, 4, 128, seed=4).sparse(4096)


def test_many_requests():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 40, 4096)
    Batch(lens, 16, 1, 2, 64, seed=5).dense(rows=range(0, 4096, 37))
    Batch(rng.integers(0, 90, 1000), 8, 2, 2, 64, 4, seed=6).sparse(20, rows=range(0, 1000, 31))


def test_empty_batches():
    Batch([0, 0, 0]).dense()
    Batch([0, 0, 0], Nq=2).sparse(5)
    b = Batch([0])
    e = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    q = torch.empty((0, 8, 64), dtype=torch.bfloat16, device="cuda")
    att = Q4Attention(e[:, 0].contiguous(), e, q, b.cache)
    att()
    assert att.device_error() == 0


@pytest.mark.parametrize("v_scale,q_scale", [
    (1e-3, 1.0), (1e-6, 1.0), (100.0, 1.0), (1e4, 1.0), (3e4, 1.0), (1.0, 0.0), (1.0, 1e-30), (1.0, 8.0)])
def test_sizes_of_values_and_queries(v_scale, q_scale):
    """Scales from subnormal to near fp16's end, and scores from all equal to one token's."""
    b = Batch([300, 40, 5], 16, 2, 4, 128, seed=7, q_scale=q_scale, v_scale=v_scale)
    b.dense()
    b.sparse(64)


def test_scales_that_grow_along_a_request():
    """A token's values a million times those before it, and the largest score late."""
    b = Batch([2000], 16, 2, 4, 128, seed=8, v_scale=1e-2)
    b.v[1500] *= 3e6
    b.v[777] *= 1e3
    b.k[1900] *= 4
    b.write()
    b.dense()


def test_sm_scale():
    b = Batch(LENS, 16, 2, 4, 64, 2, seed=9)
    b.dense(sm_scale=0.5, causal=True)
    b.sparse(20, sm_scale=0.01)


@pytest.mark.parametrize("sm_scale", [1e-12, 1e-17, 1e-20, 1e-30, 1e-38, 1e-44])
@pytest.mark.parametrize("q_scale", [0.0, 1e-30, 1.0])
def test_small_sm_scale(sm_scale, q_scale):
    """Scores that are all but 0: the mean of the tokens that are there."""
    b = Batch(LENS, 16, 2, 4, 64, 2, seed=25, q_scale=q_scale)
    b.dense(sm_scale=sm_scale, causal=True)
    b.sparse(20, holes=True, sm_scale=sm_scale)


@pytest.mark.parametrize("q_scale,sm_scale", [(1e37, 0.0), (3e38, 0.0), (1e37, 1e-37), (1e38, 1e-38),
                                              (1.0, 1e38), (1e-30, 1e30), (1.0, 3e38),
                                              (1e-32, 1e32), (1e-37, 1e37), (3e-39, 1e38)])
def test_large_queries_and_sm_scale(q_scale, sm_scale):
    """Keys of 0 have scores of 0, and sizes of queries and sm_scale may cancel."""
    b = Batch([37, 300], 16, 2, 4, 64, 2, seed=26)
    b.q = (b.q.float().clamp(-1, 1) * q_scale).to(torch.bfloat16)
    cancel = 0 < q_scale * sm_scale < 10
    if not cancel:
        b.k.zero_()
        b.write()
    b.dense(sm_scale=sm_scale, causal=True)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_tokens_that_a_query_does_not_see_are_without_influence(what):
    """The last of four drafted tokens has no finite K and V: the three queries before it see
    nothing of it, its own query gets NaN.  The same for a token that is not selected."""
    b = Batch([37, 80, 4], 16, 2, 4, 128, 4, seed=10)
    for e in b.starts[1:]:
        b.k[e - 1, :, 3] = what
        b.v[e - 1, :, 64:] = what
    b.write()
    att = Q4Attention(b.len_d, b.table, b.q, b.cache, causal=True, lse=True)
    out = att()
    assert bool(out[:, 3].isnan().all()) and bool(att.lse[:, 3].isnan().all())
    b.Nq = 3
    b.lens, lens = [n - 1 for n in b.lens], b.lens
    starts = b.starts
    k, v = b.k, b.v
    # the restatement over the tokens that the first three queries see
    keep = [i for s, e in zip(starts, starts[1:]) for i in range(s, e - 1)]
    b.starts = np.concatenate([[0], np.cumsum(b.lens)]).tolist()
    b.k, b.v = k[keep], v[keep]
    b.check(out, att.lse, causal=True)
    b.lens, b.starts, b.Nq = lens, starts, 4
    lists = np.stack([np.stack([np.arange(3)] * 4)] * 3)
    lists[2, 3] = [3, -1, 0]
    att = Q4SparseAttention(b.len_d, b.table, i32(lists), b.q, b.cache, lse=True)
    out = att()
    assert bool(out[2, 3].isnan().all()) and bool(out[:2].isfinite().all())
    assert bool(out[2, :3].isfinite().all())


@pytest.mark.parametrize("s", [0xffff, 0x7c00, 0xfc00, 0x3800])
@pytest.mark.parametrize("m", [0xffff, 0x7c00, 0xfc00, 0x3800])
@pytest.mark.parametrize("Hkv,G,D", [(2, 2, 64), (8, 4, 128), (5, 4, 128), (1, 1, 128)])
def test_bytes_that_a_query_does_not_see_are_without_influence(s, m, Hkv, G, D):
    """The pairs of the last of four drafted tokens, raw in its pages: scales and minima that a
    write never stores, in all groups or in one."""
    lens = [37, 80, 4, 33]
    b = Batch(lens, 16, Hkv, G, D, 4, seed=27)
    att = Q4Attention(b.len_d, b.table, b.q, b.cache, causal=True, lse=True)
    want, want_lse = att().clone(), att.lse.clone()
    pair = torch.tensor([s & 255, s >> 8, m & 255, m >> 8], dtype=torch.uint8, device="cuda")
    rec = D // 2 + D // 8
    for r, n in enumerate(lens):
        at = b.tab[r, (n - 1) // 16], (n - 1) % 16
        for pool in (b.cache.k, b.cache.v):
            row = pool[at]
            for i in range(D // 32 if r % 2 == 0 else 1):
                o = (Hkv - 1) * rec + D // 2 + 4 * i
                row[o:o + 4] = pair
    out = att()
    assert torch.equal(out[:, :3], want[:, :3]) and torch.equal(att.lse[:, :3], want_lse[:, :3])
    heads = (Hkv - 1) * G
    assert torch.equal(out[:, 3, :heads], want[:, 3, :heads])
    if s != 0x3800 or m != 0x3800:
        assert not out[:, 3, heads:, :32].isfinite().any()
    else:
        assert bool(out.isfinite().all())


def test_queries_that_are_not_finite_stay_their_own():
    b = Batch([50], 16, 2, 4, 64, seed=11)
    q = b.q.clone()
    b.q[0, 0, 3, 5] = float("nan")
    b.q[0, 0, 6, 0] = float("inf")
    att = Q4Attention(b.len_d, b.table, b.q, b.cache, lse=True)
    out = att().clone()
    assert bool(out[0, 0, [3, 6]].isnan().all())
    b.q.copy_(q)
    want = att()
    keep = [0, 1, 2, 4, 5, 7]
    assert torch.equal(out[0, 0, keep], want[0, 0, keep])


def test_bad_entries_are_skipped_and_told():
    b = Batch([64, 40, 33], 16, 2, 4, 64, seed=12)
    table = b.tab.copy()
    table[1, 1] = b.cache.k.shape[0]
    att = Q4Attention(b.len_d, i32(table), b.q, b.cache, lse=True)
    out = att()
    assert att.device_error() == 1 and att.device_error() == 0
    b.check(out, att.lse, rows=[0, 2])
    lists = [[t] for t in (np.arange(64), np.r_[np.arange(16), np.arange(32, 40)], np.arange(33))]
    b.check(out, att.lse, lists=lists)  # request 1 without the page's tokens
    lists = np.array([[[0, 5, 64, 7]], [[-1, 39, 40, -2]], [[1, 2, 3, -1]]])
    att = Q4SparseAttention(b.len_d, b.table, i32(lists), b.q, b.cache, lse=True)
    out = att()
    assert att.device_error() == 2
    b.check(out, att.lse, lists=lists)
    att = Q4Attention(i32([64, -3, 10 ** 6]), b.table, b.q, b.cache, lse=True)
    out = att()
    assert att.device_error() == 3
    b.check(out, att.lse, rows=[0])
    assert not out[1:].any()


def test_runs_give_the_same_bits():
    b = Batch([3000, 5000, 77], 16, 8, 8, 128, seed=13)
    att = b.dense()
    first, lse = att.out.clone(), att.lse.clone()
    for _ in range(20):
        att()
        assert torch.equal(att.out, first) and torch.equal(att.lse, lse)


@pytest.mark.parametrize("Hkv,G,D,Nq", [(1, 4, 64, 1), (1, 12, 128, 1), (2, 2, 64, 2), (3, 5, 64, 2),
                                        (6, 3, 64, 1), (13, 2, 64, 1), (10, 9, 64, 1)])
def test_small_rows_by_lanes(Hkv, G, D, Nq):
    """Stage behind stage of tokens that lanes copy by rows which other lanes looked up, some of
    them missing so that the lanes part: the same bits every time."""
    b = Batch([5000, 40, 3100], 5, Hkv, G, D, Nq, seed=24)
    att = b.sparse(3000, holes=True)
    first, lse = att.out.clone(), att.lse.clone()
    for _ in range(10):
        att()
        assert torch.equal(att.out, first) and torch.equal(att.lse, lse)


def test_a_position_twice_counts_twice():
    b = Batch([100, 40], 16, 2, 4, 64, seed=21)
    lists = b.lists(30)
    lists[0, 0, 10:20] = lists[0, 0, 5]
    lists[1, 0, :] = 39
    att = Q4SparseAttention(b.len_d, b.table, i32(lists), b.q, b.cache, lse=True)
    b.check(att(), att.lse, lists=lists)


def test_two_threads_and_streams():
    """Objects of their own over one cache, each called from a thread on a stream of its own."""
    b = Batch([3000, 700, 77], 16, 8, 4, 128, seed=22)
    want = b.dense().out.clone()
    atts = [Q4Attention(b.len_d, b.table, b.q, b.cache) for _ in range(2)]
    torch.cuda.synchronize()
    wrong = []

    def run(att, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(50):
                    att.out.zero_()
                    if not torch.equal(att(), want):
                        wrong.append(att)
        except BaseException as e:  # noqa: BLE001 (told below)
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(a, torch.cuda.Stream())) for a in atts]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert all(a.device_error() == 0 for a in atts)


def test_first_call_of_a_process_is_captured():
    code = """
import torch
from q4_cases import Batch, Q4Attention
b = Batch([300, 20], 16, 8, 4, 128, seed=23)
att = Q4Attention(b.len_d, b.table, b.q, b.cache, lse=True)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    att()
g.replay()
b.check(att.out, att.lse)
"""
    here = Path(__file__).parent
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(here), str(here.parent)]))
    subprocess.run([sys.executable, "-c", code], env=env, check=True, timeout=300)


def test_graphs_that_share_a_workspace_and_follow_lengths():
    b = Batch([300, 500, 77], 16, 2, 4, 64, seed=14)
    att = b.dense()
    lists = b.lists(50)
    sel = Q4SparseAttention(b.len_d, b.table, i32(lists), b.q, b.cache, trim=True, lse=True)
    if sel.workspace.numel() <= att.workspace.numel():
        sel.args.workspace, sel.args.workspace_bytes = att.args.workspace, att.args.workspace_bytes
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for a in (att, sel):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a()
        graphs.append(g)
    lens = b.lens
    for cut in (0, 1, 60, 76):
        b.lens = [n - cut for n in lens]
        b.len_d.copy_(i32(b.lens))
        for g in graphs:
            g.replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        full, b.lens = b.lens, lens
        seen = [[np.arange(n)] for n in full]
        b.check(att.out, att.lse, lists=seen)
        short = []
        for i, n in enumerate(full):  # trim: the first min(k, len) entries, those in reach
            t = lists[i][0][:min(50, n)]
            short.append([t[t < n]])
        b.check(sel.out, sel.lse, lists=short)
        b.lens = lens
        if cut:
            sel.device_error()


def test_graphs_that_share_a_workspace_and_join_parts():
    """Two objects whose segments several CTAs hold, so that both write the plan and the parts of
    the one workspace, replayed in turn with lengths that change in between."""
    b = Batch([9000, 5001, 77, 0, 3000], 16, 8, 4, 128, 2, seed=28)
    lists = b.lists(2500, seed=28)
    att = Q4Attention(b.len_d, b.table, b.q, b.cache, causal=True, lse=True)
    sel = Q4SparseAttention(b.len_d, b.table, i32(lists), b.q, b.cache, trim=True, lse=True)
    ws = torch.zeros(max(a.workspace.numel() for a in (att, sel)), dtype=torch.uint8, device="cuda")
    for a in (att, sel):
        a.workspace = ws
        a.args.workspace, a.args.workspace_bytes = ws.data_ptr(), ws.numel()
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a in (att, sel):
        a()
        assert bool((ws[256:] != 0).any())  # (the plan and the parts, not the error word alone)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            a()
        graphs.append(g)
    full = b.lens
    for cut in (0, 1, 2500, 4000, 0):
        b.lens = [max(0, n - cut) for n in full]
        b.len_d.copy_(i32(b.lens))
        short = [[t[:min(2500, n)] for t in rows] for rows, n in zip(lists, b.lens)]
        for order in ((0, 1), (1, 0)):
            for a in (att, sel):
                a.out.fill_(float("nan"))
                a.lse.fill_(float("nan"))
            for i in order:
                graphs[i].replay()
            torch.cuda.synchronize()
            now, b.lens = b.lens, full
            dense = [[np.arange(max(0, n - 1 + i)) for i in range(2)] for n in now]
            b.check(att.out, att.lse, lists=dense)
            b.check(sel.out, sel.lse, lists=[[t[t < n] for t in rows]
                                             for rows, n in zip(short, now)])
            b.lens = now
        sel.device_error()
        b.lens = full


def test_further_layers():
    """One object over the queries and caches of several layers."""
    b, c = (Batch([100, 30], 16, 2, 4, 64, seed=s) for s in (15, 15))
    c.q = torch.randn_like(c.q.float()).to(torch.bfloat16)
    c.k, c.v = c.k * 0.5, c.v * 2
    c.write()
    att = b.dense()
    first = att.out.clone()
    out = att.attend(c.q, c.cache)
    c.check(out, att.lse)
    with pytest.raises(ValueError):
        att.attend(b.q[:, :, :4])
    with pytest.raises(TypeError):
        att.attend(b.q.float())
    c.check(att(), att.lse)
    assert torch.equal(att.attend(b.q, b.cache), first)


@pytest.mark.parametrize("page", [16, 5])
def test_a_wait_that_runs_out_is_told(page):
    """A limit far below what a copy takes: the warps give up, the call ends with device error
    5 and the context stays usable.  Of a short batch the copies may have landed before they
    are waited for; its result is then the right one."""
    b = Batch([3000, 5000], page, 8, 8, 128, seed=16)
    att = Q4Attention(b.len_d, b.table, b.q, b.cache, wait_limit=10, lse=True)
    att()
    code = att.device_error()
    assert code in (0, 5)
    if code == 0:
        b.check(att.out, att.lse)
    # ten times as many stages as the ring holds: some warp has to wait
    b = Batch([300000], page, 8, 8, 128, seed=17)
    att = Q4Attention(b.len_d, b.table, b.q, b.cache, wait_limit=10)
    att()
    assert att.device_error() == 5
    b.dense()


def test_long_tables_and_large_pools():
    """Rows beyond 2^31 bytes of a pool."""
    N, page, Hkv, D = 60000, 64, 8, 128
    cache = Q4Cache(N, page, Hkv, D)
    b = Batch([130], page, Hkv, 4, D, seed=17)
    tab = np.array([[N - 1, 3, N - 2, -7]])
    b.cache, b.tab, b.table = cache, tab, i32(tab)
    b.write()
    att = Q4Attention(b.len_d, b.table, b.q, cache, lse=True)
    out = att()
    small = Batch([130], page, Hkv, 4, D, seed=17)
    want = small.dense()
    assert torch.equal(out, want.out) and torch.equal(att.lse, want.lse)
