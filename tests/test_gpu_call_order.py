"""Calls right behind one another on a stream and in a graph: kernels that were
launched while the one before still runs read what it writes.  Lengths, tables
and queries come from the page calls or the staging copy; every result has to be
the one of the same calls with the stream idle in between."""

import numpy as np
import pytest
import torch

from gpu_cases import prepare
from top_sparse_attention_pks_gb300 import build, pks
from top_sparse_attention_pks_gb300.decoder import (MlaAttention, MlaDecodeStep, PageTable,
                                                    PrefixAttention, SparseDecodeStep)
from top_sparse_attention_pks_gb300.workloads import (MLA_WORKLOADS, WORKLOADS, draw_host,
                                                      draw_mla_tensors)

pytestmark = pytest.mark.gpu

REPEATS = 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def dev(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def doubled(t, *names):
    for name in names:
        t[name] = torch.cat([t[name], t[name].flip(0)])
    return [t[name] for name in names]


class Table:
    """The worked example's requests (61 of 64 pages) with as many empty rows behind
    them and pools of twice the pages (`doubled`), so that all rows can grow; its
    state put back by `reset` (plain copies, which wait for everything before them)."""

    def __init__(self, wl, t, pools):
        rows = 2 * wl.B
        self.rows, self.B = rows, wl.B
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.lens[: wl.B] = t["seq_lens"]
        self.table = torch.full((rows, wl.max_pages), -1, dtype=torch.int32, device="cuda")
        self.table[: wl.B] = t["block_table"]
        self.pages = PageTable(self.lens, self.table, 2 * wl.num_pages, wl.page_size, pools=pools)
        self.mine = [self.lens, self.table, self.pages.state] + list(pools)
        self.saved = [x.clone() for x in self.mine]
        full = int(self.lens.max())
        add = torch.full((rows,), 2, dtype=torch.int32, device="cuda")
        add[wl.B:] = 5
        src, dst = dev(range(wl.B)), dev(range(wl.B, rows))
        some, keep = dev([0, 2, 4]), dev([full // 2, 0, 7])
        self.calls = {
            "extend": lambda: self.pages.extend(add),
            "fork": lambda: self.pages.fork(src, dst),
            "free": lambda: self.pages.free(some, keep),
            "fork_extend_free": lambda: (self.pages.fork(src, dst), self.pages.extend(add),
                                         self.pages.free(some)),
            "compact": lambda: (self.pages.free(some, keep), self.pages.compact()),
        }

    def reset(self):
        for x, was in zip(self.mine, self.saved):
            x.copy_(was)


def check(table, name, step, results, idle=None):
    """`step` behind the page call against `step` on an idle device, eager and in a
    graph; `idle`: what it needs to know of the tables after the call."""
    call = table.calls[name]
    table.reset()
    call()
    torch.cuda.synchronize()
    if idle:
        idle()
        torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    want = [r.clone() for r in results()]
    assert table.pages.device_error() == 0

    def compare(what):
        torch.cuda.synchronize()
        for got, w in zip(results(), want):
            assert torch.equal(got, w), f"{what}: {name}"
        for r in results():
            r.fill_(0)

    for i in range(REPEATS):
        table.reset()
        if i % 2:
            torch.cuda.synchronize()
        call()
        step()
        compare(f"eager {i}")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        table.reset()
        call()
        step()
    for i in range(REPEATS):
        g.replay()
        compare(f"replay {i}")


CALLS = ["extend", "fork", "free", "fork_extend_free", "compact"]


def mla_tensors():
    wl = MLA_WORKLOADS["mla_paging_example"]
    h = draw_host(wl)
    pool = pks.Pool(wl.num_pages, wl.page_size, h["free_order"])
    bt, _ = pool.build_block_table(h["seq_lens"], wl.max_pages, h["prefix_group"], wl.prefix_len)
    pool.close()
    t = draw_mla_tensors(wl, "cuda")
    t["seq_lens"], t["block_table"] = h["seq_lens"].cuda(), torch.from_numpy(bt).cuda()
    return wl, t


def last_tokens(lens, idx):
    """Each row's last min(k, len) tokens, -1 after them (none behind `lens`)."""
    k = idx.shape[1]
    n = lens.clamp(max=k)[:, None]
    j = torch.arange(k, device="cuda")[None, :]
    idx.copy_(torch.where(j < n, lens[:, None] - 1 - j, -1))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("splits,trim", [(1, True), (2, False)])
def test_mla_behind_page_calls(name, splits, trim):
    wl, t = mla_tensors()
    tab = Table(wl, t, doubled(t, "kv"))
    q = t["q"].repeat(2, 1, 1).contiguous()
    idx = torch.full((tab.rows, wl.k), -1, dtype=torch.int32, device="cuda")
    att = MlaAttention(tab.lens, tab.table, idx, q, t["kv"], trim=trim, splits=splits)
    check(tab, name, att, lambda: [att.out], lambda: last_tokens(tab.lens, idx))
    assert att.device_error() == 0


@pytest.mark.parametrize("name", CALLS)
def test_mla_step_behind_page_calls(name):
    wl, t = mla_tensors()
    tab = Table(wl, t, doubled(t, "kv", "idx_k"))
    t.update(seq_lens=tab.lens, block_table=tab.table, q=t["q"].repeat(2, 1, 1).contiguous(),
             q_idx=t["q_idx"].repeat(2, 1, 1).contiguous())
    step = MlaDecodeStep(t, wl.k)
    check(tab, name, step, lambda: [step.out, step.topk_idx])


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("topk_mode", [0, 1])
def test_sparse_step_behind_page_calls(name, topk_mode):
    wl = WORKLOADS["paging_example"]
    t, _, _ = prepare(wl)
    tab = Table(wl, t, doubled(t, "kv_k", "kv_v", "idx_k"))
    t.update(seq_lens=tab.lens, block_table=tab.table, q=t["q"].repeat(2, 1, 1).contiguous(),
             q_idx=t["q_idx"].repeat(2, 1, 1).contiguous())
    step = SparseDecodeStep(t, wl.k, topk_mode=topk_mode)
    check(tab, name, step, lambda: [step.out, step.topk_idx])
    # the attention alone, over each row's last tokens
    check(tab, name, step.attention_only, lambda: [step.out],
          lambda: last_tokens(tab.lens, step.topk_idx))
    assert step.device_error() == 0


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("Nq", [1, 5])
def test_prefix_attention_behind_page_calls(name, Nq):
    wl = WORKLOADS["paging_example"]
    t, _, _ = prepare(wl)
    tab = Table(wl, t, doubled(t, "kv_k", "kv_v"))
    q = torch.randn((tab.rows, Nq, wl.Hq, wl.D), device="cuda").to(torch.bfloat16)
    group = dev(list(range(wl.B)) * 2)
    att = PrefixAttention(tab.lens, tab.table, q, t["kv_k"], t["kv_v"], prefix_group=group,
                          causal=True, lse=True, min_shared=16)
    check(tab, name, att, lambda: [att.out, att.lse])
    assert att.device_error() == 0


def test_attention_behind_the_staging_copy():
    """Queries, lengths and lists staged in from the host right in front."""
    wl, t = mla_tensors()
    sets = []
    for s in range(2):
        lens = (t["seq_lens"] - 13 * s).cpu()
        idx = torch.full((wl.B, wl.k), -1, dtype=torch.int32, device="cuda")
        last_tokens(lens.cuda(), idx)
        sets.append([x.cpu().pin_memory() for x in (t["q"] * (1 + s), lens, idx)])
    q, lens = t["q"].clone(), t["seq_lens"].clone()
    idx = torch.empty((wl.B, wl.k), dtype=torch.int32, device="cuda")
    att = MlaAttention(lens, t["block_table"], idx, q, t["kv"], trim=True)
    want = []
    for s in sets:
        pks.pks_stage_copy(list(zip((q, lens, idx), s)))
        torch.cuda.synchronize()
        want.append(att().clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    for i in range(2 * REPEATS):
        pks.pks_stage_copy(list(zip((q, lens, idx), sets[i % 2])))
        att()
        torch.cuda.synchronize()
        assert torch.equal(att.out, want[i % 2]), i
    assert att.device_error() == 0


def test_mla_step_behind_the_staging_copy():
    """The step in one call, its queries and lengths staged in right in front: as
    the two calls on an idle device."""
    wl, t = mla_tensors()
    names = ("q", "q_idx", "seq_lens")
    sets = [[t[n].cpu().pin_memory() for n in names],
            [x.cpu().pin_memory() for x in (t["q"] * 2, t["q_idx"] // 2, t["seq_lens"] - 13)]]
    step = MlaDecodeStep(t, wl.k)
    want = []
    for s in sets:
        pks.pks_stage_copy(list(zip((t[n] for n in names), s)))
        torch.cuda.synchronize()
        step.select()
        torch.cuda.synchronize()
        step.attention()
        torch.cuda.synchronize()
        want.append((step.out.clone(), step.topk_idx.clone()))
    assert not torch.equal(want[0][0], want[1][0])
    g = []
    for s in sets:
        g.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(g[-1]):
            pks.pks_stage_copy(list(zip((t[n] for n in names), s)))
            step()
    for i in range(4 * REPEATS):
        if i < 2 * REPEATS:
            pks.pks_stage_copy(list(zip((t[n] for n in names), sets[i % 2])))
            step()
        else:
            g[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want[i % 2][0]) and torch.equal(step.topk_idx, want[i % 2][1])
        step.out.fill_(0)
    assert step.attention.device_error() == 0
