"""The decode step over a 4-bit cache, and a decode loop: rows forked, grown, written and
attended over, call behind call and in a graph."""

import numpy as np
import pytest
import torch

from gpu_cases import oracle_topk, prepare
from q4_cases import Batch, i32
from top_sparse_attention_pks_gb300 import build
from top_sparse_attention_pks_gb300.decoder import (PageTable, Q4Attention, Q4Cache, Q4DecodeStep,
                                                    Q4SparseAttention, SparseDecodeStep)
from top_sparse_attention_pks_gb300.workloads import WORKLOADS, draw_float_weights, draw_fp8_indexer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


class Case(Batch):
    """The worked example with its K/V rows in a 4-bit cache."""

    def __init__(self, wl, nq=1, seed=3):
        super().__init__([int(n) for n in wl.seq_lens], wl.page_size, wl.Hkv, wl.Hq // wl.Hkv,
                         wl.D, nq, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        N, B = self.cache.k.shape[0], len(self.lens)
        self.t = dict(
            seq_lens=self.len_d, block_table=torch.where(self.table < 0, -1, self.table),
            q=self.q if nq > 1 else self.q[:, 0].contiguous(),
            q_idx=torch.randint(-127, 128, (B, nq, wl.Hi, wl.Di), dtype=torch.int8, device="cuda",
                                generator=g),
            w_idx=torch.ones(wl.Hi, dtype=torch.int32, device="cuda"),
            idx_k=torch.randint(-127, 128, (N, wl.page_size, wl.Di), dtype=torch.int8,
                                device="cuda", generator=g))
        if nq == 1:
            self.t["q_idx"] = self.t["q_idx"][:, 0].contiguous()


@pytest.mark.parametrize("nq,hi,mode", [(1, 1, 0), (1, 4, 1), (4, 1, 0), (2, 2, 1)])
def test_step(nq, hi, mode):
    wl = WORKLOADS["paging_example"].replace(Hi=hi)
    c = Case(wl, nq)
    step = Q4DecodeStep(c.t, c.cache, wl.k, topk_mode=mode, lse=True)
    out, idx = step()
    torch.cuda.synchronize()
    assert step.device_error() == 0
    # the selection: that of the step over 16-bit pools
    kv = torch.zeros((c.cache.k.shape[0], c.P, c.Hkv, c.D), dtype=torch.bfloat16, device="cuda")
    _, want = SparseDecodeStep(dict(c.t, kv_k=kv, kv_v=kv), wl.k, topk_mode=mode)()
    assert torch.equal(idx, want)
    lists = idx.cpu().numpy().reshape(len(c.lens), nq, wl.k)
    c.check(out.view(c.q.shape), step.lse.view(c.q.shape[:-1]), lists=lists)
    # the same bits as the two calls
    first = out.clone()
    assert torch.equal(step.select(), want)
    att = Q4SparseAttention(c.len_d, c.t["block_table"], idx, c.t["q"], c.cache, trim=True)
    assert torch.equal(att(), first)


@pytest.mark.parametrize("fp8", [None, torch.int8, torch.float8_e4m3fn])
def test_step_with_real_weights_and_fp8(fp8):
    wl = WORKLOADS["b32_4k"].replace(B=4, seq_lens=(4096, 700, 0, 1500))
    t, _, _ = prepare(wl)
    t["w_idx_f"] = draw_float_weights(wl, "cuda", signed=True)
    if fp8 is not None:
        t["q_idx"], t["idx_k"] = (x.view(fp8) for x in draw_fp8_indexer(wl, "cuda"))
        t["idx_fp8"] = True
    _, want = SparseDecodeStep(t, wl.k)()
    cache = Q4Cache(wl.num_pages, wl.page_size, wl.Hkv, wl.D)
    lens = [int(n) for n in wl.seq_lens]
    starts = i32(np.concatenate([[0], np.cumsum(lens)]))
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((sum(lens), wl.Hkv, wl.D), generator=g, device="cuda") for _ in range(2))
    cache.write(k, v, t["seq_lens"], t["block_table"], starts)
    del t["kv_k"], t["kv_v"]
    step = Q4DecodeStep(t, cache, wl.k)
    out, idx = step()
    assert torch.equal(idx, want) and step.device_error() == 0
    att = Q4SparseAttention(t["seq_lens"], t["block_table"], want, t["q"], cache, trim=True)
    assert torch.equal(att(), out) and bool(out[0].any()) and not out[2].any()


@pytest.mark.parametrize("name", ["q_idx", "idx_k", "w_idx", "block_table"])
def test_step_refuses_tensors_on_the_host(name):
    wl = WORKLOADS["paging_example"]
    c = Case(wl)
    with pytest.raises(ValueError):
        Q4DecodeStep(dict(c.t, **{name: c.t[name].cpu()}), c.cache, wl.k)


def test_step_against_the_oracle():
    wl = WORKLOADS["b32_4k"].replace(B=4, seq_lens=(4096, 700, 0, 1500))
    t, _, _ = prepare(wl)
    cache = Q4Cache(wl.num_pages, wl.page_size, wl.Hkv, wl.D)
    lens = [int(n) for n in wl.seq_lens]
    starts = i32(np.concatenate([[0], np.cumsum(lens)]))
    rows = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((rows, wl.Hkv, wl.D), generator=g, device="cuda") for _ in range(2))
    cache.write(k, v, t["seq_lens"], t["block_table"], starts)
    step = Q4DecodeStep(t, cache, wl.k)
    out, idx = step()
    _, want = oracle_topk(wl, t)
    assert (idx.cpu().numpy() == want).all() and step.device_error() == 0
    att = Q4SparseAttention(t["seq_lens"], t["block_table"], i32(want), t["q"], cache, trim=True)
    assert torch.equal(att(), out) and not out[2].any()


class Loop:
    """Requests over prompts in a 4-bit cache; a step grows every row, writes the new tokens'
    K/V, a slice of one tensor, and attends over all tokens and over some."""

    def __init__(self, seed=0):
        self.P, self.Hkv, self.D, B = 16, 8, 128, 6
        N = 64
        lens = [70, 33, 5, 0, 0, 0]
        table = np.full((B, 12), -1, np.int64)
        deal = np.random.default_rng(seed).permutation(N)
        table[0, :5], table[1, :3], table[2, :1] = deal[:5], deal[5:8], deal[8:9]
        self.lens, self.table = i32(lens), i32(table)
        self.cache = Q4Cache(N, self.P, self.Hkv, self.D)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = torch.randn((2, 108, self.Hkv, self.D), generator=g, device="cuda")
        self.cache.write(rows[0], rows[1], self.lens, self.table,
                         i32([0, 70, 103, 108, 108, 108, 108]))
        self.pages = PageTable(self.lens, self.table, N, self.P,
                               pools=[self.cache.k, self.cache.v])
        self.add = i32([2] * B)
        self.starts = i32([2 * i for i in range(B + 1)])
        self.qkv = torch.randn((2 * B, 32 + 2 * self.Hkv, self.D), generator=g, device="cuda"
                               ).to(torch.bfloat16)
        q = torch.randn((B, 2, 32, self.D), generator=g, device="cuda").to(torch.bfloat16)
        self.list = i32(np.tile([0, 3, 1, -1, 4, 2], (B, 2, 1)))
        self.att = Q4Attention(self.lens, self.table, q, self.cache, causal=True, lse=True)
        self.sel = Q4SparseAttention(self.lens, self.table, self.list, q, self.cache, lse=True)
        self.pages.fork(i32([0, 1, 2]), i32([3, 4, 5]))
        torch.cuda.synchronize()
        self.mine = [self.lens, self.table, self.pages.state, self.cache.k, self.cache.v]
        self.saved = [x.clone() for x in self.mine]

    def reset(self):
        for x, was in zip(self.mine, self.saved):
            x.copy_(was)

    def step(self, wait=lambda: None):
        self.pages.extend(self.add)
        wait()
        self.cache.write(self.qkv[:, 32:32 + self.Hkv], self.qkv[:, 32 + self.Hkv:], self.lens,
                         self.table, self.starts)
        wait()
        self.att()
        wait()
        self.sel()
        wait()

    def results(self):
        return [self.att.out, self.att.lse, self.sel.out, self.sel.lse, self.cache.k, self.cache.v,
                self.lens, self.table]


def test_calls_right_behind_one_another():
    loop = Loop()
    for _ in range(3):
        loop.step(torch.cuda.synchronize)
    want = [x.clone() for x in loop.results()]
    assert loop.pages.device_error() == loop.cache.device_error() == 0
    assert loop.att.device_error() == loop.sel.device_error() == 0
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        loop.step()
    for _ in range(20):
        for go in (loop.step, graph.replay):
            loop.reset()
            for x in loop.results()[:4]:
                x.fill_(float("nan"))
            for _ in range(3):
                go()
            torch.cuda.synchronize()
            for got, w in zip(loop.results(), want):
                assert torch.equal(got, w)


def test_a_loop_gives_what_the_rows_say():
    """After the loop: forked rows differ from their sources only in what was written."""
    loop = Loop(1)
    for _ in range(2):
        loop.step()
    lens = [74, 37, 9] * 2
    assert loop.lens.tolist() == lens
    out = torch.empty((2, sum(lens), loop.Hkv, loop.D), device="cuda")
    starts = np.concatenate([[0], np.cumsum(lens)])
    loop.cache.read(loop.lens, loop.table, i32(starts), out[0], out[1])
    for b in range(3):
        n = lens[b] - 4
        src, dst = starts[b], starts[b + 3]
        assert torch.equal(out[:, src:src + n], out[:, dst:dst + n])
        assert not torch.equal(out[:, src + n:src + n + 4], out[:, dst + n:dst + n + 4])
