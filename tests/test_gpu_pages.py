"""The page table on the device against sequential code: tables, lengths, holder
counts, free pages and the pools' contents have to be equal after every call."""

import numpy as np
import pytest
import torch

from pages_reference import PagesReference, pages_of
from top_sparse_attention_pks_gb300 import build, pks
from top_sparse_attention_pks_gb300.decoder import PageTable, SparseDecodeStep
from top_sparse_attention_pks_gb300.workloads import WORKLOADS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def dev(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


class Both:
    """The same calls on the device and on the reference, compared after each."""

    def __init__(self, lens, table, num_pages, page_size, pools):
        self.ref = PagesReference(lens, table, num_pages, page_size,
                                  [p.cpu().numpy() for p in pools])
        self.lens, self.table, self.pools = dev(lens), dev(table), pools
        self.pages = PageTable(self.lens, self.table, num_pages, page_size, pools=pools)
        self.compare("init")

    def compare(self, what):
        torch.cuda.synchronize()
        r = self.ref
        assert self.pages.device_error() == r.error, what
        r.error = 0
        assert (self.lens.cpu().numpy() == r.lens).all(), what
        assert (self.table.cpu().numpy() == r.table).all(), what
        assert (self.pages.refs.cpu().numpy() == r.ref).all(), what
        assert int(self.pages.n_free) == r.n_free(), what
        off = pks.pks_pages_offsets(r.N)["free_map"]
        words = self.pages.state[off: off + 4 * -(-r.N // 32)].cpu().numpy()
        bits = np.unpackbits(words, bitorder="little")[: r.N]
        assert (bits == (r.ref == 0)).all(), what
        for got, want in zip(self.pools, r.pools):
            assert (got.cpu().numpy() == want).all(), what

    def fork(self, src, dst, tokens=None):
        self.pages.fork(dev(src), dev(dst), None if tokens is None else dev(tokens))
        self.ref.fork(list(src), list(dst), tokens)
        self.compare(f"fork {src} {dst} {tokens}")

    def extend(self, add):
        self.pages.extend(dev(add))
        granted = self.ref.extend(list(add))
        assert int(self.pages.granted) == int(granted)
        self.compare(f"extend {list(add)[:8]}")
        return granted

    def free(self, rows, keep=None):
        self.pages.free(dev(rows), None if keep is None else dev(keep))
        self.ref.free(list(rows), keep)
        self.compare(f"free {rows} {keep}")

    def compact(self):
        got = self.pages.compact()
        want = self.ref.compact()
        self.compare("compact")
        assert (got.cpu().numpy() == want).all()


def pools_for(num_pages, page_size, kinds):
    g = torch.Generator().manual_seed(num_pages)
    out = []
    for kind in kinds:
        shape = (num_pages, page_size) + {"kv": (2, 64), "idx": (64,), "odd": (3,), "word": (5,),
                                          "wide": (8, 128)}[kind]
        t = torch.randint(-100, 100, shape, generator=g)
        t = t.to({"odd": torch.int8, "idx": torch.int8, "word": torch.int32}.get(kind, torch.float16))
        out.append(t.cuda())
    return out


def start(rng, B, page_size, num_pages, max_pages, fill, kinds=("kv", "idx")):
    """Rows of random lengths on randomly dealt pages; `fill` of the rows hold something."""
    lens = np.where(rng.random(B) < fill, rng.integers(0, max_pages * page_size // 2 + 1, B), 0)
    need = [pages_of(int(n), page_size) for n in lens]
    while sum(need) > num_pages * 0.7:
        lens = lens // 2
        need = [pages_of(int(n), page_size) for n in lens]
    deal = rng.permutation(num_pages)
    table = np.full((B, max_pages), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = deal[at:at + n]
        at += n
    return Both(lens, table, num_pages, page_size, pools_for(num_pages, page_size, kinds))


@pytest.mark.parametrize("page_size,num_pages,max_pages,B,kinds", [
    (16, 300, 32, 12, ("kv", "idx")),
    (1, 500, 100, 7, ("kv", "odd")),
    (3, 65, 9, 20, ("word",)),
    (17, 1000, 20, 40, ("odd", "word", "idx", "kv")),
    (64, 40, 8, 5, ()),
    (128, 31, 4, 9, ("wide",)),
])
def test_random_sequences(page_size, num_pages, max_pages, B, kinds):
    rng = np.random.default_rng(page_size * 1000 + B)
    t = start(rng, B, page_size, num_pages, max_pages, 0.5, kinds)
    for step in range(25):
        kind = rng.integers(0, 4)
        if kind == 0:
            empty = np.nonzero(t.ref.lens == 0)[0]
            held = np.nonzero(t.ref.lens > 0)[0]
            if len(empty) and len(held):
                n = rng.integers(1, len(empty) + 1)
                src = rng.choice(held, n)
                tokens = [int(rng.integers(-1, t.ref.lens[s] + 1)) for s in src]
                t.fork(src, rng.permutation(empty)[:n], tokens if rng.random() < 0.6 else None)
        elif kind == 1:
            add = rng.integers(0, 2 * page_size + 1, B) * (rng.random(B) < 0.7)
            t.extend(np.minimum(add, t.ref.max_len - t.ref.lens))
        elif kind == 2:
            n = rng.integers(1, max(2, B // 3))
            rows = rng.permutation(B)[:n]
            keep = [int(rng.integers(0, t.ref.lens[r] + 1)) for r in rows]
            t.free(rows, keep if rng.random() < 0.7 else None)
        else:
            t.compact()


def test_extend_copies_shared_pages_once_per_extra_holder():
    """Five rows on one prompt of 20 tokens in 8-token pages: all grow (the last
    keeps the page), then a fork grows alone, then none shares a partial page."""
    table = np.full((8, 10), -1)
    table[0, :3] = [7, 3, 5]
    t = Both([20] + [0] * 7, table, 40, 8, pools_for(40, 8, ("kv",)))
    t.fork([0, 0, 0, 0], [1, 2, 3, 4])
    t.extend([1] * 5 + [0] * 3)
    assert len({int(t.ref.table[b, 2]) for b in range(5)}) == 5
    assert t.ref.table[4, 2] == 5, "the highest of the growing holders keeps the page"
    t.fork([2], [6])
    t.extend([0, 0, 0, 0, 0, 0, 9, 0])
    assert t.ref.table[6, 2] != t.ref.table[2, 2]
    before = t.ref.n_free()
    t.extend([3, 0, 0, 0, 0, 0, 0, 0])
    assert t.ref.n_free() == before, "a page of its own grows in place"
    t.fork([3], [7], [16])  # whole pages only: nothing to copy
    t.extend([0] * 7 + [1])
    assert t.ref.n_free() == before - 1


def test_out_of_pages_changes_nothing():
    table = np.full((3, 8), -1)
    table[0, :2], table[1, :1] = [0, 1], [2]
    t = Both([7, 3, 0], table, 6, 4, pools_for(6, 4, ("kv",)))
    assert not t.extend([9, 4, 1])  # needs 2 + 1 + 1 of 3 free pages
    assert t.extend([9, 4, 0])
    assert not t.extend([0, 0, 1])
    assert t.extend([0, 1, 0])  # grows in place
    t.free([1])
    assert t.extend([0, 0, 4])


def test_refused_rows():
    table = np.full((6, 4), -1)
    table[0, :2], table[1, :3] = [4, 2], [7, 1, 0]
    t = Both([5, 12, 0, 0, 0, 0], table, 12, 4, pools_for(12, 4, ("odd",)))
    t.fork([0, 0], [2, 2])       # a destination twice: the first counts
    t.fork([0], [1])             # not empty
    t.fork([0, 3], [3, 4])       # row 3 on both sides: neither
    t.fork([0, 0], [6, -1])      # out of range
    t.fork([0], [3], [6])        # more than the source holds
    t.fork([0], [0])
    t.fork([5], [3])             # an empty source gives an empty row
    t.free([1, 1], [9, 2])       # a row twice: the first counts
    t.free([0], [6])
    t.free([0], [-1])
    t.free([7], [0])
    assert not t.extend([12, 0, 0, 0, 0, 0])   # past max_pages * page_size
    assert not t.extend([0, -1, 0, 0, 0, 0])
    t.extend([0] * 6)
    t.fork([1], [4], [0])


def test_bad_pages_are_flagged_and_not_followed():
    lens, table = dev([9, 4, 0]), dev([[1, 99, 2, -5], [3, -1, -1, -1], [-1] * 4])
    pool = pools_for(8, 4, ("kv",))
    pg = PageTable(lens, table, 8, 4, pools=pool)
    assert pg.device_error() == 1
    assert pg.refs.cpu().tolist() == [0, 1, 1, 1, 0, 0, 0, 0]
    pg.fork(dev([0]), dev([2]))
    assert pg.device_error() == 1 and int(lens[2]) == 0
    pg.free(dev([0]))
    assert pg.device_error() == 1
    assert pg.refs.cpu().tolist() == [0, 0, 0, 1, 0, 0, 0, 0] and int(pg.n_free) == 7
    bad = dev([500, -3])
    pg2 = PageTable(bad, dev([[0, 1], [2, 3]]), 8, 4)
    assert pg2.device_error() == 3 and int(pg2.n_free) == 8


def test_large_table_many_rows():
    """4096 rows; more bitmap words than the planning block has threads."""
    rng = np.random.default_rng(5)
    num_pages, B = 140_000, 4096
    lens = rng.integers(0, 400, B)
    table = np.full((B, 64), -1)
    deal, at = rng.permutation(num_pages), 0
    for b, n in enumerate(lens):
        k = pages_of(int(n), 16)
        table[b, :k] = deal[at:at + k]
        at += k
    t = Both(lens, table, num_pages, 16, pools_for(num_pages, 16, ("odd",)))
    t.extend(rng.integers(0, 300, B))
    t.free(rng.permutation(B)[:3000], None)
    spare = np.nonzero(t.ref.lens == 0)[0]
    held = np.nonzero(t.ref.lens)[0]
    t.fork(rng.choice(held, len(spare) - 1), spare[:-1])
    t.extend(np.ones(B, int))
    t.compact()
    t.compact()  # nothing left to move


def test_needs_past_32_bits_are_refused():
    """2100 rows that ask for 2^20 pages each: 2.2e9 pages, more than an int holds."""
    rows, width = 2100, 1 << 20
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    table = torch.empty((rows, width), dtype=torch.int32, device="cuda")
    pg = PageTable(lens, table, 1000, 1)
    pg.extend(torch.full((rows,), width, dtype=torch.int32, device="cuda"))
    assert pg.device_error() == 6
    assert int(pg.granted) == 0 and int(pg.n_free) == 1000 and not lens.any()
    assert not pg.refs.any()
    pg.extend(dev(np.arange(rows) < 1000))
    assert pg.device_error() == 0 and int(pg.n_free) == 0


def test_tensors_elsewhere_are_refused():
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        PageTable(lens, table.cuda(), 4, 2)
    with pytest.raises(ValueError):
        PageTable(lens.cuda(), table.cuda(), 4, 2, pools=[torch.zeros(4, 2, 8)])


def test_empty_calls_and_full_pool():
    t = start(np.random.default_rng(3), 4, 16, 64, 8, 1.0)
    t.fork([], [])
    t.free([])
    pg = PageTable(dev(np.zeros(0)), dev(np.zeros((0, 3))), 5, 4)
    pg.extend(dev(np.zeros(0)))
    pg.compact()
    assert pg.device_error() == 0 and int(pg.n_free) == 5
    one = Both([0], [[-1]], 1, 1, pools_for(1, 1, ("odd",)))
    one.extend([1])
    assert not one.extend([1])
    one.compact()
    one.free([0])
    one.compact()


def test_captured_and_replayed():
    """fork, extend and free in one CUDA graph: each replay works on the tables
    as they stand."""
    table = np.full((4, 16), -1)
    table[0, :2] = [9, 4]
    t = Both([20, 0, 0, 0], table, 64, 16, pools_for(64, 16, ("kv", "odd")))
    src, dst, add, drop = dev([0, 0]), dev([1, 2]), dev([5, 3, 17, 0]), dev([1, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t.pages.fork(src, dst)
        t.pages.extend(add)
        t.pages.free(drop)
        t.pages.compact()
    for _ in range(4):
        g.replay()
        t.ref.fork([0, 0], [1, 2])
        t.ref.extend([5, 3, 17, 0])
        t.ref.free([1, 2])
        t.ref.compact()
        t.compare("replay")


def test_two_tables_on_two_streams():
    rng = np.random.default_rng(11)
    tabs = [start(rng, 30, 16, 600, 30, 0.6) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    adds = [dev(rng.integers(0, 20, 30)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for t, s, a in zip(tabs, streams, adds):
            t.pages.extend(a, stream=s)
            t.pages.compact(stream=s)
    torch.cuda.synchronize()
    for t, a in zip(tabs, adds):
        for _ in range(5):
            t.ref.extend(a.cpu().numpy())
            t.ref.compact()
        t.compare("two streams")


def test_table_feeds_the_decode_step():
    """Rows forked, freed and compacted between decode steps: the sparse decode
    step selects and attends as the oracle does, a fork selects what its source
    selects, and compaction changes no bit of a step (the work is split over the
    CTAs by the lengths alone)."""
    from gpu_cases import check_attention, oracle_attention, oracle_topk, prepare
    wl = WORKLOADS["paging_example"]
    t, _, _ = prepare(wl)
    rows = 2 * wl.B
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    lens[: wl.B] = t["seq_lens"]
    table = torch.full((rows, wl.max_pages), -1, dtype=torch.int32, device="cuda")
    table[: wl.B] = t["block_table"]
    t.update(seq_lens=lens, block_table=table, q=t["q"].repeat(2, 1, 1).contiguous(),
             q_idx=t["q_idx"].repeat(2, 1, 1).contiguous())
    pages = PageTable(lens, table, wl.num_pages, wl.page_size,
                      pools=[t["kv_k"], t["kv_v"], t["idx_k"]])
    pages.fork(dev(range(wl.B)), dev(range(wl.B, rows)))
    out, idx = SparseDecodeStep(t, wl.k)()
    want = oracle_topk(wl, t)[1]
    assert (idx.cpu().numpy() == want).all()
    assert (want[wl.B:] == want[: wl.B]).all()
    check_attention(out, oracle_attention(wl, t, want), "forked")
    pages.free(dev([0, 2]))     # the forks hold their pages now
    assert int(pages.n_free) == wl.num_pages - 61
    pages.free(dev([1]))
    pages.free(dev([6]))        # request 1 and its fork: six pages
    assert int(pages.n_free) == wl.num_pages - 61 + 6
    before = {k: v.clone() for k, v in t.items()}
    pages.compact()
    assert int(table.max()) < 61 - 6 <= int(before["block_table"].max())
    step = SparseDecodeStep(t, wl.k)
    out, idx = step()
    out0, idx0 = SparseDecodeStep(before, wl.k)()
    assert torch.equal(out, out0) and torch.equal(idx, idx0)
    assert step.device_error() == 0 and pages.device_error() == 0


def test_arguments_elsewhere_are_refused(monkeypatch):
    """Arguments on the host, and calls while another device is the current one."""
    lens, table = dev([20, 0, 0]), dev([[0, 1, -1], [-1] * 3, [-1] * 3])
    pages = PageTable(lens, table, 6, 16)
    rows = torch.tensor([1], dtype=torch.int32)
    calls = [lambda r: pages.fork(dev([0]), r), lambda r: pages.fork(r, dev([1])),
             lambda r: pages.fork(dev([0]), dev([1]), r), lambda r: pages.free(r),
             lambda r: pages.free(dev([0]), r),
             lambda r: pages.extend(torch.cat([r, r, r]))]
    for call in calls:
        with pytest.raises(ValueError):
            call(rows)
    with pytest.raises(ValueError):
        PageTable(lens.cpu(), table, 6, 16)
    here = rows.cuda()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for call in [lambda: pages.free(here), lambda: pages.fork(here, here), pages.compact,
                     lambda: pages.extend(lens)]:
            with pytest.raises(ValueError):
                call()
    assert pages.device_error() == 0 and int(pages.n_free) == 4


def test_states_of_other_pages_are_refused():
    """A state that was not filled, or for other pages, changes nothing."""
    lens, table = dev([20, 0, 5]), dev([[0, 1, -1], [-1] * 3, [2, -1, -1]])
    pool = torch.arange(8 * 16, dtype=torch.int32, device="cuda").view(8, 16, 1)
    size = pks.pks_pages_state_bytes(8)
    for fill in (0, 7):
        state = torch.zeros(size, dtype=torch.uint8, device="cuda")
        full = pks.make_pages_args(seq_lens=lens, block_table=table, num_pages=8, page_size=16,
                                   state=state, pools=[pool])
        if fill:  # for seven pages
            pks.pks_pages_init(pks.make_pages_args(seq_lens=lens, block_table=table, num_pages=7,
                                                   page_size=16, state=state))
        before = [x.clone() for x in (lens, table, pool)]
        calls = [lambda: pks.pks_pages_fork(full, dev([0]), dev([1])),
                 lambda: pks.pks_pages_free(full, dev([0])),
                 lambda: pks.pks_pages_extend(full, dev([1, 1, 30])),
                 lambda: pks.pks_pages_compact(full)]
        for call in calls:
            call()
            assert pks.pks_pages_device_error(full) == 4
        for was, x in zip(before, (lens, table, pool)):
            assert torch.equal(was, x)


def test_fewer_free_pages_than_counted():
    lens, table = dev([20, 0, 5]), dev([[0, 1, -1], [-1] * 3, [2, -1, -1]])
    pages = PageTable(lens, table, 8, 16)
    pages.n_free.fill_(7)  # five are free
    pages.extend(dev([28, 48, 43]))  # six pages
    assert int(pages.granted) == 0 and pages.device_error() == 4
    assert lens.tolist() == [20, 0, 5]
    assert table.tolist() == [[0, 1, -1], [-1] * 3, [2, -1, -1]]


@pytest.mark.parametrize("entry", [-1, -2, 6, 2 ** 31 - 1])
def test_free_flags_any_bad_entry(entry):
    lens, table = dev([40, 0]), dev([[0, 1, 2], [-1] * 3])
    pages = PageTable(lens, table, 6, 16)
    table[0, 1] = entry
    pages.free(dev([0]))
    assert pages.device_error() == 1
    assert lens.tolist() == [0, 0] and int(table.max()) == -1
    assert pages.refs.tolist() == [0, 1, 0, 0, 0, 0] and int(pages.n_free) == 5


def _bitmap(pages):
    off = pks.pks_pages_offsets(pages.refs.numel())["free_map"]
    return pages.state[off: off + 4 * -(-pages.refs.numel() // 32)].clone()


@pytest.mark.parametrize("num_pages,held", [(8, 3), (3000, 5), (140_000, 9)])
def test_extend_with_fewer_free_pages_than_counted_takes_none(num_pages, held):
    """The pages that are free stay so: growth that fits them is granted afterwards."""
    B, width = 64, held + -(-num_pages // 64) + 2
    table = np.full((B, width), -1)
    table[0, :held] = np.random.default_rng(num_pages).permutation(num_pages)[:held]
    lens, table = dev([16 * held] + [0] * (B - 1)), dev(table)
    pages = PageTable(lens, table, num_pages, 16)
    before = [x.clone() for x in (lens, table, pages.refs)] + [_bitmap(pages)]
    pages.n_free.fill_(num_pages - 1)
    need = np.full(B, (num_pages - held + 1) // B)
    need[: (num_pages - held + 1) % B] += 1  # one page more than there are
    pages.extend(dev(16 * need))
    assert int(pages.granted) == 0 and pages.device_error() == 4
    for was, x in zip(before, [lens, table, pages.refs, _bitmap(pages)]):
        assert torch.equal(was, x)
    pages.n_free.fill_(num_pages - held)
    need[0] -= 1
    pages.extend(dev(16 * need))
    assert int(pages.granted) == 1 and pages.device_error() == 0
    assert int(pages.n_free) == 0 and bool((pages.refs == 1).all())
    assert not _bitmap(pages).any()


@pytest.mark.parametrize("counted", [7, 4, 8, 9, -1, 0, 2 ** 31 - 1, -2 ** 31])
def test_compact_with_another_count_of_free_pages_changes_nothing(counted):
    """Three of eight pages are held, two of them at or above the third."""
    lens, table = dev([20, 0, 5]), dev([[0, 6, -1], [-1] * 3, [7, -1, -1]])
    pool = torch.arange(8 * 16 * 3, dtype=torch.int32, device="cuda").view(8, 16, 3)
    pages = PageTable(lens, table, 8, 16, pools=[pool])
    mine = [lens, table, pages.refs, pool, pages.page_map]
    pages.page_map.fill_(-9)
    before = [x.clone() for x in mine] + [_bitmap(pages)]
    pages.n_free.fill_(counted)
    pages.compact()
    assert pages.device_error() == 4 and int(pages.n_free) == counted
    for was, x in zip(before, mine + [_bitmap(pages)]):
        assert torch.equal(was, x)
    pages.n_free.fill_(5)
    assert pages.compact().tolist() == [0, -1, -1, -1, -1, -1, 1, 2]
    assert pages.device_error() == 0 and table[[0, 2]].tolist() == [[0, 1, -1], [2, -1, -1]]
    assert pages.refs.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
