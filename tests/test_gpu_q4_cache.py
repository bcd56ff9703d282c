"""Writing a 4-bit cache and reading it back, against the definition in 64 bits:
codes, scales and minima are compared bit for bit, and what is read back as well: it is
m + s n rounded to fp32 (one fused operation) and from there to the rows' type."""

import numpy as np
import pytest
import torch

import q4_reference as ref
from top_sparse_attention_pks_gb300 import build, pks
from top_sparse_attention_pks_gb300.decoder import PageTable, Q4Cache

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def layout(lens, page, seed=0, spare=3):
    rng = np.random.default_rng(seed)
    pages = [-(-n // page) for n in lens]
    deal = rng.permutation(sum(pages) + spare)
    table = np.full((len(lens), max(pages + [1]) + 1), -9, np.int64)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = deal[at:at + n]
        at += n
    return table, len(deal)


def rows(n, Hkv, D, dtype, seed, fused=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((2, n, Hkv, D), generator=g, device="cuda")
    x = x * (torch.randn((2, 1, Hkv, D), generator=g, device="cuda") * 0.5).exp()
    x[0] += torch.randn((Hkv, D), generator=g, device="cuda")
    x = x.to(dtype)
    if not fused:
        return x[0].contiguous(), x[1].contiguous()
    qkv = torch.full((n, fused + 2 * Hkv, D), float("nan"), dtype=dtype, device="cuda")
    qkv[:, fused:fused + Hkv], qkv[:, fused + Hkv:] = x[0], x[1]
    return qkv[:, fused:fused + Hkv], qkv[:, fused + Hkv:]


def check(cache, k, v, lens, table, starts, before=None, skip=()):
    """Every row's codes and pairs; all other bytes as they were."""
    page = cache.k.shape[1]
    where = [w for w in ref.places(lens, table, starts, page) if w[0] not in skip]
    for kind, x, pool in (("k", k, cache.k), ("v", v, cache.v)):
        n, s, m = ref.unpack(pool.cpu().numpy(), cache.Hkv, cache.D, kind)
        if where:
            i, pg, sl = (np.array(c) for c in zip(*where))
            wn, ws, wm = ref.quantise(x.float().cpu().numpy()[i])
            np.testing.assert_array_equal(s[pg, sl], ws, err_msg=f"{kind} s")
            np.testing.assert_array_equal(m[pg, sl], wm, err_msg=f"{kind} m")
            np.testing.assert_array_equal(n[pg, sl], wn, err_msg=f"{kind} codes")
        if before is not None:
            keep = np.ones(pool.shape[:2], bool)
            for _, pg, sl in where:
                keep[pg, sl] = False
            now, was = pool.cpu().numpy(), before[kind]
            used = cache.Hkv * ref.record_bytes(cache.D)
            assert (now[keep] == was[keep]).all()
            if used < now.shape[2]:  # what fills a row up
                assert (now[..., used:] == was[..., used:]).all()


def check_read(cache, lens, table, starts, dtype, n_rows=None, skip=()):
    page, Hkv, D = cache.k.shape[1], cache.Hkv, cache.D
    n = starts[-1] if n_rows is None else n_rows
    out = torch.full((2, n, Hkv, D), 77.0, dtype=dtype, device="cuda")
    cache.read(i32(lens), i32(table), i32(starts), out[0], out[1])
    where = [w for w in ref.places(lens, table, starts, page) if w[0] not in skip]
    for j, (kind, pool) in enumerate((("k", cache.k), ("v", cache.v))):
        got = out[j].float().cpu().numpy().astype(np.float64)
        want = np.full((n, Hkv, D), 77.0)
        if where:
            i, pg, sl = (np.array(c) for c in zip(*where))
            x = ref.values(*(a[pg, sl] for a in
                             ref.unpack(pool.cpu().numpy(), Hkv, D, kind)))
            want[i] = torch.from_numpy(x.astype(np.float32)).to(dtype).double().numpy()
        np.testing.assert_array_equal(got, want, err_msg=kind)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("Hkv,D,page,fused", [
    (8, 128, 64, 0), (2, 64, 16, 8), (1, 64, 5, 0), (1, 128, 1, 1), (3, 64, 17, 0), (5, 128, 16, 3),
    (16, 64, 8, 0), (16, 128, 3, 0), (7, 64, 48, 1)])
def test_write_and_read(dtype, Hkv, D, page, fused):
    lens = [0, 1, 37, 200, 16, 5]
    new = [0, 1, 37, 9, 0, 3]
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    table, N = layout(lens, page)
    cache = Q4Cache(N, page, Hkv, D)
    for pool in (cache.k, cache.v):
        pool.copy_(torch.randint(0, 256, pool.shape, dtype=torch.uint8, device="cuda"))
    before = {"k": cache.k.cpu().numpy(), "v": cache.v.cpu().numpy()}
    k, v = rows(starts[-1], Hkv, D, TYPES[dtype], 3, fused)
    cache.write(k, v, i32(lens), i32(table), i32(starts))
    check(cache, k, v, lens, table, starts, before)
    check_read(cache, lens, table, starts, TYPES[dtype])
    assert cache.device_error() == 0


def test_rows_of_any_strides():
    """Heads before rows, one row for all, one head for all."""
    lens, starts = [40, 3], [0, 40, 43]
    table, N = layout(lens, 16, 9)
    cache = Q4Cache(N, 16, 4, 64)
    k, v = rows(43, 4, 64, torch.bfloat16, 10)
    for a, b in ((k.transpose(0, 1).contiguous().transpose(0, 1), v), (k[:1].expand(43, 4, 64), v),
                 (k, v[:, :1].expand(43, 4, 64))):
        cache.write(a, b, i32(lens), i32(table), i32(starts))
        check(cache, a, b, lens, table, starts)
    out = torch.full((2, 4, 43, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    got = cache.read(i32(lens), i32(table), i32(starts), *out.transpose(1, 2))
    same = torch.empty((2, 43, 4, 64), dtype=torch.bfloat16, device="cuda")
    want = cache.read(i32(lens), i32(table), i32(starts), *same)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    with pytest.raises(pks.PksError):
        cache.read(i32(lens), i32(table), i32(starts), k[:1].expand(43, 4, 64), v)
    assert cache.device_error() == 0


def test_prompts_of_many_rows():
    """More rows than blocks: blocks take eight rows at a time, more than once."""
    lens = [9000, 1, 4321, 0, 2777]
    starts = np.concatenate([[0], np.cumsum(lens)]).tolist()
    table, N = layout(lens, 16, 5)
    cache = Q4Cache(N, 16, 2, 64)
    k, v = rows(starts[-1], 2, 64, torch.bfloat16, 6)
    cache.write(k, v, i32(lens), i32(table), i32(starts))
    check(cache, k, v, lens, table, starts)
    check_read(cache, lens, table, starts, torch.bfloat16)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_groups_that_are_hard_to_round(dtype):
    """Equal values, values that halve a step, a mean far from 0, subnormal scales, fp16's
    ends, infinities and NaN."""
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(1)
    r = torch.randn((400, 1, 128), generator=g)
    x = torch.cat([
        torch.zeros(1, 1, 128), torch.full((1, 1, 128), -0.0), torch.full((1, 1, 128), 3.0),
        torch.arange(128).float().view(1, 1, 128), (torch.arange(128) % 31).float().view(1, 1, 128),
        (torch.arange(128) % 31 / 2 - 7).view(1, 1, 128), r[:40] * 0.01 + 100.0,
        r[40:80] * 1e-3 - 64.0, r[80:120] * 1e-7, r[120:160] * 3e-5, r[160:180] * 1e4,
        r[180:200] * 3e5, (r[200:300] * 8).round() / 8, (r[300:400] * 4).round() * 0.75]).to(t)
    x[-1, 0, 5], x[-2, 0, 40], x[-3, 0, 70] = float("nan"), float("inf"), -float("inf")
    x[-4, 0, 100:] = 65504.0
    x[-5, 0, :32] = -65504.0
    x[-6, 0, 3] = 1e-30
    x[-7, 0, 3] = -1e-30
    n = x.shape[0]
    x = x.cuda()
    lens, starts = [n], [0, n]
    table, N = layout(lens, 16)
    cache = Q4Cache(N, 16, 1, 128)
    y = x.flip(2).contiguous()
    cache.write(x, y, i32(lens), i32(table), i32(starts))
    check(cache, x, y, lens, table, starts)
    check_read(cache, lens, table, starts, torch.float32)


def test_a_value_is_rounded_to_fp32_and_from_there():
    """m + s n = 1.00390625 + 2^-24, which lies above the middle of two bf16 numbers: fp32 rounds
    it to that middle."""
    cache = Q4Cache(1, 16, 1, 64)
    x = torch.full((1, 1, 64), 2.0 ** -24, device="cuda")
    x[0, 0, 0], x[0, 0, 32] = 15 * 1.00390625, 1.00390625
    x[0, 0, 1] = x[0, 0, 33] = 1.00390625
    cache.write(x, x, i32([1]), i32([[0]]), i32([0, 1]))
    _, s, m = ref.unpack(cache.k.cpu().numpy(), 1, 64, "k")
    assert s[0, 0, 0, 0] == 1.00390625 and m[0, 0, 0, 0] == 2.0 ** -24
    for dtype, want in (("fp32", 1.00390625), ("fp16", 1.00390625), ("bf16", 1.0)):
        out = torch.empty((2, 1, 1, 64), dtype=TYPES[dtype], device="cuda")
        cache.read(i32([1]), i32([[0]]), i32([0, 1]), out[0], out[1])
        assert float(out[0, 0, 0, 1]) == float(out[1, 0, 0, 1]) == want


def border_rows(dtype, seed, n=600):
    """Rows of a group each whose minimum is small beside its scale, and whose values stand at
    the borders between two codes, rounded to the type, or next to them."""
    rng = np.random.default_rng(seed)
    m = (rng.integers(1024, 2048, n) * 2.0 ** rng.integers(-28, -12, n)).astype(np.float16)
    m[: n // 8] = rng.integers(1, 1024, n // 8) * 2.0 ** -24  # subnormal ones
    m[n // 8: n // 4] *= -1
    m = m.astype(np.float64)
    s = (rng.integers(1024, 2048, n) * 2.0 ** rng.integers(-14, -8, n)).astype(np.float64)
    top = m + 15 * s
    x = np.empty((n, 32))
    x[:, 0], x[:, 1] = m, top
    x[:, 2:] = (m[:, None] + (np.arange(30) // 2 + 0.5) * s[:, None])
    x = torch.from_numpy(x).to(torch.float32).to(dtype)
    bits = x.view(torch.int32 if dtype == torch.float32 else torch.int16)
    off = torch.from_numpy(rng.integers(-1, 2, (n, 32)))
    off[:, :2] = 0
    off[:, 2::2] = 0
    bits += off.to(bits.dtype)
    return x


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_values_at_the_borders_between_codes(dtype):
    """Minima whose last bits lie below the place of a border m + (n + 1/2) s in fp32."""
    t = TYPES[dtype]
    x = border_rows(t, 5)
    odd = torch.zeros((4, 32))
    odd[0, :30], odd[0, 30], odd[0, 31] = 2.0 ** -14 * (1 + 2.0 ** -10), 7.5 + 2.0 ** -14, 15.0
    odd[1, :30], odd[1, 30], odd[1, 31] = 0.0004887580871582031, 8.3984375, 19.375
    odd[2, :30], odd[2, 30], odd[2, 31] = 2.0 ** -24, 7.5, 15.0
    odd[3, :30], odd[3, 30], odd[3, 31] = -2.0 ** -24, 7.5, 15.0
    x = torch.cat([odd.to(t), x])
    x = x[: len(x) // 2 * 2].reshape(-1, 1, 64).cuda()
    n = x.shape[0]
    table, N = layout([n], 16)
    cache = Q4Cache(N, 16, 1, 64)
    y = x.flip(2).contiguous()
    cache.write(x, y, i32([n]), i32(table), i32([0, n]))
    check(cache, x, y, [n], table, [0, n])
    check_read(cache, [n], table, [0, n], torch.float32)


def test_padded_rows_and_rows_without_a_place():
    """Rows behind the last request, a page out of range, a length out of range and more rows
    than tokens: those rows are skipped, all others written; a read leaves theirs alone."""
    page, Hkv, D = 16, 2, 64
    lens = [20, 30, 40, 3, 10]
    new = [4, 20, 5, 5, 2]  # request 3 has three tokens only
    starts = (np.concatenate([[0], np.cumsum(new)]) + 2).tolist()  # rows 0 and 1 unused
    table, N = layout(lens, page)
    n_rows = starts[-1] + 7
    k, v = rows(n_rows, Hkv, D, torch.bfloat16, 8)
    for bad, code in (("none", 2), ("page", 1), ("length", 3)):
        cache = Q4Cache(N, page, Hkv, D)
        cache.k.fill_(255)
        cache.v.fill_(255)
        before = {"k": cache.k.cpu().numpy(), "v": cache.v.cpu().numpy()}
        tb, ln = table.copy(), list(lens)
        own_starts = list(starts)
        skip = set(range(starts[3], starts[3] + 2))
        if bad != "none":  # request 3's fault away
            ln[3], own = 5, 5
            tb[3, 0] = table[3, 0]
            skip = set()
        if bad == "page":
            tb[1, 1] = N + 3  # positions 16.. of request 1
            skip = {i for i, pg, _ in ref.places(ln, tb, own_starts, page) if pg == N + 3}
        if bad == "length":
            ln[4] = 10 ** 6
            skip = set(range(starts[4], starts[5]))
        cache.write(k, v, i32(ln), i32(tb), i32(own_starts))
        check(cache, k, v, ln, tb, own_starts, before, skip)
        assert cache.device_error() == code and cache.device_error() == 0
        check_read(cache, ln, tb, own_starts, torch.bfloat16, n_rows, skip)
        assert cache.device_error() == code


def test_starts_that_go_back_stay_inside():
    """Starts that are no starts skip rows; nothing outside the requests' tokens changes."""
    page, Hkv, D = 16, 2, 64
    lens = [40, 40, 40]
    table, N = layout(lens, page)
    k, v = rows(30, Hkv, D, torch.bfloat16, 9)
    for starts in ([0, 25, 10, 30], [5, 0, 40, 12], [-3, 10, 20, 30], [0, 10 ** 9, -10 ** 9, 30],
                   [0, 0, 0, 1000], [30, 20, 10, 0]):
        cache = Q4Cache(N, page, Hkv, D)
        cache.write(k, v, i32(lens), i32(table), i32(starts))
        held = np.zeros((N, page), bool)
        for b in range(3):
            for t in range(40):
                held[table[b, t // page], t % page] = True
        assert not cache.k.cpu().numpy()[~held].any()


def test_nothing_to_do():
    cache = Q4Cache(4, 16, 2, 64)
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache.write(k, k, i32([0]), i32([[0]]), i32([0, 0]))
    e = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache.write(k, k, e[:, 0], e, i32([0]))
    torch.cuda.synchronize()
    assert not cache.k.any() and not cache.v.any()


def test_in_a_graph_and_on_another_stream():
    """A captured write and read follow what lengths, table and rows hold at a replay."""
    lens = [33, 64]
    table, N = layout([80, 80], 16)
    cache = Q4Cache(N, 16, 8, 128)
    k, v = rows(6, 8, 128, torch.bfloat16, 1)
    d_lens, d_table, d_starts = i32(lens), i32(table), i32([0, 2, 6])
    out = torch.empty((2, 6, 8, 128), dtype=torch.bfloat16, device="cuda")
    cache.write(k, v, d_lens, d_table, d_starts)
    cache.read(d_lens, d_table, d_starts, out[0], out[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.write(k, v, d_lens, d_table, d_starts)
        cache.read(d_lens, d_table, d_starts, out[0], out[1])
    for step in range(3):
        k2, v2 = rows(6, 8, 128, torch.bfloat16, 10 + step)
        lens = [lens[0] + 2, lens[1] + 4]
        d_lens.copy_(i32(lens))
        k.copy_(k2)
        v.copy_(v2)
        graph.replay()
        torch.cuda.synchronize()
        check(cache, k, v, lens, table, [0, 2, 6])
        n, s, m = ref.quantise(k.float().cpu().numpy())
        want = torch.from_numpy(ref.values(n, s, m).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(out[0].cpu(), want)
    with torch.cuda.stream(side):
        k3, v3 = rows(6, 8, 128, torch.bfloat16, 30)
        cache.write(k3, v3, d_lens, d_table, d_starts)
    cache.write(k, v, i32([2, 4]), d_table, d_starts, stream=side)
    side.synchronize()
    check(cache, k3, v3, lens, table, [0, 2, 6])
    check(cache, k, v, [2, 4], table, [0, 2, 6])


def test_rows_move_with_their_pages():
    """Pages that are forked, grown (copy-on-write) and compacted keep what their rows stand
    for: the pools are pools like any other."""
    page, Hkv, D, N = 8, 8, 128, 40
    lens = [19, 0, 0, 30]
    table = np.full((4, 8), -1, np.int64)
    table[0, :3], table[3, :4] = [31, 7, 22], [39, 1, 12, 38]
    d_lens, d_table = i32(lens), i32(table)
    cache = Q4Cache(N, page, Hkv, D)
    k, v = rows(49, Hkv, D, torch.bfloat16, 2)
    cache.write(k, v, d_lens, d_table, i32([0, 19, 19, 19, 49]))
    pages = PageTable(d_lens, d_table, N, page, pools=[cache.k, cache.v])
    pages.fork(i32([0, 0]), i32([1, 2]), i32([19, 13]))
    pages.extend(i32([1, 2, 3, 4]))
    k2, v2 = rows(10, Hkv, D, torch.bfloat16, 4)
    starts = i32([0, 1, 3, 6, 10])
    cache.write(k2, v2, d_lens, d_table, starts)
    pages.compact()
    out = torch.empty((2, 20 + 21 + 16 + 34, Hkv, D), dtype=torch.bfloat16, device="cuda")
    cache.read(d_lens, d_table, i32([0, 20, 41, 57, 91]), out[0], out[1])
    assert pages.device_error() == 0 and cache.device_error() == 0
    assert d_lens.tolist() == [20, 21, 16, 34]
    for j, (x, x2) in enumerate(((k, k2), (v, v2))):
        want = torch.cat([x[:19], x2[:1], x[:19], x2[1:3], x[:13], x2[3:6], x[19:49], x2[6:10]])
        want = ref.values(*ref.quantise(want.float().cpu().numpy()))
        want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(out[j].cpu(), want)


def test_tables_of_more_than_2_to_31_bytes():
    """Offsets beyond 32 bits: the last page of a pool of 2.7 GB."""
    N, page, Hkv, D = 65536, 64, 8, 128
    cache = Q4Cache(N, page, Hkv, D)
    k, v = rows(40, Hkv, D, torch.bfloat16, 12)
    table = np.array([[N - 1]])
    cache.write(k, v, i32([40]), i32(table), i32([0, 40]))
    out = torch.empty((2, 40, Hkv, D), dtype=torch.bfloat16, device="cuda")
    cache.read(i32([40]), i32(table), i32([0, 40]), out[0], out[1])
    want = ref.values(*ref.quantise(k.float().cpu().numpy()))
    assert torch.equal(out[0].cpu(), torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))
    assert not cache.k[:N - 1].any()
