"""What the host refuses of the 4-bit cache's calls before any launch (no GPU), and the
sizes it gives."""

import ctypes

import pytest
import torch

import q4_reference as ref
from top_sparse_attention_pks_gb300 import build, pks
from top_sparse_attention_pks_gb300.decoder import Q4Cache, Q4DecodeStep, _select_args


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def attention(**change):
    """Arguments without memory (the pointers are not followed before they are refused)."""
    a = pks.pks_q4_attention_args()
    a.B, a.Hq, a.Hkv, a.D, a.n_queries = 2, 8, 2, 64, 1
    a.page_size, a.max_pages, a.num_pages = 16, 32, 64
    for name in ("seq_lens", "block_table", "q", "pool_k", "pool_v", "out"):
        setattr(a, name, 4096)
    a.workspace, a.workspace_bytes = 4096, 1 << 40
    for k, v in change.items():
        setattr(a, k, v)
    return a


def rows(**change):
    a = pks.pks_q4_rows_args()
    a.B, a.n_rows, a.Hkv, a.D, a.page_size, a.max_pages, a.num_pages = 2, 5, 2, 64, 16, 32, 64
    a.k_row, a.k_head, a.v_row, a.v_head = 128, 64, 128, 64
    for name in ("seq_lens", "block_table", "starts", "k", "v", "pool_k", "pool_v"):
        setattr(a, name, 4096)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("Hkv,D", [(1, 64), (3, 64), (8, 64), (1, 128), (8, 128), (17, 128)])
def test_token_bytes(Hkv, D):
    n = pks.pks_q4_token_bytes(Hkv, D)
    assert n == -(-Hkv * ref.record_bytes(D) // 16) * 16


@pytest.mark.parametrize("Hkv,D,want", [(0, 64, -1), (1, 96, -6), (1025, 64, -6), (1, 256, -6)])
def test_token_bytes_refused(Hkv, D, want):
    n = ctypes.c_size_t()
    assert pks.lib().pks_q4_token_bytes(Hkv, D, ctypes.byref(n)) == want
    assert pks.lib().pks_q4_token_bytes(1, 64, None) == -1


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(Hq=9), -1), (dict(D=96), -6),
    (dict(page_size=0), -1), (dict(max_pages=0), -1), (dict(num_pages=0), -1),
    (dict(n_queries=-1), -1), (dict(n_queries=65), -6), (dict(causal=2), -1), (dict(k=-1), -1),
    (dict(trim=1), -1), (dict(k=4), -1), (dict(wait_limit=-1), -1), (dict(reserved=1), -1),
    (dict(sm_scale=-1.0), -1), (dict(sm_scale=float("nan")), -1),
    (dict(sm_scale=float("inf")), -1), (dict(Hq=34), -6), (dict(B=4097), -6),
    (dict(B=2049, n_queries=2), -6), (dict(Hkv=1025, Hq=1025), -6), (dict(max_pages=1 << 21), -6),
    (dict(num_pages=1 << 28), -6), (dict(seq_lens=None), -1), (dict(block_table=None), -1),
    (dict(q=None), -1), (dict(q=4104), -1), (dict(pool_k=None), -1), (dict(pool_v=4100), -1),
    (dict(out=None), -1), (dict(out=4098), -1), (dict(workspace=None), -7),
    (dict(workspace=4112), -7), (dict(workspace_bytes=256), -7)])
def test_attention_refused(change, want):
    assert pks.lib().pks_q4_attention(ctypes.byref(attention(**change)), None) == want
    assert pks.lib().pks_q4_attention(None, None) == -1


@pytest.mark.parametrize("change,want", [
    (dict(k=0), -1), (dict(topk_idx=None), -1), (dict(causal=1), -1), (dict(k=65537), -6),
    (dict(trim=2), -1), (dict(workspace_bytes=256), -7)])
def test_sparse_refused(change, want):
    a = attention(**{**dict(k=8, topk_idx=4096), **change})
    assert pks.lib().pks_q4_sparse_attention(ctypes.byref(a), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), -1), (dict(n_rows=-1), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1),
    (dict(Hkv=0), -1), (dict(D=32), -6), (dict(page_size=0), -1), (dict(k_row=4), -1),
    (dict(v_head=-64), -1), (dict(dtype=2, k_row=6), -1), (dict(seq_lens=None), -1),
    (dict(starts=None), -1), (dict(block_table=None), -1), (dict(k=None), -1), (dict(v=4104), -1),
    (dict(pool_k=None), -1), (dict(pool_v=4104), -1), (dict(B=4097), -6), (dict(Hkv=2000), -6)])
def test_rows_refused(change, want):
    for call in (pks.lib().pks_q4_write, pks.lib().pks_q4_read):
        assert call(ctypes.byref(rows(**change)), None) == want
        assert call(None, None) == -1


@pytest.mark.parametrize("change", [
    dict(k_row=0), dict(v_row=0), dict(k_head=0), dict(v_head=32), dict(k_row=64), dict(v_row=120),
    dict(k_row=64, k_head=256), dict(v_row=32, v_head=1024)])
def test_rows_to_read_into_share_no_values(change):
    assert pks.lib().pks_q4_read(ctypes.byref(rows(**change)), None) == -1


def test_cache_keeps_its_pools():
    for name in ("k", "v", "error"):
        with pytest.raises(AttributeError):
            setattr(Q4Cache.__new__(Q4Cache), name, torch.zeros(1))


def test_empty_calls_launch_nothing():
    L = pks.lib()
    assert L.pks_q4_attention(ctypes.byref(attention(B=0)), None) == 0
    assert L.pks_q4_sparse_attention(ctypes.byref(attention(B=0, k=4)), None) == 0
    assert L.pks_q4_write(ctypes.byref(rows(B=0)), None) == 0
    assert L.pks_q4_read(ctypes.byref(rows(n_rows=0)), None) == 0


@pytest.mark.parametrize("which,change,want", [
    ("a", dict(B=3), -1), ("s", dict(B=3), -1), ("a", dict(k=63), -1), ("s", dict(k=63), -1),
    ("a", dict(topk_idx=8192), -1), ("a", dict(n_queries=2), -1), ("s", dict(n_queries=2), -1),
    ("a", dict(q=None), -1), ("s", dict(q_idx=None), -1), ("s", dict(Hi=9), -6),
    ("a", dict(Hq=40), -6), ("s", dict(workspace=None), -7), ("a", dict(workspace=None), -7)])
def test_step_refused(which, change, want):
    s = pks.pks_decode_args()
    s.B, s.Hq, s.Hkv, s.D, s.Hi, s.Di = 2, 1, 1, 64, 1, 64
    s.page_size, s.max_pages, s.num_pages, s.k = 16, 32, 64, 64
    for name in ("seq_lens", "block_table", "topk_idx", "q_idx", "w_idx", "idx_k"):
        setattr(s, name, 4096)
    s.workspace, s.workspace_bytes = 4096, 1 << 40
    a = attention(k=64, topk_idx=4096, trim=1)
    for k, v in change.items():
        setattr(s if which == "s" else a, k, v)
    assert pks.lib().pks_q4_decode_step(ctypes.byref(s), ctypes.byref(a), None) == want
    assert pks.lib().pks_q4_decode_step(None, ctypes.byref(a), None) == -1
    assert pks.lib().pks_q4_decode_step(ctypes.byref(s), None, None) == -1


def host_step(nq, **change):
    """Tensors of a step and its cache, on the host."""
    i = torch.int32
    cache = Q4Cache.__new__(Q4Cache)
    cache.Hkv, cache.D = 2, 64
    cache._k = cache._v = torch.zeros((4, 16, pks.pks_q4_token_bytes(2, 64)), dtype=torch.uint8)
    lead = (2, nq) if nq else (2,)
    t = dict(seq_lens=torch.zeros(2, dtype=i), block_table=torch.zeros((2, 3), dtype=i),
             q=torch.zeros(lead + (8, 64), dtype=torch.bfloat16),
             q_idx=torch.zeros(lead + (4, 64), dtype=torch.int8), w_idx=torch.ones(4, dtype=i),
             idx_k=torch.zeros((4, 16, 64), dtype=torch.int8))
    t.update({name: (x if isinstance(x, torch.Tensor) else torch.zeros(x, dtype=t[name].dtype))
              for name, x in change.items()})
    return t, cache


@pytest.mark.parametrize("nq,change", [
    (0, dict(q_idx=(2, 3, 4, 64))), (0, dict(q_idx=(1, 4, 64))), (0, dict(q_idx=(4, 64))),
    (3, dict(q_idx=(2, 4, 64))), (3, dict(q_idx=(2, 2, 4, 64))), (3, dict(q_idx=(1, 3, 4, 64))),
    (0, dict(idx_k=(3, 16, 64))), (0, dict(idx_k=(4, 8, 64))), (0, dict(idx_k=(4, 16, 128))),
    (0, dict(idx_k=(8, 8, 64))), (3, dict(seq_lens=(3,))), (0, dict(block_table=(3, 3))),
    (0, dict(block_table=(6,))), (0, dict(w_idx=(3,))), (0, dict(w_idx_f=torch.zeros(4))),
    (3, dict(w_idx_f=torch.zeros(2, 4)))])
def test_step_refuses_shapes_that_disagree(nq, change):
    t, cache = host_step(nq, **change)
    with pytest.raises(ValueError):
        Q4DecodeStep(t, cache, 8)


def test_step_takes_fp8_tensors_as_their_bits():
    t, _ = host_step(0)
    top = torch.zeros((2, 8), dtype=torch.int32)
    for name in ("q_idx", "idx_k"):
        f8 = dict(t, **{name: t[name].view(torch.float8_e4m3fn)})
        assert getattr(_select_args(f8, top, 4, 16, 0), name) == t[name].data_ptr()
        with pytest.raises(TypeError):
            _select_args(dict(t, **{name: t[name].view(torch.uint8)}), top, 4, 16, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Nq", [(4096, 1), (64, 64), (1, 3)])
def test_all_heads_fit(D, B, Nq):
    """Every number of heads leaves the ring of stages its least length in shared memory."""
    for Hkv in list(range(1, 34)) + [40, 64, 127, 1024]:
        for G in (1, 3, 16) if Hkv <= 64 else (1,):
            for k in (0, 9):
                for page in (1, 7, 16, 64):
                    a = attention(B=B, Hkv=Hkv, Hq=Hkv * G, D=D, n_queries=Nq, k=k, page_size=page)
                    assert pks.pks_q4_workspace_size(a) > 0


def test_workspace_grows_with_the_rows():
    sizes = [pks.pks_q4_workspace_size(attention(Hq=g * 2)) for g in (4, 8, 16)]
    assert 0 < sizes[0] == sizes[1] < sizes[2]
    assert pks.pks_q4_workspace_size(attention(n_queries=4)) >= sizes[2]


def test_binding_refuses_shapes_that_disagree():
    i = torch.int32
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    pool = torch.zeros((4, 16, pks.pks_q4_token_bytes(2, 64)), dtype=torch.uint8)
    ok = dict(seq_lens=torch.zeros(2, dtype=i), block_table=torch.zeros((2, 3), dtype=i), q=q,
              pool_k=pool, pool_v=pool, Hkv=2)
    pks.make_q4_attention_args(**ok)
    for change in (dict(q=q[0]), dict(q=q.float()), dict(seq_lens=torch.zeros(3, dtype=i)),
                   dict(block_table=torch.zeros((3, 3), dtype=i)), dict(pool_v=pool[:3]),
                   dict(pool_k=pool[..., :48], pool_v=pool[..., :48]), dict(Hkv=1),
                   dict(topk_idx=torch.zeros((2, 0), dtype=i)),
                   dict(topk_idx=torch.zeros((2, 1, 4), dtype=i)),
                   dict(out=torch.zeros((2, 8, 32), dtype=torch.bfloat16)),
                   dict(lse=torch.zeros(2)), dict(q=torch.zeros((2, 0, 8, 64)).bfloat16())):
        with pytest.raises((ValueError, TypeError)):
            pks.make_q4_attention_args(**{**ok, **change})
    k = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    ok = dict(k=k, v=k, seq_lens=torch.zeros(2, dtype=i), block_table=torch.zeros((2, 3), dtype=i),
              starts=torch.zeros(3, dtype=i), pool_k=pool, pool_v=pool)
    pks.make_q4_rows_args(**ok)
    for change in (dict(k=k[0]), dict(v=k[:4]), dict(v=k.half()), dict(k=k.double(), v=k.double()),
                   dict(starts=torch.zeros(2, dtype=i)), dict(seq_lens=torch.zeros(1, dtype=i)),
                   dict(pool_k=pool.view(torch.int8)), dict(starts=torch.zeros(3)),
                   dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            pks.make_q4_rows_args(**{**ok, **change})
