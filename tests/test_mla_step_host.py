"""Refusals of the DSA step in one call that the host makes before any launch (no
GPU)."""

import ctypes

import pytest

from top_sparse_attention_pks_gb300 import build, pks


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def pair(B=2):
    """Arguments that differ in nothing and have no memory (the pointers are not
    followed before they are refused)."""
    s, m = pks.pks_decode_args(), pks.pks_mla_args()
    s.B, s.Hq, s.Hkv, s.D, s.Hi, s.Di = B, 1, 1, 64, 1, 64
    m.B, m.H, m.d_latent, m.d_rope = B, 128, 512, 64
    for a in (s, m):
        a.page_size, a.max_pages, a.num_pages, a.k = 16, 32, 64, 64
        for name in ("seq_lens", "block_table", "topk_idx"):
            setattr(a, name, 4096)
    for name in ("q_idx", "w_idx", "idx_k"):
        setattr(s, name, 4096)
    for name in ("q", "kv", "out"):
        setattr(m, name, 4096)
    for a in (s, m):
        a.workspace, a.workspace_bytes = 4096, 1 << 40
    return s, m


def code(s, m):
    return pks.lib().pks_mla_decode_step(s and ctypes.byref(s), m and ctypes.byref(m), None)


@pytest.mark.parametrize("which,change,want", [
    ("s", dict(B=3), -1), ("m", dict(B=3), -1), ("s", dict(k=63), -1), ("m", dict(k=65), -1),
    ("s", dict(topk_idx=8192), -1), ("m", dict(topk_idx=8192), -1), ("s", dict(n_queries=2), -1),
    ("s", dict(seq_lens=None), -1), ("m", dict(seq_lens=None), -1), ("s", dict(q_idx=None), -1),
    ("m", dict(q=None), -1), ("m", dict(q=4104), -1), ("m", dict(trim=2), -1),
    ("m", dict(d_rope=32), -6), ("s", dict(Hi=9), -6), ("s", dict(workspace=None), -7),
    ("m", dict(workspace=None), -7), ("m", dict(workspace_bytes=8), -7),
    ("s", dict(workspace_bytes=8), -7), ("m", dict(workspace=4112), -7)])
def test_refused(which, change, want):
    s, m = pair()
    for k, v in change.items():
        setattr(s if which == "s" else m, k, v)
    assert code(s, m) == want


def test_nothing_and_an_empty_batch():
    s, m = pair()
    assert code(None, m) == -1 and code(s, None) == -1
    assert code(*pair(B=0)) == 0
