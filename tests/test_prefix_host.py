"""Refusals of the shared-prefix attention that the host makes before any launch
(no GPU), and the size of its workspace."""

import pytest
import torch

from top_sparse_attention_pks_gb300 import build, pks


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def tensors(B=2, Nq=1, Hq=8, Hkv=2, D=64, N=4, P=16):
    return dict(seq_lens=torch.zeros(B, dtype=torch.int32),
                block_table=torch.zeros((B, 5), dtype=torch.int32),
                prefix_group=torch.zeros(B, dtype=torch.int32),
                q=torch.zeros((B, Nq, Hq, D), dtype=torch.bfloat16),
                kv_k=torch.zeros((N, P, Hkv, D), dtype=torch.bfloat16),
                kv_v=torch.zeros((N, P, Hkv, D), dtype=torch.bfloat16),
                out=torch.zeros((B, Nq, Hq, D), dtype=torch.bfloat16))


def args(**kw):
    t = tensors(**kw)
    a = pks.make_prefix_args(**t)
    raw = torch.zeros(pks.pks_prefix_workspace_size(a) + 256, dtype=torch.uint8)
    a.workspace = raw.data_ptr() + -raw.data_ptr() % 256
    a.workspace_bytes = raw.numel() - 256
    a.keep = (t, raw)
    return a


def refused(code, call, a):
    with pytest.raises(pks.PksError) as e:
        call(a)
    assert e.value.code == code


@pytest.mark.parametrize("change,code", [
    (dict(B=-1), -1), (dict(Hq=0), -1), (dict(Hkv=3), -1), (dict(D=0), -1), (dict(D=96), -6),
    (dict(page_size=0), -1), (dict(max_pages=0), -1), (dict(num_pages=0), -1),
    (dict(n_queries=-1), -1), (dict(n_queries=65), -6), (dict(causal=2), -1),
    (dict(wait_limit=-1), -1), (dict(reserved=3), -1), (dict(sm_scale=-1.0), -1),
    (dict(sm_scale=float("nan")), -1), (dict(sm_scale=float("inf")), -1),
    (dict(Hq=34, Hkv=2), -6), (dict(B=4097), -6), (dict(B=1025, n_queries=4), -6),
    (dict(num_pages=1 << 28), -6), (dict(max_pages=1 << 21), -6)])
def test_shapes(change, code):
    a = args()
    for k, v in change.items():
        setattr(a, k, v)
    for call in (pks.pks_prefix_workspace_size, pks.pks_prefix_plan, pks.pks_prefix_attention,
                 pks.pks_prefix_device_error):
        refused(code, call, a)


def test_pointers_and_workspace():
    for name in ("block_table", "q", "kv_k", "kv_v", "out"):
        a = args()
        setattr(a, name, None)
        refused(-1, pks.pks_prefix_attention, a)
    for name in ("q", "kv_k", "kv_v", "out"):
        a = args()
        setattr(a, name, getattr(a, name) + 8)
        refused(-1, pks.pks_prefix_attention, a)
    for name in ("seq_lens", "block_table"):
        a = args()
        setattr(a, name, None)
        refused(-1, pks.pks_prefix_plan, a)
    for change in (dict(workspace=None), dict(workspace_bytes=256)):
        a = args()
        for k, v in change.items():
            setattr(a, k, v)
        for call in (pks.pks_prefix_plan, pks.pks_prefix_attention, pks.pks_prefix_device_error):
            refused(-7, call, a)
    a = args()
    a.workspace += 16
    refused(-7, pks.pks_prefix_plan, a)


def test_tensors():
    for name, bad in [("q", torch.zeros((2, 8, 32), dtype=torch.bfloat16)),
                      ("q", torch.zeros((2, 8), dtype=torch.bfloat16)),
                      ("q", torch.zeros((2, 0, 8, 64), dtype=torch.bfloat16)),
                      ("kv_v", torch.zeros((4, 16, 1, 64), dtype=torch.bfloat16)),
                      ("seq_lens", torch.zeros(3, dtype=torch.int32)),
                      ("block_table", torch.zeros(10, dtype=torch.int32)),
                      ("prefix_group", torch.zeros(1, dtype=torch.int32)),
                      ("out", torch.zeros((2, 8, 64), dtype=torch.bfloat16)),
                      ("kv_k", torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16).transpose(1, 2))]:
        with pytest.raises(ValueError):
            pks.make_prefix_args(**dict(tensors(), **{name: bad}))
    for name, bad in [("q", torch.zeros((2, 1, 8, 64))), ("prefix_group", torch.zeros(2)),
                      ("seq_lens", torch.zeros(2, dtype=torch.int64))]:
        with pytest.raises(TypeError):
            pks.make_prefix_args(**dict(tensors(), **{name: bad}))
    with pytest.raises(ValueError):
        pks.make_prefix_args(**tensors(), lse=torch.zeros((2, 8)))


def test_workspace_size():
    """Partials: each row once a KV head, in up to twice the rows of short items,
    and one item a CTA; nothing for the wide kernel where it never runs."""
    small = pks.pks_prefix_workspace_size(args())
    t = tensors()
    t["prefix_group"] = None
    assert pks.pks_prefix_workspace_size(pks.make_prefix_args(**t)) < small
    a = args()
    a.B, a.Hq, a.Hkv, a.D = 4096, 128, 8, 128
    rows = 4096 * 128
    assert pks.pks_prefix_workspace_size(a) < 5 * rows * (128 + 2) * 4
    a = args()
    a.B = 0  # an empty batch is no error and launches nothing
    pks.pks_prefix_plan(a)
    pks.pks_prefix_attention(a)


def test_min_shared():
    for change in (dict(min_shared=-1), dict(reserved2=1)):
        a = args()
        for k, v in change.items():
            setattr(a, k, v)
        for call in (pks.pks_prefix_workspace_size, pks.pks_prefix_plan, pks.pks_prefix_attention):
            refused(-1, call, a)
