"""Refusals of the page calls that the host makes before any launch (no GPU)."""

import pytest
import torch

from top_sparse_attention_pks_gb300 import build, pks


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def args(num_pages=8, page_size=4, B=3, max_pages=5, pools=None):
    lens = torch.zeros(B, dtype=torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    raw = torch.zeros(pks.pks_pages_state_bytes(num_pages) + 256, dtype=torch.uint8)
    state = raw[-raw.data_ptr() % 256:][: pks.pks_pages_state_bytes(num_pages)]
    pools = [torch.zeros(num_pages, page_size, 6)] if pools is None else pools
    a = pks.make_pages_args(seq_lens=lens, block_table=table, num_pages=num_pages,
                            page_size=page_size, state=state, pools=pools)
    a.keep = (lens, table, raw, pools)
    return a


def refused(code, call, *a):
    with pytest.raises(pks.PksError) as e:
        call(*a)
    assert e.value.code == code


def test_state_size_and_offsets():
    for n in (1, 31, 32, 33, 1000, 1 << 20):
        total = pks.pks_pages_state_bytes(n)
        off = pks.pks_pages_offsets(n)
        assert off["ref"] % 256 == 0 and off["free_map"] % 256 == 0
        assert off["ref"] + 4 * n <= off["free_map"] < total
    for n in (0, -1, (1 << 24) + 1):
        refused(-1, pks.pks_pages_state_bytes, n)


def test_shapes_and_pointers():
    ids = torch.zeros(4, dtype=torch.int32)
    for change, code in [(dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(B=-1), -1),
                         (dict(max_pages=0), -1), (dict(reserved=1), -1), (dict(n_pools=9), -1),
                         (dict(n_pools=-1), -1), (dict(B=4097), -6), (dict(seq_lens=None), -1),
                         (dict(block_table=None), -1), (dict(state=None), -7),
                         (dict(state_bytes=100), -7), (dict(max_pages=1 << 23), -6),
                         (dict(num_pages=1 << 24, page_size=1 << 10), -6)]:
        a = args()
        for k, v in change.items():
            setattr(a, k, v)
        for call in (pks.pks_pages_init, pks.pks_pages_device_error):
            refused(code, call, a)
        refused(code, pks.pks_pages_fork, a, ids[:1], ids[1:2])
        refused(code, pks.pks_pages_free, a, ids[:1])
    a = args()
    a.state += 16
    refused(-7, pks.pks_pages_init, a)
    a = args()
    a.pools[0].data = None
    refused(-1, pks.pks_pages_compact, a)
    a = args()
    a.pools[0].token_bytes = 0
    refused(-1, pks.pks_pages_compact, a)


def test_lists():
    a = args()
    ids = torch.zeros(4, dtype=torch.int32)
    refused(-1, pks.pks_pages_fork, a, ids, ids)   # more forks than rows
    refused(-1, pks.pks_pages_free, a, ids)
    with pytest.raises(ValueError):
        pks.pks_pages_fork(a, ids[:2], ids[:1])
    with pytest.raises(ValueError):
        pks.pks_pages_fork(a, ids[:2], ids[:2], ids[:1])
    with pytest.raises(ValueError):
        pks.pks_pages_free(a, ids[:2], ids[:1])
    with pytest.raises(ValueError):
        pks.pks_pages_extend(a, ids)
    with pytest.raises(TypeError):
        pks.pks_pages_extend(a, ids[:3].long())
    with pytest.raises(ValueError):
        pks.pks_pages_compact(a, ids)
    with pytest.raises(ValueError):
        pks.pks_pages_fork(a, torch.zeros(6, dtype=torch.int32)[::2], ids[:3])


def test_pools():
    with pytest.raises(ValueError):
        args(pools=[torch.zeros(8, 5, 6)])
    with pytest.raises(ValueError):
        args(pools=[torch.zeros(8)])
    with pytest.raises(ValueError):
        args(pools=[torch.zeros(8, 4, 2)] * 9)
    with pytest.raises(ValueError):
        args(pools=[torch.zeros(4, 8, 6).transpose(0, 1)])
    assert args(pools=[torch.zeros(8, 4, 3, dtype=torch.int8)]).pools[0].token_bytes == 3
    assert args(pools=[torch.zeros(8, 4)]).pools[0].token_bytes == 4
