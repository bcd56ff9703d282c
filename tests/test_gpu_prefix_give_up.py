"""Waits of the shared-prefix attention that run out at any point: the kernels give
up with code 5 (or finish, when nothing ran out), copies and products in flight
end before shared and tensor memory are given up, and the same buffers give the
right results afterwards, beside work that was launched right behind."""

import pytest
import torch

from test_gpu_prefix import Batch
from top_sparse_attention_pks_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


LIMITS = (1, 300, 1000, 3000, 10000, 30000)


def give_up(b, causal, **kw):
    """Runs with every limit, each followed by a whole run of another object, and
    then without a limit, which has to be right."""
    att, after = b.attention(causal=causal, **kw), b.attention(causal=causal, **kw)
    codes = []
    for limit in LIMITS:
        att.args.wait_limit = limit
        att()
        out = after()
        codes.append(att.device_error())
        assert after.device_error() == 0
        b.check(out, after.lse, causal, what=f"behind limit {limit}")
    assert codes[0] == 5 and set(codes) <= {0, 5}
    att.args.wait_limit = 0
    for _ in range(2):
        att.out.fill_(float("nan"))
        out = att()
        assert att.device_error() == 0
        b.check(out, att.lse, causal, what="without a limit")


@pytest.mark.parametrize("page", [5, 16, 128])  # row by row, boxes by four warps, by one
@pytest.mark.parametrize("D,Nq", [(64, 3), (128, 3)])
@pytest.mark.parametrize("tokens", [256, 4000])  # two tiles a CTA: the loads never wait; more
def test_wide(page, D, Nq, tokens):
    """24 rows a request and KV head: the wide kernel alone, prefix and own tokens."""
    lens = [tokens + 3, tokens + 100] + ([tokens] * 30 if tokens == 4000 else [])
    b = Batch(lens, [0] * len(lens), [tokens] * len(lens), page=page, Hkv=2, G=8, D=D, Nq=Nq,
              seed=page + D + tokens)
    give_up(b, causal=True, min_shared=128)


@pytest.mark.parametrize("page", [1, 16, 64])  # row by row, by boxes
@pytest.mark.parametrize("D,Hkv,G,Nq",
                         [(64, 1, 4, 1), (128, 8, 4, 3), (128, 4, 8, 1), (64, 3, 5, 2)])
@pytest.mark.parametrize("tokens", [32, 30000])  # two tiles a CTA: its ring is never full; more
def test_narrow(page, D, Hkv, G, Nq, tokens):
    """Own tokens of up to 16 rows, no groups: the narrow kernel alone."""
    lens = [tokens, tokens - 7, 1, 0, 90]
    b = Batch(lens, [-1] * 5, [0] * 5, page=page, Hkv=Hkv, G=G, D=D, Nq=Nq, seed=page + Hkv,
              groups_passed=False)
    give_up(b, causal=Nq > 1)


@pytest.mark.parametrize("page", [5, 16, 128])
def test_both(page):
    """Prefixes by the wide kernel and own tokens by the narrow one beside it."""
    lens = [2000 + 150 * i for i in range(8)]
    b = Batch(lens, [0] * 8, [1920] * 8, page=page, Hkv=4, G=4, D=128, Nq=2, seed=page)
    give_up(b, causal=True, min_shared=128)
