"""The tests of attention over shared prefixes once more, with every prefix of a
tile or more taken once: left to itself the plan leaves the short ones of these
small batches to the requests' own parts."""

import pytest

import test_gpu_prefix as base
from test_gpu_prefix import *  # noqa: F401,F403 (the tests themselves)
from test_gpu_prefix import Batch, build, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


@pytest.fixture(autouse=True)
def _every_prefix(monkeypatch):
    plain = base.Batch.attention

    def attention(self, **kw):
        kw.setdefault("min_shared", 128)
        return plain(self, **kw)
    monkeypatch.setattr(base.Batch, "attention", attention)


@pytest.mark.parametrize("min_shared", [1, 63, 64, 65, 1 << 30])
def test_from_how_many_tokens_on(min_shared):
    """Prefixes shorter than a tile, and none."""
    b = Batch([403, 96, 241, 30, 176], [0, 0, 0, -1, -1], [64, 64, 64, 0, 0])
    att = b.attention(min_shared=min_shared)
    out = att()
    torch.cuda.synchronize()
    assert att.device_error() == 0
    assert int(att.workspace[8:12].view(torch.int32)) == (1 if min_shared <= 64 else 0)  # items
    b.check(out, att.lse)


def test_left_to_the_plan():
    """The bytes that the groups save together decide, except with many rows a
    request, which the same kernel reads in any case."""
    for tokens, Nq, want in ((2000, 1, 0), (6016, 1, 1), (256, 5, 1)):
        lens = [tokens + 40 * i for i in range(8)]
        b = Batch(lens, [0] * 8, [tokens] * 8, page=64, Hkv=8, G=4, D=128, Nq=Nq, seed=tokens)
        att = b.attention(min_shared=0)
        out = att()
        torch.cuda.synchronize()
        assert att.device_error() == 0
        items = int(att.workspace[8:12].view(torch.int32))
        assert (items > 0) == bool(want)
        b.check(out, att.lse, rows=[0, 3, 7])
