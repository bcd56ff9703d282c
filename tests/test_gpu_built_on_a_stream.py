"""Objects built for a stream that is not torch's current one, while that one is
busy and the memory they get holds what others left: their buffers belong to their
own stream."""

import numpy as np
import pytest
import torch

from test_gpu_prefix import Batch
from top_sparse_attention_pks_gb300 import build
from top_sparse_attention_pks_gb300.decoder import PageTable

pytestmark = pytest.mark.gpu

BUSY = 400_000_000  # cycles: about 0.2 s


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def dev(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()


def leave_behind(stream, sizes):
    """Blocks of these sizes, filled with 0x7f, free for the next on `stream`."""
    with torch.cuda.stream(stream):
        for _ in range(2):
            held = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes]
            torch.cuda.synchronize()
            del held


@pytest.mark.parametrize("requests", [3, 40])  # the plan by one block, by several
@pytest.mark.parametrize("raw", [False, True])
def test_prefix_attention(requests, raw):
    torch.cuda._sleep(1)
    b = Batch([700 + i for i in range(requests)], [0] * requests, [640] * requests, D=64,
              seed=requests)
    probe = b.attention()
    probe()  # (kernels are loaded on their first launch, which may wait for the device)
    sizes = [probe.workspace.numel()] + [x.numel() * x.element_size()
                                         for x in (probe.out, probe.lse)]
    del probe
    side = torch.cuda.Stream()
    for s in (side, torch.cuda.current_stream()):
        leave_behind(s, sizes)
    torch.cuda._sleep(BUSY)
    on = side.cuda_stream if raw else side
    att = b.attention(stream=on)
    out = att(stream=on)
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "still busy: nothing was waited for"
    assert att.device_error(on) == 0
    got, lse = out.clone(), att.lse.clone()
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    b.check(got, lse)


def test_page_table():
    lens, table = dev([20, 0, 5]), dev([[0, 6, -1], [-1] * 3, [7, -1, -1]])
    add = dev([1, 17, 0])
    before = lens.clone(), table.clone()
    probe = PageTable(lens, table, 8, 16)
    probe.extend(add)  # (as above)
    lens.copy_(before[0])
    table.copy_(before[1])
    size = [probe.state.numel(), probe.page_map.numel() * 4]
    del probe
    side = torch.cuda.Stream()
    for s in (side, torch.cuda.current_stream()):
        leave_behind(s, size)
    busy = torch.empty(size[0], dtype=torch.uint8, device="cuda")  # the current stream's block
    torch.cuda._sleep(BUSY)
    busy.fill_(0x55)  # ... is still to be written by it when the state is built
    del busy
    pages = PageTable(lens, table, 8, 16, stream=side)
    pages.extend(add, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert pages.device_error(side) == 0 and int(pages.n_free) == 3
    assert table.tolist() == [[0, 6, -1], [1, 2, -1], [7, -1, -1]]
    assert pages.refs.tolist() == [1, 1, 1, 0, 0, 0, 1, 1]
