"""Partial sums handed from one CTA pair to another while other streams load the
memory: the result has the same bits as on an idle GPU, call after call."""
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev
from test_gpu_newton_schulz import check, gaussian

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    fp8.fp8_clear_error()
    yield
    assert fp8.fp8_get_error() == 0


@pytest.mark.parametrize("shape", [(200, 9001), (256, 12000), (520, 4096), (2, 300, 5000)])
def test_same_bits_under_memory_traffic(shape):
    g = gaussian(shape, sum(shape))
    want = fp8.fp8_newton_schulz(g)
    check(g, want)
    ws = torch.empty(fp8.fp8_newton_schulz_workspace_bytes(*(shape if len(shape) == 3 else (1, *shape))), dtype=torch.uint8,
                     device=dev())
    a, b = (torch.empty(1 << 26, device=dev()) for _ in range(2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):
            b.copy_(a)
    outs = [fp8.fp8_newton_schulz(g, workspace=ws) for _ in range(20)]
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)
