"""Newton-Schulz products whose tiles are cut along the contraction: the partial
sums handed from one CTA pair to another through the workspace, at shapes that
cut them into few and many parts, next to each other on two streams, and in
batches.  Bound (1) of the iteration's own tests holds whatever the order of the
sums (it counts K roundings of FP32 accumulation)."""
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


# long contractions over few tiles: one tile in many parts, column halves and
# parts, a ragged last half, a few matrices, and whole waves before the cut ones
SHAPES = [(40, 9001), (9001, 40), (256, 8192), (4096, 512), (500, 6000), (1300, 7777), (3, 300, 5000), (5, 5000, 130),
          (2048, 4096), (6144, 2048)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gaussian(shape, dtype):
    g = gaussian(shape, sum(shape), dtype)
    out = fp8.fp8_newton_schulz(g)
    check(g, out)
    for _ in range(3):                                     # the parts are added in order, whichever comes first
        assert torch.equal(fp8.fp8_newton_schulz(g), out)


def test_workspace_contents_do_not_matter():
    for shape in ((4096, 512), (512, 4096)):
        g = gaussian(shape, 3)
        want = fp8.fp8_newton_schulz(g)
        ws = torch.empty(fp8.fp8_newton_schulz_workspace_bytes(1, *shape), dtype=torch.uint8, device=dev())
        for fill in (0, 1, 0x7F, 0xFF):
            ws.fill_(fill)
            assert torch.equal(fp8.fp8_newton_schulz(g, workspace=ws), want)
        # and what a call leaves there does no harm to the next, of fewer steps or another shape
        a = fp8.fp8_newton_schulz(g, coefficients=[(1.5, -0.5, 0.0)], workspace=ws)
        assert torch.equal(a, fp8.fp8_newton_schulz(g, coefficients=[(1.5, -0.5, 0.0)]))
        small = gaussian((256, 2048), 4)
        assert torch.equal(fp8.fp8_newton_schulz(small, workspace=ws), fp8.fp8_newton_schulz(small))
        assert torch.equal(fp8.fp8_newton_schulz(g, workspace=ws), want)


def test_at_once_on_several_streams():
    shapes = [(4096, 512), (512, 4096), (256, 8192)]
    cases = [gaussian(s, 10 + i) for i, s in enumerate(shapes)]
    want = [fp8.fp8_newton_schulz(g) for g in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = [fp8.fp8_newton_schulz(g, stream=st) for g, st in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_captured():
    g = gaussian((4096, 512), 21)
    other = gaussian((4096, 512), 22)
    want = fp8.fp8_newton_schulz(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8.fp8_newton_schulz(g)
    g.copy_(other)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
