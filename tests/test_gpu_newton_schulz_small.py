"""Newton-Schulz on matrices small enough for one launch (a shorter side of up to
128, a longer one of 2432 there and of up to 8192 at 48), at every number of CTAs a
matrix takes, at the edges of the range and just behind them.  Bounds as in the iteration's own tests:
the roundings are the same."""
import math

import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev
from test_gpu_newton_schulz import check, gaussian, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    fp8.fp8_clear_error()
    yield
    assert fp8.fp8_get_error() == 0


LONG = [128, 129, 257, 300, 520, 641, 900, 1024, 1025, 1500, 2047, 2048, 2049]


@pytest.mark.parametrize("short", [64, 100, 128, 129])
@pytest.mark.parametrize("long", LONG)
def test_wide_and_tall(short, long):
    g = gaussian((short, long), short + long)
    out = fp8.fp8_newton_schulz(g)
    check(g, out)
    tall = g.T.contiguous()
    check(tall, fp8.fp8_newton_schulz(tall))


@pytest.mark.parametrize("short", [1, 2, 15, 16, 17, 31, 33, 48, 49])
@pytest.mark.parametrize("long", [49, 97, 255, 256, 257, 1030, 2048])
def test_thin(short, long):
    """Too few singular values for the noise model: the worst-case bound alone."""
    for dtype in (torch.float32, torch.bfloat16):
        g = gaussian((short, long), short * long, dtype)
        check(g, fp8.fp8_newton_schulz(g), noise=False)
        tall = g.T.contiguous()
        check(tall, fp8.fp8_newton_schulz(tall), noise=False)


@pytest.mark.parametrize("shape", [(300, 20, 30), (7, 128, 700), (5, 700, 128), (9, 1, 2048), (149, 64, 64)])
def test_batches(shape):
    g = gaussian(shape, sum(shape), torch.bfloat16)
    want = torch.stack([fp8.fp8_newton_schulz(m.contiguous()) for m in g])
    out = fp8.fp8_newton_schulz(g)
    assert torch.equal(out, want)
    for _ in range(3):
        assert torch.equal(fp8.fp8_newton_schulz(g), out)
    bad = g.clone()
    bad[1] = 0.0
    bad[2, 0, 5] = math.nan
    bad[3, 0, 0] = math.inf
    got = fp8.fp8_newton_schulz(bad)
    assert torch.equal(got[0], want[0]) and torch.equal(got[4], want[4])
    assert bool((got[1] == 0).all()) and bool(got[2].isnan().all()) and bool(got[3].isnan().all())


def test_steps_and_coefficients():
    for shape in ((90, 500), (500, 90), (30, 200)):
        g = gaussian(shape, 5)
        for coeff in ([(1.5, -0.5, 0.0)], [(2.0, -1.5, 0.5)] * 2, [(3.4445, -4.775, 2.0315)] * 3, [(0.0, 0.0, 0.0)],
                      [(1.5, -0.5, 0.0)] * 32):
            check(g, fp8.fp8_newton_schulz(g, coefficients=coeff, eps=1e-3), coeff, 1e-3, noise=False)


def test_agrees_with_the_large_matrices_way():
    """A matrix with zero rows behind it has the same iteration: [128, n] and
    [129, n] take the two ways."""
    g = gaussian((128, 1000), 6)
    small = fp8.fp8_newton_schulz(g).double()
    large = fp8.fp8_newton_schulz(torch.cat([g, torch.zeros(1, 1000, device=dev())])).double()
    assert bool((large[128] == 0).all())
    want, err = reference(g)
    assert float((small - large[:128]).norm()) <= 2.2 * err + 2.0 ** -7 * float(want.norm())


def test_outputs_stay_inside_their_buffers():
    for shape in ((2, 100, 333), (2, 333, 100), (1, 3, 5), (3, 128, 2048)):
        g = gaussian(shape, 15)
        want = fp8.fp8_newton_schulz(g)
        n = g.numel() * 2
        buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=dev())
        out = buf[256:256 + n].view(torch.bfloat16).view(shape)
        need = fp8.fp8_newton_schulz_workspace_bytes(*shape)
        ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=dev())
        assert torch.equal(fp8.fp8_newton_schulz(g, out=out, workspace=ws[256:256 + need]), want)
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n:] == 0xA5).all())
        assert bool((ws[:256] == 0xFF).all()) and bool((ws[256 + need:] == 0xFF).all())


def test_streams_and_graph():
    cases = [gaussian((4, 128, 1500), 20 + i) for i in range(3)]
    want = [fp8.fp8_newton_schulz(g) for g in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = [fp8.fp8_newton_schulz(g, stream=st) for g, st in zip(cases, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    g = cases[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8.fp8_newton_schulz(g)
    g.copy_(cases[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])


# More matrices than run at once: wider shares, several rounds of clusters, or the
# launch per product.
@pytest.mark.parametrize("shape", [(20, 128, 1000), (40, 64, 900), (200, 500, 100), (80, 100, 600), (300, 33, 130)])
def test_many(shape):
    g = gaussian(shape, sum(shape), torch.bfloat16)
    out = fp8.fp8_newton_schulz(g)
    assert torch.equal(fp8.fp8_newton_schulz(g), out)
    for i in (0, 1, shape[0] // 2, shape[0] - 1):
        check(g[i], out[i], noise=min(shape[1:]) >= 64)


@pytest.mark.parametrize("shape", [(40, 90), (300, 280)])
def test_norm_far_below_eps(shape):
    """X is then |G| / eps times a unit matrix, and each step multiplies it by at most
    a = 3.4445 (its cube no longer counts): digits may be lost, nothing may be made up.
    FP16 in its subnormals, of X times more than sqrt(mn) / 2, is off by 2^-25 an element,
    2^-24 of the norm, at the start and after each step: 2^-24 (a^5 + a^4 + ...) < 2^-23 a^5."""
    g = gaussian(shape, 5)
    for norm in (1e-13, 1e-20):
        out = fp8.fp8_newton_schulz(g * (norm / float(g.norm()))).double()
        assert float(out.norm()) <= 1.01 * (norm / 1e-7) * 3.4445 ** 5 + 3.4445 ** 5 * 2.0 ** -23


# The longest that fit a cluster's shared memory, and the first that do not.
@pytest.mark.parametrize("shape", [(128, 2432), (128, 2433), (112, 3000), (96, 3840), (96, 3841), (80, 4992), (80, 4999),
                                   (65, 4900), (64, 6528), (64, 6529), (48, 8191), (48, 8192), (48, 8193), (33, 5000)])
def test_longest(shape):
    for dtype in (torch.float32, torch.bfloat16):
        g = gaussian(shape, sum(shape), dtype)
        check(g, fp8.fp8_newton_schulz(g), noise=shape[0] >= 64)
        tall = g.T.contiguous()
        check(tall, fp8.fp8_newton_schulz(tall), noise=shape[0] >= 64)


@pytest.mark.parametrize("shape", [(1, 8192), (3, 8001), (17, 8192), (32, 7777)])
def test_longest_thin(shape):
    g = gaussian((2, *shape), sum(shape))
    out = fp8.fp8_newton_schulz(g)
    check(g, out, noise=False)
    assert torch.equal(out[0], fp8.fp8_newton_schulz(g[0].contiguous()))
