"""Newton-Schulz orthogonalisation on the GPU, against the iteration in 64 bits.

Two bounds.  (1) Worst case, in Frobenius norms, from the reference's own
matrices: an error e of X passes a step multiplied by at most the largest
divided difference of f(t) = a t + b t^3 + c t^5 over the singular values (of
either sign); a step adds the FP16 roundings (half a step, 2^-11) of S, Q and
the new X, and FP32 accumulation over K terms, at most K 2^-23 |X|_F^2 of S
(the tensor cores may cut instead of rounding) and likewise for the others:
  S: 2^-11 |S|_F + K 2^-23 |X|_F^2, times (|b| + 2 |c| |S|_2) |X|_2
  Q: (2^-11 |Q|_F + |c| K 2^-23 |S|_F^2) |X|_2,   X: 2^-11 |X|_F + K 2^-23 |Q|_F |X|_F
and the result's bfloat16 rounding adds 2^-8 |X|_F.
(2) For Gaussian matrices the roundings act like independent noise: 16 of them,
each 1/8 of a bfloat16 rounding's, none amplified in the mean much beyond the
matrix itself, make sqrt(16) / 8 = 0.5 of the result's own rounding error:
together 1.12 times what rounding the exact result gives.  2 is asserted."""
import math

import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev

pytestmark = pytest.mark.gpu

COEFF = fp8.NEWTON_SCHULZ_COEFFICIENTS


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    fp8.fp8_clear_error()
    yield
    assert fp8.fp8_get_error() == 0


def gaussian(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(dev())


def reference(g, coeff=COEFF, eps=1e-7):
    """The iteration in 64 bits for one matrix: the result and bound (1)
    without the last rounding."""
    x = g.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.mT
    err = 2.0 ** -11 * float(x.norm())
    u, u32 = 2.0 ** -11, 2.0 ** -23
    K = x.shape[1]
    for a, b, c in coeff:
        s = x @ x.mT
        q = b * s + c * (s @ s)
        q.diagonal().add_(a)
        y = q @ x
        t = torch.linalg.svdvals(x)
        t = torch.cat([t, -t, torch.zeros(1, device=t.device, dtype=t.dtype)])
        f = a * t + b * t ** 3 + c * t ** 5
        if len(t) > 400:                                   # the extreme slopes are enough: f is smooth
            t = torch.linspace(-float(t.max()), float(t.max()), 401, device=t.device, dtype=t.dtype)
            f = a * t + b * t ** 3 + c * t ** 5
        dt = t[:, None] - t[None, :]
        slope = torch.where(dt.abs() > 1e-9, (f[:, None] - f[None, :]) / torch.where(dt.abs() > 1e-9, dt, 1.0),
                            (a + 3 * b * t ** 2 + 5 * c * t ** 4)[:, None].expand_as(dt)).abs().max()
        xf, x2, sf, s2, qf = (float(v) for v in (x.norm(), torch.linalg.matrix_norm(x, 2), s.norm(),
                                                 torch.linalg.matrix_norm(s, 2), q.norm()))
        err = float(slope) * err + (u * sf + K * u32 * xf * xf) * (abs(b) + 2 * abs(c) * s2) * x2 \
            + (u * qf + abs(c) * s.shape[0] * u32 * sf * sf) * x2 + u * float(y.norm()) + s.shape[0] * u32 * qf * xf
        x = y
    return (x.mT if tall else x), err


def check(g, out, coeff=COEFF, eps=1e-7, noise=True):
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    gs, os_ = (g, out) if g.dim() == 3 else (g[None], out[None])
    for k in range(gs.shape[0]):
        want, err = reference(gs[k], coeff, eps)
        off = float((os_[k].double() - want).norm())
        # (the recursion is first order: its square is allowed for by 10%)
        assert off <= 1.1 * err + 2.0 ** -8 * float(want.norm()) + 1e-12, (k, off, err)
        if noise:
            best = float((want.bfloat16().double() - want).norm())
            assert off <= 2 * best, (k, off, best)


SHAPES = [(64, 64), (128, 300), (300, 128), (256, 256), (257, 513), (513, 257), (1000, 1001), (4, 520, 1100),
          (3, 1100, 520), (2, 72, 2056)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gaussian(shape, dtype):
    g = gaussian(shape, sum(shape), dtype)
    check(g, fp8.fp8_newton_schulz(g))


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (7, 1), (2, 2), (33, 17), (17, 33), (5, 9, 31), (1, 5000), (5000, 1),
                                   (40, 3, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tiny_and_thin(shape, dtype):
    """Too few elements for the noise model: the worst-case bound alone."""
    g = gaussian(shape, sum(shape), dtype)
    check(g, fp8.fp8_newton_schulz(g), noise=False)


def test_low_rank_and_wide_spectrum():
    u, v = gaussian((700, 5), 1), gaussian((5, 400), 2)
    g = u @ v
    check(g, fp8.fp8_newton_schulz(g), noise=False)
    s = torch.logspace(0, -6, 300, device=dev())
    q1, q2 = torch.linalg.qr(gaussian((300, 300), 3))[0], torch.linalg.qr(gaussian((500, 300), 4))[0]
    g = (q1 * s) @ q2.mT
    check(g, fp8.fp8_newton_schulz(g), noise=False)


def test_singular_values_come_near_one():
    g = gaussian((384, 1024), 9)
    t = torch.linalg.svdvals(fp8.fp8_newton_schulz(g).double())
    assert 0.6 < float(t.min()) and float(t.max()) < 1.3     # the quintic's fixed interval, with margin


def test_other_coefficients_and_step_counts():
    g = gaussian((200, 264), 11)
    for coeff in ([(1.5, -0.5, 0.0)], [(2.0, -1.5, 0.5)] * 3, [(3.4445, -4.775, 2.0315), (1.5, -0.5, 0.0)],
                  [(0.0, 0.0, 0.0)], [(1.0, 0.0, 0.0)] * 2):
        check(g, fp8.fp8_newton_schulz(g, coefficients=coeff, eps=1e-3), coeff, 1e-3, noise=False)


def test_scale_does_not_matter():
    g = gaussian((130, 260), 12)
    want = fp8.fp8_newton_schulz(g, eps=0.0)
    for k in (-100, -60, -1, 7, 90):
        assert torch.equal(fp8.fp8_newton_schulz(g * 2.0 ** k, eps=0.0), want), k
    tiny = gaussian((64, 72), 13) * 1e-42                   # subnormal
    check(tiny, fp8.fp8_newton_schulz(tiny, eps=0.0), eps=0.0, noise=False)


def test_matrices_of_a_batch_do_not_touch_each_other():
    for shape in ((5, 200, 333), (5, 333, 200)):
        g = gaussian(shape, 14)
        want = torch.stack([fp8.fp8_newton_schulz(m.contiguous()) for m in g])
        assert torch.equal(fp8.fp8_newton_schulz(g), want)
        bad = g.clone()
        bad[1] = 0.0
        bad[3, 7, 9] = math.nan
        bad[4, 0, 0] = math.inf
        out = fp8.fp8_newton_schulz(bad)
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
        assert bool((out[1] == 0).all()) and bool(out[3].isnan().all()) and bool(out[4].isnan().all())
        zero = torch.zeros(shape[1:], device=dev())
        assert bool((fp8.fp8_newton_schulz(zero, eps=0.0) == 0).all())


@pytest.mark.parametrize("shape", [(2, 129, 257), (2, 257, 129), (2, 200, 264), (1, 3, 5)])
def test_outputs_and_workspace_stay_inside_their_buffers(shape):
    g = gaussian(shape, 15)
    want = fp8.fp8_newton_schulz(g)
    n = g.numel() * 2
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=dev())
    out = buf[256:256 + n].view(torch.bfloat16).view(shape)
    need = fp8.fp8_newton_schulz_workspace_bytes(*shape)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=dev())    # NaNs before the call
    got = fp8.fp8_newton_schulz(g, out=out, workspace=ws[256:256 + need])
    assert torch.equal(got, want)
    for b, k in ((buf, n),):
        assert bool((b[:256] == 0xA5).all()) and bool((b[256 + k:] == 0xA5).all())
    assert bool((ws[:256] == 0xFF).all()) and bool((ws[256 + need:] == 0xFF).all())
    with pytest.raises(fp8.Fp8Error) as err:
        fp8.fp8_newton_schulz(g, workspace=ws[256:256 + need - 16])
    assert err.value.status == 2


def test_streams_and_graph():
    cases = [gaussian((300, 700), 20 + i) for i in range(2)]
    want = [fp8.fp8_newton_schulz(g) for g in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
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


def test_main_gradient_to_update():
    """wgrad into an FP32 main gradient over two micro-batches, then its
    orthogonalised update."""
    M, N, K = 256, 384, 256
    dw = torch.zeros(N, K, device=dev())
    for k in range(2):
        dy, x = gaussian((M, N), 30 + k, torch.bfloat16), gaussian((M, K), 40 + k, torch.bfloat16)
        _, _, dyqT, sdyT = fp8.fp8_quantize_act_1x128(dy, fp8.COLWISE)
        _, _, xqT, sxT = fp8.fp8_quantize_act_1x128(x, fp8.COLWISE)
        fp8.fp8_block_gemm_wgrad_accum_f32(dyqT, sdyT, xqT, sxT, dw)
    check(dw, fp8.fp8_newton_schulz(dw), noise=False)


