"""Residual addition + RMSNorm + quantization and its gradient on the GPU.

Forward: the sum is bfloat16's correctly rounded x + residual; rstd lies within
one float32 ulp of the oracle's (another order of the FP64 sum); and, given the
rstd the kernel wrote, codes and scales equal the oracle's bit for bit.

Gradient: against the formula in 64 bits.  The kernel rounds ds once to
bfloat16 (at most half a step, 2^-8 of the value) after FP32 arithmetic whose
terms are r g, r n m and dresidual with m = mean(g n): each carries a handful
of roundings (at most 2^-24 each; n = s r, dy n, g n, its product with m, the
final sums: under 16), and m a sum whose longest chain of additions is at most
8 * 8 (a lane's elements) + 5 (shuffles) + 8 (warps) < 96 roundings of
mean |g n|.  dgamma is a sum over rows of products with three roundings each,
whose chain of additions is at most rows + blocks' partial sums: (rows + 64)
roundings of sum |dy n| bound it whatever the split."""
import numpy as np
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8
import oracle
from blockwise_fp8_pretraining_b200 import synthetic as syn

from _parity import assert_bits_equal, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    yield
    assert fp8.fp8_get_error() == 0


def norm_case(rows, cols, seed):
    g = syn.generator(seed)
    x = syn.activation_bf16(rows, cols, max(1, cols // 100), 30.0, g).float()
    res = (2.0 * torch.randn(rows, cols, generator=g)).bfloat16().float()
    gamma = (1.0 + 0.2 * torch.randn(cols, generator=g)).float()
    x[0] = 0.0                                     # a zero row without the residual
    if rows > 2:
        res[1] = -x[1]                             # the sum cancels to zero
        x[2], res[2] = 1e-38, 3e-39                # tiny and subnormal values
    gamma[: min(8, cols)] = torch.tensor([0.0, -0.0, 1e-38, -1.0, 1.0, 3.0, 1e-5, 100.0])[: min(8, cols)]
    return x.bfloat16(), res.bfloat16(), gamma.bfloat16()


def check_forward(x, res, gamma, mode, eps=1e-6, **out):
    d = dev()
    xs = x if res is None else (x.float() + res.float()).bfloat16()
    s, rstd, q_row, s_row, q_colT, s_col = fp8.fp8_add_rmsnorm_quantize_1x128(
        x.to(d), gamma.to(d), residual=None if res is None else res.to(d), eps=eps, mode=mode, **out)
    torch.cuda.synchronize()
    sb, gb = syn.bf16_bits(xs), syn.bf16_bits(gamma)
    assert_bits_equal(s.view(torch.int16), sb.view(np.int16), "sum")
    got = rstd.cpu().numpy()
    want = oracle.rmsnorm_rstd(sb, eps)
    assert np.abs(got.view(np.int32).astype(np.int64) - want.view(np.int32).astype(np.int64)).max() <= 1
    y = oracle.rmsnorm_apply(sb, got, gb)
    if mode & fp8.ROWWISE:
        q_o, s_o = oracle.quantize_act_rowwise(y)
        assert_bits_equal(q_row, q_o, "row codes")
        assert_bits_equal(s_row, s_o, "row scales")
    else:
        assert q_row is None and s_row is None
    if mode & fp8.COLWISE:
        q_o, s_o = oracle.quantize_act_colwise(y)
        assert_bits_equal(q_colT, q_o, "column codes")
        assert_bits_equal(s_col, s_o, "column scales")
    else:
        assert q_colT is None and s_col is None
    return s, rstd, q_row, s_row, q_colT, s_col


@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 2048), (3, 384), (5, 16384), (130, 8320), (301, 256), (333, 2176),
                                       (400, 512), (1037, 1024), (2049, 128), (700, 6144), (310, 16384)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_rowwise_any_rows(rows, cols, with_residual):
    x, res, gamma = norm_case(rows, cols, rows + cols)
    check_forward(x, res if with_residual else None, gamma, fp8.ROWWISE)


@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 384), (384, 1024), (128, 1152), (256, 2048), (128, 2176),
                                       (256, 4096), (128, 4224), (128, 6144), (128, 16384)])
@pytest.mark.parametrize("mode", [fp8.COLWISE, fp8.BOTH])
def test_tiles(rows, cols, mode):
    x, res, gamma = norm_case(rows, cols, 3 * rows + cols + mode)
    check_forward(x, res, gamma, mode)
    check_forward(x, None, gamma, mode)


def test_many_row_blocks_and_other_eps():
    x, res, gamma = norm_case(128 * 41, 640, 5)
    check_forward(x, res, gamma, fp8.BOTH, eps=0.25)


def test_agrees_with_the_separate_entry_points():
    x, res, gamma = (t.to(dev()) for t in norm_case(256, 2048, 9))
    s, rstd, q_row, s_row, q_colT, s_col = fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=res)
    ref = fp8.fp8_rmsnorm_quantize_1x128(s, rstd, gamma)
    for a, b in zip((q_row, s_row, q_colT, s_col), ref):
        assert torch.equal(a, b)
    one = fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=res, mode=fp8.ROWWISE)
    # the statistic's summation order differs between the two kernels
    same = one[1] == rstd
    assert same.float().mean() > 0.9
    assert torch.equal(one[2][same], q_row[same])


@pytest.mark.parametrize("mode,rows", [(fp8.ROWWISE, 77), (fp8.BOTH, 256)])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_sum_in_place(mode, rows, which):
    x, res, gamma = (t.to(dev()) for t in norm_case(rows, 768, 11))
    want = fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=res, mode=mode)
    xi, ri = x.clone(), res.clone()
    got = fp8.fp8_add_rmsnorm_quantize_1x128(xi, gamma, residual=ri, mode=mode, sum_out=xi if which == "x" else ri)
    for a, b in zip(want, got):
        assert (a is None and b is None) or torch.equal(a, b)
    assert torch.equal(ri if which == "x" else xi, res if which == "x" else x)


@pytest.mark.parametrize("rows,cols,mode", [(3, 384, fp8.ROWWISE), (128, 640, fp8.BOTH), (128, 4224, fp8.BOTH)])
def test_outputs_stay_inside_their_buffers(rows, cols, mode):
    """Outputs as views into sentinel-filled buffers."""
    d = dev()
    x, res, gamma = norm_case(rows, cols, 21)
    pads = {}

    def view(name, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=d)
        pads[name] = (buf, n)
        return buf[256:256 + n].view(dtype).view(shape)

    out = {"sum_out": view("sum", (rows, cols), torch.bfloat16), "rstd": None,
           "q_row": view("qr", (rows, cols), torch.uint8), "s_row": view("sr", (cols // 128, rows), torch.float32)}
    if mode & fp8.COLWISE:
        out["q_colT"] = view("qc", (cols, rows), torch.uint8)
        out["s_col"] = view("sc", (rows // 128, cols), torch.float32)
    out["rstd"] = view("r", (rows,), torch.float32)
    check_forward(x, res, gamma, mode, **out)
    for name, (buf, n) in pads.items():
        assert bool((buf[:256] == 0xA5).all()) and bool((buf[256 + n:] == 0xA5).all()), name


# ------------------------------------------------------------------ gradient

def reference_backward(dy, s, rstd, gamma, dres):
    """ds, dgamma and their error bounds, in 64 bits on the CPU."""
    dy, s, r, g0 = dy.double(), s.double(), rstd.double()[:, None], gamma.double()
    n, g = s * r, dy * g0
    m = (g * n).mean(1, keepdim=True)
    ds = r * (g - n * m) + (dres.double() if dres is not None else 0.0)
    terms = (r * g).abs() + (r * n * m).abs() + (dres.double().abs() if dres is not None else 0.0)
    ds_tol = 2.0 ** -8 * ds.abs() + U * (16 * terms + 96 * (r * n).abs() * (g * n).abs().mean(1, keepdim=True)) + 1e-40
    dgamma = (dy * n).sum(0)
    dgamma_tol = U * (dy.shape[0] + 64) * (dy * n).abs().sum(0) + 1e-40
    return ds, ds_tol, dgamma, dgamma_tol


def grad_case(rows, cols, seed):
    g = syn.generator(seed)
    s = syn.activation_bf16(rows, cols, max(1, cols // 100), 30.0, g)
    dy = syn.normal_bf16((rows, cols), 1e-3, g)
    dres = syn.normal_bf16((rows, cols), 1e-3, g)
    gamma = (1.0 + 0.2 * torch.randn(cols, generator=g)).bfloat16()
    if rows > 1:
        s[1] = 0.0                                  # rstd = eps^-1/2
    rstd = torch.from_numpy(oracle.rmsnorm_rstd(syn.bf16_bits(s), 1e-6))
    return dy, s, rstd, gamma, dres


def within(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    assert bool(torch.isfinite(got).all()), what
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).max()):.3g} of the tolerance"


@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 2048), (2, 16384), (3, 384), (7, 1536), (333, 5120), (150, 8192),
                                       (601, 16384), (129, 2176), (4099, 256), (1025, 1024), (2500, 2048)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_backward(rows, cols, with_residual):
    dy, s, rstd, gamma, dres = grad_case(rows, cols, rows + cols)
    if not with_residual:
        dres = None
    ds, dgamma = fp8.fp8_rmsnorm_backward(*(t.to(dev()) for t in (dy, s, rstd, gamma)),
                                          dresidual=None if dres is None else dres.to(dev()))
    want_ds, ds_tol, want_dg, dg_tol = reference_backward(dy, s, rstd, gamma, dres)
    within(ds, want_ds, ds_tol, "ds")
    within(dgamma, want_dg, dg_tol, "dgamma")


def test_backward_against_differences():
    """Directional differences, in 64 bits, of <dy, gamma s r(s)> over the
    gradient's own inputs."""
    dy, s, rstd, gamma, _ = grad_case(64, 512, 3)
    s[1] = s[0]                                     # (a zero row's norm curves too sharply for differences)
    rstd = torch.from_numpy(oracle.rmsnorm_rstd(syn.bf16_bits(s), 1e-6))
    ds, dgamma = fp8.fp8_rmsnorm_backward(*(t.to(dev()) for t in (dy, s, rstd, gamma)))

    def loss(sv, gv):
        return float((dy.double() * gv * sv * (sv.square().mean(1, keepdim=True) + 1e-6).rsqrt()).sum())

    sd, gd = s.double(), gamma.double()
    g = syn.generator(8)
    for _ in range(4):
        v, w = torch.randn(64, 512, generator=g).double(), torch.randn(512, generator=g).double()
        h = 1e-4
        num = (loss(sd + h * v, gd) - loss(sd - h * v, gd)) / (2 * h)
        # each ds element is off by its bfloat16 rounding (2^-8): the signed
        # sum's error is at most 2^-8 sum |ds v|; h^2 and rstd's rounding are far below
        assert abs(num - float((ds.double().cpu() * v).sum())) <= 2.0 ** -8 * float((ds.double().cpu() * v).abs().sum())
        num = (loss(sd, gd + h * w) - loss(sd, gd - h * w)) / (2 * h)
        assert abs(num - float((dgamma.double().cpu() * w).sum())) <= 1e-5 * float((dgamma.double().cpu() * w).abs().sum())


def test_backward_accumulates_and_repeats():
    dy, s, rstd, gamma, dres = (t.to(dev()) for t in grad_case(700, 1024, 4))
    ds, dgamma = fp8.fp8_rmsnorm_backward(dy, s, rstd, gamma, dres)
    start = torch.randn(1024, generator=syn.generator(5)).to(dev())
    acc = start.clone()
    fp8.fp8_rmsnorm_backward(dy, s, rstd, gamma, dres, dgamma=acc, accumulate=True)
    assert torch.equal(acc, start + dgamma)
    ds2, dgamma2 = fp8.fp8_rmsnorm_backward(dy, s, rstd, gamma, dres)
    assert torch.equal(ds, ds2) and torch.equal(dgamma, dgamma2)
    # rows without the second kernel
    few = [t[:2].contiguous() for t in (dy, s, rstd)]
    acc = start.clone()
    _, dg = fp8.fp8_rmsnorm_backward(*few, gamma)
    fp8.fp8_rmsnorm_backward(*few, gamma, dgamma=acc, accumulate=True)
    assert torch.equal(acc, start + dg)


@pytest.mark.parametrize("which", ["dy", "dresidual"])
def test_backward_in_place(which):
    dy, s, rstd, gamma, dres = (t.to(dev()) for t in grad_case(300, 2048, 6))
    want, _ = fp8.fp8_rmsnorm_backward(dy, s, rstd, gamma, dres)
    a, b = dy.clone(), dres.clone()
    got, _ = fp8.fp8_rmsnorm_backward(a, s, rstd, gamma, b, ds=a if which == "dy" else b)
    assert torch.equal(want, got)


def test_backward_without_rows():
    d = dev()
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=d)
    ds, dgamma = fp8.fp8_rmsnorm_backward(e, e, torch.empty(0, device=d), torch.ones(256, device=d).bfloat16())
    assert ds.shape == (0, 256) and bool((dgamma == 0).all())


def test_backward_refuses_a_small_workspace():
    dy, s, rstd, gamma, _ = (t.to(dev()) for t in grad_case(700, 1024, 4))
    need = fp8.fp8_rmsnorm_backward_workspace_bytes(700, 1024)
    assert need > 0 and need % (4 * 1024) == 0
    with pytest.raises(fp8.Fp8Error) as err:
        fp8.fp8_rmsnorm_backward(dy, s, rstd, gamma, workspace=torch.empty(need - 4, dtype=torch.uint8, device=dev()))
    assert err.value.status == 2


def test_streams_and_graph():
    """Two streams at once with their own workspaces, then a captured and
    replayed forward + backward on new contents."""
    d = dev()
    cases = [[t.to(d) for t in grad_case(512, 1024, 30 + i)] for i in range(2)]
    want = [fp8.fp8_rmsnorm_backward(dy, s, r, g, e) for dy, s, r, g, e in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for st, (dy, s, r, g, e) in zip(streams, cases):
        got.append(fp8.fp8_rmsnorm_backward(dy, s, r, g, e, stream=st))
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, e)

    x, res, gamma = (t.to(d) for t in norm_case(256, 1024, 50))
    dy = cases[0][0][:256].contiguous()

    def step():
        s, r, q, sc, qT, scT = fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=res)
        return [q, sc, qT, scT, *fp8.fp8_rmsnorm_backward(dy, s, r, gamma, dy)]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x2, res2, _ = norm_case(256, 1024, 51)
    x.copy_(x2)
    res.copy_(res2)
    graph.replay()
    torch.cuda.synchronize()
    held = [t.clone() for t in out]
    for a, b in zip(held, step()):
        assert torch.equal(a, b)
