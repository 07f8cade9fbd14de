"""Forms of the operators around the linears that their own tests leave out: rows
that fill their last warp only in part at two and four chunks per lane, outputs
that only the C entry points can leave out, Newton-Schulz on long thin matrices and
on norms far below eps."""
import ctypes

import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev
from test_gpu_addnorm import check_forward, grad_case, norm_case, reference_backward, within
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


def ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


# cols / 8 chunks over warps of 32 lanes with 1, 2 or 4 chunks each
RAGGED = [4224, 4352, 6016, 7936, 8064, 8320, 12416, 16256]


@pytest.mark.parametrize("cols", RAGGED)
@pytest.mark.parametrize("rows", [5, 299, 640])
def test_ragged_rows_forward(rows, cols):
    x, res, gamma = norm_case(rows, cols, rows + cols)
    check_forward(x, res, gamma, fp8.ROWWISE)
    check_forward(x, None, gamma, fp8.BOTH if rows % 128 == 0 else fp8.ROWWISE)


@pytest.mark.parametrize("cols", RAGGED)
@pytest.mark.parametrize("rows", [1, 5, 299, 640])
def test_ragged_rows_backward(rows, cols):
    dy, s, rstd, gamma, dres = grad_case(rows, cols, rows + cols)
    for e in (dres, None):
        ds, dgamma = fp8.fp8_rmsnorm_backward(*(t.to(dev()) for t in (dy, s, rstd, gamma)),
                                              dresidual=None if e is None else e.to(dev()))
        want_ds, ds_tol, want_dg, dg_tol = reference_backward(dy, s, rstd, gamma, e)
        within(ds, want_ds, ds_tol, "ds")
        within(dgamma, want_dg, dg_tol, "dgamma")


@pytest.mark.parametrize("rows,cols", [(3, 384), (700, 1024), (640, 8320), (310, 16384)])
def test_gradient_without_the_weights(rows, cols):
    """dgamma = NULL: the same ds, no workspace."""
    dy, s, rstd, gamma, dres = (t.to(dev()) for t in grad_case(rows, cols, 7))
    want, _ = fp8.fp8_rmsnorm_backward(dy, s, rstd, gamma, dres)
    ds = torch.empty_like(s)
    st = fp8.load().fp8_rmsnorm_backward(ptr(dy), ptr(s), ptr(rstd), ptr(gamma), ptr(dres), rows, cols, ptr(ds), None, 0, None,
                                         0, stream())
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(ds, want)


@pytest.mark.parametrize("rows,vocab", [(1, 151936), (7, 1003), (300, 40)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_without_some_outputs(rows, vocab, dtype):
    """logprob or entropy NULL, with and without alternatives: the others are the same."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    logits = torch.randn(rows, vocab, generator=g, device=dev()).to(dtype)
    targets = torch.randint(0, vocab, (rows,), generator=g, device=dev())
    for k in (0, 5):
        want = fp8.fp8_token_logprobs(logits, targets, topk=k)
        for leave in ((0,), (1,), (0, 1)):
            out = [None if i in leave or w is None else torch.empty_like(w) for i, w in enumerate(want)]
            st = fp8.load().fp8_token_logprobs(ptr(logits), 0 if dtype == torch.bfloat16 else 1, rows, vocab, vocab,
                                               ptr(None if 0 in leave else targets), k, *map(ptr, out), stream())
            torch.cuda.synchronize()
            assert st == 0
            for o, w in zip(out, want):
                assert o is None or torch.equal(o, w)


def test_padded_row_in_place_and_one_row_of_many():
    """One row: its stride does not matter, in place or not."""
    buf = torch.randn(5, 1024, device=dev())
    logits, targets = buf[2:3, :1000], torch.tensor([3], device=dev())
    _, entropy, stats, _, _ = fp8.fp8_token_logprobs(logits, targets)
    g = torch.ones(1, device=dev())
    want = fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, g)
    rest = buf.clone()
    assert torch.equal(fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, g, dlogits=logits), want)
    assert torch.equal(buf[2:3, :1000], want) and torch.equal(buf[2, 1000:], rest[2, 1000:])
    assert torch.equal(buf[[0, 1, 3, 4]], rest[[0, 1, 3, 4]])


@pytest.mark.parametrize("shape", [(1, 8193), (1, 20000), (3, 20001), (17, 9000), (2, 5, 32768), (60, 10007)])
def test_long_and_thin(shape):
    """A shorter side of a few rows with a longer one that no cluster holds: worst-case bound."""
    g = gaussian(shape, sum(shape))
    check(g, fp8.fp8_newton_schulz(g), noise=False)
    tall = g.mT.contiguous()
    check(tall, fp8.fp8_newton_schulz(tall), noise=False)


@pytest.mark.parametrize("shape", [(40, 90), (90, 40), (300, 280), (129, 600)])
@pytest.mark.parametrize("norm", [1e-11, 1e-12, 1e-13])
def test_norm_far_below_eps_against_64_bits(shape, norm):
    """X is |G| / eps times a unit matrix and each step multiplies it by a = 3.4445 (its
    cube no longer counts).  FP16 in its subnormals, of X times more than sqrt(mn) / 2,
    is off by 2^-25 an element, 2^-24 of the norm, at the start and after each step:
    2^-24 (a^5 + a^4 + ...) < 2^-23 a^5 = 5.8e-5, besides the roundings of the iteration's
    own bound and of the result."""
    g = gaussian(shape, 5)
    g = g * (norm / float(g.norm()))
    want, err = reference(g)
    out = fp8.fp8_newton_schulz(g).double()
    size = float(want.norm())
    assert size > 4 * 2.0 ** -23 * 3.4445 ** 5          # there is something to be right about
    assert float((out - want).norm()) <= 2.0 ** -23 * 3.4445 ** 5 + 1.1 * err + 2.0 ** -8 * size
    assert float(out.norm()) > 0.5 * size
