"""Slices of longer tensors as arguments: the next-token loss (logits[:-1] with
targets[1:]), a loss in chunks of an odd number of rows, one matrix of a stack of
odd sizes.  Such views begin at any multiple of their element; the results are
those of the same values in tensors of their own, bit for bit."""
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    fp8.fp8_clear_error()
    yield
    assert fp8.fp8_get_error() == 0


def same(a, b):
    for u, v in zip(a, b):
        assert (u is None) == (v is None)
        assert u is None or torch.equal(u, v)


def rows_of(rows, vocab, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(rows, vocab, generator=g, device=dev()).to(dtype)
    return logits, torch.randint(0, vocab, (rows,), generator=g, device=dev()), torch.randn(rows, generator=g, device=dev())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("on_stream", [False, True])
def test_next_token_loss(dtype, on_stream):
    logits, tokens, g = rows_of(50, 1003, dtype, 1)
    st = torch.cuda.Stream() if on_stream else None
    torch.cuda.synchronize()
    out = fp8.fp8_token_logprobs(logits[:-1], tokens[1:], topk=3, stream=st)
    grad = fp8.fp8_token_logprobs_backward(logits[:-1], tokens[1:], out[2], g[1:], out[1], g[1:], stream=st)
    torch.cuda.synchronize()
    want = fp8.fp8_token_logprobs(logits[:-1], tokens[1:].clone(), topk=3)
    same(out, want)
    assert torch.equal(grad, fp8.fp8_token_logprobs_backward(logits[:-1], tokens[1:].clone(), want[2], g[1:].clone(), want[1],
                                                             g[1:].clone()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("chunk", [1, 7, 33])
def test_loss_in_chunks(dtype, chunk):
    """Every per-row argument a slice, outputs given, none written outside its slice."""
    rows, vocab, k = 99, 515, 5
    logits, targets, g = rows_of(rows, vocab, dtype, 2)
    want = fp8.fp8_token_logprobs(logits, targets, topk=k)
    grad = fp8.fp8_token_logprobs_backward(logits, targets, want[2], g, want[1], g)
    new = [torch.full_like(t, -7) for t in want]
    dlogits = torch.empty_like(logits)
    for i in range(0, rows, chunk):
        part = [t[i:i + chunk] for t in new]
        out = fp8.fp8_token_logprobs(logits[i:i + chunk], targets[i:i + chunk], topk=k, logprob=part[0], entropy=part[1],
                                     stats=part[2], top_logprob=part[3], top_index=part[4])
        assert all(a is b for a, b in zip(out, part))
        for t, w in zip(new, want):
            assert torch.equal(t[:i + chunk], w[:i + chunk]) and bool((t[i + chunk:] == -7).all())
        d = fp8.fp8_token_logprobs_backward(logits[i:i + chunk], targets[i:i + chunk], part[2], g[i:i + chunk], part[1],
                                            g[i:i + chunk], dlogits=dlogits[i:i + chunk])
        assert d.data_ptr() == dlogits[i:i + chunk].data_ptr()
    assert torch.equal(dlogits, grad)


def test_captured():
    logits, tokens, _ = rows_of(20, 300, torch.float32, 3)
    want = fp8.fp8_token_logprobs(logits[:-1], tokens[1:].clone())
    fp8.fp8_token_logprobs(logits[:-1], tokens[1:])
    store = torch.zeros(20, device=dev())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8.fp8_token_logprobs(logits[:-1], tokens[1:], logprob=store[1:])
    tokens.copy_(tokens.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    now = fp8.fp8_token_logprobs(logits[:-1], tokens[1:].clone())
    assert not torch.equal(now[0], want[0])
    assert torch.equal(out[0], now[0]) and torch.equal(store[1:], now[0]) and float(store[0]) == 0.0


def test_norm_gradient_in_chunks():
    g = torch.Generator(device="cuda").manual_seed(4)
    dy, s = (torch.randn(37, 256, generator=g, device=dev()).bfloat16() for _ in range(2))
    rstd, gamma = torch.rand(37, generator=g, device=dev()), torch.randn(256, generator=g, device=dev()).bfloat16()
    for i in (1, 2, 3, 5):
        got = fp8.fp8_rmsnorm_backward(dy[i:], s[i:], rstd[i:], gamma)
        same(got, fp8.fp8_rmsnorm_backward(dy[i:], s[i:], rstd[i:].clone(), gamma))


@pytest.mark.parametrize("shape", [(3, 5, 7), (3, 33, 77), (3, 129, 257), (4, 257, 131), (3, 300, 1001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_matrix_of_a_stack(shape, dtype):
    g = torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(5), device=dev()).to(dtype)
    out = torch.full(shape, 9.0, dtype=torch.bfloat16, device=dev())
    for i in range(shape[0]):
        want = fp8.fp8_newton_schulz(g[i].clone())
        assert torch.equal(fp8.fp8_newton_schulz(g[i]), want)
        given = out[i]
        assert fp8.fp8_newton_schulz(g[i], out=given) is given
        assert torch.equal(out[i], want) and bool((out[i + 1:] == 9.0).all())
