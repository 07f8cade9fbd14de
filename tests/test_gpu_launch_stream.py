"""Calls with stream= while the current stream is still at work: their new
outputs and scratch take no memory that queued work of another stream has yet to
read or write, and give none up that queued work of the caller has yet to read."""
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev

pytestmark = pytest.mark.gpu

SPIN = 100_000_000              # clocks: some 50 ms


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    fp8.fp8_clear_error()
    yield
    assert fp8.fp8_get_error() == 0


def cases():
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev())

    x, res, dy = (randn(512, 1024).bfloat16() for _ in range(3))
    gamma = randn(1024).bfloat16()
    rstd = torch.rand(512, generator=g, device=dev())
    logits, targets = randn(300, 5003), torch.randint(0, 5003, (300,), generator=g, device=dev())
    stats = fp8.fp8_token_logprobs(logits, targets)[2]
    up, w = randn(256, 1024).bfloat16(), randn(512, 1024).bfloat16()
    xq, sx, xqT, sxT = fp8.fp8_quantize_act_1x128(up)
    wq, sw, wqT = fp8.fp8_quantize_weight_128x128(w)
    dq, sd, dqT, sdT = fp8.fp8_quantize_act_1x128(randn(256, 512).bfloat16())
    small, large = randn(3, 100, 900), randn(300, 5000)
    return {
        "norm": lambda **k: fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=res, **k),
        "norm_grad": lambda **k: fp8.fp8_rmsnorm_backward(dy, x, rstd, gamma, res, **k),
        "logp": lambda **k: fp8.fp8_token_logprobs(logits, targets, topk=5, **k),
        "logp_grad": lambda **k: fp8.fp8_token_logprobs_backward(logits, targets, stats, rstd[:300].contiguous(), **k),
        "quantize": lambda **k: fp8.fp8_quantize_act_1x128(up, **k),
        "quantize_weight": lambda **k: fp8.fp8_quantize_weight_128x128(w, **k),
        "swiglu": lambda **k: fp8.fp8_swiglu_quantize_1x128(up, **k),
        "rstd": lambda **k: fp8.fp8_rmsnorm_rstd(up, **k),
        "norm_of_rstd": lambda **k: fp8.fp8_rmsnorm_quantize_1x128(x, rstd, gamma, **k),
        "fprop": lambda **k: fp8.fp8_block_gemm_fprop(xq, sx, wq, sw, **k),
        "dgrad": lambda **k: fp8.fp8_block_gemm_dgrad(dq, sd, wqT, sw, **k),
        "wgrad": lambda **k: fp8.fp8_block_gemm_wgrad(dqT, sdT, xqT, sxT, **k),
        "cast": lambda **k: fp8.fp8_cast_e4m3_scaled(logits, 2.0, **k),
        "newton_schulz_small": lambda **k: fp8.fp8_newton_schulz(small, **k),
        "newton_schulz": lambda **k: fp8.fp8_newton_schulz(large, **k),
    }


NAMES = ["norm", "norm_grad", "logp", "logp_grad", "quantize", "quantize_weight", "swiglu", "rstd", "norm_of_rstd", "fprop",
         "dgrad", "wgrad", "cast", "newton_schulz_small", "newton_schulz"]


def outputs(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_queued_work_is_left_alone(name, handle):
    call = cases()[name]
    want = [t.clone() for t in outputs(call())]
    scratch = {"norm_grad": fp8.fp8_rmsnorm_backward_workspace_bytes(512, 1024),
               "newton_schulz_small": fp8.fp8_newton_schulz_workspace_bytes(3, 100, 900),
               "newton_schulz": fp8.fp8_newton_schulz_workspace_bytes(1, 300, 5000)}.get(name)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the outputs' and the scratch's sizes, freed with reads and writes of them still queued
    held = [torch.full_like(t, 3) for t in want]
    if scratch:
        held.append(torch.full((scratch,), 3, dtype=torch.uint8, device=dev()))
    copies = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    for c, t in zip(copies, held):
        c.copy_(t)
        t.fill_(5)
    del held, t
    got = outputs(call(stream=st.cuda_stream if handle else st))
    torch.cuda.synchronize()
    for c in copies:
        assert bool((c == 3).all()), "a queued read saw the call's output"
    for a, b in zip(got, want):
        assert torch.equal(a, b), "a queued write reached the call's output"


@pytest.mark.parametrize("name", NAMES)
def test_outputs_read_by_the_caller_are_not_given_away(name):
    """Freed with the caller's reads of them still queued, then a call on the
    side stream again."""
    call = cases()[name]
    want = [t.clone() for t in outputs(call())]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = outputs(call(stream=st))
    copies = [torch.empty_like(t) for t in got]
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(SPIN)
    for c, t in zip(copies, got):
        c.copy_(t)
    shapes = [(t.shape, t.dtype) for t in got]
    del got, t
    with torch.cuda.stream(st):
        other = [torch.zeros(s, dtype=d, device=dev()) for s, d in shapes]
    torch.cuda.synchronize()
    assert len(other) == len(copies)
    for a, b in zip(copies, want):
        assert torch.equal(a, b)


def test_current_stream_given_by_name():
    """stream= of the stream that is current anyway: nothing is tied to another."""
    call = cases()["logp"]
    want = outputs(call())
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        got = outputs(call(stream=st))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_on_a_forked_stream():
    call = cases()["norm"]
    want = outputs(call())
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = outputs(call(stream=side))
        torch.cuda.current_stream().wait_stream(side)
    for t in got:
        t.fill_(1)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
