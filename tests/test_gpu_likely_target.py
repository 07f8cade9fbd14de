"""The gradient of a target that has almost all the probability keeps its digits:
g (1 - p) comes from log p, not from the difference of g and g p.

Tolerance: log p = (x - m) - L is one rounding (2^-24) of the logit's distance to
the maximum, which is exact here, and stats; expm1f is off by 2^-23 at most and
the product by 2^-24, relative, and 1 - p follows log p with a factor of at most
one: under 2^-22 in all, plus the result's own rounding."""
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
    yield
    assert fp8.fp8_get_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,offset", [(33, 0), (33, 1), (4099, 0), (4099, 3), (151936, 0)])
@pytest.mark.parametrize("with_entropy", [False, True])
def test_relative_accuracy(dtype, vocab, offset, with_entropy):
    places = [0, 1, 7, 8, vocab // 2, vocab - 2, vocab - 1]              # head, whole vectors and tail of a row
    heights = [9.0, 12.0, 16.0, 20.0, 24.0, 30.0]                         # 1 - p from some 1e-2 down to 1e-11
    rows = len(places) * len(heights)
    buf = torch.zeros(rows * vocab + offset, device=dev(), dtype=dtype)
    logits = buf[offset:].view(rows, vocab)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    logits.copy_(0.5 * torch.randn(rows, vocab, generator=g, device=dev()))
    targets = torch.tensor(places, device=dev()).repeat(len(heights))
    top = torch.tensor(heights, device=dev()).repeat_interleave(len(places))
    logits.scatter_(1, targets[:, None], top[:, None].to(dtype))
    _, entropy, stats, _, _ = fp8.fp8_token_logprobs(logits, targets)
    dlp = 1 + torch.rand(rows, generator=g, device=dev())
    dent = torch.rand(rows, generator=g, device=dev()) if with_entropy else None
    out = fp8.fp8_token_logprobs_backward(logits, targets, stats, dlp, entropy if with_entropy else None, dent)
    x = logits.double().gather(1, targets[:, None])[:, 0]
    lp = x - stats[:, 0].double() - stats[:, 1].double()
    want = -dlp.double() * torch.expm1(lp)
    tol = 2.0 ** -22 * want.abs()
    if with_entropy:
        # h p (log p + H): exp's 2^-22, and the sum's rounding
        part = dent.double() * lp.exp()
        want = want - part * (lp + entropy.double())
        tol = tol + part * ((2.0 ** -22 + 2.0 ** -23) * (lp + entropy.double()).abs() + 2.0 ** -23 * (lp.abs() + entropy.double()))
    tol = tol + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * want.abs() + 2.0 ** -133
    err = (out.gather(1, targets[:, None])[:, 0].double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_target_and_empty_rows(dtype):
    """A target of probability 0 gets g itself."""
    logits = torch.randn(4, 1003, device=dev()).to(dtype)
    targets = torch.tensor([5, 1002, 0, 600], device=dev())
    logits[torch.arange(4), targets] = -torch.inf
    logits[3] = -torch.inf
    _, entropy, stats, _, _ = fp8.fp8_token_logprobs(logits, targets)
    g = torch.tensor([1.0, -2.0, 0.5, 4.0], device=dev())
    for h in (None, g):
        out = fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, h)
        assert torch.equal(out[torch.arange(4), targets].float(), g)
        assert bool(out.isfinite().all())
    # no gradient of log p, or no target: the entropy's part alone
    none = fp8.fp8_token_logprobs_backward(logits, None, stats, None, entropy, g)
    away = fp8.fp8_token_logprobs_backward(logits, torch.full_like(targets, -1), stats, g, entropy, g)
    assert torch.equal(none, away)
