"""Token log probabilities, entropy, alternatives and their gradient on the
GPU, against 64-bit arithmetic on the same logits.

Tolerances.  Each exponential is off by a relative 2^-22 (ex2.approx) plus the
rounding of its argument: d = x - m, d * log2(e) and the constant, at most three
times 2^-24 |d|.  Averaged with the weights p they give 2^-22 + 3 2^-24 a with
a = sum p |d|; a sum of n terms adds at most (longest chain of additions) 2^-24:
a thread's own elements (two interleaved sums of at most V / 256 + 32 elements)
and 14 levels of joins (each referring a sum to a new maximum: 4 roundings).
So L = log(sum) is off by dL = 2^-22 + 2^-24 (3 a + V / 256 + 32 + 64), and the
entropy by dL + the same relative error, with b = sum p d^2 in the place of a,
of a.  Differences and roundings of the results add 2^-24 of what they are
taken of."""
import math

import numpy as np
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

from _parity import dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = math.inf


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    yield
    assert fp8.fp8_get_error() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def case(rows, vocab, dtype, seed, masked=False, pad=0, offset=0):
    """Logits as a view of a buffer with row stride vocab + pad, starting
    `offset` elements into it; the padding holds values that would show."""
    g = gen(seed)
    buf = torch.full((rows * (vocab + pad) + offset + 8,), 1e4, device=dev(), dtype=dtype)
    logits = buf[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    x = torch.randn(rows, vocab, generator=g, device=dev()) * 3.0
    targets = torch.randint(0, vocab, (rows,), generator=g, device=dev())
    x.scatter_add_(1, targets[:, None], 14 * torch.rand(rows, 1, generator=g, device=dev()))
    if masked:
        x.masked_fill_(torch.rand(rows, vocab, generator=g, device=dev()) < 0.3, -INF)
        targets[torch.rand(rows, generator=g, device=dev()) < 0.2] = -1
        x[rows // 2] = -INF
        if rows > 3:
            x[0] = torch.finfo(dtype).min               # a mask of the type's lowest value
            x[1] = torch.finfo(dtype).max / 2
            x[2] = -INF
            x[2, vocab // 2] = 3.0                      # one token left
    logits.copy_(x)
    return logits, targets


def reference(logits, targets):
    x = logits.double()
    m = x.amax(1)
    empty = m == -INF
    d = x - m.masked_fill(empty, 0.0)[:, None]
    e = d.exp()
    total = e.sum(1)
    L = total.log().masked_fill(empty, 0.0)
    p = e / total.masked_fill(empty, 1.0)[:, None]
    dz = d.masked_fill(d == -INF, 0.0)
    a, b = (p * dz.abs()).sum(1), (p * dz * dz).sum(1)
    H = (L + a).masked_fill(empty, 0.0)
    lp = d - L[:, None]
    at = lp.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    logp = torch.where(targets < 0, 0.0, at)
    chain = x.shape[1] / 256 + 96
    rel = 2.0 ** -22 + U * (3 * a + chain)
    # the joins' log1p / log: one more rounding of L
    L_tol = rel + U * L
    logp_tol = L_tol + 2 * U * (torch.where(at.isinf(), 0.0, at.abs()) + L)
    H_tol = L_tol + a * (rel + 2.0 ** -22 + U * (chain + 4)) + 3 * U * b + 2 * U * H
    return dict(m=m, L=L, H=H, logp=logp, lp=lp, p=p, empty=empty, L_tol=L_tol, logp_tol=logp_tol, H_tol=H_tol)


def near(got, want, tol, what):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), what
    err = (got - want)[fine].abs()
    worst = (err / tol.expand_as(want)[fine]).max() if err.numel() else 0.0
    assert bool((err <= tol.expand_as(want)[fine]).all()), f"{what}: {float(worst):.3g} of the tolerance"


def check_forward(logits, targets, topk):
    ref = reference(logits, targets)
    logp, entropy, stats, top_lp, top_i = fp8.fp8_token_logprobs(logits, targets, topk=topk)
    torch.cuda.synchronize()
    assert torch.equal(stats[:, 0].double(), ref["m"])
    near(stats[:, 1], ref["L"], ref["L_tol"], "log sum")
    near(logp, ref["logp"], ref["logp_tol"], "logprob")
    near(entropy, ref["H"], ref["H_tol"], "entropy")
    if topk:
        order = (logits.float() + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :topk]
        assert torch.equal(top_i, order)
        want = ref["lp"].gather(1, order)
        tol = ref["L_tol"][:, None] + 2 * U * (torch.where(want.isinf(), 0.0, want.abs()) + ref["L"][:, None])
        near(top_lp, want, tol, "alternatives")
    else:
        assert top_lp is None and top_i is None
    return logp, entropy, stats


SHAPES = [(1, 1), (2, 2), (5, 7), (4, 33), (300, 40), (7, 127), (64, 1000), (9, 4099), (5, 32001), (1, 151936),
          (40, 151936), (1, 8191), (2500, 517)]


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("masked", [False, True])
def test_forward(rows, vocab, dtype, masked):
    logits, targets = case(rows, vocab, dtype, rows + vocab, masked)
    for topk in {0, min(1, vocab), min(20, vocab), min(32, vocab)}:
        check_forward(logits, targets, topk)


@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (64, 5), (1, 7)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padded_and_misaligned_rows(pad, offset, dtype):
    for rows, vocab in [(6, 5), (6, 300), (17, 20011), (2, 151936)]:
        logits, targets = case(rows, vocab, dtype, vocab + pad, pad=pad, offset=offset)
        check_forward(logits, targets, min(5, vocab))
        check_backward(logits, targets, True, pad=2 * pad)


def test_equal_logits_rank_by_index():
    for dtype in (torch.bfloat16, torch.float32):
        for vocab in (40, 5003, 70000):
            logits = torch.zeros(3, vocab, device=dev(), dtype=dtype)
            logits[1, ::2] = -0.0                       # equal to +0
            logits[2] = torch.randint(0, 3, (vocab,), generator=gen(1), device=dev()).to(dtype)
            check_forward(logits, torch.zeros(3, dtype=torch.int64, device=dev()), 32)


def test_increasing_and_decreasing_rows():
    """The orders in which the bound of the alternatives and the running
    maximum change most and least often."""
    up = torch.arange(70001, device=dev(), dtype=torch.float32) / 3000
    check_forward(torch.stack([up, up.flip(0)]), torch.tensor([70000, 3], device=dev()), 32)


def test_one_token_with_almost_all_probability():
    """log p of the likely token and the entropy keep their digits."""
    for dtype in (torch.bfloat16, torch.float32):
        for vocab in (33, 4099, 151936):
            logits = torch.randn(1, vocab, generator=gen(vocab), device=dev()).to(dtype)
            logits[0, vocab // 3] = 40.0
            targets = torch.tensor([vocab // 3], device=dev())
            lp = torch.log_softmax(logits.double(), 1)
            rest = (logits.double() - 40.0).exp()
            rest[0, vocab // 3] = 0.0
            want = -torch.log1p(rest.sum(1))
            logp, entropy, _, _, _ = fp8.fp8_token_logprobs(logits, targets)
            # relative: the exponentials' 2^-22 + 3 2^-24 * 45 and the sums
            assert abs(float((logp.double() - want) / want)) < 2.0 ** -22 + U * (3 * 45 + vocab / 256 + 100)
            p = lp.exp()
            H = -(p * lp).sum(1) + 0.0
            H = (rest * (40.0 - logits.double())).sum(1) / (1 + rest.sum(1)) + torch.log1p(rest.sum(1))
            assert abs(float((entropy.double() - H) / H)) < 2 * (2.0 ** -22 + U * (3 * 45 + vocab / 256 + 100))


def test_targets_outside_and_nan():
    logits = torch.randn(6, 1000, generator=gen(2), device=dev())
    logits[3, 17] = math.nan
    logits[4, 17] = INF
    targets = torch.tensor([-5, 1000, 999, 1, 2, 0], device=dev())
    logp, entropy, stats, top_lp, top_i = fp8.fp8_token_logprobs(logits, targets, topk=4)
    assert float(logp[0]) == 0.0 and math.isnan(float(logp[1]))
    assert math.isnan(float(logp[3])) and math.isnan(float(entropy[3])) and math.isnan(float(logp[4]))
    assert 17 not in top_i[3].tolist() and int(top_i[4, 0]) == 17
    assert torch.equal(top_i[5], logits[5].sort(descending=True).indices[:4])
    few = torch.full((1, 9), math.nan, device=dev())
    few[0, 5] = 1.0
    _, _, _, top_lp, top_i = fp8.fp8_token_logprobs(few, topk=3)
    assert top_i[0].tolist() == [5, -1, -1] and bool(top_lp.isnan().all())
    grad = fp8.fp8_token_logprobs_backward(logits, targets, stats, torch.ones(6, device=dev()))
    assert bool((grad[0] == 0).all()) and bool(grad[1].isnan().all()) and bool(grad[2].isfinite().all())


def test_repeats_bit_for_bit():
    logits, targets = case(3, 151936, torch.bfloat16, 3)
    a = fp8.fp8_token_logprobs(logits, targets, topk=20)
    for _ in range(3):
        for u, v in zip(a, fp8.fp8_token_logprobs(logits, targets, topk=20)):
            assert torch.equal(u, v)


def test_without_targets_and_with_given_outputs():
    logits, targets = case(5, 2000, torch.bfloat16, 4)
    want = fp8.fp8_token_logprobs(logits, targets, topk=3)
    logp, entropy, stats, _, _ = fp8.fp8_token_logprobs(logits)
    assert logp is None and torch.equal(entropy, want[1]) and torch.equal(stats, want[2])
    out = {"logprob": torch.empty(5, device=dev()), "stats": torch.empty(5, 2, device=dev()),
           "top_index": torch.empty(5, 3, dtype=torch.int64, device=dev())}
    got = fp8.fp8_token_logprobs(logits, targets, topk=3, **out)
    assert got[0] is out["logprob"] and got[2] is out["stats"] and got[4] is out["top_index"]
    for u, v in zip(got, want):
        assert torch.equal(u, v)


# ------------------------------------------------------------------ gradient

def check_backward(logits, targets, with_entropy, with_logprob=True, pad=0, seed=1):
    rows, vocab = logits.shape
    g = gen(seed)
    ref = reference(logits, targets)
    stats = torch.stack([ref["m"], ref["L"]], 1).float()
    dlp = torch.randn(rows, generator=g, device=dev()) if with_logprob else None
    dent = torch.randn(rows, generator=g, device=dev()) if with_entropy else None
    entropy = ref["H"].float() if with_entropy else None
    buf = torch.full((rows, vocab + pad), 7.0, device=dev(), dtype=logits.dtype)
    out = fp8.fp8_token_logprobs_backward(logits, targets, stats, dlp, entropy, dent, dlogits=buf[:, :vocab])
    torch.cuda.synchronize()
    assert bool((buf[:, vocab:] == 7.0).all())
    # at the given (rounded) stats and entropy
    lse = torch.where(ref["empty"], INF, stats.double().sum(1))
    lp = logits.double() - stats[:, :1].double().masked_fill(ref["empty"][:, None], 0.0) - stats[:, 1:].double()
    p = lp.exp()
    lpz = lp.masked_fill(lp == -INF, 0.0)
    gg = torch.where(targets < 0, 0.0, dlp.double())[:, None] if with_logprob else torch.zeros(rows, 1, device=dev()).double()
    hh = dent.double()[:, None] if with_entropy else 0.0
    HH = entropy.double()[:, None] if with_entropy else 0.0
    want = -p * (gg + hh * (lpz + HH))
    hot = torch.zeros_like(want).scatter_(1, targets.clamp(min=0)[:, None], 1.0) * gg
    want = want + hot
    size = p * (gg.abs() + abs(hh) * (lpz.abs() + HH)) if with_entropy else p * gg.abs()
    tol = size * (2.0 ** -22 + U * (3 * lpz.abs() + 8)) + U * hot.abs() + 1e-37
    tol = tol + (2.0 ** -8 if logits.dtype == torch.bfloat16 else U) * want.abs() + 2.0 ** -133
    near(out, want, tol, "dlogits")
    assert not bool(lse.isnan().any())
    return out


@pytest.mark.parametrize("rows,vocab", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("masked", [False, True])
def test_backward(rows, vocab, dtype, masked):
    logits, targets = case(rows, vocab, dtype, rows + vocab + 1, masked)
    check_backward(logits, targets, False)
    check_backward(logits, targets, True)
    check_backward(logits, targets, True, with_logprob=False)


def test_backward_in_place():
    for dtype in (torch.bfloat16, torch.float32):
        logits, targets = case(9, 5003, dtype, 6, pad=3)
        _, entropy, stats, _, _ = fp8.fp8_token_logprobs(logits, targets)
        g = torch.randn(9, generator=gen(3), device=dev())
        want = fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, g)
        got = fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, g, dlogits=logits)
        assert got is logits and torch.equal(got, want)


def test_gradient_against_differences():
    """Differences in 64 bits of sum g logp + h H over random directions."""
    logits, targets = case(6, 700, torch.float32, 8)
    _, entropy, stats, _, _ = fp8.fp8_token_logprobs(logits, targets)
    g, h = torch.randn(6, generator=gen(1), device=dev()), torch.randn(6, generator=gen(2), device=dev())
    grad = fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, h).double()

    def loss(x):
        lp = torch.log_softmax(x, 1)
        return float((g.double() * lp.gather(1, targets[:, None])[:, 0]).sum() - (h.double() * (lp.exp() * lp).sum(1)).sum())

    x = logits.double()
    for k in range(4):
        v = torch.randn(6, 700, generator=gen(20 + k), device=dev()).double()
        step = 1e-5
        num = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
        assert abs(num - float((grad * v).sum())) <= 1e-6 * float((grad * v).abs().sum()) + 1e-8


def test_large_offsets():
    """Rows beyond 2^31 elements into the logits (a strided view, so that
    only two rows' pages hold data)."""
    vocab, ld = 1000, (1 << 30) + 3
    buf = torch.empty(2 * ld + vocab + 8, dtype=torch.bfloat16, device=dev())
    logits = buf.as_strided((3, vocab), (ld, 1))
    logits.copy_(torch.randn(3, vocab, generator=gen(5), device=dev()))
    targets = torch.tensor([1, 2, 999], device=dev())
    check_forward(logits, targets, 5)
    want = fp8.fp8_token_logprobs(logits.contiguous(), targets)
    g = torch.ones(3, device=dev())
    a = fp8.fp8_token_logprobs_backward(logits.contiguous(), targets, want[2], g)
    b = fp8.fp8_token_logprobs_backward(logits, targets, want[2], g, dlogits=logits)
    assert torch.equal(a, b)


def test_streams_and_graph():
    logits, targets = case(30, 20011, torch.bfloat16, 12)
    g = torch.randn(30, generator=gen(4), device=dev())

    def step():
        logp, entropy, stats, tl, ti = fp8.fp8_token_logprobs(logits, targets, topk=8)
        return [logp, entropy, stats, tl, ti, fp8.fp8_token_logprobs_backward(logits, targets, stats, g, entropy, g)]

    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    other, _ = case(30, 20011, torch.bfloat16, 13)
    torch.cuda.synchronize()
    a = fp8.fp8_token_logprobs(other, targets, topk=8, stream=st)
    b = step()
    torch.cuda.synchronize()
    for u, v in zip(want, b):
        assert torch.equal(u, v)
    for u, v in zip(a, fp8.fp8_token_logprobs(other, targets, topk=8)):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    logits.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    held = [t.clone() for t in out]
    for u, v in zip(held, step()):
        assert torch.equal(u, v)
