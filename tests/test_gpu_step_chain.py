"""The operators around the linears run together as a training step uses them:
residual + norm + quantization, the output projection, the token log
probabilities and their gradient, the linear's gradients, the norm's gradient
and the orthogonalised update, eagerly, captured into a graph and on two streams
at once.  Each stage is held against 64-bit arithmetic on that stage's own
inputs, with the tolerances its own tests derive."""
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8
from blockwise_fp8_pretraining_b200 import synthetic as syn

from _parity import dev

pytestmark = pytest.mark.gpu

M, K, V = 256, 384, 1152          # tokens, hidden, vocabulary
U = 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    fp8.fp8_clear_error()
    yield
    assert fp8.fp8_get_error() == 0


class Step:
    """One micro-batch's forward, backward and update of norm + output
    projection, with the buffers a program keeps."""

    def __init__(self, seed):
        g = syn.generator(seed)
        d = dev()
        self.x = syn.activation_bf16(M, K, 4, 30.0, g).to(d)
        self.residual = syn.normal_bf16((M, K), 2.0, g).to(d)
        self.dresidual = syn.normal_bf16((M, K), 1e-3, g).to(d)
        self.gamma = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16().to(d)
        self.w = syn.normal_bf16((V, K), 0.05, g).to(d)
        self.targets = torch.randint(0, V, (M,), generator=g).to(d)
        self.targets[3] = -1                                        # a position without a target
        self.dw = torch.zeros(V, K, device=d)
        self.dgamma = torch.zeros(K, device=d)

    def run(self):
        o = self
        self.s, self.rstd, q, sq, qT, sqT = fp8.fp8_add_rmsnorm_quantize_1x128(o.x, o.gamma, residual=o.residual)
        wq, sw, wqT = fp8.fp8_quantize_weight_128x128(o.w)
        self.logits = fp8.fp8_block_gemm_fprop(q, sq, wq, sw)
        self.logp, self.entropy, self.stats, self.top_logp, self.top = fp8.fp8_token_logprobs(o.logits, o.targets, topk=4)
        count = (o.targets >= 0).sum().clamp(min=1)
        self.dlogp = -torch.ones(M, device=dev()) / count            # the mean negative log probability
        self.dent = torch.full((M,), -0.01 / M, device=dev())        # with an entropy bonus
        self.dlogits = fp8.fp8_token_logprobs_backward(o.logits, o.targets, o.stats, o.dlogp, o.entropy, o.dent)
        dq, sd, dqT, sdT = fp8.fp8_quantize_act_1x128(o.dlogits)
        self.dy = fp8.fp8_block_gemm_dgrad(dq, sd, wqT, sw)
        fp8.fp8_block_gemm_wgrad_accum_f32(dqT, sdT, qT, sqT, o.dw)
        self.ds, _ = fp8.fp8_rmsnorm_backward(o.dy, o.s, o.rstd, o.gamma, o.dresidual, dgamma=o.dgamma, accumulate=True)
        self.update = fp8.fp8_newton_schulz(o.dw)
        self.quantized = (q, sq, qT, sqT)
        return [self.s, self.rstd, q, sq, qT, sqT, self.logits, self.logp, self.entropy, self.stats, self.top_logp, self.top,
                self.dlogits, self.dy, self.ds, self.update]


def test_each_stage_on_its_own_inputs():
    st = Step(1)
    st.run()
    torch.cuda.synchronize()
    # the sum, the statistic and the quantized norm
    assert torch.equal(st.s, (st.x.float() + st.residual.float()).bfloat16())
    r = (st.s.double().square().mean(1) + 1e-6).rsqrt()
    assert float(((st.rstd.double() - r) / r).abs().max()) <= 2.0 ** -23
    ref = fp8.fp8_rmsnorm_quantize_1x128(st.s, st.rstd, st.gamma)
    for a, b in zip(st.quantized, ref):
        assert torch.equal(a, b)
    # log probabilities: FP32 arithmetic on rows of V, the bounds of their own tests
    x = st.logits.double()
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    H = -(p * lp).sum(1)
    spread = (x.amax(1, keepdim=True) - x).mul(p).sum(1) + 1
    tol = 2.0 ** -22 + U * (3 * spread + V / 256 + 100) + 4 * U * lp.abs().amax(1)
    want = torch.where(st.targets < 0, 0.0, lp.gather(1, st.targets.clamp(min=0)[:, None])[:, 0])
    assert bool(((st.logp.double() - want).abs() <= tol).all())
    assert bool(((st.entropy.double() - H).abs() <= tol * (2 + H)).all())
    assert torch.equal(st.top, st.logits.float().sort(dim=1, descending=True, stable=True).indices[:, :4])
    # their gradient: FP32 arithmetic, one rounding to bfloat16 (2^-8)
    g = torch.where(st.targets < 0, 0.0, st.dlogp.double())[:, None]
    hot = torch.zeros_like(x).scatter_(1, st.targets.clamp(min=0)[:, None], 1.0)
    d = g * (hot - p) - st.dent.double()[:, None] * p * (lp + H[:, None])
    size = p * (g.abs() + st.dent.double().abs()[:, None] * (lp.abs() + H[:, None])) + hot * g.abs()
    assert bool(((st.dlogits.double() - d).abs() <= 2.0 ** -8 * d.abs() + size * (2.0 ** -20 + 32 * U * lp.abs()) + 1e-38).all())
    # the norm's gradient, joined by the residual path's
    n, dy, rr = st.s.double() * st.rstd.double()[:, None], st.dy.double(), st.rstd.double()[:, None]
    gd = dy * st.gamma.double()
    ds = rr * (gd - n * (gd * n).mean(1, keepdim=True)) + st.dresidual.double()
    terms = (rr * gd).abs() + (rr * n).abs() * (gd * n).abs().mean(1, keepdim=True) * 6 + st.dresidual.double().abs()
    assert bool(((st.ds.double() - ds).abs() <= 2.0 ** -8 * ds.abs() + 16 * U * terms + 1e-40).all())
    dgamma = (dy * n).sum(0)
    assert bool(((st.dgamma.double() - dgamma).abs() <= U * (M + 64) * (dy * n).abs().sum(0) + 1e-40).all())
    # the update: singular values near one, in the gradient's directions
    t = torch.linalg.svdvals(st.update.double())
    strong = torch.linalg.svdvals(st.dw.double()) > 1e-2 * torch.linalg.matrix_norm(st.dw.double(), 2)
    assert 0.6 < float(t[strong].min()) and float(t.max()) < 1.3


def test_captured_step_equals_the_eager_one():
    """Main gradients accumulate over two micro-batches, once eagerly and once
    by replaying a graph on new contents."""
    eager, graphed, other = Step(2), Step(2), Step(3)
    eager.run()
    for name in ("x", "residual", "targets"):
        getattr(eager, name).copy_(getattr(other, name))
    want = [t.clone() for t in eager.run()] + [eager.dw.clone(), eager.dgamma.clone()]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                                    # (warm-up: library state, allocator)
        Step(4).run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.run()
    graph.replay()
    for name in ("x", "residual", "targets"):
        getattr(graphed, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, out + [graphed.dw, graphed.dgamma]):
        assert torch.equal(a, b)


def test_two_steps_at_once():
    """Two streams, each with its own buffers: results as one after the other."""
    alone = [Step(5), Step(6)]
    want = [[t.clone() for t in st.run()] for st in alone]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [Step(5), Step(6)]
    torch.cuda.synchronize()
    got = [None, None]
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            got[k] = both[k].run()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_gradient_of_the_whole_step_in_64_bits():
    """The step's ds and dgamma against autograd in 64 bits.  FP8 codes carry
    4 significant bits (2^-4 of a value, 2^-8 of a group's largest at the least),
    so the gradients agree as directions: each group of roundings is independent
    noise of at most 2^-4 / sqrt(3) relative, four of them (codes of y, W, dlogits
    and W again) make under 2^-4 * 4 / sqrt(3) = 0.15 of the norm."""
    st = Step(7)
    st.run()
    x = st.s.double().requires_grad_(True)
    gamma = st.gamma.double().requires_grad_(True)
    y = gamma * x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    lp = torch.log_softmax(y @ st.w.double().T, 1)
    keep = st.targets >= 0
    loss = -lp.gather(1, st.targets.clamp(min=0)[:, None])[:, 0][keep].sum() / keep.sum() + 0.01 / M * (lp.exp() * lp).sum()
    loss.backward()
    ds = st.ds.double() - st.dresidual.double()
    # (the residual path's part is taken out again: bfloat16's rounding of the sum stays, 2^-8 of it)
    off = float((ds - x.grad).norm())
    assert off <= 0.15 * float(x.grad.norm()) + 2.0 ** -8 * float(st.ds.double().norm())
    assert float((st.dgamma.double() - gamma.grad).norm()) <= 0.15 * float(gamma.grad.norm())
