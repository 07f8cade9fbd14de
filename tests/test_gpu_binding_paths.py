"""The binding's two ways to the same entry points on the GPU: the compiled
host side (plain calls on the current stream) and the Python one give the same
results bit for bit, hand back the same given tensors and refuse the same calls
with the same errors."""
import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8
from blockwise_fp8_pretraining_b200 import _abi

from _parity import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fp8.load()
    assert _abi._host is not None, "the compiled host side is not built"
    yield
    assert fp8.fp8_get_error() == 0


def both_ways(monkeypatch, call):
    """call() through the compiled host side and through Python."""
    seen = []
    plain = _abi._plain
    with monkeypatch.context() as m:
        m.setattr(_abi, "_plain", lambda *a: seen.append(plain(*a)) or seen[-1])
        first = call()
    with monkeypatch.context() as m:
        m.setattr(_abi, "_host", None)
        second = call()
    return seen, first, second


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for u, v in zip(a, b):
        assert (u is None) == (v is None)
        if u is not None:
            assert u.dtype == v.dtype and u.shape == v.shape and u.device == v.device and u.is_contiguous() == v.is_contiguous()
            assert torch.equal(u, v)


def tensors(rows, cols, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r, dy = (torch.randn(rows, cols, generator=g, device=dev()).bfloat16() for _ in range(3))
    gamma = (1 + 0.1 * torch.randn(cols, generator=g, device=dev())).bfloat16()
    return x, r, dy, gamma


@pytest.mark.parametrize("rows,cols", [(0, 256), (1, 2048), (5, 384), (128, 640), (256, 4224)])
@pytest.mark.parametrize("mode", [fp8.ROWWISE, fp8.COLWISE, fp8.BOTH])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm(monkeypatch, rows, cols, mode, with_residual):
    if mode & fp8.COLWISE and rows % 128:
        pytest.skip("groups along tokens need whole blocks of 128")
    x, r, dy, gamma = tensors(rows, cols)
    res = r if with_residual else None
    seen, a, b = both_ways(monkeypatch, lambda: fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=res, mode=mode))
    assert seen[0] is not None
    same(a, b)
    assert (a[0] is x) == (not with_residual)
    rstd = torch.rand(rows, device=dev())
    seen, a, b = both_ways(monkeypatch, lambda: fp8.fp8_rmsnorm_backward(dy, x, rstd, gamma, res))
    assert seen[0] is not None
    same(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("topk", [0, 7])
@pytest.mark.parametrize("with_targets", [True, False])
def test_logprobs(monkeypatch, dtype, topk, with_targets):
    buf = torch.randn(9, 1003, device=dev()).to(dtype)
    for logits in (buf, buf[:, :1000], buf[:1], buf[:0]):
        targets = torch.arange(logits.shape[0], device=dev()) if with_targets else None
        seen, a, b = both_ways(monkeypatch, lambda: fp8.fp8_token_logprobs(logits, targets, topk=topk))
        assert seen[0] is not None
        same(a, b)
        g = torch.rand(logits.shape[0], device=dev())
        lp = g if with_targets else None
        for h in (None, g):
            seen, c, d = both_ways(monkeypatch, lambda: fp8.fp8_token_logprobs_backward(logits, targets, a[2], lp, a[1], h))
            assert seen[0] is not None
            same(c, d)


def test_given_outputs_come_back(monkeypatch):
    x, r, dy, gamma = tensors(128, 256)
    s, rstd, q = torch.empty_like(x), torch.empty(128, device=dev()), torch.empty(128, 256, dtype=torch.uint8, device=dev())
    seen, a, b = both_ways(monkeypatch, lambda: fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=r, sum_out=s, rstd=rstd, q_row=q))
    assert seen[0] is not None and a[0] is s and a[1] is rstd and a[2] is q and b[0] is s and b[2] is q
    dg = torch.zeros(256, device=dev())
    ws = torch.empty(fp8.fp8_rmsnorm_backward_workspace_bytes(128, 256), dtype=torch.uint8, device=dev())
    seen, a, b = both_ways(monkeypatch, lambda: fp8.fp8_rmsnorm_backward(dy, x, rstd, gamma, dgamma=dg, accumulate=True, workspace=ws))
    assert seen[0] is not None and a[1] is dg and b[1] is dg
    logits, targets = torch.randn(4, 50, device=dev()), torch.zeros(4, dtype=torch.int64, device=dev())
    ti = torch.empty(4, 3, dtype=torch.int64, device=dev())
    seen, a, b = both_ways(monkeypatch, lambda: fp8.fp8_token_logprobs(logits, targets, topk=3, top_index=ti))
    assert seen[0] is not None and a[4] is ti and b[4] is ti
    out = torch.empty(4, 60, device=dev())[:, :50]
    seen, c, d = both_ways(monkeypatch, lambda: fp8.fp8_token_logprobs_backward(logits, targets, a[2], dlogprob=a[0], dlogits=out))
    assert seen[0] is not None and c is out and d is out


def test_refusals_are_alike(monkeypatch):
    x, r, dy, gamma = tensors(130, 256)
    rstd = torch.ones(130, device=dev())
    logits, targets = torch.randn(4, 50, device=dev()), torch.zeros(4, dtype=torch.int64, device=dev())
    stats = torch.zeros(4, 2, device=dev())
    N, B, L, LB = fp8.fp8_add_rmsnorm_quantize_1x128, fp8.fp8_rmsnorm_backward, fp8.fp8_token_logprobs, fp8.fp8_token_logprobs_backward
    calls = [
        lambda: N(x, gamma),                                           # 130 rows in groups along tokens
        lambda: N(x, gamma, mode=7), lambda: N(x, gamma, mode=0), lambda: N(x, gamma, eps=-1.0),
        lambda: N(x.float(), gamma), lambda: N(x[0], gamma), lambda: N(x, gamma[:128]), lambda: N(x, gamma.cpu()),
        lambda: N(x.cpu(), gamma), lambda: N(x[:, :128], gamma[:128], mode=1), lambda: N(x, gamma, residual=r[:1], mode=1),
        lambda: N(x, gamma, sum_out=r, mode=1), lambda: N(x[:, :200].contiguous(), gamma[:200], mode=1),
        lambda: N(x, gamma, mode=1, q_row=torch.empty(130, 256, device=dev())),
        lambda: N(x, gamma, mode=1, rstd=torch.empty(131, device=dev())[1:]),      # not 16-byte aligned
        lambda: N(x, gamma, mode=1, rstd=torch.empty(130)),
        lambda: B(dy, x, rstd.double(), gamma), lambda: B(dy, x, rstd, gamma, accumulate=True),
        lambda: B(dy[:5], x, rstd, gamma), lambda: B(dy, x, rstd, gamma, workspace=torch.empty(16, dtype=torch.uint8, device=dev())),
        lambda: B(dy, x, rstd, gamma, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
        lambda: L(logits.half()), lambda: L(logits, topk=51), lambda: L(logits, topk=-1), lambda: L(logits, topk=33),
        lambda: L(logits.T), lambda: L(logits, targets.int()), lambda: L(logits, targets[:3]), lambda: L(logits.cpu()),
        lambda: L(logits, entropy=torch.empty(5, device=dev())),
        lambda: LB(logits, None, stats, rstd[:4]), lambda: LB(logits, targets, stats, dentropy=rstd[:4]),
        lambda: LB(logits, targets, stats[:3]), lambda: LB(logits, targets, stats, dlogits=logits.bfloat16()),
        lambda: LB(logits, targets, stats, dlogits=logits.T), lambda: LB(logits, targets, stats, dlogits=logits.cpu()),
    ]
    for i, call in enumerate(calls):
        errors = []
        for host in (_abi._host, None):
            with monkeypatch.context() as m:
                m.setattr(_abi, "_host", host)
                with pytest.raises((ValueError, TypeError, fp8.Fp8Error)) as err:
                    call()
                errors.append((type(err.value), getattr(err.value, "status", None), str(err.value)))
        assert errors[0] == errors[1], i


def test_a_stream_given_by_handle():
    x, r, _, gamma = tensors(64, 512)
    want = fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=r, mode=fp8.ROWWISE)
    dy = r.clone()
    grad = fp8.fp8_rmsnorm_backward(dy, want[0], want[1], gamma)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=r, mode=fp8.ROWWISE, stream=st.cuda_stream)
    g2 = fp8.fp8_rmsnorm_backward(dy, got[0], got[1], gamma, stream=st.cuda_stream)
    torch.cuda.synchronize()
    same(want, got)
    same(grad, g2)
    with torch.cuda.stream(st):                                        # the current stream is another one
        same(want, fp8.fp8_add_rmsnorm_quantize_1x128(x, gamma, residual=r, mode=fp8.ROWWISE))
    torch.cuda.synchronize()

