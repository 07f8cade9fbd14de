"""The workspace fp8_newton_schulz asks for: a page where one launch takes the
batch, whatever the GPU; else X in two FP16 parts, twice, and S and Q."""
import ctypes

import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from blockwise_fp8_pretraining_b200 import build

    build.build()
    fp8.load()


ONE_LAUNCH = [(4096, 64, 2048), (4096, 2048, 64), (300, 80, 640), (4096, 128, 128), (1, 128, 2048), (1, 2048, 128), (7, 1, 1),
              (12, 48, 8192), (3, 80, 4992)]
PRODUCTS = [(2, 100, 130), (2, 130, 100), (1, 129, 129), (100, 128, 1000), (5, 81, 129), (2, 1, 8193), (1, 128, 2433),
            (1, 12288, 2048)]


@pytest.mark.parametrize("shape", ONE_LAUNCH)
def test_one_launch_asks_for_a_page(shape):
    assert fp8.fp8_newton_schulz_workspace_bytes(*shape) == 4096


@pytest.mark.parametrize("shape", PRODUCTS)
def test_products_ask_for_their_operands(shape):
    batch, m, n = shape
    s, ld = min(m, n), (n + 63) // 64 * 64
    need = 4 * batch * m * ld * 2 + 2 * batch * s * ((s + 63) // 64 * 64) * 2
    assert need <= fp8.fp8_newton_schulz_workspace_bytes(*shape) <= need + batch * 8192 + (64 << 20)


@pytest.mark.parametrize("shape", ONE_LAUNCH + PRODUCTS)
def test_too_small_a_workspace_is_refused(shape):
    lib, a16 = fp8.load(), ctypes.c_void_p(0x10000)
    table = (ctypes.c_float * 3)(1.5, -0.5, 0.0)
    need = fp8.fp8_newton_schulz_workspace_bytes(*shape)
    assert lib.fp8_newton_schulz(a16, 1, *shape, ctypes.cast(table, ctypes.c_void_p), 1, 1e-7, a16, a16, need - 16, None) == 2


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(300, 64, 500), (40, 80, 640), (1, 128, 2048), (1, 2048, 128), (200, 128, 128), (2, 80, 4992),
                                   (5, 81, 129), (100, 128, 1000), (60, 128, 1024), (36, 1024, 128), (1, 100, 640), (1, 96, 3500)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_workspace_asked_for_is_enough(shape, dtype):
    """Every way a batch may take, and nothing written behind the workspace."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    need = fp8.fp8_newton_schulz_workspace_bytes(*shape)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    out = fp8.fp8_newton_schulz(g, workspace=ws[256:256 + need])
    torch.cuda.synchronize()
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + need:] == 0xA5).all())
    if need == 4096:
        assert bool((ws == 0xA5).all())
    assert torch.equal(out, fp8.fp8_newton_schulz(g))
    x = g[-1].double()
    x = x / (x.norm() + 1e-7)
    for a, b, c in fp8.NEWTON_SCHULZ_COEFFICIENTS:
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    # (the operator's own tests derive the bounds: this is twice the result's own rounding)
    assert float((out[-1].double() - x).norm()) <= 2 * float((x.bfloat16().double() - x).norm())
