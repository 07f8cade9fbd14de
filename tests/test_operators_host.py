"""Refusals and marshalling of the operators around the linears, without a
GPU: bad arguments come back as a status before anything is launched (the fake
pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import blockwise_fp8_pretraining_b200 as fp8

OK, NULL, SHAPE, ALIGN, MODE = 0, 1, 2, 3, 4
A16, MIS = 0x10000, 0x10008
S = ctypes.c_void_p(0)


def P(v):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    from blockwise_fp8_pretraining_b200 import build

    build.build()
    return fp8.load()


def test_limits_match_the_header():
    import re

    from blockwise_fp8_pretraining_b200 import build

    defines = dict(re.findall(r"#define\s+(FP8_\w+)\s+(\d+)", open(build.HEADER).read()))
    assert int(defines["FP8_MAX_NORM_COLS"]) == fp8.MAX_NORM_COLS
    assert int(defines["FP8_MAX_TOPK"]) == fp8.MAX_TOPK


def test_add_rmsnorm_quantize_rejections(lib):
    def call(x=A16, res=A16, rows=256, cols=256, eps=1e-6, gamma=A16, mode=3, s=A16, r=A16, qr=A16, sr=A16, qc=A16,
             sc=A16):
        return lib.fp8_add_rmsnorm_quantize_1x128(P(x), P(res), rows, cols, eps, P(gamma), mode, P(s), P(r), P(qr),
                                                  P(sr), P(qc), P(sc), S)

    for mode in (0, 4, -1):
        assert call(mode=mode) == MODE
    assert call(cols=200) == SHAPE
    assert call(cols=fp8.MAX_NORM_COLS + 128) == SHAPE
    assert call(rows=-1) == SHAPE
    assert call(rows=100) == SHAPE and call(rows=100, mode=2) == SHAPE     # groups along tokens need 128
    assert call(eps=-1.0) == SHAPE and call(eps=float("nan")) == SHAPE and call(eps=float("inf")) == SHAPE
    for name in ("x", "gamma", "s", "r", "qr", "sr", "qc", "sc"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: MIS}) == ALIGN, name
    assert call(res=MIS) == ALIGN
    assert call(rows=0, x=None) == OK and call(cols=0, x=None) == OK


def test_rmsnorm_backward_rejections(lib):
    def call(dy=A16, s=A16, r=A16, g=A16, e=A16, rows=256, cols=256, ds=A16, dg=A16, acc=0, ws=A16, n=1 << 30):
        return lib.fp8_rmsnorm_backward(P(dy), P(s), P(r), P(g), P(e), rows, cols, P(ds), P(dg), acc, P(ws), n, S)

    assert call(acc=2) == MODE
    assert call(cols=100) == SHAPE and call(rows=-1) == SHAPE and call(cols=fp8.MAX_NORM_COLS + 128) == SHAPE
    for name in ("dy", "s", "r", "g", "ds"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: MIS}) == ALIGN, name
    for name in ("e", "dg", "ws"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(cols=0, dy=None) == OK
    assert call(rows=0, dy=None, dg=None) == OK
    assert lib.fp8_rmsnorm_backward_workspace_bytes(128, 128, None) == NULL
    n = ctypes.c_size_t(7)
    assert lib.fp8_rmsnorm_backward_workspace_bytes(128, 100, ctypes.byref(n)) == SHAPE
    assert lib.fp8_rmsnorm_backward_workspace_bytes(0, 128, ctypes.byref(n)) == OK and n.value == 0


def test_binding_refuses_before_the_library(lib):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    g = torch.zeros(256, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fp8.fp8_add_rmsnorm_quantize_1x128(x.float(), g)
    with pytest.raises(ValueError):                  # not on a GPU
        fp8.fp8_add_rmsnorm_quantize_1x128(x, g)
    with pytest.raises(TypeError):
        fp8.fp8_rmsnorm_backward(x, x.float(), torch.zeros(4), g)
    with pytest.raises(ValueError):
        fp8.fp8_rmsnorm_backward(x, x, torch.zeros(4), g)


def test_token_logprobs_rejections(lib):
    def call(x=A16, dtype=0, rows=4, vocab=1000, ld=1000, y=A16, k=5, lp=A16, h=A16, st=A16, tl=A16, ti=A16):
        return lib.fp8_token_logprobs(P(x), dtype, rows, vocab, ld, P(y), k, P(lp), P(h), P(st), P(tl), P(ti), S)

    assert call(dtype=2) == MODE and call(dtype=-1) == MODE
    assert call(rows=-1) == SHAPE and call(vocab=0) == SHAPE and call(ld=999) == SHAPE and call(vocab=1 << 31, ld=1 << 31) == SHAPE
    assert call(ld=(1 << 40) + 1) == SHAPE
    assert call(k=-1) == SHAPE and call(k=fp8.MAX_TOPK + 1) == SHAPE and call(k=6, vocab=5) == SHAPE
    for name in ("x", "st", "y", "tl", "ti"):
        assert call(**{name: None}) == NULL, name
    for name in ("y", "lp", "h", "st", "tl", "ti"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(x=A16 + 1) == ALIGN and call(x=A16 + 2, dtype=1) == ALIGN
    assert call(rows=0, x=None) == OK


def test_token_logprobs_backward_rejections(lib):
    def call(x=A16, dtype=1, rows=4, vocab=1000, ld=1000, y=A16, st=A16, g=A16, H=A16, h=A16, out=A16 + 0x10000, ldo=1000):
        return lib.fp8_token_logprobs_backward(P(x), dtype, rows, vocab, ld, P(y), P(st), P(g), P(H), P(h), P(out), ldo, S)

    assert call(dtype=7) == MODE
    assert call(rows=-1) == SHAPE and call(vocab=0) == SHAPE and call(ld=999) == SHAPE and call(ldo=999) == SHAPE
    assert call(ldo=1008, out=A16) == SHAPE                                 # in place with another stride
    for name in ("x", "st", "out", "y", "H"):
        assert call(**{name: None}) == NULL, name
    for name in ("y", "st", "g", "H", "h"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(x=A16 + 2) == ALIGN and call(out=A16 + 2) == ALIGN
    assert call(rows=0, x=None) == OK


def test_logits_binding_refuses(lib):
    x = torch.zeros(4, 100)
    with pytest.raises(ValueError):                  # not on a GPU
        fp8.fp8_token_logprobs(x)
    with pytest.raises(TypeError):
        fp8.fp8_token_logprobs(x.half())
    with pytest.raises(TypeError):
        fp8.fp8_token_logprobs(x[0])


def test_newton_schulz_rejections(lib):
    def call(g=A16, dtype=1, batch=1, m=64, n=64, coeff=(1.0, 2.0, 3.0), steps=1, eps=0.0, out=A16, ws=A16, size=1 << 40):
        table = (ctypes.c_float * max(1, len(coeff)))(*coeff) if coeff is not None else None
        c = ctypes.cast(table, ctypes.c_void_p) if table is not None else None
        return lib.fp8_newton_schulz(P(g), dtype, batch, m, n, c, steps, eps, P(out), P(ws), size, S)

    assert call(dtype=2) == MODE
    assert call(batch=-1) == SHAPE and call(m=0) == SHAPE and call(n=0) == SHAPE and call(m=32769) == SHAPE
    assert call(batch=4097) == SHAPE and call(steps=0) == SHAPE and call(steps=33) == SHAPE
    assert call(eps=-1.0) == SHAPE and call(eps=float("nan")) == SHAPE
    assert call(coeff=(1.0, float("nan"), 0.0)) == SHAPE and call(coeff=(1.0, 65.0, 0.0)) == SHAPE
    assert call(coeff=None) == NULL
    for name in ("g", "out", "ws"):
        assert call(**{name: None}) == NULL and call(**{name: MIS}) == ALIGN, name
    assert call(size=1024) == SHAPE
    assert call(batch=0, g=None) == OK
    n = ctypes.c_size_t(7)
    assert lib.fp8_newton_schulz_workspace_bytes(1, 64, 64, None) == NULL
    assert lib.fp8_newton_schulz_workspace_bytes(1, 0, 64, ctypes.byref(n)) == SHAPE
    assert lib.fp8_newton_schulz_workspace_bytes(0, 64, 64, ctypes.byref(n)) == OK and n.value == 0
    assert lib.fp8_newton_schulz_workspace_bytes(2, 100, 130, ctypes.byref(n)) == OK
    assert n.value >= 2 * (2 * 100 * 192 + 2 * 100 * 128) * 2


def test_newton_schulz_binding_refuses(lib):
    g = torch.zeros(8, 8)
    with pytest.raises(ValueError):                  # not on a GPU
        fp8.fp8_newton_schulz(g)
    with pytest.raises(TypeError):
        fp8.fp8_newton_schulz(g.half())
    with pytest.raises(TypeError):
        fp8.fp8_newton_schulz(g[0])
