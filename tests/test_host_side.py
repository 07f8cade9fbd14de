"""The binding's compiled host side, without a GPU: it is built beside the
library and loaded, leaves every call on tensors that are not on a GPU to the
Python checks, and refuses a wrong number of arguments."""
import pytest
import torch

from blockwise_fp8_pretraining_b200 import _abi, build


@pytest.fixture(scope="module")
def host():
    build.build()
    _abi.load()
    assert _abi._host is not None
    return _abi._host


def test_calls_off_the_gpu_are_left_to_python(host):
    x, g, r = torch.zeros(4, 256).bfloat16(), torch.zeros(256).bfloat16(), torch.zeros(4)
    none = [None] * 7
    assert host.add_rmsnorm_quantize(x, g, None, 1e-6, 1, *none[:6]) is None
    assert host.rmsnorm_backward(x, x, r, g, None, None, None, False, None) is None
    assert host.token_logprobs(torch.zeros(4, 9), None, 0, *none[:5]) is None
    assert host.token_logprobs_backward(torch.zeros(4, 9), None, torch.zeros(4, 2), *none[:4]) is None


@pytest.mark.parametrize("what", [None, 3, "x", [1.0], object()])
def test_other_objects_are_left_to_python(host, what):
    assert host.add_rmsnorm_quantize(what, None, None, 1e-6, 1, None, None, None, None, None, None) is None
    assert host.rmsnorm_backward(None, what, None, None, None, None, None, False, None) is None
    assert host.token_logprobs(what, None, 0, None, None, None, None, None) is None
    assert host.token_logprobs_backward(what, None, None, None, None, None, None) is None


def test_argument_counts(host):
    for f in (host.add_rmsnorm_quantize, host.rmsnorm_backward, host.token_logprobs, host.token_logprobs_backward, host.bind):
        with pytest.raises(TypeError):
            f()
        with pytest.raises(TypeError):
            f(*range(20))
