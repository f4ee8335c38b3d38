"""Flags that have no truth value: the native marshalling leaves the call to Python, whose error the caller sees."""

import os

import pytest
import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.MARSHAL):
    _build.build()
from bit_quantized_finetuning_amd import qlora as q  # noqa: E402

VAGUE = torch.ones(2)  # a tensor of two values is neither true nor false
X = torch.zeros(3, 16, dtype=torch.bfloat16)
CODES, SCALES = torch.zeros(16, 16, dtype=q.E4M3), torch.zeros(1, 1)


@pytest.mark.parametrize("call", [
    lambda m: m.rmsnorm_forward(X, None, None, 1e-6, VAGUE, 2, False, 0, 0),
    lambda m: m.rmsnorm_forward(X, None, None, 1e-6, True, 2, VAGUE, 0, 0),
    lambda m: m.rmsnorm_backward(X, X, None, torch.zeros(3), None, VAGUE, 0, 0),
    lambda m: m.fp8_forward(CODES, SCALES, 16, 16, X, None, None, 1.0, None, None, 2, VAGUE, None, 0, 0),
    lambda m: m.fp8_backward(CODES, SCALES, 16, 16, X, X, None, None, 1.0, None, VAGUE, False, False, 2, None, 0, 0)])
def test_native_marshalling_leaves_vague_flags_to_python(call):
    assert call(q._marshal) is None


@pytest.mark.gpu
def test_a_vague_flag_raises():
    print("norm with a vague flag", flush=True)
    with pytest.raises(RuntimeError, match="ambiguous"):
        q.qlora_rmsnorm_forward(X.cuda(), want_y=VAGUE, fmt=q.E4M3)
