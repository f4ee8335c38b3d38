"""Modules that were saved before there was a choice of base run on the 4-bit one."""

import os

import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.LIB):
    _build.build()
from bit_quantized_finetuning_amd import layer, stack  # noqa: E402


class _Three(torch.nn.Module):
    def forward(self, x):
        return x, x[:, :2], x[:, :2]


class _Two(torch.nn.Module):
    def forward(self, x):
        return x, x


def _restored(cls, **state):
    """A module as unpickling makes it: without __init__, from the attributes that it was saved with."""
    m = cls.__new__(cls)
    torch.nn.Module.__init__(m)
    for k, v in state.items():
        setattr(m, k, v)
    return m


def test_decoder_layer_without_a_base():
    m = _restored(stack.DecoderProjections, hidden=4, kv=2, head=2, qkv=_Three(), o=torch.nn.Identity(), gate_up=_Two(),
                  down=torch.nn.Identity())
    x = torch.randn(5, 4)
    y = m(x)
    q = stack.rms_norm(x)
    a = (q.view(5, 1, 2, 2) * torch.sigmoid(q[:, :2].view(5, 1, 1, 2)) + q[:, :2].view(5, 1, 1, 2)).reshape(5, 4)
    n = stack.rms_norm(x + a)
    torch.testing.assert_close(y, x + a + torch.nn.functional.silu(n) * n)


def test_projections_without_a_base():
    for cls in (layer.QLoRALinear, layer.QLoRAFusedLinear):
        m = _restored(cls, d_w_out=64, d_in=64, codes=torch.zeros(2048, dtype=torch.uint8), qscale=torch.zeros(64, dtype=torch.uint8),
                      smax=torch.zeros(1))
        assert type(m.w) is layer.q.NF4Weight and m.w.codes is m.codes
