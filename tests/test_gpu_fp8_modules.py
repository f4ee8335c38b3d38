"""Gradients of the modules over the 8-bit base (needs an MI355X), in both formats of the upstream gradient."""

import zlib

import pytest
import torch

import ops_ref as R
from gpu_common import product, say

q = product("qlora")
layer = product("layer")
stack = product("stack")


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [None, R.E4M3, R.E5M2])
def test_format_of_the_upstream_gradient(fmt):
    say(f"fp8 modules, upstream gradient in {fmt}")
    g = _gen("fmt")
    W = _randn(g, 384, 400) * 0.02
    x, dh = _randn(g, 37, 400).bfloat16(), _randn(g, 37, 384).bfloat16()
    lin = layer.QLoRALinear(W, r=16, base="fp8", generator=_gen("a"), grad_fmt=fmt)
    fused = layer.QLoRAFusedLinear([W[:128], W[128:]], r=8, adapted=[True, False], base="fp8", generator=_gen("b"), grad_fmt=fmt)
    with torch.no_grad():
        lin.B.copy_(_randn(g, 384, 16) * 0.02)
        fused.B[0].copy_(_randn(g, 128, 8) * 0.02)
    for m, A, B in ((lin, lin.A, lin.B), (fused, *fused.stacked_adapter())):
        xg = x.clone().requires_grad_(True)
        h = m(xg)
        (torch.cat(h, 1) if isinstance(h, tuple) else h).backward(dh)
        outs = {f: q.qlora_fp8_backward(m.w, x, dh, A.detach(), B.detach(), 16.0, fmt=f)[0] for f in (R.E4M3, R.E5M2)}
        assert not torch.equal(outs[R.E4M3], outs[R.E5M2])
        assert torch.equal(xg.grad, outs[fmt or R.E4M3])


@pytest.mark.gpu
def test_stack_passes_the_format_on():
    say("fp8 stack, upstream gradients in e5m2")
    shapes = {"q": (256, 256), "k": (128, 256), "v": (128, 256), "o": (256, 256), "gate": (384, 256), "up": (384, 256), "down": (256, 384)}
    grads = []
    for fmt in (None, R.E4M3, R.E5M2):
        st = stack.DecoderStack(layers=2, shapes=shapes, r=8, seed=5, device=torch.device("cuda:0"), head=64, base="fp8", grad_fmt=fmt)
        for lay in st.layers:
            assert all(m.grad_fmt is (fmt or R.E4M3) for m in (lay.qkv, lay.o, lay.gate_up, lay.down))
        x = _randn(_gen("x"), 45, 256).bfloat16().requires_grad_(True)
        st(x).backward(_randn(_gen("dy"), 45, 256).bfloat16())
        grads.append(x.grad)
    assert torch.equal(grads[0], grads[1]) and not torch.equal(grads[0], grads[2])
    assert torch.isfinite(grads[2]).all()


def test_format_is_for_the_eight_bit_base():
    W = torch.zeros(64, 64)
    for make in (lambda **k: layer.QLoRALinear(W, **k), lambda **k: layer.QLoRAFusedLinear([W], **k)):
        with pytest.raises(ValueError, match="grad_fmt"):
            make(base="nf4", grad_fmt=R.E5M2)
        with pytest.raises(TypeError, match="float8"):
            make(base="fp8", grad_fmt=torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_broadcast_and_transposed_inputs(dtype):
    """Rows that overlap or are not dense, as the projections' modules take them: values and gradients of the dense copy."""
    say(f"norm module, broadcast and transposed inputs {dtype}")
    g = _gen("broadcast")
    n = layer.QLoRARMSNorm(64, weight=1 + 0.1 * _randn(g, 64), trainable=True, fmt=R.E4M3)
    row, wide, deep = _randn(g, 1, 1, 64).to(dtype), _randn(g, 64, 5).to(dtype), _randn(g, 3, 64, 5).to(dtype)
    views = ((row, lambda t: t.expand(3, 5, 64)), (wide, lambda t: t.t()), (wide, lambda t: t.t()[::2]),
             (deep, lambda t: t.transpose(1, 2)))
    for src, make in views:
        shape = make(src).shape
        for res in (None, _randn(g, 64).to(dtype).expand(shape)):
            a, b = src.clone().requires_grad_(True), src.clone().requires_grad_(True)
            dy = _randn(g, *shape).to(dtype)
            got = n(make(a), res)
            want = n(make(b).contiguous(), None if res is None else res.contiguous())
            for s, t in zip(got, want):
                assert torch.equal(s, t)
            got[0].backward(dy)
            want[0].backward(dy)
            assert torch.equal(a.grad, b.grad)


@pytest.mark.gpu
def test_gradients_of_gradients_are_refused():
    """The library's backward is not differentiable: a second derivative raises instead of leaving its terms out."""
    say("fp8 modules, second derivatives")
    g = _gen("twice")
    n = layer.QLoRARMSNorm(64, weight=1 + 0.1 * _randn(g, 64))
    lin = layer.QLoRALinear(_randn(g, 64, 64) * 0.02, r=8, base="fp8", generator=g)
    for f in (lambda x: n(x)[0], lin):
        x = _randn(g, 5, 64).bfloat16().requires_grad_(True)
        a = _randn(g, 5, 64).bfloat16().requires_grad_(True)
        # d/dx of a sum over f(x a): a times what the library gives, which itself depends on a
        (dx,) = torch.autograd.grad(f(x * a).float().square().sum(), x, create_graph=True)
        for second in (lambda: torch.autograd.grad(dx.float().square().sum(), a, retain_graph=True), lambda: dx.float().sum().backward()):
            with pytest.raises(RuntimeError, match="gradients of gradients"):
                second()
        a.grad = x.grad = None
        f(x * a).sum().backward(create_graph=True)  # once it is
        first = x.grad.detach().clone()
        x.grad = None
        f(x * a).sum().backward()
        assert torch.isfinite(first).all() and torch.equal(first, x.grad)
