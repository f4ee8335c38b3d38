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


def _check(name, got, ref, bound):
    worst = ((got.double() - ref).abs() / bound.clamp_min(1e-300)).max().item()
    say(f"    {name}: largest error / bound = {worst:.3f}")
    assert got.shape == ref.shape and worst <= 1.0, f"{name}: {worst} times the bound"


def _projection_gradients(x, dY, w, fmt, adapters=(), s=0.0):
    """dX of a projection over the base w from the upstream gradient that it got, and dA, dB of its adapters (first output
    row, A, B): (value, bound) each, in 64 bits.

    dX: the base's product of dY's 8-bit rows (R.product_bound), and each adapter's s (dY B) A with v = dY B off by a
    float32 step per term and 2^-15 left out of s v by its two bf16 terms. dA, dB: float32 operands with all their bits,
    float32 sums over the tokens."""
    T, N = dY.shape
    codes, scales = R.quantize_rows(dY, fmt)
    yh, wh = codes * R.spread_cols(scales, N), R.restored_weight(w.codes, w.scales).t()
    ref, extra, grads = yh @ wh.t(), 0.0, []
    X, lim = x.double(), (T + 8) * 2.0 ** -23
    for row, A, B in adapters:
        Ad, Bd, D = A.detach().double(), B.detach().double(), dY[:, row:row + B.shape[0]].double()
        v, vb = D @ Bd, (N + 4) * 2.0 ** -23 * (D.abs() @ Bd.abs())
        U, ub = X @ Ad.t(), (X.shape[1] + 4) * 2.0 ** -23 * (X.abs() @ Ad.abs().t())
        ref = ref + s * v @ Ad
        lost = 2.0 ** -15 + (2 * 256 + 8) * 2.0 ** -23
        extra = extra + s * (lost * v.abs() + (1 + lost) * vb) @ Ad.abs()
        grads.append(((s * v.t() @ X, s * (lim * v.abs().t() + vb.t()) @ X.abs()),
                      (s * D.t() @ U, s * D.abs().t() @ (lim * U.abs() + ub))))
    return (ref, R.product_bound(yh, wh, ref, extra)), grads


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [R.E4M3, R.E5M2])
@pytest.mark.parametrize("T", [5, 37, 300])
def test_gradients_of_fused_projections(T, fmt):
    """Against the formulas in 64 bits, each projection's adapter from its own rows of the stacked gradient."""
    say(f"fp8 fused gradients T={T} {fmt}")
    g = _gen("fused", T)
    outs = (256, 144, 128)
    f = layer.QLoRAFusedLinear([_randn(g, n, 400) * 0.02 for n in outs], r=24, alpha=32.0, adapted=[True, False, True], base="fp8",
                               generator=g, grad_fmt=fmt)
    with torch.no_grad():
        for B in f.B:
            B.copy_(_randn(g, *B.shape) * 0.05)
    x = _randn(g, T, 400).bfloat16().requires_grad_(True)
    dY = (_randn(g, T, sum(outs)) * torch.exp2(_randn(g, T, 1))).bfloat16()
    torch.cat(f(x), 1).backward(dY)
    (dX, bound), grads = _projection_gradients(x.detach(), dY, f.w, fmt, [(0, f.A[0], f.B[0]), (400, f.A[1], f.B[1])], 32.0 / 24)
    _check("dX", x.grad, dX, bound)
    for k, (a, b) in enumerate(grads):
        _check(f"dA {k}", f.A[k].grad_fp32, *a)
        _check(f"dB {k}", f.B[k].grad_fp32, *b)
        assert torch.equal(f.A[k].grad, f.A[k].grad_fp32.bfloat16()) and torch.equal(f.B[k].grad, f.B[k].grad_fp32.bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [R.E4M3, R.E5M2])
def test_gradients_inside_the_stack(fmt):
    """Every projection and norm of every layer: its gradients against the 64-bit formulas, from the inputs and the upstream
    gradient that it really got."""
    say(f"fp8 stack gradients {fmt}")
    shapes = {"q": (256, 256), "k": (128, 256), "v": (128, 256), "o": (256, 256), "gate": (384, 256), "up": (384, 256), "down": (256, 384)}
    st = stack.DecoderStack(layers=3, shapes=shapes, r=8, seed=5, device=torch.device("cuda:0"), checkpoint=False, head=64, base="fp8",
                            grad_fmt=fmt)
    g = _gen("inside")
    seen = []

    def note(module, args, out):
        ins = [t for t in args if torch.is_tensor(t) and t.requires_grad]
        outs = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None and t.requires_grad]
        for t in (*ins, *outs):
            if not t.is_leaf:
                t.retain_grad()
        seen.append((module, args, ins, out, outs))

    with torch.no_grad():
        for lay in st.layers:
            for B in lay.qkv.B:
                B.copy_(_randn(g, *B.shape) * 0.05)
    for lay in st.layers:
        for m in (lay.qkv, lay.o, lay.gate_up, lay.down, lay.norm):
            m.register_forward_hook(note)
        lay.norm.register_forward_hook(lambda m, a, k, o: seen.append((m, a + (k["residual"],), None, o, None)) if k else None,
                                       with_kwargs=True)
    x = _randn(g, 45, 256).bfloat16().requires_grad_(True)
    st(x).backward(_randn(g, 45, 256).bfloat16())
    checked = 0
    for module, args, ins, out, outs in seen:
        if outs is None or isinstance(module, layer.QLoRARMSNorm):
            continue
        dY = torch.cat([t.grad for t in outs], 1)
        adapters = []
        if isinstance(module, layer.QLoRAFusedLinear) and len(module.A):
            adapters = [(0, module.A[0], module.B[0]), (module.d_outs[0] + module.d_outs[1], module.A[1], module.B[1])]
        (dX, bound), grads = _projection_gradients(args[0].detach(), dY, module.w, fmt, adapters, 16.0 / 8)
        assert len(ins) == 1 and ins[0] is args[0]
        _check(f"dX of {tuple(module.codes.shape)}", ins[0].grad, dX, bound)
        for k, (a, b) in enumerate(grads):
            _check(f"dA {k}", module.A[k].grad_fp32, *a)
            _check(f"dB {k}", module.B[k].grad_fp32, *b)
        checked += 1
    assert checked == 12
    # the norms before the MLPs: dx + ds of the sum, from y's and s's own gradients (the residual's reaches the same sum)
    norms = 0
    for module, args, _, out, outs in seen:
        if not isinstance(module, layer.QLoRARMSNorm) or outs is not None or len(args) < 2:
            continue
        y, s = out[0], out[1]
        sd = s.detach().double().requires_grad_(True)
        yd = sd * torch.rsqrt(sd.square().mean(-1, keepdim=True) + 1e-6)
        dy, ds = y.grad.double(), s.grad.double()
        ref = torch.autograd.grad((yd * dy).sum(), sd)[0] + ds
        # float32 sums of 256 terms of size |dy xh| rstd, then one rounding to bf16
        rstd = torch.rsqrt(sd.detach().square().mean(-1, keepdim=True) + 1e-6)
        xh = (sd.detach() * rstd).abs()
        acc = (256 + 16) * 2.0 ** -23 * (rstd * (dy.abs() + xh * (dy.abs() * xh).mean(-1, keepdim=True)) + ds.abs())
        _check("dx of the norm", args[0].grad, ref, 2.0 ** -8 * (ref.abs() + acc) + acc)
        norms += 1
    assert norms == 3
