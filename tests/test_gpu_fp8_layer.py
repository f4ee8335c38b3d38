"""The modules over the 8-bit base (needs an MI355X): QLoRALinear and QLoRAFusedLinear with base="fp8", QLoRARMSNorm,
the decoder stack with base="fp8", FlatAdamW; and one training step of them together, every stage against a 64-bit
reference of that stage on the inputs it really got."""

import zlib

import pytest
import torch

import ops_ref as R
from gpu_common import product, say

pytestmark = pytest.mark.gpu

q = product("qlora")
layer = product("layer")
optim = product("optim")
stack = product("stack")


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _check(name, got, ref, bound):
    worst = ((got.double() - ref).abs() / bound.clamp_min(1e-300)).max().item()
    say(f"    {name}: largest error / bound = {worst:.3f}")
    assert got.shape == ref.shape and worst <= 1.0, f"{name}: {worst} times the bound"


def _product_ref(xq, xs, w, u=None, B=None, s=0.0):
    """Value and bound of one projection: 8-bit rows, base, and the adapter's s u B^T (u as the kernel had it)."""
    xh, wh = xq.double() * R.spread_cols(xs, xq.shape[1]), R.restored_weight(w.codes, w.scales)
    ref, extra = xh @ wh.t(), 0.0
    if u is not None:
        ref = ref + s * u.double() @ B.double().t()
        extra = s * (2.0 ** -8 + (u.shape[1] + 4) * 2.0 ** -23) * u.double().abs() @ B.double().abs().t()
    return ref, R.product_bound(xh, wh, ref, extra)


@pytest.mark.parametrize("freeze_A", [False, True])
@pytest.mark.parametrize("recompute_u", [False, True])
def test_linear_is_the_calls(freeze_A, recompute_u):
    say(f"fp8 linear freeze_A={freeze_A} recompute_u={recompute_u}")
    g = _gen("lin")
    m = layer.QLoRALinear(_randn(g, 272, 400) * 0.02, r=16, alpha=32.0, freeze_A=freeze_A, recompute_u=recompute_u, base="fp8",
                          generator=g)
    with torch.no_grad():
        m.B.copy_(_randn(g, 272, 16) * 0.02)
    x = _randn(g, 3, 11, 400).bfloat16().requires_grad_(True)
    dh = _randn(g, 3, 11, 272).bfloat16()
    m(x).backward(dh)
    x2, dh2 = x.detach().view(-1, 400), dh.view(-1, 272)
    h, u = q.qlora_fp8_forward(m.w, x2, m.A, m.B, 32.0, save_u=True)
    dX, dA, dB = q.qlora_fp8_backward(m.w, x2, dh2, m.A, m.B, 32.0, u_saved=u)
    assert torch.equal(m(x).detach().view(-1, 272), h) and torch.equal(x.grad.view(-1, 400), dX)
    assert torch.equal(m.B.grad_fp32, dB) and torch.equal(m.B.grad, dB.bfloat16())
    assert (m.A.grad is None) if freeze_A else torch.equal(m.A.grad_fp32, dA)
    assert not any(b.requires_grad for b in m.buffers())
    with pytest.raises(ValueError, match="4-bit"):
        m.merged_weight()
    with pytest.raises(ValueError, match="base"):
        layer.QLoRALinear(torch.zeros(64, 64, device="cuda"), base="int3")


def test_eight_bit_rows_are_for_the_eight_bit_base():
    g = _gen("rows")
    m = layer.QLoRALinear(_randn(g, 64, 128), r=0)
    x = _randn(g, 4, 128).bfloat16()
    with pytest.raises(ValueError, match="8-bit"):
        m(x, *q.qlora_fp8_quantize_rows(x))


def test_casts_and_state_dict_keep_the_base():
    say("fp8 casts, state dict")
    g = _gen("sd")
    m = layer.QLoRALinear(_randn(g, 128, 256), r=8, base="fp8", generator=g).half()
    assert m.codes.dtype is R.E4M3 and m.scales.dtype is torch.float32 and m.A.dtype is torch.bfloat16
    other = layer.QLoRALinear(_randn(g, 128, 256), r=8, base="fp8", generator=g)
    other.load_state_dict(m.state_dict())
    x = _randn(g, 5, 256).bfloat16()
    assert torch.equal(m(x), other(x))


def test_fused_projections_equal_single_ones():
    """Each d_out a multiple of 128: the stacked quantization is each projection's own."""
    say("fp8 fused")
    g = _gen("fused")
    ws = [_randn(g, n, 256).bfloat16() for n in (256, 128, 128)]
    f = layer.QLoRAFusedLinear(ws, r=8, adapted=[True, False, True], base="fp8", generator=_gen("f"))
    with torch.no_grad():
        for B in f.B:
            B.copy_(_randn(g, *B.shape) * 0.02)
    x = _randn(g, 37, 256).bfloat16()
    outs = f(x, *q.qlora_fp8_quantize_rows(x))
    k = 0
    for w, o, ad in zip(ws, outs, (True, False, True)):
        one = q.qlora_fp8_quantize(w)
        if not ad:
            assert torch.equal(o, q.qlora_fp8_forward(one, x, None, None, 1.0)[0])
            continue
        xq, xs = q.qlora_fp8_quantize_rows(x)
        A, B = f.A[k].detach(), f.B[k].detach()
        u = (x.double() @ A.double().t()).float()
        ref, bound = _product_ref(xq, xs, one, u, B, 16.0 / 8)
        _check("fused", o, ref, bound)
        k += 1


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("uses", ["y", "s", "both"])
def test_norm_module_gradients(with_residual, uses):
    """Against 64-bit autograd of the formula, on the stored sum."""
    if uses != "y" and not with_residual:
        return  # s is x itself: nothing of the module
    say(f"norm module residual={with_residual} uses={uses}")
    g = _gen("norm", with_residual, uses)
    d = 640
    n = layer.QLoRARMSNorm(d, weight=1 + 0.2 * _randn(g, d), trainable=True, fmt=R.E4M3)
    x = _randn(g, 2, 9, d).bfloat16().requires_grad_(True)
    r = _randn(g, 2, 9, d).bfloat16().requires_grad_(True) if with_residual else None
    y, s, yq, ys = n(x, r)
    assert not yq.requires_grad and yq.shape == (18, d) and ys.shape == (18, 5)
    cy, cs = _randn(g, 2, 9, d).bfloat16(), _randn(g, 2, 9, d).bfloat16()
    loss = 0
    if uses != "s":
        loss = loss + (y * cy).float().sum()
    if uses != "y":
        loss = loss + (s * cs).float().sum()
    loss.backward()
    sd = s.detach().double().requires_grad_(True)
    w = n.weight.detach().double().requires_grad_(True)
    yd = sd * torch.rsqrt(sd.square().mean(-1, keepdim=True) + 1e-6) * w
    ref = 0
    if uses != "s":
        ref = ref + (yd * cy.double()).sum()
    if uses != "y":
        ref = ref + (sd * cs.double()).sum()
    ref.backward()
    # one bf16 rounding of the result, float32 sums before it (their terms are within 8 of each other here)
    bound = 2.0 ** -8 * sd.grad.abs() + 2.0 ** -16 * (sd.grad.abs().amax(-1, keepdim=True) + 1)
    _check("dx", x.grad, sd.grad, bound)
    if with_residual:
        assert torch.equal(x.grad, r.grad)
    if uses == "s":
        assert n.weight.grad is None
    else:
        _check("dw", n.weight.grad, w.grad, 2.0 ** -17 * (cy.double() * yd.detach()).abs().sum((0, 1)) + 1e-6)


def test_one_training_step_of_all_of_them():
    """residual add + norm -> 8-bit rows -> projection with adapter -> loss -> backward -> clipped 8-bit AdamW."""
    say("fp8 training step")
    T, d, N, r, alpha = 70, 1040, 528, 16, 32.0
    g = _gen("step")
    lin = layer.QLoRALinear(_randn(g, N, d) * 0.02, r=r, alpha=alpha, base="fp8", generator=g)
    norm = layer.QLoRARMSNorm(d, weight=1 + 0.1 * _randn(g, d), fmt=R.E4M3)
    with torch.no_grad():
        lin.B.copy_(_randn(g, N, r) * 0.02)
    x, res = _randn(g, T, d).bfloat16().requires_grad_(True), _randn(g, T, d).bfloat16()
    y, s, yq, ys = norm(x, res)
    h = lin(y, yq, ys)
    c = (_randn(g, T, N) * 1e-2).bfloat16()
    opt = optim.FlatAdamW([lin.A, lin.B], lr=1e-2, weight_decay=0.1, bits=8, max_norm=0.5, seed=9)
    A0, B0 = lin.A.detach().clone(), lin.B.detach().clone()
    (h.float() * c.float()).sum().backward()
    # forward
    assert torch.equal(s, (x.detach().double() + res.double()).bfloat16())
    u = (y.detach().double() @ A0.double().t()).float()
    ref, bound = _product_ref(yq, ys, lin.w, u, B0, alpha / r)
    _check("h", h.detach(), ref, bound)
    # backward: the gradients of the adapter from y and c, then x's from the projection's dX
    dA = alpha / r * (c.double() @ B0.double()).t() @ y.detach().double()
    dB = alpha / r * c.double().t() @ (y.detach().double() @ A0.double().t())
    mags = alpha / r * (c.double().abs() @ B0.double().abs()).t() @ y.detach().double().abs()
    _check("dA", lin.A.grad_fp32, dA, 2.0 ** -13 * mags)
    _check("dB", lin.B.grad_fp32, dB, 2.0 ** -13 * alpha / r * c.double().abs().t() @ (y.detach().double().abs() @ A0.double().abs().t()))
    dY, _, _ = q.qlora_fp8_backward(lin.w, y.detach(), c, A0, B0, alpha)
    dx, _ = q.qlora_rmsnorm_backward(dY, s.detach(), norm.weight, 1 / torch.sqrt(s.detach().double().square().mean(-1) + 1e-6).float())
    assert ((x.grad.double() - dx.double()).abs() <= 2.0 ** -7 * dx.double().abs() + 1e-6).all()
    # the step
    grads = R.flat([lin.A.grad_fp32, lin.B.grad_fp32])
    p0 = R.flat([A0, B0])
    opt.step()
    zero = torch.zeros_like(p0)
    rp, rm, rv, rn = R.adamw(1, grads, p0, zero, zero, 1e-2, 0.9, 0.999, 1e-8, 0.1, max_norm=0.5)
    assert abs(opt.norm.item() / rn.item() - 1) <= 2.0 ** -22
    # the first step's update is lr g / (|g| + eps'): where g is far above eps its size is lr
    _check("p", opt.master, rp, 1e-2 * 2.0 ** -18 + 4 * 2.0 ** -24 * p0.abs() + 1e-2 * 1e-3 * (grads.abs() < 1e-5).double())
    n = lin.A.numel()
    assert torch.equal(lin.A.detach().reshape(-1), opt.master[:n].bfloat16())
    assert torch.equal(lin.B.detach().reshape(-1), opt.master[R.padded(n):R.padded(n) + lin.B.numel()].bfloat16())


SHAPES = {"q": (256, 256), "k": (128, 256), "v": (128, 256), "o": (256, 256), "gate": (384, 256), "up": (384, 256),
          "down": (256, 384)}


def _stack(checkpoint):
    st = stack.DecoderStack(layers=3, shapes=SHAPES, r=8, alpha=16.0, seed=5, device=torch.device("cuda:0"),
                            checkpoint=checkpoint, head=64, base="fp8")
    g = _gen("stack")
    with torch.no_grad():
        for lay in st.layers:
            for B in lay.qkv.B:
                B.copy_(_randn(g, *B.shape) * 0.02)
    return st, _randn(g, 45, 256).bfloat16().requires_grad_(True), _randn(g, 45, 256).bfloat16()


def test_stack_runs_and_checkpointing_changes_nothing():
    say("fp8 stack")
    runs = []
    for checkpoint in (False, True):
        st, x, dy = _stack(checkpoint)
        seen = []
        hook = st.layers[1].gate_up.register_forward_hook(lambda m, a, o: seen.append((a, o)))
        y = st(x)
        y.backward(dy)
        hook.remove()
        assert torch.isfinite(y).all()
        # gate/up of the middle layer from exactly the 8-bit rows that its norm wrote
        (n, nq, ns), (gate, up) = seen[0]
        codes, scales = R.quantize_rows(n.detach(), R.E4M3)
        off = (nq.double() * R.spread_cols(ns, 256) - n.detach().double()).abs()
        assert (off <= (2.0 ** -4 + 2.0 ** -7) * n.detach().double().abs() + 2.0 ** -9 * R.spread_cols(ns, 256)).all()
        ref, bound = _product_ref(nq, ns, st.layers[1].gate_up.w)
        _check("gate/up", torch.cat([gate, up], 1).detach(), ref, bound)
        runs.append([y.detach(), x.grad] + [p.grad_fp32 for lay in st.layers for p in (*lay.qkv.A, *lay.qkv.B)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [8, 32])
def test_flat_adamw(bits):
    """Several steps with a parameter whose gradient is missing once; the state survives a save and a load."""
    say(f"flat adamw bits={bits}")
    g = _gen("flat", bits)
    mk = lambda: [torch.nn.Parameter(p.clone()) for p in start]  # noqa: E731
    start = [(_randn(g, n) * 0.02).bfloat16() for n in (300, 4096, 77)]
    grads = [[(_randn(g, p.numel()) * 1e-2).bfloat16() for p in start] for _ in range(4)]
    grads[2][1] = None

    def run(params, opt, ks):
        for k in ks:
            for p, gr in zip(params, grads[k]):
                p.grad, p.grad_fp32 = gr, None if gr is None else gr.float()
            opt.step()
            opt.zero_grad()

    a = mk()
    oa = optim.FlatAdamW(a, lr=1e-3, bits=bits, max_norm=0.1, seed=4)
    run(a, oa, range(4))
    b = mk()
    ob = optim.FlatAdamW(b, lr=1e-3, bits=bits, max_norm=0.1, seed=4)
    run(b, ob, range(2))
    c = [torch.nn.Parameter(p.detach().clone()) for p in b]
    oc = optim.FlatAdamW(c, lr=1e-3, bits=bits, max_norm=0.1, seed=4)
    oc.load_state_dict({k: v.clone() if torch.is_tensor(v) else v for k, v in ob.state_dict().items()})
    run(c, oc, range(2, 4))
    for x, y in zip(a, c):
        assert torch.equal(x, y)
    # 64-bit reference, the second parameter left out of the third step
    p, m, v = R.flat(start), 0 * R.flat(start), 0 * R.flat(start)
    real = R.flat([torch.ones_like(s) for s in start]).bool()
    second = torch.zeros_like(real)
    second[512:512 + 4096] = True
    for k in range(4):
        gk = R.flat([torch.zeros_like(s) if gr is None else gr for s, gr in zip(start, grads[k])])
        np_, nm, nv, _ = R.adamw(k + 1, gk, p, m, v, 1e-3, 0.9, 0.999, 1e-8, 0.0, max_norm=0.1)
        keep = second if k == 2 else torch.zeros_like(real)
        p, m, v = torch.where(keep, p, np_), torch.where(keep, m, nm), torch.where(keep, v, nv)
    # 32 bits: float32 roundings, at most 2^-16 of the update's size over four steps. 8 bits: m is off by at most an
    # eighth of itself (or the least code of its block, far below what moves p) per step, sqrt(v) too, so an update of
    # size lr by at most 2/7 + 2/7 ... of it: three of the four steps read rounded moments
    lim = 4e-3 * 2.0 ** -16 if bits == 32 else 3 * 1e-3 * 1.5
    got = oa.master.double()
    assert ((got - p).abs()[real] <= lim + 2.0 ** -22 * p.abs()[real]).all()
    if bits == 8:
        assert (got - p).norm() <= 0.1 * (p - R.flat(start)).norm()


def test_flat_adamw_refuses():
    with pytest.raises(ValueError):
        optim.FlatAdamW([torch.nn.Parameter(torch.zeros(4, device="cuda"), requires_grad=False)])
    with pytest.raises(ValueError):
        optim.FlatAdamW([torch.nn.Parameter(torch.zeros(4, device="cuda"))], bits=4)
    with pytest.raises(TypeError):
        optim.FlatAdamW([torch.nn.Parameter(torch.zeros(4, device="cuda").half())])
    with pytest.raises(TypeError):
        optim.FlatAdamW([torch.nn.Parameter(torch.zeros(4, device="cuda")), torch.nn.Parameter(torch.zeros(4, device="cuda").bfloat16())])
    a = optim.FlatAdamW([torch.nn.Parameter(torch.zeros(4, device="cuda"))], bits=8)
    b = optim.FlatAdamW([torch.nn.Parameter(torch.zeros(400, device="cuda"))], bits=8)
    with pytest.raises(ValueError):
        b.load_state_dict(a.state_dict())
