"""The modules between a decoder layer's projections and the stack that runs them together, on the GPU (needs an MI355X).

The modules' results and gradients are the entry points' (held against 64 bits in their own tests), bit for bit where
nothing is added; in the stack every call of the attention is checked against float64 from its actual inputs."""

import zlib

import pytest
import torch

import attention_ref as R
from gpu_common import product, say

pytestmark = pytest.mark.gpu

q_, L, S_ = product("qlora"), product("layer"), product("stack")
HALF = 2.0 ** -8
SHAPES = {"q": (256, 256), "k": (128, 256), "v": (128, 256), "o": (256, 256), "gate": (384, 256), "up": (384, 256),
          "down": (256, 384)}
HEAD = 64


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _bf(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _turn(x, angle, interleaved):
    """x [..., T, H, D] turned by angle [..., T, dim / 2] in float64."""
    n = angle.shape[-1]
    c, s = angle.cos()[..., None, :], angle.sin()[..., None, :]
    x = x.double()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    y = x.clone()
    ya, yb = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = ya, yb
    else:
        y[..., :n], y[..., n:2 * n] = ya, yb
    return y


def _near_turn(got, x, ref):
    """bf16 results: half a step, and 2^-21 of the pair's magnitudes for the float32 arithmetic inside."""
    slack = 2.0 ** -21 * x.double().abs().amax(-1, keepdim=True) * 2
    assert ((got.double() - ref).abs() <= HALF * (ref.abs() + slack) + slack).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_module(interleaved):
    say("rotary module")
    g = _gen("rotary", interleaved)
    m = L.QLoRARotary(48, theta=500.0, interleaved=interleaved)
    m.to(torch.bfloat16)  # a cast leaves the frequencies as they are
    assert m.freqs.dtype == torch.float64
    x = _bf(g, 2, 9, 6 * 64).requires_grad_(True)
    q, k, _ = (t.unflatten(-1, (-1, 64)) for t in torch.split(x, [192, 128, 64], dim=-1))
    dq, dk = _bf(g, 2, 9, 3, 64), _bf(g, 2, 9, 2, 64)
    for positions in (None, torch.randint(0, 4000, (9,), generator=g, device="cuda"),
                      torch.randint(0, 4000, (2, 9), generator=g, device="cuda", dtype=torch.int32)):
        at = torch.arange(9, device="cuda") if positions is None else positions
        angle = at.double()[..., None] * m.freqs
        q2, k2 = m(q, k, positions)
        _near_turn(q2, q, _turn(q, angle, interleaved))
        _near_turn(k2, k, _turn(k, angle, interleaved))
        (gx,) = torch.autograd.grad((q2, k2), x, (dq, dk), retain_graph=True)
        _near_turn(gx[..., :192].unflatten(-1, (3, 64)), dq, _turn(dq, -angle, interleaved))
        _near_turn(gx[..., 192:320].unflatten(-1, (2, 64)), dk, _turn(dk, -angle, interleaved))
        assert not gx[..., 320:].any()
        for part, d in ((0, dq), (1, dk)):  # a gradient of one of them alone
            (one,) = torch.autograd.grad((q2, k2)[part], x, d, retain_graph=True)
            lo, hi = ((0, 192), (192, 320))[part]
            assert torch.equal(one[..., lo:hi], gx[..., lo:hi]) and not one[..., :lo].any() and not one[..., hi:].any()
        (wide,) = torch.autograd.grad(q2, x, torch.ones((), device="cuda").bfloat16().expand(q2.shape), retain_graph=True)
        assert torch.equal(wide, torch.autograd.grad(q2.sum(), x, retain_graph=True)[0])
    alone, none = m(q, None, positions)
    assert none is None and torch.equal(alone, q2)
    # the derivative of the derivative turns forward again
    up = dq.clone().requires_grad_(True)
    (gx,) = torch.autograd.grad(m(q, k, positions)[0], x, up, create_graph=True)
    (again,) = torch.autograd.grad(gx, up, x.detach())
    assert torch.equal(again, m(q, k, positions)[0])
    with pytest.raises(ValueError):
        m(q, k, positions[:, :8])
    with pytest.raises(ValueError):
        m(q, k[:, :8])


@pytest.mark.parametrize("lengths,offsets", [(None, None), ((40, 13), (0, 0)), ((40, 25), (-3, 11))])
def test_attention_module(lengths, offsets):
    say(f"attention module {lengths} {offsets}")
    g = _gen("attention", lengths)
    B, T, H, G, D, window, sinks, scale = 2, 40, 4, 2, 64, 9, 2, 0.2
    x = _bf(g, B, T, (H + 2 * G) * D).requires_grad_(True)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in torch.split(x, [H * D, G * D, G * D], dim=-1))
    m = L.QLoRAAttention(window, sinks, scale)
    n, off = (None if t is None else _ints(*t) for t in (lengths, offsets))
    o = m(q, k, v, n, off)
    want, lse = q_.qlora_attention_forward(q, k, v, window, sinks, scale, n, off, save_lse=True)
    assert torch.equal(o, want)
    do = _bf(g, B, H, T, D).transpose(1, 2)  # heads in front: taken as it lies
    grads = q_.qlora_attention_backward(do, q, k, v, o, lse, window, sinks, scale, n, off)
    (gx,) = torch.autograd.grad(o, x, do, retain_graph=True)
    assert torch.equal(gx, torch.cat([t.flatten(2) for t in grads], 2))
    (gq,) = torch.autograd.grad(o, q, do.transpose(2, 3).contiguous().transpose(2, 3), retain_graph=True)  # copied
    assert torch.equal(gq, grads[0])
    ones = torch.ones(B, T, H, D, device="cuda").bfloat16()
    (gs,) = torch.autograd.grad(o.sum(), x, retain_graph=True)  # an upstream gradient without strides
    assert torch.equal(gs, torch.autograd.grad(o, x, ones, retain_graph=True)[0])
    with torch.no_grad():
        assert torch.equal(m(q, k, v, n, off), want)
        odd = torch.empty(B, T, G, D + 4, device="cuda").bfloat16()[..., :D].copy_(k)  # strides that do not fit: a copy
        assert torch.equal(m(q, odd, v, n, off), want)
    (gk,) = torch.autograd.grad(o, k, do, create_graph=True)
    with pytest.raises(RuntimeError, match="gradients of gradients"):
        gk.sum().backward()
    if n is not None:  # an argument that changes before the backward is noticed
        o = m(q, k, v, n, off)
        n.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            o.sum().backward()


@pytest.mark.parametrize("r,adapted", [(0, None), (8, None), (16, (False, True))])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_module(act, r, adapted):
    say(f"gated module {act} r={r} {adapted}")
    g = _gen("gated", act, r)
    gate, up = _bf(g, 272, 192) * 0.05, _bf(g, 272, 192) * 0.05
    m = L.QLoRAGated(gate, up, r=r, alpha=12.0, adapted=adapted, act=act, generator=g)
    same = L.QLoRAFusedLinear([gate, up], r=r, alpha=12.0, adapted=adapted)
    same.load_state_dict(m.state_dict())  # one state
    assert torch.equal(same.codes, m.codes)
    with torch.no_grad():
        for B in m.B:
            B.copy_(_bf(g, *B.shape) * 0.1)
    for x in (_bf(g, 2, 21, 192), _bf(g, 1, 192)):
        x.requires_grad_(True)
        a = m(x)
        A, B = m.stacked_adapter()
        n = len(m.A)
        alpha = 12.0 * max(n, 1)
        x2 = x.detach().reshape(-1, 192)
        want, h, u = q_.qlora_gated_forward(m.w, x2, A, B, alpha, act, save_h=True, save_u=True)
        assert a.shape == (*x.shape[:-1], 272) and torch.equal(a.reshape(-1, 272), want)
        with torch.no_grad():
            assert torch.equal(m(x), a)
        da = _bf(g, *a.shape)
        dX, dA, dB = q_.qlora_gated_backward(m.w, x2, h, da.reshape(-1, 272), A, B, alpha, act, u_saved=u)
        m.zero_grad()
        x.grad = None
        a.backward(da, retain_graph=True)
        assert torch.equal(x.grad.reshape(-1, 192), dX)
        if r:
            row = {2: (0, 272), 1: (272,)}[n]
            for i in range(n):
                gA, gB = dA[i * r:(i + 1) * r], dB[row[i]:row[i] + 272, i * r:(i + 1) * r]
                assert torch.equal(m.A[i].grad_fp32, gA) and torch.equal(m.A[i].grad, gA.bfloat16())
                assert torch.equal(m.B[i].grad_fp32, gB) and torch.equal(m.B[i].grad, gB.bfloat16())
            a.backward(da, retain_graph=True)
            assert torch.equal(m.B[0].grad_fp32, 2 * dB[row[0]:row[0] + 272, :r])
        (gx,) = torch.autograd.grad(a, x, da, create_graph=True)
        with pytest.raises(RuntimeError, match="gradients of gradients"):
            gx.sum().backward()


def test_gated_module_against_the_formula():
    """x and the adapters' gradients against central differences of the 64-bit product over the restored weights: the
    gradients' own bf16 roundings (of dh, of the adapter's intermediate, of the result) are half steps of the magnitudes
    that enter, taken here as 4 half steps of the products of magnitudes; a step of 2^-10 of a smooth function of O(1)
    arguments is below 2^-14 of them off."""
    say("gated module against differences")
    g = _gen("gated formula")
    d, f, r, T = 64, 32, 8, 3
    m = L.QLoRAGated(_bf(g, f, d) * 0.1, _bf(g, f, d) * 0.1, r=r, alpha=8.0, generator=g)
    with torch.no_grad():
        for B in m.B:
            B.copy_(_bf(g, *B.shape) * 0.1)
    W = q_.qlora_dequantize(m.w).double()
    A, B = ([t.detach().double() for t in p] for p in (m.A, m.B))
    x, da = _bf(g, T, d).requires_grad_(True), _bf(g, T, f)
    (dx,) = torch.autograd.grad(m(x), x, da)

    def loss(xd):
        h = [xd @ W[i * f:(i + 1) * f].t() + xd @ A[i].t() @ B[i].t() for i in range(2)]
        return (h[0] * torch.sigmoid(h[0]) * h[1] * da.double()).sum(-1)

    xd = x.detach().double()
    step = 2.0 ** -10
    ref = torch.stack([(loss(xd + step * e) - loss(xd - step * e)) / (2 * step) for e in torch.eye(d, dtype=torch.float64, device="cuda")], 1)
    h = [xd @ W[i * f:(i + 1) * f].t() + xd @ A[i].t() @ B[i].t() for i in range(2)]
    s = torch.sigmoid(h[0])
    dh = [(da.double() * h[1] * (s + h[0] * s * (1 - s))).abs(), (da.double() * h[0] * s).abs()]
    # (h itself is kept in bf16: half a step of it moves the slopes by at most 1.13 and 1 of it)
    eh = [HALF * t.abs() for t in h]
    moved = [da.double().abs() * (1.13 * eh[1] + h[1].abs() * eh[0]), da.double().abs() * 1.13 * eh[0]]
    size = sum((4 * HALF * dh[i] + 2 * moved[i]) @ (W[i * f:(i + 1) * f].abs() + B[i].abs() @ A[i].abs()) for i in range(2))
    worst = ((dx.double() - ref).abs() / (size + HALF * ref.abs() + 2.0 ** -14 * (1 + ref.abs()))).max().item()
    say(f"    largest error / bound = {worst:.3f}")
    assert worst <= 1.0


# --- the stack ---------------------------------------------------------------

def _stack(**kw):
    st = S_.DecoderStack(layers=2, shapes=SHAPES, r=8, alpha=16.0, seed=11, device="cuda", head=HEAD,
                         **{"attention": True, "window": 24, "sinks": 3, "theta": 1000.0, "gated": "silu", **kw})
    g = _gen("stack")
    with torch.no_grad():
        for layer in st.layers:
            for B in layer.qkv.B:
                B.copy_(_bf(g, *B.shape) * 0.02)
    return st, g


def _watch(st):
    """The inputs and outputs of every call of the layers' modules."""
    calls = {"rotary": [], "attention": [], "gate_up": []}
    for layer in st.layers:
        for name, kept in calls.items():
            getattr(layer, name).register_forward_hook(
                lambda m, args, out, kept=kept: kept.append(([t.detach().clone() if torch.is_tensor(t) else t for t in args], out)))
    return calls


def _check_attention(call, window, sinks):
    (q, k, v, n, off), o = call
    worst = 0.0
    for b in range(q.shape[0]):
        keys = k.shape[1] if n is None else int(n[b])
        first = keys - q.shape[1] if off is None else int(off[b])
        mask = R.seen(q.shape[1], k.shape[1], keys, first, window, sinks)
        for h in range(q.shape[2]):
            g = h * k.shape[2] // q.shape[2]
            ro, _, _, eo, _, _ = R.head(q[b, :, h].double(), k[b, :, g].double(), v[b, :, g].double(), mask, HEAD ** -0.5)
            worst = max(worst, R.worst(o[b, :, h], ro, eo))
    say(f"    attention in the stack: largest error / bound = {worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("T,lengths", [(70, None), (70, (70, 33)), (1, (1, 0))])
def test_a_training_step(T, lengths):
    say(f"stack, a training step T={T} lengths={lengths}")
    st, g = _stack()
    B = 2
    n = None if lengths is None else _ints(*lengths)
    own = torch.ones(B, T, dtype=torch.bool, device="cuda")
    if n is not None:
        own = torch.arange(T, device="cuda")[None] < n[:, None]
    x = _bf(g, B, T, 256).requires_grad_(True)
    dy = _bf(g, B, T, 256) * own[..., None]
    calls = _watch(st)

    def run(x):
        x.grad = None
        st.zero_grad()
        y = st(x, n)
        y.backward(dy)
        return [y.detach(), x.grad.clone()] + [p.grad_fp32.clone() for p in st.parameters()]

    first = run(x)
    assert all(torch.isfinite(t).all() for t in first)
    assert all(t.any() for t in first[2:]) or T == 1  # (over one key the weights are 1: no gradient of q)
    assert len(calls["attention"]) == 4  # two layers, run again in the backward
    for call in calls["attention"][:2]:
        _check_attention(call, 24, 3)
    for (q, k), (q2, k2) in calls["rotary"][:2]:
        angle = torch.arange(T, device="cuda").double()[:, None] * st.layers[0].rotary.freqs
        _near_turn(q2, q, _turn(q, angle, False))
        _near_turn(k2, k, _turn(k, angle, False))
    for layer, ((y,), a) in zip(st.layers, calls["gate_up"][:2]):
        assert torch.equal(a, q_.qlora_gated_forward(layer.gate_up.w, y, None, None, 16.0)[0])
    st.use_checkpoint = False  # what checkpointing keeps has no part in the results
    for a, b in zip(first, run(x)):
        assert torch.equal(a, b)
    # what stands in the padding reaches nothing
    x2 = torch.where(own[..., None], x.detach(), _bf(g, B, T, 256) * 100).requires_grad_(True)
    for a, b in zip(first[:2], run(x2)[:2]):
        assert torch.equal(a[own], b[own])
    if n is None:  # one sequence as it is, and as a batch of one
        a, b = st(x[0]), st(x[:1])
        assert torch.equal(a, b[0]) and a.shape == (T, 256)


def test_the_modules_may_be_mixed():
    say("stack, each operator alone")
    x = _bf(_gen("mixed"), 19, 256)
    plain, _ = _stack(attention=False, window=None, sinks=0, gated=None)
    alone, _ = _stack(attention=False, window=None, sinks=0)
    assert {k: v.shape for k, v in plain.state_dict().items()} == {k: v.shape for k, v in alone.state_dict().items()}
    with torch.no_grad():
        y, z = plain(x), alone(x)
    # the same but for the roundings of gate, up and the activation between
    assert torch.allclose(y.float(), z.float(), rtol=0.05, atol=0.05 * y.float().abs().max().item())
    wide, _ = _stack(gated=None, base="fp8", window=None, sinks=0)
    calls = {"attention": []}
    for layer in wide.layers:
        layer.attention.register_forward_hook(lambda m, args, out: calls["attention"].append(([t.detach() if torch.is_tensor(t) else t for t in args], out.detach())))
    xs = x.clone().requires_grad_(True)
    wide(xs).sum().backward()
    assert torch.isfinite(xs.grad).all() and len(calls["attention"]) == 4
    _check_attention(calls["attention"][0], 1 << 30, 0)
    with pytest.raises(ValueError):
        plain(x, _ints(19))
    with pytest.raises(ValueError):
        plain.caches(1, 8)


def test_a_prompt_and_tokens_behind_it():
    say("stack, prompts of two lengths and tokens behind them")
    st, g = _stack()
    caches = st.caches(2, 64)
    n = _ints(37, 20)
    x = _bf(g, 2, 37, 256)
    with torch.no_grad():
        whole = st(x, n)
        calls = _watch(st)
        y = st(x, n, caches)
        for b in range(2):  # the prompt alone: the same call but for the keys behind it, which are masked
            assert torch.equal(y[b, :n[b]], whole[b, :n[b]])
        turned = [out[1] for _, out in calls["rotary"]]
        for c, k in zip(caches, turned):
            assert c.lengths.tolist() == [37, 20] and c.used == 37
            for b in range(2):
                assert torch.equal(c.k[b, :n[b]], k[b, :n[b]]) and not c.k[b, n[b]:].any()
        for step in range(5):
            for kept in calls.values():
                kept.clear()
            st(_bf(g, 2, 1, 256), None, caches)
            for i, c in enumerate(caches):
                (q, k, _), (q2, k2) = calls["rotary"][i]
                at = _ints(37 + step, 20 + step)
                angle = at.double()[:, None, None] * st.layers[0].rotary.freqs
                _near_turn(k2, k, _turn(k, angle, False))
                assert c.lengths.tolist() == [38 + step, 21 + step]
                for b in range(2):
                    assert torch.equal(c.k[b, at[b]], k2[b, 0])
                _check_attention(calls["attention"][i], 24, 3)
        with pytest.raises(ValueError):
            st(_bf(g, 2, 30, 256), None, caches)
        with pytest.raises(ValueError):
            st(x, None, caches[:1])
    with pytest.raises(RuntimeError):
        st(_bf(g, 2, 1, 256), None, caches)


def test_a_captured_token():
    """A step of one token, captured and replayed with eager work between: the lengths advance on the device; what a replay
    appends to a full cache is dropped."""
    say("stack, a captured token")
    st, g = _stack()
    x = _bf(g, 2, 12, 256)
    steps = [_bf(g, 2, 1, 256) for _ in range(6)]
    with torch.no_grad():
        eager, seen = st.caches(2, 16), []
        st(x, _ints(12, 7), eager)
        for t in steps[:4]:
            seen.append(st(t, None, eager))
        caches = st.caches(2, 16)
        st(x, _ints(12, 7), caches)
        keep = [(c._kv.clone(), c.lengths.clone()) for c in caches]
        token = steps[0].clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            st(token, None, caches)  # (warms the workspaces of this stream)
        torch.cuda.current_stream().wait_stream(stream)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = st(token, None, caches)
        for c, (kv, n) in zip(caches, keep):
            c._kv.copy_(kv)
            c.lengths.copy_(n)
        for i, t in enumerate(steps):
            token.copy_(t)
            graph.replay()
            if i < 4:
                assert torch.equal(y, seen[i])
            torch.cuda.synchronize()
            (x.float() @ x.float().transpose(1, 2)).sum().item()
        for c, e in zip(caches, eager):
            assert c.lengths.tolist() == [16, 13]
            assert torch.equal(c.k[0], e.k[0]) and torch.equal(c.v[1, :11], e.v[1, :11])


def test_a_captured_training_step():
    say("stack, a captured training step")
    st, g = _stack(checkpoint=False)
    n = _ints(50, 31)
    x, dy = _bf(g, 2, 50, 256), _bf(g, 2, 50, 256)
    xs = x.clone().requires_grad_(True)

    def run():
        return torch.autograd.grad(st(xs, n), [xs, *st.parameters()], dy)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = [t.clone() for t in run()]  # (nothing of its graph lives on)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with torch.no_grad():
            st(x, n)


def test_training_moves_the_adapters():
    """The stack with all operators under the library's optimizer: its float32 gradients reach it, it steps, and the next
    step runs."""
    say("stack under the optimizer")
    optim = product("optim")
    st, g = _stack()
    params = [p for p in st.parameters() if p.requires_grad]
    opt = optim.PagedAdamW(params, lr=1e-3)
    x, dy = _bf(g, 2, 33, 256), _bf(g, 2, 33, 256)
    before = [p.detach().clone() for p in params]
    for _ in range(2):
        opt.zero_grad()
        st(x.clone().requires_grad_(True)).backward(dy)
        opt.step()
    torch.cuda.synchronize()
    assert all(not torch.equal(a, b) and torch.isfinite(b).all() for a, b in zip(before, params))


def test_a_cache_that_replays_filled_refuses():
    """After replays have filled a cache a call outside of the graph is refused instead of being dropped; with rows taken
    back it lands behind what the replays appended."""
    say("a cache after replays")
    g = _gen("cache after replays")
    c = L.KeyValueCache(2, 8, 1, 64)
    t = _bf(g, 2, 1, 1, 64)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.append(t, t)
    assert c.used == 0 and c.lengths.tolist() == [0, 0]
    kept = []
    for _ in range(6):
        t.copy_(_bf(g, 2, 1, 1, 64))
        kept.append(t.clone())
        graph.replay()
    c.append(t, t)
    assert c.lengths.tolist() == [7, 7] and c.used == 7
    graph.replay()
    with pytest.raises(ValueError, match="8"):
        c.append(t, t)
    graph.replay()  # dropped
    torch.cuda.synchronize()
    want = torch.cat(kept + [t, t], 1)
    assert torch.equal(c.k, want) and torch.equal(c.v, want) and c.lengths.tolist() == [8, 8]
    c.lengths.copy_(_ints(2, 5))
    new = _bf(g, 2, 3, 1, 64)
    assert c.append(new, new).tolist() == [2, 5] and torch.equal(c.k[0, 2:5], new[0]) and torch.equal(c.k[1, 5:], new[1])
    c.reset()
    graph.replay()
    torch.cuda.synchronize()
    assert c.lengths.tolist() == [1, 1] and torch.equal(c.k[:, :1], t)
