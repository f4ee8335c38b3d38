"""AdamW over many tensors on the GPU (needs an MI355X): moments in 32 and in 8 bits, float32 and bf16 gradients and
parameters, the clip to a global norm, sizes around a block, empty tensors, more tensors than one launch takes,
against 64-bit references; what lies between tensors, norms that are not finite, capture into a graph."""

import zlib

import pytest
import torch

import ops_ref as R
from gpu_common import product, say

pytestmark = pytest.mark.gpu

q = product("qlora")
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
SIZES = {
    "edges": [1, 255, 0, 256, 257, 511, 1000, 3],
    "one": [100_003],
    "many": [64 + 7 * i for i in range(300)],  # three launches of the step, two of the norm
    "middle": [100 + 5 * i for i in range(200)],  # two launches and one
    "empty": [0, 0],
    "none": [],
}


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _flat_of(g, sizes, fill):
    """Flat float32 values, and a mask of the places that belong to a tensor."""
    total = q.adamw_state_elements(sizes)
    t, real = torch.full((total,), fill, device="cuda"), torch.zeros(total, dtype=torch.bool, device="cuda")
    o = 0
    for n in sizes:
        t[o:o + n] = torch.randn(n, generator=g, device="cuda")
        real[o:o + n] = True
        o += R.padded(n)
    return t, real


class Setup:
    def __init__(self, sizes, bits, grad, param, key, pad=0.0):
        g = _gen(key)
        self.sizes = sizes
        self.grads = [(torch.randn(n, generator=g, device="cuda") * 1e-2).to(grad) for n in sizes]
        flat, self.real = _flat_of(g, sizes, pad)
        flat = torch.where(self.real, flat * 0.02, flat)
        offs = [0]
        for n in sizes:
            offs.append(offs[-1] + R.padded(n))
        self.offs = offs
        self.master = flat if param is torch.bfloat16 else None
        self.params = [flat[o:o + n].to(param).clone() for o, n in zip(offs, sizes)]
        m, _ = _flat_of(g, sizes, pad)
        v, _ = _flat_of(g, sizes, pad)
        m, v = m * 3e-3, (v * 1e-2).square()
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = m, v
        else:
            def held(t):
                if not t.numel():
                    return t.to(R.E4M3), t
                sc = t.view(-1, 256).abs().amax(-1).clamp_min(R.TINY) / 448
                return (t.view(-1, 256) / sc[:, None]).clamp(-448, 448).to(R.E4M3).view(-1), sc
            self.m, self.ms = held(m)
            self.v, self.vs = held(v.sqrt())
        self.bits = bits

    def clone(self):
        import copy
        return copy.deepcopy(self)

    def values(self):
        """p, m, v, grads flat in float64, zero outside the tensors."""
        if self.bits == 32:
            m, v = self.m.double(), self.v.double()
        else:
            m = self.m.double() * self.ms.double().repeat_interleave(256)
            v = (self.v.double() * self.vs.double().repeat_interleave(256)).square()
        z = torch.zeros((), dtype=torch.float64, device="cuda")
        p = self.master.double() if self.master is not None else (
            R.flat(self.params) if self.sizes else torch.zeros(0, dtype=torch.float64, device="cuda"))
        g = R.flat(self.grads) if self.sizes else p
        return torch.where(self.real, p, z), torch.where(self.real, m, z), torch.where(self.real, v, z), g

    def step(self, k, **kw):
        return q.qlora_adamw_many(k, self.grads, self.params, self.m, self.v, self.ms, self.vs, master=self.master, **{**HP, **kw})


def _within(name, got, ref, bound):
    worst = ((got.double() - ref).abs() / bound).max().item() if ref.numel() else 0.0
    say(f"    {name}: largest error / bound = {worst:.3f}")
    assert worst <= 1.0, f"{name}: {worst} times the bound"


@pytest.mark.parametrize("clip", [None, 0.05])
@pytest.mark.parametrize("param", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("which", list(SIZES))
def test_step(which, bits, grad, param, clip):
    say(f"adamw many {which} bits={bits} grad={grad} param={param} clip={clip}")
    step, seed = 7, 123
    s = Setup(SIZES[which], bits, grad, param, which)
    p, m, v, g = s.values()
    norm = s.step(step, max_norm=clip, seed=seed)
    rp, rm, rv, rn = R.adamw(step, g, p, m, v, **HP, max_norm=clip)
    if clip is None:
        assert norm is None
    else:
        assert abs(norm.item() - rn.item()) <= 2.0 ** -23 * rn.item() + 1e-30
    u = 2.0 ** -24
    c = 1.0 if clip is None else min(1.0, clip / (rn.item() + 1e-6))
    # float32: a product or sum costs u of its result. g c: 4u (the norm, the quotient, the product). m: its terms'
    # magnitudes once more each. v = the squares: twice g's.
    mb = 8 * u * (0.9 * m.abs() + 0.1 * (c * g).abs()) + 1e-37
    vb = 14 * u * rv + 1e-37
    b1c, b2c = 1 - 0.9 ** step, 1 - 0.999 ** step
    den = (rv / b2c).sqrt() + HP["eps"]
    ub = (mb + 24 * u * rm.abs()) / b1c / den
    pb = HP["lr"] * ub + 4 * u * (p.abs() + rp.abs()) + 1e-37
    got_p = s.master if s.master is not None else (R.flat(s.params) if s.sizes else p)
    _within("p", torch.where(s.real, got_p.double(), 0.0), torch.where(s.real, rp, 0.0), pb)
    if param is torch.bfloat16:
        for o, n, t in zip(s.offs, s.sizes, s.params):
            assert torch.equal(t, s.master[o:o + n].bfloat16())
    if bits == 32:
        _within("m", s.m, torch.where(s.real, rm, 0.0), mb)
        _within("v", s.v, torch.where(s.real, rv, 0.0), vb)
        return
    bits_ = R.random_bits(p.numel(), seed, step, "cuda")
    for name, codes, scale, t, tb, r in (("m", s.m, s.ms, rm, mb, bits_ & 0xFFFF), ("v", s.v, s.vs, rv.sqrt(), 8 * u * rv.sqrt() + 1e-37, bits_ >> 16)):
        t = torch.where(s.real, t, 0.0)
        if not t.numel():
            continue
        amax = t.view(-1, 256).abs().amax(-1).clamp_min(R.TINY)
        _within(name + " scale", scale, amax / 448, (tb.view(-1, 256).amax(-1) + 2 * u * amax) / 448)
        x = t.abs() * (448 / amax).repeat_interleave(256)
        want, ulp = R.round_up_or_down(x, r)
        if name == "v":
            want = torch.where((x > 0) & (want == 0), 2.0 ** -9, want)
        got = codes.double().abs()
        # one grid step at most (the least code for a root that would round to zero), and the same choice but where
        # the value and its random bits are within the float32 error of the border
        assert ((got - x).abs() <= ulp * (1 + 1e-4) + 1e-12).all(), name
        assert (codes.double() * t >= 0).all()
        differ = (got != want).double().mean().item()
        say(f"    {name}: {differ:.2e} of the codes differ")
        assert differ <= 1e-3 + 2 / got.numel()


@pytest.mark.parametrize("bits", [8, 32])
def test_what_lies_between_tensors_is_left_alone(bits):
    """Other bytes in the padding neither change nor reach a scale."""
    say(f"adamw many padding bits={bits}")
    sizes = [1, 255, 257, 300]
    a, b = Setup(sizes, bits, torch.float32, torch.bfloat16, "p"), Setup(sizes, bits, torch.float32, torch.bfloat16, "p")
    for t in (b.m, b.v) if bits == 32 else (b.m.view(torch.uint8), b.v.view(torch.uint8)):
        t[~b.real] = 0x7E if bits == 8 else 1e30
    b.master[~b.real] = 5.0
    a.step(3, max_norm=1.0)
    b.step(3, max_norm=1.0)
    for x, y in ((a.m, b.m), (a.v, b.v), (a.master, b.master)):
        x, y = (t.view(torch.uint8) if t.dtype is R.E4M3 else t for t in (x, y))
        assert torch.equal(x[a.real], y[b.real])
    assert (b.master[~b.real] == 5.0).all()
    pad = b.m.view(torch.uint8)[~b.real] if bits == 8 else b.m[~b.real]
    assert (pad == (0x7E if bits == 8 else 1e30)).all()
    if bits == 8:
        assert torch.equal(a.ms, b.ms) and torch.equal(a.vs, b.vs)


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_norm_that_is_not_finite_changes_nothing(bits, bad):
    say(f"adamw many not finite bits={bits} {bad}")
    s = Setup([300, 1000], bits, torch.float32, torch.bfloat16, "n")
    before = s.clone()
    s.grads[1][77] = bad
    norm = s.step(2, max_norm=1.0)
    assert not torch.isfinite(norm).any()
    for a, b in ((s.m, before.m), (s.v, before.v), (s.master, before.master), (s.params[0], before.params[0]), (s.params[1], before.params[1])):
        assert torch.equal(a.float(), b.float())


def test_norm_of_large_and_small_gradients():
    """Squares that leave float32's range: the norm is summed in 64 bits."""
    say("adamw many norm range")
    for size in (1e25, 1e-25):
        s = Setup([1000, 50], 32, torch.float32, torch.float32, "r")
        s.grads = [torch.full((n,), size, device="cuda") for n in s.sizes]
        norm = s.step(1, max_norm=1.0)
        assert abs(norm.item() / (size * 1050 ** 0.5) - 1) < 1e-6
        assert all(torch.isfinite(p).all() for p in s.params)


def test_same_seed_same_bits_and_other_seed_other_bits():
    say("adamw many seeds")
    runs = []
    for seed in (5, 5, 6):
        s = Setup([5000], 8, torch.float32, torch.bfloat16, "s")
        s.step(4, seed=seed)
        runs.append(s)
    assert torch.equal(runs[0].m.view(torch.uint8), runs[1].m.view(torch.uint8))
    assert not torch.equal(runs[0].m.view(torch.uint8), runs[2].m.view(torch.uint8))


def test_rounding_is_unbiased():
    """400 seeds of one step: the mean of the stored root is the root itself. Each stored value is within a grid step
    (at most 1/8 of the value, normal range) of it, so the mean's standard deviation is below 1/8 / 2 / sqrt(400) of
    it; six of those allowed. Rounding to nearest would be off by up to 1/16 everywhere."""
    say("adamw many unbiased")
    acc = 0
    for seed in range(400):
        s = Setup([256 * 8], 8, torch.float32, torch.bfloat16, "u")
        if seed == 0:
            p, m, v, g = s.values()
            _, _, rv, _ = R.adamw(9, g, p, m, v, **HP)
        s.step(9, seed=seed)
        acc = acc + s.v.double() * s.vs.double().repeat_interleave(256)
    root = rv.sqrt()
    amax = root.view(-1, 256).amax(-1).repeat_interleave(256)
    big = root > amax / 1000
    assert ((acc / 400 / root - 1).abs()[big] <= 6 / 16 / 20).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_step(bits):
    say(f"adamw many graph bits={bits}")
    a = Setup([1000, 77, 4096], bits, torch.bfloat16, torch.bfloat16, "g")
    b = a.clone()
    warm = a.clone()
    warm.step(5, max_norm=0.01)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        norm = b.step(5, max_norm=0.01)
    for k in range(3):
        for s, t in zip(a.grads, b.grads):
            s.mul_(-0.5)
            t.copy_(s)
        want = a.step(5, max_norm=0.01)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, norm), k
        for x, y in ((a.m, b.m), (a.v, b.v), (a.master, b.master)):
            assert torch.equal(x.float(), y.float()), k


@pytest.mark.parametrize("clip", [None, 0.01])
@pytest.mark.parametrize("missing", [[0], [1, 2], [4], [0, 2, 4], [0, 1, 2, 3, 4]])
def test_tensors_without_a_gradient_are_left_alone(missing, clip):
    """The others get what they get in a call of their own (32-bit moments: nothing depends on the place)."""
    say(f"adamw many without gradients {missing} clip={clip}")
    sizes = [300, 5000, 256, 0, 777]
    a = Setup(sizes, 32, torch.float32, torch.bfloat16, "h")
    before = a.clone()
    for i in missing:
        a.grads[i] = None
    a.step(3, max_norm=clip)
    b = before.clone()
    here = [i for i in range(5) if i not in missing]
    if here:
        cut = lambda t: torch.cat([t[b.offs[i]:b.offs[i] + R.padded(sizes[i])] for i in here])  # noqa: E731
        m, v, master = cut(b.m), cut(b.v), cut(b.master)
        q.qlora_adamw_many(3, [b.grads[i] for i in here], [b.params[i] for i in here], m, v, master=master, max_norm=clip, **HP)
        assert torch.equal(cut(a.m), m) and torch.equal(cut(a.v), v) and torch.equal(cut(a.master), master)
    for i in range(5):
        o = slice(a.offs[i], a.offs[i] + sizes[i])
        if i in missing:
            assert torch.equal(a.m[o], before.m[o]) and torch.equal(a.master[o], before.master[o])
            assert torch.equal(a.params[i], before.params[i])
        else:
            assert torch.equal(a.params[i], b.params[i])


def test_python_and_native_marshalling_agree(monkeypatch):
    say("adamw many python marshalling")
    runs = []
    for native in (True, False):
        if not native:
            monkeypatch.setattr(q, "_marshal", _Refuses())
        s = Setup(SIZES["edges"], 8, torch.float32, torch.bfloat16, "m")
        s.grads[4] = None
        norm = s.step(4, max_norm=0.05, seed=3)
        runs.append((s.m.view(torch.uint8), s.v.view(torch.uint8), s.ms, s.vs, s.master, norm, *s.params))
    for x, y in zip(*runs):
        assert torch.equal(x, y)


class _Refuses:
    def __getattr__(self, name):
        return lambda *a: None


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_past_32_bit_places(bits):
    """A tensor of more than 2^31 elements and one after it: their last elements as in a call on those alone. (8-bit
    moments round by their place, so their own bits are compared in steps of the format: at most one apart.)"""
    say(f"adamw {bits}-bit past 32 bits")
    n, tail = (1 << 31) + 300, 256 + 300
    total = q.adamw_state_elements([n, 1000])
    g = _gen("huge", bits)
    grads = [torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16), _randn16(g, 1000)]
    params = [torch.randn(n, generator=g, device="cuda"), torch.randn(1000, generator=g, device="cuda")]
    cut = n - tail
    small = q.adamw_state_elements([tail, 1000])
    few_p, few_g = [params[0][cut:].clone(), params[1].clone()], [grads[0][cut:].clone(), grads[1]]
    if bits == 32:
        state = [torch.rand(total, generator=g, device="cuda") for _ in range(2)]
        few = [t[cut:].clone() for t in state]
        scales, few_scales = [None, None], [None, None]
    else:
        state = [torch.randint(0, 120, (total,), generator=g, device="cuda", dtype=torch.uint8).view(R.E4M3) for _ in range(2)]
        scales = [torch.rand(total // 256, generator=g, device="cuda") * 1e-4 for _ in range(2)]
        few = [t[cut:].clone() for t in state]
        few_scales = [t[cut // 256:].clone() for t in scales]
    assert few[0].numel() == small
    q.qlora_adamw_many(3, grads, params, *state, *scales, **HP)
    q.qlora_adamw_many(3, few_g, few_p, *few, *few_scales, **HP)
    assert torch.equal(params[0][cut:], few_p[0]) and torch.equal(params[1], few_p[1])
    for a, b, sa, sb in zip(state, few, scales, few_scales):
        a = a[cut:]
        if bits == 32:
            assert torch.equal(a, b)
            continue
        assert torch.equal(sa[cut // 256:], sb)
        # the codes of e4m3 of one sign are in order: neighbours differ by one (a zero's sign aside)
        x, y = (torch.where(t >= 128, -(t.int() & 127), t.int()) for t in (a.view(torch.uint8), b.view(torch.uint8)))
        assert ((x - y).abs() <= 1).all()


def _randn16(g, n):
    return torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)
