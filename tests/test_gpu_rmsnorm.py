"""The root-mean-square norm on the GPU (needs an MI355X): forward with the residual's addition, bf16 / float32 and
8-bit outputs, backward, against 64-bit references; widths around every variant's edge, odd widths, row strides,
unaligned rows, no rows at all."""

import zlib

import pytest
import torch

import ops_ref as R
from gpu_common import product, say

pytestmark = pytest.mark.gpu

q = product("qlora")
WIDTHS = [1, 2, 7, 8, 64, 127, 128, 129, 512, 513, 1000, 1024, 1032, 2048, 2049, 4096, 5120, 6152, 8192, 8200, 16384,
          20001, 32768]
# A row's sum: at most 32 values one after another in a thread, then 6 + 16 additions across lanes and waves
SUM = 64 * 2.0 ** -24


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _x(g, T, d, dtype, pad=0, off=0):
    """[T, d] with rows d + pad apart, starting `off` elements into its memory."""
    buf = _randn(g, T * (d + pad) + off).to(dtype)
    return buf[off:].view(T, d + pad)[:, :d] if T else buf[:0].view(0, d)


def _within(name, got, ref, bound):
    worst = ((got.double() - ref).abs() / bound.clamp_min(1e-300)).max().item() if ref.numel() else 0.0
    say(f"    {name}: largest error / bound = {worst:.3f}")
    assert got.shape == ref.shape and worst <= 1.0, f"{name}: {worst} times the bound"


def _check_forward(o, x, w, res, eps, fmt, dtype):
    s = x if res is None else (x.double() + res.double()).to(dtype)
    if res is not None:
        assert torch.equal(o.s, s)
    sd = s.double()
    rstd = 1 / torch.sqrt(sd.square().mean(-1) + eps)
    _within("rstd", o.rstd, rstd, SUM * rstd)
    y = sd * rstd[:, None] * (1 if w is None else w.double())
    if o.y is not None:
        _within("y", o.y, y, (R.HALF[dtype] + 2 * SUM) * y.abs() + 2.0 ** -133)
    if fmt is not None:
        scale = o.ys.double()
        want = R.row_scales(y, fmt)
        # a scale differs only where the largest value is within the float32 error of a power of two's edge
        near = torch.where(scale == want, 0, 1).bool()
        amax = torch.nn.functional.pad(y.abs(), (0, -y.shape[1] % 128)).view(y.shape[0], -1, 128).amax(-1)
        edge = (amax / R.TOP[fmt] / torch.minimum(scale, want) - 1).abs() <= 4 * SUM
        assert (edge | ~near).all()
        sc = R.spread_cols(scale, y.shape[1])
        v = o.yq.double() * sc
        step = torch.exp2((torch.frexp(y / sc)[1] - 1).clamp_min(R.LOW[fmt]).double() - R.MANT[fmt]) * sc
        _within("yq", v, y, step / 2 + 4 * SUM * y.abs() + 1e-300)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_widths(d, dtype):
    say(f"norm forward d={d} {dtype}")
    for T, fmt, want_y, with_res, wdt in ((1, R.E4M3, False, True, torch.float32), (5, R.E5M2, True, False, torch.bfloat16),
                                          (9, None, True, True, None)):
        g = _gen(d, T)
        x, res = _x(g, T, d, dtype), _x(g, T, d, dtype) if with_res else None
        w = None if wdt is None else (1 + 0.3 * _randn(g, d)).to(wdt)
        o = q.qlora_rmsnorm_forward(x, w, residual=res, eps=1e-5, want_y=want_y, fmt=fmt, save_rstd=True)
        assert (o.y is not None) == want_y and (o.yq is not None) == (fmt is not None) and (o.s is not None) == with_res
        _check_forward(o, x, w, res, 1e-5, fmt, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("d", [256, 515, 4096])
def test_forward_strides(d, pad, off, dtype):
    say(f"norm forward strides d={d} pad={pad} off={off} {dtype}")
    g = _gen(d, pad, off)
    x, res = _x(g, 6, d, dtype, pad, off), _x(g, 6, d, dtype, 0, 1)
    w = _randn(g, d + 1)[1:].contiguous()
    o = q.qlora_rmsnorm_forward(x, w, residual=res, fmt=R.E4M3, save_rstd=True)
    _check_forward(o, x, w, res, 1e-6, R.E4M3, dtype)


def test_rows_of_zeros_and_values_that_are_not_finite():
    say("norm zeros, not finite")
    x = _x(_gen("z"), 4, 1024, torch.bfloat16).clone()
    clean = q.qlora_rmsnorm_forward(x, None, fmt=R.E4M3)
    x[0] = 0
    x[1, 7], x[2, 9] = float("inf"), float("nan")
    o = q.qlora_rmsnorm_forward(x, None, fmt=R.E4M3, save_rstd=True)
    assert (o.y[0] == 0).all() and (o.yq[0].float() == 0).all() and torch.isfinite(o.ys[0]).all()
    assert torch.isnan(o.y[1, 7]) and torch.isnan(o.y[2]).all()
    for r in (1, 2):  # whatever reads the 8-bit row gets values that are not finite
        v = o.yq[r].float() * o.ys[r].repeat_interleave(128)
        assert not torch.isfinite(v).all()
    assert torch.equal(o.y[3], clean.y[3]) and torch.equal(o.yq[3].view(torch.uint8), clean.yq[3].view(torch.uint8))


def test_no_rows():
    say("norm without rows")
    x = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    o = q.qlora_rmsnorm_forward(x, None, residual=x, fmt=R.E4M3, save_rstd=True)
    assert o.y.shape == (0, 100) and o.ys.shape == (0, 1)
    dx, dw = q.qlora_rmsnorm_backward(x, x, None, o.rstd, need_dw=True)
    assert dx.shape == (0, 100) and (dw == 0).all()


def _ref_backward(dy, s, w, rstd, ds):
    dyd, sd, r = dy.double(), s.double(), rstd.double()[:, None]
    g = dyd * (1 if w is None else w.double())
    xh = sd * r
    mean = (g * xh).mean(-1, keepdim=True)
    dx = r * (g - xh * mean)
    mag = r * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.double()
        mag = mag + ds.double().abs()
    return dx, mag, (dyd * xh).sum(0), (dyd * xh).abs().sum(0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", WIDTHS)
def test_backward_widths(d, dtype):
    say(f"norm backward d={d} {dtype}")
    for T, with_ds, wdt, need_dw in ((1, True, torch.float32, True), (37, False, None, True), (11, True, torch.bfloat16, False)):
        g = _gen(d, T)
        s, dy = _x(g, T, d, dtype), _x(g, T, d, dtype)
        ds = _x(g, T, d, dtype) if with_ds else None
        w = None if wdt is None else (1 + 0.3 * _randn(g, d)).to(wdt)
        rstd = torch.rsqrt(s.float().square().mean(-1) + 1e-6)
        dx, dw = q.qlora_rmsnorm_backward(dy, s, w, rstd, ds=ds, need_dw=need_dw)
        rdx, mag, rdw, wmag = _ref_backward(dy, s, w, rstd, ds)
        _within("dx", dx, rdx, R.HALF[dtype] * rdx.abs() + (1 + R.HALF[dtype]) * 2 * SUM * mag)
        if need_dw:
            _within("dw", dw, rdw, (T + 8) * 2.0 ** -24 * wmag)
        else:
            assert dw is None


@pytest.mark.parametrize("T,d", [(2051, 640), (1500, 5120), (700, 333), (4100, 96)])
def test_backward_many_rows_and_strides(T, d):
    say(f"norm backward T={T} d={d} strided")
    g = _gen(T, d)
    s, dy, ds = _x(g, T, d, torch.bfloat16, 8), _x(g, T, d, torch.bfloat16, 16), _x(g, T, d, torch.bfloat16, 0, 1)
    w = 1 + 0.3 * _randn(g, d)
    rstd = torch.rsqrt(s.float().square().mean(-1) + 1e-6)
    dx, dw = q.qlora_rmsnorm_backward(dy, s, w, rstd, ds=ds, need_dw=True)
    rdx, mag, rdw, wmag = _ref_backward(dy, s, w, rstd, ds)
    _within("dx", dx, rdx, R.HALF[torch.bfloat16] * rdx.abs() + (1 + 2.0 ** -8) * 2 * SUM * mag)
    _within("dw", dw, rdw, (T + 8) * 2.0 ** -24 * wmag)
    again = q.qlora_rmsnorm_backward(dy, s, w, rstd, ds=ds, need_dw=True)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_gradient_against_differences():
    """Central differences in 64 bits of sum(c y) + sum(k s), step 1e-4: their own error is 1e-8 of the third
    derivative, below the float32 roundings that the bound counts."""
    say("norm gradient against differences")
    g = _gen("d")
    T, d = 3, 40
    x, res, w, c, k = (_randn(g, *sh) for sh in ((T, d), (T, d), (d,), (T, d), (T, d)))
    o = q.qlora_rmsnorm_forward(x, w, residual=res, eps=1e-6, save_rstd=True)
    dx, dw = q.qlora_rmsnorm_backward(c, o.s, w, o.rstd, ds=k, need_dw=True)

    def loss(s, w):
        return (c.double() * s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-6) * w).sum() + (k.double() * s).sum()

    s, wd, e = o.s.double(), w.double(), 1e-4
    for i in range(T * d):
        u = torch.zeros(T * d, dtype=torch.float64, device="cuda")
        u[i] = e
        u = u.view(T, d)
        num = (loss(s + u, wd) - loss(s - u, wd)) / (2 * e)
        assert abs(num - dx.double().view(-1)[i]) <= 2e-6 * (1 + abs(num)) * 4
    for i in range(d):
        u = torch.zeros(d, dtype=torch.float64, device="cuda")
        u[i] = e
        num = (loss(s, wd + u) - loss(s, wd - u)) / (2 * e)
        assert abs(num - dw.double()[i]) <= 2e-6 * (1 + abs(num)) * 4


def test_captured_norm():
    say("norm graph")
    g = _gen("g")
    x, res, w, dy = _x(g, 33, 2560, torch.bfloat16), _x(g, 33, 2560, torch.bfloat16), _randn(g, 2560), _x(g, 33, 2560, torch.bfloat16)

    def call():
        o = q.qlora_rmsnorm_forward(x, w, residual=res, fmt=R.E4M3, save_rstd=True)
        return tuple(o) + q.qlora_rmsnorm_backward(dy, o.s, w, o.rstd, ds=dy, need_dw=True)

    call()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = call()
    for _ in range(3):
        x.copy_(_x(g, 33, 2560, torch.bfloat16))
        want = call()
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a.float(), b.float())


class _Refuses:
    def __getattr__(self, name):
        return lambda *a: None


def test_python_and_native_marshalling_agree(monkeypatch):
    say("norm python marshalling")
    g = _gen("m")
    x, res, w, dy = _x(g, 7, 515, torch.bfloat16, 3, 1), _x(g, 7, 515, torch.bfloat16), _randn(g, 515), _x(g, 7, 515, torch.bfloat16)
    runs = []
    for native in (True, False):
        if not native:
            monkeypatch.setattr(q, "_marshal", _Refuses())
        o = q.qlora_rmsnorm_forward(x, w, residual=res, fmt=R.E5M2, save_rstd=True)
        runs.append(tuple(o) + q.qlora_rmsnorm_backward(dy, o.s, w, o.rstd, ds=dy, need_dw=True))
    for a, b in zip(*runs):
        assert torch.equal(a.float(), b.float())


def test_many_rows_and_far_apart():
    """More rows than one launch takes, rows past 2^31 bytes, and a row stride of 2^22 elements."""
    T, d = (1 << 20) + 3, 1032
    say(f"norm {T}x{d}")
    g = _gen("many")
    x, res = (torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = 1 + 0.3 * _randn(g, d)
    o = q.qlora_rmsnorm_forward(x, w, residual=res, fmt=R.E4M3, save_rstd=True)
    dx, _ = q.qlora_rmsnorm_backward(x, o.s, w, o.rstd, ds=res)
    dx2, dw = q.qlora_rmsnorm_backward(x, o.s, w, o.rstd, ds=res, need_dw=True)
    assert torch.equal(dx, dx2)
    at = torch.tensor([0, 1, T // 2, T - 5, T - 4, T - 3, T - 2, T - 1], device="cuda")
    some = q.RMSNormOut(*(t[at] for t in o))
    _check_forward(some, x[at], w, res[at], 1e-6, R.E4M3, torch.bfloat16)
    ref, mag, _, _ = _ref_backward(x[at], some.s, w, some.rstd, res[at])
    _within("dx", dx[at], ref, (R.HALF[torch.bfloat16] + 4 * SUM) * mag)
    total = torch.zeros(2, d, dtype=torch.float64, device="cuda")
    for i in range(0, T, 1 << 17):
        p = x[i:i + (1 << 17)].double() * (o.s[i:i + (1 << 17)].double() * o.rstd[i:i + (1 << 17), None].double())
        total += torch.stack([p.sum(0), p.abs().sum(0)])
    _within("dw", dw, total[0], (T + 8) * 2.0 ** -23 * total[1])
    del x, res, o, dx, dx2
    far = torch.empty(600 << 22, dtype=torch.bfloat16, device="cuda").view(600, 1 << 22)[:, :520]
    far.copy_(_randn(g, 600, 520))
    a = q.qlora_rmsnorm_forward(far, None, save_rstd=True)
    b = q.qlora_rmsnorm_forward(far.contiguous(), None, save_rstd=True)
    assert torch.equal(a.y, b.y) and torch.equal(a.rstd, b.rstd)


@pytest.mark.parametrize("fmt", [R.E4M3, R.E5M2])
@pytest.mark.parametrize("d", [4096, 777])
def test_largest_values_where_the_scale_doubles(d, fmt):
    """Each group's largest value within a few float32 steps of the format's largest times a power of two: the scale is
    that of the value before its roundings. (The squares are powers of four, so their float32 sums are exact.)"""
    say(f"norm edge d={d} {fmt}")
    g = _gen("edge", d)
    wrong = 0
    for T in range(20):
        x = torch.exp2(torch.randint(-2, 3, (1, d), generator=g, device="cuda").float())
        rstd = 1 / (x.double().square().mean() + 1e-6).sqrt()
        w = torch.rand(d, generator=g, device="cuda") * 2.0 ** -6
        at = torch.arange(0, d, 128, device="cuda") + 5
        off = 1 + (torch.rand(len(at), generator=g, device="cuda").double() - 0.5) * 2.0 ** -21
        w[at] = (R.TOP[fmt] * 2.0 ** -9 * off / (x[0, at].double() * rstd)).float()
        y = x.double() * rstd * w.double()
        o = q.qlora_rmsnorm_forward(x, w, eps=1e-6, want_y=False, fmt=fmt)
        assert torch.equal(o.ys.double(), R.row_scales(y, fmt).double())
        assert torch.isfinite(o.yq.float()).all()
        wrong += (R.row_scales((x * rstd.float() * w).double(), fmt).double() != o.ys.double()).sum().item()
    say(f"    scales that float32 alone would have got wrong: {wrong}")
