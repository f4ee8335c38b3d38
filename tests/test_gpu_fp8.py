"""The 8-bit frozen base on the GPU (needs an MI355X): the quantizers bit for bit, the forward and backward against
64-bit references within bounds counted from the formats, cut blocks, single tokens, any finite scales, values that
are not finite, rows past the last token, streams, and calls captured into a graph."""

import zlib

import pytest
import torch

import ops_ref as R
from gpu_common import product, say

pytestmark = pytest.mark.gpu

q = product("qlora")
FMTS = [R.E4M3, R.E5M2]


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, T, d):
    x = _randn(g, T, d) * torch.exp2(torch.randint(-6, 7, (T, 1), generator=g, device="cuda").float())
    return (x * (1 + 15 * (torch.rand(d, generator=g, device="cuda") < 0.02))).bfloat16()


def _weight(g, N, K, scales="amax"):
    w = q.qlora_fp8_quantize(_randn(g, N, K) * 0.02)
    if scales == "any":  # a checkpoint's own: of any size and sign, some zero
        s = _randn(g, *w.scales.shape) * 1e-3
        s[torch.rand(s.shape, generator=g, device="cuda") < 0.1] = 0
        w.scales.copy_(s)
    return w


def _adapter(g, N, K, r):
    if not r:
        return None, None
    return (_randn(g, r, K) * 0.02).bfloat16(), (_randn(g, N, r) * 0.02).bfloat16()


def _check(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    worst = ((got - ref).abs() / bound.clamp_min(1e-300)).max().item()
    say(f"    {name}: largest error / bound = {worst:.3f}")
    assert worst <= 1.0, f"{name}: {worst} times the bound"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 128), (3, 144), (7, 2048), (5, 2064), (33, 5120)])
def test_quantize_rows_bit_exact(T, d, dtype, fmt):
    say(f"fp8 rows {T}x{d} {dtype} {fmt}")
    g = _gen(T, d)
    x = _rows(g, T, d).to(dtype)
    if dtype is torch.float32:
        x = x + _randn(g, T, d) * 1e-3
    x[0, : min(d, 128)] = 0  # a group of zeros
    xq, xs = q.qlora_fp8_quantize_rows(x, fmt)
    codes, scales = R.quantize_rows(x, fmt)
    assert torch.equal(xs.double(), scales)
    assert torch.equal(xq.double(), codes)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_rows_extremes(fmt):
    """The largest values of a binade on both sides of 1.75, subnormal bf16, the largest finite value."""
    say(f"fp8 rows extremes {fmt}")
    x = torch.zeros(6, 128, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 1.75, 1.75 + 2.0 ** -22, 1.9999
    x[3, 0], x[3, 1] = 2.0 ** -133, -(2.0 ** -130)
    x[4, 0], x[4, 1] = 3.3895313892515355e38, -1e30
    x[5] = torch.linspace(-448, 448, 128, device="cuda")
    xq, xs = q.qlora_fp8_quantize_rows(x, fmt)
    codes, scales = R.quantize_rows(x, fmt)
    assert torch.equal(xs.double(), scales) and torch.equal(xq.double(), codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 272), (400, 1040)])
def test_quantize_weight(N, K, dtype):
    """scale = amax / 448 to one float32 rounding; every code is the nearest value of w * (448 / amax), up to the two
    float32 roundings of that product (a code may fall on the other side of a tie only when the exact quotient is
    within 2^-22 of it)."""
    say(f"fp8 weight {N}x{K} {dtype}")
    W = (_randn(_gen(N, K), N, K) * 0.02).to(dtype)
    w = q.qlora_fp8_quantize(W)
    amax = R.block_amax(W)
    assert ((w.scales.double() - amax / 448).abs() <= 2.0 ** -24 * amax / 448).all()
    x = W.double() * (448 / amax).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp_min(-6).double() - 3)
    assert ((w.codes.double() - x).abs() <= step / 2 + 2.0 ** -22 * x.abs()).all()


SHAPES = [  # T, d_out, d_in, r
    (1, 16, 16, 0), (1, 128, 128, 8), (1, 1040, 2064, 16), (2, 400, 144, 24), (15, 256, 512, 0), (16, 1024, 1024, 64),
    (17, 272, 400, 8), (33, 528, 1296, 16), (64, 256, 256, 256), (65, 128, 4096, 8), (100, 640, 784, 40),
    (255, 256, 384, 0), (256, 512, 512, 16), (257, 784, 656, 64), (515, 1808, 1040, 8), (1030, 272, 2576, 0),
]


# tokens, outputs, contracted width: large tiles of 256 outputs x 256, 192 and 128 tokens and of 192 x 192, whole and with
# their last round cut into K ranges
LARGE = [(776, 5168, 288), (3166, 2608, 256), (2964, 4560, 256), (201, 13520, 4720), (1031, 15136, 2704),
         (1781, 13696, 3344), (1204, 14208, 4800), (325, 10960, 3104), (519, 14048, 528), (518, 13248, 272),
         (206, 8496, 4784), (212, 8240, 4224), (263, 14240, 272), (780, 9936, 272), (582, 13392, 528), (2160, 8176, 2560),
         (1937, 8960, 3824), (976, 10832, 272), (1296, 3104, 4688), (1060, 14352, 2176), (515, 13824, 400),
         (516, 13552, 16), (535, 13344, 144), (198, 16416, 16), (195, 17344, 144), (399, 16496, 16), (581, 16432, 144)]


@pytest.mark.parametrize("T,N,K", LARGE)
def test_forward_large(T, N, K):
    test_forward(T, N, K, 16, True)


@pytest.mark.parametrize("T,K,N", LARGE)
def test_backward_large(T, N, K):
    test_backward(T, N, K, 16)


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("T,N,K,r", SHAPES)
def test_forward(T, N, K, r, given):
    fmt = FMTS[(T + N // 16) % 2]
    say(f"fp8 forward T={T} {N}x{K} r={r} {fmt} given={given}")
    g = _gen(T, N, K, r, given)
    w = _weight(g, N, K, "any" if given else "amax")
    x = _rows(g, T, K)
    A, B = _adapter(g, N, K, r)
    xq, xs = q.qlora_fp8_quantize_rows(x, fmt)
    if given:  # scales of any kind
        xs = xs * (0.5 + torch.rand(xs.shape, generator=g, device="cuda"))
    big = torch.full((T + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    h, u = q.qlora_fp8_forward(w, x, A, B, 16.0, xq=xq if given else None, xs=xs if given else None, fmt=fmt,
                               save_u=True, h=big[:T])
    assert h.data_ptr() == big.data_ptr() and (big[T:] == 7).all()
    xh, wh = xq.double() * R.spread_cols(xs, K), R.restored_weight(w.codes, w.scales)
    ref, extra = xh @ wh.t(), 0.0
    if r:
        s = 16.0 / r
        uref = x.double() @ A.double().t()
        umag = x.double().abs() @ A.double().abs().t()
        # u: float32 sums of exact products; s u is rounded to bf16 (half a step) before its product with B
        ubound = (K + 4) * 2.0 ** -23 * umag
        _check("u", u, uref, ubound)
        ref = ref + s * uref @ B.double().t()
        extra = s * ((2.0 ** -8 * uref.abs() + (1 + 2.0 ** -8) * ubound) @ B.double().abs().t()
                     + (r + 4) * 2.0 ** -23 * uref.abs() @ B.double().abs().t())
    else:
        assert u is None
    _check("h", h, ref, R.product_bound(xh, wh, ref, extra))
    h2, _ = q.qlora_fp8_forward(w, x, A, B, 16.0, xq=xq if given else None, xs=xs if given else None, fmt=fmt)
    assert torch.equal(h2, h)


@pytest.mark.parametrize("T,N,K,r", SHAPES)
def test_backward(T, N, K, r):
    fmt = FMTS[(T + K // 16) % 2]
    say(f"fp8 backward T={T} {N}x{K} r={r} {fmt}")
    g = _gen(T, N, K, r, "b")
    w = _weight(g, N, K, "any")
    x, dY = _rows(g, T, K), _rows(g, T, N)
    A, B = _adapter(g, N, K, r)
    big = torch.full((T + 2, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dX, dA, dB = q.qlora_fp8_backward(w, x, dY, A, B, 16.0, fmt=fmt, dX=big[:T])
    assert (big[T:] == 7).all()
    codes, scales = R.quantize_rows(dY, fmt)
    yh, wh = codes * R.spread_cols(scales, N), R.restored_weight(w.codes, w.scales).t()
    ref, extra = yh @ wh.t(), 0.0
    if r:
        s, D, Bd, Ad, X = 16.0 / r, dY.double(), B.double(), A.double(), x.double()
        v, vb = D @ Bd, (N + 4) * 2.0 ** -23 * (D.abs() @ Bd.abs())
        ref = ref + s * v @ Ad
        extra = s * ((2.0 ** -8 * v.abs() + (1 + 2.0 ** -8) * vb) @ Ad.abs() + (r + 4) * 2.0 ** -23 * v.abs() @ Ad.abs())
        # dA, dB: a float32 operand enters the matrix units as three bf16 terms (24 bits), float32 sums over the tokens
        lim = (T + 8) * 2.0 ** -23
        _check("dA", dA, s * v.t() @ X, s * (lim * v.abs().t() + vb.t()) @ X.abs())
        U, ub = X @ Ad.t(), (K + 4) * 2.0 ** -23 * (X.abs() @ Ad.abs().t())
        _check("dB", dB, s * D.t() @ U, s * D.abs().t() @ (lim * U.abs() + ub))
    else:
        assert dA is None and dB is None
    _check("dX", dX, ref, R.product_bound(yh, wh, ref, extra))


@pytest.mark.parametrize("T,N,K,r", [(1, 16, 272, 8), (2, 528, 16, 16), (5, 1040, 784, 24), (33, 256, 512, 64),
                                     (40, 272, 144, 72), (64, 144, 1040, 128), (65, 784, 400, 136), (97, 512, 256, 256)])
def test_adapter_gradients_keep_float32(T, N, K, r):
    """The intermediates enter with all their bits. u is given, in float32. v = dY B has 24 bits by construction: each
    column of B holds 1, 2^-8 and 2^-16 at three rows, and each sum over dY's values there is exact in float32."""
    say(f"fp8 adapter gradients T={T} {N}x{K} r={r}")
    g = _gen(T, N, K, r, "keep")
    w = _weight(g, N, K)
    x, u = _rows(g, T, K), _randn(g, T, r)
    dY = ((128 + torch.randint(0, 128, (T, N), generator=g, device="cuda")) / 256.0).bfloat16()  # 1/2 .. 1, 8 bits
    B = torch.zeros(N, r, device="cuda")
    for j in range(r):
        for i, at in enumerate(torch.randperm(N, generator=g, device="cuda")[:3].tolist()):
            B[at, j] = 2.0 ** (-8 * i)
    A, B = _adapter(g, N, K, r)[0], B.bfloat16()
    v = dY.double() @ B.double()
    assert torch.equal(v.float().double(), v)
    s = 32.0 / r
    # three terms leave at most 2^-25 of a value behind; T sums, the scale and its product, one step each
    lim = s * (T + 4) * 2.0 ** -23
    for want in ("both", "dA", "dB"):
        _, dA, dB = q.qlora_fp8_backward(w, x, dY, A, B, 32.0, u_saved=u, need_dx=False, need_dA=want != "dB", need_dB=want != "dA")
        if want != "dB":
            _check(f"dA ({want})", dA, s * v.t() @ x.double(), lim * v.abs().t() @ x.double().abs())
        else:
            assert dA is None
        if want != "dA":
            _check(f"dB ({want})", dB, s * dY.double().t() @ u.double(), lim * dY.double().abs().t() @ u.double().abs())
        else:
            assert dB is None


@pytest.mark.parametrize("T,r", [(40, 8), (300, 64)])
def test_adapter_gradients_of_the_largest_values(T, r):
    """u at the end of float32's range, infinite and NaN: products as the formula has them, in their own column only."""
    say(f"fp8 adapter gradients, large values T={T} r={r}")
    g = _gen("large", T)
    N = K = 272
    w, x = _weight(g, N, K), _rows(g, T, K)
    A, B = _adapter(g, N, K, r)
    dY = torch.exp2(torch.randint(-12, -8, (T, N), generator=g, device="cuda").float()).bfloat16()
    u = _randn(g, T, r)
    plain = q.qlora_fp8_backward(w, x, dY, A, B, float(r), u_saved=u, need_dx=False, need_dA=False)[2]
    u[:, 1] = 0
    u[3, 1] = torch.finfo(torch.float32).max
    u[5, 2] = float("inf")
    u[7, 4] = float("nan")
    dB = q.qlora_fp8_backward(w, x, dY, A, B, float(r), u_saved=u, need_dx=False, need_dA=False)[2]
    assert torch.equal(dB[:, 1], u[3, 1] * dY[3].float())  # a power of two times it: exact
    assert (dB[:, 2] == float("inf")).all() and torch.isnan(dB[:, 4]).all()
    rest = [j for j in range(r) if j not in (1, 2, 4)]
    assert torch.equal(dB[:, rest], plain[:, rest])


@pytest.mark.parametrize("fmt", FMTS)
def test_what_the_matrix_unit_keeps(fmt):
    """A large product and its negative beside a small one: among the same eight k the small one survives down to
    2^-13 of the large one, in another eight down to 2^-23 at least. Every bound on a product here rests on it."""
    say(f"fp8 matrix unit {fmt}")
    for place in range(128):
        if place in (3, 5):
            continue
        n = 13 if place < 8 else 23
        small = 16 - n
        x, w = torch.zeros(16, 128, device="cuda"), torch.zeros(16, 128, device="cuda")
        x[:, 3], w[:, 3], x[:, 5], w[:, 5] = 256, 256, 256, -256
        x[:, place], w[:, place] = 2.0 ** (small // 2), 2.0 ** (small - small // 2)
        h, _ = q.qlora_fp8_forward(q.Fp8Weight(16, 128, w.to(R.E4M3), torch.ones(1, 1, device="cuda")), None, None, None,
                                   1.0, xq=x.to(fmt), xs=torch.ones(16, 1, device="cuda"), fmt=fmt)
        assert (h == 2.0 ** small).all(), place


def test_adapter_gradients_against_differences():
    """The loss sum(c * h) is bilinear in A and B: central differences of it in 64 bits are exact but for rounding."""
    say("fp8 gradients against differences")
    T, N, K, r = 20, 48, 80, 8
    g = _gen("diff")
    w = _weight(g, N, K)
    x, c = _rows(g, T, K), _randn(g, T, N).bfloat16()
    A, B = _adapter(g, N, K, r)
    dX, dA, dB = q.qlora_fp8_backward(w, x, c, A, B, 16.0)
    xd, cd, wh = x.double(), c.double(), R.restored_weight(w.codes, w.scales)

    def loss(A, B, x=xd):
        return (cd * (x @ wh.t() + 16.0 / r * (x @ A.t()) @ B.t())).sum()

    Ad, Bd = A.double(), B.double()
    for k in range(12):
        dirA, dirB = torch.randn_like(Ad), torch.randn_like(Bd)
        da = (loss(Ad + dirA, Bd) - loss(Ad - dirA, Bd)) / 2
        db = (loss(Ad, Bd + dirB) - loss(Ad, Bd - dirB)) / 2
        mag_a = ((cd.abs() @ Bd.abs()).t() @ xd.abs() * 2 * dirA.abs()).sum()
        mag_b = (cd.abs().t() @ (xd.abs() @ Ad.abs().t()) * 2 * dirB.abs()).sum()
        assert abs(da - (dA.double() * dirA).sum()) <= 2.0 ** -15 * mag_a
        assert abs(db - (dB.double() * dirB).sum()) <= 2.0 ** -15 * mag_b
        # in x: the base sees the gradient in 8 bits (half a step, 2^-4), the result is rounded to bf16 (2^-8)
        dirx = torch.randn_like(xd)
        dx = (loss(Ad, Bd, xd + dirx) - loss(Ad, Bd, xd - dirx)) / 2
        lim = (2.0 ** -4 + 2.0 ** -10) * (cd.abs() @ wh.abs() * dirx.abs()).sum()
        lim = lim + 2.0 ** -7 * (((cd.abs() @ Bd.abs()) @ Ad.abs() * 2 + cd.abs() @ wh.abs()) * dirx.abs()).sum()
        assert abs(dx - (dX.double() * dirx).sum()) <= lim


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_values_that_are_not_finite_stay_in_their_rows(T):
    say(f"fp8 not finite T={T}")
    N, K = 272, 400
    g = _gen("nan", T)
    w = _weight(g, N, K)
    x = _rows(g, T, K)
    clean, _ = q.qlora_fp8_forward(w, x, None, None, 1.0)
    bad = x.clone()
    bad[T // 2, 5] = float("nan")
    bad[T - 1, 300] = float("inf")
    h, _ = q.qlora_fp8_forward(w, bad, None, None, 1.0)
    rows = sorted({T // 2, T - 1})
    assert not torch.isfinite(h[rows]).any()
    keep = [t for t in range(T) if t not in rows]
    assert torch.equal(h[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 70])
def test_codes_of_nan_past_a_cut_block_are_not_read(T):
    """d_in = 144: the second block holds 16 columns; what follows a row in memory (the next row's codes, here NaN
    rows) does not reach it."""
    say(f"fp8 cut block T={T}")
    N, K = 64, 144
    g = _gen("cut", T)
    w = _weight(g, N, K)
    x = _rows(g, T, K)
    clean, _ = q.qlora_fp8_forward(w, x, None, None, 1.0)
    codes = w.codes.view(torch.uint8).clone()
    codes[1::2] = 0x7F
    h, _ = q.qlora_fp8_forward(q.Fp8Weight(N, K, codes.view(R.E4M3), w.scales), x, None, None, 1.0)
    assert torch.equal(h[:, 0::2], clean[:, 0::2]) and torch.isnan(h[:, 1::2]).all()


def test_frozen_a_and_recomputed_u():
    say("fp8 frozen A, recomputed u")
    T, N, K, r = 70, 256, 512, 16
    g = _gen("fa")
    w, x, dY = _weight(g, N, K), _rows(g, T, K), _rows(g, T, N)
    A, B = _adapter(g, N, K, r)
    _, u = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True)
    full = q.qlora_fp8_backward(w, x, dY, A, B, 16.0)
    dX, dA, dB = q.qlora_fp8_backward(w, None, dY, A, B, 16.0, u_saved=u, need_dA=False)
    assert dA is None and torch.equal(dX, full[0]) and torch.equal(dB, full[2])


def test_own_workspaces_on_two_streams():
    say("fp8 two streams")
    g = _gen("streams")
    jobs = []
    for T, N, K in ((16, 1024, 2048), (300, 528, 784)):
        w, x = _weight(g, N, K), _rows(g, T, K)
        A, B = _adapter(g, N, K, 16)
        ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, 16), dtype=torch.uint8, device="cuda")
        jobs.append((w, x, A, B, ws, q.qlora_fp8_forward(w, x, A, B, 16.0)[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = []
    for _ in range(3):
        for st, (w, x, A, B, ws, _) in zip(streams, jobs):
            with torch.cuda.stream(st):
                outs.append(q.qlora_fp8_forward(w, x, A, B, 16.0, ws=ws)[0])
    torch.cuda.synchronize()
    for i, h in enumerate(outs):
        assert torch.equal(h, jobs[i % 2][5])


@pytest.mark.parametrize("T", [1, 16, 100])
def test_captured_calls(T):
    """Forward and backward captured into two graphs, replayed in turn with eager calls between: every replay gives
    the eager results for the inputs of the moment."""
    say(f"fp8 graph T={T}")
    N, K, r = 528, 1040, 16
    g = _gen("graph", T)
    w = _weight(g, N, K)
    A, B = _adapter(g, N, K, r)
    x, dY = _rows(g, T, K), _rows(g, T, N)
    call = lambda: q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True)  # noqa: E731
    back = lambda: q.qlora_fp8_backward(w, x, dY, A, B, 16.0)  # noqa: E731
    call(), back()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for fn in (call, back):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(fn())
        graphs.append(gr)
    for k in range(4):
        x.copy_(_rows(g, T, K))
        dY.copy_(_rows(g, T, N))
        want = [call(), back()]
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        q.qlora_fp8_forward(_weight(g, 64, 64), _rows(g, 5, 64), None, None, 1.0)
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            for s, t in zip(a, b):
                assert torch.equal(s, t), k


@pytest.mark.parametrize("T,N,K,r", [(1, 512, 1040, 8), (5, 1024, 2064, 40), (16, 4096, 4096, 256)])
def test_streaming_forward_without_its_producers(T, N, K, r):
    """With the waits cut to one tick, readers that find a partial of x A^T missing form it themselves: the same bits."""
    say(f"fp8 stream fallback T={T} {N}x{K} r={r}")
    g = _gen("fallback", T)
    w, x = _weight(g, N, K), _rows(g, T, K)
    A, B = _adapter(g, N, K, r)
    ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")
    h, u = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws)
    q.qlora_workspace_set_wait_limit(ws, 1)
    for _ in range(3):
        h1, u1 = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws)
        assert torch.equal(h1, h) and torch.equal(u1, u)
    say(f"    partials formed by readers: {q.qlora_workspace_fallbacks(ws)}")
    q.qlora_workspace_set_wait_limit(ws, 0)


@pytest.mark.parametrize("T,N,K,r", [(200, 512, 512, 8), (333, 1024, 272, 64), (64, 528, 400, 136)])
def test_adapter_gradients_without_waiting(T, N, K, r):
    """With the waits cut to one tick, the last range to arrive adds what the others left: the same bits."""
    say(f"fp8 adapter gradients, no waits T={T} {N}x{K} r={r}")
    g = _gen("no waits", T)
    w, x, dY = _weight(g, N, K), _rows(g, T, K), _rows(g, T, N)
    A, B = _adapter(g, N, K, r)
    ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")
    want = q.qlora_fp8_backward(w, x, dY, A, B, 16.0, ws=ws)
    q.qlora_workspace_set_wait_limit(ws, 1)
    for _ in range(3):
        for a, b in zip(want, q.qlora_fp8_backward(w, x, dY, A, B, 16.0, ws=ws)):
            assert torch.equal(a, b)
    say(f"    waits that ended early: {q.qlora_workspace_fallbacks(ws)}")
    q.qlora_workspace_set_wait_limit(ws, 0)


class _Refuses:
    def __getattr__(self, name):
        return lambda *a: None


@pytest.mark.parametrize("T", [3, 70])
def test_python_and_native_marshalling_agree(T, monkeypatch):
    say(f"fp8 python marshalling T={T}")
    N, K, r = 272, 400, 16
    g = _gen("m", T)
    w, x, dY = _weight(g, N, K), _rows(g, T, K), _rows(g, T, N)
    A, B = _adapter(g, N, K, r)
    xq, xs = q.qlora_fp8_quantize_rows(x, R.E5M2)
    runs = []
    for native in (True, False):
        if not native:
            monkeypatch.setattr(q, "_marshal", _Refuses())
        runs.append(q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True) + q.qlora_fp8_forward(w, None, None, None, 1.0, xq=xq, xs=xs, fmt=R.E5M2)[:1]
                    + q.qlora_fp8_backward(w, x, dY, A, B, 16.0))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def _some_rows(T):
    return torch.tensor(sorted({0, 1, T // 3, T // 2 + 1, T - 130, T - 2, T - 1}), device="cuda")


def test_forward_past_32_bit_offsets():
    """Rows whose 8-bit values, and outputs whose bytes, lie past 2^31 of their tensor's start."""
    for T, N, K in ((140003, 144, 16400), (70001, 16400, 144)):
        say(f"fp8 forward T={T} {N}x{K}")
        g = _gen(T, N)
        w = _weight(g, N, K)
        x = torch.randn(T, K, generator=g, device="cuda", dtype=torch.bfloat16)
        A, B = _adapter(g, N, K, 8)
        h, u = q.qlora_fp8_forward(w, x, A, B, 8.0, save_u=True)
        at = _some_rows(T)
        codes, scales = R.quantize_rows(x[at], R.E4M3)
        xh, wh, Ad, Bd, X = codes * R.spread_cols(scales, K), R.restored_weight(w.codes, w.scales), A.double(), B.double(), x[at].double()
        uref, ubound = X @ Ad.t(), (K + 4) * 2.0 ** -23 * (X.abs() @ Ad.abs().t())
        _check("u", u[at], uref, ubound)
        ref = xh @ wh.t() + uref @ Bd.t()
        extra = (2.0 ** -8 * uref.abs() + (1 + 2.0 ** -8) * ubound) @ Bd.abs().t() + 12 * 2.0 ** -23 * uref.abs() @ Bd.abs().t()
        _check("h", h[at], ref, R.product_bound(xh, wh, ref, extra))


def test_backward_past_32_bit_offsets():
    T, N, K = 140003, 16400, 144
    say(f"fp8 backward T={T} {N}x{K}")
    g = _gen(T, N, "b")
    w = _weight(g, N, K)
    x = torch.randn(T, K, generator=g, device="cuda", dtype=torch.bfloat16)
    dY = torch.randn(T, N, generator=g, device="cuda", dtype=torch.bfloat16)
    A, B = _adapter(g, N, K, 8)
    u = _randn(g, T, 8)
    dX, dA, dB = q.qlora_fp8_backward(w, x, dY, A, B, 8.0, u_saved=u)
    at = _some_rows(T)
    codes, scales = R.quantize_rows(dY[at], R.E4M3)
    yh, wh, Ad, Bd, D = codes * R.spread_cols(scales, N), R.restored_weight(w.codes, w.scales).t(), A.double(), B.double(), dY[at].double()
    v, vb = D @ Bd, (N + 4) * 2.0 ** -23 * (D.abs() @ Bd.abs())
    ref = yh @ wh.t() + v @ Ad
    extra = (2.0 ** -8 * v.abs() + (1 + 2.0 ** -8) * vb) @ Ad.abs() + 12 * 2.0 ** -23 * v.abs() @ Ad.abs()
    _check("dX", dX[at], ref, R.product_bound(yh, wh, ref, extra))
    # The gradients sum over all tokens. A sum of n float32 values in any order is off by at most n steps; the last 300
    # tokens alone, in a call of their own, show that rows past the offset are the ones that are read.
    lim = (T + 8) * 2.0 ** -23
    cols = torch.tensor([0, 5, N // 2, N - 1], device="cuda")
    Dc, U = dY[:, cols].double(), u.double()
    _check("dB", dB[cols], Dc.t() @ U, Dc.abs().t() @ (lim * U.abs()))
    V, Vb, Xd = torch.zeros(T, 8, device="cuda", dtype=torch.float64), torch.zeros(T, 8, device="cuda", dtype=torch.float64), x.double()
    for i in range(0, T, 20000):
        d = dY[i:i + 20000].double()
        V[i:i + 20000], Vb[i:i + 20000] = d @ Bd, d.abs() @ Bd.abs()
    _check("dA", dA, V.t() @ Xd, (lim * V.abs() + (N + 4) * 2.0 ** -23 * Vb).t() @ Xd.abs())
    x[:-300] = 0
    dY[:-300] = 0
    _, dA, dB = q.qlora_fp8_backward(w, x, dY, A, B, 8.0, u_saved=u, need_dx=False)
    _, da, db = q.qlora_fp8_backward(w, x[-300:].contiguous(), dY[-300:].contiguous(), A, B, 8.0, u_saved=u[-300:].contiguous(),
                                     need_dx=False)
    V, Xd, Dd, U, lim = V[-300:], x[-300:].double(), dY[-300:].double(), u[-300:].double(), 2 * 308 * 2.0 ** -23
    _check("dA of the last", dA, da.double(), (lim * V.abs() + 2 * (N + 4) * 2.0 ** -23 * Vb[-300:]).t() @ Xd.abs())
    _check("dB of the last", dB, db.double(), lim * Dd.abs().t() @ U.abs())


@pytest.mark.parametrize("T,N,K", [(1, 1 << 20, 16), (1, 16, 1 << 20), (40, 1 << 20, 32), (40, 32, 1 << 20), (300, 16, 1 << 20),
                                   (1 << 24, 16, 16)])
def test_the_largest_sizes(T, N, K):
    say(f"fp8 largest T={T} {N}x{K}")
    g = _gen(T, N, K, "most")
    w = _weight(g, N, K)
    x = torch.randn(T, K, generator=g, device="cuda", dtype=torch.bfloat16)
    dY = torch.randn(T, N, generator=g, device="cuda", dtype=torch.bfloat16)
    A, B = _adapter(g, N, K, 8)
    at = _some_rows(T) if T > 1000 else torch.arange(T, device="cuda")
    Ad, Bd, wh = A.double(), B.double(), R.restored_weight(w.codes, w.scales)
    h, u = q.qlora_fp8_forward(w, x, A, B, 8.0, save_u=True)
    dX, dA, dB = q.qlora_fp8_backward(w, x, dY, A, B, 8.0, u_saved=u)
    for rows, got, W_, P, Q in ((x, h, wh, Ad, Bd.t()), (dY, dX, wh.t(), Bd.t(), Ad)):
        width = rows.shape[1]
        codes, scales = R.quantize_rows(rows[at], R.E4M3)
        xh, X = codes * R.spread_cols(scales, width), rows[at].double()
        v, vb = X @ P.t(), (width + 4) * 2.0 ** -23 * (X.abs() @ P.abs().t())
        ref = xh @ W_.t() + v @ Q
        extra = (2.0 ** -8 * v.abs() + (1 + 2.0 ** -8) * vb) @ Q.abs() + 12 * 2.0 ** -23 * v.abs() @ Q.abs()
        _check("h" if rows is x else "dX", got[at], ref, R.product_bound(xh, W_, ref, extra))
    lim = (T + 8) * 2.0 ** -23
    D, U, X = dY.double(), u.double(), x.double()
    _check("dB", dB, D.t() @ U, D.abs().t() @ (lim * U.abs()))
    V, vb = D @ Bd, (N + 4) * 2.0 ** -23 * (D.abs() @ Bd.abs())
    _check("dA", dA, V.t() @ X, (lim * V.abs() + vb).t() @ X.abs())


def test_backward_on_two_streams_and_one_workspace_in_turn():
    """Backward calls that overlap, each with a workspace of its own; then one workspace for the 4-bit and the 8-bit
    base's calls in turn, few tokens after many: every result as with a fresh workspace."""
    say("fp8 backward on two streams, one workspace for both bases")
    g = _gen("turns")
    jobs = []
    for T, N, K, r in ((333, 1024, 2048, 16), (200, 2048, 784, 64)):
        w, x, dY = _weight(g, N, K), _rows(g, T, K), _rows(g, T, N)
        A, B = _adapter(g, N, K, r)
        ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")
        jobs.append(((w, x, dY, A, B, 16.0), ws, q.qlora_fp8_backward(w, x, dY, A, B, 16.0)))
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in jobs], []
    for _ in range(4):
        for st, (args, ws, _) in zip(streams, jobs):
            with torch.cuda.stream(st):
                outs.append(q.qlora_fp8_backward(*args, ws=ws))
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert all(torch.equal(a, b) for a, b in zip(got, jobs[i % 2][2]))

    N, K, r = 1024, 2048, 64
    W = _randn(g, N, K) * 0.02
    w8, w4 = q.qlora_fp8_quantize(W), q.qlora_quantize(W)
    A, B = _adapter(g, N, K, r)
    T = 200
    need = max(f(N, K, t, r) for f in (q.qlora_fp8_workspace_bytes, q.qlora_workspace_bytes) for t in (1, 4, 16, T))
    shared = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for k in range(2):
        for t in (T, 1, 4, T, 16, 2):
            x = _rows(g, t, K)
            for f, w in ((q.qlora_forward, w4), (q.qlora_fp8_forward, w8)):
                fresh = torch.zeros(need, dtype=torch.uint8, device="cuda")
                want = f(w, x, A, B, 16.0, save_u=True, ws=fresh)
                got = f(w, x, A, B, 16.0, save_u=True, ws=shared)
                assert all(torch.equal(a, b) for a, b in zip(got, want)), (k, t)
    assert not shared[:q.COUNTER_BYTES].any()
