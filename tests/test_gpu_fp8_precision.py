"""Precision of the adapter's term over the 8-bit base (needs an MI355X): with a base of zeros it is all of the result, so
that nothing covers the rounding of its intermediate."""

import zlib

import pytest
import torch

import ops_ref as R
from gpu_common import product, say

pytestmark = pytest.mark.gpu

q = product("qlora")


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _bound(v, vb, Q, ref, s, r):
    """One rounding to bf16 of s v Q: v (off by vb) enters as two bf16 terms, which hold all but 2^-15 of s v; s v is one
    float32 rounding; 2 r products and their sum are float32, one step each at most, and a few more for the joins."""
    lost = 2.0 ** -15 + 2.0 ** -24 + (2 * r + 8) * 2.0 ** -23
    acc = s * (lost * v.abs() + (1 + lost) * vb) @ Q.abs()
    return R.HALF[torch.bfloat16] * (ref.abs() + acc) + acc


def _check(name, got, ref, bound):
    worst = ((got.double() - ref).abs() / bound.clamp_min(1e-300)).max().item()
    error = ((got.double() - ref).norm() / ref.norm()).item()
    say(f"    {name}: largest error / bound = {worst:.3f}, relative error {error:.2e}")
    assert got.shape == ref.shape and worst <= 1.0, f"{name}: {worst} times the bound"


# one token: readers add the slices' partials; more: the last slice hands the sums over; then small tiles (in K ranges and
# whole) and large ones
@pytest.mark.parametrize("T,N,K,r", [(1, 4096, 4096, 16), (1, 272, 144, 8), (4, 1040, 784, 16), (5, 528, 4096, 40), (16, 1024, 2048, 64),
                                     (16, 512, 1040, 256), (40, 272, 4096, 24), (70, 1024, 1040, 128), (300, 5120, 528, 64),
                                     (515, 13824, 144, 16), (1031, 4096, 400, 256)])
def test_adapter_alone(T, N, K, r):
    say(f"fp8 adapter alone T={T} {N}x{K} r={r}")
    g = _gen(T, N, K, r)
    s = 32.0 / r
    codes = torch.zeros(N, K, device="cuda").to(R.E4M3)
    w = q.Fp8Weight(N, K, codes, torch.ones(-(-N // 128), -(-K // 128), device="cuda"))
    x, dY = _randn(g, T, K).bfloat16(), _randn(g, T, N).bfloat16()
    A, B = (_randn(g, r, K) * 0.02).bfloat16(), (_randn(g, N, r) * 0.02).bfloat16()
    h, u = q.qlora_fp8_forward(w, x, A, B, 32.0, save_u=True)
    dX, _, _ = q.qlora_fp8_backward(w, x, dY, A, B, 32.0, u_saved=u, need_dA=False, need_dB=False)
    for name, got, rows, P, Q in (("h", h, x, A.double().t(), B.double().t()), ("dX", dX, dY, B.double(), A.double())):
        v = rows.double() @ P
        vb = (P.shape[0] + 4) * 2.0 ** -23 * (rows.double().abs() @ P.abs())
        ref = s * v @ Q
        _check(name, got, ref, _bound(v, vb, Q, ref, s, r))


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_adapter_of_large_and_infinite_values(T):
    """s u near the end of float32's range (its bf16 would be infinite), infinite and NaN, each in a token of its own."""
    say(f"fp8 adapter, large values T={T}")
    N, K, r = 272, 144, 8
    g = _gen("large", T)
    w = q.Fp8Weight(N, K, torch.zeros(N, K, device="cuda").to(R.E4M3), torch.zeros(3, 2, device="cuda"))
    A, B = torch.zeros(r, K, device="cuda"), torch.zeros(N, r, device="cuda")
    A[0, 0] = A[0, 1] = 1.0
    B[:, 0] = torch.exp2(torch.randint(-60, -50, (N,), generator=g, device="cuda").float())
    x = torch.zeros(T, K, device="cuda")
    top, low = 2.0 ** 127 * (2 - 2.0 ** -7), 2.0 ** 119 * (2 - 2.0 ** -7)  # their sum has 16 bits, and no bf16 near it is finite
    x[0, 0], x[0, 1] = top, low
    if T > 2:
        x[T // 2, 0], x[T - 1, 0] = float("inf"), float("nan")
    A, B, x = A.bfloat16(), B.bfloat16(), x.bfloat16()
    h, u = q.qlora_fp8_forward(w, x, A, B, float(r), xq=torch.zeros(T, K, device="cuda").to(R.E4M3), xs=torch.ones(T, 2, device="cuda"),
                               save_u=True)
    assert u[0, 0].item() == top + low
    assert torch.equal(h[0].double(), ((top + low) * B[:, 0].double()).bfloat16().double())
    if T > 2:
        assert u[T // 2, 0].item() == float("inf")  # and the infinity times the zeros of A's other rows is NaN in the formula
        assert torch.isnan(h[T // 2]).all() and torch.isnan(h[T - 1]).all()
        assert not h[1:T // 2].any()


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_infinite_intermediate_stays_infinite(T):
    say(f"fp8 adapter, infinite u T={T}")
    N, K, r = 272, 144, 8
    w = q.Fp8Weight(N, K, torch.zeros(N, K, device="cuda").to(R.E4M3), torch.zeros(3, 2, device="cuda"))
    A, B = torch.zeros(r, K, device="cuda"), torch.ones(N, r, device="cuda")
    A[:, 0] = 1.0
    x = torch.zeros(T, K, device="cuda")
    x[T - 1, 0] = float("-inf")
    h, _ = q.qlora_fp8_forward(w, x.bfloat16(), A.bfloat16(), B.bfloat16(), float(r), xq=torch.zeros(T, K, device="cuda").to(R.E4M3),
                               xs=torch.ones(T, 2, device="cuda"))
    assert (h[T - 1] == float("-inf")).all() and not h[:T - 1].any()
