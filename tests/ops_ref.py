"""64-bit references of the operators around the frozen base (torch float64, on whatever device the inputs are),
and the error bounds that their tests use."""

import numpy as np
import torch

GROUP, BLOCK, TINY = 128, 256, 2.0 ** -100
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4M3: 448.0, E5M2: 57344.0}
MANT = {E4M3: 3, E5M2: 2}
LOW = {E4M3: -6, E5M2: -14}  # exponent of the least normal value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def ngroups(d):
    return -(-d // GROUP)


def nearest(x, fmt):
    """The format's value nearest to each x (|x| <= TOP), ties to even."""
    ulp = torch.exp2((torch.frexp(x)[1] - 1).clamp_min(LOW[fmt]).double() - MANT[fmt])
    return torch.round(x / ulp) * ulp


def row_scales(y, fmt):
    """The least power of two s with amax <= TOP s per row and group of 128."""
    T, d = y.shape
    g = torch.nn.functional.pad(y.abs().double(), (0, -d % GROUP)).view(T, -1, GROUP).amax(-1).clamp_min(TINY)
    f, e = torch.frexp(g / TOP[fmt])
    return torch.exp2((e - (f == 0.5).int()).double())


def spread_cols(scales, d):
    return scales.double().repeat_interleave(GROUP, 1)[:, :d]


def quantize_rows(y, fmt):
    s = row_scales(y, fmt)
    return nearest(y.double() / spread_cols(s, y.shape[1]), fmt), s


def block_amax(W):
    N, K = W.shape
    p = torch.nn.functional.pad(W.abs().double(), (0, -K % GROUP, 0, -N % GROUP))
    return p.view(p.shape[0] // GROUP, GROUP, p.shape[1] // GROUP, GROUP).amax((1, 3)).clamp_min(TINY)


def restored_weight(codes, scales):
    N, K = codes.shape
    return codes.double() * scales.double().repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]


ALIGN = 2.0 ** -13  # what the matrix unit keeps beside the largest of eight products (see product_bound)


def product_bound(xh, wh, ref, extra=0.0):
    """Bound on |bf16 result - ref| of a block-scaled product of 8-bit values.

    * The matrix unit brings eight products (eight consecutive k) to the exponent of the largest of them before it
      adds them, and drops what lies below 2^-13 of that (test_what_the_matrix_unit_keeps pins it): each of the eight
      is off by less than 2^-13 of the largest, which is at most the largest |x| times the largest |w| of the eight.
    * The sums of the eights, the two scale factors' roundings and the sum over the blocks are float32: at most one
      step (2^-23) of the terms' magnitudes each, GROUP / 8 + 4 + the number of blocks of them.
    * Half a step of bf16 on the result."""
    T, K = xh.shape
    mags = xh.abs() @ wh.abs().t()
    eights = xh.abs().view(T, K // 8, 8).amax(-1) @ wh.abs().reshape(-1, K // 8, 8).amax(-1).t()
    acc = 8 * ALIGN * eights + (GROUP // 8 + 4 + ngroups(K)) * 2.0 ** -23 * mags + extra
    return HALF[torch.bfloat16] * (ref.abs() + acc) + acc


def random_bits(n, seed, step, device, start=0):
    """The 32 bits of each place of the moments, in Python's arithmetic modulo 2^32."""
    M = (1 << 32) - 1
    key = (seed * 0x9E3779B1 + step * 0x85157AF5) & M
    key ^= key >> 16
    i = np.arange(start, start + n, dtype=np.uint64)
    x = (i * np.uint64(0x9E3779B1) + np.uint64(key)) & np.uint64(M)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x6A09E667)) & np.uint64(M)
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0x3C6EF373)) & np.uint64(M)
    x = x ^ (x >> np.uint64(16))
    return torch.from_numpy(x.astype(np.int64)).to(device)


def round_up_or_down(x, r16):
    """Non-negative x <= 448 to e4m3: up with probability its place between its neighbours; also its grid step."""
    ulp = torch.exp2((torch.frexp(x)[1] - 1).clamp_min(-6).double() - 3)
    return (torch.floor(x / ulp + r16.double() / 65536.0) * ulp).clamp_max(448.0), ulp


def padded(n):
    return -(-n // BLOCK) * BLOCK


def flat(tensors):
    """Tensors side by side, each padded with zeros to a multiple of 256."""
    return torch.cat([torch.nn.functional.pad(t.reshape(-1).double(), (0, -t.numel() % BLOCK)) for t in tensors])


def adamw(step, g, p, m, v, lr, beta1, beta2, eps, weight_decay, max_norm=None):
    """One step in float64. v is v itself."""
    norm = g.square().sum().sqrt()
    if max_norm is not None:
        g = g * min(1.0, max_norm / (float(norm) + 1e-6))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    upd = (m / (1 - beta1 ** step)) / ((v / (1 - beta2 ** step)).sqrt() + eps)
    return p * (1 - lr * weight_decay) - lr * upd, m, v, norm
