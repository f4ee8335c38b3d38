"""Gradients of attention against central differences of its definition in float64, block by block of rows and head by head,
along the signs of the exact gradient: the derivative in that direction is the sum of the block's magnitudes, and a gradient of
another size, sign or form misses it."""

import math

import torch

import attention_ref as R

STEP = 2.0 ** -18
BLOCK = 16  # rows


def loss(q, k, v, do, mask, scale):
    """sum(do o) [T, H, D], [S, G, D] in float64, and the sum of the magnitudes that enter it."""
    H, G = q.shape[1], k.shape[1]
    total = size = 0.0
    for h in range(H):
        g = h * G // H
        z = torch.where(mask, q[:, h] @ k[:, g].t() * scale, -math.inf)
        P = torch.where(mask, torch.softmax(torch.where(mask.any(1, keepdim=True), z, 0.0), 1), 0.0)
        total = total + (do[:, h] * (P @ v[:, g])).sum()
        size = size + (do[:, h].abs() * (P @ v[:, g].abs())).sum()
    return total, size


def bounds(q, k, v, do, mask, scale):
    """What the roundings inside may add up to in dq, dk and dv, before their own (attention_ref.py), with an o as far off as
    the forward's may be."""
    H, G = q.shape[1], k.shape[1]
    out = [torch.zeros_like(t) for t in (q, k, v)]
    for h in range(H):
        g = h * G // H
        o, _, P, eo, el, rel = R.head(q[:, h], k[:, g], v[:, g], mask, scale)
        off = o + R.HALF * (o.abs() + eo) + eo
        _, (eq, ek, ev) = R.head_grads(q[:, h], k[:, g], v[:, g], do[:, h], P, mask, scale, o, off, rel, el)
        out[0][:, h] += eq
        out[1][:, g] += ek
        out[2][:, g] += ev
    return out


def third(q, k, v, do, mask, scale, i, u):
    """A bound on the third derivative of the loss along u for argument i. Of a row with scores moving by a_j per step and
    weights P, that of sum_j P_j w_j is E[a'^3 w'] - 3 E[a'^2] E[a' w'] (' less the mean): below 19 max|a|^3 max|w|."""
    H, G = q.shape[1], k.shape[1]
    total = 0.0
    for h in range(H):
        g = h * G // H
        if i == 2:
            continue
        a = (u[:, h] @ k[:, g].t() if i == 0 else q[:, h] @ u[:, g].t()) * scale
        w = do[:, h] @ v[:, g].t()
        a, w = (torch.where(mask, t.abs(), 0.0).amax(1) for t in (a, w))
        total = total + (19 * a ** 3 * w).sum()
    return total


def ratios(grads, q, k, v, do, mask, scale):
    """|the gradient along a direction - the derivative by differences| over the bound, the largest of all blocks, for dq, dk
    and dv. One sequence ([T, H, D], [S, G, D]); the bound counts half a step of bf16 for each value, what the roundings inside
    may do to it, the differences' third order and float64's own roundings."""
    x, do = [t.double().requires_grad_(True) for t in (q, k, v)], do.double()
    exact = torch.autograd.grad(loss(*x, do, mask, scale)[0], x)
    x = [t.detach() for t in x]
    inside = bounds(*x, do, mask, scale)
    out = []
    for i, g in enumerate(grads):
        g, worst = g.double(), 0.0
        signs = torch.where(exact[i] < 0, -1.0, 1.0).double()
        each = R.HALF * (g.abs() + inside[i]) + inside[i] + 2.0 ** -133
        for head in range(g.shape[1]):
            for lo in range(0, g.shape[0], BLOCK):
                u = torch.zeros_like(signs)
                u[lo:lo + BLOCK, head] = signs[lo:lo + BLOCK, head]
                up, down = (loss(*[t + s * STEP * u if j == i else t for j, t in enumerate(x)], do, mask, scale) for s in (1, -1))
                diff = (up[0] - down[0]) / (2 * STEP)
                bound = each[lo:lo + BLOCK, head].sum() + 2.0 ** -44 / STEP * (up[1] + down[1])
                bound = bound + STEP ** 2 / 6 * third(*x, do, mask, scale, i, u)
                worst = max(worst, (((g * u).sum() - diff).abs() / bound).item())
        out.append(worst)
    return out
