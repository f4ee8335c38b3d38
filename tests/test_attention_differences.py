"""The check of attention's gradients against differences, on the CPU: it accepts the exact gradients, rounded, and refuses
those of every mistake planted here."""

import math

import pytest
import torch

import attention_differences as A
import attention_ref as R

CASES = [(70, 4, 2, 64, 20, 3), (90, 3, 1, 128, 1 << 30, 0), (33, 2, 2, 64, 5, 1)]


def _case(T, H, G, D, window, sinks):
    g = torch.Generator().manual_seed(T)
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    return 2 * bf(T, H, D), bf(T, G, D), bf(T, G, D), bf(T, H, D), R.seen(T, T, T, 0, window, sinks, device="cpu"), D ** -0.5


def _grads(q, k, v, do, mask, scale, mistake=""):
    """dq, dk, dv by the formula in float64, with one mistake."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    T, H, G = q.shape[0], q.shape[1], k.shape[1]
    o, dq, dk, dv = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    if mistake == "window":  # one key too many
        mask = mask | (torch.arange(T)[:, None] - torch.arange(T)[None] == 20)
    if mistake == "causal":  # the query's own key is missing
        mask = mask & ~torch.eye(T, dtype=torch.bool) | (torch.arange(T)[:, None] == 0) & mask
    for h in range(H):
        g = h * G // H
        P = torch.softmax(torch.where(mask, q[:, h] @ k[:, g].t() * scale, -math.inf), 1)
        o[:, h] = P @ v[:, g]
        dP = do[:, h] @ v[:, g].t()
        delta = (do[:, h] * o[:, h]).sum(1, keepdim=True)
        if mistake == "delta":
            delta = 0 * delta
        dS = P * (dP - delta) * (1.0 if mistake == "scale" else scale)
        if mistake == "weights":
            dS = dS * P
        dq[:, h] = dS @ k[:, g]
        if mistake == "heads" and h % (H // G):
            continue
        dk[:, g] += dS.t() @ q[:, h]
        dv[:, g] += (P.t() if mistake != "half" else P.t() / 2) @ do[:, h]
    if mistake == "half":
        dq, dk = dq / 2, dk / 2
    if mistake == "sign":
        dq, dk, dv = -dq, -dk, -dv
    if mistake == "rows":  # a tile's last rows are lost
        dq[-8:], dk[-8:], dv[-8:] = 0, 0, 0
        dk[:8], dv[:8] = 0, 0
    return dq, dk, dv


@pytest.mark.parametrize("case", CASES)
def test_exact_gradients_pass(case):
    x = _case(*case)
    grads = _grads(*x)
    for got in (grads, [t.bfloat16() for t in grads]):
        assert max(A.ratios(got, *x)) <= 1.0


@pytest.mark.parametrize("mistake,wrong", [("half", (0, 1, 2)), ("sign", (0, 1, 2)), ("delta", (0, 1)), ("scale", (0, 1)), ("weights", (0, 1)),
                                           ("heads", (1, 2)), ("window", (0, 1, 2)), ("causal", (0, 1, 2)), ("rows", (0, 1, 2))])
def test_mistakes_are_refused(mistake, wrong):
    x = _case(*CASES[0])
    grads = _grads(*x, mistake=mistake)
    found = A.ratios([t.bfloat16() for t in grads], *x)
    assert all(found[i] > 1.0 for i in wrong), (mistake, found)
