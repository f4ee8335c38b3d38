"""Paths of the 8-bit base that few calls take (needs an MI355X): the fallbacks of every wait, counted so that the test
knows that they ran, and values that are not finite in each of the large tiles."""

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


def _inputs(g, T, N, K, r):
    w = q.qlora_fp8_quantize(_randn(g, N, K) * 0.02)
    x, dY = _randn(g, T, K).bfloat16(), _randn(g, T, N).bfloat16()
    A, B = ((_randn(g, r, K) * 0.02).bfloat16(), (_randn(g, N, r) * 0.02).bfloat16()) if r else (None, None)
    return w, x, dY, A, B


def _with_waits_cut(call, ws, most=40):
    """Results of calls whose waits end after one tick, until some wait has ended early (at most `most` calls)."""
    assert q.qlora_workspace_fallbacks(ws) == 0
    q.qlora_workspace_set_wait_limit(ws, 1)
    outs = []
    for k in range(most):
        outs.append(call())
        n = q.qlora_workspace_fallbacks(ws)
        if k >= 2 and n:
            break
    q.qlora_workspace_set_wait_limit(ws, 0)
    say(f"    waits that ended early: {n} in {len(outs)} calls")
    assert n > 0, "no wait took its fallback"
    return outs


# Readers that are done before the first workgroups: few steps of K to stream, or more ranks and slices to form. Few
# tokens (tokens x ranks x slices at most 512): they add the slices' partials, one slice and several; more: the last
# slice hands the sums over.
@pytest.mark.parametrize("T,N,K,r", [(1, 4096, 128, 8), (2, 4096, 128, 16), (16, 4096, 1040, 16), (2, 4096, 2064, 64), (1, 4096, 1040, 256),
                                     (5, 4096, 128, 256), (16, 4096, 2048, 64), (16, 4096, 4096, 256), (5, 1024, 2064, 40)])
def test_readers_form_what_they_miss(T, N, K, r):
    say(f"fp8 stream fallback, counted T={T} {N}x{K} r={r}")
    w, x, _, A, B = _inputs(_gen("miss", T, r), T, N, K, r)
    ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")
    h, u = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws)
    for h1, u1 in _with_waits_cut(lambda: q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws), ws):
        assert torch.equal(h1, h) and torch.equal(u1, u)
    assert not ws[:q.COUNTER_BYTES - 4].any()


# ranges of tokens of the adapter gradients; ranges of K of the rows' product with more than 32 ranks
@pytest.mark.parametrize("T,N,K,r,parts", [(512, 512, 512, 8, "gradients"), (2048, 1024, 272, 64, "gradients"),
                                           (64, 8192, 8192, 64, "rows"), (70, 8192, 4096, 256, "rows")])
def test_the_last_to_arrive_adds_what_is_left(T, N, K, r, parts):
    say(f"fp8 split sums, counted T={T} {N}x{K} r={r} {parts}")
    w, x, dY, A, B = _inputs(_gen("left", T, r), T, N, K, r)
    ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")
    if parts == "rows":
        call = lambda: q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws)  # noqa: E731
    else:
        u = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True)[1]
        call = lambda: q.qlora_fp8_backward(w, x, dY, A, B, 16.0, u_saved=u, need_dx=False, need_dA=False, ws=ws)[2:]  # noqa: E731
    want = call()
    for got in _with_waits_cut(call, ws):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not ws[:q.COUNTER_BYTES - 4].any()


# tokens, outputs, contracted width: large tiles of each form, whole and with the last round in K ranges
@pytest.mark.parametrize("r", [0, 16])
@pytest.mark.parametrize("T,N,K", [(776, 5168, 288), (3166, 2608, 256), (201, 13520, 4720), (1031, 15136, 2704), (515, 13824, 400),
                                   (1781, 13696, 3344), (206, 8496, 4784)])
def test_values_that_are_not_finite_stay_in_their_rows(T, N, K, r):
    say(f"fp8 not finite, large tiles T={T} {N}x{K} r={r}")
    g = _gen("nan", T, N)
    w, x, _, A, B = _inputs(g, T, N, K, r)
    wt = q.qlora_fp8_quantize(_randn(g, K, N) * 0.02)  # K outputs, N inputs: its backward contracts K
    forward = lambda v: q.qlora_fp8_forward(w, v, A, B, 16.0)[0]  # noqa: E731
    At, Bt = (B.t().contiguous(), A.t().contiguous()) if r else (None, None)
    backward = lambda v: q.qlora_fp8_backward(wt, None, v, At, Bt, 16.0, need_dA=False, need_dB=False)[0]  # noqa: E731
    rows = sorted({0, T // 3, T // 2 + 1, T - 1})
    bad = x.clone()
    for i, t in enumerate(rows):
        bad[t, (i * K // 3) % K] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[rows] = False
    for name, f in (("h", forward), ("dX", backward)):
        clean, got = f(x), f(bad)
        assert torch.isfinite(clean).all(), name
        assert not torch.isfinite(got[rows]).any(), name
        assert torch.equal(got[keep], clean[keep]), name
