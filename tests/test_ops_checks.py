"""Refusals of the 8-bit base, the norm and the many-tensor AdamW step, without a GPU: the C entry points on made-up
addresses (every case fails its checks, so nothing is enqueued), the binding on CPU tensors."""

import ctypes
import os

import pytest
import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.LIB):
    _build.build()
from bit_quantized_finetuning_amd import qlora as q  # noqa: E402

NULL, SHAPE, ALIGN, WORKSPACE, DTYPE, VALUE = -1, -2, -3, -4, -5, -9
OK, OFF = 0x10000, 0x10001
F32, BF16, E4M3, E5M2 = 0, 1, 2, 3
BIG = 1 << 40


def _w(d_out=64, d_in=128, codes=OK, scales=OK):
    return ctypes.byref(q._Fp8Weight(d_out, d_in, codes, scales))


def test_fp8_quantizers_refuse():
    f, r = q.lib.qlora_fp8_quantize, q.lib.qlora_fp8_quantize_rows
    assert f(None, 0, _w(), None) == NULL
    assert f(OK, 0, None, None) == NULL
    assert f(OK, 0, _w(codes=None), None) == NULL
    assert f(OK, 0, _w(scales=None), None) == NULL
    assert f(OK, E4M3, _w(), None) == DTYPE
    assert f(OFF, 0, _w(), None) == ALIGN
    for bad in ((0, 128), (64, 0), (24, 128), (64, 136), (16, (1 << 20) + 16)):
        assert f(OK, 0, _w(*bad), None) == SHAPE
    assert r(None, BF16, 1, 16, E4M3, OK, OK, None) == NULL
    assert r(OK, BF16, 1, 16, E4M3, None, OK, None) == NULL
    assert r(OK, BF16, 1, 16, BF16, OK, OK, None) == DTYPE
    assert r(OK, E5M2, 1, 16, E4M3, OK, OK, None) == DTYPE
    for T, d in ((0, 16), (-1, 16), ((1 << 24) + 1, 16), (1, 0), (1, 24), (1, (1 << 20) + 16)):
        assert r(OK, BF16, T, d, E4M3, OK, OK, None) == SHAPE
    assert r(OK, BF16, 1, 16, E4M3, OFF, OK, None) == ALIGN


def _fwd(w=None, xq=OK, xs=OK, fmt=E4M3, x=OK, T=4, A=OK, B=OK, r=8, h=OK, u=None, ws=OK, n=BIG):
    return q.lib.qlora_fp8_forward(w or _w(), xq, xs, fmt, x, T, A, B, r, 16.0, h, u, ws, n, None)


def test_fp8_forward_refuses():
    assert _fwd(w=_w(d_in=24)) == SHAPE
    assert _fwd(h=None) == NULL
    assert _fwd(fmt=BF16) == DTYPE
    assert _fwd(T=0) == SHAPE and _fwd(r=12) == SHAPE and _fwd(r=264) == SHAPE and _fwd(r=-8) == SHAPE
    assert _fwd(A=None) == NULL and _fwd(B=None) == NULL
    assert _fwd(xs=None) == NULL and _fwd(xq=None) == NULL
    assert _fwd(xq=None, xs=None, x=None, A=None, B=None) == NULL
    assert _fwd(x=None) == NULL  # the adapter needs it
    assert _fwd(xq=OFF) == ALIGN and _fwd(xs=OFF) == ALIGN and _fwd(u=OFF) == ALIGN and _fwd(h=OFF) == ALIGN
    need = q.qlora_fp8_workspace_bytes(64, 128, 4, 8)
    assert _fwd(n=need - 1) == WORKSPACE and _fwd(ws=None) == NULL and _fwd(ws=OFF) == ALIGN


def _bwd(w=None, x=OK, dY=OK, fmt=E5M2, T=4, A=OK, B=OK, r=8, u=None, dX=OK, dA=OK, dB=OK, ws=OK, n=BIG):
    return q.lib.qlora_fp8_backward(w or _w(), x, dY, fmt, T, A, B, r, 16.0, u, dX, dA, dB, ws, n, None)


def test_fp8_backward_refuses():
    assert _bwd(dY=None) == NULL and _bwd(fmt=F32) == DTYPE and _bwd(T=0) == SHAPE
    assert _bwd(A=None, B=None) == SHAPE  # gradients of an adapter that is not there
    assert _bwd(x=None) == NULL and _bwd(x=None, dA=None) == NULL
    assert _bwd(dX=OFF) == ALIGN and _bwd(u=OFF) == ALIGN and _bwd(dA=OFF) == ALIGN
    need = q.qlora_fp8_workspace_bytes(64, 128, 4, 8)
    assert _bwd(n=need - 1) == WORKSPACE and _bwd(ws=None) == NULL
    assert _bwd(dX=None, dA=None, dB=None, n=need) == 0  # nothing asked, nothing done


def test_fp8_workspace_and_storage_bytes():
    assert q.qlora_fp8_storage_bytes(272, 400) == 272 * 400 + 4 * 3 * 4
    assert q.qlora_fp8_storage_bytes(0, 4) == 0
    assert q.qlora_fp8_workspace_bytes(64, 128, 0, 8) == 0 and q.qlora_fp8_workspace_bytes(64, 128, 1, 257) == 0
    assert q.qlora_fp8_workspace_bytes(64, 128, 4, 0) >= 65536 + 4 * 128


def _norm(x=OK, ldx=64, res=None, ldr=0, dt=BF16, T=4, d=64, w=OK, wdt=F32, eps=1e-6, s=None, y=OK, yq=None, ys=None,
          fmt=E4M3, rstd=None):
    return q.lib.qlora_rmsnorm_forward(x, ldx, res, ldr, dt, T, d, w, wdt, eps, s, y, yq, ys, fmt, rstd, None)


def test_rmsnorm_forward_refuses():
    assert _norm(x=None) == NULL and _norm(y=None) == NULL
    assert _norm(yq=OK) == NULL and _norm(ys=OK) == NULL
    assert _norm(res=OK, ldr=64) == NULL and _norm(s=OK) == NULL  # s and the residual come together
    assert _norm(dt=E4M3) == DTYPE and _norm(wdt=7) == DTYPE and _norm(yq=OK, ys=OK, fmt=F32) == DTYPE
    assert _norm(T=-1) == SHAPE and _norm(d=0) == SHAPE and _norm(d=32769, ldx=40000) == SHAPE
    assert _norm(ldx=63) == SHAPE and _norm(res=OK, s=OK, ldr=63) == SHAPE
    assert _norm(eps=-1.0) == VALUE and _norm(eps=float("nan")) == VALUE and _norm(eps=float("inf")) == VALUE
    assert _norm(x=OFF) == ALIGN and _norm(w=0x10002) == ALIGN and _norm(y=0x10008) == ALIGN
    assert _norm(T=0, x=None) == 0


def _nback(dy=OK, ldy=64, s=OK, lds=64, ds=None, ldd=0, dt=BF16, T=4, d=64, w=OK, wdt=F32, rstd=OK, dx=OK, dw=None,
           ws=None, n=0):
    return q.lib.qlora_rmsnorm_backward(dy, ldy, s, lds, ds, ldd, dt, T, d, w, wdt, rstd, dx, dw, ws, n, None)


def test_rmsnorm_backward_refuses():
    for k in ("dy", "s", "rstd", "dx"):
        assert _nback(**{k: None}) == NULL
    assert _nback(ldy=63) == SHAPE and _nback(lds=1) == SHAPE and _nback(ds=OK, ldd=5) == SHAPE
    assert _nback(dt=5) == DTYPE and _nback(d=0) == SHAPE
    assert _nback(dy=OFF) == ALIGN and _nback(dw=OFF) == ALIGN and _nback(rstd=0x10002) == ALIGN
    need = q.lib.qlora_rmsnorm_workspace_bytes(4, 64)
    assert need >= 4 * 64 * 4
    assert _nback(dw=OK, n=need - 1, ws=OK) == WORKSPACE and _nback(dw=OK, n=need) == NULL
    assert _nback(T=0, dy=None) == 0
    assert q.lib.qlora_rmsnorm_workspace_bytes(4, 40000) == 0


def _many(jobs=((OK, OK, 100),), hp=(1e-3, 0.9, 0.999, 1e-8, 0.0), step=1, count=None, gd=F32, pd=F32, sd=F32, m=OK,
          v=OK, ms=None, vs=None, master=None, max_norm=0.0, norm=None, ws=None, n=0, state=True):
    arr = (q._AdamWJob * max(1, len(jobs)))(*[q._AdamWJob(*j) for j in jobs])
    st = q._AdamWState(sd, m, v, ms, vs, master)
    return q.lib.qlora_adamw_many(ctypes.byref(q._AdamWManyHparams(*hp)) if hp else None, step, arr,
                                  len(jobs) if count is None else count, gd, pd, ctypes.byref(st) if state else None,
                                  max_norm, norm, 0, ws, n, None)


def test_adamw_many_refuses():
    assert _many(hp=None) == NULL and _many(state=False) == NULL
    assert _many(count=-1) == SHAPE
    assert _many(gd=E4M3) == DTYPE and _many(pd=9) == DTYPE and _many(sd=BF16) == DTYPE and _many(sd=E5M2) == DTYPE
    for hp in ((-1.0, 0.9, 0.999, 1e-8, 0.0), (1e-3, 1.0, 0.999, 1e-8, 0.0), (1e-3, 0.9, -0.1, 1e-8, 0.0),
               (1e-3, 0.9, 0.999, 0.0, 0.0), (1e-3, 0.9, 0.999, 1e-8, -1.0), (float("nan"), 0.9, 0.999, 1e-8, 0.0)):
        assert _many(hp=hp) == VALUE
    assert _many(step=0) == VALUE and _many(max_norm=-1.0) == VALUE and _many(max_norm=float("nan")) == VALUE
    assert _many(jobs=((OK, OK, -1),)) == SHAPE and _many(jobs=((OK, OK, 1 << 38),)) == SHAPE
    assert _many(jobs=((OK, OK, (1 << 38) - 256),) * 3) == SHAPE  # 2^31 blocks and more
    assert _many(jobs=((OK, OK, 5), (OK, None, 1))) == NULL
    assert _many(jobs=((OK, OK, 5), (OFF, OK, 1))) == ALIGN
    assert _many(m=None) == NULL and _many(m=OFF) == ALIGN
    assert _many(sd=E4M3) == NULL and _many(sd=E4M3, ms=OK) == NULL  # scales
    assert _many(pd=BF16) == NULL  # master copy
    assert _many(max_norm=1.0) == NULL
    need = q.lib.qlora_adamw_many_workspace_bytes(1)
    assert _many(max_norm=1.0, norm=OK, ws=OK, n=need - 1) == WORKSPACE
    assert _many(max_norm=1.0, norm=OK, n=need) == NULL
    assert _many(jobs=(), m=None, v=None) == 0 and _many(jobs=((None, None, 0),), m=None, v=None) == 0
    assert _many(jobs=((None, OK, 5),)) == 0  # no gradient: left as it is


# --- the binding -------------------------------------------------------------

def _fp8(d_out=64, d_in=128):
    return q.Fp8Weight(d_out, d_in, torch.zeros(d_out, d_in, dtype=q.E4M3), torch.zeros(-(-d_out // 128), -(-d_in // 128)))


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_binding_refuses_fp8():
    w = _fp8()
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_fp8_forward(w, _bf(4, 128), None, None, 1.0)
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_fp8_backward(w, None, _bf(4, 64), None, None, 1.0)
    for call, err in (
            (lambda: q.qlora_fp8_forward(w, _bf(4, 64), None, None, 1.0), ValueError),
            (lambda: q.qlora_fp8_forward(w, torch.zeros(4, 128), None, None, 1.0), TypeError),
            (lambda: q.qlora_fp8_forward(w, None, None, None, 1.0), ValueError),
            (lambda: q.qlora_fp8_forward(w, _bf(0, 128), None, None, 1.0), ValueError),
            (lambda: q.qlora_fp8_forward(w, _bf(4, 128), None, None, 1.0, xq=torch.zeros(4, 128, dtype=q.E4M3)), ValueError),
            (lambda: q.qlora_fp8_forward(w, None, None, None, 1.0, xq=torch.zeros(4, 128, dtype=q.E5M2), xs=torch.zeros(4, 1)), TypeError),
            (lambda: q.qlora_fp8_forward(w, None, None, None, 1.0, xq=torch.zeros(4, 128, dtype=q.E4M3), xs=torch.zeros(4, 2)), ValueError),
            (lambda: q.qlora_fp8_forward(w, None, _bf(8, 128), _bf(64, 8), 1.0, xq=torch.zeros(4, 128, dtype=q.E4M3), xs=torch.zeros(4, 1)), ValueError),
            (lambda: q.qlora_fp8_forward(w, _bf(4, 128), _bf(8, 128), None, 1.0), ValueError),
            (lambda: q.qlora_fp8_forward(w, _bf(4, 128), _bf(12, 128), _bf(64, 12), 1.0), ValueError),
            (lambda: q.qlora_fp8_forward(w, _bf(4, 128), None, None, 1.0, fmt=torch.bfloat16), TypeError),
            (lambda: q.qlora_fp8_forward(w, _bf(4, 128), None, None, 1.0, ws=torch.zeros(8, dtype=torch.uint8)), ValueError),
            (lambda: q.qlora_fp8_forward(_fp8(64, 120), _bf(4, 120), None, None, 1.0), ValueError),
            (lambda: q.qlora_fp8_backward(w, None, _bf(4, 64), _bf(8, 128), _bf(64, 8), 1.0), ValueError),
            (lambda: q.qlora_fp8_backward(w, None, _bf(4, 64), None, None, 1.0, dA=torch.zeros(8, 128)), ValueError),
            (lambda: q.qlora_fp8_quantize(_bf(64, 120)), ValueError),
            (lambda: q.qlora_fp8_quantize(torch.zeros(64, 128, dtype=torch.float16)), TypeError),
            (lambda: q.qlora_fp8_quantize(_bf(128, 64).t()), ValueError),
            (lambda: q.qlora_fp8_quantize_rows(_bf(4, 24)), ValueError),
            (lambda: q.qlora_fp8_quantize_rows(_bf(0, 16)), ValueError),
            (lambda: q.qlora_fp8_quantize_rows(_bf(4, 16), fmt=torch.int8), TypeError)):
        with pytest.raises(err):
            call()
    h = _bf(4, 64)
    x = torch.zeros(4 * 128 + 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="overlaps"):
        q.qlora_fp8_forward(w, x[:512].view(4, 128), None, None, 1.0, h=x[:256].view(4, 64))
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_fp8_forward(w, x[:512].view(4, 128), None, None, 1.0, h=h)


def test_binding_refuses_norm():
    x = _bf(4, 64)
    for call, err in (
            (lambda: q.qlora_rmsnorm_forward(x), ValueError),  # no GPU
            (lambda: q.qlora_rmsnorm_forward(x.half()), TypeError),
            (lambda: q.qlora_rmsnorm_forward(x[0]), ValueError),
            (lambda: q.qlora_rmsnorm_forward(_bf(2, 40000)), ValueError),
            (lambda: q.qlora_rmsnorm_forward(x, want_y=False), ValueError),
            (lambda: q.qlora_rmsnorm_forward(x.t()), ValueError),
            (lambda: q.qlora_rmsnorm_forward(_bf(1, 64).expand(4, 64)), ValueError),  # rows that overlap
            (lambda: q.qlora_rmsnorm_forward(x, residual=_bf(4, 32)), ValueError),
            (lambda: q.qlora_rmsnorm_forward(x, residual=torch.zeros(4, 64)), TypeError),
            (lambda: q.qlora_rmsnorm_forward(x, weight=torch.ones(63)), ValueError),
            (lambda: q.qlora_rmsnorm_forward(x, weight=torch.ones(64, dtype=torch.float64)), TypeError),
            (lambda: q.qlora_rmsnorm_forward(x, fmt=torch.float32), TypeError),
            (lambda: q.qlora_rmsnorm_backward(x, x, None, torch.ones(3)), ValueError),
            (lambda: q.qlora_rmsnorm_backward(x.float(), x, None, torch.ones(4)), TypeError),
            (lambda: q.qlora_rmsnorm_backward(None, x, None, torch.ones(4)), TypeError),
            (lambda: q.qlora_rmsnorm_backward(x, x, None, None), TypeError),
            (lambda: q.qlora_rmsnorm_backward(x, x, None, torch.ones(4)), ValueError)):  # no GPU
        with pytest.raises(err):
            call()


def test_binding_refuses_adamw_many():
    g, p = torch.zeros(300), torch.zeros(300)
    m, v = torch.zeros(512), torch.zeros(512)
    m8 = torch.zeros(512, dtype=q.E4M3)
    two = torch.zeros(2)
    for call, err in (
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v), ValueError),  # no GPU
            (lambda: q.qlora_adamw_many(1, [g], [], m, v), ValueError),
            (lambda: q.qlora_adamw_many(1, [g.half()], [p], m, v), TypeError),
            (lambda: q.qlora_adamw_many(1, [g, g.bfloat16()], [p, p.clone()], torch.zeros(1024), torch.zeros(1024)), TypeError),
            (lambda: q.qlora_adamw_many(1, [g[:200]], [p], m, v), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m[:300], v[:300]), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m.double(), v.double()), TypeError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m8, m8.clone()), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, two, two), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, master=m.clone()), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p.bfloat16()], m, v), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, max_norm=0.0), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, max_norm=float("nan")), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, max_norm=1e-60), ValueError),  # nothing in float32
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, norm=torch.zeros(1)), ValueError),
            (lambda: q.qlora_adamw_many(1, [g], [p], m, v, seed=-1), ValueError)):
        with pytest.raises(err):
            call()
    with pytest.raises(ValueError, match="overlap"):  # one parameter twice
        q.qlora_adamw_many(1, [g, g], [p, p], torch.zeros(1024), torch.zeros(1024))
    for call in (lambda: q.qlora_adamw_many(1, [g], [p], m, m),  # one buffer for two things
                 lambda: q.qlora_adamw_many(1, [g], [m[:300]], m, v),
                 lambda: q.qlora_adamw_many(1, [g], [p], m, v, max_norm=1.0, norm=v[511:])):
        with pytest.raises(ValueError, match="overlap"):
            call()
    assert q.adamw_state_elements([0, 1, 256, 257]) == 256 + 256 + 512
