"""Refusals of the operators between a layer's projections, without a GPU: the C entry points on made-up addresses (every
case fails its checks, so nothing is enqueued), the binding on CPU tensors."""

import ctypes
import math
import os

import pytest
import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.LIB):
    _build.build()
from bit_quantized_finetuning_amd import qlora as q  # noqa: E402

NULL, SHAPE, ALIGN, WORKSPACE, DTYPE, VALUE = -1, -2, -3, -4, -5, -9
OK, OFF = 0x10000, 0x10001
F32, BF16, E4M3 = 0, 1, 2
BIG = 1 << 40


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


# --- rotary ------------------------------------------------------------------

def _rot(x=OK, y=OK, xt=128, xh=64, yt=128, yh=64, heads=2, count=1, dt=BF16, T=4, D=64, dim=64, pos=OK, bits=64, freqs=OK, amp=1.0,
         rows=True):
    arr = (q._RotaryRows * 2)(q._RotaryRows(x, y, xt, xh, yt, yh, heads), q._RotaryRows(OK, OK, 128, 64, 128, 64, 2))
    return q.lib.qlora_rotary(arr if rows else None, count, dt, T, D, dim, pos, bits, freqs, amp, 0, 0, None)


def test_rotary_refuses():
    assert _rot(rows=False) == NULL and _rot(x=None) == NULL and _rot(y=None) == NULL and _rot(freqs=None) == NULL
    assert _rot(pos=None) == NULL and _rot(bits=0) == NULL
    assert _rot(dt=E4M3) == DTYPE and _rot(bits=16) == DTYPE
    for bad in (dict(count=0), dict(count=3), dict(T=-1), dict(T=(1 << 24) + 1), dict(D=0), dict(D=1026, dim=64), dict(dim=0),
                dict(dim=66), dict(dim=63), dict(heads=0), dict(heads=1025), dict(xt=-1), dict(yh=-64)):
        assert _rot(**bad) == SHAPE, bad
    assert _rot(amp=math.inf) == VALUE and _rot(amp=math.nan) == VALUE
    assert _rot(x=OFF) == ALIGN and _rot(y=OFF) == ALIGN and _rot(freqs=OK + 4) == ALIGN and _rot(pos=OK + 4) == ALIGN
    assert _rot(x=OK + 2, dt=F32) == ALIGN
    assert _rot(T=0, x=None, y=None) == 0


def test_binding_refuses_rotary():
    x, f = _bf(4, 2, 64), torch.zeros(32, dtype=torch.float64)
    for call, err in (
            (lambda: q.qlora_rotary(x, None, None, f), ValueError),  # no GPU
            (lambda: q.qlora_rotary(x.half(), None, None, f), TypeError),
            (lambda: q.qlora_rotary(x[0], None, None, f), ValueError),
            (lambda: q.qlora_rotary(x, x.float(), None, f), TypeError),
            (lambda: q.qlora_rotary(x, _bf(3, 2, 64), None, f), ValueError),
            (lambda: q.qlora_rotary(x, _bf(4, 2, 32), None, f), ValueError),
            (lambda: q.qlora_rotary(_bf(4, 64, 2).transpose(1, 2), None, None, f), ValueError),
            (lambda: q.qlora_rotary(x, None, None, f.float()), TypeError),
            (lambda: q.qlora_rotary(x, None, None, torch.zeros(33, dtype=torch.float64)), ValueError),
            (lambda: q.qlora_rotary(x, None, None, torch.zeros(0, dtype=torch.float64)), ValueError),
            (lambda: q.qlora_rotary(x, None, torch.zeros(3, dtype=torch.int64), f), ValueError),
            (lambda: q.qlora_rotary(x, None, torch.zeros(4), f), TypeError),
            (lambda: q.qlora_rotary(x, None, None, f, amplitude=math.inf), ValueError),
            (lambda: q.qlora_rotary(x, None, None, f, amplitude=1e39), ValueError),
            (lambda: q.qlora_rotary(x, None, None, None), TypeError),
            (lambda: q.qlora_rotary(_bf(4, 2, 1026), None, None, f), ValueError)):
        with pytest.raises(err):
            call()
    for a, b in ((x, x), (x, x[:, 1:]), (x[:1].expand(4, 2, 64), None), (x.view(8, 1, 64).expand(8, 2, 64), None)):
        with pytest.raises(ValueError, match="overlap"):
            q.qlora_rotary(a, b, None, f, inplace=True)
    y = _bf(4, 6 * 64)
    with pytest.raises(ValueError, match="GPU"):  # side by side: nothing overlaps
        q.qlora_rotary(y[:, :128].view(4, 2, 64), y[:, 128:256].view(4, 2, 64), None, f, inplace=True)


def test_rotary_frequencies():
    f, amp = q.rotary_frequencies(64, device="cpu")
    assert amp == 1.0 and f.dtype == torch.float64 and f[0] == 1.0 and abs(f[31] - 10000.0 ** (-62 / 64)) < 1e-18
    lin, _ = q.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, f / 4)
    base, _ = q.rotary_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert base[0] == 1.0 and abs(base[31] / f[31] * 4 - 1) < 1e-12
    bands, amp = q.rotary_frequencies(64, scaling="bands", factor=8.0, trained=4096, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert abs(amp - (1 + math.log(8) / 10)) < 1e-15
    assert torch.equal(bands[turns >= 32], f[turns >= 32]) and torch.allclose(bands[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    for bad in (dict(dim=3), dict(dim=0), dict(dim=64, theta=0.0), dict(dim=64, factor=0.5), dict(dim=64, scaling="other"),
                dict(dim=64, scaling="bands", factor=2.0), dict(dim=2, scaling="base"), dict(dim=2000)):
        with pytest.raises(ValueError):
            q.rotary_frequencies(**{"device": "cpu", **bad})


# --- the gated block -----------------------------------------------------------

def _w(d_out=64, d_in=128, codes=OK, qs=OK, sm=OK):
    return ctypes.byref(q._Nf4Weight(d_out, d_in, codes, qs, sm))


def _gf(w=None, x=OK, T=4, A=OK, B=OK, r=8, act=0, a=OK, h=None, u=None, ws=OK, n=BIG):
    return q.lib.qlora_gated_forward(w or _w(), x, T, A, B, r, 16.0, act, a, h, u, ws, n, None)


def _gb(w=None, x=OK, h=OK, da=OK, T=4, A=OK, B=OK, r=8, act=0, u=None, dX=OK, dA=OK, dB=OK, dh=None, ws=OK, n=BIG):
    return q.lib.qlora_gated_backward(w or _w(), x, h, da, T, A, B, r, 16.0, act, u, dX, dA, dB, dh, ws, n, None)


def test_gated_forward_refuses():
    assert _gf(w=_w(d_out=48)) == SHAPE and _gf(w=_w(d_in=100)) == SHAPE and _gf(w=_w(d_out=1 << 20, d_in=1 << 17)) == SHAPE
    assert _gf(act=2) == VALUE and _gf(act=-1) == VALUE
    assert _gf(x=None) == NULL and _gf(a=None) == NULL and _gf(A=None) == NULL and _gf(w=_w(codes=None)) == NULL
    assert _gf(T=0) == SHAPE and _gf(r=12) == SHAPE and _gf(T=(1 << 24) + 1) == SHAPE
    assert _gf(a=OFF) == ALIGN and _gf(h=OFF) == ALIGN and _gf(u=OFF) == ALIGN
    need = q.qlora_workspace_bytes(64, 128, 4, 8)
    assert _gf(n=need - 1) == WORKSPACE and _gf(ws=None) == NULL and _gf(ws=OFF) == ALIGN


def test_gated_backward_refuses():
    assert _gb(w=_w(d_out=48)) == SHAPE and _gb(act=7) == VALUE
    assert _gb(h=None) == NULL and _gb(da=None) == NULL and _gb(B=None) == NULL
    assert _gb(A=None, B=None) == SHAPE and _gb(x=None) == NULL and _gb(x=None, dA=None) == NULL
    assert _gb(dh=OFF) == ALIGN and _gb(da=OFF) == ALIGN and _gb(dX=OFF) == ALIGN and _gb(T=0) == SHAPE
    need = q.qlora_gated_workspace_bytes(64, 128, 4, 8)
    assert need >= q.qlora_workspace_bytes(64, 128, 4, 8) + 4 * 64 * 2
    assert _gb(n=need - 1) == WORKSPACE and _gb(ws=None) == NULL
    assert _gb(n=q.qlora_workspace_bytes(64, 128, 4, 8) - 1, dh=OK) == WORKSPACE
    assert _gb(dX=None, dA=None, dB=None, n=need) == 0  # nothing asked, nothing done
    assert q.qlora_gated_workspace_bytes(64, 128, 0, 8) == 0


def test_binding_refuses_gated():
    def weight(d_out=64, d_in=128):
        n = d_out * d_in
        return q.NF4Weight(d_out, d_in, torch.zeros(n // 2, dtype=torch.uint8), torch.zeros(n // 64, dtype=torch.uint8),
                           torch.zeros(-(-n // 64 // 256)))

    w, x, h, da = weight(), _bf(4, 128), _bf(4, 64), _bf(4, 32)
    fp8 = q.Fp8Weight(64, 128, torch.zeros(64, 128, dtype=q.E4M3), torch.zeros(1, 1))
    f, b = q.qlora_gated_forward, q.qlora_gated_backward
    for call, err in (
            (lambda: f(w, x, None, None, 1.0), ValueError),  # no GPU
            (lambda: b(w, None, h, da, None, None, 1.0), ValueError),
            (lambda: f(fp8, x, None, None, 1.0), TypeError),
            (lambda: f(weight(48), x, None, None, 1.0), ValueError),
            (lambda: f(w, x, None, None, 1.0, act="relu"), ValueError),
            (lambda: f(w, x.float(), None, None, 1.0), TypeError),
            (lambda: f(w, _bf(0, 128), None, None, 1.0), ValueError),
            (lambda: f(w, _bf(4, 64), None, None, 1.0), ValueError),
            (lambda: f(w, x, _bf(8, 128), None, 1.0), ValueError),
            (lambda: f(w, x, _bf(8, 128), _bf(32, 8), 1.0), ValueError),
            (lambda: f(w, x, None, None, 1.0, a=_bf(4, 64)), ValueError),
            (lambda: f(w, x, None, None, 1.0, u=torch.zeros(4, 8)), ValueError),
            (lambda: f(w, x, None, None, 1.0, ws=torch.zeros(8, dtype=torch.uint8)), ValueError),
            (lambda: b(w, None, None, da, None, None, 1.0), TypeError),
            (lambda: b(w, None, h, h, None, None, 1.0), ValueError),
            (lambda: b(w, None, h, da, _bf(8, 128), _bf(64, 8), 1.0), ValueError),
            (lambda: b(w, None, h, da, None, None, 1.0, dA=torch.zeros(8, 128)), ValueError),
            (lambda: b(w, None, h, da, None, None, 1.0, act=None), ValueError)):
        with pytest.raises(err):
            call()
    with pytest.raises(ValueError, match="overlaps"):
        f(w, x, None, None, 1.0, a=x.view(-1)[:128].view(4, 32))
    with pytest.raises(ValueError, match="overlaps"):
        b(w, None, h, da, None, None, 1.0, dh=h)


# --- attention -------------------------------------------------------------------

def _at(B=1, T=4, S=8, heads=4, kv=2, D=64, window=16, sinks=1, scale=0.125, lengths=None, offsets=None):
    return q._Attention(B, T, S, heads, kv, D, window, sinks, scale, lengths, offsets)


def _rows(p=OK, batch=2048, token=256, head=64):
    return ctypes.byref(q._AttentionRows(p, batch, token, head))


def _af(p=None, rq=None, rk=None, rv=None, o=OK, lse=None, ws=OK, n=BIG, none=()):
    args = [ctypes.byref(p or _at()), rq or _rows(), rk or _rows(), rv or _rows()]
    return q.lib.qlora_attention_forward(*[None if i in none else a for i, a in enumerate(args)], o, lse, ws, n, None)


def _ab(p=None, rd=None, rq=None, rk=None, rv=None, ro=None, lse=OK, dq=OK, dk=OK, dv=OK, ws=OK, n=BIG, none=()):
    args = [ctypes.byref(p or _at())] + [r or _rows() for r in (rd, rq, rk, rv, ro)]
    return q.lib.qlora_attention_backward(*[None if i in none else a for i, a in enumerate(args)], lse, dq, dk, dv, ws, n, None)


def test_attention_refuses():
    for call in (_af, _ab):
        for i in range(4 if call is _af else 6):
            assert call(none=(i,)) == NULL
        for bad in (dict(B=0), dict(T=0), dict(S=0), dict(T=(1 << 24) + 1), dict(heads=0), dict(heads=1025), dict(heads=3),
                    dict(kv=0), dict(D=96), dict(D=0), dict(B=1 << 24, T=1 << 10), dict(B=1 << 25)):
            assert call(p=_at(**bad)) == SHAPE, bad
        for bad in (dict(window=0), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
                    dict(scale=1e-40), dict(scale=3e38)):
            assert call(p=_at(**bad)) == VALUE, bad
        assert call(p=_at(lengths=OK + 2)) == ALIGN and call(p=_at(offsets=OK + 1)) == ALIGN
        assert call(rq=_rows(p=None)) == NULL and call(rk=_rows(p=OK + 8)) == ALIGN and call(rv=_rows(head=4)) == ALIGN
        assert call(rq=_rows(batch=4)) == ALIGN and call(rk=_rows(token=257)) == ALIGN
        assert call(rq=_rows(token=56)) == SHAPE and call(rk=_rows(head=-64)) == SHAPE and call(rv=_rows(token=1 << 41)) == SHAPE
        assert call(rk=_rows(token=1 << 24)) == SHAPE  # 66 rows past 2^31 bytes
        assert call(ws=None) == NULL and call(ws=OFF) == ALIGN
    assert _af(o=None) == NULL and _af(o=OFF) == ALIGN and _af(lse=OK + 2) == ALIGN
    assert _ab(lse=None) == NULL and _ab(dq=None) == NULL and _ab(dk=OFF) == ALIGN and _ab(dv=None) == NULL
    f, b = q.lib.qlora_attention_workspace_bytes, q.lib.qlora_attention_backward_workspace_bytes
    assert f(1, 4, 8, 4, 2, 64, 16, 1) >= q.COUNTER_BYTES and b(1, 4, 8, 4, 2, 64, 16, 1) >= 4 * 4 * 4
    assert f(0, 4, 8, 4, 2, 64, 16, 1) == 0 and b(1, 4, 8, 4, 3, 64, 16, 1) == 0 and f(1, 4, 8, 4, 2, 64, 0, 1) == 0
    assert _af(n=f(1, 4, 8, 4, 2, 64, 16, 1) - 1) == WORKSPACE
    assert _ab(n=b(1, 4, 8, 4, 2, 64, 16, 1) - 1) == WORKSPACE


def test_binding_refuses_attention():
    x, kv = _bf(2, 3, 4, 64), _bf(2, 5, 2, 64)
    lse = torch.zeros(2, 4, 3)
    f, b = q.qlora_attention_forward, q.qlora_attention_backward
    for call, err in (
            (lambda: f(x, kv, kv), ValueError),  # no GPU
            (lambda: b(x, x, kv, kv, x, lse), ValueError),
            (lambda: f(x.float(), kv, kv), TypeError),
            (lambda: f(x, kv, None), TypeError),
            (lambda: f(x[0], kv, kv), ValueError),
            (lambda: f(x, kv, kv[:, :4]), ValueError),
            (lambda: f(x, kv[:1], kv[:1]), ValueError),
            (lambda: f(_bf(2, 3, 5, 64), kv, kv), ValueError),
            (lambda: f(_bf(2, 3, 4, 96), _bf(2, 5, 2, 96), _bf(2, 5, 2, 96)), ValueError),
            (lambda: f(_bf(2, 3, 64, 4).transpose(2, 3), kv, kv), ValueError),
            (lambda: f(_bf(2 * 3 * 4 * 68).view(2, 3, 4, 68)[..., :64], kv, kv), ValueError),
            (lambda: f(_bf(2 * 3 * 256 + 4)[4:].view(2, 3, 4, 64), kv, kv), ValueError),
            (lambda: f(x[:, :1].expand(2, 3, 4, 64), kv, kv), ValueError),
            (lambda: f(x, kv, kv, window=0), ValueError),
            (lambda: f(x, kv, kv, window=2.5), TypeError),
            (lambda: f(x, kv, kv, sinks=-1), ValueError),
            (lambda: f(x, kv, kv, scale=0.0), ValueError),
            (lambda: f(x, kv, kv, scale=math.nan), ValueError),
            (lambda: f(x, kv, kv, lengths=torch.zeros(2, dtype=torch.int64)), TypeError),
            (lambda: f(x, kv, kv, offsets=torch.zeros(3, dtype=torch.int32)), ValueError),
            (lambda: b(x, x, kv, kv, x, None), TypeError),
            (lambda: b(x[:, :2], x, kv, kv, x, lse), ValueError),
            (lambda: b(x, x, kv, kv, x.float(), lse), TypeError),
            (lambda: b(x, x, kv, kv, x, lse[:, :2]), ValueError)):
        with pytest.raises(err):
            call()


def test_attention_backward_scratch_is_bounded():
    """The rows' statistics (32 bytes a row) and at most a workgroup or two per compute unit of sums over the sinks' rows
    (128 keys, dK and dV in float32), whatever the window and the sinks."""
    f = q.lib.qlora_attention_backward_workspace_bytes
    for B, T, S, H, G, D, window, sinks in ((1, 1 << 20, 1 << 20, 1, 1, 128, (1 << 20) - 1, 4), (2, 4096, 4096, 40, 8, 128, 1024, 4),
                                            (1, 4096, 1 << 24, 8, 8, 128, 1024, 1 << 24), (1, 1 << 24, 1 << 24, 1, 1, 64, 1, 1 << 24),
                                            (64, 512, 512, 32, 32, 128, 64, 1), (1, 1 << 20, 1 << 20, 8, 8, 128, 1, 128)):
        n = f(B, T, S, H, G, D, window, sinks)
        assert 32 * B * T * H <= n <= 32 * B * T * H + 512 * 2 * 128 * D * 4, (B, T, S, window, sinks, n)


def test_attention_takes_heads_that_lie_far_apart():
    """Heads in front of many tokens: only the rows of a head have to lie less than 2^24 values apart. (The workspace is too
    small in every call, so that nothing is enqueued.)"""
    T = 1 << 20
    p = dict(B=1, T=T, S=T, heads=8, kv=1, D=128)
    far = lambda: _rows(batch=8 * 128 * T, token=128, head=128 * T)  # noqa: E731
    assert _af(p=_at(**p), rq=far(), rk=far(), rv=far(), n=0) == WORKSPACE
    assert _ab(p=_at(**p), rd=far(), rq=far(), rk=far(), rv=far(), ro=far(), n=0) == WORKSPACE
    assert _af(rq=_rows(head=1 << 40, batch=1 << 40), n=0) == WORKSPACE and _af(rq=_rows(head=1 << 41), n=0) == SHAPE
    for call, names in ((_af, ("rq", "rk", "rv")), (_ab, ("rd", "rq", "rk", "rv", "ro"))):
        for name in names:
            assert call(**{name: _rows(token=(1 << 24) - 8)}, n=0) == WORKSPACE, name
            assert call(**{name: _rows(token=1 << 24)}, n=0) == SHAPE, name
    # (no memory behind it that a check could touch)
    far = torch.empty(0, dtype=torch.bfloat16, device="meta").new_empty(2 * 3 << 24).as_strided((2, 3, 4, 64), (3 << 24, 1 << 24, 64, 1))
    with pytest.raises(ValueError, match="strides"):
        q._attention_rows(far, "q", (2, 3, 4, 64))
    near = far.as_strided((2, 3, 4, 64), (3 << 24, (1 << 24) - 8, 64, 1))
    assert q._attention_rows(near, "q", (2, 3, 4, 64)).token == (1 << 24) - 8


def test_attention_refuses_more_workgroups_than_a_launch_takes():
    """2^24 workgroups of 256 threads are one too many: refused as a shape, not by the launch. (Else the workspace is too
    small, so that nothing is enqueued.)"""
    most = 1 << 24
    for sizes, err in ((dict(B=most, T=1, S=1, heads=1, kv=1), SHAPE), (dict(B=most - 1, T=1, S=1, heads=1, kv=1), WORKSPACE),
                       (dict(B=most // 16, T=1, S=128, heads=16, kv=16), SHAPE),
                       (dict(B=most // 16 - 1, T=1, S=128, heads=16, kv=16), WORKSPACE),
                       (dict(B=most // 32, T=129, S=1, heads=16, kv=16), SHAPE), (dict(B=most // 32, T=33, S=1, heads=64, kv=16), SHAPE),
                       (dict(B=most // 32, T=32, S=1, heads=64, kv=16), WORKSPACE)):
        for call in (_af, _ab):
            assert call(p=_at(**sizes), n=0) == err, sizes
    x = torch.empty(0, dtype=torch.bfloat16, device="meta").new_empty(most, 1, 1, 64)
    with pytest.raises(ValueError, match="too many"):
        q.qlora_attention_forward(x, x, x)


def test_attention_scales_end_where_its_backward_does():
    """lse of up to log(2^24) over the scale is added to the scores in float32: at 1e-38 that would be infinite. Every entry has
    the binding's limits."""
    for call in (_af, _ab):
        for scale in (1e-38, 9e-39, 5e-38, 9e-31, 2e30, 1e38):
            assert call(p=_at(scale=scale), n=0) == VALUE, scale
        for scale in (2e-30, 1.0, 9e29):
            assert call(p=_at(scale=scale), n=0) == WORKSPACE, scale
    assert math.log(1 << 24) / 2e-30 < 3.4e38 < math.log(1 << 24) / 4e-38


def test_scales_that_the_binding_takes_pass_the_entry_too():
    """The binding compares in 64 bits, the entries the float32 that they get: one just above 1e-30 rounds to it."""
    for scale in (1e-30 * (1 + 1e-12), 1e30 * (1 - 1e-12)):
        assert 1e-30 < scale < 1e30
        for call in (_af, _ab):
            assert call(p=_at(scale=scale), n=0) == WORKSPACE, scale
