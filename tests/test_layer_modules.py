"""The modules between a layer's projections without a GPU: what they refuse, and the cache's bookkeeping."""

import os

import pytest
import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.LIB):
    _build.build()
from bit_quantized_finetuning_amd import layer, stack  # noqa: E402


def test_constructors_refuse():
    w = torch.zeros(32, 64)
    for call in (lambda: layer.QLoRAGated(w, torch.zeros(48, 64)), lambda: layer.QLoRAGated(torch.zeros(8, 64), torch.zeros(8, 64)),
                 lambda: layer.QLoRAGated(w, w, act="relu"), lambda: layer.QLoRAAttention(0), lambda: layer.QLoRAAttention(4, -1),
                 lambda: layer.QLoRARotary(63, device="cpu"), lambda: layer.QLoRARotary(64, scaling="other", device="cpu"),
                 lambda: layer.KeyValueCache(1, 0, 1, 64, device="cpu"),
                 lambda: stack.DecoderProjections({}, base="fp8", gated="silu"), lambda: stack.DecoderProjections({}, window=4),
                 lambda: stack.DecoderProjections({}, sinks=1)):
        with pytest.raises(ValueError):
            call()


def test_modules_refuse():
    r = layer.QLoRARotary(64, device="cpu")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: r(x), lambda: r(x[0]), lambda: r(x, x[:3]), lambda: r(x, None, torch.arange(3)),
                 lambda: layer.QLoRAAttention()(x, x, x), lambda: layer.QLoRAAttention()(x[None], x[None], x[None])):
        with pytest.raises(ValueError):  # the last ones for want of a GPU
            call()


def test_rotary_keeps_its_frequencies():
    r = layer.QLoRARotary(64, theta=100.0, scaling="bands", factor=8.0, trained=128, device="cpu").half()
    assert r.freqs.dtype == torch.float64 and r.freqs.shape == (32,) and r.amplitude > 1 and not r.state_dict()


def test_cache():
    c = layer.KeyValueCache(3, 10, 2, 64, device="cpu")
    g = torch.Generator().manual_seed(0)

    def rows(T):
        return torch.randn(3, T, 2, 64, generator=g).bfloat16(), torch.randn(3, T, 2, 64, generator=g).bfloat16()

    k, v = rows(4)
    before = c.append(k, v, torch.tensor([4, 0, 2], dtype=torch.int32))
    assert before.tolist() == [0, 0, 0] and c.lengths.tolist() == [4, 0, 2] and c.used == 4
    k2, v2 = rows(3)
    assert c.positions(3).tolist() == [[4, 5, 6], [0, 1, 2], [2, 3, 4]]
    at = c.lengths
    before = c.append(k2, v2)
    assert before.tolist() == [4, 0, 2] and c.lengths is at and at.tolist() == [7, 3, 5]
    for got, a, b in ((c.k, k, k2), (c.v, v, v2)):
        assert torch.equal(got[0, :7], torch.cat((a[0], b[0]))) and torch.equal(got[1, :3], b[1])
        assert torch.equal(got[2, :5], torch.cat((a[2, :2], b[2])))
        assert not got[0, 7:].any() and not got[1, 3:].any() and not got[2, 5:].any()
    with pytest.raises(ValueError):
        c.append(*rows(4))
    for bad in ((k2[:2], v2[:2]), (k2, v), (k2[0], v2[0]), (k2[..., :32], v2[..., :32])):
        with pytest.raises(ValueError):
            c.append(*bad)
    with pytest.raises(ValueError):
        c.append(k2, v2, torch.tensor([1, 1, 1]))
    # counts that the host cannot see are held within the rows, and rows that do not fit are dropped
    c.append(k2, v2, torch.tensor([9, -5, 1], dtype=torch.int32))
    assert c.lengths.tolist() == [10, 3, 6]
    c.used = 0
    c.append(k2, v2)
    assert c.lengths.tolist() == [10, 6, 9] and torch.equal(c.k[1, 3:6], k2[1]) and torch.equal(c.k[0, 7:], k2[0])
    c.reset()
    assert c.lengths.tolist() == [0, 0, 0] and c.used == 0


def test_cache_counts_what_sequences_hold():
    """A padded prompt that fills the cache's rows leaves the room behind each sequence; only what does not fit is refused,
    and a refused call changes nothing."""
    c = layer.KeyValueCache(2, 64, 1, 64, device="cpu")
    g = torch.Generator().manual_seed(1)

    def rows(T):
        return torch.randn(2, T, 1, 64, generator=g).bfloat16()

    k = rows(64)
    c.append(k, k, torch.tensor([10, 7], dtype=torch.int32))
    tokens = [rows(1) for _ in range(54)]
    for t in tokens:
        c.append(t, t)
    assert c.lengths.tolist() == [64, 61] and c.used == 64
    assert torch.equal(c.k[0], torch.cat([k[0, :10]] + [t[0] for t in tokens]))
    assert torch.equal(c.v[1, :61], torch.cat([k[1, :7]] + [t[1] for t in tokens]))
    before = c._kv.clone()
    for n in (None, torch.tensor([1, 0], dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)):
        with pytest.raises(ValueError, match="64"):
            c.append(rows(5), rows(5), n)
    assert torch.equal(c._kv, before) and c.lengths.tolist() == [64, 61]
    t = rows(5)  # no row of the longer one, three of the other's
    assert c.append(t, t, torch.tensor([0, 3], dtype=torch.int32)).tolist() == [64, 61]
    assert c.lengths.tolist() == [64, 64] and torch.equal(c.k[1, 61:], t[1, :3]) and torch.equal(c.k[0], before[0, 0, :64])
    c.lengths.copy_(torch.tensor([3, 5]))  # tokens taken back
    t = rows(59)
    assert c.append(t, t).tolist() == [3, 5] and c.used == 64 and torch.equal(c.k[1, 5:], t[1])
    t = rows(70)  # more rows than the cache has, few of them a sequence's
    c.reset()
    c.append(t, t, torch.tensor([64, 2], dtype=torch.int32))
    assert c.lengths.tolist() == [64, 2] and torch.equal(c.k[0], t[0, :64]) and torch.equal(c.k[1, :2], t[1, :2])
    c.reset()
    with pytest.raises(ValueError):
        c.append(t, t)


def test_layers_refuse_heads_that_attention_has_not():
    """At the construction, not in the first call; without attention any width goes on (here to the missing weights)."""
    for head in (32, 96, 256):
        with pytest.raises(ValueError, match="64 or 128"):
            stack.DecoderProjections({}, head=head, attention=True)
        with pytest.raises(KeyError):
            stack.DecoderProjections({}, head=head)
    with pytest.raises(KeyError):
        stack.DecoderProjections({}, head=64, attention=True)
