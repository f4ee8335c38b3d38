"""A stack of decoder layers built from the QLoRA projections: the chained-layer setting of the pages' 14B runs.

"8GB, 12GB, 16GB, 24GB GPU에서 몇 B 모델까지 LoRA 학습이 될까", section "무엇을 돌렸나": a 14B model (hidden
5120, MLP 17408, 40 layers) with 4-bit NF4 + double-quant base weights, LoRA r = 8, alpha = 16 on q_proj and
v_proj only, bf16 compute, gradient checkpointing, one sequence of 2048 tokens.

Each layer holds its seven projections as the library's frozen NF4 weights: q/k/v stacked into one call that
reads the normalized input once (q and v adapted), o, gate/up stacked into one call, and down. k and v are
1024 x 5120 (8 KV heads of 128 for 40 query heads). Everything between the projections is plain torch glue and
stands in for parts of the model that are not on this path:
  * RMS normalization (no weight) before q/k/v and before gate/up;
  * attention is replaced by a gate that mixes q with k and v expanded to the query heads,
    a = q * sigmoid(k) + v, so that every projection's output reaches the loss;
  * the MLP activation is SiLU(gate) * up; residual adds around both halves.
With checkpoint=True each layer keeps only its input and runs its forward again in the backward
(torch.utils.checkpoint, non-reentrant).

base="fp8" keeps the projections' frozen weights in 8-bit floating point instead: the norms are then the library's
(QLoRARMSNorm), which write the 8-bit rows that q/k/v and gate/up multiply, and the one before the MLP adds the
residual in the same pass. grad_fmt is then the 8-bit format of the projections' upstream gradients.

With attention=True the gate in attention's place gives way to the library's attention: q and k are turned to their
positions (QLoRARotary over the whole head), and causal attention with a sliding window and sinks follows
(QLoRAAttention). x is then one sequence [T, hidden] or a batch [B, T, hidden], with `lengths` (int32 [B]) for sequences
that are padded behind their end; and with a KeyValueCache per layer (DecoderStack.caches) the tokens of x continue the
sequences that the cache holds, a prompt at once or token by token (inference only). gated="silu" or "gelu" forms the
activation's product within the gate/up call (QLoRAGated, 4-bit base only; "gelu" is its form in tanh).

Weights come from the seeded device generator of the synthetic-input module, one seed per layer, so that a
layer's weights can be drawn again to check it.
"""

from __future__ import annotations

import torch
import torch.nn.functional as F
from torch.utils.checkpoint import checkpoint

from . import synth
from . import qlora as q_
from .layer import KeyValueCache, QLoRAAttention, QLoRAFusedLinear, QLoRAGated, QLoRALinear, QLoRARMSNorm, QLoRARotary

HEAD = 128


def rms_norm(x: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    """x / sqrt(mean(x^2) + eps) over the last dimension, bf16 in and out (torch's fused norm)."""
    return F.rms_norm(x, (x.shape[-1],), eps=eps)


class DecoderProjections(torch.nn.Module):
    """One decoder layer of projections (see the module docstring); `weights` maps q, k, v, o, gate, up, down to
    bf16 [d_out, d_in] tensors."""

    # of layers saved before there was a choice
    base = "nf4"
    attends = False
    gated = None

    def __init__(self, weights: dict, r: int = 8, alpha: float = 16.0, generator: torch.Generator | None = None,
                 head: int = HEAD, base: str = "nf4", grad_fmt=None, attention: bool = False, window: int | None = None,
                 sinks: int = 0, theta: float = 10000.0, gated: str | None = None):
        super().__init__()
        if gated is not None and base != "nf4":
            raise ValueError("gated is for the 4-bit base")
        if not attention and (window is not None or sinks):
            raise ValueError("window and sinks are for attention=True")
        if attention and head not in (64, 128):
            raise ValueError(f"attention has heads of 64 or 128 values, got {head}")
        self.base, self.attends, self.gated = base, bool(attention), gated
        self.hidden, self.kv, self.head = weights["q"].shape[0], weights["k"].shape[0], head
        if self.hidden % head or self.kv % head or self.hidden % self.kv:
            raise ValueError("q and k/v widths must be multiples of the head width, q's of k's")
        self.qkv = QLoRAFusedLinear([weights["q"], weights["k"], weights["v"]], r=r, alpha=alpha,
                                    adapted=[True, False, True], generator=generator, base=base, grad_fmt=grad_fmt)
        self.o = QLoRALinear(weights["o"], r=0, base=base, grad_fmt=grad_fmt)
        if gated is None:
            self.gate_up = QLoRAFusedLinear([weights["gate"], weights["up"]], r=0, base=base, grad_fmt=grad_fmt)
        else:
            self.gate_up = QLoRAGated(weights["gate"], weights["up"], r=0, act=gated)
        self.down = QLoRALinear(weights["down"], r=0, base=base, grad_fmt=grad_fmt)
        self.norm = QLoRARMSNorm(self.hidden, fmt=q_.E4M3) if base == "fp8" else None
        if attention:
            self.rotary = QLoRARotary(head, theta, device=weights["q"].device)
            self.attention = QLoRAAttention(window, sinks)

    def _heads(self, t: torch.Tensor, rep: int) -> torch.Tensor:
        """[T, n * head] -> [T, kv heads, rep, head] (a view; k and v broadcast over the query heads they serve)."""
        return t.view(t.shape[0], self.kv // self.head, rep, self.head)

    def forward(self, x: torch.Tensor, lengths: torch.Tensor | None = None, cache: KeyValueCache | None = None):
        """x [T, hidden], with attention=True also [B, T, hidden]. lengths (int32 [B]): the tokens of each sequence that
        are its own; cache: the sequences that x continues."""
        if not self.attends:
            if lengths is not None or cache is not None:
                raise ValueError("lengths and cache are for attention=True")
            return self._layer(x, self._mix)
        if x.dim() not in (2, 3):
            raise ValueError(f"x must be [T, hidden] or [B, T, hidden], got {tuple(x.shape)}")
        B, T = (1, x.shape[0]) if x.dim() == 2 else x.shape[:2]
        y = self._layer(x.reshape(B * T, self.hidden), lambda q, k, v: self._attend(q, k, v, B, T, lengths, cache))
        return y.reshape(x.shape)

    def _layer(self, x: torch.Tensor, between) -> torch.Tensor:
        if self.base == "fp8":
            y, _, yq, ys = self.norm(x)
            q, k, v = self.qkv(y, yq, ys)
            a = between(q, k, v)
            y, x1, yq, ys = self.norm(self.o(a.reshape(x.shape[0], self.hidden)), residual=x)
            g, u = self.gate_up(y, yq, ys)
            return x1 + self.down(F.silu(g) * u)
        q, k, v = self.qkv(rms_norm(x))
        a = between(q, k, v)
        x1 = x + self.o(a.reshape(x.shape[0], self.hidden))
        if self.gated is not None:
            return x1 + self.down(self.gate_up(rms_norm(x1)))
        g, u = self.gate_up(rms_norm(x1))
        return x1 + self.down(F.silu(g) * u)

    def _attend(self, q, k, v, B: int, T: int, lengths, cache) -> torch.Tensor:
        """Attention of q [B T, hidden] over k, v [B T, kv], or over the cache once they are in it."""
        q, k, v = (t.unflatten(-1, (-1, self.head)).unflatten(0, (B, T)) for t in (q, k, v))
        if cache is None:
            q, k = self.rotary(q, k)
            return self.attention(q, k, v, lengths, None if lengths is None else torch.zeros_like(lengths))
        if torch.is_grad_enabled():
            raise RuntimeError("a cache is for inference: call it under torch.no_grad()")
        q, k = self.rotary(q, k, cache.positions(T))
        before = cache.append(k, v, lengths)
        return self.attention(q, cache.k, cache.v, cache.lengths, before)

    def _mix(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
        rep = self.hidden // self.kv  # query heads per KV head
        # a = q * sigmoid(k) + v with k and v broadcast to the query heads (one bf16 rounding, float32 inside)
        return torch.addcmul(self._heads(v, 1), self._heads(q, rep), torch.sigmoid(self._heads(k, 1)))


class DecoderStack(torch.nn.Module):
    """`layers` decoder layers of projections; layer i's weights are synth.stack_layer_weights(i) (shapes default
    to the 14B-style layer) and its adapters' A are drawn from synth.stack_adapter_init(i) (B starts at zero)."""

    def __init__(self, layers: int = 40, shapes: dict | None = None, r: int = 8, alpha: float = 16.0,
                 seed: int = 0, device="cuda", checkpoint: bool = True, head: int = HEAD, base: str = "nf4",
                 grad_fmt=None, attention: bool = False, window: int | None = None, sinks: int = 0,
                 theta: float = 10000.0, gated: str | None = None):
        super().__init__()
        self.shapes = dict(synth.STACK_SHAPES if shapes is None else shapes)
        self.seed = seed
        self.use_checkpoint = checkpoint
        self.layers = torch.nn.ModuleList()
        for i in range(layers):
            ws = synth.stack_layer_weights(i, device, self.shapes, seed)
            gen = synth.stack_adapter_init(i, device, seed)
            self.layers.append(DecoderProjections(ws, r=r, alpha=alpha, generator=gen, head=head, base=base,
                                                  grad_fmt=grad_fmt, attention=attention, window=window, sinks=sinks,
                                                  theta=theta, gated=gated))
            del ws

    def caches(self, batch: int, tokens: int) -> list[KeyValueCache]:
        """One cache per layer for `batch` sequences of up to `tokens` tokens (attention=True)."""
        if not all(layer.attends for layer in self.layers):
            raise ValueError("caches are for attention=True")
        return [KeyValueCache(batch, tokens, layer.kv // layer.head, layer.head, layer.qkv.codes.device)
                for layer in self.layers]

    def forward(self, x: torch.Tensor, lengths: torch.Tensor | None = None, caches=None) -> torch.Tensor:
        """lengths, caches: see DecoderProjections.forward; one cache per layer."""
        if caches is not None and len(caches) != len(self.layers):
            raise ValueError(f"{len(caches)} caches for {len(self.layers)} layers")
        for i, layer in enumerate(self.layers):
            more = {} if lengths is None else {"lengths": lengths}
            if caches is not None:
                more["cache"] = caches[i]
            if self.use_checkpoint and torch.is_grad_enabled():
                x = checkpoint(layer, x, use_reentrant=False, **more)
            else:
                x = layer(x, **more)
        return x
