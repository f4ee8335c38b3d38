"""The AdamW step over many tensors writes its parameters and state while it reads its gradients: calls where these share
memory are refused before anything is enqueued, by the binding without a GPU and by the native marshalling with one."""

import os

import pytest
import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.LIB):
    _build.build()
from bit_quantized_finetuning_amd import qlora as q  # noqa: E402


def _overlaps(device):
    """(what shares memory with a gradient, the call)"""
    z = lambda n, **kw: torch.zeros(n, device=device, **kw)  # noqa: E731

    def call(grads=None, params=None, m=None, v=None, **kw):
        grads, params = grads or [z(300)], params or [z(300)]
        n = q.adamw_state_elements([p.numel() for p in params])
        return lambda: q.qlora_adamw_many(1, grads, params, z(n) if m is None else m, z(n) if v is None else v, **kw)

    p, m, both = z(300), z(512), z(1000)
    yield "its own parameter", call([p], [p])
    yield "its parameter, shifted", call([both[4:304]], [both[:300]])
    yield "another parameter", call([z(300), p], [p, z(300)])
    yield "m", call([m[4:304]], m=m)
    yield "the end of m", call([m[240:252]], [z(12)], m=m[:256], v=m[256:])
    yield "v", call([m[260:272]], [z(12)], m=m[:256], v=m[256:])
    master = z(512)
    yield "the master copy", call([master.view(torch.bfloat16)[:300]], [z(300, dtype=torch.bfloat16)], master=master)
    m8, scale = z(512).to(q.E4M3), z(2)
    yield "8-bit m", call([m8.view(torch.float32)[:100]], [z(100)], m=m8[:256], v=z(256).to(q.E4M3), m_scale=z(1), v_scale=z(1))
    yield "a scale", call([scale[:1]], [z(1)], m=z(256).to(q.E4M3), v=z(256).to(q.E4M3), m_scale=scale[:1], v_scale=z(1))
    norm = z(4)
    yield "norm", call([norm], [z(4)], max_norm=1.0, norm=norm[:1])


CASES = [name for name, _ in _overlaps("cpu")]


@pytest.mark.parametrize("name", CASES)
def test_binding_refuses(name):
    with pytest.raises(ValueError, match="overlap"):
        dict(_overlaps("cpu"))[name]()


def test_binding_refuses_a_workspace_among_the_arguments():
    buf = torch.zeros(1 << 16, dtype=torch.uint8)
    inside, apart = buf[-400:].view(torch.float32), torch.zeros(100)
    for grad, param in ((inside, apart), (apart, inside)):
        with pytest.raises(ValueError, match="overlap"):
            q.qlora_adamw_many(1, [grad], [param], torch.zeros(256), torch.zeros(256), max_norm=1.0, ws=buf)


def test_gradients_may_overlap_each_other():
    """And lie beside the parameters: the call gets as far as asking for a GPU."""
    buf = torch.zeros(700)
    g = buf[:300]
    with pytest.raises(ValueError, match="GPU"):
        q.qlora_adamw_many(1, [g, g], [buf[300:600], torch.zeros(300)], torch.zeros(1024), torch.zeros(1024))


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_native_marshalling_refuses(name):
    print(f"adamw overlap: {name}", flush=True)
    with pytest.raises(ValueError, match="overlap"):
        dict(_overlaps("cuda"))[name]()


@pytest.mark.gpu
def test_native_marshalling_takes_shared_gradients():
    """One gradient for two parameters, gradients and parameters side by side in one buffer."""
    print("adamw: one gradient twice, beside the parameters", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(5)
    buf = torch.randn(1024, generator=gen, device="cuda")
    g, p, p2 = buf[:256], buf[256:512], buf[512:768]
    apart = [t.clone() for t in (g, g, p, p2)]
    state = lambda: (torch.zeros(512, device="cuda"), torch.zeros(512, device="cuda"))  # noqa: E731
    q.qlora_adamw_many(1, [g, g], [p, p2], *state(), max_norm=1.0)
    q.qlora_adamw_many(1, apart[:2], apart[2:], *state(), max_norm=1.0)
    assert torch.equal(p, apart[2]) and torch.equal(p2, apart[3]) and torch.equal(g, apart[0])
