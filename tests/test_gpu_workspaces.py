"""Calls and modules that name no workspace (needs an MI355X): on overlapping streams, from threads that share a stream,
and captured into graphs that are replayed beside each other; every result as from the same call alone."""

import threading
import zlib

import pytest
import torch

from gpu_common import product, say

pytestmark = pytest.mark.gpu

q = product("qlora")
layer = product("layer")


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


SIZES = [(16, 1024, 2048, 64), (300, 528, 784, 16), (1, 4096, 1040, 8), (333, 1024, 2048, 16), (40, 272, 4096, 128)]


def _calls(base):
    """One forward and one backward of each size over the base, as functions without arguments."""
    out = []
    for T, N, K, r in SIZES:
        if base == "nf4" and K % 64:
            K = 64 * (K // 64)
        g = _gen(base, T, N, K)
        W = _randn(g, N, K) * 0.02
        w = q.qlora_fp8_quantize(W) if base == "fp8" else q.qlora_quantize(W)
        x, dY = _randn(g, T, K).bfloat16(), _randn(g, T, N).bfloat16()
        A, B = (_randn(g, r, K) * 0.02).bfloat16(), (_randn(g, N, r) * 0.02).bfloat16()
        fwd, bwd = (q.qlora_fp8_forward, q.qlora_fp8_backward) if base == "fp8" else (q.qlora_forward, q.qlora_backward)
        out.append(lambda f=fwd, a=(w, x, A, B, 16.0): f(*a, save_u=True))
        out.append(lambda f=bwd, a=(w, x, dY, A, B, 16.0): f(*a))
    return out


def _same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("base", ["fp8", "nf4"])
def test_overlapping_streams(base):
    say(f"default workspaces on two streams, {base}")
    calls = _calls(base)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(4):
        for i in range(len(calls)):
            for s, st in enumerate(streams):  # the streams run through the calls from different ends
                j = i if s == 0 else len(calls) - 1 - i
                with torch.cuda.stream(st):
                    got.append((j, calls[j]()))
    torch.cuda.synchronize()
    for j, out in got:
        assert _same(out, want[j]), j


@pytest.mark.parametrize("base", ["fp8", "nf4"])
def test_threads_that_share_a_stream(base):
    say(f"default workspace from two threads, {base}")
    calls = _calls(base)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def run(s):
        try:
            for k in range(4):
                for i in range(len(calls)):
                    j = i if s == 0 else len(calls) - 1 - i
                    got[s].append((j, calls[j]()))
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(s,)) for s in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for j, out in got[0] + got[1]:
        assert _same(out, want[j]), j


def test_modules_on_overlapping_streams():
    """Forward and backward of modules over the 8-bit base, which give no way to pass a workspace."""
    say("fp8 modules on two streams")
    jobs = []
    for k, (T, N, K) in enumerate(((333, 1024, 2048), (16, 2048, 784))):
        g = _gen("modules", k)
        m = layer.QLoRALinear(_randn(g, N, K) * 0.02, r=16, base="fp8", generator=g)
        with torch.no_grad():
            m.B.copy_(_randn(g, N, 16) * 0.02)
        jobs.append((m, _randn(g, T, K).bfloat16(), _randn(g, T, N).bfloat16()))

    def step(m, x, dh):
        x = x.detach().requires_grad_(True)
        m.A.grad = m.B.grad = m.A.grad_fp32 = m.B.grad_fp32 = None
        h = m(x)
        h.backward(dh)
        return h.detach(), x.grad, m.A.grad_fp32, m.B.grad_fp32

    want = [step(*j) for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], []
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((i, step(*jobs[i])))
    torch.cuda.synchronize()
    for i, out in got:
        assert _same(out, want[i]), i


@pytest.mark.parametrize("base", ["fp8", "nf4"])
def test_graphs_replayed_beside_each_other(base):
    """Two graphs of all calls, replayed on two streams at once with eager calls on a third; the first calls of a graph
    find no workspace yet, and later ones need a larger one."""
    say(f"default workspaces in two graphs, {base}")
    calls = _calls(base)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append([c() for c in (calls if s == 0 else calls[::-1])])
        graphs.append(gr)
    assert q._capture_id(torch.device("cuda", 0), torch.cuda.current_stream().cuda_stream) == 0
    streams = [torch.cuda.Stream() for _ in graphs]
    for k in range(4):
        for o in outs:
            for out in o:
                for t in out:
                    t.fill_(7)
        torch.cuda.synchronize()
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        eager = [c() for c in calls]
        torch.cuda.synchronize()
        for i, w in enumerate(want):
            assert _same(outs[0][i], w) and _same(outs[1][len(calls) - 1 - i], w) and _same(eager[i], w), (k, i)


@pytest.mark.parametrize("T,r", [(1, 16), (16, 64), (5, 256)])
def test_one_workspace_on_two_streams_in_turn(T, r):
    """The adapter's x A^T travels between workgroups in the workspace: calls on two streams, ordered by events, that
    find the other stream's values there, each with new inputs."""
    say(f"fp8 one workspace, two streams in turn T={T} r={r}")
    N, K = 1024, 2064
    g = _gen("turns", T, r)
    w = q.qlora_fp8_quantize(_randn(g, N, K) * 0.02)
    A, B = (_randn(g, r, K) * 0.02).bfloat16(), (_randn(g, N, r) * 0.02).bfloat16()
    xs = [_randn(g, T, K).bfloat16() for _ in range(40)]
    fresh = lambda: torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")  # noqa: E731
    want = [q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=fresh()) for x in xs]
    ws = fresh()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for k, x in enumerate(xs):
        st = streams[k % 2]
        st.wait_stream(streams[(k + 1) % 2])
        with torch.cuda.stream(st):
            got.append(q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws))
    torch.cuda.synchronize()
    for k, (a, b) in enumerate(zip(got, want)):
        assert _same(a, b), k


@pytest.mark.parametrize("T,r", [(1, 16), (16, 64)])
def test_captured_call_with_a_given_workspace(T, r):
    """A replay finds the values of the replay before it in the workspace: it takes its own."""
    say(f"fp8 captured call, given workspace T={T} r={r}")
    N, K = 1024, 2064
    g = _gen("replay", T, r)
    w = q.qlora_fp8_quantize(_randn(g, N, K) * 0.02)
    A, B = (_randn(g, r, K) * 0.02).bfloat16(), (_randn(g, N, r) * 0.02).bfloat16()
    x = _randn(g, T, K).bfloat16()
    ws = torch.zeros(q.qlora_fp8_workspace_bytes(N, K, T, r), dtype=torch.uint8, device="cuda")
    q.qlora_fp8_forward(w, x, A, B, 16.0, ws=ws)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True, ws=ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(12):
        x.copy_(_randn(g, T, K))
        want = q.qlora_fp8_forward(w, x, A, B, 16.0, save_u=True)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[k % 2]):
            gr.replay()
        torch.cuda.synchronize()
        assert _same(out, want), k
