"""Which workspace a call takes, without a GPU: one per stream, one per captured graph and stream, and whole calls of
threads that share a stream one after another. (The buffers are host memory here; streams and captures are numbers.)"""

import os
import subprocess
import threading
import time

import pytest
import torch

from bit_quantized_finetuning_amd import build as _build

if not os.path.exists(_build.LIB):
    _build.build()
from bit_quantized_finetuning_amd import qlora as q  # noqa: E402


@pytest.fixture
def now(monkeypatch):
    """The current stream and the capture it takes part in."""
    at = {"stream": 0, "capture": 0}
    monkeypatch.setattr(q, "_stream_id", lambda dev: at["stream"])
    monkeypatch.setattr(q, "_capture_id", lambda dev, stream: at["capture"])
    monkeypatch.setattr(q, "_workspaces", {})
    monkeypatch.setattr(q, "_captured", {})
    return at


def test_one_per_stream(now):
    a = q.workspace("cpu", 1000)
    assert q.workspace("cpu", 5000) is a and a.numel() >= 5000 and not a.any()
    now["stream"] = 7
    b = q.workspace("cpu", 1000)
    assert b is not a and b.data_ptr() != a.data_ptr()
    now["stream"] = 0
    assert q.workspace("cpu", 1000) is a
    big = q.workspace("cpu", a.numel() + 1)
    assert big.numel() >= 2 * a.numel() and not big.any()
    assert q.workspace("cpu", 1) is big
    now["stream"] = 7
    assert q.workspace("cpu", 1) is b


def test_one_per_captured_graph_and_stream(now):
    eager = q.workspace("cpu", 1000)
    now["capture"] = 3
    a = q.workspace("cpu", 1000)
    assert a is not eager and not a[:q.COUNTER_BYTES].any()
    a[:q.COUNTER_BYTES] = 1
    assert q.workspace("cpu", 2000) is a and a[:q.COUNTER_BYTES].all()  # cleared once, at the first call
    now["stream"] = 9
    assert q.workspace("cpu", 1000) is not a
    now.update(stream=0, capture=4)
    b = q.workspace("cpu", 1000)
    assert b is not a and not b[:q.COUNTER_BYTES].any()
    grown = q.workspace("cpu", b.numel() + 1)
    assert grown.numel() > b.numel() and not grown[:q.COUNTER_BYTES].any()
    now["capture"] = 0
    assert q.workspace("cpu", 1000) is eager


def test_threads_enqueue_whole_calls(now):
    log = []

    def call(k):
        for _ in range(5):
            with q._ws_for(None, torch.device("cpu"), 1000):
                log.append((k, "first launch"))
                time.sleep(0.001)
                log.append((k, "last launch"))

    threads = [threading.Thread(target=call, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(log) == 30
    for first, last in zip(log[::2], log[1::2]):
        assert first[0] == last[0] and (first[1], last[1]) == ("first launch", "last launch")


def test_a_given_workspace_is_the_callers(now):
    ws = torch.zeros(100, dtype=torch.uint8)
    with q._ws_for(ws, torch.device("cpu"), 100) as got:
        assert got is ws
    with pytest.raises(ValueError, match="at least 101 bytes"):
        with q._ws_for(ws, torch.device("cpu"), 101):
            pass
    assert not q._workspaces and not q._captured


def test_capture_number_refuses():
    assert q.lib.qlora_stream_capture_id(None, None) == -1


def test_marks_of_the_exchange(tmp_path):
    """What a single-token launch's workgroups hand each other carries a mark that no other launch has, whatever its
    stream or queue."""
    root = _build.ROOT
    exe = tmp_path / "exchange_check"
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", _build.CSRC, os.path.join(root, "tests", "c_abi", "exchange_check.cpp"),
                    "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout == "shared marks 0\nfinite 0 lost 0 zero 0\n", run.stdout
