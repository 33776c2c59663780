"""The binding's kept scratch where calls could meet in it: current streams, threads, graph capture."""
import threading

import numpy as np
import pytest
import torch

import synthetic
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

# small enough for the kept scratch, large enough to be under way when the next call comes
T, H, E = 2000, 256, 8


class _Call:
    """One operator call of each kind that takes scratch, and what it gives with memory of its own."""

    def __init__(self, m, seed):
        self.m = m
        rng = np.random.default_rng(seed)
        self.x, self.w = synthetic.random_bf16((T, H), seed).cuda(), synthetic.random_bf16((E, H), seed + 1, std=0.02).cuda()
        self.z = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
        self.ids = torch.from_numpy(rng.integers(0, E, (T, 2)).astype(np.int32)).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sizes = m.mxg_router_linear_bwd_workspace_bytes(T, H, E), m.mxg_balance_loss_workspace_bytes(T, E)
        assert max(sizes) <= m._lib._ScratchCache.BYTES and min(sizes) > 0
        self.expected = self.run([torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes])
        torch.cuda.synchronize()

    def run(self, ws=(None, None)):
        out = self.m.mxg_router_linear_bwd(self.x, self.w, self.z, None, self.status, workspace=ws[0])
        return (*out, *self.m.mxg_balance_loss_fwd(self.z, self.ids, 0.1, self.status, workspace=ws[1]))

    def check(self, outs):
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, self.expected))
        assert int(self.status.item()) == 0


def test_current_streams_in_turn():
    m = require_gpu()
    calls = [_Call(m, 10 * i) for i in range(3)]
    streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], [], []]
    for _ in range(40):
        for s, c, o in zip(streams, calls, outs):
            with torch.cuda.stream(s):
                o.append(c.run())
    torch.cuda.synchronize()
    for c, o in zip(calls, outs):
        c.check(o)


@pytest.mark.parametrize("own_stream", [True, False])
def test_threads(own_stream):
    m = require_gpu()
    calls = [_Call(m, 10 * i + 5) for i in range(3)]
    outs, errors, start = [[], [], []], [], threading.Barrier(3)

    def work(i):
        try:
            start.wait()
            with torch.cuda.stream(torch.cuda.Stream() if own_stream else torch.cuda.current_stream()):
                for _ in range(40):
                    outs[i].append(calls[i].run())
                torch.cuda.current_stream().synchronize()
        except BaseException as e:                            # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for c, o in zip(calls, outs):
        c.check(o)


def test_capture_has_memory_of_its_own(monkeypatch):
    """What a graph holds is not the kept scratch, so calls outside may come between its replays, on any stream."""
    m = require_gpu()
    a, b = _Call(m, 3), _Call(m, 4)
    b.run()                                                    # the scratch is there
    graph = torch.cuda.CUDAGraph()
    with monkeypatch.context() as p:
        p.setattr(m._lib._ScratchCache, "get", lambda *_: pytest.fail("kept scratch in a graph"))
        with torch.cuda.graph(graph):
            captured = a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        for t in captured:
            t.zero_()
        graph.replay()
        outs.append(b.run())
        with torch.cuda.stream(side):
            outs.append(b.run())
    torch.cuda.synchronize()
    a.check([captured])
    b.check(outs)


def test_given_stream_has_memory_of_its_own(monkeypatch):
    m = require_gpu()
    c = _Call(m, 6)
    s = torch.cuda.Stream()
    monkeypatch.setattr(m._lib._ScratchCache, "get", lambda *_: pytest.fail("kept scratch on a given stream"))
    dx, dw = m.mxg_router_linear_bwd(c.x, c.w, c.z, None, c.status, stream=s)
    s.synchronize()
    assert torch.equal(dx, c.expected[0]) and torch.equal(dw, c.expected[1])
