"""Norm gradients with dW of one config on several streams: the partial sums of
one call are not another's.  Every dX and dW equals, bit for bit, that of the
same call made alone."""
import ctypes
import re

import pytest
import torch

import tile_scheduling_persistent_amd as pg
from tests.gpu_util import config, note, sync
from tests.test_gpu_rms_grad_rows import normal

pytestmark = pytest.mark.gpu

ROUNDS = 12


class Call:
    """One gradient with inputs of its own, and its result when made alone."""

    def __init__(self, rows, cols, seed):
        g = torch.Generator(device="cuda:0")
        g.manual_seed(seed)
        self.H, self.dY = normal(g, rows, cols).bfloat16(), normal(g, rows, cols).bfloat16()
        self.W = (1 + 0.3 * normal(g, cols)).bfloat16()
        self.T = torch.rsqrt(self.H.float().square().mean(1) + 1e-6)
        self.shape = rows, cols
        self.want = self.outputs()
        self.run(self.want)
        sync()

    def outputs(self):
        return torch.full_like(self.H, float("nan")), torch.full((self.shape[1],), float("nan"), device="cuda:0")

    def run(self, out, cfg=None, stream=None):
        pg.prms_grad_run(cfg or config(), self.dY, self.H, self.W, self.T, *out, *self.shape, stream=stream)

    def same(self, out):
        return all(torch.equal(a, b) for a, b in zip(out, self.want))


SIZES = [((4096, 4096), (700, 8192)), ((8192, 1024), (8192, 1024)), ((300, 20000), (2000, 2048))]


@pytest.mark.parametrize("one,two", SIZES)
def test_calls_on_two_streams(one, two):
    calls = [Call(*one, 1), Call(*two, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[c.outputs() for _ in range(ROUNDS)] for c in calls]
    sync()
    note(f"gradients on two streams {one} {two}")
    for i in range(ROUNDS):
        for c, s, o in zip(calls, streams, outs):
            c.run(o[i], stream=s)
    calls[0].run(calls[0].outputs())  # and on the null stream
    sync("two streams")
    for c, o in zip(calls, outs):
        assert all(c.same(x) for x in o)


@pytest.mark.parametrize("one,two", SIZES)
def test_eager_calls_beside_replays(one, two):
    captured, eager = Call(*one, 3), Call(*two, 4)
    outs = [captured.outputs() for _ in range(4)]
    st, other, g = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    captured.run(outs[0], stream=st)  # warm-up on the stream of the capture
    sync("warm-up", stream=st)
    with torch.cuda.graph(g, stream=st):
        for o in outs:
            captured.run(o)
    for turn in range(3):
        results = [eager.outputs() for _ in range(ROUNDS)]
        for o in outs:
            for t in o:
                t.zero_()
        sync("cleared")
        note(f"replay {captured.shape} beside eager {eager.shape}")
        with torch.cuda.stream(st):
            g.replay()
        for o in results:
            eager.run(o, stream=other)
        sync("replay beside eager calls")
        assert all(captured.same(o) for o in outs) and all(eager.same(o) for o in results), turn


def runtime():
    for line in open("/proc/self/maps"):
        m = re.search(r"(/\S*libamdhip64\.so\S*)", line)
        if m:
            return ctypes.CDLL(m.group(1))
    raise AssertionError("no HIP runtime loaded")


def test_streams_that_were_destroyed():
    """The stream of the call before is gone: when the second stream comes, and
    again when the calls already wait for each other."""
    cfg, call, hip = pg.Config(0), Call(500, 1024, 5), runtime()
    outs = [call.outputs() for _ in range(4)]
    sync()
    note("gradients on streams that end, and on torch's")
    for first, second in (outs[:2], outs[2:]):
        s = ctypes.c_void_p()
        assert hip.hipStreamCreate(ctypes.byref(s)) == 0
        call.run(first, cfg, s.value)
        assert hip.hipStreamSynchronize(s) == 0 and hip.hipStreamDestroy(s) == 0
        call.run(second, cfg)
    sync()
    assert all(call.same(o) for o in outs)
    cfg.close()
