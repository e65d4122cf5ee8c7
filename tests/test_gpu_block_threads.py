"""The join called from several host threads at once, and at several widths in one
captured graph: one kernel serves all widths, so what a call asks of the driver for
its own width must not take anything from another's."""
import threading

import pytest
import torch

import fsdp_sharded_mixed_shard_gb300 as Z
from test_gpu_block import NAMES, at, join_case, params_of, weights_of
from train_util import ZT

pytestmark = pytest.mark.gpu

ROWS = 2000
# one kernel each way for both of a pair's widths, with 80 and 128 KB (RMS) or 96
# and 192 KB (layer norm) of shared memory forward, 144 and 192 KB backward
PAIRS = [(False, 2048, 8192), (True, 2048, 8192), (False, 2047, 8191)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


class Call:
    """A join and its gradient with all parameters, at one width."""

    def __init__(self, cols, layer, seed):
        names = NAMES if layer else ("w_post", "gate", "w_pre")
        self.c = join_case("bf16", ROWS, cols, cols, 0, layer, names, 0.0, 1.0, 0.5, seed=seed)
        new = lambda *s: torch.empty(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.h_out, self.z, self.dh, self.dy = (new(ROWS, cols) for _ in range(4))
        self.stats = torch.empty(ROWS, 4, device="cuda")
        self.g = {k: None if v is None else torch.empty_like(v) for k, v in self.c["w"].items()}
        self.work = torch.empty(Z.zero_block_join_workspace_bytes(ROWS, cols), dtype=torch.uint8,
                                device="cuda")
        self.p, self.w, self.dw = params_of(self.c), weights_of(self.c["w"]), weights_of(self.g)

    def run(self, st):
        c, cols = self.c, self.c["cols"]
        Z.zero_block_join(self.p, self.w, at(c["h"]), at(c["y"]), ROWS, cols, cols, ZT["bf16"],
                          at(self.h_out), at(self.z), at(self.stats), st)
        Z.zero_block_join_grad(self.p, self.w, at(self.h_out), at(c["y"]), at(self.stats),
                               at(c["dz"]), at(c["dh_out"]), ROWS, cols, cols, ZT["bf16"],
                               at(self.dh), at(self.dy), self.dw, at(self.work), st)

    def outputs(self):
        out = [self.h_out, self.z, self.stats, self.dh, self.dy]
        return out + [t for t in self.g.values() if t is not None]

    def clear(self):
        for t in self.outputs():
            t.zero_()


def alone(calls):
    st = torch.cuda.current_stream().cuda_stream
    for c in calls:
        c.run(st)
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.outputs()] for c in calls]
    for c in calls:
        c.clear()
    torch.cuda.synchronize()
    return want


def same(calls, want):
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        for a, b in zip(c.outputs(), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("layer,narrow,wide", PAIRS)
def test_widths_from_two_threads(layer, narrow, wide):
    calls = [Call(narrow, layer, 1), Call(wide, layer, 2)]
    want = alone(calls)
    streams = [torch.cuda.Stream() for _ in calls]
    start, errors = threading.Barrier(2), []

    def repeat(call, st):
        start.wait()
        for _ in range(1500):
            try:
                call.run(st)
            except Z.ZeroError as e:
                errors.append((call.c["cols"], str(e)))
                return

    threads = [threading.Thread(target=repeat, args=(c, s.cuda_stream))
               for c, s in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == []
    same(calls, want)


@pytest.mark.parametrize("layer,narrow,wide", PAIRS)
def test_widths_in_one_graph(layer, narrow, wide):
    """The narrow calls are captured after the wide ones, before the graph is made."""
    calls = [Call(wide, layer, 3), Call(narrow, layer, 4)]
    want = alone(calls)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        for c in calls:
            c.run(torch.cuda.current_stream().cuda_stream)
    for _ in range(2):
        for c in calls:
            c.clear()
        torch.cuda.synchronize()
        graph.replay()
        same(calls, want)
