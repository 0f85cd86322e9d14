"""The gated forward that keeps 8 bits on more tiles than there are clusters (CTAs, for gathered rows), under both tile
schedules: the same bits, those of the definition on sampled rows, from call to call, replayed from a graph and beside
another launch.  Operands are whole numbers, so every sum is exact in fp32 and codes and scales have to be the
definition's."""
import contextlib

import numpy as np
import pytest
import torch

import act8_ref as ref
import unpermute_route_hist_gb300 as gg
from gpu_util import dev, status_of, status_tensor
from unpermute_route_hist_gb300 import _lib

pytestmark = pytest.mark.gpu

# rows per expert (ragged, one expert without), K, I.  256-row pairs x 256 columns: 37 x 9, 19 x 5 and 18 x 5
# tiles for 76 clusters; 1000 and 3200 columns are 16 and 50 reduction blocks (the automatic schedule turns dynamic at 48)
SIZES = {"short": ((2500, 1, 0, 900, 257, 3000, 128, 1300, 106), 128, 1048),
         "odd": ((700, 2100, 33, 0, 1500), 1000, 520),
         "long": ((1500, 0, 600, 1731, 265), 3200, 520)}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@contextlib.contextmanager
def schedule(mode):
    prev = gg.set_gemm_schedule(mode)
    try:
        yield
    finally:
        gg.set_gemm_schedule(prev)


class Problem:
    def __init__(self, name, topk=1, gathered=False):
        sizes, self.K, self.I = SIZES[name]
        g = torch.Generator().manual_seed(len(sizes) + topk)
        R, E = sum(sizes), len(sizes)
        T = R // topk
        assert T * topk == R
        self.sizes, self.topk, self.gathered = np.array(sizes), topk, gathered
        self.order = torch.randperm(R, generator=g).to(torch.int32)
        self.X = torch.randint(-4, 5, (T if gathered else R, self.K), generator=g).bfloat16()
        self.W = torch.randint(-4, 5, (E, 2 * self.I, self.K), generator=g).bfloat16()
        self.on = [t.to(dev()) for t in (self.X, self.W, torch.tensor(sizes, dtype=torch.int32), self.order)]

    def run(self, fmt, status=None, **kw):
        X, W, m, order = self.on
        return gg.forward_swiglu_act8(X, W, m, order, self.topk, self.gathered, fmt=fmt, status=status, **kw)

    def check(self, kept, A, fmt, n=150):
        """Sampled rows, the experts' first and last ones among them, against the definition."""
        ends = np.cumsum(self.sizes)
        at = np.random.default_rng(1).integers(0, ends[-1], n)
        at = np.unique(np.concatenate([at, ends[self.sizes > 0] - 1, (ends - self.sizes)[self.sizes > 0]]))
        e = np.searchsorted(ends, at, side="right")
        src = self.order.numpy()[at] // self.topk if self.gathered else at
        H = np.empty((len(at), 2 * self.I))
        for x in np.unique(e):
            H[e == x] = self.X[src[e == x]].double().numpy() @ self.W[int(x)].double().numpy().T
        want_c, want_s = ref.pack(H, fmt)
        rows = torch.from_numpy(at).to(dev())
        assert np.array_equal(kept.scales[rows].cpu().numpy()[:, :want_s.shape[1]], want_s)
        assert np.array_equal(ref.TABLE[fmt][kept.codes[rows].cpu().numpy()], ref.TABLE[fmt][want_c])
        gate, up = H[:, 0::2], H[:, 1::2]
        with np.errstate(over="ignore"):
            act = gate / (1 + np.exp(-gate)) * up
        # bf16's half step, the quotient's and exp's fp32 steps, and 0 in place of less than 88 2^-126 < 2^-119
        off = np.abs(A[rows].double().cpu().numpy() - act)
        assert (off <= 2.0 ** -8 * np.abs(act) + 2.0 ** -24 * (16 + 4 * np.abs(gate)) * np.abs(act) +
                2.0 ** -119 * np.abs(up)).all()


def same(a, b):
    nb = -(-a[0].cols // 32)
    return torch.equal(a[0].codes, b[0].codes) and torch.equal(a[0].scales[:, :nb], b[0].scales[:, :nb]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("name,topk,gathered", [("short", 1, False), ("odd", 1, False), ("long", 1, False), ("short", 8, True),
                                                ("long", 4, True)])
def test_schedules_give_the_definition(name, topk, gathered, fmt):
    p = Problem(name, topk, gathered)
    st = status_tensor()
    got = {}
    for mode in (_lib.GG_SCHEDULE_STATIC, _lib.GG_SCHEDULE_DYNAMIC, _lib.GG_SCHEDULE_AUTO):
        with schedule(mode):
            got[mode] = p.run(fmt, st)
            assert same(got[mode], p.run(fmt, st))
    assert status_of(st) == 0
    first = got[_lib.GG_SCHEDULE_STATIC]
    assert all(same(first, v) for v in got.values())
    p.check(*first, fmt)


def test_counters_reset_across_many_launches():
    """More dynamic launches than there are counters, into the same outputs."""
    p = Problem("odd")
    st = status_tensor()
    with schedule(_lib.GG_SCHEDULE_DYNAMIC):
        want = p.run("int8", st)
        out, act = gg.Act8.empty(p.sizes.sum(), 2 * p.I, "int8", dev()), torch.empty_like(want[1])
        bad = 0
        for i in range(1100):
            if i % 50 == 49:
                out.codes.zero_()
                out.scales.zero_()
                act.zero_()
            got = p.run("int8", st, out=out, out_act=act)
            if i % 50 == 49:
                bad += int(not same(got, want))
    assert status_of(st) == 0 and bad == 0


def test_graph_replays_and_two_streams():
    p = Problem("odd")
    R, E = int(p.sizes.sum()), len(p.sizes)
    X, W, m, order = p.on
    st = status_tensor()
    with schedule(_lib.GG_SCHEDULE_DYNAMIC):
        want = p.run("e4m3", st)
        dY = torch.ones(R, 2 * p.I, dtype=torch.bfloat16, device=dev())
        dX = gg.backward_dX(dY, W, m, order, R, 1, status=st)
        torch.cuda.synchronize()
        out, act = gg.Act8.empty(R, 2 * p.I, "e4m3", dev()), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.run("e4m3", st, out=out, out_act=act)
        for _ in range(5):
            out.codes.zero_()
            act.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert same((out, act), want)
        streams = [torch.cuda.Stream() for _ in range(2)]
        dX2 = torch.empty_like(dX)
        for _ in range(20):
            for s in streams:
                s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[0]):
                p.run("e4m3", st, out=out, out_act=act)
            with torch.cuda.stream(streams[1]):
                gg.backward_dX(dY, W, m, order, R, 1, out=dX2, status=st)
            torch.cuda.synchronize()
            assert same((out, act), want) and torch.equal(dX2, dX)
    assert status_of(st) == 0
