"""The adapter gradients take the V of their own call: gg_lora_backward starts their kernel
beside dX's last tiles, and what the low-rank product wrote (V, its remainder, the cleared
counters) has to be seen there.

A call that missed it would sum what an earlier call left in the same workspace, so calls on
two batches alternate in one workspace without a host wait between them, and every result is
compared bit for bit with the batch's own in a workspace of its own (the reduction orders are
fixed: no tolerance)."""
import pytest
import torch

from gpu_util import dev, status_of, status_tensor
from test_gpu_lora import make, on_gpu

pytestmark = pytest.mark.gpu

# few rows and long reductions (split clusters), many rows (2-CTA tiles, whole and cut), a call
# whose dX outlasts the low-rank product by far, one whose dX is shorter, every rank class
SHAPES = [(1, 64, 72, 2, 8, "mixed"), (200, 2048, 520, 3, 16, "runs"), (300, 136, 2904, 3, 24, "mixed"),
          (777, 520, 1032, 5, 64, "mixed"), (2570, 1040, 1096, 11, 24, "mixed"), (2560, 4096, 200, 3, 72, "runs"),
          (2305, 264, 4096, 3, 256, "runs")]


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


@pytest.mark.parametrize("want", [(True, True, True), (True, True, False), (True, False, True), (False, True, True)])
@pytest.mark.parametrize("T,K,N,L,r,order", SHAPES)
def test_gradients_take_their_own_calls_v(gg, T, K, N, L, r, order, want):
    st = status_tensor()
    batches = []
    for seed in (1, 2):
        g = on_gpu(make(T, K, N, L, r, order, seed=seed))
        plan = gg.lora_plan(g["ids"], L, status=st)
        U = gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan, status=st)[1]
        batches.append((g["dY"], g["X"], g["W"], g["A"], g["B"], g["scale"], plan, U))
    size = gg.lora_backward_workspace_size(T, r)
    own = []
    for b in batches:
        ws = torch.full((size,), 255, dtype=torch.uint8, device=dev())
        own.append(gg.lora_backward(*b, want=want, workspace=ws, status=st))
        torch.cuda.synchronize()
    ws = torch.full((size,), 255, dtype=torch.uint8, device=dev())
    got = [gg.lora_backward(*batches[i & 1], want=want, workspace=ws, status=st) for i in range(12)]
    assert status_of(st) == 0
    for i, out in enumerate(got):
        for name, x, y in zip(("dX", "dA", "dB"), out, own[i & 1]):
            assert (x is None and y is None) or torch.equal(x, y), (i, name)


def test_two_streams_side_by_side(gg):
    """Calls on two streams, each with a plan and a workspace of its own, give the bits they give
    alone."""
    st = status_tensor()
    jobs = []
    for seed, (T, K, N, L, r, order) in ((1, (777, 520, 1032, 5, 64, "mixed")), (2, (200, 2048, 520, 3, 16, "runs"))):
        g = on_gpu(make(T, K, N, L, r, order, seed=seed))
        size = gg.lora_backward_workspace_size(T, r)

        def call(g=g, L=L, ws=torch.full((size,), 255, dtype=torch.uint8, device=dev())):
            plan = gg.lora_plan(g["ids"], L, status=st)
            args = (g["X"], g["W"], g["A"], g["B"], g["scale"], plan)
            Y, U = gg.lora_forward(*args, status=st)
            return (Y, U) + gg.lora_backward(g["dY"], *args, U, workspace=ws, status=st)

        jobs.append((call, call(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    for _ in range(8):
        for i, (call, _, stream) in enumerate(jobs):
            with torch.cuda.stream(stream):
                got[i].append(call())
    torch.cuda.synchronize()
    assert status_of(st) == 0
    for (_, want, _), outs in zip(jobs, got):
        for out in outs:
            for name, x, y in zip(("Y", "U", "dX", "dA", "dB"), out, want):
                assert torch.equal(x, y), name
