"""Adapters and rotary positions in a captured graph: the backward's chain of three launches, two of
them started beside the one before, on both projection paths, replayed on other inputs than the
captured ones.  Every replay gives the bits of the plain call (fixed reduction orders)."""
import pytest
import torch

from gpu_util import dev, status_of, status_tensor
from test_gpu_lora import make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


def captured(fn):
    """fn once by itself, then its graph and what the captured call returned."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = fn()
    return graph, out


# split clusters; 2-CTA tiles: few and whole, more than a round with a cut one; ranks of one and of several chunks
@pytest.mark.parametrize("T,K,N,L,r,order", [(48, 256, 264, 5, 16, "mixed"), (513, 2904, 520, 5, 136, "runs"),
                                             (777, 520, 1032, 4, 24, "runs"), (2600, 264, 2056, 4, 24, "mixed"),
                                             (2600, 1032, 1800, 3, 256, "runs")])
def test_forward_and_backward(gg, T, K, N, L, r, order):
    st = status_tensor()
    batches = [on_gpu(make(T, K, N, L, r, order, seed=s)) for s in (1, 2, 3)]
    held = {k: v.clone() for k, v in batches[0].items()}
    plan_buf = torch.empty(gg.lora_plan_size(T, L), dtype=torch.uint8, device=dev())
    ws = torch.full((gg.lora_backward_workspace_size(T, r),), 255, dtype=torch.uint8, device=dev())

    def step(g, workspace=None, out=None):
        plan = gg.lora_plan(g["ids"], L, out=out, status=st)
        args = (g["X"], g["W"], g["A"], g["B"], g["scale"], plan)
        Y, U = gg.lora_forward(*args, status=st)
        return (Y, U) + gg.lora_backward(g["dY"], *args, U, workspace=workspace, status=st)

    graph, outs = captured(lambda: step(held, ws, plan_buf))
    for g in (batches[1], batches[2], batches[0], batches[1]):
        want = step(g)
        for k in held:
            held[k].copy_(g[k])
        graph.replay()
        torch.cuda.synchronize()
        for name, x, y in zip(("Y", "U", "dX", "dA", "dB"), outs, want):
            assert torch.equal(x, y), name
    assert status_of(st) == 0


@pytest.mark.parametrize("T", [1, 2500])
def test_projection_with_positions(gg, T):
    """AdaptedQKV forward and backward, the heads turned in place and back."""
    from unpermute_route_hist_gb300.adapters import AdaptedQKV
    n_q, n_kv, D, hid, L, r = 4, 2, 64, 512, 3, 16
    N = (n_q + 2 * n_kv) * D
    g = torch.Generator(device=dev()).manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev()).mul_(0.2).bfloat16()
    layer = AdaptedQKV(rnd(N, hid), rnd(L, r, hid), rnd(L, N, r), None, n_q, n_kv, D, gg.rope_freqs(D, device=dev()))
    draw = lambda: (rnd(T, hid), rnd(T, N), torch.randint(-1, L, (T,), generator=g, device=dev(), dtype=torch.int32),
                    torch.randint(0, 9999, (T,), generator=g, device=dev(), dtype=torch.int32))

    def step(x, dy, ids, pos):
        plan = gg.lora_plan(ids, L)
        q, k, v, saved = layer.forward(x, plan, pos)
        return (q, k, v) + layer.backward(dy.clone(), saved)

    held = [t.clone() for t in draw()]
    graph, outs = captured(lambda: step(*held))
    for _ in range(3):
        batch = draw()
        want = step(*batch)
        for a, b in zip(held, batch):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for name, x, y in zip(("q", "k", "v", "dX", "dA", "dB"), outs, want):
            assert torch.equal(x, y), name
