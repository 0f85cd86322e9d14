"""Where the adapters' backward rounds: small whole numbers, every product and sum of which is
exact in fp32, so each output has one right value."""
import pytest
import torch

from gpu_util import dev, status_of, status_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gg():
    import __graft_entry__ as g
    g.build()
    import unpermute_route_hist_gb300 as gg
    return gg


def zeros(*s):
    return torch.zeros(*s, dtype=torch.bfloat16, device=dev())


@pytest.mark.parametrize("T,K,N", [(16, 64, 8), (2560, 1024, 1024)])  # split clusters, 2-CTA tiles
def test_dx_takes_v_in_bf16_and_da_with_its_remainder(gg, T, K, N):
    """V = (257, -256) in the first row: bf16 holds 256 and -256, so dX through A = (1, 1) is 0, not
    1.  The second row's V = (-256, 0), so dA's first rank sums 257 - 256 = 1 with the remainder,
    0 without."""
    X, W, A, B, dY = zeros(T, K), zeros(N, K), zeros(1, 8, K), zeros(1, N, 8), zeros(T, N)
    B[0, 0, 0], B[0, 1, 0], B[0, 2, 1], B[0, 3, 0] = 256, 1, -256, -256
    dY[0, :3], dY[1, 3] = 1, 1
    A[0, :2, 5], X[:2, 3] = 1, 1
    st = status_tensor()
    plan = gg.lora_plan(torch.zeros(T, dtype=torch.int32, device=dev()), 1, status=st)
    dX, dA, _ = gg.lora_backward(dY, X, W, A, B, None, plan, zeros(T, 8), status=st)
    assert status_of(st) == 0
    assert float(dX[0, 5]) == 0.0 and float(dX[1, 5]) == -256.0
    assert float(dA[0, 0, 3]) == 1.0 and float(dA[0, 1, 3]) == -256.0
    dX[1, 5] = 0
    dA[0, :2, 3] = 0
    assert not dX.any() and not dA.any()
