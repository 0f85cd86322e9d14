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


@pytest.mark.parametrize("T,K,N,r,order", [(40, 64, 72, 8, "mixed"), (300, 200, 136, 64, "runs"), (700, 136, 264, 136, "mixed"),
                                           (2600, 1032, 520, 24, "runs")])
def test_an_infinity_in_x_or_dy_stays_one_in_da(gg, T, K, N, r, order):
    """dA[a] sums outer(V[t], X[t]): one infinite X[t, k] makes column k of its adapter infinite with
    V's signs, one infinite dY[t, n] makes all of it infinite with the signs of B and X, and a
    zero V times infinity is NaN; never NaN from how V is held.  V here is whole numbers, many of
    them a bf16 and many not (a remainder of zero, of V's sign and of the other)."""
    L = 3
    g = torch.Generator().manual_seed(T)
    ids = torch.arange(T) % L if order == "mixed" else torch.arange(T) * L // T
    X = torch.randint(1, 4, (T, K), generator=g) * (torch.randint(0, 2, (T, K), generator=g) * 2 - 1)
    B = torch.randint(-9, 10, (L, N, r), generator=g)
    dY = torch.randint(-9, 10, (T, N), generator=g)
    V = torch.stack([dY[t] @ B[ids[t]] for t in range(T)])
    assert int(V.abs().max()) > 512 and (V % 2).any()  # past bf16's whole numbers
    of = [int((ids == a).nonzero()[1]) for a in range(L)]
    dY[of[2]] = 0                                      # adapter 2: a row of zero V
    V[of[2]] = 0
    Xf, dYf = X.double(), dY.double()
    Xf[of[0], 5], Xf[of[2], 9] = float("inf"), -float("inf")
    dYf[of[1], 7] = float("inf")                       # adapter 1: an infinite V
    B[1, 7][B[1, 7] == 0] = 1
    put = lambda t: t.to(torch.bfloat16).to(dev())
    st = status_tensor()
    plan = gg.lora_plan(ids.to(torch.int32).to(dev()), L, status=st)
    args = (put(torch.zeros(N, K)), put(torch.zeros(L, r, K)), put(B), None, plan, zeros(T, r))
    dA = gg.lora_backward(put(dYf), put(Xf), *args, want=(False, True, False), status=st)[1].double().cpu()
    both = gg.lora_backward(put(dYf), put(Xf), *args, want=(True, True, False), status=st)[1].double().cpu()
    clean = gg.lora_backward(put(dY), put(X), *args, want=(False, True, False), status=st)[1].double().cpu()
    assert status_of(st) == 0
    want = clean.clone()
    v = V[of[0]].double()
    want[0, :, 5] = torch.where(v == 0, float("nan"), torch.sign(v) * float("inf"))
    want[1] = float("inf") * torch.sign(B[1, 7].double())[:, None] * Xf[of[1]][None]
    want[2, :, 9] = float("nan")
    torch.testing.assert_close(dA, want, rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(both, want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("K,N", [(0, 16), (16, 0), (0, 0)])
def test_empty_widths(gg, K, N):
    """No input or no output columns: what has elements is zero, what has none is empty."""
    T, L, r = 37, 2, 8
    st = status_tensor()
    ones = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device=dev())
    plan = gg.lora_plan(torch.arange(T, dtype=torch.int32, device=dev()) % L, L, status=st)
    args = (ones(T, K), ones(N, K), ones(L, r, K), ones(L, N, r), None, plan)
    dirty = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev())
    Y, U = gg.lora_forward(*args, out=dirty(T, N), out_u=dirty(T, r), status=st)
    dX, dA, dB = gg.lora_backward(ones(T, N), *args, U, out=dirty(T, K), out_da=dirty(L, r, K), out_db=dirty(L, N, r),
                                  status=st)
    assert status_of(st) == 0
    assert bool((U == K).all()) and Y.shape == (T, N) and not Y.any()
    assert dX.shape == (T, K) and dA.shape == (L, r, K) and dB.shape == (L, N, r)
    assert not dX.any() and not dA.any() and not dB.any()
