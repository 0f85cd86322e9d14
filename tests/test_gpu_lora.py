"""Low-rank adapters beside a shared projection: gg_lora_plan, gg_lora_forward and
gg_lora_backward against the formulas in float64 on the CPU.

Bounds, elementwise, from the arithmetic (derived before any run):
  - a stored bf16 value is rounded once: 2^-9 of itself, 2^-8 allowed;
  - products accumulate in fp32: at most n 2^-24 of the sum of the terms'
    magnitudes M, n <= 1024 here, so 2^-14 M (the tensor core may truncate);
  - U and V enter the second product as bf16 (2^-9 each, 2^-8 allowed of the
    magnitudes they meet); in dA, V carries its remainder, 2^-16."""
import numpy as np
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


def bf(x):
    """float64 -> nearest bf16, as float64."""
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).to(torch.float64).numpy()


def put(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).to(dev())


def get(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(T, K, N, L, r, order, seed=0, bare=0.2):
    g = np.random.default_rng(seed)
    d = dict(X=bf(g.standard_normal((T, K))), W=bf(g.standard_normal((N, K)) * 0.1),
             A=bf(g.standard_normal((L, r, K)) * 0.1), B=bf(g.standard_normal((L, N, r)) * 0.1),
             dY=bf(g.standard_normal((T, N))), scale=g.uniform(0.5, 2.0, L).astype(np.float32))
    if order == "mixed":
        ids = g.integers(0, L, T)
        ids[g.random(T) < bare] = -1
    elif order == "bare":
        ids = np.full(T, -1)
    else:  # runs of one adapter's rows, some without
        ids = np.repeat(g.integers(-1, L, T), g.integers(1, 90, T))[:T]
    d["ids"] = ids.astype(np.int32)
    return d


def forward_ref(d):
    T, N = d["X"].shape[0], d["W"].shape[0]
    L, r, _ = d["A"].shape
    U, Ua = np.zeros((T, r)), np.zeros((T, r))
    Y, M = d["X"] @ d["W"].T, np.abs(d["X"]) @ np.abs(d["W"]).T
    E = np.zeros((T, N))
    for a in range(L):
        i = np.flatnonzero(d["ids"] == a)
        U[i] = d["scale"][a] * (d["X"][i] @ d["A"][a].T)
        Ua[i] = d["scale"][a] * (np.abs(d["X"][i]) @ np.abs(d["A"][a]).T)
        Y[i] += U[i] @ d["B"][a].T
        E[i] += (2.0 ** -8 * np.abs(U[i]) + 2.0 ** -14 * Ua[i]) @ np.abs(d["B"][a]).T
        M[i] += np.abs(U[i]) @ np.abs(d["B"][a]).T
    return Y, U, 2.0 ** -8 * np.abs(Y) + E + 2.0 ** -14 * M, 2.0 ** -8 * np.abs(U) + 2.0 ** -14 * Ua


def backward_ref(d, U):
    T, K = d["X"].shape
    L, r, _ = d["A"].shape
    N = d["W"].shape[0]
    dX, M = d["dY"] @ d["W"], np.abs(d["dY"]) @ np.abs(d["W"])
    E = np.zeros((T, K))
    dA, dB, eA, eB = (np.zeros(s) for s in ((L, r, K), (L, N, r), (L, r, K), (L, N, r)))
    for a in range(L):
        i = np.flatnonzero(d["ids"] == a)
        V = d["scale"][a] * (d["dY"][i] @ d["B"][a])
        Va = d["scale"][a] * (np.abs(d["dY"][i]) @ np.abs(d["B"][a]))
        dX[i] += V @ d["A"][a]
        E[i] += (2.0 ** -8 * np.abs(V) + 2.0 ** -14 * Va) @ np.abs(d["A"][a])
        M[i] += np.abs(V) @ np.abs(d["A"][a])
        dA[a] = V.T @ d["X"][i]
        eA[a] = ((2.0 ** -16 + 2.0 ** -14) * np.abs(V) + 2.0 ** -14 * Va).T @ np.abs(d["X"][i])
        dB[a] = d["dY"][i].T @ U[i]
        eB[a] = 2.0 ** -14 * np.abs(d["dY"][i]).T @ np.abs(U[i])
    return (dX, dA, dB, 2.0 ** -8 * np.abs(dX) + E + 2.0 ** -14 * M, 2.0 ** -8 * np.abs(dA) + eA,
            2.0 ** -8 * np.abs(dB) + eB)


def within(got, ref, bound, what):
    got = get(got)
    assert got.shape == ref.shape, what
    bad = np.argwhere(~(np.abs(got - ref) <= bound + 1e-30))
    assert len(bad) == 0, "%s: %d of %d off, first %s got %r want %r bound %r" % (
        what, len(bad), ref.size, bad[0], got[tuple(bad[0])], ref[tuple(bad[0])], bound[tuple(bad[0])])


def on_gpu(d):
    g = {k: put(d[k]) for k in ("X", "W", "A", "B", "dY")}
    g["scale"] = torch.from_numpy(d["scale"]).to(dev())
    g["ids"] = torch.from_numpy(d["ids"]).to(dev())
    return g


# T, K, N, L, r, order: one row to several units, widths around the 64- and
# 128-column tiles, every rank class, few and many adapters; the last rows have
# enough tiles for 2-CTA pairs in one direction or both
SHAPES = [
    (1, 8, 8, 1, 8, "mixed"), (1, 256, 264, 3, 16, "runs"), (2, 72, 136, 2, 24, "mixed"),
    (7, 64, 16, 5, 8, "mixed"), (33, 520, 128, 40, 16, "mixed"), (48, 1024, 520, 32, 16, "mixed"),
    (127, 128, 256, 2, 32, "runs"), (128, 264, 136, 7, 40, "mixed"), (129, 256, 72, 3, 64, "runs"),
    (255, 136, 264, 300, 8, "mixed"), (256, 192, 128, 1, 128, "runs"), (257, 64, 520, 4, 72, "mixed"),
    (300, 328, 200, 2, 256, "runs"), (520, 256, 256, 9, 136, "mixed"), (640, 512, 384, 6, 48, "runs"),
    (1000, 24, 24, 2, 8, "bare"), (2600, 200, 1032, 5, 16, "runs"), (2600, 1032, 200, 5, 16, "runs"),
    (2570, 1040, 1096, 11, 24, "mixed"), (2816, 1024, 1024, 3, 64, "runs"), (2305, 1032, 1288, 3, 136, "mixed"),
    (2400, 1096, 1032, 70, 8, "mixed"), (2560, 1024, 1024, 2, 256, "runs"),
    # as many adapters as there may be, in one unit's plan and in several
    (256, 64, 72, 2048, 8, "mixed"), (600, 72, 64, 2048, 8, "mixed"),
    # long reductions of few tiles, split over clusters (forward: K, backward: N)
    (300, 2904, 136, 3, 24, "mixed"), (300, 136, 2904, 3, 24, "mixed"), (513, 2904, 520, 5, 136, "runs"),
    (513, 520, 2904, 5, 136, "runs"),
    # more pair tiles than a round of the GPU holds
    (2600, 264, 2056, 4, 24, "runs"), (2600, 136, 1800, 6, 72, "mixed"), (2600, 2056, 264, 4, 24, "runs"),
    (2600, 1800, 136, 6, 72, "mixed"), (2560, 200, 4856, 3, 8, "runs"), (2560, 4856, 200, 3, 8, "runs"),
]


@pytest.mark.parametrize("T,K,N,L,r,order", SHAPES)
def test_forward(gg, T, K, N, L, r, order):
    d = make(T, K, N, L, r, order, seed=T + K)
    g, st = on_gpu(d), status_tensor()
    plan = gg.lora_plan(g["ids"], L, status=st)
    Y, U = gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan, status=st)
    assert status_of(st) == 0
    ref, refu, bound, boundu = forward_ref(d)
    within(U, refu, boundu, "U")
    within(Y, ref, bound, "Y")


@pytest.mark.parametrize("T,K,N,L,r,order", SHAPES)
def test_backward(gg, T, K, N, L, r, order):
    d = make(T, K, N, L, r, order, seed=T + N)
    g, st = on_gpu(d), status_tensor()
    U = bf(forward_ref(d)[1])
    plan = gg.lora_plan(g["ids"], L, status=st)
    got = gg.lora_backward(g["dY"], g["X"], g["W"], g["A"], g["B"], g["scale"], plan, put(U), status=st)
    assert status_of(st) == 0
    ref = backward_ref(d, U)
    for k, name in enumerate(("dX", "dA", "dB")):
        within(got[k], ref[k], ref[3 + k], name)


def test_backward_against_differences(gg):
    """<dY, Y(x + h) - Y(x - h)> / 2h against the gradients, along random directions
    of X, A and B.  Y is linear in each alone, so any h gives the derivative; the
    directions have the operands' size, and the bound is the forward's (2^-8 of Y a
    side) times |dY|."""
    d = make(70, 64, 72, 3, 8, "mixed", seed=5)
    g = on_gpu(d)
    plan = gg.lora_plan(g["ids"], 3)
    U = bf(forward_ref(d)[1])
    grads = [get(t) for t in gg.lora_backward(g["dY"], g["X"], g["W"], g["A"], g["B"], g["scale"], plan, put(U))]
    rng = np.random.default_rng(6)
    for name, grad in zip(("X", "A", "B"), grads):
        h = bf(rng.standard_normal(d[name].shape) * np.abs(d[name]).mean())
        up, dn = dict(d, **{name: bf(d[name] + h)}), dict(d, **{name: bf(d[name] - h)})
        ys = []
        for e in (up, dn):
            ge = on_gpu(e)
            ys.append(get(gg.lora_forward(ge["X"], ge["W"], ge["A"], ge["B"], ge["scale"], plan)[0]))
        num = float((d["dY"] * (ys[0] - ys[1])).sum())
        ana = float((grad * (up[name] - dn[name])).sum())
        err = sum(float((np.abs(d["dY"]) * forward_ref(e)[2]).sum()) for e in (up, dn))
        err += 2.0 ** -7 * float((np.abs(grad) * np.abs(up[name] - dn[name])).sum())
        assert abs(num - ana) <= err, (name, num, ana, err)


@pytest.mark.parametrize("T,N", [(200, 264), (2570, 1096)])
def test_rows_take_their_own_adapter_alone(gg, T, N):
    """Infinities and NaN in one adapter, or in rows, reach no other row and no other
    adapter's gradient: everything else is bit for bit as without them."""
    d = make(T, 256, N, 4, 16, "mixed", seed=3)
    U = bf(forward_ref(d)[1])

    def call(e, u):
        g = on_gpu(e)
        plan = gg.lora_plan(g["ids"], 4)
        y, u2 = gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan)
        return [get(t) for t in (y, u2) + gg.lora_backward(g["dY"], g["X"], g["W"], g["A"], g["B"], g["scale"], plan,
                                                            put(u))]

    clean = call(d, U)
    e, u = {k: v.copy() for k, v in d.items()}, U.copy()
    e["A"][1, 3, 5], e["B"][1, 7, 2], e["A"][1, 4, 6] = np.inf, -np.inf, np.nan
    bad = np.flatnonzero(d["ids"] == 1)
    e["X"][bad[0], 9], e["dY"][bad[1], 11], u[bad[2], 1] = np.inf, np.nan, np.inf
    got = call(e, u)
    other = d["ids"] != 1
    for k in (0, 1, 2):  # Y, U, dX by rows
        np.testing.assert_array_equal(got[k][other], clean[k][other])
    for k in (3, 4):     # dA, dB by adapter
        for a in (0, 2, 3):
            np.testing.assert_array_equal(got[k][a], clean[k][a])
    assert np.isnan(got[0][bad]).any() and not np.isfinite(got[3][1]).all()


def test_repeats_bit_for_bit_and_on_another_stream(gg):
    d = make(700, 520, 392, 6, 24, "mixed", seed=8)
    g = on_gpu(d)
    U = put(bf(forward_ref(d)[1]))

    def call():
        plan = gg.lora_plan(g["ids"], 6)
        return gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan) + gg.lora_backward(
            g["dY"], g["X"], g["W"], g["A"], g["B"], g["scale"], plan, U)

    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = call()
    s.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_graph_capture(gg):
    d = make(48, 256, 264, 5, 16, "mixed", seed=9)
    g = on_gpu(d)
    plan = gg.lora_plan(g["ids"], 5)
    want = gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan)[0].clone()
    Y, U = torch.zeros_like(want), torch.zeros(48, 16, dtype=torch.bfloat16, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
        gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan, out=Y, out_u=U)
        graph.capture_end()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_offsets_past_32_bits(gg):
    """270000 tokens of width 8192: elements past 2^31 of X, Y, dY and dX.  The last 70
    tokens have an adapter of their own, so its gradients are theirs alone."""
    T, W, r, last = 270000, 8192, 8, 70
    g = torch.Generator(device=dev()).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev(), dtype=torch.bfloat16)
    ids = torch.zeros(T, dtype=torch.int32, device=dev())
    ids[-last:] = 1
    plan, scale = gg.lora_plan(ids, 2), torch.tensor([1.0, 0.5], device=dev())
    cpu = lambda t: t.double().cpu().numpy()
    big = rnd(T, W)
    tail = cpu(big[-last:])
    # wide input: X past 2^31, then dX and dA
    d = dict(X=tail, W=cpu(rnd(16, W)), A=cpu(rnd(2, r, W) * 0.01), B=cpu(rnd(2, 16, r)), dY=cpu(rnd(T, 16)[-last:]))
    d["ids"], d["scale"] = np.ones(last, np.int32), np.array([1.0, 0.5], np.float32)
    dY = torch.zeros(T, 16, dtype=torch.bfloat16, device=dev())
    dY[-last:] = put(d["dY"])
    ops = [put(d[k]) for k in ("W", "A", "B")]
    Y, U = gg.lora_forward(big, *ops, scale, plan)
    ref = forward_ref(d)
    within(U[-last:], ref[1], ref[3] * 8, "U")      # sums of 8192 terms: 8 times the bound's 1024
    within(Y[-last:], ref[0], ref[2] * 8, "Y")
    dX, dA, _ = gg.lora_backward(dY, big, *ops, scale, plan, U, want=(True, True, False))
    ref = backward_ref(d, get(U[-last:]))
    within(dX[-last:], ref[0], ref[3], "dX")
    within(dA[1:], ref[1][1:], ref[4][1:] , "dA")
    assert not get(dX[:1000]).any()
    del dX
    # wide output: Y and dY past 2^31, then dB
    d = dict(X=cpu(rnd(T, 16)[-last:]), W=cpu(rnd(W, 16)), A=cpu(rnd(2, r, 16)), B=cpu(rnd(2, W, r) * 0.1), dY=tail,
             ids=d["ids"], scale=d["scale"])
    X = torch.zeros(T, 16, dtype=torch.bfloat16, device=dev())
    X[-last:] = put(d["X"])
    ops = [put(d[k]) for k in ("W", "A", "B")]
    Y, U = gg.lora_forward(X, *ops, scale, plan)
    ref = forward_ref(d)
    within(Y[-last:], ref[0], ref[2], "Y, wide")
    dB = gg.lora_backward(big, X, *ops, scale, plan, U, want=(False, False, True))[2]
    ref = backward_ref(d, get(U[-last:]))
    within(dB[1:], ref[2][1:], ref[5][1:], "dB")


def test_scale_none_and_wanted_gradients(gg):
    d = make(130, 128, 136, 3, 16, "mixed", seed=10)
    d["scale"][:] = 1.0
    g = on_gpu(d)
    plan = gg.lora_plan(g["ids"], 3)
    U = put(bf(forward_ref(d)[1]))
    args = (g["dY"], g["X"], g["W"], g["A"], g["B"])
    Y, _ = gg.lora_forward(*args[1:], None, plan)
    within(Y, forward_ref(d)[0], forward_ref(d)[2], "Y")
    full = gg.lora_backward(*args, None, plan, U)
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)):
        some = gg.lora_backward(*args, None, plan, U, want=want)
        for k in range(3):
            assert (some[k] is None) if not want[k] else torch.equal(some[k], full[k])


def test_no_tokens_and_bad_ids(gg):
    d = make(4, 64, 72, 3, 8, "mixed", seed=11)
    g, st = on_gpu(d), status_tensor()
    empty = gg.lora_plan(g["ids"][:0], 3)
    Y, U = gg.lora_forward(g["X"][:0], g["W"], g["A"], g["B"], g["scale"], empty)
    assert Y.shape == (0, 72) and U.shape == (0, 8)
    dX, dA, dB = gg.lora_backward(g["dY"][:0], g["X"][:0], g["W"], g["A"], g["B"], g["scale"], empty, U)
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()
    from unpermute_route_hist_gb300 import _lib
    ids = torch.tensor([0, 3, -2, 1], dtype=torch.int32, device=dev())
    plan = gg.lora_plan(ids, 3, status=st)
    Y, U = gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan, status=st)
    assert gg.read_status(st) == (_lib.GG_ERR_DEVICE_CHECK, _lib.GG_DEV_BAD_ADAPTER_ID)
    d["ids"] = np.array([0, -1, -1, 1], np.int32)  # ids out of range count as no adapter
    within(Y, forward_ref(d)[0], forward_ref(d)[2], "Y")


def test_refusals(gg):
    d = make(16, 64, 72, 3, 8, "mixed", seed=12)
    g = on_gpu(d)
    plan = gg.lora_plan(g["ids"], 3)
    ok = (g["X"], g["W"], g["A"], g["B"], g["scale"], plan)
    with pytest.raises(TypeError):
        gg.lora_forward(g["X"].float(), *ok[1:])
    with pytest.raises(ValueError):
        gg.lora_forward(g["X"][:8], *ok[1:])                       # another number of tokens than the plan's
    with pytest.raises(ValueError):
        gg.lora_forward(g["X"], g["W"], g["A"][:2].contiguous(), g["B"], None, plan)
    with pytest.raises(ValueError):
        gg.lora_forward(g["X"], g["W"], g["A"], g["B"][:, :64].contiguous(), g["scale"], plan)
    with pytest.raises(ValueError):
        gg.lora_forward(g["X"].t().contiguous().t(), *ok[1:])      # rows not contiguous
    with pytest.raises(gg.GGError):
        gg.lora_forward(*ok[:2], g["A"][:, :4].contiguous(), g["B"][..., :4].contiguous(), g["scale"], plan)
    with pytest.raises(gg.GGError):
        gg.lora_plan(g["ids"], 3, out=torch.empty(64, dtype=torch.uint8, device=dev()))
    with pytest.raises(gg.GGError):
        gg.lora_backward(g["dY"], *ok, torch.zeros(16, 8, dtype=torch.bfloat16, device=dev()),
                         workspace=torch.empty(16, dtype=torch.uint8, device=dev()))


@pytest.mark.parametrize("T,r", [(1, 8), (31, 24), (300, 256), (777, 16), (2049, 136), (5000, 64)])
@pytest.mark.parametrize("order", ["all", "first half", "every third", "all but the last"])
def test_rows_without_an_adapter_in_dirty_memory(gg, T, r, order):
    """U of a row without an adapter is zero whatever stood there, its Y and dX are the shared
    product's alone, and a backward in a dirty workspace gives finite sums."""
    K, N, L = 136, 72, 3
    d = make(T, K, N, L, r, "runs", seed=T + r)
    ids, at = np.sort(d["ids"] % L), np.arange(T)
    bare = {"all": at >= 0, "first half": at < T // 2, "every third": at % 3 == 0, "all but the last": at < T - 1}[order]
    d["ids"] = np.where(bare, -1, ids).astype(np.int32)
    g, st = on_gpu(d), status_tensor()
    plan = gg.lora_plan(g["ids"], L, status=st)
    dirty = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev())
    Y, U = gg.lora_forward(g["X"], g["W"], g["A"], g["B"], g["scale"], plan, out=dirty(T, N), out_u=dirty(T, r), status=st)
    ref, refu, bound, boundu = forward_ref(d)
    within(U, refu, boundu, "U")
    within(Y, ref, bound, "Y")
    assert not U[torch.from_numpy(bare).to(dev())].any()
    ws = torch.full((gg.lora_backward_workspace_size(T, r),), 255, dtype=torch.uint8, device=dev())
    got = gg.lora_backward(g["dY"], g["X"], g["W"], g["A"], g["B"], g["scale"], plan, U, out=dirty(T, K),
                           out_da=dirty(L, r, K), out_db=dirty(L, N, r), workspace=ws, status=st)
    assert status_of(st) == 0
    ref = backward_ref(d, get(U))
    for i, what in enumerate(("dX", "dA", "dB")):
        within(got[i], ref[i], ref[3 + i], what)
