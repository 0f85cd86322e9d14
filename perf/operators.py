"""The measured cases of the adapter and rotary operators.

Three operators, each with its plain form (elementary torch operations in
32 bits, rounded once at the end), the framework's call, and the definition
in 64 bits:

  adapt       Y = X W^T + U B[a]^T,  U = scale[a] X A[a]^T: one shared projection
              with the low-rank adapter a = ids[t] of each token beside it
              (ids -1: no adapter)
  adapt_bwd   its gradients dX, dA, dB from dY, X and the kept U (W is frozen)
  rotary      rotary positions on the q and k heads of a packed projection,
              forward, or backward (the gradient)

Shapes are the repository's own hidden sizes (2048, 4096; 1536 and 768 of the
fine-grained layer) with generic head layouts.  own selects the framework's
kernels; the tools set it.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --

def _adapt(name, T, K, N, L, r, order, bare=0.0):
    return {"name": name, "op": "adapt", "T": T, "K": K, "N": N, "L": L, "r": r, "order": order, "bare": bare}


def _adapt_bwd(name, T, K, N, L, r, order, bare=0.0):
    return {"name": name, "op": "adapt_bwd", "T": T, "K": K, "N": N, "L": L, "r": r, "order": order, "bare": bare}


def _rotary(name, T, Hq, Hk, D, rot, layout, dtype, scaling, maxpos, sections, backward, inplace):
    return {"name": name, "op": "rotary", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot, "layout": layout,
            "dtype": dtype, "scaling": scaling, "maxpos": maxpos, "sections": sections, "backward": backward,
            "inplace": inplace}


def listed():
    return [
        # one request decoding one token: the q|k|v projection of hidden size 4096
        _adapt("adapt_decode_1", 1, 4096, 6144, 8, 16, "runs"),
        # a serving batch of 48 requests decoding, 32 adapters in use, a few requests on the bare model
        _adapt("adapt_decode_48", 48, 4096, 6144, 32, 16, "mixed", 0.1),
        # a ragged prefill of five short prompts, odd length, hidden size 2048
        _adapt("adapt_prefill_777", 777, 2048, 2560, 5, 24, "runs", 0.15),
        # a packed training batch, eight adapters trained side by side
        _adapt("adapt_train_8192", 8192, 4096, 6144, 8, 32, "runs"),
        # a small odd training step of rank 8
        _adapt_bwd("adapt_bwd_201", 201, 2048, 1536, 3, 8, "runs", 0.1),
        # tokens of sixteen adapters in no order (rows already shuffled), rank 64
        _adapt_bwd("adapt_bwd_mixed_2048", 2048, 2048, 4096, 16, 64, "mixed", 0.05),
        # the training step of adapt_train_8192
        _adapt_bwd("adapt_bwd_train_8192", 8192, 4096, 6144, 8, 32, "runs"),
        # decoding: q and k heads of the packed projection rotated in place, 48 requests
        _rotary("rotary_decode_48", 48, 32, 8, 128, 128, "half", "bfloat16", "none", 32768, 0, False, True),
        # a training batch, in place on the packed projection
        _rotary("rotary_train_16384", 16384, 32, 8, 128, 128, "half", "bfloat16", "ntk", 16384, 0, False, True),
        # part of the head, interleaved pairs, positions scaled for a long context, 32-bit tensors, odd length
        _rotary("rotary_part_long_4097", 4097, 16, 1, 192, 64, "interleaved", "float32", "yarn", 131072, 0, False, False),
        # the backward of image and text positions (three axes), out of place
        _rotary("rotary_bwd_sections_8192", 8192, 32, 8, 128, 128, "half", "bfloat16", "none", 4096, 3, True, False),
        # an odd head width in 16-bit floats
        _rotary("rotary_odd_999", 999, 7, 3, 80, 20, "interleaved", "float16", "linear", 65536, 0, False, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _not_3072(n, step=8):
    return n + step if n == 3072 else n


def draw(rng):
    kind = rng.choice(["adapt", "adapt", "adapt_bwd", "adapt_bwd", "rotary"])
    if kind != "rotary":
        r = 8 * _log_int(rng, 1, 16)
        L = _log_int(rng, 1, 64)
        T = _not_3072(_log_int(rng, 1, 8192), 1)
        K = _not_3072(8 * rng.randint(32, 512))
        N = _not_3072(8 * rng.randint(32, 768))
        most = 8192 * 4096 * 6144
        order = rng.choice(["runs", "mixed"])
        while T * (K * N + (L if order == "mixed" else 1) * r * (K + N)) > most:
            T = _not_3072(T // 2 + 1, 1)
        return {"op": kind, "T": T, "K": K, "N": N, "L": L, "r": r, "order": order,
                "bare": rng.choice([0.0, 0.1, 0.5])}
    D = 4 * rng.randint(8, 64)
    rot = 2 * rng.randint(2, D // 2)
    Hk = rng.randint(1, 8)
    Hq = Hk * rng.randint(1, 6)
    T = _log_int(rng, 1, 16384)
    dtype = rng.choice(["bfloat16", "float16", "float32"])
    size = 4 if dtype == "float32" else 2
    while T * (Hq + Hk) * D * size > 16384 * 40 * 128 * 2:
        T //= 2
    T = _not_3072(T, 1)
    return {"op": "rotary", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
            "layout": rng.choice(["half", "interleaved"]), "dtype": dtype,
            "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "maxpos": _log_int(rng, 64, 131072),
            "sections": rng.choice([0, 0, 3]) if rot >= 8 else 0, "backward": rng.random() < 0.4,
            "inplace": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs --

def _adapter_ids(case, seed):
    """Token -> adapter: runs of one request's tokens, or every token on its own; a share `bare` without one."""
    g = np.random.default_rng([int(seed), 11])
    T, L = case["T"], case["L"]
    if case["order"] == "mixed":
        ids = g.integers(0, L, size=T)
        ids[g.random(T) < case["bare"]] = -1
        return ids.astype(np.int32)
    nruns = min(T, 2 * L)
    cuts = np.sort(g.choice(np.arange(1, T), size=nruns - 1, replace=False)) if nruns > 1 else np.zeros(0, np.int64)
    which = np.concatenate([g.permutation(L) for _ in range(2)])[:nruns]
    which = np.where(g.random(nruns) < case["bare"], -1, which)
    return np.repeat(which, np.diff(np.concatenate([[0], cuts, [T]]))).astype(np.int32)


def _normal(gen, shape, std, dtype=torch.bfloat16):
    x = torch.empty(shape, dtype=torch.float32, device=DEV)
    x.normal_(0.0, std, generator=gen)
    return x.to(dtype)


def _adapter_inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    T, K, N, L, r = (case[k] for k in ("T", "K", "N", "L", "r"))
    s = {"X": _normal(gen, (T, K), 1.0), "W": _normal(gen, (N, K), 0.02),
         "A": _normal(gen, (L, r, K), K ** -0.5), "B": _normal(gen, (L, N, r), 0.02)}
    g = np.random.default_rng([int(seed), 12])
    s["scale"] = torch.from_numpy(g.uniform(0.5, 2.0, size=L).astype(np.float32)).to(DEV)
    s["ids"] = torch.from_numpy(_adapter_ids(case, seed)).to(DEV)
    if case["op"] == "adapt_bwd":
        s["dY"] = _normal(gen, (T, N), 0.02)
        # U as the forward keeps it: [T, r], zero where a token has no adapter
        s["U"] = _normal(gen, (T, r), 1.0) * (s["ids"] >= 0).unsqueeze(1).to(torch.bfloat16)
    return s


def _sections(case):
    """Pairs of each position axis: time, height, width (a quarter and the rest split in two)."""
    half = case["rot"] // 2
    if not case["sections"]:
        return None
    a = max(1, half // 4)
    b = max(1, (half - a) // 2)
    return (a, b, half - a - b)


_SCALINGS = {"none": {}, "linear": {"scaling": "linear", "factor": 4.0}, "ntk": {"scaling": "ntk", "factor": 2.0},
             "yarn": {"scaling": "yarn", "factor": 32.0, "original_length": 4096}}


def _inv_freq(case):
    """(pair frequencies in radians a position, attention factor), 64 bits."""
    rot, base = case["rot"], 10000.0
    s = _SCALINGS[case["scaling"]]
    f = s.get("factor", 1.0)
    if case["scaling"] == "ntk" and rot > 2:
        base = base * f ** (rot / (rot - 2.0))
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] == "yarn":
        # turns over the original context: kept above 32, interpolated below 1, blended in pair index between
        def at(turns):
            return rot * math.log(s["original_length"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _rotary_inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
    # the packed projection q | k | v: q and k are views of it, tokens strided over all three
    qkv = _normal(gen, (T, (Hq + 2 * Hk) * D), 1.0, getattr(torch, case["dtype"]))
    g = np.random.default_rng([int(seed), 13])
    axes = 3 if case["sections"] else 1
    pos = g.integers(0, case["maxpos"], size=(axes, T)).astype(np.int32)
    return {"qkv": qkv, "pos": torch.from_numpy(pos if axes > 1 else pos[0]).to(DEV)}


def _heads(case, qkv):
    T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
    return (qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D))


def prepare(case, seed):
    state = {"case": dict(case)}
    if case["op"] == "rotary":
        state.update(_rotary_inputs(case, seed))
        state["q"], state["k"] = _heads(case, state["qkv"])
        # phase steps of each pair, in 2^-44 turns a position: exact in whole numbers
        inv, m = _inv_freq(case)
        state["steps"] = torch.from_numpy(np.round(inv / (2 * math.pi) * 2.0 ** 44).astype(np.int64)).to(DEV)
        state["m"] = m
        sec = _sections(case)
        axis = np.zeros(case["rot"] // 2, np.int64) if sec is None else np.repeat(np.arange(3), sec)
        state["axis"] = torch.from_numpy(axis).to(DEV)
        if own:
            import unpermute_route_hist_gb300 as gg
            # the frequencies of the model's layers, made once
            state["freqs"] = gg.rope_freqs(case["rot"], base=10000.0, sections=sec, device=DEV,
                                           **_SCALINGS[case["scaling"]])
        return state
    state.update(_adapter_inputs(case, seed))
    if own:
        import unpermute_route_hist_gb300 as gg
        # made once for a batch, used by every layer's projections
        state["plan"] = gg.lora_plan(state["ids"], case["L"])
    return state


# -------------------------------------------------------------------- run --

def _run_own(state):
    import unpermute_route_hist_gb300 as gg
    case = state["case"]
    if case["op"] == "adapt":
        return gg.lora_forward(state["X"], state["W"], state["A"], state["B"], state["scale"], state["plan"])
    if case["op"] == "adapt_bwd":
        return gg.lora_backward(state["dY"], state["X"], state["W"], state["A"], state["B"], state["scale"],
                                state["plan"], state["U"])
    fn = gg.rope_bwd if case["backward"] else gg.rope
    outs = {"out_q": state["q"], "out_k": state["k"]} if case["inplace"] else {}
    return fn(state["q"], state["k"], state["pos"], state["freqs"], interleaved=case["layout"] == "interleaved", **outs)


def _plain_adapt(state):
    X, W = state["X"].float(), state["W"].float()
    ids = state["ids"]
    Y = X @ W.t()
    U = torch.zeros(X.shape[0], state["A"].shape[1], device=X.device)
    for a in range(state["A"].shape[0]):
        mask = (ids == a).unsqueeze(1)
        Ua = torch.where(mask, state["scale"][a] * (X @ state["A"][a].float().t()), torch.zeros_like(U))
        Y += Ua @ state["B"][a].float().t()
        U += Ua
    return Y.to(torch.bfloat16), U.to(torch.bfloat16)


def _plain_adapt_bwd(state):
    dY, X, W, U = (state[k].float() for k in ("dY", "X", "W", "U"))
    ids = state["ids"]
    dX = dY @ W
    dA, dB = [], []
    for a in range(state["A"].shape[0]):
        mask = (ids == a).unsqueeze(1)
        Va = torch.where(mask, state["scale"][a] * (dY @ state["B"][a].float()), torch.zeros_like(U))
        dX += Va @ state["A"][a].float()
        dA.append((Va.t() @ X).to(torch.bfloat16))
        dB.append((dY.t() @ torch.where(mask, U, torch.zeros_like(U))).to(torch.bfloat16))
    return dX.to(torch.bfloat16), torch.stack(dA), torch.stack(dB)


def _plain_rotary(state):
    case = state["case"]
    rot, half = case["rot"], case["rot"] // 2
    pos = state["pos"].to(torch.int64)
    pos = pos.unsqueeze(0) if pos.dim() == 1 else pos
    phase = (pos[state["axis"]].t() * state["steps"]) & ((1 << 44) - 1)          # [T, rot/2]
    angle = phase.float() * (2 * math.pi / 2.0 ** 44)
    cos, sin = torch.cos(angle) * state["m"], torch.sin(angle) * state["m"]
    if case["backward"]:
        sin = -sin
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    out = []
    for x in (state["q"], state["k"]):
        f = x.float()
        if case["layout"] == "half":
            x1, x2 = f[..., :half], f[..., half:rot]
            turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
        else:
            x1, x2 = f[..., 0:rot:2], f[..., 1:rot:2]
            turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
        out.append(torch.cat([turned, f[..., rot:]], dim=-1).to(x.dtype))
    if case["inplace"]:
        state["q"].copy_(out[0])
        state["k"].copy_(out[1])
        return state["q"], state["k"]
    return tuple(out)


def run(state):
    if own:
        return _run_own(state)
    return {"adapt": _plain_adapt, "adapt_bwd": _plain_adapt_bwd, "rotary": _plain_rotary}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    """The definition in 64 bits, token by token group, on the host's or the card's float64."""
    if case["op"] == "rotary":
        s = _rotary_inputs(case, seed)
        inv, m = _inv_freq(case)
        sec = _sections(case)
        pos = s["pos"].cpu().numpy().astype(np.float64)
        pos = pos[None] if pos.ndim == 1 else pos
        axis = [0] * (case["rot"] // 2) if sec is None else [a for a in range(3) for _ in range(sec[a])]
        theta = np.stack([pos[axis[i]] * inv[i] for i in range(case["rot"] // 2)], axis=1)
        z = torch.from_numpy(m * np.exp((-1j if case["backward"] else 1j) * theta)).to(DEV)[:, None, :]
        outs = []
        for x in _heads(case, s["qkv"]):
            d = x.double()
            y = d.clone()
            half = case["rot"] // 2
            first = slice(0, half) if case["layout"] == "half" else slice(0, case["rot"], 2)
            second = slice(half, case["rot"]) if case["layout"] == "half" else slice(1, case["rot"], 2)
            w = torch.complex(d[..., first], d[..., second]) * z
            y[..., first], y[..., second] = w.real, w.imag
            outs.append(y.cpu().numpy())
        return tuple(outs)
    s = _adapter_inputs(case, seed)
    ids = s["ids"].cpu().numpy()
    X, W = s["X"].double(), s["W"].double()
    rows = {a: torch.from_numpy(np.flatnonzero(ids == a)).to(DEV) for a in range(case["L"])}
    scale = s["scale"].double()
    if case["op"] == "adapt":
        Y = X @ W.t()
        U = torch.zeros(case["T"], case["r"], dtype=torch.float64, device=DEV)
        for a, ix in rows.items():
            if len(ix):
                U[ix] = scale[a] * (X[ix] @ s["A"][a].double().t())
                Y[ix] += U[ix] @ s["B"][a].double().t()
        return Y.cpu().numpy(), U.cpu().numpy()
    dY = s["dY"].double()
    dX = dY @ W
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV)
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=DEV)
    for a, ix in rows.items():
        if len(ix):
            V = scale[a] * (dY[ix] @ s["B"][a].double())
            dX[ix] += V @ s["A"][a].double()
            dA[a] = V.t() @ X[ix]
            dB[a] = dY[ix].t() @ s["U"][ix].double()
    return dX.cpu().numpy(), dA.cpu().numpy(), dB.cpu().numpy()


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "rotary":
        size = 4 if case["dtype"] == "float32" else 2
        # in place, the part of the head that is not rotated is neither read nor written
        width = case["rot"] if case["inplace"] else case["D"]
        n = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * n * width * size + 4 * case["T"] * (3 if case["sections"] else 1), "flops": 3 * n * case["rot"]}
    T, K, N, L, r = (case[k] for k in ("T", "K", "N", "L", "r"))
    used = min(L, T)
    fwd = 2 * T * N * K + 2 * T * r * (K + N)
    if case["op"] == "adapt":
        return {"bytes": 2 * (T * K + N * K + used * r * (K + N) + T * N + T * r) + 4 * T, "flops": fwd}
    return {"bytes": 2 * (2 * T * K + T * N + N * K + used * r * (K + N) + T * r + L * r * (K + N)) + 4 * T,
            "flops": fwd + 2 * T * r * (K + N)}
