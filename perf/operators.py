"""The group-scaled int4 operators of this library, as a set of measurable cases.

Two operators work on the same weights: 4-bit codes, two per byte, with one scale for each
group of consecutive columns of a row (``group`` columns; 0: one scale for the whole row).

``linear``  y[t, n] = sum_k x[t, k] c[n, k] s[n, k // group]  (+ a[t, n])
    the dense projections beside the expert layers (decode: one to a few tokens; prompts: more)
``few``     a whole mixture-of-experts layer for a few tokens: sigmoid + bias router, top-K,
    SwiGLU experts and the shared expert with such weights, the weighted combine (+ residual)

``own`` false: the formulas in elementary torch operations; ``own`` true: the library's calls.
"""
import torch

own = False

DEVICE = "cuda"
_SCALES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_WIDTH = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def _linear(name, T, N, K, group, scales, add=False):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "group": group, "scales": scales, "add": add}


def _few(name, T, H, E, K, I, Is, group, scales, scaling=1.0, residual=True):  # noqa: E741
    return {"name": name, "op": "few", "T": T, "H": H, "E": E, "K": K, "I": I, "Is": Is, "group": group,
            "scales": scales, "scaling": scaling, "residual": residual}


def listed():
    return [
        # a square projection at the small model's hidden size, one token: launch latency counts
        _linear("linear nano T1", 1, 1024, 1024, 128, "bf16"),
        # a square projection at the large layer's hidden size, one token: the weight stream
        _linear("linear large T1", 1, 6144, 6144, 128, "bf16", add=True),
        # a dense feed-forward's gate and up rows, four speculated tokens, fine groups in f32
        _linear("linear gate-up T4", 4, 12288, 6144, 32, "f32"),
        # odd everything: rows that fill no tile, a last group of half a length, an odd token count
        _linear("linear odd T7", 7, 5001, 1120, 64, "f16", add=True),
        # a decode batch, the down projection's aspect
        _linear("linear batch T16", 16, 6144, 2048, 128, "bf16"),
        # the largest decode batch of the weight-streaming kernels
        _linear("linear batch T64", 64, 6144, 6144, 128, "bf16", add=True),
        # a prompt through the shared expert's gate and up rows
        _linear("linear prompt T512", 512, 4096, 6144, 64, "bf16"),
        # one layer of the small model's decode, one token, fine groups
        _few("few nano T1", 1, 1024, 64, 2, 512, 2048, 32, "f32"),
        # the same with four speculated tokens and one scale a row (the weights of the other layer calls)
        _few("few nano T4", 4, 1024, 64, 2, 512, 2048, 0, "f32"),
        # the largest pass of the small model
        _few("few nano T8", 8, 1024, 64, 2, 512, 2048, 128, "bf16"),
        # the large layer, one token: 8 of 256 experts and the shared one
        _few("few large T1", 1, 6144, 256, 8, 2048, 2048, 128, "bf16", scaling=2.5),
        # the large layer verifying five speculated tokens; an expert seldom serves two of them
        _few("few large T5", 5, 6144, 256, 8, 2048, 2048, 64, "bf16", scaling=2.5, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    group = rng.choice([0, 32, 32, 64, 128, 128, 256])
    scales = rng.choice(["f32", "bf16", "bf16", "f16"])
    if rng.random() < 0.55:
        T, N, K = _log(rng, 1, 512), _log(rng, 200, 12288), 32 * _log(rng, 4, 256)
        return {"op": "linear", "T": T, "N": min(N, max(200, 2 ** 33 // (T * K))), "K": K, "group": group,
                "scales": scales, "add": rng.random() < 0.5}
    E = _log(rng, 4, 256)
    T, H, K = _log(rng, 1, 8), 128 * _log(rng, 2, 48), min(E, _log(rng, 1, 8))
    I = 128 * min(_log(rng, 1, 16), max(1, 3 * 10 ** 8 // (128 * T * K * H)))  # noqa: E741
    return {"op": "few", "T": T, "H": H, "E": E, "K": K, "I": I,
            "Is": 128 * rng.choice([0, 1, 4, _log(rng, 1, 16)]), "group": group, "scales": scales,
            "scaling": rng.choice([1.0, 2.5]), "residual": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs
def _codes(g, *shape):
    """Packed codes, bell-shaped over -8..7: each nibble is the sum of four short random numbers."""
    n = 1
    for d in shape:
        n *= d
    r = [torch.randint(-2 ** 63, 2 ** 63 - 1, (-(-n // 8),), generator=g, device=DEVICE).view(torch.uint8)[:n]
         for _ in range(4)]
    b = (r[0] & 0x33) + (r[1] & 0x33) + (r[2] & 0x77) + ((r[3] & 0x11) << 1)
    return (b ^ 0x88).view(shape)


def _scales(g, case, rows, cols):
    """Scales of weights with a deviation near 0.02, one for each group of each row."""
    n = (-(-cols // case["group"]),) if case["group"] else ()
    return torch.rand((*rows, *n), generator=g, device=DEVICE).mul_(0.006).add_(0.004).to(_SCALES[case["scales"]])


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"] = _normal(g, T, K).to(torch.bfloat16)
        s["w"], s["s"] = _codes(g, N, K // 2), _scales(g, case, (N,), K)
        s["a"] = _normal(g, T, N).to(torch.bfloat16) if case["add"] else None
    else:
        T, H, E, K, I, Is = (case[k] for k in ("T", "H", "E", "K", "I", "Is"))
        L = {"router_w": _normal(g, E, H).mul_(0.02),
             "router_bias": torch.rand((E,), generator=g, device=DEVICE).mul_(0.2).sub_(0.1),
             "w13": _codes(g, E, 2 * I, H // 2), "s13": _scales(g, case, (E, 2 * I), H),
             "w2": _codes(g, E, H, I // 2), "s2": _scales(g, case, (E, H), I)}
        if Is:
            L |= {"sh_w13": _codes(g, 2 * Is, H // 2), "sh_s13": _scales(g, case, (2 * Is,), H),
                  "sh_w2": _codes(g, H, Is // 2), "sh_s2": _scales(g, case, (H,), Is)}
        s["layer"] = L
        # tokens whose K-th and next router keys are apart: a tie to rounding may go either way
        x = _normal(g, 4 * T + 32, H).to(torch.bfloat16)
        keys = torch.sigmoid(x.double() @ L["router_w"].double().T) + L["router_bias"].double()
        keys = keys.sort(dim=1, descending=True).values
        gap = keys[:, K - 1] - keys[:, K] if K < E else torch.ones_like(keys[:, 0])
        s["x"] = x[(gap < 1e-5).to(torch.int32).argsort(stable=True)[:T]].contiguous()
    if own:
        import int4_expert_ffn_sigmoid_b200 as moe
        if case["op"] == "linear":
            s["call"] = moe.Int4Linear(s["w"], s["s"], group=case["group"])
        else:
            import workloads
            shape = workloads.LayerShape(H=H, E=E, K=K, I=I, Is=Is, routed_scaling=case["scaling"])
            s["call"] = moe.MoEFewLayer(s["layer"], shape, group=case["group"], max_tokens=T)
    return s


# ------------------------------------------------------------- plain forms
def _weights(codes, scales, group):
    """The f32 weights of packed codes [..., n / 2] and their scales."""
    lo, hi = codes & 15, codes >> 4
    c = torch.stack((lo, hi), dim=-1).flatten(-2).to(torch.float32)
    c = torch.where(c < 8, c, c - 16)
    if not group:
        return c * scales.float()[..., None]
    return c * scales.float().repeat_interleave(group, dim=-1)[..., : c.shape[-1]]


def _ffn(x, w13, s13, w2, s2, group):
    """SwiGLU of x [..., H] with matrices of the same leading dimensions: f32 [..., H]."""
    gu = (_weights(w13, s13, group) @ x.float()[..., None])[..., 0]
    g, u = gu.chunk(2, dim=-1)
    h = g / (1 + torch.exp(-g)) * u
    return (_weights(w2, s2, group) @ h[..., None])[..., 0]


def run(state):
    if own:
        if state["op"] == "linear":
            return state["call"](state["x"], add=state["a"])
        return state["call"](state["x"], residual=state["residual"])
    x, group = state["x"], state["group"]
    if state["op"] == "linear":
        y = x.float() @ _weights(state["w"], state["s"], group).T
        return (y if state["a"] is None else y + state["a"].float()).to(torch.bfloat16)
    L, K = state["layer"], state["K"]
    # scores in 64 bits: a pick is a comparison of two of them
    score = 1 / (1 + torch.exp(-(x.double() @ L["router_w"].double().T)))
    idx = (score + L["router_bias"].double()).sort(dim=1, descending=True, stable=True).indices[:, :K]
    picked = score.gather(1, idx)
    w = (state["scaling"] * picked / picked.sum(dim=1, keepdim=True)).float()
    y = _ffn(x[:, None], L["w13"][idx], L["s13"][idx], L["w2"][idx], L["s2"][idx], group)
    y = (y * w[..., None]).sum(dim=1)
    if state["Is"]:
        y = y + _ffn(x, L["sh_w13"], L["sh_s13"], L["sh_w2"], L["sh_s2"], group)
    return (y + x.float() if state["residual"] else y).to(torch.bfloat16)


def work(case):
    n = lambda rows, cols: rows * (cols / 2 + (-(-cols // (case["group"] or cols))) * _WIDTH[case["scales"]])  # noqa: E731
    T = case["T"]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": n(N, K) + 2 * T * K + (4 if case["add"] else 2) * T * N, "flops": 2 * T * N * K}
    H, E, K, I, Is = (case[k] for k in ("H", "E", "K", "I", "Is"))
    touched = E * (1 - (1 - K / E) ** T)  # experts that T tokens are expected to pick
    return {"bytes": touched * (n(2 * I, H) + n(H, I)) + n(2 * Is, H) + (n(H, Is) if Is else 0) + 4 * E * (H + 1) + 4 * T * H,
            "flops": 2 * T * (E * H + 3 * H * (K * I + Is))}


# --------------------------------------------------- the definition, 64 bits
def _matrix64(codes, scales, group):
    rows, half = codes.shape
    q = torch.empty((rows, 2 * half), dtype=torch.float64, device=codes.device)
    b = codes.to(torch.int32)
    q[:, 0::2] = ((b << 28) >> 28).double()
    q[:, 1::2] = ((b << 24) >> 28).double()
    at = torch.arange(2 * half, device=codes.device) // (group or 2 * half)
    return q * scales.reshape(rows, -1).double()[:, at]


def _expert64(x, w13, s13, w2, s2, group):
    z = _matrix64(w13, s13, group) @ x
    half = z.shape[0] // 2
    return _matrix64(w2, s2, group) @ (z[:half] * torch.sigmoid(z[:half]) * z[half:])


def exact(case, seed):
    s = prepare(case, seed)
    group = case["group"]
    if case["op"] == "linear":
        y = torch.stack([_matrix64(s["w"], s["s"], group) @ v for v in s["x"].double()]) if case["T"] <= 2 else \
            s["x"].double() @ _matrix64(s["w"], s["s"], group).t()
        return y + s["a"].double() if case["add"] else y
    L, rows = s["layer"], []
    names = ("w13", "s13", "w2", "s2")
    for x in s["x"].double():
        score = torch.sigmoid(L["router_w"].double() @ x)
        key = score + L["router_bias"].double()
        picks = []
        for _ in range(case["K"]):
            e = int((key == key.max()).nonzero()[0])  # the lowest index of the largest key
            key[e] = -torch.inf
            picks.append(e)
        y = x.clone() if case["residual"] else torch.zeros_like(x)
        for e in picks:
            y += case["scaling"] * score[e] / score[picks].sum() * _expert64(x, *(L[n][e] for n in names), group)
        if case["Is"]:
            y += _expert64(x, *(L["sh_" + n] for n in names), group)
        rows.append(y)
    return torch.stack(rows)
