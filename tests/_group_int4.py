"""Inputs and 64-bit references of the group-scaled int4 operators' tests."""
import types

import torch

SCALES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def shape_of(H, E, K, I, Is, routed_scaling=1.0):  # noqa: E741
    return types.SimpleNamespace(H=H, E=E, K=K, I=I, Is=Is, routed_scaling=routed_scaling)


def gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def codes(g, *shape):
    """Uniformly random packed codes: every one of the 16 values, -8 included."""
    return torch.randint(0, 256, shape, generator=g, device=g.device, dtype=torch.uint8)


def scales(g, rows, cols, group, stype="f32"):
    n = (-(-cols // group),) if group else ()
    return torch.rand((*rows, *n), generator=g, device=g.device).mul_(0.008).add_(0.002).to(SCALES[stype])


def weights64(w, s, group):
    """float64 [..., n] from packed codes [..., n/2] and their scales."""
    b = w.to(torch.int64)
    q = torch.stack(((b & 15 ^ 8) - 8, (b >> 4 ^ 8) - 8), -1).flatten(-2).double()
    if not group:
        return q * s.double()[..., None]
    return q * s.double().repeat_interleave(group, -1)[..., : q.shape[-1]]


def linear64(x, w, s, group, add=None):
    y = x.double() @ weights64(w, s, group).t()
    return y if add is None else y + add.double()


def block_max(x, n):
    """[T, K]: the largest magnitude of the n-column block that each element lies in."""
    T, K = x.shape
    p = torch.nn.functional.pad(x.double().abs(), (0, -K % n)).view(T, -1, n)
    return p.amax(-1, keepdim=True).expand_as(p).reshape(T, -1)[:, :K]


def streams(T, N, half):
    """Whether a projection of these sizes surely runs on the weight-streaming kernel (148 SMs)."""
    K = 2 * half
    return T <= 8 and T * 2 * (K + 320) <= 113 * 1024 and (T <= 4 or N > 16 * 148 or T * K <= 28000)


def linear_bound(x, w, s, group, add=None):
    """How far an f32 result may be from linear64, element by element.  The weight-streaming kernel (streams)
    holds an activation to within 2^-15 of the largest of its 256-column block; the tensor-core kernel rounds
    code * scale to bf16, half a step of which is 2^-8 of the weight, from a scale held to 2^-16.  Sums: every product or group sum enters one f32 addition
    chain no longer than K / 16 + 64 (2^-24 of the running magnitude each, doubled for the tensor cores' truncation)."""
    W = weights64(w, s, group).abs()
    mag = x.double().abs() @ W.t()
    b = 2.0 ** -15 * (block_max(x, 256) @ W.t()) if streams(x.shape[0], *w.shape) else (2.0 ** -8 + 2.0 ** -16) * mag
    b = b + (x.shape[1] / 16 + 64) * 2.0 ** -23 * mag
    return b if add is None else b + 2.0 ** -23 * (mag + add.double().abs())


def linear_rms(T, N, half):
    """Bound of the relative L2 error of an f32 result: activations to 2^-15 of a block's largest value (under 2^-13 of
    its r.m.s.), or weights rounded to bf16 (uniform within half a step of at most 2^-8: r.m.s. 2^-8 / sqrt(3) < 2^-8.7,
    independent errors)."""
    return 2.0 ** -12 if streams(T, N, half) else 2.0 ** -8.7


def make_layer(shape, group, stype="f32", seed=0, device="cuda"):
    g = gen(seed, device)
    H, E, I, Is = shape.H, shape.E, shape.I, shape.Is  # noqa: E741
    L = {"router_w": torch.randn((E, H), generator=g, device=device) * (2.0 / H ** 0.5),
         "router_bias": torch.rand((E,), generator=g, device=device) * 0.2 - 0.1,
         "w13": codes(g, E, 2 * I, H // 2), "s13": scales(g, (E, 2 * I), H, group, stype),
         "w2": codes(g, E, H, I // 2), "s2": scales(g, (E, H), I, group, stype)}
    if Is:
        L |= {"sh_w13": codes(g, 2 * Is, H // 2), "sh_s13": scales(g, (2 * Is,), H, group, stype),
              "sh_w2": codes(g, H, Is // 2), "sh_s2": scales(g, (H,), Is, group, stype)}
    return L


def route64(x, L, shape, topp=0.0):
    """Per token: (picked experts in pick order, their weights), and the smallest distance of a decision from
    falling the other way."""
    out, margin = [], float("inf")
    score = torch.sigmoid(x.double() @ L["router_w"].double().t()).cpu()
    key = (score + L["router_bias"].double().cpu()).nan_to_num(nan=-torch.inf)
    for s, k in zip(score, key):
        order = sorted(range(shape.E), key=lambda e: (-float(k[e]), e))
        picks = order[:shape.K]
        ks = [float(k[e]) for e in order[:shape.K + 1]]
        margin = min([margin] + [a - b for a, b in zip(ks, ks[1:])])
        if 0 < topp < 1:
            total, kept, run = sum(float(s[e]) for e in picks), [], 0.0
            for e in sorted(picks, key=lambda e: (-float(s[e]), e)):
                margin = min(margin, abs(run - topp * total)) if kept else margin
                if run < topp * total:
                    kept.append(e)
                run += float(s[e])
            picks = [e for e in picks if e in kept]
        tot = sum(float(s[e]) for e in picks)
        out.append((picks, [shape.routed_scaling * float(s[e]) / tot for e in picks]))
    return out, margin


def _ffn64(x, w13, s13, w2, s2, group):
    z = weights64(w13, s13, group) @ x
    a, b = z.chunk(2)
    return weights64(w2, s2, group) @ (a * torch.sigmoid(a) * b)


def few64(x, L, shape, group, residual=False, topp=0.0, picks=None):
    """The layer in 64 bits; ``picks``: int [T, K] experts to use (-1: none) instead of its own choice."""
    own, _ = route64(x, L, shape, topp)
    rows = []
    for t, v in enumerate(x.double()):
        es, ws = own[t]
        if picks is not None:
            es = [int(e) for e in picks[t] if e >= 0]
            sc = torch.sigmoid(L["router_w"][es].double() @ v)
            ws = [float(shape.routed_scaling * a / sc.sum()) for a in sc]
        y = v.clone() if residual else torch.zeros_like(v)
        for e, wt in zip(es, ws):
            y += wt * _ffn64(v, L["w13"][e], L["s13"][e], L["w2"][e], L["s2"][e], group)
        if shape.Is:
            y += _ffn64(v, L["sh_w13"], L["sh_s13"], L["sh_w2"], L["sh_s2"], group)
        rows.append(y)
    return torch.stack(rows)
