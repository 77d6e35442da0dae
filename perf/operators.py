"""What the expert-layer operators are measured on.

Five operators: the routing of tokens to experts (scores, choice, weights and the order of the
rows by expert, with the gradient of the weights), the quantisation of rows to 8 bits, the 8-bit
integer product with a scale for each token and channel (for one matrix, and for the experts'
matrices over rows sorted by expert), and the weighted sum of the experts' rows with its gradient.

``run`` computes them in elementary torch operations in 32 bits, or, with ``own``, through the
library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1), "f16": (torch.float16, 2)}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
LARGEST = 2.0 * 8192 ** 3  # operations of the largest product


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a served batch: 16 tokens, many experts in groups, a bias for balance
        dict(name="route_decode", kind="route", T=16, E=256, k=8, score="sigmoid", groups=8, kept=4, top=2,
             renorm=True, bias=True, type="f32", padded=0),
        # a prompt batch with padded tokens at its end, softmax scores, no groups
        dict(name="route_prompt", kind="route", T=16384, E=64, k=6, score="softmax", groups=1, kept=1, top=1,
             renorm=True, bias=False, type="bf16", padded=515),
        # the router's gradient of a training step
        dict(name="route_backward", kind="route_backward", T=16384, E=256, k=8, score="sigmoid", groups=1, kept=1,
             top=1, renorm=True, bias=True, type="f32", padded=0),
        # a single token through one linear layer: latency and the reading of the weights
        dict(name="product_token", kind="product", M=1, N=4096, K=4096, out="bf16"),
        # a decode batch against a wide layer
        dict(name="product_skinny", kind="product", M=128, N=16384, K=4096, out="bf16"),
        # a ragged batch, odd in every direction, 32-bit outputs
        dict(name="product_odd", kind="product", M=777, N=4101, K=4001, out="f32"),
        # a prompt through one linear layer, from 16-bit activations: quantised, then multiplied
        dict(name="linear_square", kind="linear", M=8192, N=8192, K=8192, type="bf16", out="bf16"),
        # the experts' product of a decode step: few rows for each expert, some have none
        dict(name="experts_decode", kind="experts", M=96, E=64, N=4096, K=2048, out="bf16"),
        # the experts' product of a prompt batch
        dict(name="experts_prompt", kind="experts", M=32768, E=64, N=4096, K=2048, out="bf16"),
        # the sum of the experts' rows of a prompt batch
        dict(name="combine", kind="combine", T=4096, E=64, k=6, N=4096, type="bf16", padded=100),
        # its gradient
        dict(name="combine_backward", kind="combine_backward", T=4096, E=64, k=6, N=4096, type="bf16", padded=100),
        # a whole expert layer: routed, quantised, two products with a gate between them, summed
        dict(name="layer", kind="layer", T=256, E=64, k=6, score="softmax", groups=1, kept=1, top=1, renorm=True,
             bias=False, type="bf16", padded=0, H=2048, F=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _route_draw(rng, T):
    E = rng.choice([8, 16, 60, 64, 72, 128, 160, 256, 384])
    groups = rng.choice([1, 1, 4]) if E % 8 == 0 else 1
    kept = 2 if groups == 4 else 1
    k = rng.randint(1, min(10, E // groups * kept))
    return dict(T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), groups=groups, kept=kept,
                top=rng.choice([1, 2]), renorm=rng.random() < 0.6, bias=rng.random() < 0.5,
                type=rng.choice(["f32", "bf16"]), padded=rng.choice([0, T // 9]))


def draw(rng):
    kind = rng.choice(["route", "route_backward", "product", "product", "linear", "experts", "experts", "combine",
                       "combine_backward", "layer"])
    if kind in ("route", "route_backward"):
        return dict(_route_draw(rng, _log(rng, 1, 16384)), kind=kind)
    if kind in ("product", "linear"):
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 16384), N=_log(rng, 64, 16384), K=_log(rng, 64, 16384),
                     out=rng.choice(["bf16", "f16", "f32"]))
            if 2.0 * c["M"] * c["N"] * c["K"] <= LARGEST / 2:
                break
        return dict(c, type=rng.choice(["bf16", "f16", "f32"])) if kind == "linear" else c
    if kind == "experts":
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 32768), E=rng.choice([8, 16, 60, 64, 128]), N=_log(rng, 64, 4096),
                     K=_log(rng, 64, 4096), out=rng.choice(["bf16", "f32"]))
            if 2.0 * c["M"] * c["N"] * c["K"] <= LARGEST / 4 and c["E"] * c["N"] * c["K"] <= 64 * 4096 * 2048:
                return c
    if kind in ("combine", "combine_backward"):
        T = _log(rng, 1, 4096)
        E = rng.choice([8, 60, 64, 128])
        return dict(kind=kind, T=T, E=E, k=rng.randint(1, 8), N=_log(rng, 64, 4096),
                    type=rng.choice(["bf16", "f16", "f32"]), padded=rng.choice([0, T // 9]))
    c = _route_draw(rng, _log(rng, 1, 512))
    while c["E"] > 72:
        c = _route_draw(rng, c["T"])
    return dict(c, kind=kind, type="bf16", padded=0, H=16 * _log(rng, 8, 128), F=16 * _log(rng, 8, 128))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _int8(g, *shape):
    """Quantised normal values; rows padded to a multiple of 16 bytes, as the library's leading dimensions are."""
    ld = -(-shape[-1] // 16) * 16
    q = torch.empty(*shape[:-1], ld, dtype=torch.int8, device=DEV)
    if q.dim() == 3:
        for i in range(shape[0]):
            q[i] = (torch.randn(shape[1], ld, generator=g, device=DEV) * 32).round().clamp_(-127, 127).to(torch.int8)
    else:
        q.copy_((torch.randn(*shape[:-1], ld, generator=g, device=DEV) * 32).round().clamp_(-127, 127))
    return q


def _scales(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV) * 0.02 + 0.002


def _choice64(logits, bias, c):
    """Scores, and what the choice goes by, in 64 bits; the scores of the groups that are kept."""
    x = logits.double()
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    return s, s + bias.double() if bias is not None else x


def _logits(g, c):
    """Router logits. Two experts of a token whose scores agree in their first 20 bits or so have no order that
    survives rounding: such tokens are replaced by others, so that the choice has one right answer."""
    T, E = c["T"], c["E"]
    n = T + 64
    x = (torch.randn(n, E, generator=g, device=DEV) * 1.5).to(TYPES[c["type"]][0])
    bias = None
    if c["bias"]:  # as a run of sign updates of 0.001 leaves it
        bias = torch.randint(-60, 61, (E,), generator=g, device=DEV).float() * 0.001
    s, by = _choice64(x, bias, c)
    v = by.sort(-1).values
    gap = v[:, 1:] - v[:, :-1]
    bad = ((gap > 0) & (gap < 1e-6)).any(-1)
    if c["groups"] > 1:
        t = (s if bias is None else by).view(n, c["groups"], -1).topk(min(c["top"], E // c["groups"]), -1).values.sum(-1)
        v = t.sort(-1).values
        bad |= ((v[:, 1:] - v[:, :-1]) < 1e-6).any(-1)
    if bias is not None:  # 16-bit logits and a common step of the bias: equal in 64 bits, not in 32, and the reverse
        v = by.float().sort(-1).values
        bad |= ((v[:, 1:] == v[:, :-1]) & (by.sort(-1).values[:, 1:] != by.sort(-1).values[:, :-1])).any(-1)
    good = torch.nonzero(~bad).flatten()
    if good.numel() == 0:
        good = torch.arange(n, device=DEV)
    pick = torch.arange(T, device=DEV)
    pick = torch.where(bad[:T], good[pick % good.numel()], pick)
    x = x[pick].contiguous()
    if c["padded"]:
        x[T - c["padded"]:] = -math.inf
    return x, bias


def _counts(g, M, E):
    """Rows of each expert: uneven, as a router leaves them; with few rows some have none."""
    p = torch.softmax(torch.randn(E, generator=g, device=DEV) * 0.5, 0)
    of = torch.multinomial(p, M, replacement=True, generator=g)
    return torch.bincount(of, minlength=E)


def _pairs(g, c):
    """Experts of each token without repetition (-1 for padded tokens), in a drawn order, and the order by expert."""
    ids = torch.rand(c["T"], c["E"], generator=g, device=DEV).argsort(-1)[:, :c["k"]].to(torch.int32)
    if c["padded"]:
        ids[c["T"] - c["padded"]:] = -1
    return ids, _plan(ids, c["E"])


def prepare(case, seed):
    c, g = case, _gen(seed)
    kind = c["kind"]
    s = dict(case=c)
    if kind in ("route", "route_backward", "layer"):
        s["logits"], s["bias"] = _logits(g, c)
        T, E, k = c["T"], c["E"], c["k"]
        s["weights"] = torch.empty(T, k, device=DEV)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    if kind in ("route", "layer"):
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        s["workspace"] = torch.empty(4 << 20, dtype=torch.uint8, device=DEV)
    if kind == "route_backward":
        s["ids"] = _route(s["logits"], s["bias"], c)[1]
        s["dweights"] = torch.randn(T, k, generator=g, device=DEV)
        s["dlogits"] = torch.empty_like(s["logits"])
    if kind in ("product", "linear"):
        M, N, K = c["M"], c["N"], c["K"]
        s["B"], s["sb"] = _int8(g, N, K), _scales(g, N)
        s["D"] = torch.empty(M, N, dtype=TYPES[c["out"]][0], device=DEV)
        s["A"], s["sa"] = _int8(g, M, K), _scales(g, M)
        if kind == "linear":
            s["X"] = torch.randn(M, K, generator=g, device=DEV).to(TYPES[c["type"]][0])
    if kind == "experts":
        M, E, N, K = c["M"], c["E"], c["N"], c["K"]
        n = _counts(g, M, E)
        s["capacity"] = int(n.max())
        s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        s["A"], s["sa"] = _int8(g, M, K), _scales(g, M)
        s["B"], s["sb"] = _int8(g, E, N, K), _scales(g, E, N)
        s["D"] = torch.empty(M, N, dtype=TYPES[c["out"]][0], device=DEV)
    if kind in ("combine", "combine_backward"):
        T, k, N = c["T"], c["k"], c["N"]
        t = TYPES[c["type"]][0]
        ids, plan = _pairs(g, c)
        s["slots"] = plan[1]
        s["weights"] = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["Y"] = torch.randn(T * k, N, generator=g, device=DEV).to(t)
        s["D"] = torch.empty(T, N, dtype=t, device=DEV)
        if kind == "combine_backward":
            s["dD"] = torch.randn(T, N, generator=g, device=DEV).to(t)
            s["dY"] = torch.zeros(T * k, N, dtype=t, device=DEV)
            s["dweights"] = torch.empty(T, k, device=DEV)
    if kind == "layer":
        H, F = c["H"], c["F"]
        s["X"] = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
        s["B1"], s["sb1"] = _int8(g, E, 2 * F, H), torch.rand(E, 2 * F, generator=g, device=DEV) * 0.001 + 0.0002
        s["B2"], s["sb2"] = _int8(g, E, H, F), torch.rand(E, H, generator=g, device=DEV) * 0.001 + 0.0002
        s["capacity"] = int(torch.bincount(_route(s["logits"], s["bias"], c)[1].flatten(), minlength=E).max())
        R = T * k
        s["A1"], s["sa1"] = torch.empty(R, H, dtype=torch.int8, device=DEV), torch.empty(R, device=DEV)
        s["Y1"] = torch.empty(R, 2 * F, device=DEV)
        s["A2"], s["sa2"] = torch.empty(R, F, dtype=torch.int8, device=DEV), torch.empty(R, device=DEV)
        s["Y2"] = torch.empty(R, H, device=DEV)
        s["D"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softmax(x):
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _route(logits, bias, c):
    """Weights and experts of each token: -1 and 0 where no expert is left."""
    x = logits.float()
    s = _sigmoid(x) if c["score"] == "sigmoid" else _softmax(x)
    by = torch.where(x == -math.inf, x, s + bias if bias is not None else x)
    T, E = x.shape
    if c["groups"] > 1:
        of = torch.where(x == -math.inf, x, s + bias if bias is not None else s).view(T, c["groups"], -1)
        t = of.sort(-1, descending=True).values[..., :c["top"]]
        t = torch.where(t == -math.inf, torch.zeros_like(t), t).sum(-1)
        t = torch.where(of.amax(-1) == -math.inf, torch.full_like(t, -math.inf), t)
        kept = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device)
        kept.scatter_(1, t.sort(dim=-1, descending=True, stable=True).indices[:, :c["kept"]], True)
        by = torch.where(kept.repeat_interleave(E // c["groups"], 1), by, torch.full_like(by, -math.inf))
    v, ids = by.sort(dim=-1, descending=True, stable=True)
    v, ids = v[:, :c["k"]], ids[:, :c["k"]]
    none = v == -math.inf
    w = torch.where(none, torch.zeros_like(v), s.gather(1, ids))
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return w * 2.5, torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32)


def _plan(ids, E):
    """offsets[e]: first row of expert e; slots: the row of each pair; tokens: the token of each row."""
    T, k = ids.shape
    key = torch.where(ids < 0, torch.full_like(ids, E), ids).flatten().long()
    order = key.sort(stable=True).indices
    n = (key[:, None] == torch.arange(E, device=ids.device)).sum(0) if key.numel() * E <= 1 << 27 else torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([n.new_zeros(1), n.cumsum(0)])
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=ids.device)
    slots = torch.where(key == E, torch.full_like(slots, -1), slots).view(T, k)
    tokens = torch.where(key[order] == E, torch.full_like(order, -1), order // k)
    return offsets.to(torch.int32), slots.to(torch.int32), tokens.to(torch.int32)


def _route_grad(logits, ids, dw, c):
    x = logits.float()
    none = ids < 0
    at = torch.where(none, torch.zeros_like(ids), ids).long()
    dw = torch.where(none, torch.zeros_like(dw), dw) * 2.5
    s = _sigmoid(x) if c["score"] == "sigmoid" else _softmax(x)
    p = torch.where(none, torch.zeros_like(dw), s.gather(1, at))
    if c["renorm"]:
        total = p.sum(-1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        ds = (dw - (dw * p).sum(-1, keepdim=True) / total) / total
    else:
        ds = dw
    ds = torch.where(none, torch.zeros_like(ds), ds)
    full = torch.zeros_like(x).scatter_add_(1, at, ds)
    if c["score"] == "sigmoid":
        d = full * s * (1.0 - s)
    else:
        d = s * (full - (full * s).sum(-1, keepdim=True))
    return d.to(logits.dtype)


def _quantise(x):
    """Rows to whole numbers of at most 127, and their scales."""
    x = x.float()
    scale = x.abs().amax(-1) / 127.0
    q = torch.round(x / torch.where(scale == 0, torch.ones_like(scale), scale)[:, None])
    return q, scale


def _products(q, sa, offsets, B, sb, K, capacity):
    """The experts' products over rows sorted by expert."""
    E, M = B.shape[0], q.shape[0]
    row = torch.arange(M, device=q.device)
    e = (row[:, None] >= offsets[None, 1:]).sum(1).clamp_(max=E - 1)
    place = row - offsets[e].long()
    x = torch.zeros(E, capacity, K, device=q.device)
    x[e, place] = q.float()
    y = torch.bmm(x, B[..., :K].float().transpose(1, 2))[e, place]
    return y * sa[:, None] * sb[e]


def _combine(y, slots, w):
    rows = torch.where(slots < 0, torch.zeros_like(slots), slots).long()
    w = torch.where(slots < 0, torch.zeros_like(w), w)
    return (y[rows].float() * w[..., None]).sum(1)


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "route":
        w, ids = _route(s["logits"], s["bias"], c)
        offsets, slots, tokens = _plan(ids, c["E"])
        return dict(weights=w, ids=ids, offsets=offsets, slots=slots, tokens=tokens)
    if kind == "route_backward":
        return dict(dlogits=_route_grad(s["logits"], s["ids"], s["dweights"], c))
    if kind == "product":
        y = s["A"][:, :c["K"]].float() @ s["B"][:, :c["K"]].float().t()
        return dict(D=(y * s["sa"][:, None] * s["sb"]).to(s["D"].dtype))
    if kind == "linear":
        q, sa = _quantise(s["X"])
        return dict(D=((q @ s["B"][:, :c["K"]].float().t()) * sa[:, None] * s["sb"]).to(s["D"].dtype))
    if kind == "experts":
        y = _products(s["A"][:, :c["K"]], s["sa"], s["offsets"], s["B"], s["sb"], c["K"], s["capacity"])
        return dict(D=y.to(s["D"].dtype))
    if kind == "combine":
        return dict(D=_combine(s["Y"], s["slots"], s["weights"]).to(s["D"].dtype))
    if kind == "combine_backward":
        none = s["slots"] < 0
        rows = torch.where(none, torch.zeros_like(s["slots"]), s["slots"]).long()
        dw = torch.where(none, torch.zeros_like(s["weights"]), (s["Y"][rows].float() * s["dD"].float()[:, None]).sum(-1))
        R = s["Y"].shape[0]
        dy = torch.zeros(R + 1, c["N"], device=DEV)  # the last row takes the pairs that have none
        dy[torch.where(none, torch.full_like(rows, R), rows)] = s["weights"][..., None] * s["dD"].float()[:, None]
        return dict(dY=dy[:R].to(s["Y"].dtype), dweights=dw)
    w, ids = _route(s["logits"], s["bias"], c)
    offsets, slots, tokens = _plan(ids, c["E"])
    q, sa = _quantise(s["X"][tokens.long()])
    y = _products(q, sa, offsets, s["B1"], s["sb1"], c["H"], s["capacity"])
    gate, up = y[:, :c["F"]], y[:, c["F"]:]
    q, sa = _quantise(gate / (1.0 + torch.exp(-gate)) * up)
    y = _products(q, sa, offsets, s["B2"], s["sb2"], c["F"], s["capacity"])
    return dict(D=_combine(y, slots, w).to(torch.bfloat16), ids=ids)


# ------------------------------------------------------------------ the library

def _rule(G, c):
    return dict(score=G.ROUTE_SIGMOID if c["score"] == "sigmoid" else G.ROUTE_SOFTMAX, groups=c["groups"],
                group_top=c["top"], groups_kept=c["kept"], renormalize=int(c["renorm"]), scale=2.5)


def _library(s):
    import smem_swizzle_layouts_gb300 as G
    c = s["case"]
    kind = c["kind"]
    code = TYPES[c["type"]][1] if "type" in c else 0
    out = TYPES[c["out"]][1] if "out" in c else code
    if kind in ("route", "layer"):
        T, E, k = c["T"], c["E"], c["k"]
        G.gemm_route(T, E, s["logits"], code, E, s["bias"], k, _rule(G, c), s["weights"], s["ids"])
        G.gemm_route_plan(T, E, k, s["ids"], s["offsets"], s["slots"], s["tokens"], s["workspace"],
                          s["workspace"].numel())
        if kind == "route":
            return dict(weights=s["weights"], ids=s["ids"], offsets=s["offsets"], slots=s["slots"], tokens=s["tokens"])
    if kind == "route_backward":
        T, E, k = c["T"], c["E"], c["k"]
        G.gemm_route_backward(T, E, s["logits"], code, E, k, _rule(G, c), s["ids"], s["dweights"], s["dlogits"], E)
        return dict(dlogits=s["dlogits"])
    if kind in ("product", "linear"):
        M, N, K = c["M"], c["N"], c["K"]
        A, sa, B = s["A"], s["sa"], s["B"]
        if kind == "linear":
            G.gemm_quantize_int8(M, K, s["X"], code, M, K, None, G.QUANT_PLAIN, A, A.stride(0), sa)
        G.gemm_int8(M, N, K, A, A.stride(0), sa, B, B.stride(0), s["sb"], s["D"], N, out)
        return dict(D=s["D"])
    if kind == "experts":
        M, E, N, K = c["M"], c["E"], c["N"], c["K"]
        A, B = s["A"], s["B"]
        G.gemm_int8_grouped(M, N, K, E, s["offsets"], A, A.stride(0), s["sa"], B, B.stride(1), B.stride(0), s["sb"],
                            s["D"], N, out)
        return dict(D=s["D"])
    if kind == "combine":
        G.gemm_route_combine(c["T"], c["N"], c["k"], s["Y"], code, c["T"] * c["k"], c["N"], s["slots"], s["weights"],
                             s["D"], code, c["N"])
        return dict(D=s["D"])
    if kind == "combine_backward":
        N = c["N"]
        G.gemm_route_combine_backward(c["T"], N, c["k"], s["dD"], code, N, s["Y"], code, c["T"] * c["k"], N,
                                      s["slots"], s["weights"], s["dY"], N, s["dweights"])
        return dict(dY=s["dY"], dweights=s["dweights"])
    R, H, F = T * k, c["H"], c["F"]
    G.gemm_quantize_int8(R, H, s["X"], 1, T, H, s["tokens"], G.QUANT_PLAIN, s["A1"], H, s["sa1"])
    G.gemm_int8_grouped(R, 2 * F, H, E, s["offsets"], s["A1"], H, s["sa1"], s["B1"], H, 2 * F * H, s["sb1"], s["Y1"],
                        2 * F, G.OUT_F32)
    G.gemm_quantize_int8(R, F, s["Y1"], 0, R, 2 * F, None, G.QUANT_GATED, s["A2"], F, s["sa2"])
    G.gemm_int8_grouped(R, H, F, E, s["offsets"], s["A2"], F, s["sa2"], s["B2"], F, H * F, s["sb2"], s["Y2"], H,
                        G.OUT_F32)
    G.gemm_route_combine(T, H, k, s["Y2"], 0, R, H, s["slots"], s["weights"], s["D"], 1, H)
    return dict(D=s["D"], ids=s["ids"])


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ work and the values in 64 bits

def work(case):
    c = case
    kind = c["kind"]
    if kind in ("route", "route_backward", "layer"):
        T, E, k, b = c["T"], c["E"], c["k"], BYTES[c["type"]]
        routed = T * E * b + T * k * 8 + (E * 4 if c["bias"] else 0)
    if kind == "route":
        return dict(bytes=routed + T * k * 8 + E * 4, flops=10 * T * E)
    if kind == "route_backward":
        return dict(bytes=2 * T * E * b + T * k * 8, flops=10 * T * E)
    if kind in ("product", "linear", "experts"):
        M, N, K, o = c["M"], c["N"], c["K"], BYTES[c["out"]]
        x = M * K * (BYTES[c["type"]] if kind == "linear" else 1)
        used = min(c["E"], M) if kind == "experts" else 1
        return dict(bytes=x + used * N * (K + 4) + 4 * M + M * N * o, flops=2.0 * M * N * K)
    if kind in ("combine", "combine_backward"):
        T, k, N, b = c["T"] - c["padded"], c["k"], c["N"], BYTES[c["type"]]
        if kind == "combine":
            return dict(bytes=T * k * N * b + c["T"] * N * b + c["T"] * k * 8, flops=2 * T * k * N)
        return dict(bytes=2 * T * k * N * b + T * N * b + c["T"] * k * 12, flops=3 * T * k * N)
    H, F, used = c["H"], c["F"], min(E, T * k)
    return dict(bytes=routed + 4 * T * H + used * (3 * F * H + 8 * F + 4 * H), flops=6.0 * T * k * F * H)


def _route64(logits, bias, c):
    x = logits.double()
    s, _ = _choice64(logits, bias, c)
    s = torch.nan_to_num(s)
    by = s + bias.double() if bias is not None else x
    groups = s + bias.double() if bias is not None else s
    T, E = x.shape
    per = E // c["groups"]
    if c["groups"] > 1:
        t = groups.view(T, c["groups"], per).topk(min(c["top"], per), -1).values.sum(-1)
        cut = t.sort(dim=-1, descending=True, stable=True).indices[:, c["kept"]:]
        out = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV)
        out[torch.arange(T, device=DEV)[:, None], cut] = True
        by = by.masked_fill(out[:, :, None].expand(T, c["groups"], per).reshape(T, E), -math.inf)
    ids = by.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    masked = (x == -math.inf).all(-1, keepdim=True)
    return (w * 2.5).masked_fill(masked, 0.0), ids.masked_fill(masked, -1)


def _order64(ids, E):
    key = ids.flatten().tolist()
    rows = [[] for _ in range(E)]
    for p, e in enumerate(key):
        if e >= 0:
            rows[e].append(p)
    flat = [p for r in rows for p in r]
    ends = [0]
    for r in rows:
        ends.append(ends[-1] + len(r))
    slots = [-1] * len(key)
    for i, p in enumerate(flat):
        slots[p] = i
    tokens = [p // ids.shape[1] for p in flat] + [-1] * (len(key) - len(flat))
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return t(ends), t(slots).view(ids.shape), t(tokens)


def _rows64(x):
    x = x.double()
    scale = x.abs().amax(-1, keepdim=True) / 127
    return torch.round(x / scale.clamp(min=1e-300)), scale


def _experts64(q, sa, ends, B, sb, K):
    y = torch.zeros(q.shape[0], B.shape[1], dtype=torch.float64, device=DEV)
    for e in range(B.shape[0]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            y[a:b] = (q[a:b].double() @ B[e, :, :K].double().t()) * sa[a:b].double() * sb[e].double()
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "route":
        w, ids = _route64(s["logits"], s["bias"], c)
        offsets, slots, tokens = _order64(ids, c["E"])
        return dict(weights=w, ids=ids.to(torch.int32), offsets=offsets, slots=slots, tokens=tokens)
    if kind == "route_backward":
        x = s["logits"].double().masked_fill((s["logits"] == -math.inf).all(-1, keepdim=True), 0.0).requires_grad_()
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
        live = (s["ids"] >= 0).double()
        w = p.gather(1, s["ids"].long().clamp(min=0)) * live
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        (w * 2.5 * live * s["dweights"].double()).sum().backward()
        return dict(dlogits=x.grad)
    if kind in ("product", "linear"):
        if kind == "linear":
            q, sa = _rows64(s["X"])
        else:
            q, sa = s["A"][:, :c["K"]].double(), s["sa"].double()[:, None]
        return dict(D=(q @ s["B"][:, :c["K"]].double().t()) * sa * s["sb"].double())
    if kind == "experts":
        ends = s["offsets"].tolist()
        return dict(D=_experts64(s["A"][:, :c["K"]], s["sa"][:, None], ends, s["B"], s["sb"], c["K"]))
    if kind in ("combine", "combine_backward"):
        T, k, N = c["T"], c["k"], c["N"]
        D, dw = torch.zeros(T, N, dtype=torch.float64, device=DEV), torch.zeros(T, k, dtype=torch.float64, device=DEV)
        dy = torch.zeros(T * k, N, dtype=torch.float64, device=DEV)
        for j in range(k):
            t = torch.nonzero(s["slots"][:, j] >= 0).flatten()
            r = s["slots"][t, j].long()
            w = s["weights"][t, j].double()[:, None]
            if kind == "combine":
                D[t] += w * s["Y"][r].double()
            else:
                dy[r] = w * s["dD"][t].double()
                dw[t, j] = (s["dD"][t].double() * s["Y"][r].double()).sum(-1)
        return dict(D=D) if kind == "combine" else dict(dY=dy, dweights=dw)
    w, ids = _route64(s["logits"], s["bias"], c)
    offsets, slots, tokens = _order64(ids, c["E"])
    ends = offsets.tolist()
    q, sa = _rows64(s["X"][tokens.long()])
    y = _experts64(q, sa, ends, s["B1"], s["sb1"], c["H"])
    gate, up = y[:, :c["F"]], y[:, c["F"]:]
    q, sa = _rows64(gate * torch.sigmoid(gate) * up)
    y = _experts64(q, sa, ends, s["B2"], s["sb2"], c["F"])
    D = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
    for j in range(c["k"]):
        D += w[:, j:j + 1] * y[slots[:, j].long()]
    return dict(D=D, ids=ids.to(torch.int32))
