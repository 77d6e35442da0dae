"""What the operators at the two ends of a training step, and its routers' balance loss, are measured on.

Three operators with their gradients: the softmax cross entropy of a linear head over a large vocabulary, whose logits
are never kept; a router's balance loss with its counts per expert; the rows of a token table times a factor, whose
gradient is summed by token. The head and the table may be the same matrix.

``run`` computes them in elementary torch operations in 32 bits, or, with ``own``, through the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1), "f16": (torch.float16, 2)}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
LARGEST = 8.0 * 8192 * 131072 * 2048  # operations of the largest step


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the probability of one token: latency and the reading of the head's weights
        dict(name="score_token", kind="loss", T=1, V=131072, K=4096, masked=0.0, type="bf16"),
        # a few scored continuations, odd in every direction
        dict(name="score_odd", kind="loss", T=77, V=50001, K=2001, masked=0.2, type="f16"),
        # the loss of a batch that is only evaluated
        dict(name="loss_prompt", kind="loss", T=8192, V=65536, K=4096, masked=0.1, type="bf16"),
        # the gradients of a micro batch, with a penalty on the normaliser
        dict(name="loss_backward", kind="loss_backward", T=4096, V=32768, K=4096, masked=0.0, type="bf16", z=True),
        # a fine-tuning batch, a third of whose tokens carry no loss, odd in every direction
        dict(name="loss_backward_odd", kind="loss_backward", T=777, V=50001, K=1001, masked=0.34, type="f16", z=False),
        # loss and gradients of a training step
        dict(name="loss_step", kind="loss_step", T=8192, V=131072, K=2048, masked=0.05, type="bf16"),
        # the balance loss of a training step: many experts, sigmoid scores, all tokens together
        dict(name="balance", kind="balance", T=16384, E=256, k=8, score="sigmoid", S=1, padded=0, type="f32"),
        # its gradient for each of a few ragged sequences, with padded tokens behind the last
        dict(name="balance_backward", kind="balance_backward", T=16384, E=64, k=6, score="softmax", S=7, padded=515,
             type="bf16"),
        # the table's rows of a decode step
        dict(name="embed_token", kind="embed", T=16, V=131072, N=4096, padded=0, type="bf16", out="bf16"),
        # the table's rows of a batch, kept in 32 bits
        dict(name="embed_prompt", kind="embed", T=8192, V=65536, N=4096, padded=100, type="bf16", out="f32"),
        # the table's gradient, written whole: tokens repeat as they do in text
        dict(name="embed_backward", kind="embed_backward", T=16384, V=32768, N=2048, padded=100, type="bf16", out="bf16"),
        # all of them around an expert model with a tied table: rows, balance loss, head's loss, and back
        dict(name="ends", kind="ends", T=2048, V=32768, K=1024, E=64, k=6, score="softmax", S=4, padded=48, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    return {"loss": 2.0, "loss_backward": 6.0, "loss_step": 8.0, "ends": 8.0}[c["kind"]] * c["T"] * c["V"] * c["K"]


def draw(rng):
    kind = rng.choice(["loss", "loss", "loss_backward", "loss_backward", "loss_step", "balance", "balance_backward", "embed",
                       "embed_backward", "embed_backward", "ends"])
    if kind in ("loss", "loss_backward", "loss_step"):
        while True:
            c = dict(kind=kind, T=_log(rng, 1, 8192), V=_log(rng, 1000, 131072), K=_log(rng, 64, 4096),
                     masked=rng.choice([0.0, 0.05, 0.4]), type=rng.choice(["bf16", "f16"]))
            if _cost(c) <= LARGEST / 2:
                break
        return dict(c, z=rng.random() < 0.5) if kind == "loss_backward" else c
    if kind in ("balance", "balance_backward"):
        T = _log(rng, 1, 16384)
        E = rng.choice([8, 16, 60, 64, 72, 128, 160, 256, 384])
        return dict(kind=kind, T=T, E=E, k=rng.randint(1, min(10, E)), score=rng.choice(["softmax", "sigmoid"]),
                    S=rng.choice([1, 1, 2, 5, 16]), padded=rng.choice([0, T // 9]), type=rng.choice(["f32", "bf16", "f16"]))
    if kind == "embed":
        T = _log(rng, 1, 8192)
        return dict(kind=kind, T=T, V=_log(rng, 1000, 65536), N=_log(rng, 64, 4096), padded=rng.choice([0, T // 9]),
                    type=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]))
    if kind == "embed_backward":
        T = _log(rng, 1, 16384)
        return dict(kind=kind, T=T, V=_log(rng, 1000, 32768), N=_log(rng, 64, 2048), padded=rng.choice([0, T // 9]),
                    type=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]))
    T = _log(rng, 8, 2048)
    E = rng.choice([8, 60, 64, 128])
    return dict(kind=kind, T=T, V=_log(rng, 1000, 32768), K=_log(rng, 64, 1024), E=E, k=rng.randint(1, 8),
                score=rng.choice(["softmax", "sigmoid"]), S=rng.choice([1, 3, 4]), padded=rng.choice([0, T // 9]),
                type=rng.choice(["bf16", "f16"]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rows(n, width, type):
    """Rows that start on 16-byte words, as the library's leading dimensions are."""
    ld = -(-width // 8) * 8
    return torch.empty(n, ld, dtype=TYPES[type][0], device=DEV)[:, :width]


def _room(n):
    return torch.empty(int(n), dtype=torch.uint8, device=DEV)


def _tokens(g, T, V, padded):
    """Token ids as frequent as words are (the r-th most frequent one about 1 / r), -1 for padded places at the end."""
    r = (torch.rand(T, generator=g, device=DEV, dtype=torch.float64) * math.log(V)).exp().long() - 1
    ids = torch.randperm(V, generator=g, device=DEV)[r.clamp_(0, V - 1)].to(torch.int32)
    if padded:
        ids[T - padded:] = -1
    return ids


def _table(g, V, K, type):
    """A head's weights: logits of rows of unit variance have a deviation of about 2."""
    w = _rows(V, K, type)
    for a in range(0, V, 16384):
        b = min(V, a + 16384)
        w[a:b] = torch.randn(b - a, K, generator=g, device=DEV) * (2.0 / math.sqrt(K))
    return w


def _hidden(g, W, targets, T, K, type):
    """Rows that know something of their targets: those get between 0 and 12 more than the other logits."""
    x = torch.randn(T, K, generator=g, device=DEV)
    at = targets.clamp(min=0).long()
    x += W[at].float() * (torch.rand(T, 1, generator=g, device=DEV) * 3.0)
    out = _rows(T, K, type)
    out.copy_(x)
    return out


def _targets(g, c):
    y = _tokens(g, c["T"], c["V"], 0)
    y[torch.rand(c["T"], generator=g, device=DEV) < c["masked"]] = -100
    return y


def _head(s, g, c, targets, W=None):
    T, V, K = c["T"], c["V"], c["K"]
    s["W"] = _table(g, V, K, c["type"]) if W is None else W
    s["targets"] = targets
    s["X"] = _hidden(g, s["W"], targets, T, K, c["type"])
    live = (targets >= 0).float()
    s["dlosses"] = live / live.sum().clamp(min=1.0)
    s["dlse"] = None
    s["losses"], s["lse"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    s["workspace"] = _room(T * V // 8 + (1 << 20))
    if c["kind"] != "loss":
        s["dX"], s["dW"] = _rows(T, K, c["type"]), _rows(V, K, c["type"])
        s["back"] = _room((320 << 20) + 16 * T * K + 2 * T * min(V + 256, 32768))


def _router(s, g, c):
    """A router's logits, the ids that it chose (-1 for padded tokens) and the ends of its sequences."""
    T, E, S = c["T"], c["E"], c["S"]
    x = torch.randn(T, E, generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV) * 0.5
    ids = x.argsort(-1, descending=True)[:, :c["k"]].to(torch.int32).contiguous()
    live = T - c["padded"]
    if c["padded"]:
        x[live:] = -math.inf
        ids[live:] = -1
    s["logits"], s["ids"] = x.to(TYPES[c["type"]][0]), ids
    cuts = torch.rand(S - 1, generator=g, device=DEV).mul(live).long().sort().values
    ends = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), live)])
    s["offsets"] = ends.to(torch.int32)
    s["counts"] = torch.empty(S, E, dtype=torch.int32, device=DEV)
    s["tokens"] = torch.empty(S, dtype=torch.int32, device=DEV)
    s["means"], s["balance"] = torch.empty(S, E, device=DEV), torch.empty(S, device=DEV)
    s["dbalance"] = torch.full((S,), 0.01 / S, device=DEV)
    s["dlogits"] = torch.zeros_like(s["logits"])
    s["router_room"] = _room(16 << 20)


def prepare(case, seed):
    c, g = case, _gen(seed)
    kind = c["kind"]
    s = dict(case=c)
    if kind in ("loss", "loss_backward", "loss_step"):
        _head(s, g, c, _targets(g, c))
    if kind == "loss_backward":
        s["losses"], s["lse"] = _loss(s)
        if c["z"]:
            s["dlse"] = 2e-4 * s["lse"] * s["dlosses"]
    if kind in ("balance", "balance_backward", "ends"):
        _router(s, g, c)
    if kind == "balance_backward":
        s["counts"], s["tokens"], s["means"], s["balance"] = _balance(s)
    if kind in ("embed", "embed_backward", "ends"):
        T, V, N = c["T"], c["V"], c["K"] if kind == "ends" else c["N"]
        s["scale"] = math.sqrt(N)
        s["words"] = _tokens(g, T, V, c["padded"])
        out = c["type"] if kind == "ends" else c["out"]
        s["rows"] = torch.empty(T, N, dtype=TYPES[out][0], device=DEV)
        if kind == "embed":
            s["table"] = (torch.randn(V, N, generator=g, device=DEV) * 0.02).to(TYPES[c["type"]][0])
        else:
            s["drows"] = (torch.randn(T, N, generator=g, device=DEV) * 0.1).to(TYPES[out][0])
            s["dtable"] = torch.empty(V, N, dtype=TYPES[c["type"]][0], device=DEV) if kind == "embed_backward" else None
            s["sums_room"] = _room((8 << 20) + 64 * T + 2 * T * N)
    if kind == "ends":
        targets = s["words"].roll(-1).clamp(min=-1)
        targets[-1] = -1
        _head(s, g, c, targets)
    return s


# ------------------------------------------------------------------ plain forms

def _loss(s):
    y = s["targets"]
    l = s["X"].float() @ s["W"].float().t()  # noqa: E741
    top = l.amax(-1)
    top = torch.where(top.abs() == math.inf, torch.zeros_like(top), top)
    lse = torch.log(torch.exp(l - top[:, None]).sum(-1)) + top
    none = (y < 0) | (y >= s["W"].shape[0])
    at = torch.where(none, torch.zeros_like(y), y).long()
    losses = lse - l.gather(1, at[:, None])[:, 0]
    return torch.where(none, torch.zeros_like(lse), losses), torch.where(none, torch.zeros_like(lse), lse)


def _loss_grad(s, lse):
    y = s["targets"]
    x, w = s["X"].float(), s["W"].float()
    none = (y < 0) | (y >= w.shape[0])
    at = torch.where(none, torch.zeros_like(y), y).long()
    d1 = torch.where(none, torch.zeros_like(lse), s["dlosses"])
    total = d1 if s["dlse"] is None else d1 + torch.where(none, torch.zeros_like(lse), s["dlse"])
    d = torch.exp(x @ w.t() - lse[:, None]) * total[:, None]
    d[torch.arange(y.numel(), device=DEV), at] -= d1
    d = torch.where(none[:, None], torch.zeros_like(d), d)
    return (d @ w).to(s["X"].dtype), (d.t() @ x).to(s["W"].dtype)


def _scores(s, c):
    x = s["logits"].float()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p, total, p / torch.where(total == 0, torch.ones_like(total), total)


def _sequences(s, c):
    """The sequence of each token (S where it has none, or where none of its ids is an expert's)."""
    t = torch.arange(c["T"], device=DEV)
    of = (t[:, None] >= s["offsets"][None, 1:]).sum(-1)
    live = ((s["ids"] >= 0) & (s["ids"] < c["E"])).any(-1) & (t >= s["offsets"][0])
    return torch.where(live, of, torch.full_like(of, c["S"]))


def _balance(s):
    c = s["case"]
    E, S, k = c["E"], c["S"], c["k"]
    of = _sequences(s, c)
    p = _scores(s, c)[2]
    tokens = (of[:, None] == torch.arange(S, device=DEV)).sum(0)
    ids = s["ids"].long()
    pair = torch.where((ids >= 0) & (of[:, None] < S), of[:, None] * E + ids, torch.full_like(ids, S * E)).flatten()
    counts = torch.zeros(S * E + 1, dtype=torch.int64, device=DEV).index_add_(0, pair, torch.ones_like(pair))[:-1].view(S, E)
    sums = torch.zeros(S + 1, E, device=DEV).index_add_(0, of, p)[:S]
    n = tokens.clamp(min=1).float()[:, None]
    means = sums / n
    losses = E * (counts.float() / (k * n) * means).sum(-1)
    return counts.to(torch.int32), tokens.to(torch.int32), means, losses


def _balance_grad(s, counts, tokens):
    c = s["case"]
    E, S, k = c["E"], c["S"], c["k"]
    of = _sequences(s, c)
    n = tokens.clamp(min=1).float()[:, None]
    by = s["dbalance"][:, None] * E * counts.float() / (k * n) / n
    by = torch.cat([by, by.new_zeros(1, E)])[of]
    score, total, p = _scores(s, c)
    d = by - (p * by).sum(-1, keepdim=True)
    d = d * (score * (1.0 - score) / torch.where(total == 0, torch.ones_like(total), total) if c["score"] == "sigmoid" else p)
    return d.to(s["logits"].dtype)


def _embed(s, table):
    ids = s["words"]
    none = (ids < 0) | (ids >= table.shape[0])
    rows = table[torch.where(none, torch.zeros_like(ids), ids).long()].float() * s["scale"]
    return torch.where(none[:, None], torch.zeros_like(rows), rows).to(s["rows"].dtype)


def _embed_grad(s, V):
    ids = s["words"]
    at = torch.where((ids < 0) | (ids >= V), torch.full_like(ids, V), ids).long()
    d = torch.zeros(V + 1, s["drows"].shape[1], device=DEV)
    return d.index_add_(0, at, s["drows"].float())[:V] * s["scale"]


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "loss":
        losses, lse = _loss(s)
        return dict(losses=losses, lse=lse)
    if kind == "loss_backward":
        dx, dw = _loss_grad(s, s["lse"])
        return dict(dX=dx, dW=dw)
    if kind == "loss_step":
        losses, lse = _loss(s)
        dx, dw = _loss_grad(s, lse)
        return dict(losses=losses, dX=dx, dW=dw)
    if kind == "balance":
        counts, tokens, means, losses = _balance(s)
        return dict(counts=counts, tokens=tokens, means=means, losses=losses)
    if kind == "balance_backward":
        return dict(dlogits=_balance_grad(s, s["counts"], s["tokens"]))
    if kind == "embed":
        return dict(rows=_embed(s, s["table"]))
    if kind == "embed_backward":
        return dict(dtable=_embed_grad(s, c["V"]).to(s["dtable"].dtype))
    rows = _embed(s, s["W"])
    counts, tokens, _, balance = _balance(s)
    losses, lse = _loss(s)
    dx, dw = _loss_grad(s, lse)
    # the head's gradient is a gradient of its own, rounded, before the table's rows are added to it
    dw = (dw.float() + _embed_grad(s, c["V"])).to(dw.dtype)
    return dict(rows=rows, losses=losses, balance=balance, dX=dx, dW=dw, dlogits=_balance_grad(s, counts, tokens))


# ------------------------------------------------------------------ the library

def _library(s):
    import smem_swizzle_layouts_gb300 as G
    c = s["case"]
    kind, code = c["kind"], TYPES[c["type"]][1]
    T = c["T"]
    if kind in ("embed", "ends"):
        table = s["table"] if kind == "embed" else s["W"]
        rows = s["rows"]
        G.gemm_embed(T, rows.shape[1], c["V"], s["words"], table, code, table.stride(0), s["scale"], rows,
                     TYPES[c["out"]][1] if kind == "embed" else code, rows.stride(0))
        if kind == "embed":
            return dict(rows=rows)
    if kind in ("balance", "ends"):
        rule = dict(score=G.ROUTE_SIGMOID if c["score"] == "sigmoid" else G.ROUTE_SOFTMAX)
        G.gemm_route_balance(T, c["E"], s["logits"], code, c["E"], c["k"], rule, s["ids"], c["S"], s["offsets"], s["counts"],
                             s["tokens"], s["means"], s["balance"], s["router_room"], s["router_room"].numel())
        if kind == "balance":
            return dict(counts=s["counts"], tokens=s["tokens"], means=s["means"], losses=s["balance"])
    if kind in ("loss", "loss_step", "ends"):
        G.gemm_cross_entropy(code % 2, T, c["V"], c["K"], s["X"], s["X"].stride(0), s["W"], s["W"].stride(0), s["targets"],
                             s["losses"], s["lse"], s["workspace"], s["workspace"].numel())
        if kind == "loss":
            return dict(losses=s["losses"], lse=s["lse"])
    if kind in ("loss_backward", "loss_step", "ends"):
        G.gemm_cross_entropy_backward(code % 2, T, c["V"], c["K"], s["X"], s["X"].stride(0), s["W"], s["W"].stride(0),
                                      s["targets"], s["lse"], s["dlosses"], s["dlse"], s["dX"], code, s["dX"].stride(0),
                                      s["dW"], code, s["dW"].stride(0), 0, s["back"], s["back"].numel())
        if kind == "loss_backward":
            return dict(dX=s["dX"], dW=s["dW"])
        if kind == "loss_step":
            return dict(losses=s["losses"], dX=s["dX"], dW=s["dW"])
    if kind in ("embed_backward", "ends"):
        d, table = s["drows"], s["dW"] if kind == "ends" else s["dtable"]
        G.gemm_embed_backward(T, d.shape[1], c["V"], s["words"], d, code if kind == "ends" else TYPES[c["out"]][1], d.stride(0),
                              s["scale"], table, code, table.stride(0), int(kind == "ends"), s["sums_room"],
                              s["sums_room"].numel())
        if kind == "embed_backward":
            return dict(dtable=table)
    rule = dict(score=G.ROUTE_SIGMOID if c["score"] == "sigmoid" else G.ROUTE_SOFTMAX)
    G.gemm_route_balance_backward(T, c["E"], s["logits"], code, c["E"], c["k"], rule, s["ids"], c["S"], s["offsets"],
                                  s["counts"], s["tokens"], s["dbalance"], s["dlogits"], c["E"], 0)
    if kind == "balance_backward":
        return dict(dlogits=s["dlogits"])
    return dict(rows=s["rows"], losses=s["losses"], balance=s["balance"], dX=s["dX"], dW=s["dW"], dlogits=s["dlogits"])


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------ work and the values in 64 bits

def work(case):
    c = case
    kind, T, b = c["kind"], c["T"], BYTES[c["type"]]
    if kind in ("loss", "loss_backward", "loss_step", "ends"):
        V, K = c["V"], c["K"]
        head = (T + V) * K * b
    if kind == "loss":
        return dict(bytes=head + 12 * T, flops=2.0 * T * V * K)
    if kind in ("loss_backward", "loss_step"):
        return dict(bytes=2 * head + 16 * T, flops=6.0 * T * V * K)
    if kind in ("balance", "balance_backward", "ends"):
        E, S = c["E"], c["S"]
        router = T * E * b + T * c["k"] * 4 + 8 * S * E
    if kind == "balance":
        return dict(bytes=router, flops=8.0 * T * E)
    if kind == "balance_backward":
        return dict(bytes=router + T * E * b, flops=10.0 * T * E)
    if kind == "ends":
        rows = T * K * b
        return dict(bytes=2 * head + 2 * router + T * E * b + 3 * rows + min(T, V) * K * b, flops=6.0 * T * V * K)
    V, N, o = c["V"], c["N"], BYTES[c["out"]]
    live = T - c["padded"]
    if kind == "embed":
        return dict(bytes=4 * T + min(live, V) * N * b + T * N * o, flops=T * N)
    return dict(bytes=4 * T + live * N * o + V * N * b, flops=T * N)


def _loss64(s):
    V = s["W"].shape[0]
    l = s["X"].double() @ s["W"].double().t()  # noqa: E741
    live = (s["targets"] >= 0) & (s["targets"] < V)
    lse = torch.logsumexp(l, -1)
    losses = lse - l[torch.arange(l.shape[0], device=DEV), s["targets"].long().clamp(0, V - 1)]
    return losses * live, lse * live


def _loss_grad64(s, lse):
    """Gradients of sum(dlosses * losses + dlse * lse) at the given normalisers."""
    V = s["W"].shape[0]
    x, w = s["X"].double(), s["W"].double()
    live = (s["targets"] >= 0) & (s["targets"] < V)
    a = s["dlosses"].double() * live
    z = torch.zeros_like(a) if s["dlse"] is None else s["dlse"].double() * live
    p = (x @ w.t()).sub_(lse.double()[:, None]).exp_().mul_((a + z)[:, None])
    y = s["targets"].long().clamp(0, V - 1)
    p.scatter_add_(1, y[:, None], -a[:, None])
    return p @ w, p.t() @ x


def _scores64(s, c):
    x = s["logits"].double()
    x = x.masked_fill((x == -math.inf).all(-1, keepdim=True), 0.0).requires_grad_()
    if c["score"] == "softmax":
        return x, torch.softmax(x, -1)
    p = torch.sigmoid(x)
    return x, p / p.sum(-1, keepdim=True)


def _balance64(s):
    """Counts, live tokens, mean scores and losses of each sequence, the scores differentiable in the logits."""
    c = s["case"]
    E, k = c["E"], c["k"]
    x, p = _scores64(s, c)
    ends = s["offsets"].tolist()
    counts, tokens, means, losses = [], [], [], []
    for a, b in zip(ends[:-1], ends[1:]):
        ids = s["ids"][a:b]
        live = (ids >= 0).any(-1)
        n = int(live.sum())
        of = torch.bincount(ids[ids >= 0].long().flatten(), minlength=E)
        mean = p[a:b][live].sum(0) / max(n, 1)
        counts.append(of)
        tokens.append(n)
        means.append(mean)
        losses.append(E * (of.double() / (k * max(n, 1)) * mean).sum())
    return x, torch.stack(counts).to(torch.int32), torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.stack(means), torch.stack(losses)


def _embed_grad64(s, V):
    ids = s["words"].long()
    live = (ids >= 0) & (ids < V)
    d = torch.zeros(V, s["drows"].shape[1], dtype=torch.float64, device=DEV)
    return d.index_put_((ids[live],), s["drows"][live].double(), accumulate=True).mul_(float(torch.tensor(s["scale"])))


def _embed64(s, table):
    ids = s["words"].long()
    live = (ids >= 0) & (ids < table.shape[0])
    out = torch.zeros(ids.numel(), table.shape[1], dtype=torch.float64, device=DEV)
    out[live] = table[ids[live]].double() * float(torch.tensor(s["scale"]))
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "loss":
        losses, lse = _loss64(s)
        return dict(losses=losses, lse=lse)
    if kind == "loss_backward":
        dx, dw = _loss_grad64(s, s["lse"])
        return dict(dX=dx, dW=dw)
    if kind == "loss_step":
        losses, lse = _loss64(s)
        dx, dw = _loss_grad64(s, lse)
        return dict(losses=losses, dX=dx, dW=dw)
    if kind in ("balance", "balance_backward", "ends"):
        x, counts, tokens, means, losses = _balance64(s)
        if kind == "balance":
            return dict(counts=counts, tokens=tokens, means=means.detach(), losses=losses.detach())
        (losses * s["dbalance"].double()).sum().backward()
        if kind == "balance_backward":
            return dict(dlogits=x.grad)
    if kind == "embed":
        return dict(rows=_embed64(s, s["table"]))
    if kind == "embed_backward":
        return dict(dtable=_embed_grad64(s, c["V"]))
    head, lse = _loss64(s)
    dx, dw = _loss_grad64(s, lse)
    return dict(rows=_embed64(s, s["W"]), losses=head, balance=losses.detach(), dX=dx, dW=dw + _embed_grad64(s, c["V"]),
                dlogits=x.grad)
