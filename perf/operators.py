"""The layer operators as timed cases: expert routing with scores, layer norm, token embedding and the
distillation head, each forward and, in training, with its gradients.

`run` makes the library's calls where `own` is true; where it is false it computes the same results with
elementary torch operations (fp32; fp64 where the choice of an expert hangs on neighbouring scores).
`exact` is the definition in fp64.
"""
import math

import torch

own = False

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = {"bf16": BF16, "fp16": FP16, "fp32": FP32}


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch of 8 sequences: grouped sigmoid routing, latency only
        dict(name="route decode", op="route", N=8, E=64, k=8, groups=8, topk_groups=4, score="sigmoid", bias=True,
             renormalize=True, scale=2.5, type="fp32", train=False),
        # a training batch of a 64-expert layer: softmax, no groups, bf16 logits from a bf16 projection
        dict(name="route 64 experts", op="route", N=16384, E=64, k=8, groups=1, topk_groups=1, score="softmax",
             bias=False, renormalize=True, scale=1.0, type="bf16", train=True),
        # a training batch of a 384-expert layer: sigmoid, balance bias, 4 of 8 groups
        dict(name="route 384 experts", op="route", N=32768, E=384, k=8, groups=8, topk_groups=4, score="sigmoid",
             bias=True, renormalize=True, scale=2.5, type="fp32", train=True),
        # a decode step's norm: 16 rows
        dict(name="norm decode", op="norm", N=16, H=2048, type="bf16", params="bf16", train=False),
        # an odd width in fp32, a ragged batch: nothing is a multiple of a vector
        dict(name="norm odd width", op="norm", N=4099, H=1001, type="fp32", params="fp32", train=True),
        # a full training batch at the widest hidden size, fp32 parameters
        dict(name="norm wide", op="norm", N=32768, H=7168, type="bf16", params="fp32", train=True),
        # a prompt's lookup: no gradient
        dict(name="embed prompt", op="embed", N=1000, V=32000, H=2048, scale=1.0, type="bf16", ids="int64",
             train=False, add=False),
        # gradient added into an existing one (tied head, gradient accumulation): touched rows only
        dict(name="embed add", op="embed", N=16384, V=32000, H=2048, scale=45.25, type="bf16", ids="int32",
             train=True, add=True),
        # the largest vocabulary, a dense gradient
        dict(name="embed dense", op="embed", N=32768, V=200000, H=4096, scale=1.0, type="bf16", ids="int64",
             train=True, add=False),
        # a small head, every size ragged
        dict(name="distill small", op="distill", N=300, H=128, V=1000, K=8, P=3, tau=1.0, train=True),
        # one micro-batch against 32,000 classes
        dict(name="distill mid", op="distill", N=2048, H=1024, V=32000, K=32, P=4, tau=2.0, train=True),
        # a full batch: 64 teacher logits per token
        dict(name="distill large", op="distill", N=8192, H=4096, V=65536, K=64, P=4, tau=2.0, train=True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "embed", "distill"])
    train = rng.random() < 0.7
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        groups = rng.choice([1, 1, 2, 4, 8]) if E % 8 == 0 else rng.choice([1, 2, 4])
        topk_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(8, topk_groups * (E // groups)))
        return dict(op=op, N=_spread(rng, 1, 32768), E=E, k=k, groups=groups, topk_groups=topk_groups,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    type=rng.choice(["fp32", "fp32", "bf16"]), train=train)
    if op == "norm":
        H = rng.choice([_spread(rng, 64, 8192) | 1, 64 * _spread(rng, 1, 40), 4096, 7168])
        t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = min(32768, 32768 * 7168 // (H * (2 if t == "fp32" else 1)))
        return dict(op=op, N=_spread(rng, 1, most), H=H, type=t, params=rng.choice(["fp32", t]), train=train)
    if op == "embed":
        H = rng.choice([_spread(rng, 64, 4096) | 1, 64 * _spread(rng, 1, 40), 4096])
        V = _spread(rng, 500, 200000)
        return dict(op=op, N=_spread(rng, 1, 32768), V=V, H=H, scale=rng.choice([1.0, round(math.sqrt(H), 2)]),
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]) if H * V < 2 ** 28 else "bf16",
                    ids=rng.choice(["int32", "int64"]), train=train, add=train and rng.random() < 0.5)
    H = rng.choice([64 * _spread(rng, 1, 40), 64 * _spread(rng, 1, 40), 4096])
    V = _spread(rng, 300, 65536)
    return dict(op=op, N=_spread(rng, 1, 8192), H=H, V=V, K=rng.choice([1, 4, 10, 32, 64]), P=rng.randint(1, 4),
                tau=rng.choice([1.0, 2.0, 4.0]), train=train)


def work(c):
    """Bytes and operations of one pass: every input read once, every output written once."""
    train = c["train"]
    if c["op"] == "route":
        b = TYPES[c["type"]].itemsize
        N, E, k = c["N"], c["E"], c["k"]
        nbytes, flops = N * E * b + N * k * 8 + E * 4 + (E * 4 if c["bias"] else 0), 4 * N * E
        if train:   # the chosen logits again (all of them where the softmax is not renormalised), dw, idx
            nbytes += N * E * b + N * k * 8 + (N * E * b if c["score"] == "softmax" and not c["renormalize"]
                                               else N * k * b)
            flops += 10 * N * k
        return dict(bytes=nbytes, flops=flops)
    if c["op"] == "norm":
        N, H, b, pb = c["N"], c["H"], TYPES[c["type"]].itemsize, TYPES[c["params"]].itemsize
        nbytes, flops = 2 * N * H * b + 2 * H * pb + 8 * N, 8 * N * H
        if train:
            nbytes += 3 * N * H * b + H * pb + 8 * N + 8 * H
            flops += 14 * N * H
        return dict(bytes=nbytes, flops=flops)
    if c["op"] == "embed":
        N, V, H, b = c["N"], c["V"], c["H"], TYPES[c["type"]].itemsize
        ib = 8 if c["ids"] == "int64" else 4
        nbytes, flops = N * ib + 2 * N * H * b, N * H
        if train:   # distinct tokens of N draws whose frequency falls as 1 / rank
            u = min(V, N) if not c["add"] else int(sum(1 - (1 - math.log1p(1 / r) / math.log(V + 1)) ** N
                                                       for r in range(1, V + 1)))
            nbytes += N * ib + N * H * b + (2 * u * H * 4 if c["add"] else V * H * 4)
            flops += 2 * N * H
        return dict(bytes=nbytes, flops=flops)
    N, H, V, K = c["N"], c["H"], c["V"], c["K"]
    nbytes, flops = 2 * (N * H + V * H) + 8 * N * K + 8 * N + 4, 2 * N * H * V
    if train:   # X, W, the teacher, lse, dloss again; dX and dW out; the logits again and two products
        nbytes += 2 * (N * H + V * H) + 8 * N * K + 8 * N + 2 * (N * H + V * H)
        flops *= 4
    return dict(bytes=nbytes, flops=flops)


# ------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, type=FP32):
        return (torch.randn(*shape, device="cuda", generator=g) * std + mean).to(type)

    s = dict(c)
    if c["op"] == "route":
        s["logits"] = normal(c["N"], c["E"], std=1.5, type=TYPES[c["type"]])
        s["b"] = normal(c["E"], std=0.05) if c["bias"] else None
        s["dw"] = normal(c["N"], c["k"])
    elif c["op"] == "norm":
        t, pt = TYPES[c["type"]], TYPES[c["params"]]
        s["x"] = normal(c["N"], c["H"], std=2.0, mean=0.5, type=t)
        s["weight"], s["b"] = normal(c["H"], std=0.2, mean=1.0, type=pt), normal(c["H"], std=0.2, type=pt)
        s["dy"] = normal(c["N"], c["H"], type=t)
    elif c["op"] == "embed":
        t = TYPES[c["type"]]
        s["table"] = torch.empty(c["V"], c["H"], device="cuda", dtype=t).normal_(0, 0.02, generator=g)
        u = torch.rand(c["N"], device="cuda", generator=g, dtype=torch.float64)
        rank = (torch.exp(u * math.log(c["V"] + 1)) - 1).long().clamp_(0, c["V"] - 1)
        name = torch.randperm(c["V"], device="cuda", generator=g)
        s["tokens"] = name[rank].to(torch.int64 if c["ids"] == "int64" else torch.int32)
        s["dy"] = normal(c["N"], c["H"], type=t)
        if c["add"]:
            s["grad"] = normal(c["V"], c["H"], std=0.1)
    else:
        s["X"] = normal(c["N"], c["H"], type=BF16)
        s["W"] = normal(c["V"], c["H"], std=2.0 / math.sqrt(c["H"]), type=BF16)
        # K different classes a row: K places of the vocabulary's K-th parts
        part = c["V"] // c["K"]
        at = torch.randint(0, part, (c["N"], c["K"]), device="cuda", generator=g)
        at = at + torch.arange(c["K"], device="cuda") * part
        order = torch.rand(c["N"], c["K"], device="cuda", generator=g).argsort(dim=1)
        s["t_idx"] = at.gather(1, order).to(torch.int32).contiguous()
        s["t_logits"] = normal(c["N"], c["K"], std=2.0).sort(dim=1, descending=True).values.contiguous()
        # some rows come with fewer entries, a few with none
        few = torch.rand(c["N"], 1, device="cuda", generator=g)
        keep = torch.where(few < 0.02, 0, torch.where(few < 0.2, (c["K"] + 1) // 2, c["K"]))
        s["t_idx"].masked_fill_(torch.arange(c["K"], device="cuda") >= keep, -1)
        s["dloss"] = torch.full((c["N"],), 1.0 / c["N"], device="cuda")
    if own:
        import top_softmax_router_gb300 as M
        if c["op"] == "route":
            s["unit"] = M.ScoreRouter(M.ScoreRouterConfig(
                N=c["N"], E=c["E"], k=c["k"], groups=c["groups"], topk_groups=c["topk_groups"], score=c["score"],
                renormalize=c["renormalize"], scale=c["scale"]))
        elif c["op"] == "norm":
            s["unit"] = M.LayerNorm(M.LayerNormConfig(N=c["N"], H=c["H"], eps=1e-5))
        elif c["op"] == "embed":
            s["unit"] = M.TokenEmbedding(M.EmbeddingConfig(N=c["N"], V=c["V"], H=c["H"], scale=c["scale"]))
        else:
            s["unit"] = M.VocabDistill(M.DistillConfig(N=c["N"], H=c["H"], V=c["V"], K=c["K"], P=c["P"],
                                                       temperature=c["tau"]))
    return s


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _own_route(s):
    idx, w, counts = s["unit"].forward(s["logits"], s["b"])
    if not s["train"]:
        return idx, w, counts
    return idx, w, counts, s["unit"].backward(s["logits"], idx, s["dw"])


def _own_norm(s):
    y, mean, rstd = s["unit"].forward(s["x"], s["weight"], s["b"])
    if not s["train"]:
        return y, mean, rstd
    return (y, mean, rstd) + tuple(s["unit"].backward(s["x"], s["weight"], mean, rstd, s["dy"]))


def _own_embed(s):
    y = s["unit"].forward(s["tokens"], s["table"])
    if not s["train"]:
        return y
    # a pass adds into a copy of the gradient so far, so that every pass gives the same
    return y, s["unit"].backward(s["tokens"], s["dy"], into=s["grad"].clone() if s["add"] else None)


def _own_distill(s):
    loss, lse, mean = s["unit"].forward(s["X"], s["W"], s["t_idx"], s["t_logits"])
    if not s["train"]:
        return loss, lse, mean
    return (loss, lse, mean) + tuple(s["unit"].backward(s["X"], s["W"], s["t_idx"], s["t_logits"], lse, s["dloss"]))


def _plain_route(s):
    N, E, k, G, kg = s["N"], s["E"], s["k"], s["groups"], s["topk_groups"]
    l = s["logits"].double()      # neighbouring scores decide between experts
    if s["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.exp(l - l.max(dim=1, keepdim=True).values)
        p = p / p.sum(dim=1, keepdim=True)
    c = p + s["b"].double() if s["b"] is not None else p
    if G > 1:
        top = c.view(N, G, E // G).sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        best = top.sort(dim=1, descending=True, stable=True).indices[:, :kg]
        open_ = torch.zeros(N, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = c.masked_fill(~open_.repeat_interleave(E // G, dim=1), -math.inf)
    idx = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    chosen = p.gather(1, idx)
    total = chosen.sum(dim=1, keepdim=True) if s["renormalize"] else 1.0
    w = (s["scale"] * chosen / total).float()
    counts = torch.zeros(E, dtype=torch.int32, device=l.device)
    counts.index_add_(0, idx.flatten(), torch.ones_like(idx.flatten(), dtype=torch.int32))
    out = (idx.to(torch.int32), w, counts)
    if not s["train"]:
        return out
    p, chosen, dw = p.float(), chosen.float(), s["dw"]
    if s["renormalize"]:
        total = chosen.sum(dim=1, keepdim=True)
        ds = s["scale"] / total * (dw - (dw * chosen).sum(dim=1, keepdim=True) / total)
    else:
        ds = s["scale"] * dw
    dense = torch.zeros_like(p).scatter_(1, idx, ds)
    if s["score"] == "sigmoid":
        dl = dense * p * (1 / (1 + torch.exp(s["logits"].float())))
    else:
        dl = p * (dense - (dense * p).sum(dim=1, keepdim=True))
        if s["renormalize"]:   # the sum is zero by algebra: what is not chosen has no gradient
            dl = p * dense
    return out + (dl.to(s["logits"].dtype),)


def _plain_norm(s):
    x, weight = s["x"].float(), s["weight"].float()
    mean = x.mean(dim=1, keepdim=True)
    centred = x - mean
    rstd = 1 / torch.sqrt((centred * centred).mean(dim=1, keepdim=True) + 1e-5)
    xh = centred * rstd
    y = (xh * weight + s["b"].float()).to(s["x"].dtype)
    out = (y, mean.flatten(), rstd.flatten())
    if not s["train"]:
        return out
    dy = s["dy"].float()
    t = dy * weight
    dx = rstd * (t - t.mean(dim=1, keepdim=True) - xh * (t * xh).mean(dim=1, keepdim=True))
    return out + (dx.to(s["x"].dtype), (dy * xh).sum(dim=0), dy.sum(dim=0))


def _plain_embed(s):
    ids = s["tokens"].long()
    y = (s["table"][ids].float() * s["scale"]).to(s["table"].dtype)
    if not s["train"]:
        return y
    grad = s["grad"].clone() if s["add"] else torch.zeros(s["V"], s["H"], device=ids.device)
    return y, grad.index_add_(0, ids, s["dy"].float() * s["scale"])


def _plain_distill(s):
    X, W, tau = s["X"].float(), s["W"].float(), s["tau"]
    z = (X @ W.t()) / tau
    top = z.max(dim=1, keepdim=True).values
    lse = top + torch.log(torch.exp(z - top).sum(dim=1, keepdim=True))
    there = s["t_idx"] >= 0
    at = s["t_idx"].clamp(min=0).long()
    t = (s["t_logits"] / tau).masked_fill(~there, -math.inf)
    t = t - t.max(dim=1, keepdim=True).values.clamp(min=-1e30)
    e = torch.exp(t)
    total = e.sum(dim=1, keepdim=True)
    some = total > 0
    q = torch.where(some, e / total, 0.0)
    log_q = torch.where(there, t, 0.0) - torch.where(some, torch.log(total), 0.0)
    loss = tau * tau * (q * (log_q - z.gather(1, at) + lse)).sum(dim=1)
    out = (loss, lse.flatten(), loss.mean().view(1))
    if not s["train"]:
        return out
    d = torch.exp(z - lse) * some
    d = d.scatter_add_(1, at, -q) * (s["dloss"] * tau)[:, None]
    return out + ((d @ W).to(BF16), (d.t() @ X).to(BF16))


_run_own = dict(route=_own_route, norm=_own_norm, embed=_own_embed, distill=_own_distill)
_run_plain = dict(route=_plain_route, norm=_plain_norm, embed=_plain_embed, distill=_plain_distill)


# ------------------------------------------------------------------------------------------------- definition
def exact(c, seed):
    s = prepare(c, seed)
    f64 = torch.float64
    if c["op"] == "route":
        x = s["logits"].to(f64)
        prob = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, dim=1)
        gain = prob if s["b"] is None else prob + s["b"].to(f64)
        if c["groups"] > 1:
            by_group = gain.unflatten(1, (c["groups"], -1))
            value = by_group.topk(min(2, by_group.shape[2]), dim=2).values.sum(dim=2)
            # a group is open where fewer than topk_groups others come before it
            before = (value[:, None, :] > value[:, :, None]).sum(dim=2)
            gain = torch.where((before < c["topk_groups"])[:, :, None], by_group, -math.inf).flatten(1)
        idx = torch.argsort(-gain, dim=1, stable=True)[:, :c["k"]]
        mine = torch.take_along_dim(prob, idx, dim=1)
        part = mine / mine.sum(dim=1, keepdim=True) if c["renormalize"] else mine
        counts = torch.bincount(idx.flatten(), minlength=c["E"]).to(torch.int32)
        out = (idx.to(torch.int32), c["scale"] * part, counts)
        if not c["train"]:
            return out
        dw = s["dw"].to(f64) * c["scale"]
        if c["score"] == "softmax" and c["renormalize"]:
            # weights are a softmax over the chosen logits alone
            d = torch.zeros_like(x).scatter_(1, idx, part * (dw - (dw * part).sum(dim=1, keepdim=True)))
            return out + (d,)
        if c["renormalize"]:
            dw = (dw - (dw * part).sum(dim=1, keepdim=True)) / mine.sum(dim=1, keepdim=True)
        if c["score"] == "sigmoid":
            inner = torch.take_along_dim(torch.sigmoid(-x), idx, dim=1) * mine
            return out + (torch.zeros_like(x).scatter_(1, idx, dw * inner),)
        d = torch.zeros_like(x).scatter_(1, idx, dw * mine)
        return out + (d - prob * d.sum(dim=1, keepdim=True),)
    if c["op"] == "norm":
        x, weight = s["x"].to(f64), s["weight"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = (var + 1e-5) ** -0.5
        y = (x - mean) * rstd
        out = (y * weight + s["b"].to(f64), mean[:, 0], rstd[:, 0])
        if not c["train"]:
            return out
        dy = s["dy"].to(f64)
        dweight, dbias = torch.einsum("nh,nh->h", dy, y), dy.sum(dim=0)
        dy = dy * weight
        along = torch.einsum("nh,nh->n", dy, y)[:, None] / c["H"]
        return out + ((dy - dy.mean(dim=1, keepdim=True) - y * along) * rstd, dweight, dbias)
    if c["op"] == "embed":
        ids, scale = s["tokens"].to(torch.int64), c["scale"]
        y = torch.index_select(s["table"], 0, ids).to(f64) * scale
        if not c["train"]:
            return y
        grad = torch.zeros(c["V"], c["H"], dtype=f64, device=y.device)
        grad.index_put_((ids,), s["dy"].to(f64), accumulate=True)
        grad *= scale
        return y, grad + s["grad"] if c["add"] else grad
    if c["N"] * c["H"] * c["V"] > 2.5e12:
        return None
    X, W, tau = s["X"].to(f64), s["W"].to(f64), c["tau"]
    logp = torch.log_softmax(X @ W.t() / tau, dim=1)
    teacher = torch.full((c["N"], c["V"] + 1), -math.inf, dtype=f64, device=X.device)
    teacher.scatter_(1, torch.where(s["t_idx"] < 0, c["V"], s["t_idx"]).long(), s["t_logits"].to(f64) / tau)
    teacher = teacher[:, :c["V"]]
    q = torch.nan_to_num(torch.softmax(teacher, dim=1), nan=0.0)
    loss = tau ** 2 * torch.where(q > 0, q * (torch.log(q) - logp), 0.0).sum(dim=1)
    z0 = (X * W[0]).sum(dim=1) / tau
    out = (loss, z0 - logp[:, 0], loss.mean().view(1))
    if not c["train"]:
        return out
    d = (torch.exp(logp) * q.sum(dim=1, keepdim=True) - q) * (tau * s["dloss"].to(f64)[:, None])
    return out + (d @ W, d.t() @ X)
