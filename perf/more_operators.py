"""The 8-bit path around the block as timed cases: RMS norm with the residual's addition and 8-bit output, activation
checkpoints in 8 bits, and products by expert in bf16 and in 8 bits with a scale for each block of 128, forward and, in
training, with their gradients.

`run` makes the library's calls where `own` is true; where it is false it computes the same results with elementary
torch operations in fp32.  `exact` is the definition in fp64.
"""
import math
import random

import torch

own = False

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TYPES = {"bf16": BF16, "fp16": FP16, "fp32": FP32, "e4m3": E4M3}
BLOCK = 128
EPS = 1e-6


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 16 sequences: the residual added, the norm's output in 8 bits; latency only
        dict(name="rms decode", op="rms", N=16, H=2048, type="bf16", params="bf16", residual=True, codes=True,
             train=False),
        # an odd width: no row is aligned, the last block of 128 is short
        dict(name="rms odd width", op="rms", N=4099, H=1001, type="bf16", params="bf16", residual=True, codes=True,
             train=True),
        # a full training batch at the widest hidden size, both upstream gradients
        dict(name="rms wide", op="rms", N=32768, H=7168, type="bf16", params="fp32", residual=True, codes=True,
             train=True),
        # a small ragged checkpoint, kept and restored
        dict(name="checkpoint ragged", op="checkpoint", N=333, H=1000, type="bf16"),
        # the inputs of a layer of 65536 tokens
        dict(name="checkpoint long", op="checkpoint", N=65536, H=4096, type="bf16"),
        # a dense 8-bit layer, one token for each of 8 sequences: the weights' bytes
        dict(name="linear8 decode", op="linear", N=8, K=7168, O=2048, E=1, type="e4m3", tail=False, train=False,
             dw="fp32"),
        # a prompt of 1000 tokens through it
        dict(name="linear8 prompt", op="linear", N=1000, K=2048, O=2816, E=1, type="e4m3", tail=False, train=False,
             dw="fp32"),
        # a training step of it
        dict(name="linear8 train", op="linear", N=16384, K=7168, O=2048, E=1, type="e4m3", tail=False, train=True,
             dw="fp32"),
        # a decode step: 64 routes over 64 experts in bf16, many experts without a row
        dict(name="experts decode", op="linear", N=64, K=2048, O=1408, E=64, type="bf16", tail=False, train=False,
             dw="fp32"),
        # all routes of 16384 tokens x 8 over 64 experts, in bf16, a training step; the buffer is longer than its rows
        dict(name="experts train", op="linear", N=131072, K=2048, O=1408, E=64, type="bf16", tail=True, train=True,
             dw="fp32"),
        # a decode step over 128 experts in 8 bits
        dict(name="experts8 decode", op="linear", N=128, K=4096, O=1536, E=128, type="e4m3", tail=False, train=False,
             dw="fp32"),
        # a training step over 128 experts in 8 bits, weight gradients in bf16
        dict(name="experts8 train", op="linear", N=65536, K=4096, O=1536, E=128, type="e4m3", tail=True, train=True,
             dw="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms", "checkpoint", "linear", "linear", "linear"])
    train = rng.random() < 0.6
    if op == "rms":
        H = rng.choice([_spread(rng, 64, 8192) | 1, 64 * _spread(rng, 1, 40), 4096, 7168])
        t = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = min(32768, 32768 * 7168 // (H * (2 if t == "fp32" else 1)))
        return dict(op=op, N=_spread(rng, 1, most), H=H, type=t, params=rng.choice(["fp32", t]),
                    residual=rng.random() < 0.7, codes=rng.random() < 0.7, train=train)
    if op == "checkpoint":
        H = rng.choice([_spread(rng, 64, 8192) | 1, 8 * _spread(rng, 8, 900), 4096])
        return dict(op=op, N=_spread(rng, 1, min(65536, 65536 * 4096 // H)), H=H,
                    type=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    E = rng.choice([1, 1, 5, 8, 64, 128])
    K, O = 16 * _spread(rng, 4, 448), 16 * _spread(rng, 4, 256)
    while E * K * O > 128 * 4096 * 1536:
        K = max(64, K // 32 * 16)
    most = max(64, min(131072, 65536 * 4096 * 1536 // (K * O)))
    return dict(op=op, N=_spread(rng, 1, most), K=K, O=O, E=E, type=rng.choice(["bf16", "e4m3"]),
                tail=rng.random() < 0.5, train=train, dw=rng.choice(["fp32", "bf16"]))


def _shares(E):
    """How likely a row is each expert's, the most likely first."""
    w = [(1 + r) ** -0.4 for r in range(E)]
    return [x / sum(w) for x in w]


def work(c):
    """Bytes and operations of one pass: every input read once, every output written once."""
    if c["op"] == "rms":
        N, H, b, pb = c["N"], c["H"], TYPES[c["type"]].itemsize, TYPES[c["params"]].itemsize
        nb = -(-H // BLOCK)
        nbytes = N * H * b + H * pb + 4 * N + (2 * N * H * b if c["residual"] else 0)
        nbytes += N * H + N * nb if c["codes"] else N * H * b
        flops = 6 * N * H
        if c["train"]:
            nbytes += 3 * N * H * b + H * pb + 4 * N + 4 * H + (N * H * b if c["residual"] else 0)
            flops += 10 * N * H
        return dict(bytes=nbytes, flops=flops)
    if c["op"] == "checkpoint":
        n = c["N"] * c["H"]
        return dict(bytes=n * TYPES[c["type"]].itemsize + 2 * (n + n // BLOCK) + n * 2, flops=4 * n)
    N, K, O, E, b = c["N"], c["K"], c["O"], c["E"], TYPES[c["type"]].itemsize
    met = sum(1 - (1 - p) ** N for p in _shares(E))      # experts that have rows
    nbytes, flops = N * K * b + met * O * K * b + N * O * 2, 2 * N * K * O
    if c["train"]:   # dy, x and the weights again; dx and the weights' gradients out
        nbytes += N * O * 2 + N * K * b + met * O * K * b + N * K * 2 + E * O * K * TYPES[c["dw"]].itemsize
        flops *= 3
    return dict(bytes=int(nbytes), flops=flops)


# ------------------------------------------------------------------------------------------------- inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, type=FP32):
        return (torch.randn(*shape, device="cuda", generator=g) * std + mean).to(type)

    def activations(n, h, type):
        """Rows of different sizes, a few columns far larger than the others."""
        column = torch.where(torch.rand(h, device="cuda", generator=g) < 0.01, 12.0, 1.0)
        x = torch.randn(n, h, device="cuda", generator=g) * column
        return x.mul_(torch.exp(normal(n, 1, std=0.5))).to(type)

    s = dict(c)
    if c["op"] == "rms":
        t = TYPES[c["type"]]
        s["x"] = activations(c["N"], c["H"], t)
        s["r"] = normal(c["N"], c["H"], std=2.0, type=t) if c["residual"] else None
        s["weight"] = normal(c["H"], std=0.2, mean=1.0, type=TYPES[c["params"]])
        s["dy"] = normal(c["N"], c["H"], std=0.1, type=t) if c["train"] else None
        s["dh"] = normal(c["N"], c["H"], std=0.1, type=t) if c["train"] and c["residual"] else None
    elif c["op"] == "checkpoint":
        s["x"] = activations(c["N"], c["H"], TYPES[c["type"]])
    else:
        N, K, O, E = c["N"], c["K"], c["O"], c["E"]
        rng = random.Random(seed)
        rows = N - (N // 32 if c["tail"] else 0)
        share = _shares(E)
        rng.shuffle(share)
        counts = [0] * E
        if rows > 64 * E:       # many rows: near the expected share, two experts without any
            left = rng.sample(range(E), 2) if E > 4 else []
            for e in range(E):
                counts[e] = 0 if e in left else int(rows * share[e] * rng.uniform(0.8, 1.2))
            counts[share.index(max(share))] += rows - sum(counts)
            while min(counts) < 0:
                counts[counts.index(max(counts))] += min(counts)
                counts[counts.index(min(counts))] = 0
        else:
            for e in rng.choices(range(E), share, k=rows):
                counts[e] += 1
        offsets = [0]
        for n in counts:
            offsets.append(offsets[-1] + n)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda") if E > 1 or c["tail"] else None
        s["rows"], s["most"], s["ends"] = offsets[-1], max(counts), offsets
        x = activations(N, K, BF16)
        w = torch.empty(E, O, K, device="cuda", dtype=BF16).normal_(0, K ** -0.5, generator=g)
        s["x_scales"] = s["w_scales"] = None
        if c["type"] == "e4m3":
            x, s["x_scales"] = _pack(x)
            w, s["w_scales"] = _pack_weight(w)
        s["x"], s["w"] = x, w
        s["dy"] = normal(N, O, std=1e-3, type=BF16) if c["train"] else None
        if rows < N:            # what lies behind the last row is no number
            s["x"].view(torch.uint8 if c["type"] == "e4m3" else torch.int16)[rows:] = 0x7F if c["type"] == "e4m3" else 0x7FC0
            if c["train"]:
                s["dy"][rows:] = math.nan
    if own:
        import top_softmax_router_gb300 as M
        if c["op"] == "rms":
            s["unit"] = M.RMSNorm(M.RMSNormConfig(N=c["N"], H=c["H"], eps=EPS))
        elif c["op"] == "checkpoint":
            s["unit"] = M.Checkpoint8(M.Checkpoint8Config(N=c["N"], H=c["H"]))
        else:
            s["unit"] = M.ExpertLinear(M.ExpertLinearConfig(N=c["N"], K=c["K"], O=c["O"], E=c["E"],
                                                            blocks8=c["type"] == "e4m3"))
    return s


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _own_rms(s):
    y, h, rstd, codes, scales = s["unit"].forward(s["x"], s["weight"], s["r"], want_y=not s["codes"],
                                                  want_codes=s["codes"])
    out = (codes, scales, rstd) if s["codes"] else (y, rstd)
    out += (h,) if s["residual"] else ()
    if s["train"]:
        out += tuple(s["unit"].backward(h, s["weight"], rstd, s["dy"], s["dh"]))
    return out


def _own_checkpoint(s):
    codes, scales = s["unit"].pack(s["x"])
    return s["unit"].unpack(codes, scales)


def _own_linear(s):
    x, w, at, xs, ws = s["x"], s["w"], s["offsets"], s["x_scales"], s["w_scales"]
    y = s["unit"].forward(x, w, at, xs, ws)
    if not s["train"]:
        return y
    return (y,) + tuple(s["unit"].backward(x, w, s["dy"], at, xs, ws, dw_dtype=TYPES[s["dw"]]))


def _scale_of(amax):
    """2^e, the smallest with amax <= 448 x 2^e; 1 for an amax of 0."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, 448 = 0.875 x 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-127)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax == 0, 0, e))


def _pack(x):
    """Codes and scales of rows: one scale for 128 columns of a row."""
    n, h = x.shape
    pad = -h % BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(n, -1, BLOCK)
    scale = _scale_of(v.abs().amax(dim=2))
    codes = (v / scale[:, :, None]).to(E4M3).view(n, h + pad)[:, :h].contiguous()
    return codes, scale.to(E8M0)


def _pack_weight(w):
    """Codes and scales of matrices: one scale for 128 x 128 values."""
    E, O, K = w.shape
    v = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -O % BLOCK)).view(E, -(-O // BLOCK), BLOCK, -(-K // BLOCK), BLOCK)
    scale = _scale_of(v.abs().amax(dim=(2, 4)).float())
    codes = (v.float() / scale[:, :, None, :, None]).to(E4M3)
    return codes.view(E, O + -O % BLOCK, K + -K % BLOCK)[:, :O, :K].contiguous(), scale.to(E8M0)


def _unpack(codes, scales):
    h = codes.shape[1]
    return codes.float() * scales.float().repeat_interleave(BLOCK, dim=1)[:, :h]


def _unpack_weight(codes, scales):
    _, O, K = codes.shape
    s = scales.float().repeat_interleave(BLOCK, dim=1)[:, :O].repeat_interleave(BLOCK, dim=2)[:, :, :K]
    return codes.float() * s


def _plain_rms(s):
    x, weight = s["x"], s["weight"].float()
    h = (x.float() + s["r"].float()).to(x.dtype) if s["residual"] else x
    v = h.float()
    rstd = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    xh = v * rstd
    y = xh * weight
    out = _pack(y) + (rstd.flatten(),) if s["codes"] else (y.to(x.dtype), rstd.flatten())
    out += (h,) if s["residual"] else ()
    if not s["train"]:
        return out
    dy = s["dy"].float()
    t = dy * weight
    dx = rstd * (t - xh * (t * xh).mean(dim=1, keepdim=True))
    if s["residual"]:
        dx = dx + s["dh"].float()
    return out + (dx.to(x.dtype), (dy * xh).sum(dim=0))


def _plain_checkpoint(s):
    return _unpack(*_pack(s["x"])).to(BF16)


def _plain_linear(s):
    """The experts' rows side by side in a padded [E, most, ...], and batched products."""
    N, E, most, rows = s["N"], s["E"], s["most"], s["rows"]
    x, w, dy = s["x"], s["w"], s["dy"]
    if s["type"] == "e4m3":
        x, w = _unpack(x, s["x_scales"]), _unpack_weight(w, s["w_scales"])
    else:
        x, w = x.float(), w.float()
    if s["offsets"] is None:
        y = (x @ w[0].t()).to(BF16)
        if not s["train"]:
            return y
        d = _unpack(*_pack(dy)) if s["type"] == "e4m3" else dy.float()
        return y, (d @ w[0]).to(BF16), (dy.float().t() @ x)[None].to(TYPES[s["dw"]])
    at = s["offsets"].long()
    row = torch.arange(rows, device=x.device)
    expert = torch.bucketize(row, at[1:], right=True)
    place = expert * most + row - at[expert]

    def padded(v):
        return torch.zeros(E * most, v.shape[1], device=v.device).index_copy_(0, place, v[:rows]).view(E, most, -1)

    def whole(v):
        out = torch.zeros(N, v.shape[2], dtype=BF16, device=v.device)
        out[:rows] = v.view(E * most, -1)[place].to(BF16)
        return out

    px = padded(x)
    y = whole(px @ w.transpose(1, 2))
    if not s["train"]:
        return y
    d = _unpack(*_pack(dy)) if s["type"] == "e4m3" else dy.float()
    return y, whole(padded(d) @ w), (padded(dy.float()).transpose(1, 2) @ px).to(TYPES[s["dw"]])


_run_own = dict(rms=_own_rms, checkpoint=_own_checkpoint, linear=_own_linear)
_run_plain = dict(rms=_plain_rms, checkpoint=_plain_checkpoint, linear=_plain_linear)


# ------------------------------------------------------------------------------------------------- definition
def _blocks64(v):
    """(codes, scales) of fp64 rows, one scale for 128 columns, the codes rounded to e4m3's steps."""
    n, h = v.shape
    full = torch.zeros(n, -(-h // BLOCK) * BLOCK, dtype=v.dtype, device=v.device)
    full[:, :h] = v
    full = full.unflatten(1, (-1, BLOCK))
    top = torch.linalg.vector_norm(full, ord=math.inf, dim=2)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-127.0))
    scale = torch.where(top > 0, scale, 1.0)
    q = full / scale.unsqueeze(2)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).flatten(1)[:, :h], scale


def exact(c, seed):
    s = prepare(c, seed)
    f64 = torch.float64
    if c["op"] == "rms":
        h = s["x"].to(f64)
        if c["residual"]:       # the sum is kept in the inputs' type
            h = (h + s["r"].to(f64)).to(s["x"].dtype).to(f64)
        scale = torch.rsqrt(h.square().sum(dim=1, keepdim=True) / c["H"] + EPS)
        n = h * scale
        y = n * s["weight"].to(f64)
        out = (*_blocks64(y), scale[:, 0]) if c["codes"] else (y, scale[:, 0])
        if c["residual"]:
            out += (h,)
        if not c["train"]:
            return out
        d = s["dy"].to(f64)
        dweight = torch.einsum("nh,nh->h", d, n)
        d = d * s["weight"].to(f64)
        dx = scale * (d - n * (torch.einsum("nh,nh->n", d, n) / c["H"])[:, None])
        return out + (dx + s["dh"].to(f64) if c["residual"] else dx, dweight)
    if c["op"] == "checkpoint":
        codes, scale = _blocks64(s["x"].to(f64))
        cols = torch.arange(c["H"], device=codes.device) // BLOCK
        return codes * scale[:, cols]
    if c["N"] * c["K"] * c["O"] > 5e11:
        return None
    N, K, O, E = c["N"], c["K"], c["O"], c["E"]
    ends = s["ends"]
    kb, ob = torch.arange(K, device="cuda") // BLOCK, torch.arange(O, device="cuda") // BLOCK
    y = torch.zeros(N, O, dtype=f64, device="cuda")
    dx = torch.zeros(N, K, dtype=f64, device="cuda") if c["train"] else None
    dw = torch.zeros(E, O, K, dtype=f64, device="cuda") if c["train"] else None
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        x, w = s["x"][a:b].to(f64), s["w"][e].to(f64)
        if c["type"] == "e4m3":
            x *= s["x_scales"][a:b].to(f64)[:, kb]
            w *= s["w_scales"][e].to(f64)[ob][:, kb]
        torch.mm(x, w.t(), out=y[a:b])
        if c["train"]:
            d = s["dy"][a:b].to(f64)
            torch.mm(d.t(), x, out=dw[e])
            if c["type"] == "e4m3":
                codes, scale = _blocks64(d)
                d = codes * scale[:, ob]
            torch.mm(d, w, out=dx[a:b])
    return (y, dx, dw) if c["train"] else y
