"""The training operators that stand beside the quantized linears -- layer norm, the head's softmax
cross entropy and the global gradient norm with clipping -- as cases to be measured.

`run` computes a case in its plain form (elementary torch operations in fp32, rounded once at the
end) or, where `own` is true, through nvfp4_quantized_b200.qt2_train.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
IGNORE = -100
EPS = 1e-5


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # scoring a few tokens against a 32k vocabulary: W's read and the launches are the time
        {"name": "loss 16 x 2048 x 32000", "op": "loss", "T": 16, "K": 2048, "V": 32000, "ignored": 0.0},
        # validation loss of a 1.9B-class model's micro-batch, odd vocabulary
        {"name": "loss 4096 x 2048 x 50257", "op": "loss", "T": 4096, "K": 2048, "V": 50257, "ignored": 0.05},
        # loss and gradients of a short ragged batch; hidden size and vocabulary fill no tile
        {"name": "step 777 x 1000 x 50257", "op": "step", "T": 777, "K": 1000, "V": 50257, "ignored": 0.2},
        # loss and gradients of an 8B-class head (hidden 4096) over a 128k-class vocabulary
        {"name": "step 8192 x 4096 x 128000", "op": "step", "T": 8192, "K": 4096, "V": 128000, "ignored": 0.05},
        # one token's norm: latency alone
        {"name": "norm fwd 1 x 2048 bf16", "op": "norm_fwd", "R": 1, "C": 2048, "x": BF16, "w": BF16},
        # the norm before an 8B-class MLP at its 16384 tokens
        {"name": "norm fwd 16384 x 4096 bf16", "op": "norm_fwd", "R": 16384, "C": 4096, "x": BF16, "w": F32},
        # the norm of the 1.1B-class block at its 32768 tokens, backward
        {"name": "norm bwd 32768 x 2048 bf16", "op": "norm_bwd", "R": 32768, "C": 2048, "x": BF16, "w": BF16},
        # a small batch, backward: the reduction over the rows is short
        {"name": "norm bwd 128 x 2048 bf16", "op": "norm_bwd", "R": 128, "C": 2048, "x": BF16, "w": F32},
        # fp32 activations, odd row length (rows padded to a multiple of 8 elements), backward
        {"name": "norm bwd 4999 x 1601 f32", "op": "norm_bwd", "R": 4999, "C": 1601, "x": F32, "w": F32},
        # a small model's gradients: many short tensors of odd sizes, packed one behind the other
        {"name": "clip 40 small mixed", "op": "clip", "n": 40, "lo": 1, "hi": 5000, "f32": 0.5, "max_norm": 1.0, "scale": 1e-2},
        # fp32 wgrads of eight 1.1B-class blocks (QKV, O, gate, up, down) and their norms' vectors
        {"name": "clip 1.1B blocks f32", "op": "clip", "n": 56, "lo": 0, "hi": 8, "f32": 1.0, "max_norm": 1.0, "scale": 1e-3},
        # a flat bucket of bf16 gradients and fp32 ones, a few hundred odd-sized tensors
        {"name": "clip 300 mixed", "op": "clip", "n": 300, "lo": 1000, "hi": 2000000, "f32": 0.3, "max_norm": 0.5, "scale": 1e-3},
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "step", "norm_fwd", "norm_bwd", "clip"])
    if op in ("loss", "step"):
        most = 8192 * 4096 * 128000 * (1 if op == "step" else 3)
        while True:
            T, K, V = _between(rng, 1, 16384), _between(rng, 64, 4100), _between(rng, 1000, 160000)
            if T * K * V <= most and T * V <= 8192 * 128000:
                return {"op": op, "T": T, "K": K, "V": V, "ignored": rng.choice([0.0, 0.05, 0.5])}
    if op in ("norm_fwd", "norm_bwd"):
        while True:
            R, C = _between(rng, 1, 65536), _between(rng, 16, 20000)
            if R * C <= 1 << 26:
                return {"op": op, "R": R, "C": C, "x": rng.choice([BF16, F32]), "w": rng.choice([BF16, F32])}
    n = _between(rng, 1, 600)
    hi = _between(rng, 2, max(3, 200000000 // n))
    return {"op": op, "n": n, "lo": min(hi, _between(rng, 1, 1000)), "hi": hi, "f32": rng.choice([0.0, 0.3, 1.0]),
            "max_norm": rng.choice([0.5, 1.0, 1e6]), "scale": rng.choice([1e-4, 1e-2, 1.0])}


# the parameters of a 1.1B-class block: QKV, O, gate, up, down and its two norms' weight vectors
_BLOCK = [6144 * 2048, 2048 * 2048, 5632 * 2048, 5632 * 2048, 2048 * 5632, 2048, 2048]


def _sizes(case):
    """Numbers of elements and types of a clip case's tensors (the same for every seed)."""
    if case["lo"] == 0:
        return [(_BLOCK[i % len(_BLOCK)], F32) for i in range(case["n"])]
    g = torch.Generator().manual_seed(case["n"] * 1000003 + case["hi"])
    u, t = torch.rand(case["n"], generator=g).tolist(), torch.rand(case["n"], generator=g).tolist()
    span = math.log(case["hi"] / case["lo"])
    return [(int(case["lo"] * math.exp(span * a)), F32 if b < case["f32"] else BF16) for a, b in zip(u, t)]


def work(case):
    op = case["op"]
    if op in ("loss", "step"):
        T, K, V = case["T"], case["K"], case["V"]
        if op == "loss":
            return {"bytes": 2 * K * (T + V) + 16 * T, "flops": 2 * T * V * K}
        # logits, dx and dw: the second forming of the logits, which not keeping them costs, is not counted
        return {"bytes": 4 * K * (T + V) + 20 * T, "flops": 6 * T * V * K}
    if op in ("norm_fwd", "norm_bwd"):
        R, C = case["R"], case["C"]
        e, w = (2 if case["x"] == BF16 else 4), (2 if case["w"] == BF16 else 4)
        if op == "norm_fwd":
            return {"bytes": 2 * R * C * e + 8 * R + 2 * C * w, "flops": 8 * R * C}
        return {"bytes": 3 * R * C * e + 8 * R + 3 * C * w, "flops": 15 * R * C}
    sizes = _sizes(case)
    b = sum(n * (4 if t == F32 else 2) for n, t in sizes)
    return {"bytes": 2 * b + 4, "flops": 3 * sum(n for n, _ in sizes)}


# ------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(R, C, dtype):
    """An uninitialised [R, C] matrix whose rows start 16-byte aligned (leading dimension a multiple of 8)."""
    return torch.empty((R, (C + 7) // 8 * 8), dtype=dtype, device="cuda")[:, :C]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"op": op, "case": case}
    if op in ("loss", "step"):
        T, K, V = case["T"], case["K"], case["V"]
        w = _rows(V, K, torch.bfloat16).copy_(_randn(g, V, K).mul_(0.02))
        # frequent words are much more frequent than rare ones
        y = (V * torch.rand(T, generator=g, device="cuda") ** 3).long().clamp_(max=V - 1)
        # hidden states of unit variance, moved toward the target's row so that its logit rises by 0 to about 12
        lift = -4 * torch.log(torch.rand((T, 1), generator=g, device="cuda").clamp_(min=0.05))
        x = _rows(T, K, torch.bfloat16).copy_(_randn(g, T, K) + lift * w[y].float() / (0.02 ** 2 * K))
        ignored = torch.rand(T, generator=g, device="cuda") < case["ignored"]
        s |= {"x": x, "w": w, "y": torch.where(ignored, IGNORE, y), "loss": torch.empty(T, device="cuda"), "lse": torch.empty(T, device="cuda")}
        if op == "step":  # the mean over the tokens that count, with a weight for each
            weight = torch.where(ignored, 0.0, 0.5 + torch.rand(T, generator=g, device="cuda"))
            s |= {"dloss": weight / weight.sum().clamp(min=0.5), "dx": _rows(T, K, torch.bfloat16), "dw": _rows(V, K, torch.bfloat16)}
    elif op in ("norm_fwd", "norm_bwd"):
        R, C, dx, dw = case["R"], case["C"], _DTYPE[case["x"]], _DTYPE[case["w"]]
        x = _randn(g, R, C)
        x[:, :: max(2, C // 4)] *= 8.0  # a few channels carry large values
        x += 0.5 * _randn(g, R, 1)
        s |= {"x": _rows(R, C, dx).copy_(x), "w": (1 + 0.1 * _randn(g, C)).to(dw), "b": (0.1 * _randn(g, C)).to(dw),
              "mean": torch.empty(R, device="cuda"), "rstd": torch.empty(R, device="cuda")}
        if op == "norm_fwd":
            s["out"] = _rows(R, C, dx)
        else:  # what the forward pass kept
            var, mean = torch.var_mean(s["x"].double(), 1, correction=0)
            s |= {"mean": mean.float(), "rstd": (var + EPS).rsqrt().float(), "dy": _rows(R, C, dx).copy_(_randn(g, R, C).mul_(1e-2)),
                  "out": _rows(R, C, dx), "dw": torch.empty_like(s["w"]), "db": torch.empty_like(s["b"])}
    else:
        sizes = _sizes(case)
        flat = {t: _randn(g, sum(n for n, u in sizes if u == t)).mul_(case["scale"]).to(_DTYPE[t]) for t in (BF16, F32)}
        flat = {t: f for t, f in flat.items() if f.numel()}
        out = {t: torch.empty_like(f) for t, f in flat.items()}
        at, grads, outs = {BF16: 0, F32: 0}, [], []
        for n, t in sizes:  # tensors packed one behind the other, as gradient buckets hold them
            if n:
                grads.append(flat[t][at[t]:at[t] + n])
                outs.append(out[t][at[t]:at[t] + n])
                at[t] += n
        s |= {"flat": flat, "out": out, "grads": grads, "outs": outs, "norm": torch.empty((), device="cuda")}
    return s


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _plain(s):
    op = s["op"]
    if op in ("loss", "step"):
        x, w, y = s["x"].float(), s["w"].float(), s["y"]
        counts, at = y != IGNORE, y.clamp(min=0)[:, None]
        logits = x @ w.T
        top = logits.amax(1, keepdim=True)
        lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(1))
        loss = torch.where(counts, lse - logits.gather(1, at)[:, 0], 0.0)
        if op == "loss":
            return loss, lse
        p = torch.exp_(logits.sub_(lse[:, None]))
        p.scatter_add_(1, at, p.new_full((1, 1), -1.0).expand_as(at))
        p.mul_(torch.where(counts, s["dloss"], 0.0)[:, None])
        return loss, lse, (p @ w).to(s["x"].dtype), (p.T @ x).to(s["w"].dtype)
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        return (d * rstd * s["w"].float() + s["b"].float()).to(s["x"].dtype), mean[:, 0], rstd[:, 0]
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        h = (s["x"].float() - s["mean"][:, None]) * rstd
        a = dy * s["w"].float()
        dx = rstd * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
        return dx.to(s["x"].dtype), (dy * h).sum(0).to(s["w"].dtype), dy.sum(0).to(s["w"].dtype)
    norm = torch.stack([f.float().square().sum() for f in s["flat"].values()]).sum().sqrt()
    scale = (s["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return norm, [(f.float() * scale).to(f.dtype) for f in s["flat"].values()]


def _own(s):
    from nvfp4_quantized_b200 import qt2, qt2_train as tr
    op = s["op"]
    if op in ("loss", "step"):
        x, w, y = s["x"], s["w"], s["y"]
        (T, K), V = x.shape, w.shape[0]
        if "ws" not in s:
            size = tr.qt2_linear_xent_fwd_workspace_size(T, K, V)
            if op == "step":
                size = max(size, tr.qt2_linear_xent_bwd_workspace_size(T, K, V))
            s["ws"] = qt2.alloc_workspace(size)
        ws = s["ws"]
        tr.qt2_linear_xent_fwd(x, w, y, T, K, V, x.stride(0), w.stride(0), IGNORE, s["loss"], s["lse"], ws, ws.numel())
        if op == "loss":
            return s["loss"], s["lse"]
        tr.qt2_linear_xent_bwd(x, w, y, s["lse"], s["dloss"], T, K, V, x.stride(0), w.stride(0), IGNORE, s["dx"],
                               s["dx"].stride(0), s["dw"], qt2.QT2_DTYPE_BF16, s["dw"].stride(0), ws, ws.numel())
        return s["loss"], s["lse"], s["dx"], s["dw"]
    if op == "norm_fwd":
        x, out = s["x"], s["out"]
        R, C = x.shape
        tr.qt2_layernorm_fwd(x, R, C, x.stride(0), s["w"], s["b"], EPS, out, out.stride(0), s["mean"], s["rstd"])
        return out, s["mean"], s["rstd"]
    if op == "norm_bwd":
        x, dy, out = s["x"], s["dy"], s["out"]
        R, C = x.shape
        if "ws" not in s:
            s["ws"] = qt2.alloc_workspace(tr.qt2_layernorm_bwd_workspace_size(R, C))
        tr.qt2_layernorm_bwd(dy, dy.stride(0), x, R, C, x.stride(0), s["w"], s["mean"], s["rstd"], out, out.stride(0),
                             s["dw"], s["db"], s["ws"], s["ws"].numel())
        return out, s["dw"], s["db"]
    if "list" not in s:
        s["list"] = tr.GradList(s["grads"], s["outs"])
        s["ws"] = qt2.alloc_workspace(tr.qt2_grad_norm_workspace_size(s["list"]))
    tr.qt2_grad_norm(s["list"], s["norm"], s["ws"], s["ws"].numel())
    tr.qt2_grad_clip(s["list"], s["norm"], s["case"]["max_norm"])
    return s["norm"], list(s["out"].values())


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("loss", "step"):
        return _exact_loss(s, op == "step")
    if op == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        return ((x - mean[:, None]) * rstd[:, None]).mul_(s["w"].double()).add_(s["b"].double()), mean, rstd
    if op == "norm_bwd":
        # the gradient as the sum of the three ways in which x moves y: itself, the mean, the deviation
        x, m, r = s["x"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        dy, C = s["dy"].double(), s["x"].shape[1]
        up = dy * s["w"].double()
        d = x - m
        dvar = -0.5 * (up * d).sum(1, keepdim=True) * r ** 3
        dmean = -(up * r).sum(1, keepdim=True) - 2 * dvar * d.mean(1, keepdim=True)
        # (the second term vanishes up to the rounding of the mean that was kept)
        return up * r + dvar * 2 * d / C + dmean / C, (dy * d * r).sum(0), dy.sum(0)
    total = sum(f.double().square().sum() for f in s["flat"].values())
    norm = total.sqrt()
    m = case["max_norm"]
    return norm, [f.double() * min(1.0, m / (float(norm) + 1e-6)) for f in s["flat"].values()]


def _exact_loss(s, step):
    """Online over pieces of the vocabulary, in 64 bits."""
    x, w, y = s["x"].double(), s["w"], s["y"]
    T, V, n = x.shape[0], w.shape[0], 8192
    lse, hit = torch.full((T,), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(T, dtype=torch.float64, device="cuda")
    here = torch.arange(T, device="cuda")
    for v in range(0, V, n):
        z = x @ w[v:v + n].double().T
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        mine = (y >= v) & (y < v + z.shape[1])
        hit[mine] = z[here[mine], y[mine] - v]
    loss = torch.where(y == IGNORE, 0.0, lse - hit)
    if not step:
        return loss, lse
    up = torch.where(y == IGNORE, 0.0, s["dloss"].double())
    dx, dw = torch.zeros_like(x), torch.empty(w.shape, dtype=torch.float64, device="cuda")
    for v in range(0, V, n):
        part = w[v:v + n].double()
        z = torch.exp(x @ part.T - lse[:, None])
        mine = (y >= v) & (y < v + z.shape[1])
        z[here[mine], y[mine] - v] -= 1.0
        z *= up[:, None]
        dx += z @ part
        dw[v:v + n] = z.T @ x
    return loss, lse, dx, dw
