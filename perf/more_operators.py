"""What a transformer block's training step needs between the quantized linears -- the gated feed-forward
product on NVFP4 operands and its backward pass, the norm of queries and keys for each head with the position
rotation, the AdamW update of many tensors -- as cases to be measured.

`run` computes a case in its plain form (elementary torch operations in fp32, rounded once at the end) or,
where `own` is true, through nvfp4_quantized_b200.qt2_train.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-6
BETA1, BETA2, ADAM_EPS, MAX_NORM = 0.9, 0.95, 1e-8, 1.0
SEED = 20


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # evaluating 128 tokens through a 1.1B-class block's gate and up projections: the weights' read
        {"name": "gated 128 x 2048 x 5632", "op": "gated", "M": 128, "K": 2048, "F": 5632, "act": "silu", "keep": False},
        # a small model whose sizes fill no pair of tiles, trained: gate and up are kept for the backward pass
        {"name": "gated 1920 x 2176 x 1408 gelu", "op": "gated", "M": 1920, "K": 2176, "F": 1408, "act": "gelu", "keep": True},
        # the 8B-class MLP at its 16384 tokens, trained
        {"name": "gated 16384 x 4096 x 14336", "op": "gated", "M": 16384, "K": 4096, "F": 14336, "act": "silu", "keep": True},
        # the small model's backward pass through the down projection and the activation
        {"name": "gated bwd 640 x 1408 x 2176", "op": "gated_bwd", "M": 640, "K": 1408, "F": 2176, "act": "gelu"},
        # the 8B-class MLP's
        {"name": "gated bwd 16384x4096x14336", "op": "gated_bwd", "M": 16384, "K": 4096, "F": 14336, "act": "silu"},
        # one token being decoded: latency alone
        {"name": "qk rope 1 x 32+8 x 128", "op": "rope", "T": 1, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "x": BF16, "w": BF16, "pairs": False},
        # the QKV projection's output of the 1.1B-class block at its 32768 tokens
        {"name": "qk rope 32768 x 16+16 x 128", "op": "rope", "T": 32768, "Hq": 16, "Hk": 16, "D": 128, "R": 128, "x": BF16, "w": F32, "pairs": False},
        # its backward pass
        {"name": "qk rope bwd 32768x16+16x128", "op": "rope_bwd", "T": 32768, "Hq": 16, "Hk": 16, "D": 128, "R": 128, "x": BF16, "w": F32, "pairs": False},
        # a short ragged batch, backward: fp32, shared key heads, half of a head rotated, neighbours as pairs
        {"name": "qk rope bwd 777 x 12+4 x 80 f32", "op": "rope_bwd", "T": 777, "Hq": 12, "Hk": 4, "D": 80, "R": 40, "x": F32, "w": F32, "pairs": True},
        # a small model's tensors, packed one behind the other: short, of odd sizes
        {"name": "adamw 40 small f32", "op": "adamw", "n": 40, "lo": 1, "hi": 5000, "kind": "f32", "state": "f32", "pack": 1},
        # eight 1.1B-class blocks with fp32 weights, gradients and states
        {"name": "adamw 1.1B blocks f32", "op": "adamw", "n": 56, "lo": 0, "hi": 8, "kind": "f32", "state": "f32", "pack": 256},
        # the same in bf16 with fp32 masters and states of 8 bits
        {"name": "adamw 1.1B blocks 8 bits", "op": "adamw", "n": 56, "lo": 0, "hi": 8, "kind": "master", "state": "e4m3", "pack": 256},
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_bwd", "rope", "rope_bwd", "adamw"])
    if op in ("gated", "gated_bwd"):
        while True:
            M, K, F = (128 * _between(rng, 1, n) for n in (256, 112, 112))
            if M * K * F <= 16384 * 4096 * 14336 and M * F <= 16384 * 14336:
                case = {"op": op, "M": M, "K": K, "F": F, "act": rng.choice(["silu", "gelu"])}
                return case | {"keep": rng.random() < 0.5} if op == "gated" else case
    if op in ("rope", "rope_bwd"):
        while True:
            T, Hq, Hk, D = _between(rng, 1, 65536), _between(rng, 1, 64), _between(rng, 1, 16), rng.choice([64, 80, 96, 128, 192, 256])
            if T * (Hq + 2 * Hk) * D <= 32768 * 6144:
                return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": rng.choice([D, D // 2]), "x": rng.choice([BF16, F32]),
                        "w": rng.choice([BF16, F32]), "pairs": rng.random() < 0.5}
    n = _between(rng, 1, 600)
    hi = _between(rng, 2, max(3, 200000000 // n))
    state = rng.choice(["f32", "e4m3"])
    return {"op": op, "n": n, "lo": min(hi, _between(rng, 1, 1000)), "hi": hi, "kind": rng.choice(["f32", "master", "bf16"]),
            "state": state, "pack": 256 if state == "e4m3" else rng.choice([1, 256])}


# the parameters of a 1.1B-class block: QKV, O, gate, up, down and its two norms' weight vectors
_BLOCK = [6144 * 2048, 2048 * 2048, 5632 * 2048, 5632 * 2048, 2048 * 5632, 2048, 2048]


def _sizes(case):
    """Numbers of elements of an AdamW case's tensors (the same for every seed)."""
    if case["lo"] == 0:
        return [_BLOCK[i % len(_BLOCK)] for i in range(case["n"])]
    g = torch.Generator().manual_seed(case["n"] * 1000003 + case["hi"])
    span = math.log(case["hi"] / case["lo"])
    return [int(case["lo"] * math.exp(span * a)) for a in torch.rand(case["n"], generator=g).tolist()]


def work(case):
    op = case["op"]
    if op == "gated":
        M, K, F = case["M"], case["K"], case["F"]
        return {"bytes": 9 * K * (M + 2 * F) // 16 + M * F * (6 if case["keep"] else 2), "flops": 4 * M * F * K}
    if op == "gated_bwd":
        M, K, F = case["M"], case["K"], case["F"]
        return {"bytes": 9 * K * (M + F) // 16 + M * F * 10, "flops": 2 * M * F * K}
    if op in ("rope", "rope_bwd"):
        T, D, e = case["T"], case["D"], 2 if case["x"] == BF16 else 4
        n = T * (case["Hq"] + case["Hk"]) * D
        return {"bytes": n * e * (2 if op == "rope" else 3) + T * 8 + min(T, _table(case)) * case["R"] * 4, "flops": n * (8 if op == "rope" else 18)}
    n = sum(_sizes(case))
    b = {"f32": 4 + 8, "master": 2 + 2 + 8, "bf16": 2 + 4}[case["kind"]] + (16 if case["state"] == "f32" else 4 + 16 / 256)
    return {"bytes": int(n * b), "flops": 15 * n}


# ------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _view(g, R, C, std):
    """An NVFP4 view of normal values: codes [R, C/2], scales in the tensor cores' order, the tensor's scale."""
    x = _randn(g, R, C // 16, 16).mul_(std)
    top = x.abs().amax(2)
    scale = top.max() / 1792
    s = (top / (6 * scale)).to(torch.float8_e4m3fn)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(x.abs() / (s.float() * scale)[:, :, None].clamp(min=1e-30), mid, out_int32=True).to(torch.uint8)
    code = (code + (x < 0).to(torch.uint8) * 8).view(R, C // 2, 2)
    order = s.view(torch.uint8).view(R // 128, 4, 32, C // 64, 4).permute(0, 3, 2, 1, 4)
    return code[:, :, 0] + 16 * code[:, :, 1], order.reshape(-1).contiguous(), scale.reshape(1)


def _table(case):
    return 8192 if case["T"] > 1 else 131072  # a decoded token may be far into its sequence


def prepare(case, seed):
    g, op = torch.Generator(device="cuda").manual_seed(seed), case["op"]
    s = {"op": op, "case": case}
    if op in ("gated", "gated_bwd"):
        M, K, F, bf = case["M"], case["K"], case["F"], torch.bfloat16
        new = lambda: torch.empty((M, F), dtype=bf, device="cuda")  # noqa: E731
        if op == "gated":
            s |= {"a": _view(g, M, K, 1.0), "gate_w": _view(g, F, K, K ** -0.5), "up_w": _view(g, F, K, K ** -0.5), "h": new()}
            s |= {"gate": new(), "up": new()} if case["keep"] else {"gate": None, "up": None}
        else:  # rotated views of the output's gradient and of the down projection
            s |= {"a": _view(g, M, K, 1e-3), "w": _view(g, F, K, K ** -0.5), "gate": _randn(g, M, F).mul_(1.5).to(bf), "up": _randn(g, M, F).to(bf),
                  "dgate": new(), "dup": new(), "h": new()}
    elif op in ("rope", "rope_bwd"):
        T, Hq, Hk, D, R, dx = case["T"], case["Hq"], case["Hk"], case["D"], case["R"], _DTYPE[case["x"]]
        H, P = Hq + Hk, _table(case)
        x = _randn(g, T, Hq + 2 * Hk, D)  # queries, keys and values of a token side by side
        x[:, :, ::17] *= 6.0  # a few channels carry large values
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float64) / (R // 2))
        # sequences of P tokens one behind the other, from somewhere in the first one on
        start = torch.randint(0, P, (1,), generator=g, device="cuda")
        s |= {"x": x.to(dx), "wq": (1 + 0.1 * _randn(g, D)).to(_DTYPE[case["w"]]), "wk": (1 + 0.1 * _randn(g, D)).to(_DTYPE[case["w"]]),
              "pos": (start + torch.arange(T, device="cuda")) % P, "cos": angle.cos().float(), "sin": angle.sin().float()}
        if op == "rope":
            s["y"] = torch.empty((T, H, D), dtype=dx, device="cuda")
        else:  # the gradient goes where the values' gradient is already
            s |= {"dy": _randn(g, T, H, D).mul_(1e-2).to(dx), "dx": torch.zeros_like(s["x"]), "dwq": torch.empty_like(s["wq"]), "dwk": torch.empty_like(s["wk"])}
    else:
        sizes, B = _sizes(case), case["pack"]
        rows = [-(-n // B) for n in sizes]  # each tensor takes whole rows of B elements of the flat arrays
        N = sum(rows) * B
        # the elements that are a tensor's, and not what fills its last row up
        live = torch.ones((N // B, B), dtype=torch.bool, device="cuda")
        if B > 1:
            ends = torch.tensor(rows, device="cuda").cumsum(0) - 1
            left = (torch.tensor(sizes, device="cuda") - 1) % B
            live[ends] = torch.arange(B, device="cuda") <= left[:, None]
        live = live.view(-1)
        f = lambda std: _randn(g, N).mul_(std).mul_(live)  # noqa: E731
        p, grad = f(0.02), f(1e-3)
        low = case["kind"] != "f32"
        s |= {"rows": torch.tensor(rows, device="cuda"), "p": p.to(torch.bfloat16) if low else p, "g": grad.to(torch.bfloat16) if low else grad,
              "master": p if case["kind"] == "master" else None}
        # states of a run under way: gradients of the same size, averaged
        m, r = f(3e-4), f(1e-3).abs_().add_(live * 2e-4)
        if case["state"] == "f32":
            s |= {"m": m, "v": r.square_(), "ms": None, "vs": None}
        else:
            for k, t in (("m", m), ("v", r)):  # v's codes stand for its root
                top = t.view(-1, B).abs().amax(1) / 448
                s[k] = (t.view(-1, B) / top.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)
                s[k + "s"] = top
        # matrices decay, vectors do not
        wd = [0.1 if n > 10000 else 0.0 for n in sizes]
        at, spans = 0, []
        for n, r in zip(sizes, rows):
            spans.append((at, at + n))
            at += r * B
        s |= {"wd": torch.tensor(wd, device="cuda"), "wds": wd, "spans": spans, "rows_list": rows, "lr": torch.full((1,), 3e-4, device="cuda"),
              "step": torch.full((1,), 1000, dtype=torch.int64, device="cuda"), "norm": grad.double().square().sum().sqrt().float().reshape(1)}
    return s


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _decode(view):
    """The values of a view without its tensor's scale, exact in fp32."""
    codes, scales, _ = view
    R, C = codes.shape[0], 2 * codes.shape[1]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    x = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], 2).view(R, C // 16, 16)
    s = scales.view(R // 128, C // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, C // 16).view(torch.float8_e4m3fn)
    return x.mul_(s.float()[:, :, None]).view(R, C)


def _sigmoid(act, x):
    """act(x) = x s, and act'(x): s, and by how much s rises with x, for SiLU and GELU (tanh)."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s, s * (1 - s)
    c = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-c * (x + 0.044715 * x * x * x)))
    return s, s * (1 - s) * c * (1 + 3 * 0.044715 * x * x)


def _halves(x, R, pairs):
    """The two members of each rotated pair, and what is not rotated."""
    if pairs:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _joined(a, b, rest, pairs):
    if pairs:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _mulhilo(a, b):
    """High and low 32 bits of the product of a constant and 32-bit numbers held in 64."""
    low = a * (b & 0xFFFF)
    mid = a * (b >> 16) + (low >> 16)
    return mid >> 16, (mid & 0xFFFF) << 16 | low & 0xFFFF


def _philox(c, seed):
    """Philox4x32-10 of the counters c (four arrays) under the 64-bit key."""
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(0xD2511F53, c[0])
        h1, l1 = _mulhilo(0xCD9E8D57, c[2])
        c = (h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0)
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def _to_e4m3(x, draws):
    """Rows of x in E4M3, rounded up or down by 16-bit draws, and the rows' scales."""
    top = x.abs().amax(1, keepdim=True)
    zero = top < 2.0 ** -100
    most = torch.full_like(top, 448)  # by an array: by a number, torch multiplies with a reciprocal
    a = x.abs() * torch.where(zero, 0.0, most / top)
    lift = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)  # below the normal numbers the step stays that of the smallest of them
    bits = (a + lift).view(torch.int32) + (draws << 4).int() & ~0xFFFFF
    a = (bits.view(torch.float32) - lift).clamp_(max=448)
    return torch.where(x < 0, -a, a).to(torch.float8_e4m3fn), torch.where(zero, 0.0, top / most)


def _plain(s):
    op, case = s["op"], s["case"]
    if op == "gated":
        a = _decode(s["a"])
        gate = (a @ _decode(s["gate_w"]).T).mul_(s["a"][2] * s["gate_w"][2])
        up = (a @ _decode(s["up_w"]).T).mul_(s["a"][2] * s["up_w"][2])
        h = (gate * _sigmoid(case["act"], gate)[0] * up).to(torch.bfloat16)
        return {"h": h, "gate": gate.to(h.dtype), "up": up.to(h.dtype)} if case["keep"] else {"h": h}
    if op == "gated_bwd":
        dh = (_decode(s["a"]) @ _decode(s["w"]).T).mul_(s["a"][2] * s["w"][2] * 2.0 ** -7)
        gate, up = s["gate"].float(), s["up"].float()
        sig, rise = _sigmoid(case["act"], gate)
        out = {"dgate": dh * up * (sig + gate * rise), "dup": dh * gate * sig, "h": gate * sig * up}
        return {k: v.to(torch.bfloat16) for k, v in out.items()}
    if op in ("rope", "rope_bwd"):
        Hq, H, R, pairs = case["Hq"], case["Hq"] + case["Hk"], case["R"], case["pairs"]
        x = s["x"][:, :H].float()
        r = torch.rsqrt((x * x).mean(2, keepdim=True) + EPS)
        cos, sin = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
        w = torch.cat([s["wq"].float().expand(Hq, -1), s["wk"].float().expand(H - Hq, -1)])
        if op == "rope":
            a, b, rest = _halves(x * r * w, R, pairs)
            return _joined(a * cos - b * sin, b * cos + a * sin, rest, pairs).to(s["x"].dtype)
        a, b, rest = _halves(s["dy"].float(), R, pairs)
        da, n = _joined(a * cos + b * sin, b * cos - a * sin, rest, pairs), x * r
        dw = da * n
        dn = da * w
        dx = r * (dn - n * (dn * n).mean(2, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dwq": dw[:, :Hq].sum((0, 1)).to(s["wq"].dtype), "dwk": dw[:, Hq:].sum((0, 1)).to(s["wk"].dtype)}
    B = case["pack"]
    tensor = torch.repeat_interleave(torch.arange(case["n"], device="cuda"), s["rows"])  # of each row
    wd = s["wd"][tensor][:, None]
    t = s["step"].double()
    c1, c2 = (1 / (1 - BETA1 ** t)).float(), (1 / (1 - BETA2 ** t)).sqrt().float()
    clip = (MAX_NORM / (s["norm"] + 1e-6)).clamp(max=1.0)
    g = s["g"].view(-1, B).float() * clip
    m, v = s["m"].view(-1, B).float(), s["v"].view(-1, B).float()
    if case["state"] == "e4m3":
        m, v = m * s["ms"][:, None], (v * s["vs"][:, None]).square()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    root = v.sqrt()
    weights = s["p"] if s["master"] is None else s["master"]
    p = weights.view(-1, B).float()
    p = p - s["lr"] * wd * p - s["lr"] * c1 * m / (root * c2 + ADAM_EPS)
    weights.copy_(p.view(-1))
    if s["master"] is not None:
        s["p"].copy_(p.view(-1))
    if case["state"] == "f32":
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
    else:  # 16 bits of an element's word for m and 16 for v
        first = s["rows"].cumsum(0) - s["rows"]
        group = (torch.arange(len(tensor), device="cuda") - first[tensor])[:, None] * (B // 4) + torch.arange(B // 4, device="cuda")
        zero = torch.zeros_like(group)
        word = torch.stack(_philox((group, zero, zero + tensor[:, None], zero + s["step"]), SEED), 2).view(-1, B)
        for k, x, draws in (("m", m, word & 0xFFFF), ("v", root, word >> 16)):
            codes, scale = _to_e4m3(x, draws)
            s[k].copy_(codes.view(-1))
            s[k + "s"].copy_(scale[:, 0])
    return _updated(s)


def _updated(s):
    return {k: s[k] for k in ("p", "master", "m", "v", "ms", "vs") if s[k] is not None}


def _own(s):
    from nvfp4_quantized_b200 import qt2, qt2_train as tr
    op, case = s["op"], s["case"]
    if op in ("gated", "gated_bwd"):
        M, K, F = case["M"], case["K"], case["F"]
        act = tr.QT2_ACT_SILU if case["act"] == "silu" else tr.QT2_ACT_GELU_TANH
        if op == "gated":
            tr.qt2_gemm_nvfp4_gated(qt2.View(*s["a"]), qt2.View(*s["gate_w"]), qt2.View(*s["up_w"]), M, F, K, 1.0, act, s["gate"], s["up"], F, s["h"], F)
            return {k: s[k] for k in ("h", "gate", "up") if s[k] is not None}
        tr.qt2_gemm_nvfp4_gated_bwd(qt2.View(*s["a"]), qt2.View(*s["w"]), M, F, K, 2.0 ** -7, act, s["gate"], s["up"], F, s["dgate"], s["dup"], F, s["h"], F)
        return {k: s[k] for k in ("dgate", "dup", "h")}
    if op in ("rope", "rope_bwd"):
        T, Hq, Hk, D, R = case["T"], case["Hq"], case["Hk"], case["D"], case["R"]
        x, P, pairing = s["x"], s["cos"].shape[0], tr.QT2_ROPE_PAIRS if case["pairs"] else tr.QT2_ROPE_HALVES
        if op == "rope":
            tr.qt2_qk_norm_rope_fwd(x, T, Hq, Hk, D, x.stride(0), D, s["wq"], s["wk"], EPS, s["pos"], s["cos"], s["sin"], P, R, pairing,
                                    s["y"], s["y"].stride(0), D)
            return s["y"]
        if "ws" not in s:
            s["ws"] = qt2.alloc_workspace(tr.qt2_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, D))
        tr.qt2_qk_norm_rope_bwd(s["dy"], s["dy"].stride(0), D, x, T, Hq, Hk, D, x.stride(0), D, s["wq"], s["wk"], EPS, s["pos"], s["cos"], s["sin"],
                                P, R, pairing, s["dx"], x.stride(0), D, s["dwq"], s["dwk"], s["ws"], s["ws"].numel())
        return {"dx": s["dx"][:, :Hq + Hk], "dwq": s["dwq"], "dwk": s["dwk"]}
    if "list" not in s:
        parts = lambda t: None if t is None else [t[a:b] for a, b in s["spans"]]  # noqa: E731
        scales = lambda t: None if t is None else list(t.split(s["rows_list"]))  # noqa: E731
        s["list"] = tr.AdamWList(parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]), parts(s["master"]), scales(s["ms"]), scales(s["vs"]), s["wds"])
    tr.qt2_adamw(s["list"], s["lr"], s["step"], BETA1, BETA2, ADAM_EPS, s["norm"], MAX_NORM, SEED)
    return _updated(s)


# ------------------------------------------------------------------------------------------- in 64 bits
def _values(view):
    """A view's values in 64 bits, from its nibbles' sign, exponent and mantissa and its scales' bits."""
    codes, scales, scale = view
    R, C = codes.shape[0], 2 * codes.shape[1]
    n = torch.arange(C, device="cuda")
    nib = (codes.long()[:, n // 2] >> (n % 2 * 4)) & 15
    e, m = nib >> 1 & 3, (nib & 1).double()
    x = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).double()) * (1 - 2 * (nib >> 3)).double()
    r, j = torch.arange(R, device="cuda")[:, None], torch.arange(C // 16, device="cuda")
    at = ((r // 128) * (C // 64) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    b = scales.long()[at]
    e, m = b >> 3, (b & 7).double() / 8
    return x * torch.where(e == 0, m * 2.0 ** -6, (1 + m) * 2.0 ** (e - 7).double()).repeat_interleave(16, 1) * scale.double()


def _act(act, x):
    """act(x) and its derivative, through tanh."""
    if act == "silu":
        t = torch.tanh(x / 2)
        return x * (1 + t) / 2, (1 + t) / 2 + x * (1 - t * t) / 4
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return x * (1 + t) / 2, (1 + t) / 2 + x * (1 - t * t) * c * (1 + 0.134145 * x * x) / 2


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gated":
        a = _values(s["a"])
        gate, up = a @ _values(s["gate_w"]).T, a @ _values(s["up_w"]).T
        h = _act(case["act"], gate)[0] * up
        return {"h": h, "gate": gate, "up": up} if case["keep"] else {"h": h}
    if op == "gated_bwd":
        dh = _values(s["a"]) @ _values(s["w"]).T / 128
        f, d = _act(case["act"], s["gate"].double())
        return {"dgate": dh * d * s["up"].double(), "dup": dh * f, "h": f * s["up"].double()}
    if op in ("rope", "rope_bwd"):
        return _exact_rope(case, s)
    # one tensor after the other
    lr, t, clip = float(s["lr"]), int(s["step"]), min(1.0, MAX_NORM / (float(s["norm"]) + 1e-6))
    out = {k: v.double() for k, v in _updated(s).items()}
    at = 0
    for rows, wd in zip(s["rows_list"], s["wds"]):
        part = slice(at * case["pack"], (at + rows) * case["pack"])
        g, m, v = s["g"][part].double() * clip, out["m"][part], out["v"][part]
        if case["state"] == "e4m3":
            each = lambda k: out[k][at:at + rows].repeat_interleave(case["pack"])  # noqa: E731
            m, v = m * each("ms"), (v * each("vs")) ** 2
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g ** 2
        p = (s["p"] if s["master"] is None else s["master"])[part].double()
        p = (1 - lr * wd) * p - lr * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + ADAM_EPS)
        out["p"][part] = p
        if "master" in out:
            out["master"][part] = p
        if case["state"] == "f32":
            out["m"][part], out["v"][part] = m, v
        else:
            for k, x in (("ms", m), ("vs", v.sqrt())):
                out[k][at:at + rows] = x.abs().view(rows, -1).amax(1) / 448
        at += rows
    if case["state"] == "e4m3":  # which of its two neighbours a code is depends on the last bits of its value
        out["m"] = out["v"] = None
    return out


def _exact_rope(case, s):
    """Pairs as complex numbers."""
    Hq, H, R, D = case["Hq"], case["Hq"] + case["Hk"], case["R"], case["D"]
    i = torch.arange(R // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + R // 2)
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"]]

    def rotate(x, turn):
        z = torch.complex(x[:, first], x[:, second]) * turn
        x = x.clone()
        x[:, first], x[:, second] = z.real, z.imag
        return x
    out = {"dx": torch.empty((case["T"], H, D), dtype=torch.float64, device="cuda")}
    dw = {"wq": 0.0, "wk": 0.0}
    for h in range(H):
        x, k = s["x"][:, h].double(), "wq" if h < Hq else "wk"
        w, rms = s[k].double(), (x.square().sum(1, keepdim=True) / D + EPS).sqrt()
        if case["op"] == "rope":
            out["dx"][:, h] = rotate(x / rms * w, turn)
            continue
        up = rotate(s["dy"][:, h].double(), turn.conj())
        dw[k] = dw[k] + (up * x / rms).sum(0)
        # the quotient's two ways: x itself and its root mean square
        out["dx"][:, h] = up * w / rms - x * (up * w * x).sum(1, keepdim=True) / (D * rms ** 3)
    if case["op"] == "rope":
        return out["dx"]
    zero = torch.zeros(D, dtype=torch.float64, device="cuda")
    return {"dx": out["dx"], "dwq": zero + dw["wq"], "dwk": zero + dw["wk"]}
