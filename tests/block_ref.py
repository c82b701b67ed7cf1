"""Plain 64-bit implementations of a transformer block's operators (gated product, norm of queries and keys
with rotation, AdamW) and the error bounds that the kernels' arithmetic allows (u = 2^-24, the half step
of fp32; an output type adds half a step of its own: train_ref.check)."""
import math

import torch

U = 2.0 ** -24
SILU, GELU = 0, 1


# ------------------------------------------------------------------------------------------ views
def random_view(R, C, seed, scale=1.0, device="cuda"):
    """(codes, scales, tensor_scale) of an [R, C] view: every code, E4M3 scales from 2^-4 to 8 and some zeros."""
    g = torch.Generator(device=device).manual_seed(seed)
    codes = torch.randint(0, 256, (R, C // 2), generator=g, device=device, dtype=torch.uint8)
    scales = torch.randint(0x18, 0x51, (R * C // 16,), generator=g, device=device, dtype=torch.uint8)
    scales[torch.rand(scales.shape, generator=g, device=device) < 0.02] = 0
    return codes, scales, torch.full((1,), scale, device=device)


def view_values(codes, scales, tensor_scale):
    """The elements' values in 64 bits."""
    R, C = codes.shape[0], 2 * codes.shape[1]
    dev = codes.device
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=dev)
    nib = torch.stack([codes & 15, codes >> 4], 2).view(R, C).long()
    x = grid[nib & 7] * (1 - 2 * (nib >> 3)).double()
    r, j = torch.arange(R, device=dev)[:, None], torch.arange(C // 16, device=dev)
    at = ((r // 128) * (C // 64) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    s = scales[at].view(torch.float8_e4m3fn).double()
    return x * s.repeat_interleave(16, 1) * tensor_scale.double()


# ------------------------------------------------------------------------------------------ gated product
def act(kind, x):
    """(act(x), act'(x), exponent) in 64 bits."""
    if kind == SILU:
        t, dt = x, torch.ones_like(x)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        t, dt = c * (x + 0.044715 * x ** 3), c * (1 + 3 * 0.044715 * x ** 2)
    s = torch.sigmoid(t)
    return x * s, s + x * s * torch.sigmoid(-t) * dt, t


def act_bounds(kind, x):
    """Errors of act and act' computed in fp32 from x.

    exp(-t): the argument's roundings (at most six) and log2(e)'s, and 2 units of ex2: relative (8 |t| + 4) u;
    s = 1 / (1 + e): e / (1 + e) of it, the sum's rounding and 2 units of the division: at most d below.
    1 - s is off by s d' where d' is that error and its own rounding u, and in act' it meets x and dt."""
    f, df, t = act(kind, x)
    s, dt = torch.sigmoid(t), (torch.ones_like(t) if kind == SILU else 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * x ** 2))
    t = t.clamp(-90, 90)
    d = (torch.sigmoid(-t) * (8 * t.abs() + 4) + 6) * U
    tiny = x.abs() * 1e-37   # exp(-t) past fp32: s = 0 (SiLU below -88, GELU from the clamp at -10 on)
    e_f = f.abs() * (d + 2 * U) + tiny
    far = torch.where(x.abs() > 10, torch.zeros_like(x), dt)
    e_df = s * d + x.abs() * s * (torch.sigmoid(-t) * (d + 6 * U) + s * d + U) * (dt if kind == SILU else far) + 2 * U * df.abs() + tiny
    return e_f, e_df


def _product(a, b, alpha, K):
    """a b^T, and what fp32 sums of the tensor cores (at most a whole step lost each time 16 products join) are off by."""
    z = alpha * (a @ b.T)
    return z, alpha * (2 * U * (K / 16 + 16) * (a.abs() @ b.abs().T)) + 4 * U * z.abs()


def gated_fwd(a, bg, bu, alpha, kind):
    """(h, g, u) and bounds, from the operands' values."""
    K = a.shape[1]
    g, e_g = _product(a, bg, alpha, K)
    u, e_u = _product(a, bu, alpha, K)
    f, df, _ = act(kind, g)
    e_f = act_bounds(kind, g)[0] + e_g * (df.abs() + 0.1) + e_g ** 2   # |act''| is below 1.6
    return (f * u, g, u), (e_f * u.abs() + (f.abs() + e_f) * e_u + 3 * U * (f * u).abs(), e_g, e_u)


def gated_bwd(a, b, alpha, kind, gate, up):
    """(dgate, dup, h) and bounds."""
    dh, e_dh = _product(a, b, alpha, a.shape[1])
    g, u = gate.double(), up.double()
    f, df, _ = act(kind, g)
    e_f, e_df = act_bounds(kind, g)
    dg, du, h = dh * u * df, dh * f, f * u
    e_dg = e_dh * (u * df).abs() + (dh.abs() + e_dh) * u.abs() * e_df + 3 * U * dg.abs()
    return (dg, du, h), (e_dg, e_dh * f.abs() + (dh.abs() + e_dh) * e_f + 2 * U * du.abs(), e_f * u.abs() + 2 * U * h.abs())


# ------------------------------------------------------------------------------------------ queries and keys
def tables(P, R, base=1e4, device="cuda"):
    """cos and sin [P, R/2] of p / base^(2 i / R), rounded to fp32 from 64 bits."""
    i = torch.arange(R // 2, dtype=torch.float64, device=device)
    angle = torch.arange(P, dtype=torch.float64, device=device)[:, None] / base ** (2 * i / max(1, R))
    return angle.cos().float(), angle.sin().float()


def _pairs(R, pairs, device):
    i = torch.arange(R // 2, device=device)
    return (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)


def _turn(x, cos, sin, R, pairs, sign):
    """x [T, H, D] with its pairs turned by cos, sin [T, R/2]; and |x|'s sum in each element."""
    p, q = _pairs(R, pairs, x.device)
    y, size = x.clone(), x.abs()
    c, s = cos[:, None], sign * sin[:, None]
    y[..., p], y[..., q] = x[..., p] * c - x[..., q] * s, x[..., q] * c + x[..., p] * s
    size[..., p], size[..., q] = (x[..., p] * c).abs() + (x[..., q] * s).abs(), (x[..., q] * c).abs() + (x[..., p] * s).abs()
    return y, size


def _weights(wq, wk, Hq, Hk, D, device):
    one = torch.ones(D, dtype=torch.float64, device=device)
    return torch.cat([(one if w is None else w.double()).expand(n, D) for w, n in ((wq, Hq), (wk, Hk))])


def qk_fwd(x, Hq, wq, wk, eps, cos, sin, R, pairs):
    """y [T, H, D] in 64 bits and its bound, x [T, H, D] and cos, sin [T, R/2] of the tokens' positions.

    Sum of squares: no term passes more than D/32 + 16 additions; rsqrt 4 u; two products and the turn's three
    roundings."""
    x = x.double()
    T, H, D = x.shape
    w = _weights(wq, wk, Hq, H - Hq, D, x.device)
    r = 1 / torch.sqrt(x.square().mean(2, keepdim=True) + eps)
    y, size = _turn(x * r * w, cos.double(), sin.double(), R, pairs, 1)
    return y, size * (D / 64 + 8 + 4 + 2 + 3 + 1) * U


def qk_bwd(dy, x, Hq, wq, wk, eps, cos, sin, R, pairs, row_depth):
    """(dx, dwq, dwk) and bounds; row_depth: additions that any term of a sum over tokens and heads passes."""
    x, dy = x.double(), dy.double()
    T, H, D = x.shape
    w = _weights(wq, wk, Hq, H - Hq, D, x.device)
    r = 1 / torch.sqrt(x.square().mean(2, keepdim=True) + eps)
    b, size = _turn(dy, cos.double(), sin.double(), R, pairs, -1)
    n = x * r
    mean = (b * w * n).mean(2, keepdim=True)
    dx = r * (b * w - n * mean)
    depth, e_r = D / 32 + 16, (D / 64 + 13) * U
    e_mean = (size * w.abs() * n.abs()).mean(2, keepdim=True) * ((depth + 9) * U + e_r)
    big = size * w.abs() + n.abs() * mean.abs()
    e_dx = r * (size * w.abs() * 5 * U + n.abs() * e_mean + big * (e_r + 4 * U)) + dx.abs() * e_r
    dw = b * n
    e_dw = size * n.abs() * ((row_depth + 6) * U + e_r)
    return ((dx, dw[:, :Hq].sum((0, 1)), dw[:, Hq:].sum((0, 1))), (e_dx, e_dw[:, :Hq].sum((0, 1)), e_dw[:, Hq:].sum((0, 1))))


# ------------------------------------------------------------------------------------------ AdamW
def adamw(p, g, m, v, lr, step, b1, b2, eps, decay, clip):
    """(p, m, v) after a step in 64 bits, and bounds.  m, v: what the states stand for; clip: the factor (64 bits).

    The factor is off by 3 u; m and v have a product's rounding on either side and the sum's; the update's
    quotient: root, correction, sum, rate, product and a division of 2 units."""
    p, g, m, v = (t.double() for t in (p, g, m, v))
    h = g * clip
    e_h = 4 * U * h.abs()
    m1, v1 = b1 * m + (1 - b1) * h, b2 * v + (1 - b2) * h * h
    # b and 1 - b rounded to fp32, the products, the sum
    e_m = 3 * U * (b1 * m).abs() + (1 - b1) * (e_h + 2 * U * h.abs()) + U * m1.abs()
    e_v = 3 * U * b2 * v + (1 - b2) * (2 * e_h * h.abs() + 3 * U * h * h) + U * v1 + 2.0 ** -148
    c1, c2 = 1 / (1 - b1 ** step), math.sqrt(1 / (1 - b2 ** step))
    root = v1.sqrt()
    # the root's own relative error: half of v's, or where v is nearly nothing what it may be at most
    e_root = torch.minimum(e_v / root.clamp(min=1e-300), e_v.sqrt()) + U * root
    den = root * c2 + eps
    up = lr * c1 * m1 / den
    e_up = lr * c1 * e_m / den + up.abs() * (c2 * e_root / den * 1.5 + 8 * U)
    p1 = p - lr * decay * p - up
    return (p1, m1, v1), (3 * U * (lr * decay * p).abs() + U * p.abs() + U * p1.abs() + e_up * 1.001, e_m, e_v)


def philox(counter, seed):
    """Words [n, 4] of Philox4x32-10 at counters [n, 4] (numpy, as published)."""
    import numpy as np
    c = [np.asarray(counter[:, i], dtype=np.uint64) for i in range(4)]
    k = [np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32 & 0xFFFFFFFF)]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & low, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(c, 1)


def e4m3_neighbours(x):
    """The E4M3 numbers at or next below and next above |x| <= 448 (64 bits)."""
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    i = torch.searchsorted(grid, x.abs().contiguous(), right=True) - 1
    return grid[i], grid[(i + 1).clamp(max=126)]
