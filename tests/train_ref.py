"""Plain 64-bit implementations of the training operators and the error bounds that the kernels'
arithmetic allows (u = 2^-24, the half step of fp32; an output type adds half a step of its own)."""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rows_like(R, C, dtype, device="cuda", pad=0, fill=None):
    """[R, C] view with a leading dimension that is a multiple of 8 (plus pad), and its whole buffer."""
    ld = (C + 7) // 8 * 8 + pad
    buf = torch.empty((R, ld), dtype=dtype, device=device)
    if fill is not None:
        buf.fill_(fill)
    return buf[:, :C], buf


# ------------------------------------------------------------------------------------------ layer norm
def norm_fwd(x, w, b, eps):
    """(y, mean, rstd) in 64 bits and bounds on the errors of the three."""
    x = x.double()
    R, C = x.shape
    w = torch.ones(C, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(C, dtype=torch.float64, device=x.device) if b is None else b.double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    d = x - mean
    h = d * rstd
    y = h * w + b
    depth = math.ceil(C / 32) + 16   # additions that any term of a row's sum passes through
    e_mean = depth * U * x.abs().mean(1, keepdim=True) + U * mean.abs()
    e_d = e_mean + U * d.abs()
    e_var = (2 * d.abs() * e_d + e_d ** 2).mean(1, keepdim=True) + (depth + 3) * U * var
    rel_r = e_var / (var + eps) + 4 * U   # half of this to first order; doubled for the higher orders
    rel_r = torch.where(var + eps > 0, rel_r, torch.zeros_like(rel_r))
    e_h = rstd * e_d * (1 + rel_r) + h.abs() * (rel_r + 2 * U)
    e_y = w.abs() * e_h + U * (2 * (h * w).abs() + y.abs())
    return (y, mean[:, 0], rstd[:, 0]), (e_y, e_mean[:, 0], (rstd * rel_r)[:, 0])


def norm_bwd(dy, x, w, mean, rstd, row_depth):
    """(dx, dw, db) in 64 bits from the statistics that were kept, and bounds; row_depth: additions
    that any term of a sum over the rows passes through."""
    dy, x, m, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    C = x.shape[1]
    w = torch.ones(C, dtype=torch.float64, device=x.device) if w is None else w.double()
    h, a = (x - m) * r, dy * w
    s, q = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    dx = r * (a - s - h * q)
    depth = math.ceil(C / 32) + 16
    e_h = 3 * U * h.abs()
    e_s = (depth + 2) * U * a.abs().mean(1, keepdim=True)
    e_q = (depth + 7) * U * (a * h).abs().mean(1, keepdim=True)
    big = a.abs() + s.abs() + (h * q).abs()
    e_dx = r * (U * a.abs() + e_s + h.abs() * e_q + e_h * q.abs() + 4 * U * big)
    dw, db = (dy * h).sum(0), dy.sum(0)
    e_dw = ((dy * h).abs().sum(0)) * (row_depth + 5) * U
    e_db = dy.abs().sum(0) * (row_depth + 1) * U
    return (dx, dw, db), (e_dx, e_dw, e_db)


# ------------------------------------------------------------------------------------------ head loss
def xent(x, w, targets, ignore, dloss=None):
    """loss, lse (and dx, dw) in 64 bits with bounds.

    Logits: exact bf16 products, added up in fp32 16 at a time by the tensor cores, with at most a
    whole step (2^-23) lost an addition.  exp and log: 2^-21 relative to the arguments' magnitude
    and result.  P is rounded to bf16; its rounding errors (at most half a step each, uniform,
    independent) add up over a sum like their root sum of squares: 8 standard deviations allowed."""
    x, w = x.double(), w.double()
    (T, K), V = x.shape, w.shape[0]
    l = x @ w.T
    e_l = 2 * U * (K / 16 + 16) * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(l, 1)
    valid = (targets != ignore) & (targets >= 0) & (targets < V)
    at = targets.clamp(0, V - 1)
    hit = l.gather(1, at[:, None])[:, 0]
    loss = torch.where(valid, lse - hit, 0.0)
    top = l.abs().amax(1)
    e_lse = e_l.amax(1) + (top + lse.abs() + 8) * 2.0 ** -21
    e_loss = torch.where(valid, e_lse + e_l.gather(1, at[:, None])[:, 0] + U * loss.abs(), 0.0)
    if dloss is None:
        return (loss, lse), (e_loss, e_lse)
    g = torch.where(valid, dloss.double(), 0.0)[:, None]
    p = torch.exp(l - lse[:, None])
    P = p.clone()
    P.scatter_add_(1, at[:, None], -torch.ones(T, 1, dtype=P.dtype, device=P.device))
    P *= g
    e_P = g.abs() * (p * (e_l + e_lse[:, None] + (l.abs() + lse.abs()[:, None] + 8) * 2.0 ** -21) + 4 * U)
    e_P = torch.where(g == 0, 0.0, e_P)
    half = half_step(torch.bfloat16)
    sigma = half / math.sqrt(3.0)
    dx, dw = P @ w, P.T @ x
    e_dx = 8 * sigma * torch.sqrt((P ** 2) @ (w ** 2)) + e_P @ w.abs() + 2 * U * (V / 16 + 64) * (P.abs() @ w.abs())
    e_dw = 8 * sigma * torch.sqrt((P ** 2).T @ (x ** 2)) + e_P.T @ x.abs() + 2 * U * (T / 16 + 16) * (P.abs().T @ x.abs())
    return (loss, lse, dx, dw), (e_loss, e_lse, e_dx, e_dw)


def check(got, want, bound, what=""):
    """|got - want| within the bound plus half a step of got's type (and its smallest normal)."""
    tol = bound + half_step(got.dtype) * (want.abs() + bound) + torch.finfo(got.dtype).tiny
    err = (got.double() - want).abs()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert torch.isfinite(err).all() and worst <= 1.0, (what, worst, err.max().item())
