"""Training operators whose arrays pass 2^31 elements (offsets of more than 32 bits), checked on
rows and slices at both ends."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref
from tests.test_gpu_grad import REL

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def test_layernorm_rows_beyond_2_31_elements():
    R, C, ld = 70000, 2000, 32768
    assert R * ld > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(0)
    x, y, dx = (torch.empty((R, ld), dtype=BF, device="cuda") for _ in range(3))
    x[:, :C] = torch.randn((R, C), generator=g, device="cuda")
    dy = torch.randn((R, C), generator=g, device="cuda").to(BF)
    w, b = torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    tr.qt2_layernorm_fwd(x, R, C, ld, w, b, 1e-5, y, ld, mean, rstd)
    ws = qt2.alloc_workspace(tr.qt2_layernorm_bwd_workspace_size(R, C))
    dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    tr.qt2_layernorm_bwd(dy, C, x, R, C, ld, w, mean, rstd, dx, ld, dw, db, ws, ws.numel())
    for rows in (slice(0, 50), slice(R // 2, R // 2 + 50), slice(R - 50, R)):
        (wy, wm, wr), (ey, em, er) = ref.norm_fwd(x[rows, :C], w, b, 1e-5)
        ref.check(y[rows, :C], wy, ey)
        ref.check(mean[rows], wm, em)
        (wdx, _, _), (edx, _, _) = ref.norm_bwd(dy[rows], x[rows, :C], w, mean[rows], rstd[rows], 1)
        ref.check(dx[rows, :C], wdx, edx)
    want, size = dy.double().sum(0), dy.double().abs().sum(0)
    ref.check(db, want, size * (R // 64 + 96) * ref.U)


def test_head_loss_weights_beyond_2_31_elements():
    T, K, V = 40, 16384, 140000
    assert V * K > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, K), generator=g, device="cuda").to(BF)
    w = torch.empty((V, K), dtype=BF, device="cuda")
    for v in range(0, V, 20000):
        w[v:v + 20000] = torch.randn((20000, K), generator=g, device="cuda") * 0.01
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[:8] = torch.arange(V - 8, V, device="cuda")
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = qt2.alloc_workspace(max(tr.qt2_linear_xent_fwd_workspace_size(T, K, V),
                                 tr.qt2_linear_xent_bwd_workspace_size(T, K, V)))
    tr.qt2_linear_xent_fwd(x, w, y, T, K, V, K, K, -100, loss, lse, ws, ws.numel())
    tr.qt2_linear_xent_bwd(x, w, y, lse, dloss, T, K, V, K, K, -100, dx, K, dw, 0, K, ws, ws.numel())
    logits = torch.cat([x.double() @ w[v:v + 20000].double().T for v in range(0, V, 20000)], 1)
    e_l = 2 * ref.U * (K / 16 + 16) * x.double().abs().sum(1, keepdim=True) * w.abs().max().double()
    want = torch.logsumexp(logits, 1)
    bound = e_l[:, 0] + (logits.abs().amax(1) + want.abs() + 8) * 2.0 ** -21
    ref.check(lse, want, bound)
    ref.check(loss, want - logits.gather(1, y[:, None])[:, 0], 2 * bound)
    P = torch.exp(logits - want[:, None])
    P.scatter_add_(1, y[:, None], -torch.ones((T, 1), dtype=P.dtype, device="cuda"))
    P *= dloss.double()[:, None]
    for v in (0, V // 2, V - 64):   # rows of dw at both ends: rounding of P and of the result, and the logits' errors
        want_dw = P[:, v:v + 64].T @ x.double()
        size = P[:, v:v + 64].abs().T @ x.double().abs()
        ref.check(dw[v:v + 64], want_dw, size * (2.0 ** -8 + 4 * bound.max()))
    want_dx = sum(P[:, v:v + 20000] @ w[v:v + 20000].double() for v in range(0, V, 20000))
    size = sum(P[:, v:v + 20000].abs() @ w[v:v + 20000].double().abs() for v in range(0, V, 20000))
    ref.check(dx, want_dx, size * (2.0 ** -8 + 4 * bound.max()))


def test_gradient_beyond_2_31_elements():
    n = (1 << 31) + 12345
    t = torch.zeros(n + 3, dtype=BF, device="cuda")[3:]
    t[: 1 << 20] = 1.0
    t[-(1 << 20):] = 2.0
    small = torch.full((1000,), 3.0, device="cuda")
    out, so = torch.full_like(t, 7.0), torch.empty_like(small)
    gl = tr.GradList([t, small], [out, so])
    norm = torch.empty(1, device="cuda")
    ws = qt2.alloc_workspace(tr.qt2_grad_norm_workspace_size(gl))
    tr.qt2_grad_norm(gl, norm, ws, ws.numel())
    want = ((1 << 20) * 5 + 9000) ** 0.5
    assert abs(norm.item() - want) <= REL * want
    tr.qt2_grad_clip(gl, norm, want / 2)
    f = torch.tensor(want / 2, device="cuda") / (norm + 1e-6)
    one, two = (torch.tensor([v], device="cuda") * f for v in (1.0, 2.0))
    assert (out[: 1 << 20] == one.to(BF)).all() and (out[-(1 << 20):] == two.to(BF)).all()
    assert (out[1 << 20:-(1 << 20)] == 0).all() and torch.equal(so, small * f)
