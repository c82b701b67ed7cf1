"""Values at the ends of the types' ranges, where the formulas still have an answer."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref
from tests.test_gpu_xent import BF, FP, backward, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V", [(5, 700), (40, 700), (40, 1), (20, 30000)])
def test_infinite_logits(T, V):
    """A logit of +inf makes lse inf, and the loss too unless the target's own is inf (inf - inf); where all
    are -inf the sum of the exponentials is 0 and lse -inf.  Other rows stay."""
    K, inf = 64, float("inf")
    x, w, y, dloss = make(T, K, V, seed=T + V, ignored=0.0)
    up = V - 1
    w[:, 0] = -1.0
    w[up, 0] = 1.0
    w[:, 1] = -1.0
    y[:] = 0
    y[2] = up
    loss0, lse0 = forward(x, w, y)
    x[1:3, 0], x[3, 1] = inf, inf
    loss, lse = forward(x, w, y)
    assert (lse[1:3] == inf).all() and lse[3] == -inf
    assert (loss[1] == inf if V > 1 else loss[1].isnan()) and loss[2].isnan() and loss[3].isnan()
    keep = torch.arange(T, device="cuda") > 3
    keep[0] = True
    assert torch.equal(lse[keep], lse0[keep]) and torch.equal(loss[keep], loss0[keep])
    assert (torch.logsumexp(x.double() @ w.double().T, 1)[1:4] == lse[1:4]).all()
    dx, _ = backward(x, w, y, lse, dloss)
    assert torch.isfinite(dx[keep]).all()


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("C", [40, 200, 500, 1000, 2000, 4000, 8000, 16000, 20000])
def test_layernorm_backward_of_small_and_large_rows(C, dtype):
    """Rows of deviation 2^-80 and 2^60: rstd is far from 1, its cube outside fp32, and dx = rstd (...) within it."""
    for scale, up in ((2.0 ** -80, 1.0), (2.0 ** 60, 2.0 ** -20)):
        R = 6
        g = torch.Generator(device="cuda").manual_seed(C)
        x, dy = ref.rows_like(R, C, dtype)[0], ref.rows_like(R, C, dtype)[0]
        x.copy_(torch.randn((R, C), generator=g, device="cuda") * scale)
        dy.copy_(torch.randn((R, C), generator=g, device="cuda") * up)
        w = 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
        var, m = torch.var_mean(x.double(), 1, correction=0)
        mean, rstd = m.float(), var.rsqrt().float()
        dx = ref.rows_like(R, C, dtype)[0]
        dw, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
        ws = torch.empty(tr.qt2_layernorm_bwd_workspace_size(R, C), dtype=torch.uint8, device="cuda")
        tr.qt2_layernorm_bwd(dy, dy.stride(0), x, R, C, x.stride(0), w, mean, rstd, dx, dx.stride(0), dw, db, ws, ws.numel())
        want, bound = ref.norm_bwd(dy, x, w, mean, rstd, 96 + R)
        for name, a, b, e in zip(("dx", "dw", "db"), (dx, dw, db), want, bound):
            ref.check(a, b, e, (name, scale))
