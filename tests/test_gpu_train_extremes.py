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
