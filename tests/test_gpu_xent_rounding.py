"""How far the head's gradients are from 64 bits before the rounding of the output itself: in an fp32 dw
nothing hides it, and a 2-norm sees what a bound on single elements leaves room for.

Bounds, with sigma = 2^-8 / sqrt 3 the standard deviation of a rounding to bf16 (at most half a step of
2^-8 relative to the value, uniform): P's entries are rounded once, the target's is exact.  dw: c x is
rounded once more for products with P's other entries (sqrt 2 sigma together); for the target's entry it
is a sum of two bf16 numbers, off by 2^-16 at most.  dx: c multiplies the sums in fp32.  Sums and
exponentials as in train_ref.xent."""
import math

import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref
from tests.test_gpu_xent import BF, FP, IGN, backward, forward, make

pytestmark = pytest.mark.gpu
SIGMA = ref.half_step(BF) / math.sqrt(3.0)


def gradients(x, w, y, dloss):
    """(dx, dw) in 64 bits, the variances of their errors, and bounds of the errors that are no roundings to bf16."""
    x, w = x.double(), w.double()
    (T, K), V = x.shape, w.shape[0]
    l = x @ w.T
    e_l = 2 * ref.U * (K / 16 + 16) * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(l, 1)
    at, live = y.clamp(0, V - 1)[:, None], (y != IGN)[:, None]
    g = torch.where(live, dloss.double()[:, None], 0.0)
    e_lse = e_l.amax(1, keepdim=True) + (l.abs().amax(1, keepdim=True) + lse.abs()[:, None] + 8) * 2.0 ** -21
    p = torch.exp(l - lse[:, None])
    e_P = g * (p * (e_l + e_lse + (l.abs() + lse.abs()[:, None] + 8) * 2.0 ** -21) + 4 * ref.U)
    P = (p.scatter_add(1, at, -torch.ones_like(at, dtype=p.dtype))) * g
    dx, dw = P @ w, P.T @ x
    hit = P.gather(1, at)
    other = P.scatter(1, at, torch.zeros_like(hit)) ** 2
    at_target = torch.zeros_like(P).scatter(1, at, hit.abs())
    var_dx, var_dw = SIGMA ** 2 * (other @ w ** 2), 2 * SIGMA ** 2 * (other.T @ x ** 2)
    e_dx = e_P @ w.abs() + 2 * ref.U * (V / 16 + 64) * (P.abs() @ w.abs())
    e_dw = e_P.T @ x.abs() + 2 * ref.U * (T / 16 + 32) * (P.abs().T @ x.abs()) + 2.0 ** -16 * (at_target.T @ x.abs())
    return (dx, dw), (var_dx, var_dw), (e_dx, e_dw)


def rounding(want, dtype):
    """The squared rounding errors of `want` itself.  They are taken from it and not as a twelfth of the step's
    square: with one c for all rows an entry of dw is close to c x, x on the grid of bf16, and where c is
    (1 + d) 2^n, 0 <= d <= 2^-8, the errors c x - 2^n x = 2^n d x are all of one sign and size (d / 2^-7 of x's step
    at the lower end of an octave, twice that at its upper one: up to 1.95e-3 of the 2-norm, where independent ones
    have 1.6e-3 to 1.7e-3).  An error before the rounding moves a value over a tie, where the two are as far off."""
    return (want.to(dtype).double() - want) ** 2 if dtype is not FP else (ref.U * want) ** 2


def check_norm(got, want, var, bound, what):
    """The 2-norm of the errors: the root of the summed variances (many independent roundings: a tenth more
    allowed) and the 2-norm of the bounds of the rest."""
    err = (got.double() - want).norm().item()
    most = 1.1 * (var + rounding(want, got.dtype)).sum().sqrt().item() + bound.norm().item()
    assert err <= most, (what, err / want.norm().item(), most / want.norm().item())


# tokens, hidden size, vocabulary: one stage of tokens and several, ends inside a stage; vocabularies of few
# tiles (with many targets each) and of many (few have one); more tokens than a block sorts; two pieces
SHAPES = [(16, 512, 3000), (31, 130, 700), (64, 256, 5000), (65, 264, 20001), (300, 1000, 8000), (777, 500, 20000),
          (1024, 512, 257), (2048, 512, 8000), (2049, 72, 3001), (4500, 64, 2500), (8200, 72, 40000)]


@pytest.mark.parametrize("equal", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients_before_their_own_rounding(shape, equal):
    x, w, y, dloss = make(*shape, seed=sum(shape))
    if equal:   # a weight that lies almost half way between two bf16 numbers, in every row
        dloss.fill_((1 + 0.98 * 2.0 ** -8) / 1024)
    _, lse = forward(x, w, y)
    want, var, bound = gradients(x, w, y, dloss)
    for dwd in (FP, BF):
        dx, dw = backward(x, w, y, lse, dloss, dwd=dwd)
        for name, g, v, s, b in zip(("dx", "dw"), (dx, dw), want, var, bound):
            check_norm(g, v, s, b, (name, dwd))
            ref.check(g, v, 8 * s.sqrt() + b, (name, dwd))
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("T", [70, 2100])
def test_tokens_that_share_a_target(T):
    """One target for all tokens, and targets at the first and last entry of the vocabulary's tiles."""
    K, V = 200, 1500
    x, w, y, dloss = make(T, K, V, seed=T, ignored=0.0)
    for targets in (torch.full_like(y, 700), torch.tensor([0, 255, 256, 511, 1279, 1280, V - 1], device="cuda")[y % 7]):
        _, lse = forward(x, w, targets)
        dx, dw = backward(x, w, targets, lse, dloss, dwd=FP)
        want, var, bound = gradients(x, w, targets, dloss)
        for name, g, v, s, b in zip(("dx", "dw"), (dx, dw), want, var, bound):
            check_norm(g, v, s, b, name)


@pytest.mark.parametrize("K", [256, 1024, 4096, 16384])
@pytest.mark.parametrize("T", [8, 64])
def test_rows_that_one_entry_dominates(T, K):
    """Logits of about 40 whose products are all of one sign, as far from zero as sums of the tensor cores get.  Of the
    target: formed again in fp32, 2^-20 of it allowed.  Of another entry: what the sums lose, a step of 2^-23 for each of
    K / 16 additions and 16 more."""
    V = 3000
    g = torch.Generator(device="cuda").manual_seed(K + T)
    w = (torch.randn((V, K), generator=g, device="cuda") * 0.1).to(BF)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    for top, most in ((y, 2.0 ** -20), ((y + 1) % V, 2 * ref.U * (K / 16 + 16) + 2.0 ** -20)):
        x = (w[top].float() * (40 / (0.01 * K))).to(BF)
        l = x.double() @ w.double().T
        assert (l.amax(1) > 20 + l.topk(2, 1).values[:, 1]).all()   # nothing else counts
        loss, lse = forward(x, w, y)
        want = torch.logsumexp(l, 1)
        assert ((lse - want).abs() <= most * l.amax(1)).all()
        assert ((loss - (want - l.gather(1, y[:, None])[:, 0])).abs() <= most * l.amax(1)).all()


@pytest.mark.parametrize("T", [70, 2500])
def test_vocabulary_of_more_tiles_than_the_sort_takes_at_a_time(T):
    """dw's rows around tile 4096 and at both ends of 1.1 million entries, targets among them."""
    K, V = 16, 1100000
    x, w, y, dloss = make(T, K, V, seed=T)
    edge = 4096 * 256
    spans = ((0, 512), (edge - 300, edge + 300), (V - 600, V))
    for k, (lo, hi) in enumerate(spans):
        y[k::9] = lo + torch.arange(len(y[k::9]), device="cuda") * 7 % (hi - lo)
    _, lse = forward(x, w, y)
    _, dw = backward(x, w, y, lse, dloss, dwd=FP)
    at, live = y.clamp(min=0)[:, None], (y != IGN)[:, None]
    for lo, hi in spans:
        l = x.double() @ w[lo:hi].double().T
        p = torch.exp(l - lse.double()[:, None])
        here = (at >= lo) & (at < hi) & live
        hit = torch.zeros_like(p).scatter(1, (at - lo).clamp(0, hi - lo - 1), here.double())
        g = torch.where(live, dloss.double()[:, None], 0.0)
        P, other = g * (p - hit), g * p * (1 - hit)
        e_l = 2 * ref.U * (K / 16 + 16) * (x.double().abs() @ w[lo:hi].double().abs().T) + (l.abs() + 24) * 2.0 ** -20
        bound = (g * (p * e_l + 4 * ref.U * hit)).T @ x.double().abs() + 2.0 ** -16 * ((g * hit).T @ x.double().abs()) \
            + 2 * ref.U * (T / 16 + 32) * (P.abs().T @ x.double().abs())
        var = 2 * SIGMA ** 2 * ((other ** 2).T @ x.double() ** 2)
        ref.check(dw[lo:hi], P.T @ x.double(), 8 * var.sqrt() + bound, (lo, hi))
        assert here.any()


def test_bad_targets_are_not_reported_again():
    x, w, y, dloss = make(50, 64, 300)
    y[13], y[14] = 300, -7
    _, lse = forward(x, w, y)
    assert tr.qt2_train_device_status() != 0
    backward(x, w, y, lse, dloss)
    assert tr.qt2_train_device_status() == 0
