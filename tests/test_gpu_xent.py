"""The head's softmax cross entropy and its gradient on the GPU against 64 bits."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
IGN = -100

# tokens, hidden size, vocabulary: one of each, below, at and across the 16, 64, 128 and 256 steps
# of the tiles, several tiles a pair, a long contraction over a short vocabulary and the reverse
SHAPES = [(1, 1, 1), (1, 8, 2), (2, 3, 5), (1, 64, 1000), (16, 64, 128), (17, 72, 129), (33, 65, 255), (128, 128, 256),
          (127, 63, 257), (129, 200, 511), (255, 256, 300), (256, 264, 512), (257, 320, 513), (300, 1000, 777),
          (64, 2048, 4096), (1000, 96, 3000), (700, 513, 2500), (5, 4096, 900), (2100, 40, 1031), (513, 1024, 1024),
          (1, 2048, 20001), (40, 300, 33333)]


def make(T, K, V, seed=0, ignored=0.1, std=None, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    std = std if std is not None else 1.5 / K ** 0.5
    x = ref.rows_like(T, K, BF, pad=pad, fill=float("nan"))[0]
    w = ref.rows_like(V, K, BF, pad=pad, fill=float("nan"))[0]
    w.copy_(torch.randn((V, K), generator=g, device="cuda") * std)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    lift = 3 * torch.rand((T, 1), generator=g, device="cuda")
    x.copy_(torch.randn((T, K), generator=g, device="cuda") + lift * w[y].float() / (std * std * K))
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, IGN, y)
    dloss = (torch.rand(T, generator=g, device="cuda") + 0.5) / T
    return x, w, y, dloss


def forward(x, w, y, ignore=IGN, ws=None, stream=None):
    (T, K), V = x.shape, w.shape[0]
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    if ws is None:
        ws = qt2.alloc_workspace(tr.qt2_linear_xent_fwd_workspace_size(T, K, V))
        ws.fill_(0xFF)
    tr.qt2_linear_xent_fwd(x, w, y, T, K, V, x.stride(0), w.stride(0), ignore, loss, lse, ws, ws.numel(), stream)
    return loss, lse


def backward(x, w, y, lse, dloss, ignore=IGN, want=(True, True), dwd=BF, ws=None, stream=None):
    (T, K), V = x.shape, w.shape[0]
    dx, bx = ref.rows_like(T, K, BF, fill=7.0)
    dw, bw = ref.rows_like(V, K, dwd, fill=7.0)
    if ws is None:
        ws = qt2.alloc_workspace(tr.qt2_linear_xent_bwd_workspace_size(T, K, V))
        ws.fill_(0xFF)
    code = qt2.QT2_DTYPE_F32 if dwd == FP else qt2.QT2_DTYPE_BF16
    tr.qt2_linear_xent_bwd(x, w, y, lse, dloss, T, K, V, x.stride(0), w.stride(0), ignore, dx if want[0] else None,
                           dx.stride(0), dw if want[1] else None, code, dw.stride(0), ws, ws.numel(), stream)
    assert (bx[:, K:] == 7.0).all() and (bw[:, K:] == 7.0).all()   # elements behind a row's end stay
    return dx, dw


def check_all(x, w, y, dloss, ignore=IGN, dwd=BF):
    loss, lse = forward(x, w, y, ignore)
    dx, dw = backward(x, w, y, lse, dloss, ignore, dwd=dwd)
    (l, s, gx, gw), (el, es, ex, ew) = ref.xent(x, w, y, ignore, dloss)
    ref.check(lse, s, es, "lse")
    ref.check(loss, l, el, "loss")
    ref.check(dx, gx, ex, "dx")
    ref.check(dw, gw, ew, "dw")
    return loss, lse, dx, dw


@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_formulas(shape):
    x, w, y, dloss = make(*shape, seed=sum(shape))
    check_all(x, w, y, dloss, dwd=FP if shape[0] % 2 else BF)
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("std", [0.0, 1e-4, 3.0])
def test_flat_and_peaked_rows(std):
    """Equal logits (lse = log V), and logits of up to some hundreds."""
    x, w, y, dloss = make(70, 96, 1500, std=max(std, 1e-3), pad=8)
    if std == 0.0:
        w.zero_()
    loss, lse, _, _ = check_all(x, w, y, dloss)
    if std == 0.0:
        torch.testing.assert_close(lse.double(), torch.full_like(lse, 1500.0).double().log(), rtol=2 ** -21, atol=0)


def test_several_pieces_of_the_vocabulary():
    """A workspace of P that holds only a part of the vocabulary: dx adds up over the pieces."""
    T, K, V = 8200, 72, 40000
    assert T * V * 2 > (512 << 20)
    x, w, y, dloss = make(T, K, V)
    loss, lse = forward(x, w, y)
    dx, dw = backward(x, w, y, lse, dloss)
    (l, s, gx, gw), (el, es, ex, ew) = ref.xent(x, w, y, IGN, dloss)
    ref.check(loss, l, el)
    ref.check(dx, gx, ex)
    ref.check(dw, gw, ew)


def test_rows_without_a_target():
    x, w, y, dloss = make(300, 64, 1000, ignored=0.0)
    y[::3] = IGN
    dloss[::6] = float("nan")   # not used where there is no target
    loss, lse, dx, dw = check_all(x, w, y, torch.where(y == IGN, 0.0, dloss))
    loss2, lse2 = forward(x, w, y)
    dx2, dw2 = backward(x, w, y, lse2, dloss)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and (loss2[::3] == 0).all() and (dx2[::3] == 0).all()
    # nor does what x holds there reach a gradient
    bad = ref.rows_like(300, 64, BF, fill=float("nan"))[0].copy_(x)
    bad[::6], bad[3::6] = float("nan"), float("inf")
    loss3, lse3 = forward(bad, w, y)
    dx3, dw3 = backward(bad, w, y, lse3, dloss)
    assert torch.equal(loss3, loss2) and torch.equal(dx3, dx2) and torch.equal(dw3, dw2)
    y[:] = IGN
    loss, lse = forward(bad, w, y)
    dx, dw = backward(bad, w, y, lse, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("ignore", [-1, 5, 10 ** 12])
def test_other_ignore_index(ignore):
    x, w, y, dloss = make(50, 64, 300, ignored=0.0)
    y[7:12] = ignore
    check_all(x, w, y, dloss, ignore=ignore)
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("bad", [-7, 300, 2 ** 31, 2 ** 32 + 3, -2 ** 63])
def test_targets_outside_the_vocabulary_are_reported(bad):
    x, w, y, dloss = make(50, 64, 300)
    y[13] = bad
    loss, lse = forward(x, w, y)
    assert tr.qt2_train_device_status() == qt2.QT2_ERR_INVALID_ARG
    dx, dw = backward(x, w, y, lse, dloss)
    assert tr.qt2_train_device_status() in (0, qt2.QT2_ERR_INVALID_ARG)
    y2 = torch.where(y == bad, IGN, y)
    assert torch.equal(loss, forward(x, w, y2)[0]) and loss[13] == 0
    dx2, dw2 = backward(x, w, y2, lse, dloss)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("shape", [(300, 72, 1031), (2500, 64, 600)])
def test_each_gradient_alone_is_the_same(shape):
    x, w, y, dloss = make(*shape)
    _, lse = forward(x, w, y)
    dx, dw = backward(x, w, y, lse, dloss)
    a, b = backward(x, w, y, lse, dloss, want=(True, False))
    assert torch.equal(a, dx) and (b == 7.0).all()
    a, b = backward(x, w, y, lse, dloss, want=(False, True))
    assert torch.equal(b, dw) and (a == 7.0).all()


def test_nonfinite_rows_stay_to_themselves_forward():
    x, w, y, dloss = make(40, 64, 700, ignored=0.0)
    loss0, lse0 = forward(x, w, y)
    x[3, 5], x[9, 0] = float("nan"), float("inf")
    y[9] = 0
    loss, lse = forward(x, w, y)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[3] = keep[9] = False
    assert loss[3].isnan() and not torch.isfinite(loss[9])
    assert torch.equal(loss[keep], loss0[keep]) and torch.equal(lse[keep], lse0[keep])
    dx, _ = backward(x, w, y, lse, dloss)
    dx0, _ = backward(*make(40, 64, 700, ignored=0.0)[:2], y, lse0, dloss)
    assert torch.equal(dx[keep], dx0[keep])


def test_gradient_against_differences():
    """Central differences of the kernel's own loss along directions on a grid that bf16 holds
    exactly.  The losses' bounds enter divided by the step.  A row's loss along d has the third
    central moment of the logits' change under the softmax as its third derivative; a variable
    that spans r has one of at most r^3 / (6 sqrt 3), and the remainder is h^2 / 6 of it."""
    T, K, V = 64, 64, 320
    g = torch.Generator(device="cuda").manual_seed(1)
    grid = 1 / 16
    x = (torch.randint(-8, 9, (T, K), generator=g, device="cuda") * grid).to(BF)
    w = (torch.randint(-8, 9, (V, K), generator=g, device="cuda") * grid).to(BF)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = torch.ones(T, device="cuda")
    _, lse = forward(x, w, y)
    dx, dw = backward(x, w, y, lse, dloss, dwd=FP)
    for name in ("x", "w"):
        d = torch.zeros((T, K) if name == "x" else (V, K), device="cuda")
        rows, cols = torch.randint(0, d.shape[0], (24,), generator=g, device="cuda"), \
            torch.randint(0, K, (24,), generator=g, device="cuda")
        d[rows, cols] = 1.0
        h = grid
        up, down = [forward((x + s * h * d).to(BF), w, y)[0] if name == "x" else
                    forward(x, (w + s * h * d).to(BF), y)[0] for s in (1, -1)]
        want = ((up.double() - down.double()).sum() / (2 * h)).item()
        got = ((dx if name == "x" else dw).double() * d).sum().item()
        (_, _), (el, _) = ref.xent(x, w, y, IGN)
        (_, _, gx, gw), (_, _, ex, ew) = ref.xent(x, w, y, IGN, dloss)
        # |x|, |w| <= 1/2: with n changed coordinates a logit changes at most n / 2 either way
        n = d.sum(1) if name == "x" else d.sum(1).max().expand(T)
        third = h * h / 6 * (n ** 3).sum().item() / (6 * 3 ** 0.5)
        e = ((ex if name == "x" else ew) * d).sum().item() + 2 ** -8 * ((gx if name == "x" else gw) * d).abs().sum().item()
        assert abs(got - want) <= third + e + el.sum().item() / h


def test_same_bits_again_on_two_streams_and_in_a_graph():
    cases = [make(600, 256, 5000, seed=s) for s in (1, 2)]
    first = []
    for x, w, y, dloss in cases:
        loss, lse = forward(x, w, y)
        first.append((loss, lse, *backward(x, w, y, lse, dloss)))
    torch.cuda.synchronize()
    T, K, V = 600, 256, 5000
    size = max(tr.qt2_linear_xent_fwd_workspace_size(T, K, V), tr.qt2_linear_xent_bwd_workspace_size(T, K, V))
    sides, wss = [torch.cuda.Stream() for _ in cases], [qt2.alloc_workspace(size) for _ in cases]
    outs = [[torch.zeros_like(t) for t in f] for f in first]
    torch.cuda.synchronize()

    def enqueue(k, stream=None):
        (x, w, y, dloss), (loss, lse, dx, dw), ws = cases[k], outs[k], wss[k]
        tr.qt2_linear_xent_fwd(x, w, y, T, K, V, K, K, IGN, loss, lse, ws, ws.numel(), stream)
        tr.qt2_linear_xent_bwd(x, w, y, lse, dloss, T, K, V, K, K, IGN, dx, K, dw, 0, K, ws, ws.numel(), stream)
    for _ in range(3):
        for k in range(2):
            enqueue(k, sides[k])
    torch.cuda.synchronize()
    for f, o in zip(first, outs):
        assert all(torch.equal(a, b) for a, b in zip(f, o))
    graph = torch.cuda.CUDAGraph()
    for o in outs[0]:
        o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=sides[0]):
        enqueue(0)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[0], outs[0]))
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("T", [5, 40])
def test_huge_logits(T):
    """Logits of up to 1e7, where the tensor cores' sums are off by up to some units: a row that expects
    its target has no loss.  (What remains is log1p(expm1(d)) - d of that d, here below 16: expm1 and
    log1p are within 2 steps each, 2^-22 relative.)"""
    K, V = 2048, 700
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn((V, K), generator=g, device="cuda") * 64).to(BF)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = w[y].clone()
    loss, lse = forward(x, w, y)
    (l, s), (el, es) = ref.xent(x, w, y, IGN)
    ref.check(lse, s, es)
    ref.check(loss, l, el)
    assert (loss.abs() <= 18 * 2.0 ** -21).all()
    dx, dw = backward(x, w, y, lse, torch.ones(T, device="cuda"))
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("dwd", [BF, FP])
@pytest.mark.parametrize("shape", [(511, 512, 1003), (513, 520, 1002), (6, 136, 301), (39, 272, 257), (577, 136, 777)])
def test_rows_that_end_inside_a_group_of_four(shape, dwd):
    """Lanes exchange parts of four neighbouring rows of P and dw before they store them, in tiles of 512 contracted
    elements at most: both ways, with T and V no multiples of four, rows 16 and 32 bytes aligned."""
    check_all(*make(*shape, seed=sum(shape)), dwd=dwd)
    assert tr.qt2_train_device_status() == 0
