"""Layer norm forward and backward on the GPU against the 64-bit formulas."""
import math

import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
EPS = 1e-5

# rows: one, fewer and more than the blocks; row lengths: one, below and across vectors, warps,
# blocks and the longest that a block keeps in registers
SHAPES = [(1, 1), (3, 2), (1, 2048), (5, 7), (7, 8), (2, 9), (130, 31), (33, 33), (257, 64), (19, 255), (64, 256),
          (77, 257), (40, 1000), (513, 1023), (31, 1025), (9, 2047), (150, 2048), (5, 4095), (6, 4096), (11, 5632),
          (3, 8191), (4, 8192), (3, 8200), (2, 14336), (2, 16384), (3, 16387), (2, 32768), (2, 40001), (1, 70003),
          (5000, 129), (2500, 1601)]


def row_depth(R):
    """No term of a sum over the rows passes through more additions than this."""
    return math.ceil(R / 64) + 96


def make(R, C, xd, wd, seed=0, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((R, C), generator=g, device="cuda") * 1.5 + offset
    x[:, ::5] *= 10
    dy = torch.randn((R, C), generator=g, device="cuda") * 1e-2
    w = (1 + 0.2 * torch.randn(C, generator=g, device="cuda")).to(wd)
    b = (0.3 * torch.randn(C, generator=g, device="cuda")).to(wd)
    xs, dys = ref.rows_like(R, C, xd, fill=float("nan"))[0], ref.rows_like(R, C, xd, fill=float("nan"))[0]
    return xs.copy_(x), dys.copy_(dy), w, b


def forward(x, w, b, eps=EPS, pad=0):
    R, C = x.shape
    y, buf = ref.rows_like(R, C, x.dtype, pad=pad, fill=7.0)
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    tr.qt2_layernorm_fwd(x, R, C, x.stride(0), w, b, eps, y, y.stride(0), mean, rstd)
    assert (buf[:, C:] == 7.0).all()   # elements behind a row's end stay
    return y, mean, rstd


def backward(dy, x, w, mean, rstd, want=(True, True, True), wd=None):
    R, C = x.shape
    wd = wd or (w.dtype if w is not None else FP)
    dx, buf = ref.rows_like(R, C, x.dtype, fill=7.0)
    dw, db = torch.full((C,), 7.0, dtype=wd, device="cuda"), torch.full((C,), 7.0, dtype=wd, device="cuda")
    ws = qt2.alloc_workspace(tr.qt2_layernorm_bwd_workspace_size(R, C))
    ws.fill_(0xFF)   # NaNs: nothing is taken from a workspace that was not written
    tr.qt2_layernorm_bwd(dy, dy.stride(0), x, R, C, x.stride(0), w, mean, rstd, dx if want[0] else None,
                         dx.stride(0), dw if want[1] else None, db if want[2] else None, ws, ws.numel())
    assert (buf[:, C:] == 7.0).all()
    return dx, dw, db


@pytest.mark.parametrize("xd,wd", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_formulas(shape, xd, wd):
    R, C = shape
    x, dy, w, b = make(R, C, xd, wd, seed=R + C)
    y, mean, rstd = forward(x, w, b)
    (wy, wm, wr), (ey, em, er) = ref.norm_fwd(x, w, b, EPS)
    ref.check(mean, wm, em, "mean")
    ref.check(rstd, wr, er, "rstd")
    ref.check(y, wy, ey, "y")
    dx, dw, db = backward(dy, x, w, mean, rstd)
    (wdx, wdw, wdb), (edx, edw, edb) = ref.norm_bwd(dy, x, w, mean, rstd, row_depth(R))
    ref.check(dx, wdx, edx, "dx")
    ref.check(dw, wdw, edw, "dw")
    ref.check(db, wdb, edb, "db")
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("C", [40, 2048, 16387, 70003])
def test_without_weight_or_bias_or_statistics(C):
    x, dy, w, b = make(6, C, BF, FP)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y, mean, rstd = forward(x, ww, bb)
        (wy, _, _), (ey, _, _) = ref.norm_fwd(x, ww, bb, EPS)
        ref.check(y, wy, ey)
        y2 = torch.empty_like(x)
        y2 = ref.rows_like(6, C, BF)[0]
        tr.qt2_layernorm_fwd(x, 6, C, x.stride(0), ww, bb, EPS, y2, y2.stride(0), None, None)
        assert torch.equal(y, y2)
    dx, dw, db = backward(dy, x, None, mean, rstd)
    (wdx, wdw, wdb), (edx, edw, edb) = ref.norm_bwd(dy, x, None, mean, rstd, row_depth(6))
    ref.check(dx, wdx, edx)
    ref.check(dw, wdw, edw)
    ref.check(db, wdb, edb)


@pytest.mark.parametrize("shape", [(5, 33), (700, 2048), (3, 20011)])
def test_each_gradient_alone_is_the_same(shape):
    x, dy, w, b = make(*shape, BF, BF)
    _, mean, rstd = forward(x, w, b)
    full = backward(dy, x, w, mean, rstd)
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, True, True),
                 (True, True, False), (True, False, True)):
        got = backward(dy, x, w, mean, rstd, want)
        for g, f, k in zip(got, full, want):
            assert torch.equal(g, f) if k else (g == 7.0).all()


@pytest.mark.parametrize("shape", [(6, 37), (300, 2048), (2, 70003)])
def test_in_place(shape):
    x, dy, w, b = make(*shape, FP, FP)
    R, C = shape
    y, mean, rstd = forward(x, w, b)
    dx, dw, db = backward(dy, x, w, mean, rstd)
    x2, dy2 = ref.rows_like(R, C, FP)[0].copy_(x), ref.rows_like(R, C, FP)[0].copy_(dy)
    tr.qt2_layernorm_fwd(x2, R, C, x2.stride(0), w, b, EPS, x2, x2.stride(0), None, None)
    assert torch.equal(x2, y)
    ws = qt2.alloc_workspace(tr.qt2_layernorm_bwd_workspace_size(R, C))
    dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
    tr.qt2_layernorm_bwd(dy2, dy2.stride(0), x, R, C, x.stride(0), w, mean, rstd, dy2, dy2.stride(0), dw2, db2, ws,
                         ws.numel())
    assert torch.equal(dy2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_large_offset_keeps_the_variance():
    """Rows far from zero: squares minus the mean's square would lose every bit of the variance."""
    x, _, w, b = make(9, 1000, FP, FP, offset=3e4)
    y, mean, rstd = forward(x, w, b)
    (wy, wm, wr), (ey, em, er) = ref.norm_fwd(x, w, b, EPS)
    ref.check(rstd, wr, er)
    ref.check(y, wy, ey)


def test_constant_rows_and_zero_eps():
    x = ref.rows_like(4, 100, BF)[0]
    x[:] = torch.tensor([0.0, 1.0, -3.0, 256.0], device="cuda")[:, None]
    w, b = torch.full((100,), 2.0, device="cuda"), torch.full((100,), 0.5, device="cuda")
    y, mean, rstd = forward(x, w, b)
    assert torch.equal(mean, x[:, 0].float()) and (y == 0.5).all()
    torch.testing.assert_close(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=4 * ref.U, atol=0)
    y, mean, rstd = forward(x, w, b, eps=0.0)   # 0 * inf, as the formula says
    assert torch.isinf(rstd).all() and torch.isnan(y).all()


@pytest.mark.parametrize("C", [100, 2048, 70003])
def test_nonfinite_rows_stay_to_themselves(C):
    x, dy, w, b = make(7, C, BF, FP)
    y0, mean0, rstd0 = forward(x, w, b)
    bad = x.clone()
    bad = ref.rows_like(7, C, BF)[0].copy_(x)
    bad[2, C // 2], bad[5, 0] = float("nan"), float("inf")
    y, mean, rstd = forward(bad, w, b)
    for r in range(7):
        if r in (2, 5):
            assert torch.isnan(y[r]).all()
        else:
            assert torch.equal(y[r], y0[r])


def test_gradient_against_differences():
    """The directional derivative of sum(dy * y) in x, w and b from the 64-bit forward pass, by
    central differences with steps that change no rounding (fp32 inputs, 64-bit evaluation)."""
    R, C = 13, 301
    x, dy, w, b = make(R, C, FP, FP, seed=3)
    _, mean, rstd = forward(x, w, b)
    dx, dw, db = backward(dy, x, w, mean, rstd)
    g = torch.Generator(device="cuda").manual_seed(5)
    dirs = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in (x, w, b)]
    h = 1e-5

    def f(s):
        (y, _, _), _ = ref.norm_fwd(x.double() + s * h * dirs[0], w.double() + s * h * dirs[1],
                                    b.double() + s * h * dirs[2], EPS)
        return (y * dy.double()).sum()
    want = ((f(1) - f(-1)) / (2 * h)).item()
    terms = [a.double() * d for a, d in zip((dx, dw, db), dirs)]
    # fp32 gradients: their bounds relative to the sum of magnitudes stay below 2^-16; the central
    # difference is off by O(h^2) and 2^-53 / h relative
    scale = sum(t.abs().sum() for t in terms).item()
    assert abs(sum(t.sum() for t in terms).item() - want) <= 2.0 ** -16 * scale


def test_same_bits_again_and_in_a_graph():
    x, dy, w, b = make(999, 2048, BF, BF)
    y, mean, rstd = forward(x, w, b)
    first = (y, *backward(dy, x, w, mean, rstd))
    again = (forward(x, w, b)[0], *backward(dy, x, w, mean, rstd))
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    R, C = x.shape
    ws = qt2.alloc_workspace(tr.qt2_layernorm_bwd_workspace_size(R, C))
    out = [torch.zeros_like(t) for t in first]
    xs, dys = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        tr.qt2_layernorm_fwd(xs, R, C, C, w, b, EPS, out[0], C, mean, rstd)
        tr.qt2_layernorm_bwd(dys, C, xs, R, C, C, w, mean, rstd, out[1], C, out[2], out[3], ws, ws.numel())
    xs.copy_(x.flip(0)), dys.copy_(dy.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], first[0].flip(0)) and torch.equal(out[1], first[1].flip(0))
    xs.copy_(x), dys.copy_(dy)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, out))
