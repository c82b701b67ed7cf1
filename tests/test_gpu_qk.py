"""Norm of queries and keys for each head with the position rotation, forward and backward, against 64 bits."""
import math

import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.train_ref import check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
EPS = 1e-6

# (T, Hq, Hk, D, R): one token, one head, shared key heads, none of either kind; heads below, at and across the
# lanes' shares; nothing, a part and all of a head turned
SHAPES = [(1, 1, 0, 8, 8), (1, 32, 8, 128, 128), (3, 0, 1, 16, 0), (5, 3, 1, 24, 16), (7, 4, 2, 32, 8), (2, 5, 5, 40, 40),
          (33, 2, 1, 64, 32), (19, 7, 3, 72, 72), (64, 12, 4, 80, 40), (50, 1, 1, 96, 96), (257, 16, 16, 128, 128), (31, 3, 0, 128, 64),
          (17, 2, 2, 136, 120), (21, 5, 2, 192, 192), (40, 2, 1, 256, 128), (9, 1, 2, 264, 256), (6, 2, 1, 512, 512), (5, 1, 1, 520, 8),
          (3, 2, 3, 1024, 1024), (2500, 6, 2, 64, 64), (1500, 9, 1, 128, 128)]


def row_depth(T, H):
    """Rows of a lane, lanes, warps and blocks that a term of dw passes."""
    return math.ceil(T * H / (148 * 3 * 8)) + 4 + 5 + 8 + 14 + 5 + 8


class Case:
    """x, dy, y and dx [T, H, D] in one of the layouts: heads of a token side by side with others between
    ("rows"), or tokens of a head ("heads")."""

    def __init__(self, T, Hq, Hk, D, R, xd=BF, wd=FP, layout="rows", P=None, seed=0, given=True):
        self.T, self.Hq, self.Hk, self.D, self.R = T, Hq, Hk, D, R
        self.H = H = Hq + Hk
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.layout, self.xd = layout, xd
        x = rn(T, H, D)
        x[:, :, ::5] *= 8
        self.x, self.dy = self.place(x.to(xd)), self.place((rn(T, H, D) * 1e-2).to(xd))
        self.wq, self.wk = ((1 + 0.3 * rn(D)).to(wd) if given else None for _ in range(2))
        self.wd = wd
        self.P = P or T + 70
        self.cos, self.sin = ref.tables(self.P, R) if R else (None, None)
        self.pos = torch.randint(0, self.P, (T,), generator=g, device="cuda")

    def place(self, x):
        """x in this layout, NaNs around it."""
        T, H, D = self.T, self.H, self.D
        if self.layout == "rows":
            buf = torch.full((T, H + self.Hk + 1, D + 8), float("nan"), dtype=self.xd, device="cuda")
            v = buf[:, :H, :D]
        else:
            buf = torch.full((H, T + 2, D), float("nan"), dtype=self.xd, device="cuda")
            v = buf[:, 1:T + 1].transpose(0, 1)
        v.copy_(x)
        return v

    def strides(self, t):
        return t.stride(0), t.stride(1)

    def out(self, fill=7.0):
        v = self.place(torch.zeros((self.T, self.H, self.D), dtype=self.xd, device="cuda"))
        v._base.fill_(fill)
        return v

    def table_rows(self, pos=None):
        pos = self.pos if pos is None else pos
        none = torch.zeros(self.T, 0, device="cuda")
        return (self.cos[pos], self.sin[pos]) if self.R else (none, none)

    def forward(self, pairs, y=None, pos="own"):
        y = self.out() if y is None else y
        pos = self.pos if isinstance(pos, str) else pos
        tr.qt2_qk_norm_rope_fwd(self.x, self.T, self.Hq, self.Hk, self.D, *self.strides(self.x), self.wq, self.wk, EPS, pos,
                                self.cos, self.sin, self.P, self.R, pairs, y, *self.strides(y))
        return y

    def backward(self, pairs, want=(True, True, True), dx=None, pos="own"):
        dx = self.out() if dx is None else dx
        pos = self.pos if isinstance(pos, str) else pos
        dwq, dwk = (torch.full((self.D,), 7.0, dtype=self.wd, device="cuda") for _ in range(2))
        ws = qt2.alloc_workspace(tr.qt2_qk_norm_rope_bwd_workspace_size(self.T, self.Hq, self.Hk, self.D))
        ws.fill_(0xFF)
        tr.qt2_qk_norm_rope_bwd(self.dy, *self.strides(self.dy), self.x, self.T, self.Hq, self.Hk, self.D, *self.strides(self.x),
                                self.wq, self.wk, EPS, pos, self.cos, self.sin, self.P, self.R, pairs, dx if want[0] else None,
                                *self.strides(dx), dwq if want[1] else None, dwk if want[2] else None, ws, ws.numel())
        return dx, dwq, dwk

    def rest(self, v):
        """What lies around v in its buffer."""
        buf = v._base.clone()
        w = buf[:, :self.H, :self.D] if self.layout == "rows" else buf[:, 1:self.T + 1]
        w.fill_(7.0)
        return buf


@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("xd,wd,layout", [(BF, FP, "rows"), (BF, BF, "heads"), (FP, FP, "heads"), (FP, BF, "rows")])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_formulas(shape, xd, wd, layout, pairs):
    c = Case(*shape, xd, wd, layout, seed=sum(shape))
    cos, sin = c.table_rows()
    y = c.forward(pairs)
    want, bound = ref.qk_fwd(c.x, c.Hq, c.wq, c.wk, EPS, cos, sin, c.R, pairs)
    check(y, want, bound, "y")
    assert (c.rest(y) == 7.0).all()
    got = c.backward(pairs)
    want, bound = ref.qk_bwd(c.dy, c.x, c.Hq, c.wq, c.wk, EPS, cos, sin, c.R, pairs, row_depth(c.T, c.H))
    for name, a, w, e in zip(("dx", "dwq", "dwk"), got, want, bound):
        check(a, w, e, name)
    assert (c.rest(got[0]) == 7.0).all()
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("shape", [(5, 3, 1, 24, 16), (300, 16, 4, 128, 128), (9, 1, 2, 264, 256)])
def test_without_weights_and_positions(shape):
    c = Case(*shape, given=False, P=shape[0])
    at = torch.arange(c.T, device="cuda")
    cos, sin = c.table_rows(at)
    y, got = c.forward(0, pos=None), c.backward(0, pos=None)
    want, bound = ref.qk_fwd(c.x, c.Hq, None, None, EPS, cos, sin, c.R, 0)
    check(y, want, bound)
    want, bound = ref.qk_bwd(c.dy, c.x, c.Hq, None, None, EPS, cos, sin, c.R, 0, row_depth(c.T, c.H))
    for a, w, e in zip(got, want, bound):
        check(a, w, e)
    assert torch.equal(y, c.forward(0, pos=at)) and all(torch.equal(a, b) for a, b in zip(got, c.backward(0, pos=at)))


@pytest.mark.parametrize("shape", [(40, 5, 3, 80, 40), (700, 4, 4, 128, 128)])
def test_gradients_alone_and_in_place(shape):
    c = Case(*shape, FP)
    full, y = c.backward(1), c.forward(1)
    for want in ((True, False, False), (False, True, False), (False, False, True), (False, True, True), (True, False, True)):
        got = c.backward(1, want)
        for g, f, k in zip(got, full, want):
            assert torch.equal(g, f) if k else (g == 7.0).all()
    keep, dy = c.x.clone(), c.dy.clone()
    got = c.backward(1, dx=c.dy)
    assert torch.equal(c.dy, full[0]) and torch.equal(got[1], full[1]) and torch.equal(got[2], full[2])
    c.dy.copy_(dy)
    c.backward(1, dx=c.x)
    assert torch.equal(c.x, full[0])
    c.x.copy_(keep)
    assert torch.equal(c.forward(1, y=c.x), y) and torch.equal(c.x, y)


def test_positions_outside_the_tables():
    c = Case(12, 2, 1, 64, 64, FP)
    y, got = c.forward(0), c.backward(0)
    for bad in (-1, c.P, 1 << 40, -(1 << 62)):
        pos = c.pos.clone()
        pos[3] = bad
        z, dz = c.forward(0, pos=pos), c.backward(0, pos=pos)
        assert tr.qt2_train_device_status() == qt2.QT2_ERR_INVALID_ARG
        keep = torch.arange(12, device="cuda") != 3
        assert torch.equal(z[keep], y[keep]) and torch.equal(dz[0][keep], got[0][keep])
        none = torch.zeros(12, 0, device="cuda")
        want, bound = ref.qk_fwd(c.x, 2, c.wq, c.wk, EPS, none, none, 0, 0)
        check(z[3], want[3], bound[3])
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("D", [64, 80, 512])
def test_zero_rows_and_nonfinite_ones_stay_to_themselves(D):
    c = Case(10, 3, 2, D, D)
    c.x[4, 1] = 0
    y, got = c.forward(0), c.backward(0)
    assert (y[4, 1] == 0).all() and all(torch.isfinite(t).all() for t in (y, *got))
    c.x[2, 0, 5], c.x[7, 4, 0], c.dy[5, 2, 1] = float("nan"), float("inf"), float("inf")
    z, dz = c.forward(0), c.backward(0)[0]
    bad = torch.zeros(10, 5, dtype=torch.bool, device="cuda")
    bad[2, 0] = bad[7, 4] = True
    assert torch.equal(z[~bad], y[~bad]) and torch.isnan(z[2, 0]).all()
    bad[5, 2] = True
    assert torch.equal(dz[~bad], got[0][~bad])


@pytest.mark.parametrize("pairs", [0, 1])
def test_gradient_against_differences(pairs):
    c = Case(11, 3, 2, 48, 32, FP, FP, seed=4)
    cos, sin = c.table_rows()
    dx, dwq, dwk = c.backward(pairs)
    g = torch.Generator(device="cuda").manual_seed(6)
    dirs = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in (c.x, c.wq, c.wk)]
    h = 1e-5

    def f(s):
        y, _ = ref.qk_fwd(c.x.double() + s * h * dirs[0], 3, c.wq.double() + s * h * dirs[1], c.wk.double() + s * h * dirs[2], EPS,
                          cos, sin, c.R, pairs)
        return (y * c.dy.double()).sum()
    want = ((f(1) - f(-1)) / (2 * h)).item()
    terms = [a.double() * d for a, d in zip((dx, dwq, dwk), dirs)]
    scale = sum(t.abs().sum() for t in terms).item()
    assert abs(sum(t.sum() for t in terms).item() - want) <= 2.0 ** -16 * scale


def test_rotation_keeps_lengths_and_differences_of_positions():
    """The product of a turned query and key depends on the distance of their positions alone, far ones included."""
    c = Case(64, 1, 1, 128, 128, FP, P=1 << 17)
    c.x.copy_(c.x[:1].expand_as(c.x))
    c.pos.copy_(torch.arange(64, device="cuda") + (1 << 17) - 64)
    y = c.forward(0).double()
    dots = torch.stack([(y[7:, 0] * y[:-7, 1]).sum(1), (y[7:, 0] * y[:-7, 1]).sum(1)[:1].expand(57)])
    size = y[0, 0].norm() * y[0, 1].norm()
    assert ((dots[0] - dots[1]).abs() <= 2.0 ** -17 * size).all()   # roundings of tables (2^-24 each) and elements


def test_in_a_graph_on_two_streams_and_again():
    cases = [Case(333, 12, 4, 128, 64, BF, FP, seed=s) for s in (1, 2)]
    want = [[t.clone() for t in (c.forward(0), *c.backward(0))] for c in cases]
    outs = [(c.out(), c.out(), torch.empty(128, device="cuda"), torch.empty(128, device="cuda"),
             qt2.alloc_workspace(tr.qt2_qk_norm_rope_bwd_workspace_size(333, 12, 4, 128))) for c in cases]

    def run(k):
        c, (y, dx, dwq, dwk, ws) = cases[k], outs[k]
        c.forward(0, y=y)
        tr.qt2_qk_norm_rope_bwd(c.dy, *c.strides(c.dy), c.x, c.T, c.Hq, c.Hk, c.D, *c.strides(c.x), c.wq, c.wk, EPS, c.pos, c.cos, c.sin,
                                c.P, c.R, 0, dx, *c.strides(dx), dwq, dwk, ws, ws.numel())
    torch.cuda.synchronize()
    graph, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        run(0)
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
        with torch.cuda.stream(other):
            run(1)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
