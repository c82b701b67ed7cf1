"""Gated feed-forward product at the ends of the gate's range: large gates, infinities and NaN, on the GPU against
64 bits."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.test_gpu_gated import backward, forward, saved, views
from tests.train_ref import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SILU, GELU = tr.QT2_ACT_SILU, tr.QT2_ACT_GELU_TANH
INF, NAN, TOP = float("inf"), float("nan"), torch.finfo(BF).max
M, F, K = 128, 256, 128


def far_bounds(kind, x):
    """ref.act_bounds where s is neither 0 nor 1, and nothing beyond: past 128 act is x or 0, act' 1 or 0, both exactly.

    In between s is 0 where it would be subnormal, which x below 128 multiplies."""
    e_f, e_df = ref.act_bounds(kind, x)
    near = x.abs() <= 128
    tiny = 128 * 2.0 ** -126
    return torch.where(near, e_f - x.abs() * 1e-37 + tiny, 0.0), torch.where(near, e_df - x.abs() * 1e-37 + tiny, 0.0)


def agree(got, want, bound, what):
    """NaN where the formula has one, infinities of its sign, and within the bound elsewhere."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    limit = torch.isinf(want)
    assert torch.equal(got.double()[limit], want[limit]), what
    finite = torch.isfinite(want)
    check(got[finite], want[finite], bound[finite], what)


@pytest.mark.parametrize("kind", [SILU, GELU])
def test_backward_at_the_ends(kind):
    a, b, _ = views(M, F, K, dy=True)
    gate, up = saved(M, F, 7)
    ends = [-TOP, TOP, -3e38, 3e38, -1e38, -1e37, -1e36, -1e30, 1e30, -1e19, 1e19, -1e4, 1e4, -89.0, -88.0, -87.0, -11.0, -10.0625, -10.0,
            -9.9375, 9.9375, 10.0, 10.0625, 11.0, 88.0, -INF, INF, NAN]
    gate[:, :len(ends)] = torch.tensor(ends, device="cuda").to(BF)
    up[:, :len(ends)] *= 0.125   # their products with up stay in the type
    gate[5, 40:] = NAN
    dh = (ref.view_values(*a) @ ref.view_values(*b).T) / 128
    e_dh = 2 * ref.U * (K / 16 + 16) * (ref.view_values(*a).abs() @ ref.view_values(*b).abs().T) / 128 + 4 * ref.U * dh.abs()
    g, u = gate.double(), up.double()
    f, df, _ = ref.act(kind, g)
    e_f, e_df = far_bounds(kind, g)
    want = dh * u * df, dh * f, f * u
    bound = (e_dh * (u * df).abs() + (dh.abs() + e_dh) * u.abs() * e_df + 3 * ref.U * want[0].abs(),
             e_dh * f.abs() + (dh.abs() + e_dh) * e_f + 2 * ref.U * want[1].abs(), e_f * u.abs() + 2 * ref.U * want[2].abs())
    assert torch.isnan(want[0][:, len(ends) - 3:len(ends)]).all()   # (of inf by the formula: x s (1 - s) is inf * 0)
    for name, x, w, e in zip(("dgate", "dup", "h"), backward(a, b, kind, gate, up), want, bound):
        assert not ((w.abs() > 0.9 * TOP) & torch.isfinite(w)).any()
        agree(x, w, e, name)
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("kind", [SILU, GELU])
def test_forward_of_large_gates(kind):
    """Gates of either sign whose products with up reach 1e37, then infinite ones and NaN."""
    a, bg, bu = views(M, F, K)
    dot = [ref.view_values(*a) @ ref.view_values(*b).T for b in (bg, bu)]
    scale = 1e37 / (dot[0].abs().max() * dot[1].abs().max().clamp(min=1)).item()
    bg = (*bg[:2], bg[2] * scale)
    h, g, u = forward(a, bg, bu, kind)
    want, bound = ref.gated_fwd(*(ref.view_values(*v) for v in (a, bg, bu)), 1.0, kind)
    assert (want[1] < -1e34).any()
    check(g, want[1], bound[1], "g")
    check(u, want[2], bound[2], "u")
    f = ref.act(kind, want[1])[0]
    check(h, f * want[2], bound[1] * want[2].abs() + (f.abs() + bound[1]) * bound[2] + 4 * ref.U * (f * want[2]).abs(), "h")
    assert (h[want[1] < -bound[1]] == 0).all()
    size = dot[0].abs()
    sure = (size > 1e-3 * size.max()) & (dot[1].abs() > 1e-3 * dot[1].abs().max())
    for value in (INF, NAN):
        h, g, u = forward(a, (*bg[:2], torch.full((1,), value, device="cuda")), bu, kind)
        gd = dot[0].sign() * value
        hd = ref.act(kind, gd)[0] * dot[1].sign()
        assert torch.isnan(hd[gd != INF]).all() and torch.isinf(hd[gd == INF]).all()
        for x, w in ((g, gd), (h, hd)):
            assert torch.equal(x.double()[sure].nan_to_num(7.0, 8.0, 9.0), w[sure].nan_to_num(7.0, 8.0, 9.0))
    assert tr.qt2_train_device_status() == 0
