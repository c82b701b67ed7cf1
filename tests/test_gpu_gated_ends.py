"""Gated feed-forward product at the ends of the gate's range: large gates, infinities and NaN, on the GPU against
64 bits."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.test_gpu_gated import forward, views
from tests.train_ref import check

pytestmark = pytest.mark.gpu
SILU, GELU = tr.QT2_ACT_SILU, tr.QT2_ACT_GELU_TANH
INF, NAN = float("inf"), float("nan")
M, F, K = 128, 256, 128


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
