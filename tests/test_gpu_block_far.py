"""A transformer block's operators on rows that lie more than 2^31 elements apart."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.test_gpu_gated import backward, forward, saved, views
from tests.train_ref import check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
STEP = (1 << 30) + 8


def far(shape, strides):
    """A bf16 tensor of these strides over a buffer of zeros."""
    n = 1 + sum((s - 1) * d for s, d in zip(shape, strides))
    return torch.zeros(n, dtype=BF, device="cuda").as_strided(shape, strides)


@pytest.mark.parametrize("T,H,ld,hs", [(3, 2, STEP, 64), (2, 3, 64, STEP)])
def test_heads_far_apart(T, H, ld, hs):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy, near = (torch.randn((T, H, 64), generator=g, device="cuda").to(BF) for _ in range(3))
    w = 1 + 0.1 * torch.randn(64, generator=g, device="cuda")
    cos, sin = ref.tables(8, 64)
    pos = torch.tensor([5, 0, 7], device="cuda")[:T]
    ws = qt2.alloc_workspace(tr.qt2_qk_norm_rope_bwd_workspace_size(T, H, 0, 64))

    def run(x, dy, y, dx):
        dw = torch.empty(64, device="cuda")
        tr.qt2_qk_norm_rope_fwd(x, T, H, 0, 64, x.stride(0), x.stride(1), w, None, 1e-6, pos, cos, sin, 8, 64, 0, y, y.stride(0), y.stride(1))
        tr.qt2_qk_norm_rope_bwd(dy, dy.stride(0), dy.stride(1), x, T, H, 0, 64, x.stride(0), x.stride(1), w, None, 1e-6, pos, cos, sin, 8, 64,
                                0, dx, dx.stride(0), dx.stride(1), dw, None, ws, ws.numel())
        return y, dx, dw
    want = run(x, dy, torch.empty_like(x), torch.empty_like(x))
    check(want[0], *ref.qk_fwd(x, H, w, None, 1e-6, cos[pos], sin[pos], 64, 0))
    spread = lambda t: far((T, H, 64), (ld, hs, 1)).copy_(t)  # noqa: E731
    got = run(spread(x), spread(dy), torch.empty_like(x), torch.empty_like(x))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = run(x, dy, spread(near), spread(near))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert tr.qt2_train_device_status() == 0


def test_gated_rows_far_apart():
    M, F, K, ld = 256, 128, 128, (1 << 23) + 64   # the last row starts behind 2^31 elements
    a, bg, bu = views(M, F, K)
    want = forward(a, bg, bu, tr.QT2_ACT_SILU)
    h = far((M, F), (ld, 1))
    tr.qt2_gemm_nvfp4_gated(qt2.View(*a), qt2.View(*bg), qt2.View(*bu), M, F, K, 1.0, tr.QT2_ACT_SILU, None, None, 0, h, ld)
    assert torch.equal(h, want[0])
    gate, up = saved(M, F, 3)
    want = backward(a, bg, tr.QT2_ACT_SILU, gate, up)
    h.zero_()
    dg, du = (torch.empty((M, F), dtype=BF, device="cuda") for _ in range(2))
    wide = [far((M, F), (ld, 1)).copy_(t) for t in (gate, up)]
    tr.qt2_gemm_nvfp4_gated_bwd(qt2.View(*a), qt2.View(*bg), M, F, K, 2.0 ** -7, tr.QT2_ACT_SILU, *wide, ld, dg, du, F, h, ld)
    assert all(torch.equal(x, y) for x, y in zip((dg, du, h), want))
    # and in place
    tr.qt2_gemm_nvfp4_gated_bwd(qt2.View(*a), qt2.View(*bg), M, F, K, 2.0 ** -7, tr.QT2_ACT_SILU, *wide, ld, *wide, ld, None, 0)
    assert torch.equal(wide[0], want[0]) and torch.equal(wide[1], want[1])
    assert tr.qt2_train_device_status() == 0
