"""Gated feed-forward product on NVFP4 operands, forward and backward, on the GPU against 64 bits."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.train_ref import check, rows_like

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SILU, GELU = tr.QT2_ACT_SILU, tr.QT2_ACT_GELU_TANH

# (M, F, K): halves of a tile's rows and columns behind the end, half a stage of K, fewer and more tiles than
# pairs of SMs, more stages than the ring
SHAPES = [(128, 128, 128), (128, 256, 384), (256, 128, 256), (384, 384, 640), (640, 2176, 1408), (1920, 1408, 256),
          (128, 14336, 128), (4096, 128, 128), (2048, 5632, 2048), (2176, 2432, 512)]


def views(M, F, K, seed=0, g_scale=0.002, dy=False):
    a = ref.random_view(M, K, seed, 1e-3 if dy else 1.0)
    return a, ref.random_view(F, K, seed + 1, g_scale), ref.random_view(F, K, seed + 2, 0.003)


def empty(M, F, pad=0, fill=7.0):
    return rows_like(M, F, BF, pad=pad, fill=fill)


def forward(a, bg, bu, kind, keep=True, pad=0, alpha=1.0):
    (M, K), F = (a[0].shape[0], 2 * a[0].shape[1]), bg[0].shape[0]
    outs = [empty(M, F, pad) for _ in range(3)]
    h, g, u = (t for t, _ in outs)
    tr.qt2_gemm_nvfp4_gated(qt2.View(*a), qt2.View(*bg), qt2.View(*bu), M, F, K, alpha, kind, g if keep else None,
                            u if keep else None, g.stride(0), h, h.stride(0))
    assert all((buf[:, F:] == 7.0).all() for _, buf in outs)   # behind the rows' ends
    return h, g, u


def saved(M, F, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 9)
    gate, up = (rows_like(M, F, BF)[0].copy_(torch.randn((M, F), generator=g, device="cuda") * s) for s in (3.0, 1.0))
    flat = gate[0, :8]
    flat.copy_(torch.tensor([0.0, -0.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4], device="cuda"))
    return gate, up


def backward(a, b, kind, gate, up, h=True, pad=0, alpha=2.0 ** -7):
    (M, K), F = (a[0].shape[0], 2 * a[0].shape[1]), b[0].shape[0]
    outs = [empty(M, F, pad) for _ in range(3)]
    dg, du, hh = (t for t, _ in outs)
    tr.qt2_gemm_nvfp4_gated_bwd(qt2.View(*a), qt2.View(*b), M, F, K, alpha, kind, gate, up, gate.stride(0), dg, du,
                                dg.stride(0), hh if h else None, hh.stride(0))
    assert all((buf[:, F:] == 7.0).all() for _, buf in outs)
    return dg, du, hh


@pytest.mark.parametrize("kind", [SILU, GELU])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_matches_the_formulas(shape, kind):
    M, F, K = shape
    a, bg, bu = views(M, F, K)
    want, bound = ref.gated_fwd(*(ref.view_values(*v) for v in (a, bg, bu)), 1.0, kind)
    got = forward(a, bg, bu, kind)
    for name, x, w, e in zip("hgu", got, want, bound):
        check(x, w, e, name)
    alone, g, u = forward(a, bg, bu, kind, keep=False)
    assert torch.equal(alone, got[0]) and (g == 7.0).all() and (u == 7.0).all()
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("kind", [SILU, GELU])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward_matches_the_formulas(shape, kind):
    M, F, K = shape
    a, b, _ = views(M, F, K, dy=True)
    gate, up = saved(M, F, K)
    want, bound = ref.gated_bwd(ref.view_values(*a), ref.view_values(*b), 2.0 ** -7, kind, gate, up)
    got = backward(a, b, kind, gate, up)
    for name, x, w, e in zip(("dgate", "dup", "h"), got, want, bound):
        check(x, w, e, name)
    dg, du, h = backward(a, b, kind, gate, up, h=False)
    assert torch.equal(dg, got[0]) and torch.equal(du, got[1]) and (h == 7.0).all()
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("pad", [0, 8, 16, 40])
def test_leading_dimensions_and_alignments(pad):
    """Rows that start on 16 bytes and not on 32, matrices that are halves of a wider one."""
    M, F, K = 384, 640, 512
    a, bg, bu = views(M, F, K)
    want = forward(a, bg, bu, SILU)
    assert all(torch.equal(x, y) for x, y in zip(forward(a, bg, bu, SILU, pad=pad), want))
    both, h = torch.full((M, 2 * F + pad), 7.0, dtype=BF, device="cuda"), torch.full((M * F + 8,), 7.0, dtype=BF, device="cuda")
    h16 = h[8:].view(M, F)   # 16 bytes off
    tr.qt2_gemm_nvfp4_gated(qt2.View(*a), qt2.View(*bg), qt2.View(*bu), M, F, K, 1.0, SILU, both[:, :F], both[:, F:], 2 * F + pad,
                            h16, F)
    assert torch.equal(h16, want[0]) and torch.equal(both[:, :F], want[1]) and torch.equal(both[:, F:2 * F], want[2])
    assert (both[:, 2 * F:] == 7.0).all() and (h[:8] == 7.0).all()
    gate, up = want[1], want[2]
    ref_b = backward(a, bg, SILU, gate, up)
    assert all(torch.equal(x, y) for x, y in zip(backward(a, bg, SILU, both[:, :F], both[:, F:2 * F], pad=pad), ref_b))
    # in place, in the halves of one matrix
    tr.qt2_gemm_nvfp4_gated_bwd(qt2.View(*a), qt2.View(*bg), M, F, K, 2.0 ** -7, SILU, both[:, :F], both[:, F:], 2 * F + pad,
                                both[:, :F], both[:, F:], 2 * F + pad, None, F)
    assert torch.equal(both[:, :F], ref_b[0]) and torch.equal(both[:, F:2 * F], ref_b[1]) and (both[:, 2 * F:] == 7.0).all()


def test_matches_the_separate_products():
    """g and u are what the library's GEMM gives for the same views."""
    M, F, K = 512, 1024, 1152
    a, bg, bu = views(M, F, K)
    h, g, u = forward(a, bg, bu, SILU)
    for b, x in ((bg, g), (bu, u)):
        c = torch.empty((M, F), dtype=BF, device="cuda")
        qt2.qt2_gemm_nvfp4(qt2.View(*a), qt2.View(*b), M, F, K, 1.0, c, qt2.QT2_DTYPE_BF16, F)
        assert torch.equal(c, x)


@pytest.mark.parametrize("kind", [SILU, GELU])
def test_gradients_against_differences(kind):
    """sum(dh * h) in the kept gate and up, dh an output gradient, by central differences in 64 bits."""
    M, F, K = 128, 256, 128
    a, b, _ = views(M, F, K, dy=True)
    gate, up = saved(M, F, 3)
    gate[0, :8] = 0.5
    dg, du, _ = backward(a, b, kind, gate, up)
    dh = (ref.view_values(*a) @ ref.view_values(*b).T) / 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    d1, d2 = (torch.randn((M, F), generator=gen, device="cuda", dtype=torch.float64) for _ in range(2))
    eps = 1e-6

    def f(s):
        return (dh * ref.act(kind, gate.double() + s * eps * d1)[0] * (up.double() + s * eps * d2)).sum()
    want = ((f(1) - f(-1)) / (2 * eps)).item()
    terms = [(dg.double() * d1), (du.double() * d2)]
    scale = sum(t.abs().sum().item() for t in terms)
    # every term is off by half a bf16 step (2^-9 of it) and what fp32 adds, far below
    assert abs(sum(t.sum().item() for t in terms) - want) <= 2.0 ** -8 * scale


def test_in_a_graph_beside_another_stream_and_again():
    M, F, K = 640, 1408, 768
    sets = [(views(M, F, K, seed=s), saved(M, F, s)) for s in (1, 20)]
    want = []
    for (a, bg, bu), (gate, up) in sets:
        want.append([t.clone() for t in (*forward(a, bg, bu, SILU), *backward(a, bg, GELU, gate, up))])
    outs = [[torch.empty((M, F), dtype=BF, device="cuda") for _ in range(6)] for _ in sets]

    def run(k):
        (a, bg, bu), (gate, up) = sets[k]
        h, g, u, dg, du, hh = outs[k]
        tr.qt2_gemm_nvfp4_gated(qt2.View(*a), qt2.View(*bg), qt2.View(*bu), M, F, K, 1.0, SILU, g, u, F, h, F)
        tr.qt2_gemm_nvfp4_gated_bwd(qt2.View(*a), qt2.View(*bg), M, F, K, 2.0 ** -7, GELU, gate, up, gate.stride(0), dg, du, F, hh, F)
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
        assert all(torch.equal(x, y) for x, y in zip(o, w))
    assert tr.qt2_train_device_status() == 0


def test_chain_reads_what_the_call_before_wrote():
    """Forward, backward on what it kept, forward again, without a wait between."""
    M, F, K = 384, 896, 256
    a, bg, bu = views(M, F, K)
    h, g, u = forward(a, bg, bu, GELU)
    torch.cuda.synchronize()
    want = [t.clone() for t in backward(a, bg, GELU, g, u)]
    torch.cuda.synchronize()
    for _ in range(20):
        g.zero_(), u.zero_()
        tr.qt2_gemm_nvfp4_gated(qt2.View(*a), qt2.View(*bg), qt2.View(*bu), M, F, K, 1.0, GELU, g, u, F, h, F)
        got = backward(a, bg, GELU, g, u)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
