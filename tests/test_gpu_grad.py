"""Global gradient norm and clipping on the GPU against 64 bits."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32

# fp32 sums of at most 8 squares (8 half steps and the square's own), then fp64: the norm is off by
# half of that, and its own rounding
REL = 5.5 * ref.U


def norm(gl):
    n = torch.full((1,), -1.0, device="cuda")
    ws = qt2.alloc_workspace(tr.qt2_grad_norm_workspace_size(gl))
    ws.fill_(0xFF)
    tr.qt2_grad_norm(gl, n, ws, ws.numel())
    return n


def packed(sizes, dtypes, seed=0, scale=1.0):
    """Tensors one behind the other in one buffer a type (any alignment), with a guard element between."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bufs = {d: torch.full((sum(sizes) + len(sizes) + 1,), 7.0, dtype=d, device="cuda") for d in (BF, FP)}
    at, out = {BF: 1, FP: 1}, []
    for n, d in zip(sizes, dtypes):
        t = bufs[d][at[d]:at[d] + n]
        t.copy_(torch.randn(n, generator=g, device="cuda") * scale)
        out.append(t)
        at[d] += n + 1
    return out, bufs


def exact_norm(ts):
    return sum(t.double().square().sum() for t in ts).sqrt().item()


def clipped(t, n, max_norm):
    f = (torch.tensor(max_norm, device="cuda") / (n + 1e-6)).clamp(max=1.0)
    return (t.float() * f).to(t.dtype)


LISTS = [
    ([1], [FP]), ([1], [BF]), ([3, 0, 5], [FP, BF, BF]), ([8191, 8192, 8193], [BF, FP, BF]),
    ([7, 8, 9, 15, 16, 17, 31, 33] * 5, [BF, FP] * 20), ([1] * 129, [BF] * 129), ([2, 0, 3] * 300, [FP, BF, BF] * 300),
    ([1 << 20, 5, (1 << 21) + 3], [FP, BF, BF]), ([12345] * 700, ([BF] * 3 + [FP]) * 175), ([16777217], [BF])]


@pytest.mark.parametrize("k", range(len(LISTS)))
def test_norm_and_clip(k):
    sizes, dtypes = LISTS[k]
    ts, bufs = packed(sizes, dtypes, seed=k)
    before = {d: b.clone() for d, b in bufs.items()}
    outs, obufs = packed(sizes, dtypes, seed=99)
    gl = tr.GradList(ts, outs)
    n = norm(gl)
    want = exact_norm(ts)
    assert abs(n.item() - want) <= REL * want
    for max_norm in (0.25 * want, 4 * want, 0.0):
        tr.qt2_grad_clip(gl, n, max_norm)
        for t, o in zip(ts, outs):
            assert torch.equal(o, clipped(t, n, max_norm))
    assert all(torch.equal(b, before[d]) for d, b in bufs.items())          # the gradients stay
    guard = {BF: 1, FP: 1}
    for s, d in zip(sizes, dtypes):   # and so do the elements between the outputs
        assert obufs[d][guard[d] - 1] == 7.0 and obufs[d][guard[d] + s] == 7.0
        guard[d] += s + 1
    # in place
    gi = tr.GradList(ts)
    tr.qt2_grad_clip(gi, n, 4 * want)
    assert all(torch.equal(b, before[d]) for d, b in bufs.items())
    expect = [clipped(t, n, 0.5 * want) for t in ts]
    tr.qt2_grad_clip(gi, n, 0.5 * want)
    assert all(torch.equal(t, e) for t, e in zip(ts, expect))
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("shift", range(8))
@pytest.mark.parametrize("dtype", [BF, FP])
def test_every_alignment(dtype, shift):
    """Source and output at every pair of offsets within 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(shift)
    for other in range(8):
        for n in (1, 5, 8, 23, 2049):
            src = torch.randn(n + 16, generator=g, device="cuda").to(dtype)
            dst = torch.full((n + 16,), 7.0, dtype=dtype, device="cuda")
            t, o = src[shift:shift + n], dst[other:other + n]
            gl = tr.GradList([t], [o])
            v = norm(gl)
            want = exact_norm([t])
            assert abs(v.item() - want) <= REL * want
            tr.qt2_grad_clip(gl, v, 0.3 * want)
            assert torch.equal(o, clipped(t, v, 0.3 * want))
            assert (dst[:other] == 7.0).all() and (dst[other + n:] == 7.0).all()


@pytest.mark.parametrize("value", [1e-30, 1e-38, 1e-42, 1e25, 3e38])
def test_squares_beyond_fp32(value):
    """Elements whose squares leave fp32's range (the fp32 norm itself fits, or overflows to inf)."""
    for n in (1, 3, 1000):
        t = torch.full((n,), value, device="cuda")
        got = norm(tr.GradList([t, t.to(BF)])).item()
        want = torch.tensor(exact_norm([t, t.to(BF)])).float().item()
        if want == float("inf"):
            assert got == want
        else:   # half a step of a subnormal norm is absolute
            assert abs(got - want) <= REL * want + 2.0 ** -149
    mixed = torch.zeros(4096, device="cuda")
    mixed[::7] = value
    mixed[1] = 1.0
    got, want = norm(tr.GradList([mixed])).item(), torch.tensor(exact_norm([mixed])).float().item()
    assert got == want or abs(got - want) <= REL * want


def test_zeros_and_nonfinite():
    z = torch.zeros(5000, dtype=BF, device="cuda")
    gl = tr.GradList([z])
    n = norm(gl)
    assert n.item() == 0.0
    tr.qt2_grad_clip(gl, n, 1.0)
    assert (z == 0).all()
    empty = tr.GradList([torch.empty(0, device="cuda")])
    n = norm(empty)
    assert n.item() == 0.0
    tr.qt2_grad_clip(empty, n, 1.0)
    for bad in (float("inf"), float("-inf"), float("nan")):
        a, b = torch.ones(3000, device="cuda"), torch.ones(9, dtype=BF, device="cuda")
        a[1234] = bad
        oa, ob = torch.empty_like(a), torch.empty_like(b)
        gl = tr.GradList([a, b], [oa, ob])
        n = norm(gl)
        assert (n.isnan() if bad != bad else n.isinf()).all()
        tr.qt2_grad_clip(gl, n, 1.0)
        if bad != bad:
            assert oa.isnan().all() and ob.isnan().all()
        else:
            assert oa[1234].isnan() and (oa[:1234] == 0).all() and (ob == 0).all()


def test_same_bits_again_in_a_graph_and_on_two_streams():
    sizes = [100003, 17, 4096, 250000] * 40
    ts, _ = packed(sizes, [BF, FP, FP, BF] * 40)
    outs = [torch.empty_like(t) for t in ts]
    gl = tr.GradList(ts, outs)
    n = norm(gl)
    tr.qt2_grad_clip(gl, n, 1.0)
    want = [o.clone() for o in outs]
    torch.cuda.synchronize()
    outs2 = [torch.empty_like(t) for t in ts]
    gl2 = tr.GradList(ts, outs2)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    ns = [torch.zeros(1, device="cuda") for _ in sides]
    wss = [qt2.alloc_workspace(tr.qt2_grad_norm_workspace_size(gl)) for _ in sides]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, l, v, ws in zip(sides, (gl, gl2), ns, wss):
            tr.qt2_grad_norm(l, v, ws, ws.numel(), s)
            tr.qt2_grad_clip(l, v, 1.0, s)
    torch.cuda.synchronize()
    for v, os in zip(ns, (outs, outs2)):
        assert torch.equal(v, n) and all(torch.equal(a, b) for a, b in zip(os, want))
    graph = torch.cuda.CUDAGraph()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=sides[0]):
        tr.qt2_grad_norm(gl, ns[0], wss[0], wss[0].numel())
        tr.qt2_grad_clip(gl, ns[0], 1.0)
    gl.c[0].numel = 0   # the list was read when the call was made
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ns[0], n) and all(torch.equal(a, b) for a, b in zip(outs, want))
