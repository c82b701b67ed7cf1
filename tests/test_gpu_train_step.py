"""A training step of the operators together, as they are used: norm, quantized linear, norm, head
loss, and back through all of them to the clipped gradients.  Every operator's outputs are checked
against the 64-bit formulas on the inputs it was given by the one before."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref
from tests.test_gpu_grad import REL
from tests.test_gpu_norm import row_depth

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
M, D, H, V, IGN, EPS, SEED = 384, 256, 512, 1031, -100, 1e-5, 77


class Step:
    """Buffers of one model's step: norm (D), quantized linear D -> H, norm (H), head H -> V."""

    def __init__(self, seed, dw_dtype=FP):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s, std=1.0, dt=BF: (torch.randn(s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
        e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.x, self.w, self.head = rn(M, D), rn(H, D, std=0.02), rn(V, H, std=0.05)
        self.g1, self.b1 = 1 + rn(D, std=0.1, dt=FP), rn(D, std=0.1, dt=FP)
        self.g2, self.b2 = 1 + rn(H, std=0.1, dt=FP), rn(H, std=0.1, dt=FP)
        self.y = torch.randint(0, V, (M,), generator=g, device="cuda")
        self.y[::9] = IGN
        self.dloss = torch.where(self.y == IGN, 0.0, 1.0 / (self.y != IGN).sum()).float()
        self.n1, self.n2, self.z = e(M, D), e(M, H), e(M, H)
        self.m1, self.r1, self.m2, self.r2, self.loss, self.lse = (e(M, dt=FP) for _ in range(6))
        self.dn2, self.dz, self.dn1, self.dx = e(M, H), e(M, H), e(M, D), e(M, D)
        self.dhead, self.dw = e(V, H, dt=dw_dtype), e(H, D, dt=FP)
        self.dg1, self.db1, self.dg2, self.db2 = e(D, dt=FP), e(D, dt=FP), e(H, dt=FP), e(H, dt=FP)
        self.grads = tr.GradList([self.dhead, self.dw, self.dg1, self.db1, self.dg2, self.db2])
        self.raw = [torch.empty_like(t) for t in self.grads.grads]
        self.norm = e(1, dt=FP)
        # one workspace: the calls follow one another on one stream
        size = max(qt2.qt2_linear_fwd_workspace_size(M, D, H), qt2.qt2_linear_bwd_workspace_size(M, D, H),
                   tr.qt2_linear_xent_fwd_workspace_size(M, H, V), tr.qt2_linear_xent_bwd_workspace_size(M, H, V),
                   tr.qt2_layernorm_bwd_workspace_size(M, max(D, H)), tr.qt2_grad_norm_workspace_size(self.grads))
        self.ws = qt2.alloc_workspace(size)

    def run(self):
        ws, n = self.ws, self.ws.numel()
        tr.qt2_layernorm_fwd(self.x, M, D, D, self.g1, self.b1, EPS, self.n1, D, self.m1, self.r1)
        qt2.qt2_linear_fwd(self.n1, self.w, M, D, H, self.z, ws, n)
        tr.qt2_layernorm_fwd(self.z, M, H, H, self.g2, self.b2, EPS, self.n2, H, self.m2, self.r2)
        tr.qt2_linear_xent_fwd(self.n2, self.head, self.y, M, H, V, H, H, IGN, self.loss, self.lse, ws, n)
        tr.qt2_linear_xent_bwd(self.n2, self.head, self.y, self.lse, self.dloss, M, H, V, H, H, IGN, self.dn2, H,
                               self.dhead, tr._DTYPE[self.dhead.dtype], H, ws, n)
        tr.qt2_layernorm_bwd(self.dn2, H, self.z, M, H, H, self.g2, self.m2, self.r2, self.dz, H, self.dg2, self.db2,
                             ws, n)
        qt2.qt2_linear_bwd(self.dz, self.n1, self.w, M, D, H, SEED, self.dn1, self.dw, qt2.QT2_DTYPE_F32, ws, n)
        tr.qt2_layernorm_bwd(self.dn1, D, self.x, M, D, D, self.g1, self.m1, self.r1, self.dx, D, self.dg1, self.db1,
                             ws, n)
        for r, t in zip(self.raw, self.grads.grads):
            r.copy_(t)
        tr.qt2_grad_norm(self.grads, self.norm, ws, n)
        tr.qt2_grad_clip(self.grads, self.norm, 0.01)

    def outputs(self):
        return [self.loss, self.dx, self.norm, *self.grads.grads]


@pytest.mark.parametrize("dw_dtype", [FP, BF])
def test_step_matches_the_formulas(dw_dtype):
    s = Step(1, dw_dtype)
    s.run()
    assert qt2.qt2_device_status() == 0 and tr.qt2_train_device_status() == 0
    for x, g, b, y, m, r in ((s.x, s.g1, s.b1, s.n1, s.m1, s.r1), (s.z, s.g2, s.b2, s.n2, s.m2, s.r2)):
        want, bound = ref.norm_fwd(x, g, b, EPS)
        for a, w, e in zip((y, m, r), want, bound):
            ref.check(a, w, e)
    want, bound = ref.xent(s.n2, s.head, s.y, IGN, s.dloss)
    for a, w, e in zip((s.loss, s.lse, s.dn2, s.raw[0]), want, bound):
        ref.check(a, w, e)
    for dy, x, g, m, r, outs in ((s.dn2, s.z, s.g2, s.m2, s.r2, (s.dz, s.raw[4], s.raw[5])),
                                 (s.dn1, s.x, s.g1, s.m1, s.r1, (s.dx, s.raw[2], s.raw[3]))):
        want, bound = ref.norm_bwd(dy, x, g, m, r, row_depth(M))
        for a, w, e in zip(outs, want, bound):
            ref.check(a, w, e)
    norm = sum(t.double().square().sum() for t in s.raw).sqrt().item()
    assert abs(s.norm.item() - norm) <= REL * norm and norm > 0.01
    f = torch.tensor(0.01, device="cuda") / (s.norm + 1e-6)
    for t, r in zip(s.grads.grads, s.raw):
        assert torch.equal(t, (r.float() * f).to(t.dtype))


def test_step_in_a_graph_and_two_at_once():
    """The step captured and replayed, beside another that runs eagerly on its own stream and
    workspace, gives the bits of the steps alone."""
    a, b = Step(1), Step(2)
    want = []
    for s in (a, b):
        s.run()
        want.append([t.clone() for t in s.outputs()])
    torch.cuda.synchronize()
    graph, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        a.run()
    for s in (a, b):
        for t in s.outputs():
            t.fill_(3.0)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
        with torch.cuda.stream(other):
            b.run()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        assert all(torch.equal(t, v) for t, v in zip(s.outputs(), w))
    assert qt2.qt2_device_status() == 0 and tr.qt2_train_device_status() == 0


def test_between_copies_and_fills_in_a_graph():
    """Nodes that are no kernels before and after each call of a captured graph."""
    a = Step(3)
    a.run()
    want = [t.clone() for t in a.outputs()]
    x = a.x.clone()
    ws, n = a.ws, a.ws.numel()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        a.n1.zero_()
        a.x.copy_(x)
        tr.qt2_layernorm_fwd(a.x, M, D, D, a.g1, a.b1, EPS, a.n1, D, a.m1, a.r1)
        qt2.qt2_linear_fwd(a.n1, a.w, M, D, H, a.z, ws, n)
        tr.qt2_layernorm_fwd(a.z, M, H, H, a.g2, a.b2, EPS, a.n2, H, a.m2, a.r2)
        a.loss.zero_()
        tr.qt2_linear_xent_fwd(a.n2, a.head, a.y, M, H, V, H, H, IGN, a.loss, a.lse, ws, n)
        ws.zero_()
        tr.qt2_linear_xent_bwd(a.n2, a.head, a.y, a.lse, a.dloss, M, H, V, H, H, IGN, a.dn2, H, a.dhead, 1, H, ws, n)
        keep = a.dn2.clone()
        a.norm.zero_()
        tr.qt2_grad_norm(a.grads, a.norm, ws, n)
        norm = a.norm.clone()
        a.norm.fill_(5.0)
    a.x.zero_(), a.loss.fill_(9.0)
    dn2 = a.dn2.clone()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.loss, want[0]) and torch.equal(keep, dn2) and (a.norm == 5.0).all()
    exact = sum(t.double().square().sum() for t in a.grads.grads).sqrt().item()
    assert abs(norm.item() - exact) <= REL * exact


def test_calls_from_several_threads():
    """Host threads that call at once, each on a stream and workspace of its own."""
    import threading
    steps = [Step(k) for k in range(4)]
    want = []
    for s in steps:
        s.run()
        want.append([t.clone() for t in s.outputs()])
        for t in s.outputs():
            t.fill_(3.0)
    torch.cuda.synchronize()
    errors = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    s.run()
        except Exception as e:   # reported by the test, not lost with the thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w))
