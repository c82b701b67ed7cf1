"""Calls that follow one another on a stream with nothing between them, each reading what the one
before it writes: every kernel is resident before its predecessor has ended.  The same chains with
the device waited for after each call give the bits to compare with."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
IGN, EPS = -100, 1e-5


class NormChain:
    """Layer norm backward -> norm of its dgamma and dbeta -> clipped in place -> their norm again -> clipped
    into the weights of a layer norm forward -> that."""

    def __init__(self, R, C, wd):
        e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.R, self.C = R, C
        self.x, self.dy, self.dx, self.y = (e(R, C) for _ in range(4))
        self.w, self.dg, self.db, self.w2, self.b2 = (e(C, dt=wd) for _ in range(5))
        self.mean, self.rstd, self.m2, self.r2 = (e(R, dt=FP) for _ in range(4))
        self.n = [e(1, dt=FP) for _ in range(3)]
        self.grads = tr.GradList([self.dg, self.db])
        self.onto = tr.GradList([self.dg, self.db], [self.w2, self.b2])
        self.ws = qt2.alloc_workspace(max(tr.qt2_layernorm_bwd_workspace_size(R, C),
                                          tr.qt2_grad_norm_workspace_size(self.grads)))

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda t, std=1.0: t.copy_(torch.randn(t.shape, generator=g, device="cuda") * std)  # noqa: E731
        rn(self.x), rn(self.dy, 1e-2 * (1 + seed)), rn(self.w)
        rn(self.mean, 0.1), self.rstd.copy_(torch.rand(self.R, generator=g, device="cuda") + 0.5)

    def calls(self):
        R, C, ws, n = self.R, self.C, self.ws, self.ws.numel()
        yield lambda: tr.qt2_layernorm_bwd(self.dy, C, self.x, R, C, C, self.w, self.mean, self.rstd, self.dx, C,
                                           self.dg, self.db, ws, n)
        yield lambda: tr.qt2_grad_norm(self.grads, self.n[0], ws, n)
        yield lambda: tr.qt2_grad_clip(self.grads, self.n[0], 0.05)
        yield lambda: tr.qt2_grad_norm(self.grads, self.n[1], ws, n)
        yield lambda: tr.qt2_grad_clip(self.onto, self.n[1], 0.01)
        yield lambda: tr.qt2_layernorm_fwd(self.x, R, C, C, self.w2, self.b2, EPS, self.y, C, self.m2, self.r2)
        yield lambda: tr.qt2_grad_norm(self.onto, self.n[2], ws, n)

    def outputs(self):
        return [self.dx, self.dg, self.db, self.w2, self.b2, self.y, self.m2, self.r2, *self.n]


class HeadChain:
    """Head loss and its gradients -> their norm -> clipped in place -> their norm again -> the clipped dx
    through a layer norm backward whose weight is a row of the clipped dw -> the norm of that."""

    def __init__(self, T, K, V, dwd):
        e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.T, self.K, self.V = T, K, V
        self.x, self.dx, self.dz, self.w = e(T, K), e(T, K), e(T, K), e(V, K)
        self.dw, self.dg = e(V, K, dt=dwd), e(K, dt=dwd)
        self.loss, self.lse, self.dloss, self.mean, self.rstd = (e(T, dt=FP) for _ in range(5))
        self.targets = e(T, dt=torch.int64)
        self.n = [e(1, dt=FP) for _ in range(3)]
        self.grads, self.last = tr.GradList([self.dw, self.dx]), tr.GradList([self.dz, self.dg])
        self.code = tr._DTYPE[dwd]
        self.ws = qt2.alloc_workspace(max(tr.qt2_linear_xent_fwd_workspace_size(T, K, V),
                                          tr.qt2_linear_xent_bwd_workspace_size(T, K, V),
                                          tr.qt2_layernorm_bwd_workspace_size(T, K),
                                          tr.qt2_grad_norm_workspace_size(self.grads)))

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda t, std=1.0: t.copy_(torch.randn(t.shape, generator=g, device="cuda") * std)  # noqa: E731
        rn(self.x), rn(self.w, 0.05), rn(self.mean, 0.1)
        self.targets.copy_(torch.randint(0, self.V, (self.T,), generator=g, device="cuda"))
        self.targets[::7] = IGN
        self.dloss.copy_(torch.rand(self.T, generator=g, device="cuda") * (1 + seed) / self.T)
        self.rstd.copy_(torch.rand(self.T, generator=g, device="cuda") + 0.5)

    def calls(self):
        T, K, V, ws, n = self.T, self.K, self.V, self.ws, self.ws.numel()
        yield lambda: tr.qt2_linear_xent_fwd(self.x, self.w, self.targets, T, K, V, K, K, IGN, self.loss, self.lse, ws, n)
        yield lambda: tr.qt2_linear_xent_bwd(self.x, self.w, self.targets, self.lse, self.dloss, T, K, V, K, K, IGN,
                                             self.dx, K, self.dw, self.code, K, ws, n)
        yield lambda: tr.qt2_grad_norm(self.grads, self.n[0], ws, n)
        yield lambda: tr.qt2_grad_clip(self.grads, self.n[0], 0.05)
        yield lambda: tr.qt2_grad_norm(self.grads, self.n[1], ws, n)
        yield lambda: tr.qt2_layernorm_bwd(self.dx, K, self.x, T, K, K, self.dw[self.V // 2], self.mean, self.rstd,
                                           self.dz, K, self.dg, None, ws, n)
        yield lambda: tr.qt2_grad_norm(self.last, self.n[2], ws, n)

    def outputs(self):
        return [self.loss, self.lse, self.dx, self.dw, self.dz, self.dg, *self.n]


CHAINS = [(NormChain, (64, 40, FP)), (NormChain, (200, 2048, BF)), (NormChain, (3000, 1600, FP)),
          (NormChain, (40, 20000, FP)), (HeadChain, (20, 128, 600, FP)), (HeadChain, (300, 264, 1500, BF)),
          (HeadChain, (700, 512, 9000, FP))]


@pytest.mark.parametrize("kind,sizes", CHAINS)
def test_next_call_sees_what_the_last_one_wrote(kind, sizes):
    s = kind(*sizes)
    want = []
    for seed in range(4):
        s.fill(seed)
        for call in s.calls():
            torch.cuda.synchronize()
            call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in s.outputs()])
        assert all(torch.isfinite(t).all() for t in want[-1]) and (want[-1][-1] > 0).all()
    # other inputs, other outputs (but the norm of what was clipped to a norm)
    assert not any(torch.equal(a, b) for a, b in zip(want[0], want[1]) if a.numel() > 1)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        for call in s.calls():
            call()
    for run in (lambda: [call() for call in s.calls()], graph.replay):
        for _ in range(3):
            for seed in range(4):
                s.fill(seed)
                torch.cuda.synchronize()
                run()
                torch.cuda.synchronize()
                for k, (a, b) in enumerate(zip(s.outputs(), want[seed])):
                    assert torch.equal(a, b), (seed, k)
        # passes right behind one another, the inputs of the first
        s.fill(0)
        torch.cuda.synchronize()
        for _ in range(5):
            run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(s.outputs(), want[0]))
    assert tr.qt2_train_device_status() == 0
