"""The head loss where what lies past 2^31 elements of w decides the result: leaving it out, or reading
it elsewhere, shifts every row's lse by units."""
import math

import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import train_ref as ref
from tests.test_gpu_xent_rounding import SIGMA, rounding

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
K, V, FAR = 16384, 140000, (1 << 31) // 16384


def pieces(lo=0, hi=V, n=20000):
    return [slice(v, min(v + n, hi)) for v in range(lo, hi, n)]


@pytest.mark.parametrize("T,dwd", [(20, FP), (40, BF)])
def test_rows_past_2_31_elements_decide(T, dwd):
    """Rows from FAR on have logits of standard deviation 3.8, the others of 0.6: log sum exp is about 16.5 with
    them and 12 without.  Sums along K of either sign stay below 32 (more than 7 standard deviations), so that each of
    their K / 16 + 16 additions loses at most 2^-23 of that: p is off by 4e-3 of itself at most."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, K), generator=g, device="cuda").to(BF)
    w = torch.empty((V, K), dtype=BF, device="cuda")
    for s in pieces(0, FAR) + pieces(FAR):
        w[s] = torch.randn((s.stop - s.start, K), generator=g, device="cuda") * (0.005 if s.start < FAR else 0.03)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::2] = FAR + torch.randint(0, V - FAR, (len(y[::2]),), generator=g, device="cuda")
    y[:2] = torch.tensor([FAR - 1, FAR], device="cuda")
    dloss = (torch.rand(T, generator=g, device="cuda") + 0.5) / T
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty((V, K), dtype=dwd, device="cuda")
    ws = qt2.alloc_workspace(max(tr.qt2_linear_xent_fwd_workspace_size(T, K, V),
                                 tr.qt2_linear_xent_bwd_workspace_size(T, K, V)))
    tr.qt2_linear_xent_fwd(x, w, y, T, K, V, K, K, -100, loss, lse, ws, ws.numel())
    tr.qt2_linear_xent_bwd(x, w, y, lse, dloss, T, K, V, K, K, -100, dx, K, dw, tr._DTYPE[dwd], K, ws, ws.numel())
    l = torch.cat([x.double() @ w[s].double().T for s in pieces()], 1)
    want = torch.logsumexp(l, 1)
    assert (want - torch.logsumexp(l[:, :FAR], 1) > 3).all() and l.abs().max() < 28
    off = 2.0 ** -23 * 32 * (K / 16 + 16)
    assert off < 4.1e-3
    assert ((lse - want).abs() <= off + 2.0 ** -20 * want.abs()).all()
    assert ((loss - (want - l.gather(1, y[:, None])[:, 0])).abs() <= off + 2.0 ** -20 * want.abs()).all()
    p = torch.exp(l - want[:, None]) * dloss.double()[:, None]
    hit = torch.zeros_like(p).scatter(1, y[:, None], dloss.double()[:, None])
    P = p - hit
    target = hit.sum(0) > 0

    def same(got, want, var, size, what):
        err = (got.double() - want).norm().item()
        most = 1.1 * (var + rounding(want, got.dtype)).sum().sqrt().item() + size
        assert err <= most, (what, err / want.norm().item(), most / want.norm().item())
        assert most <= (2 * off + 4e-3) * want.norm().item()   # of the order of the roundings: nothing left out fits in

    sums = [torch.zeros((T, K), dtype=torch.float64, device="cuda") for _ in range(3)]
    for s in pieces():
        ws64 = w[s].double()
        for acc, m, b in zip(sums, (P, torch.where(hit > 0, 0.0, P) ** 2, p), (ws64, ws64 ** 2, ws64)):
            acc += m[:, s] @ b
    same(dx, sums[0], SIGMA ** 2 * sums[1], 2 * off * sums[2].norm().item(), "dx")
    x64 = x.double()
    for s in (slice(0, 3000), slice(FAR - 2000, FAR), slice(FAR, FAR + 2000), slice(V - 3000, V)):
        for rows in (~target[s], target[s]):   # what the softmax gives alone, and with targets
            if rows.any():
                m = P[:, s][:, rows]
                var = 2 * SIGMA ** 2 * (torch.where(hit[:, s][:, rows] > 0, 0.0, m) ** 2).T @ x64 ** 2
                # p's error, and c x as two bf16 numbers (2^-8 of 2^-8 at most) at the targets
                size = 2 * off * (p[:, s][:, rows].T @ x64).norm() + 2.0 ** -16 * (hit[:, s][:, rows].T @ x64.abs()).norm()
                same(dw[s][rows], m.T @ x64, var, size.item(), ("dw", s))
    assert tr.qt2_train_device_status() == 0
