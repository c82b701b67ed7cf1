"""The training operators' library (include/qt2_train.h): exports, host-side refusals, workspace
queries and injected failures, without a GPU (fake, never-dereferenced device addresses)."""
import ctypes
import subprocess

import pytest
import torch

from nvfp4_quantized_b200 import build as qbuild
from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr

OK, ARG, SHAPE, ALIGN, WS = 0, qt2.QT2_ERR_INVALID_ARG, qt2.QT2_ERR_SHAPE, qt2.QT2_ERR_ALIGN, qt2.QT2_ERR_WORKSPACE
BF16, F32 = qt2.QT2_DTYPE_BF16, qt2.QT2_DTYPE_F32


@pytest.fixture(scope="module")
def L():
    qbuild.build_train()
    return tr.lib()


def test_exports_every_header_function(L):
    names = tr.header_functions()
    assert "qt2_linear_xent_bwd" in names
    for path in (tr.LIB_PATH, qbuild.build_train(checked=True)):
        out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True).stdout
        exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
        assert {e for e in exported if e.startswith("qt2")} == set(names)
        C = ctypes.CDLL(path)
        assert C.qt2_train_build_checked() == (path != qbuild.TRAIN_LIB)


def _norm_fwd(L, x=0x1000, xd=BF16, rows=3, cols=5, ldx=8, w=0x2000, b=0x3000, wd=F32, eps=1e-5, y=0x4000, ldy=8,
              mean=0x5000, rstd=0x6000):
    return L.qt2_layernorm_fwd(x, xd, rows, cols, ldx, w, b, wd, eps, y, ldy, mean, rstd, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), ARG), (dict(y=None), ARG), (dict(xd=2), ARG), (dict(wd=-1), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(rows=0), SHAPE), (dict(cols=0), SHAPE),
    (dict(rows=-4), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(cols=9), SHAPE), (dict(ldy=0), SHAPE),
    (dict(ldx=9), ALIGN), (dict(ldy=12), ALIGN), (dict(x=0x1008), ALIGN), (dict(y=0x4002), ALIGN),
    (dict(w=0x2004), ALIGN), (dict(b=0x3008), ALIGN), (dict(mean=0x5002), ALIGN), (dict(rstd=0x6001), ALIGN)])
def test_layernorm_fwd_refusals(L, bad, status):
    assert _norm_fwd(L, **bad) == status


def _norm_bwd(L, dy=0x1000, lddy=8, x=0x2000, xd=BF16, rows=3, cols=5, ldx=8, w=0x3000, wd=F32, mean=0x4000,
              rstd=0x5000, dx=0x6000, lddx=8, dw=0x7000, db=0x8000, ws=0x10000, n=1 << 20):
    return L.qt2_layernorm_bwd(dy, lddy, x, xd, rows, cols, ldx, w, wd, mean, rstd, dx, lddx, dw, db, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dy=None), ARG), (dict(x=None), ARG), (dict(mean=None), ARG), (dict(rstd=None), ARG),
    (dict(dx=None, dw=None, db=None), ARG), (dict(xd=7), ARG), (dict(wd=7), ARG), (dict(rows=0), SHAPE),
    (dict(cols=-1), SHAPE), (dict(lddy=4), SHAPE), (dict(lddx=4), SHAPE), (dict(lddy=9), ALIGN),
    (dict(dy=0x1008), ALIGN), (dict(dx=0x6008), ALIGN), (dict(dw=0x7004), ALIGN), (dict(db=0x8004), ALIGN),
    (dict(w=0x3002), ALIGN), (dict(ws=None), WS), (dict(n=0), WS), (dict(ws=0x10010), ALIGN)])
def test_layernorm_bwd_refusals(L, bad, status):
    assert _norm_bwd(L, **bad) == status


def _xent_fwd(L, x=0x1000, w=0x2000, t=0x3000, T=3, K=5, V=7, ldx=8, ldw=8, ignore=-100, loss=0x4000, lse=0x5000,
              ws=0x10000, n=1 << 30):
    return L.qt2_linear_xent_fwd(x, w, t, T, K, V, ldx, ldw, ignore, loss, lse, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(t=None), ARG), (dict(loss=None), ARG), (dict(lse=None), ARG),
    (dict(T=0), SHAPE), (dict(K=0), SHAPE), (dict(V=0), SHAPE), (dict(V=1 << 30), SHAPE), (dict(ldx=0), SHAPE),
    (dict(K=9), SHAPE), (dict(ldw=12), ALIGN), (dict(ldx=9), ALIGN), (dict(x=0x1008), ALIGN), (dict(w=0x2002), ALIGN),
    (dict(t=0x3004), ALIGN), (dict(loss=0x4002), ALIGN), (dict(lse=0x5002), ALIGN), (dict(ws=None), WS),
    (dict(n=8), WS), (dict(ws=0x10080), ALIGN)])
def test_xent_fwd_refusals(L, bad, status):
    assert _xent_fwd(L, **bad) == status


def _xent_bwd(L, x=0x1000, w=0x2000, t=0x3000, lse=0x4000, g=0x5000, T=3, K=5, V=7, ldx=8, ldw=8, ignore=-100,
              dx=0x6000, lddx=8, dw=0x7000, dwd=BF16, lddw=8, ws=0x10000, n=1 << 30):
    return L.qt2_linear_xent_bwd(x, w, t, lse, g, T, K, V, ldx, ldw, ignore, dx, lddx, dw, dwd, lddw, ws, n, None)


@pytest.mark.parametrize("bad,status", [
    (dict(lse=None), ARG), (dict(g=None), ARG), (dict(dx=None, dw=None), ARG), (dict(dwd=3), ARG), (dict(t=None), ARG),
    (dict(T=-1), SHAPE), (dict(lddx=0), SHAPE), (dict(lddw=4), SHAPE), (dict(lddw=9), ALIGN), (dict(lddx=12), ALIGN),
    (dict(dx=0x6008), ALIGN), (dict(dw=0x7008), ALIGN), (dict(lse=0x4002), ALIGN), (dict(g=0x5002), ALIGN),
    (dict(ws=None), WS), (dict(n=1), WS), (dict(ws=0x10001), ALIGN)])
def test_xent_bwd_refusals(L, bad, status):
    assert _xent_bwd(L, **bad) == status


def _grads(*rows):
    a = (tr.GradC * max(1, len(rows)))()
    for d, (g, o, n, t) in zip(a, rows):
        d.grad, d.out, d.numel, d.dtype = g, o, n, t
    return a


@pytest.mark.parametrize("rows,count,norm_status,clip_status", [
    ([(0x1000, 0x2000, 4, F32)], 0, SHAPE, SHAPE), ([(0x1000, 0x2000, 4, 5)], 1, ARG, ARG),
    ([(0x1000, 0x2000, -1, F32)], 1, SHAPE, SHAPE), ([(None, 0x2000, 4, F32)], 1, ARG, ARG),
    ([(0x1002, 0x2000, 4, F32)], 1, ALIGN, ALIGN), ([(0x1001, 0x2000, 4, BF16)], 1, ALIGN, ALIGN),
    ([(0x1000, None, 4, F32)], 1, None, ARG), ([(0x1000, 0x2002, 4, F32)], 1, None, ALIGN),
    ([(0x1000, 0x2000, 1 << 44, BF16)], 1, SHAPE, SHAPE)])
def test_grad_refusals(L, rows, count, norm_status, clip_status):
    a = _grads(*rows)
    n = ctypes.c_size_t(0)
    if norm_status is not None:
        assert L.qt2_grad_norm_workspace_size(ctypes.addressof(a), count, ctypes.byref(n)) == norm_status
        assert L.qt2_grad_norm(ctypes.addressof(a), count, 0x8000, 0x10000, 1 << 20, None) == norm_status
    assert L.qt2_grad_clip(ctypes.addressof(a), count, 0x8000, 1.0, None) == clip_status


def test_grad_scalar_refusals(L):
    a = _grads((0x1000, 0x2000, 4, F32))
    p = ctypes.addressof(a)
    assert L.qt2_grad_norm(None, 1, 0x8000, 0x10000, 1 << 20, None) == ARG
    assert L.qt2_grad_norm(p, 1, None, 0x10000, 1 << 20, None) == ARG
    assert L.qt2_grad_norm(p, 1, 0x8002, 0x10000, 1 << 20, None) == ALIGN
    assert L.qt2_grad_norm(p, 1, 0x8000, None, 1 << 20, None) == WS
    assert L.qt2_grad_norm(p, 1, 0x8000, 0x10000, 4, None) == WS
    assert L.qt2_grad_clip(p, 1, None, 1.0, None) == ARG
    assert L.qt2_grad_clip(p, 1, 0x8000, -1.0, None) == ARG
    assert L.qt2_grad_clip(p, 1, 0x8000, float("nan"), None) == ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_valid_calls_without_gpu_fail_loudly(L):
    a = _grads((0x1000, 0x2000, 4, F32))
    for st in (_norm_fwd(L), _norm_bwd(L), _xent_fwd(L), _xent_bwd(L),
               L.qt2_grad_norm(ctypes.addressof(a), 1, 0x8000, 0x10000, 1 << 20, None),
               L.qt2_grad_clip(ctypes.addressof(a), 1, 0x8000, 1.0, None)):
        assert st == qt2.QT2_ERR_DEVICE


def test_workspace_queries(L):
    assert tr.qt2_linear_xent_fwd_workspace_size(1, 1, 1) > 0
    # P, the largest part of the backward pass's workspace, is bounded by a piece of the vocabulary
    small, large = (tr.qt2_linear_xent_bwd_workspace_size(4096, 1024, v) for v in (65536, 1 << 20))
    assert large <= small + (64 << 20)
    for f in (tr.qt2_linear_xent_fwd_workspace_size, tr.qt2_linear_xent_bwd_workspace_size):
        for dims in ((0, 1, 1), (1, -1, 1), (1, 1, 1 << 30), ((1 << 29), (1 << 29), 1), (1, 1 << 20, 1 << 24)):
            with pytest.raises(qt2.QT2Error) as e:
                f(*dims)
            assert e.value.status == SHAPE
    with pytest.raises(qt2.QT2Error) as e:
        tr.qt2_layernorm_bwd_workspace_size(0, 8)
    assert e.value.status == SHAPE
    assert L.qt2_layernorm_bwd_workspace_size(1, 1, None) == ARG


def _calls(L):
    many = _grads(*[(0x1000 + 16 * i, 0x200000 + 16 * i, 3, BF16) for i in range(300)])
    p = ctypes.addressof(many)
    return {
        "norm_fwd": lambda: _norm_fwd(L), "norm_bwd": lambda: _norm_bwd(L), "xent_fwd": lambda: _xent_fwd(L),
        # two pieces of the vocabulary, and a contraction split
        "xent_bwd": lambda: _xent_bwd(L, T=20000, V=9000, K=64, ldx=64, ldw=64, lddx=64, lddw=64, n=1 << 40),
        "grad_norm": lambda: L.qt2_grad_norm(p, 300, 0x8000, 0x10000, 1 << 20, None),
        "grad_clip": lambda: L.qt2_grad_clip(p, 300, 0x8000, 1.0, None), "many": many}


@pytest.mark.parametrize("name", ["norm_fwd", "norm_bwd", "xent_fwd", "xent_bwd", "grad_norm", "grad_clip"])
def test_injected_failures_at_every_site(L, name):
    """Skipping every CUDA call completes with QT2_OK having touched nothing; failing the k-th one
    returns that site's error and enqueues nothing further."""
    calls = _calls(L)
    call = calls[name]
    with tr.fault_hook(lambda site: qt2.FAULT_SKIP) as h:
        assert call() == OK
    sites = list(h.sites)
    assert sites[0] == "device" and "launch" in sites
    for k in range(len(sites)):
        seen = []

        def decide(site, k=k, seen=seen):
            seen.append(site)
            return qt2.FAULT_FAIL if len(seen) == k + 1 else qt2.FAULT_SKIP
        with tr.fault_hook(decide):
            st = call()
        assert len(seen) == k + 1, (k, seen)
        assert st == (qt2.QT2_ERR_DEVICE if sites[k] == "device" else qt2.QT2_ERR_CUDA), (k, sites[k], st)


def test_binding_refuses_types_before_the_call(monkeypatch):
    """Wrong element types and tensors of another device raise without reaching the library."""
    f, h, i = torch.zeros(8), torch.zeros(8, dtype=torch.float16), torch.zeros(8, dtype=torch.int32)
    b, g, long = torch.zeros(8, dtype=torch.bfloat16), torch.zeros(8), torch.zeros(16)
    cases = [
        lambda: tr.qt2_layernorm_fwd(h, 1, 8, 8, f, f, 1e-5, h, 8, f, f),
        lambda: tr.qt2_layernorm_fwd(f, 1, 8, 8, f, b, 1e-5, f, 8, f, f),
        lambda: tr.qt2_layernorm_fwd(f, 1, 8, 8, f, f, 1e-5, b, 8, f, f),
        lambda: tr.qt2_layernorm_fwd(f, 1, 8, 8, f, f, 1e-5, f, 8, b, f),
        lambda: tr.qt2_layernorm_bwd(b, 8, f, 1, 8, 8, f, f, f, f, 8, f, f, f, 32),
        lambda: tr.qt2_linear_xent_fwd(f, b, i.long(), 1, 8, 1, 8, 8, -100, f, f, f, 32),
        lambda: tr.qt2_linear_xent_fwd(b, b, i, 1, 8, 1, 8, 8, -100, f, f, f, 32),
        lambda: tr.qt2_linear_xent_bwd(b, b, i.long(), f, f, 1, 8, 1, 8, 8, -100, b, 8, b, F32, 8, f, 32),
        lambda: tr.GradList([h]), lambda: tr.GradList([f], [b]), lambda: tr.GradList([f], []),
        lambda: tr.GradList([f], [torch.zeros(7)]), lambda: tr.GradList([torch.zeros(4, 4).t()]),
        # what one entry writes, another reads or writes
        lambda: tr.GradList([f, f]), lambda: tr.GradList([f, g], [f, f]), lambda: tr.GradList([f, g], [g, f]),
        lambda: tr.GradList([long[:8]], [long[4:12]]), lambda: tr.GradList([long[:8], f], [f, long[7:15]]),
    ]
    for k, case in enumerate(cases):
        with pytest.raises(qt2.QT2Error) as e:
            case()
        assert e.value.status == ARG, k
    tr.GradList([f, f], [g, torch.zeros(8)])   # read twice, written apart
    tr.GradList([long[:8], long[8:]], [g, f])
    tr.GradList([long[:8], long[8:]])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # CPU tensors are on no CUDA device
    with pytest.raises(qt2.QT2Error) as e:
        tr.qt2_layernorm_fwd(f, 1, 8, 8, f, f, 1e-5, f, 8, f, f)
    assert e.value.status == qt2.QT2_ERR_DEVICE
