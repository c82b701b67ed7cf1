"""A transformer block's operators (include/qt2_train.h): host-side refusals and injected failures, without a
GPU (fake, never-dereferenced device addresses)."""
import ctypes

import pytest
import torch

from nvfp4_quantized_b200 import build as qbuild
from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr

OK, ARG, SHAPE, ALIGN, WS = 0, qt2.QT2_ERR_INVALID_ARG, qt2.QT2_ERR_SHAPE, qt2.QT2_ERR_ALIGN, qt2.QT2_ERR_WORKSPACE
DEV, CUDA = qt2.QT2_ERR_DEVICE, qt2.QT2_ERR_CUDA


@pytest.fixture(scope="module")
def L():
    qbuild.build_train()
    return tr.lib()


def injected(call):
    """Skipping every CUDA call completes; failing the k-th returns that site's error and enqueues nothing further."""
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
        assert len(seen) == k + 1 and st == (DEV if sites[k] == "device" else CUDA), (k, sites[k], st)
    return sites


# ------------------------------------------------------------------------------------------ gated product
def view(codes=0x1000, scales=0x2000, scale=0x3000):
    return ctypes.byref(qt2.NVFP4ViewC(codes, scales, scale))


def gated(L, a=view(), bg=view(), bu=view(), M=128, F=256, K=384, act=0, gate=0x4000, up=0x5000, ldgu=256, h=0x6000, ldh=256):
    return L.qt2_gemm_nvfp4_gated(a, bg, bu, M, F, K, 1.0, act, gate, up, ldgu, h, ldh, None)


def gated_bwd(L, a=view(), b=view(), M=128, F=256, K=384, act=0, gate=0x4000, up=0x5000, ldgu=256, dgate=0x6000, dup=0x7000,
              lddgu=256, h=0x8000, ldh=256):
    return L.qt2_gemm_nvfp4_gated_bwd(a, b, M, F, K, 1.0, act, gate, up, ldgu, dgate, dup, lddgu, h, ldh, None)


SIZES = [(dict(M=0), SHAPE), (dict(F=0), SHAPE), (dict(K=-128), SHAPE), (dict(M=100), SHAPE), (dict(F=130), SHAPE), (dict(K=64), SHAPE),
         (dict(M=1 << 30), SHAPE), (dict(ldgu=248), SHAPE), (dict(ldh=8), SHAPE), (dict(ldgu=1 << 40), SHAPE),
         (dict(M=1 << 22, F=1 << 22, ldgu=1 << 22, ldh=1 << 22, lddgu=1 << 22), SHAPE),
         (dict(M=1 << 21, F=1 << 22, K=1 << 21, ldgu=1 << 22, ldh=1 << 22, lddgu=1 << 22), SHAPE),
         (dict(act=2), ARG), (dict(act=-1), ARG), (dict(a=None), ARG), (dict(a=view(codes=None)), ARG), (dict(a=view(scale=None)), ARG),
         (dict(a=view(codes=0x1008)), ALIGN), (dict(a=view(scales=0x2004)), ALIGN), (dict(a=view(scale=0x3002)), ALIGN),
         (dict(gate=0x4008), ALIGN), (dict(up=0x5002), ALIGN), (dict(h=0x6004), ALIGN), (dict(ldgu=260), ALIGN), (dict(ldh=257), ALIGN)]


@pytest.mark.parametrize("bad,status", SIZES + [
    (dict(bg=None), ARG), (dict(bu=view(scales=None)), ARG), (dict(gate=None), ARG), (dict(up=None), ARG), (dict(h=None), ARG),
    (dict(bg=view(codes=0x1004)), ALIGN), (dict(bu=view(codes=0x1004)), ALIGN)])
def test_gated_refusals(L, bad, status):
    bad.pop("lddgu", None)
    assert gated(L, **bad) == status


@pytest.mark.parametrize("bad,status", SIZES + [
    (dict(b=None), ARG), (dict(b=view(scale=None)), ARG), (dict(gate=None), ARG), (dict(up=None), ARG), (dict(dgate=None), ARG),
    (dict(dup=None), ARG), (dict(lddgu=128), SHAPE), (dict(lddgu=260), ALIGN), (dict(dgate=0x6002), ALIGN), (dict(dup=0x7008), ALIGN),
    (dict(b=view(scales=0x2008)), ALIGN)])
def test_gated_bwd_refusals(L, bad, status):
    if "lddgu" not in bad and bad.get("F", 0) > 1 << 20:
        bad = dict(bad, lddgu=bad["F"])
    assert gated_bwd(L, **bad) == status


@pytest.mark.parametrize("call", [gated, lambda L: gated(L, gate=None, up=None, ldgu=0), lambda L: gated(L, act=1, M=384, F=128, ldgu=128, ldh=128),
                                  gated_bwd, lambda L: gated_bwd(L, h=None, ldh=0, act=1)])
def test_gated_failures_at_every_site(L, call):
    sites = injected(lambda: call(L))
    assert sites.count("launch") == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_valid_calls_without_gpu_fail_loudly(L):
    for st in (gated(L), gated_bwd(L)):
        assert st == DEV


def test_gated_binding_refuses_before_the_call(monkeypatch):
    b, f = torch.zeros(128, 128, dtype=torch.bfloat16), torch.zeros(128, 128)

    def v(R=128, C=128, codes=None, scales=None, scale=None):
        return qt2.View(torch.zeros(R, C // 2, dtype=torch.uint8) if codes is None else codes,
                        torch.zeros(R * C // 16, dtype=torch.uint8) if scales is None else scales, torch.zeros(1) if scale is None else scale)

    def fwd(a=None, bg=None, bu=None, g=b, u=b, h=b):
        tr.qt2_gemm_nvfp4_gated(a or v(), bg or v(), bu or v(), 128, 128, 128, 1.0, 0, g, u, 128, h, 128)

    def bwd(a=None, w=None, g=b, u=b, dg=b, du=b, h=b):
        tr.qt2_gemm_nvfp4_gated_bwd(a or v(), w or v(), 128, 128, 128, 1.0, 0, g, u, 128, dg, du, 128, h, 128)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # where a CPU tensor's "device" is: types and sizes come first
    cases = [(lambda: fwd(g=f), ARG), (lambda: fwd(h=f), ARG), (lambda: bwd(dg=f), ARG), (lambda: bwd(u=f), ARG),
             (lambda: fwd(a=v(scale=torch.zeros(1).double())), ARG), (lambda: fwd(bg=v(codes=torch.zeros(128, 64, dtype=torch.int8))), ARG),
             (lambda: fwd(bu=v(codes=torch.zeros(64, 128, dtype=torch.uint8).t())), ARG), (lambda: bwd(w=v(scales=torch.zeros(2048, dtype=torch.uint8)[::2])), ARG),
             (lambda: fwd(a=v(256)), SHAPE), (lambda: fwd(bu=v(128, 256)), SHAPE), (lambda: bwd(w=v(scales=torch.zeros(512, dtype=torch.uint8))), SHAPE)]
    for k, (case, status) in enumerate(cases):
        with pytest.raises(qt2.QT2Error) as e:
            case()
        assert e.value.status == status, k
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for case in (fwd, bwd):
        with pytest.raises(qt2.QT2Error) as e:
            case()
        assert e.value.status == DEV


# ------------------------------------------------------------------------------------------ queries and keys
QK = dict(x=0x1000, xd=0, T=5, Hq=3, Hk=1, D=16, ldx=80, hsx=16, wq=0x2000, wk=0x3000, wd=1, eps=1e-6, pos=0x4000, cos=0x5000, sin=0x6000, P=9,
          R=16, pairing=0)


def qk_fwd(L, y=0x7000, ldy=64, hsy=16, **kw):
    return L.qt2_qk_norm_rope_fwd(*dict(QK, **kw).values(), y, ldy, hsy, None)


def qk_bwd(L, dy=0x8000, lddy=64, hsdy=16, dx=0x9000, lddx=80, hsdx=16, dwq=0xa000, dwk=0xb000, ws=0x10000, n=1 << 20, **kw):
    return L.qt2_qk_norm_rope_bwd(dy, lddy, hsdy, *dict(QK, **kw).values(), dx, lddx, hsdx, dwq, dwk, ws, n, None)


QK_BAD = [(dict(x=None), ARG), (dict(xd=2), ARG), (dict(wd=9), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
          (dict(pairing=2), ARG), (dict(cos=None), ARG), (dict(sin=None), ARG), (dict(T=0), SHAPE), (dict(T=1 << 30), SHAPE), (dict(Hq=-1), SHAPE),
          (dict(Hq=0, Hk=0), SHAPE), (dict(Hk=1 << 20), SHAPE), (dict(T=1 << 20, Hq=1 << 13), SHAPE), (dict(D=0), SHAPE), (dict(D=12), SHAPE),
          (dict(D=1032), SHAPE), (dict(R=24), SHAPE), (dict(R=4), SHAPE), (dict(R=-8), SHAPE), (dict(P=0), SHAPE), (dict(P=1 << 30), SHAPE),
          (dict(pos=None, P=4), SHAPE), (dict(ldx=56), SHAPE), (dict(hsx=8), SHAPE), (dict(ldx=-80), SHAPE), (dict(ldx=1 << 32), SHAPE), (dict(hsx=1 << 32, ldx=16), SHAPE),
          (dict(ldx=16, hsx=72), SHAPE), (dict(x=0x1008), ALIGN), (dict(ldx=84), ALIGN), (dict(hsx=17), ALIGN), (dict(wq=0x2008), ALIGN),
          (dict(wk=0x3004), ALIGN), (dict(pos=0x4004), ALIGN), (dict(cos=0x5008), ALIGN), (dict(sin=0x6004), ALIGN)]


@pytest.mark.parametrize("bad,status", QK_BAD + [(dict(y=None), ARG), (dict(ldy=48), SHAPE), (dict(hsy=0), SHAPE), (dict(ldy=68), ALIGN), (dict(y=0x7008), ALIGN)])
def test_qk_fwd_refusals(L, bad, status):
    assert qk_fwd(L, **bad) == status


@pytest.mark.parametrize("bad,status", QK_BAD + [
    (dict(dy=None), ARG), (dict(dx=None, dwq=None, dwk=None), ARG), (dict(lddy=48), SHAPE), (dict(hsdx=8), SHAPE), (dict(lddx=84), ALIGN),
    (dict(dy=0x8004), ALIGN), (dict(dx=0x9008), ALIGN), (dict(dwq=0xa008), ALIGN), (dict(dwk=0xb002), ALIGN), (dict(ws=None), WS), (dict(n=64), WS),
    (dict(ws=0x10080), ALIGN)])
def test_qk_bwd_refusals(L, bad, status):
    assert qk_bwd(L, **bad) == status


@pytest.mark.parametrize("kw", [dict(), dict(R=0, pos=None, cos=None, sin=None, P=0), dict(pos=None), dict(Hq=0), dict(Hk=0), dict(T=1, ldx=0),
                                dict(ldx=16, hsx=80), dict(wq=None, wk=None, xd=1, wd=0), dict(D=512, R=8, ldx=2048, hsx=512)])
def test_qk_calls_that_are_right(L, kw):
    """Either layout, nothing turned, heads of one kind; a call may give no leading dimension where there is one row."""
    wide = dict(ldy=4096, hsy=1024) if kw.get("D") else {}
    assert injected(lambda: qk_fwd(L, **wide, **kw)).count("launch") == 1
    wide = dict(lddy=4096, hsdy=1024, lddx=4096, hsdx=1024) if kw.get("D") else {}
    assert injected(lambda: qk_bwd(L, **wide, **kw)).count("launch") == 2
    assert injected(lambda: qk_bwd(L, dwq=None, dwk=None, **wide, **kw)).count("launch") == 1


def test_qk_workspace(L):
    n = ctypes.c_size_t(0)
    assert L.qt2_qk_norm_rope_bwd_workspace_size(4, 2, 1, 64, None) == ARG
    for dims in ((0, 1, 1, 64), (4, 0, 0, 64), (4, 1, 1, 60), (4, 1, 1, 2048), (4, -1, 3, 64)):
        assert L.qt2_qk_norm_rope_bwd_workspace_size(*dims, ctypes.byref(n)) == SHAPE
    assert tr.qt2_qk_norm_rope_bwd_workspace_size(1 << 20, 32, 8, 128) < 1 << 20


def test_qk_binding_refuses_before_the_call(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, w, t, pos, ws = torch.zeros(4, 64), torch.zeros(16), torch.zeros(9, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(1 << 16, dtype=torch.uint8)
    vectors = dict(wq=w, wk=w, pos=pos, cos=t, sin=t)

    def fwd(x=x, y=x, **kw):
        v = dict(vectors, **kw)
        tr.qt2_qk_norm_rope_fwd(x, 4, 3, 1, 16, 64, 16, v["wq"], v["wk"], 1e-6, v["pos"], v["cos"], v["sin"], 9, 16, 0, y, 64, 16)

    def bwd(x=x, dy=x, dx=x, dwq=w, dwk=w, ws=ws, **kw):
        v = dict(vectors, **kw)
        tr.qt2_qk_norm_rope_bwd(dy, 64, 16, x, 4, 3, 1, 16, 64, 16, v["wq"], v["wk"], 1e-6, v["pos"], v["cos"], v["sin"], 9, 16, 0, dx, 64, 16, dwq,
                                dwk, ws, 1 << 16)
    half = torch.zeros(4, 64, dtype=torch.float16)
    bad = [lambda f: f(x=half), lambda f: f(x=x.bfloat16()), lambda f: f(wq=w.bfloat16()), lambda f: f(pos=pos.int()), lambda f: f(cos=t.double()),
           lambda f: f(pos=torch.zeros(8, dtype=torch.int64)[::2]), lambda f: f(sin=torch.zeros(8, 9).t()), lambda f: f(wk=w[:1].expand(16))]
    extra = [lambda f: f(dx=half), lambda f: f(dwq=w.bfloat16()), lambda f: f(dwk=torch.zeros(32)[::2]), lambda f: f(ws=ws[::2])]
    for f, cases in ((fwd, bad + [lambda f: f(y=half)]), (bwd, bad + extra)):
        for k, case in enumerate(cases):
            with pytest.raises(qt2.QT2Error) as e:
                case(f)
            assert e.value.status == ARG, k
        with pytest.raises(qt2.QT2Error) as e:
            f()
        assert e.value.status == DEV


# ------------------------------------------------------------------------------------------ AdamW
ROW = dict(param=0x1000, master=None, grad=0x2000, m=0x3000, v=0x4000, m_scale=None, v_scale=None, numel=5, param_dtype=1, grad_dtype=1, state=0,
           weight_decay=0.0)
EIGHT = dict(m_scale=0x5000, v_scale=0x6000, state=1)


def rows(*changes):
    a = (tr.AdamWTensorC * max(1, len(changes)))()
    for c, change in zip(a, changes):
        for k, v in dict(ROW, **change).items():
            setattr(c, k, v)
    return a


def adamw(L, *changes, count=None, lr=0x7000, step=0x8000, b1=0.9, b2=0.99, eps=1e-8, norm=0x9000, max_norm=1.0):
    a = rows(*(changes or ({},)))
    return L.qt2_adamw(ctypes.addressof(a), len(changes or (1,)) if count is None else count, lr, step, b1, b2, eps, norm, max_norm, 7, None)


@pytest.mark.parametrize("bad,status", [
    (dict(param=None), ARG), (dict(grad=None), ARG), (dict(m=None), ARG), (dict(v=None), ARG), (dict(param_dtype=2), ARG), (dict(grad_dtype=-1), ARG),
    (dict(state=2), ARG), (dict(state=1), ARG), (dict(EIGHT, v_scale=None), ARG), (dict(weight_decay=float("nan")), ARG), (dict(weight_decay=float("inf")), ARG),
    (dict(master=0x5000), ARG), (dict(numel=-1), SHAPE), (dict(numel=1 << 40), SHAPE), (dict(param=0x1002), ALIGN), (dict(grad=0x2002), ALIGN),
    (dict(m=0x3002), ALIGN), (dict(v=0x4001), ALIGN), (dict(param_dtype=0, param=0x1001), ALIGN), (dict(param_dtype=0, master=0x5002), ALIGN),
    (dict(EIGHT, m_scale=0x5002), ALIGN), (dict(EIGHT, v_scale=0x6001), ALIGN)])
def test_adamw_tensor_refusals(L, bad, status):
    assert adamw(L, {}, bad) == status
    if status != SHAPE and bad.get("state", 0) != 2 and "dtype" not in str(bad) and "decay" not in str(bad) and "master" not in bad:
        with tr.fault_hook(lambda site: qt2.FAULT_SKIP):   # of an empty tensor nothing is read
            assert adamw(L, {}, dict(bad, numel=0)) == OK


@pytest.mark.parametrize("bad,status", [
    (dict(lr=None), ARG), (dict(step=None), ARG), (dict(b1=1.0), ARG), (dict(b1=-0.1), ARG), (dict(b2=1.0), ARG), (dict(b2=float("nan")), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(max_norm=-1.0), ARG), (dict(max_norm=float("nan")), ARG),
    (dict(count=0), SHAPE), (dict(count=-3), SHAPE), (dict(lr=0x7002), ALIGN), (dict(step=0x8004), ALIGN), (dict(norm=0x9001), ALIGN)])
def test_adamw_refusals(L, bad, status):
    assert adamw(L, **bad) == status


def test_adamw_calls_that_are_right(L):
    assert L.qt2_adamw(None, 1, 0x7000, 0x8000, 0.9, 0.99, 1e-8, None, 1.0, 7, None) == ARG
    for changes, kw, launches in (([{}], {}, 1), ([dict(EIGHT, m=0x3001, v=0x4003)], {}, 1), ([{}], dict(norm=None, max_norm=-1.0), 1),
                                  ([dict(numel=0, param=None, grad=None, m=None, v=None)], {}, 0), ([dict(param_dtype=0, master=0xa000)] * 33, {}, 1),
                                  ([{}, dict(numel=0)] * 400, {}, 2), ([dict(numel=(1 << 40) - 1)] * 3, {}, 3), ([{}], dict(b1=0.0, b2=0.0), 1)):
        if launches:
            assert injected(lambda: adamw(L, *changes, **kw)).count("launch") == launches
        else:
            with tr.fault_hook(lambda site: qt2.FAULT_SKIP) as h:
                assert adamw(L, *changes, **kw) == OK
            assert "launch" not in h.sites


def test_adamw_list_refuses(monkeypatch):
    f, g, m, v = (torch.zeros(300) for _ in range(4))
    b, half = torch.zeros(300, dtype=torch.bfloat16), torch.zeros(300, dtype=torch.float16)
    e, e2, s, s2 = torch.zeros(300, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(300, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(2), torch.zeros(2)
    long = torch.zeros(1200)
    cases = [
        lambda: tr.AdamWList([half], [g], [m], [v]), lambda: tr.AdamWList([f], [half], [m], [v]), lambda: tr.AdamWList([f], [g], [b], [v]),
        lambda: tr.AdamWList([f], [g], [m], [e]), lambda: tr.AdamWList([f], [g], [e], [e2]), lambda: tr.AdamWList([f], [g], [e], [e2], None, [s], None),
        lambda: tr.AdamWList([f], [g], [m], [v], None, [s], [s2]), lambda: tr.AdamWList([f], [g], [m], [v], [long[:300]]),
        lambda: tr.AdamWList([b], [g], [m], [v], [b]), lambda: tr.AdamWList([f], [g[:299]], [m], [v]), lambda: tr.AdamWList([f], [g], [e], [e2], None, [s[:1]], [s2]),
        lambda: tr.AdamWList([f], [g], [m], [v, v]), lambda: tr.AdamWList([f], [g], [m], [v], weight_decay=[0.1, 0.1]),
        lambda: tr.AdamWList([torch.zeros(20, 15).t()], [g], [m], [v]), lambda: tr.AdamWList([f], [g[:1].expand(300)], [m], [v]),
        # what the step writes, and another array
        lambda: tr.AdamWList([f], [f], [m], [v]), lambda: tr.AdamWList([f], [g], [m], [m]), lambda: tr.AdamWList([f], [g], [f], [v]),
        lambda: tr.AdamWList([long[:300]], [long[299:599]], [m], [v]), lambda: tr.AdamWList([f, long[:300]], [g, g], [m, long[200:500]], [v, torch.zeros(300)]),
        lambda: tr.AdamWList([f], [g], [e], [e2], None, [s], [s])]
    for k, case in enumerate(cases):
        with pytest.raises(qt2.QT2Error) as err:
            case()
        assert err.value.status == ARG, k
    tr.AdamWList([f, torch.zeros(300)], [g, g], [m, torch.zeros(300)], [v, torch.zeros(300)], weight_decay=[0.0, 0.1])   # a gradient of two
    ok = tr.AdamWList([b, f], [g, g], [e, m], [e2, v], [long[:300], None], [s, None], [s2, None], 0.1)
    tr.AdamWList([long[:300]], [long[300:600]], [long[600:900]], [long[900:]])
    assert tr.AdamWList([], [], [], []).count == 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    one, step = torch.zeros(1), torch.ones(1, dtype=torch.int64)
    for args, status in (((one, step, None), DEV), ((one.double(), step, None), ARG), ((one, step.int(), None), ARG), ((one, step, one.bfloat16()), ARG),
                         ((f, step, None), ARG), ((one, step, s), ARG)):
        with pytest.raises(qt2.QT2Error) as err:
            tr.qt2_adamw(ok, args[0], args[1], 0.9, 0.99, 1e-8, args[2], 1.0, 7)
        assert err.value.status == status
