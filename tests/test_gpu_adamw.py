"""AdamW over many tensors, states in fp32 and in 8 bits, on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.train_ref import check

pytestmark = pytest.mark.gpu
BF, FP, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B1, B2, EPS, LR, SEED = 0.9, 0.95, 1e-8, 1e-3, (5 << 32) + 77


def blocks(n):
    return (n + 255) // 256


class Tensors:
    """A list of tensors of the sizes: parameters, gradients and states in buffers of their own, `gap` elements (of
    value 7) before and between them."""

    def __init__(self, sizes, param=FP, grad=FP, master=False, eight=False, gap=1, seed=0, fresh=False):
        self.sizes, self.eight, self.master = sizes, eight, master
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.bufs = {}

        def place(name, dtype, values, gap=gap):
            total = sum(v.numel() for v in values) + gap * (len(values) + 1)
            buf = torch.full((total,), 7.0, device="cuda").to(dtype)
            out, at = [], gap
            for v in values:
                out.append(buf[at:at + v.numel()])
                out[-1].copy_(v.to(dtype))
                at += v.numel() + gap
            self.bufs[name] = (buf, out)
            return out
        rn = lambda n, s: torch.randn(n, generator=g, device="cuda") * s  # noqa: E731
        p = [rn(n, 0.1) for n in sizes]
        self.p = place("p", param, p)
        self.masters = place("master", FP, p) if master else None
        self.g = place("g", grad, [rn(n, 1e-2) for n in sizes])
        m = [rn(n, 0.0 if fresh else 5e-3) for n in sizes]
        root = [(rn(n, 1e-2).abs() + 1e-3) * (0.0 if fresh else 1.0) for n in sizes]
        if eight:
            tops = [[torch.stack([c.abs().max() for c in x.split(256)]) / 448 if x.numel() else x.new_zeros(0) for x in xs] for xs in (m, root)]
            codes = [[x / t.clamp(min=1e-30).repeat_interleave(256)[:x.numel()] for x, t in zip(xs, ts)] for xs, ts in zip((m, root), tops)]
            self.m, self.v = place("m", E4, codes[0]), place("v", E4, codes[1])
            self.ms, self.vs = place("ms", FP, tops[0], 1), place("vs", FP, tops[1], 1)
        else:
            self.m, self.v, self.ms, self.vs = place("m", FP, m), place("v", FP, [r * r for r in root]), None, None
        self.decay = [0.1 * (i % 3) for i in range(len(sizes))]
        self.list = tr.AdamWList(self.p, self.g, self.m, self.v, self.masters, self.ms, self.vs, self.decay)
        self.lr, self.step = torch.full((1,), LR, device="cuda"), torch.full((1,), 3, dtype=torch.int64, device="cuda")

    def states(self, i):
        """What tensor i's states stand for, in 64 bits."""
        m, v = self.m[i].double(), self.v[i].double()
        if not self.eight:
            return m, v
        each = lambda s: s.double().repeat_interleave(256)[:m.numel()]  # noqa: E731
        # fp32 products of code and scale, as the step takes them
        return (m * each(self.ms[i])).float().double(), (v * each(self.vs[i])).float().double().square().float().double()

    def run(self, norm=None, max_norm=1.0, seed=SEED):
        tr.qt2_adamw(self.list, self.lr, self.step, B1, B2, EPS, norm, max_norm, seed)

    def all(self):
        return [b for b, _ in self.bufs.values()]

    def guards(self):
        """Elements between the tensors, as they were."""
        for name, (buf, views) in self.bufs.items():
            rest = buf.float().clone()
            for v in views:
                a = v.storage_offset()
                rest[a:a + v.numel()] = 7.0
            assert (rest == 7.0).all(), name


def want(t, clip=1.0):
    out = []
    for i in range(len(t.sizes)):
        p = t.masters[i] if t.master else t.p[i]
        m, v = t.states(i)
        lr = t.lr.double().item()
        out.append(ref.adamw(p, t.g[i], m, v, lr, t.step.item(), B1, B2, EPS, np.float32(t.decay[i]).item(), clip))
    return out


def compare(t, expected):
    for i, ((p, m, v), (ep, em, ev)) in enumerate(expected):
        check(t.p[i], p, ep, ("p", i))
        if t.master:
            check(t.masters[i], p, ep, ("master", i))
            assert torch.equal(t.p[i], t.masters[i].to(t.p[i].dtype))
        if not t.eight:
            check(t.m[i], m, em, ("m", i))
            check(t.v[i], v, ev, ("v", i))
            continue
        for name, x, e, codes, scales in (("m", m, em, t.m[i], t.ms[i]), ("v", v.sqrt(), ev, t.v[i], t.vs[i])):
            if not x.numel():
                continue
            e = e if name == "m" else torch.minimum(e / x.clamp(min=1e-300), e.sqrt()) + ref.U * x
            top = torch.stack([c.abs().max() for c in x.split(256)])
            most = torch.stack([c.max() for c in e.split(256)])
            check(scales, top / 448, most / 448, (name, "scale", i))
            s = scales.double().repeat_interleave(256)[:x.numel()]
            y = torch.where(s > 0, x / s, 0.0).clamp(-448, 448)
            slack = torch.where(s > 0, e / s, 0.0) + 8 * ref.U * y.abs() + 2.0 ** -29   # and below 2^-6 what adding it rounds
            below, above = ref.e4m3_neighbours((y.abs() - slack).clamp(min=0))[0], ref.e4m3_neighbours((y.abs() + slack).clamp(max=448))[1]
            c = codes.double()
            assert ((c.abs() >= below) & (c.abs() <= above)).all(), (name, i)
            big = y.abs() > slack
            assert (torch.sign(c) * torch.sign(y))[big & (c != 0)].ge(0).all()


LISTS = [[1], [3, 0, 5], [255, 256, 257], [2047, 2048, 2049], [1, 2, 3, 4, 5, 6, 7, 8] * 9, [1000] * 400 + [3], [100003, 65536, 7], [1 << 20]]
KINDS = [(FP, FP, False), (BF, BF, True), (BF, FP, True), (BF, BF, False), (FP, BF, False)]


@pytest.mark.parametrize("gap", [0, 1, 3, 8])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("k", range(len(LISTS)))
def test_matches_the_formulas(k, eight, gap):
    """Every alignment of the arrays, alike (fp32 states of equal gaps) and not (the scales' and codes')."""
    param, grad, master = KINDS[(k + gap) % len(KINDS)]
    t = Tensors(LISTS[k], param, grad, master, eight, gap, seed=k)
    expected = want(t)
    t.run()
    compare(t, expected)
    t.guards()
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_types_and_several_steps(kind, eight):
    t = Tensors([513, 4096, 77], *kind, eight, gap=8, seed=3, fresh=True)
    t.step.fill_(0)
    for _ in range(4):
        t.step += 1
        expected = want(t)
        t.run()
        compare(t, expected)


def test_mixed_list():
    """Tensors of every kind in one list, some arrays aligned and others not."""
    parts = [Tensors([300, 5], *kind, eight, gap, seed=i) for i, (kind, eight, gap) in enumerate(
        [(k, e, g) for k in KINDS for e in (False, True) for g in (1, 8)])]
    none = lambda xs, n: [None] * n if xs is None else xs  # noqa: E731
    cat = lambda name: [x for t in parts for x in none(getattr(t, name), 2)]  # noqa: E731
    both = tr.AdamWList(cat("p"), cat("g"), cat("m"), cat("v"), cat("masters"), cat("ms"), cat("vs"), [d for t in parts for d in t.decay])
    expected = [want(t) for t in parts]
    tr.qt2_adamw(both, parts[0].lr, parts[0].step, B1, B2, EPS, None, 1.0, SEED)
    for t, e in zip(parts, expected):
        compare(t, e)
        t.guards()


def test_misaligned_arrays_give_the_same_bits():
    """One array at a time an element off the others."""
    sizes = [1000, 2500]
    for eight in (False, True):
        a = Tensors(sizes, BF, BF, True, eight, gap=8, seed=5)
        start = {n: [v.clone() for v in vs] for n, (_, vs) in a.bufs.items()}
        a.run()
        for off in ("p", "g", "m", "v", "master"):
            moved = {}
            for name, vs in start.items():
                k = 1 if name == off else 0
                moved[name] = [torch.zeros(v.numel() + 1, device="cuda").to(v.dtype)[k:k + v.numel()].copy_(v) for v in vs]
            lst = tr.AdamWList(moved["p"], moved["g"], moved["m"], moved["v"], moved["master"], moved.get("ms"), moved.get("vs"), a.decay)
            tr.qt2_adamw(lst, a.lr, a.step, B1, B2, EPS, None, 1.0, SEED)
            for name, (_, vs) in a.bufs.items():
                assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(moved[name], vs)), (eight, off, name)


def words(n, tensor, step, seed):
    group = np.arange((n + 3) // 4, dtype=np.uint64)
    c = np.stack([group & np.uint64(0xFFFFFFFF), group >> np.uint64(32), np.full_like(group, tensor), np.full_like(group, step)], 1)
    w = ref.philox(c, seed)
    for k in (0, len(group) // 2, len(group) - 1):   # the library's own generator is pinned by published vectors
        assert [int(x) for x in w[k]] == [int(x) for x in O.philox4x32_10([int(x) for x in c[k]], [seed & 0xFFFFFFFF, seed >> 32])]
    return torch.from_numpy(w.reshape(-1)[:n].astype(np.int64)).cuda()


def test_codes_are_the_stated_ones():
    """Codes and scales bit for bit, from fp32 operations one by one and the stated draws."""
    t = Tensors([1, 700, 256, 5000], BF, BF, True, True, gap=8, seed=9)
    t.step.fill_(12345)
    norm = torch.full((1,), 3.0, device="cuda")
    f32 = lambda x: torch.tensor(x, dtype=torch.float64).float().cuda()  # noqa: E731
    states = []
    for i, n in enumerate(t.sizes):
        each = lambda s: s.repeat_interleave(256)[:n]  # noqa: E731
        m, r = t.m[i].float() * each(t.ms[i]), t.v[i].float() * each(t.vs[i])
        h = t.g[i].float() * (torch.ones(1, device="cuda") / (norm + f32(1e-6)))
        m = m * f32(B1) + h * f32(1 - B1)
        v = r * r * f32(B2) + h * h * f32(1 - B2)
        states.append((m, v.sqrt()))
    t.run(norm, 1.0)
    for i, n in enumerate(t.sizes):
        w = words(n, i, 12345, SEED)
        for x, codes, scales, draw in ((states[i][0], t.m[i], t.ms[i], w & 0xFFFF), (states[i][1], t.v[i], t.vs[i], w >> 16)):
            top = torch.stack([c.abs().max() for c in x.split(256)])
            most = torch.full_like(top, 448)
            assert torch.equal(scales, top / most)
            a = x.abs() * (most / top).repeat_interleave(256)[:n]
            # the fraction of the spacing that a lies above the code below it, against the draw
            low, high = ref.e4m3_neighbours(a.double())
            exact = (a.double() - low) / (high - low).clamp(min=2.0 ** -9)
            up = torch.where(a >= 2.0 ** -6, (exact * 2 ** 20 + draw * 16 >= 2 ** 20), False)
            small = ((a + 2.0 ** -6).double() - 2.0 ** -6) * 512
            up = torch.where(a < 2.0 ** -6, (small - small.floor()) * 2 ** 20 + draw * 16 >= 2 ** 20, up)
            low = torch.where(a < 2.0 ** -6, small.floor() / 512, low)
            high = torch.where(a < 2.0 ** -6, low + 2.0 ** -9, high)
            value = torch.where(up, high, low).clamp(max=448) * torch.sign(x).double()
            assert torch.equal(codes.double(), value)


def test_rounding_keeps_the_mean():
    """Codes of one state over many seeds: their mean is the state's value, in all binades.

    A code goes up X of n times, X binomial with mean n f.  Near a code f is small and X far from normal (6 standard
    errors at n f = 0.3 are 3.3, and X >= 4 has a chance of 3e-4), so the bound is Bernstein's:
    P(|X - n f| > t) <= 2 exp(-t^2 / (2 (n f (1 - f) + t / 3))), which is 2 exp(-L) at
    t = L / 3 + sqrt(L^2 / 9 + 2 L n f (1 - f)); with L = 30 the 2048 of them exceed it with a chance of 4e-10."""
    n, seeds = 1024, 1500
    t = Tensors([n], FP, FP, False, True, gap=8, seed=2)
    g = t.g[0]
    g.copy_(torch.logspace(-7, 0, n, device="cuda") * torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0))
    start = [b.clone() for b in t.all()]
    m, v = t.states(0)
    (_, m, v), _ = ref.adamw(t.p[0], g, m, v, LR, 3, B1, B2, EPS, 0.0, 1.0)
    total = [torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2)]
    for s in range(seeds):
        for b, x in zip(t.all(), start):
            b.copy_(x)
        t.run(seed=s)
        total[0] += t.m[0].double() * t.ms[0].double().repeat_interleave(256)
        total[1] += t.v[0].double() * t.vs[0].double().repeat_interleave(256)
    for x, s, scale in ((m, total[0], t.ms[0]), (v.sqrt(), total[1], t.vs[0])):
        scale = scale.double().repeat_interleave(256)
        low, high = ref.e4m3_neighbours((x / scale).clamp(-448, 448))
        f = ((x / scale).abs() - low) / (high - low).clamp(min=2.0 ** -10)
        L, var = 30.0, seeds * (f * (1 - f)).clamp(min=0)
        counts = L / 3 + (L * L / 9 + 2 * L * var).sqrt()
        # draws have 16 bits: 2^-16 of the spacing is lost at most
        slack = (high - low) * scale * 2.0 ** -15 + 64 * ref.U * x.abs()
        assert ((s / seeds - x).abs() <= counts / seeds * (high - low) * scale + slack).all()


@pytest.mark.parametrize("eight", [False, True])
def test_clipping_is_taken_along(eight):
    """The norm of the list's gradients, and what the step does with it: as clipped gradients do alone."""
    a, b = (Tensors([3000, 41, 256], FP, FP, False, eight, gap=8, seed=4) for _ in range(2))
    gl = tr.GradList(a.g)
    norm, ws = torch.empty(1, device="cuda"), qt2.alloc_workspace(tr.qt2_grad_norm_workspace_size(gl))
    tr.qt2_grad_norm(gl, norm, ws, ws.numel())
    max_norm = norm.item() / 3
    tr.qt2_grad_clip(tr.GradList(b.g), norm, max_norm)
    a.run(norm, max_norm)
    b.run()
    for name in a.bufs:
        if name != "g":
            assert torch.equal(a.bufs[name][0].view(torch.uint8), b.bufs[name][0].view(torch.uint8)), name
    c, d = (Tensors([3000, 41, 256], FP, FP, False, eight, gap=8, seed=4) for _ in range(2))
    c.run(norm, 1e9)   # nothing to clip
    d.run()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(c.all(), d.all()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nothing_changes_where_the_norm_is_not_finite(bad):
    for eight in (False, True):
        t = Tensors([900, 3], BF, BF, True, eight, gap=3)
        before = [b.clone() for b in t.all()]
        t.run(torch.full((1,), bad, device="cuda"))
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, t.all()))
    assert tr.qt2_train_device_status() == 0


@pytest.mark.parametrize("step", [0, -5])
def test_steps_below_one_are_reported(step):
    t = Tensors([900, 3])
    before = [b.clone() for b in t.all()]
    t.step.fill_(step)
    t.run()
    assert tr.qt2_train_device_status() == qt2.QT2_ERR_INVALID_ARG
    assert all(torch.equal(x, y) for x, y in zip(before, t.all()))


def test_far_steps():
    """Corrections of one, and a step whose number takes more than 32 bits."""
    for step in (10 ** 6, (1 << 33) + 3):
        for eight in (False, True):
            t = Tensors([600], eight=eight, gap=8)
            t.step.fill_(step)
            expected = want(t)
            t.run()
            compare(t, expected)


def test_nonfinite_gradients_stay_in_their_block():
    t, u = (Tensors([1024], FP, FP, False, True, gap=8, seed=6) for _ in range(2))
    t.g[0][300], t.g[0][600] = float("nan"), float("inf")
    t.run()
    u.run()
    assert torch.isnan(t.ms[0][1:3]).all() and torch.isnan(t.vs[0][1:3]).all()
    for x, y in ((t.p, u.p), (t.m, u.m), (t.v, u.v)):
        x, y = x[0].float(), y[0].float()
        assert torch.equal(x[:256], y[:256]) and torch.equal(x[768:], y[768:])
    assert torch.equal(t.ms[0][[0, 3]], u.ms[0][[0, 3]])
    keep = torch.ones(1024, dtype=torch.bool, device="cuda")
    keep[300] = keep[600] = False
    assert torch.equal(t.p[0][keep], u.p[0][keep])   # the step itself is each element's own


@pytest.mark.parametrize("eight", [False, True])
def test_zero_blocks_and_tiny_values(eight):
    t = Tensors([768], FP, FP, False, eight, gap=8, fresh=True)
    t.g[0][:256] = 0
    t.g[0][256:512] *= 1e-34
    before = t.p[0].clone()
    expected = want(t)
    t.run()
    if eight:
        assert t.ms[0][0] == 0 and t.vs[0][0] == 0 and t.ms[0][1] == 0 and (t.m[0].float()[:512] == 0).all() and t.ms[0][2] > 0
    assert torch.equal(t.p[0][:256], before[:256])   # no decay in the list's first tensor
    assert torch.isfinite(t.p[0]).all()
    check(t.p[0][512:], expected[0][0][0][512:], expected[0][1][0][512:])


@pytest.mark.parametrize("eight", [False, True])
def test_in_a_graph_with_new_steps_and_rates(eight):
    a, b = (Tensors([5000, 33, 256 * 9], BF, BF, True, eight, gap=8, seed=8) for _ in range(2))
    a.run(), b.run()   # (the first calls of a process may load code)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    norm = torch.full((1,), 2.0, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        a.run(norm)
    for k in range(3):
        for t in (a, b):
            t.step.fill_(10 + k), t.lr.fill_(1e-3 / (k + 1))
        norm.fill_(2.0 + k)
        graph.replay()
        b.run(norm)
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a.all(), b.all()))


def test_past_2_to_31_elements():
    """A tensor whose elements' numbers take more than 31 bits: its ends, and the draws there."""
    n = (1 << 31) + 4096 + 5
    g = torch.zeros(n, dtype=BF, device="cuda")
    p = torch.zeros(n, dtype=BF, device="cuda")
    m, v = torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4), torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4)
    ms, vs = torch.zeros(blocks(n), device="cuda"), torch.zeros(blocks(n), device="cuda")
    tail = torch.randn(5000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    g[:5000], g[-5000:] = tail.to(BF), tail.to(BF)
    lst = tr.AdamWList([p], [g], [m], [v], None, [ms], [vs])
    lr, step = torch.full((1,), LR, device="cuda"), torch.ones(1, dtype=torch.int64, device="cuda")
    tr.qt2_adamw(lst, lr, step, B1, B2, EPS, None, 1.0, SEED)
    # m / (1 - b1) = g and sqrt(v / (1 - b2)) = |g| after the first step, so p = -lr g / (|g| + eps): lr, and less
    # where g is as small as eps
    first = -LR * g[-5000:].double() / (g[-5000:].double().abs() + EPS)
    for part in (p[:5000], p[-5000:]):
        torch.testing.assert_close(part.double(), first, rtol=2.0 ** -8 + 2.0 ** -18, atol=0)
    assert (p[5000:6000] == 0).all() and (p[1 << 30:(1 << 30) + 1000] == 0).all()
    # the last block's codes: 5 elements, draws of group (2^31 + 4096) / 4 on
    last = n // 256 * 256
    x = (g[last:].float() * torch.tensor(1 - B1, dtype=torch.float64).float().cuda())
    scale = ms[-1].item()
    assert scale == (x.abs().max() / torch.full((1,), 448.0, device="cuda")).item()
    low, high = ref.e4m3_neighbours((x.double() / scale).clamp(-448, 448))
    c = m[last:].double().abs()
    assert ((c == low) | (c == high)).all() and (ms[blocks(5000):blocks(5000) + 100] == 0).all()
