"""AdamW with states in 8 bits on blocks whose elements lie many binades apart."""
import math

import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.codes_ref import encode, words

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
B1, B2, EPS, SEED = 0.9, 0.95, 1e-8, (9 << 32) + 4
N, BLOCKS = 256 * 64, 64


class State:
    """One fp32 tensor of zeros with fresh states, under a rate of one: a step's update is what p moves by."""

    def __init__(self, n, eight):
        zeros = lambda dt=torch.float32, k=n: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
        self.p, self.g, self.eight = zeros(), zeros(), eight
        self.m, self.v = (zeros(torch.uint8).view(E4) if eight else zeros() for _ in range(2))
        self.ms, self.vs = (zeros(k=(n + 255) // 256) if eight else None for _ in range(2))
        self.list = tr.AdamWList([self.p], [self.g], [self.m], [self.v], None, *([[s] if eight else None for s in (self.ms, self.vs)]))
        self.lr, self.step = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(self, g):
        """The step's updates, in learning rates."""
        self.g.copy_(g)
        self.p.zero_()
        self.step += 1
        tr.qt2_adamw(self.list, self.lr, self.step, B1, B2, EPS, None, 1.0, SEED)
        return self.p.double()


def gradients(kind):
    gen = torch.Generator(device="cuda").manual_seed(11)
    rn = lambda: torch.randn(N, generator=gen, device="cuda")  # noqa: E731
    wide, spread = (3 * rn()).exp() * 1e-6, 10 ** (6 * torch.rand(N, generator=gen, device="cuda") - 7)

    def at(t):
        if kind == "lognormal":
            return rn() * wide
        if kind == "decades":
            return rn() * spread
        if kind == "rare":
            return rn() * spread * (torch.rand(N, generator=gen, device="cuda") < 0.05)
        top, stop = {"massive 1e2": (1e2, 0), "massive 1e5": (1e5, 0), "massive 1e6": (1e6, 0), "stopping": (1e5, 50)}[kind]
        g = rn() * (1e-5 if not stop or t <= stop else 0.0)
        g.view(BLOCKS, 256)[:, 7] = rn()[:BLOCKS] * 1e-5 * top
        return g
    return at


@pytest.mark.parametrize("kind", ["massive 1e2", "massive 1e5", "massive 1e6", "stopping", "lognormal", "decades", "rare"])
def test_no_step_runs_away(kind):
    """300 steps beside fp32 states: no update above 8 learning rates, and their root mean square in line.

    With exact states |m| / sqrt(v) is (1 - b1) / sqrt((1 - b2) (1 - b1^2 / b2)) = 1.17 at most (Cauchy-Schwarz).  An m
    below its smallest code is stored as that code at most, a root as its smallest at least: the largest |m| over
    the largest root of the block, 1.17 again.  Between the smallest codes an m may be rounded up to twice and a
    root down to half of itself, 4.7; of that the next step keeps b1 / sqrt(b2) = 0.92, and its own gradient adds
    (1 - b1) / sqrt(1 - b2) = 0.45: 4.8.  More takes such roundings several times in a row, each as unlikely as it
    is large (the mean stays).  The same sums, step by step on the CPU in fp32, gave 2.3 at most, and root mean
    squares of 1.18 of fp32's; a root of 0 gave 34 to 3500 (not on the first rows, whose range the codes span)."""
    grads = gradients(kind)
    a, b = State(N, True), State(N, False)
    worst, square = torch.zeros(2, dtype=torch.float64, device="cuda"), torch.zeros(2, dtype=torch.float64, device="cuda")
    for t in range(1, 301):
        g = grads(t)
        u = torch.stack([a.run(g), b.run(g)])
        worst, square = torch.maximum(worst, u.abs().amax(1)), square + u.square().mean(1)
    assert worst[1] <= 1.2
    assert worst[0] <= 8, worst.tolist()
    assert square[0].sqrt() <= 1.5 * square[1].sqrt(), square.tolist()
    # and where the codes span the block, the runs agree (elements below the smallest codes move less)
    if kind == "massive 1e2":
        assert square[0].sqrt() >= 0.9 * square[1].sqrt()
    assert tr.qt2_train_device_status() == 0


def test_codes_of_wide_blocks_are_the_stated_ones():
    """Codes and scales bit for bit through steps on blocks of every spread, zeros among them."""
    n = N - 100
    s = State(n, True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    size = 10 ** (9 * torch.rand(n, generator=gen, device="cuda") - 9)
    size[::11] = 0
    f32 = lambda x: torch.tensor(x, dtype=torch.float64).float().cuda()  # noqa: E731
    each = lambda c: c.repeat_interleave(256)[:n]  # noqa: E731
    for step in range(1, 5):
        g = torch.randn(n, generator=gen, device="cuda") * size
        m, r = s.m.float() * each(s.ms), s.v.float() * each(s.vs)
        m = m * f32(B1) + g * f32(1 - B1)
        root = (r * r * f32(B2) + g * g * f32(1 - B2)).sqrt()
        s.run(g)
        w = words(0, n, 0, step, SEED)
        for x, draw, codes, scales in ((m, w & 0xFFFF, s.m, s.ms), (root, w >> 16, s.v, s.vs)):
            want, scale = encode(x, draw, x is root)
            assert torch.equal(codes.double(), want) and torch.equal(scales, scale)
        assert torch.equal(s.v.float() == 0, root == 0)
        # there are roots below the smallest code
        assert ((root > 0) & (root / each(s.vs) < 2.0 ** -9)).any()


def test_a_root_below_its_block_is_kept_at_both_ends():
    """The smallest root that fp32 has beside the largest: its code is the smallest; a block of zeros stays zeros."""
    s = State(512, True)
    g = torch.zeros(512, device="cuda")
    g[3], g[5] = 1e18, 2e-22   # squares of 1e36 and 4e-44
    for _ in range(3):
        s.run(g)
        assert s.v[5].float() == 2.0 ** -9 and s.v[3].float() == 448
        assert (s.v.float() != 0).sum() == 2 and s.vs[1] == 0 and s.ms[1] == 0
        assert torch.isfinite(s.p).all() and s.p.abs().max() <= 1.0 + 2.0 ** -20
