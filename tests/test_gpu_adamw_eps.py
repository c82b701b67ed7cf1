"""AdamW with the smallest eps: subnormal ones are divided by too."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests import block_ref as ref
from tests.train_ref import check

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
B1, B2, LR = 0.9, 0.95, 2.0 ** -10


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("eps", [2.0 ** -149, 2.0 ** -133, 2.0 ** -126 - 2.0 ** -149, 2.0 ** -126, 2.0 ** -100])
def test_matches_the_formulas(eps, eight):
    """Elements without a gradient or a state stay; those with a gradient, or with an m alone, move as the formula says."""
    n = 768
    gen = torch.Generator(device="cuda").manual_seed(2)
    p, g = torch.randn(n, generator=gen, device="cuda"), torch.randn(n, generator=gen, device="cuda")
    g[256:] = 0
    g[::7] = 0
    m = torch.zeros(n, device="cuda")
    if not eight:
        m[512:] = eps * 100 * torch.randn(256, generator=gen, device="cuda")   # (steps of up to 3000 rates)
        states = [m, torch.zeros(n, device="cuda"), None, None]
    else:
        states = [torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4) for _ in range(2)] + [torch.zeros(3, device="cuda") for _ in range(2)]
    (want, _, _), (bound, _, _) = ref.adamw(p, g, m, torch.zeros_like(m), LR, 3, B1, B2, eps, 0.0, 1.0)
    still = (g == 0) & (m == 0)
    before = p.clone()
    scales = [None if s is None else [s] for s in states[2:]]
    lst = tr.AdamWList([p], [g], [states[0]], [states[1]], None, *scales)
    tr.qt2_adamw(lst, torch.full((1,), LR, device="cuda"), torch.full((1,), 3, dtype=torch.int64, device="cuda"), B1, B2, eps, None, 1.0, 1)
    assert torch.equal(p[still], before[still])
    # m is subnormal where eps is: its product with b1 is off by 2^-150, which eps divides
    low = torch.where(g == 0, LR / (1 - B1 ** 3) * 2.0 ** -149 / eps * (m != 0), 0.0)
    check(p, want, bound + low)
