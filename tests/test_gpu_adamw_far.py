"""AdamW's 8-bit codes bit for bit in a tensor of more than 2^31 elements (the draws' counter has a high word from 2^34
elements on, which no test reaches: such a tensor and its arrays take 100 GB)."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2_train as tr
from tests.codes_ref import encode, words

pytestmark = pytest.mark.gpu
B1, B2, SEED = 0.9, 0.95, (7 << 32) + 5
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def test_codes_and_draws_past_2_to_31_elements():
    n, far = (1 << 31) + 4096 + 5, 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(8)
    g, p = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(E4) for _ in range(2))
    ms, vs = (torch.zeros((n + 255) // 256, device="cuda") for _ in range(2))
    # the first blocks, those on both sides of 2^30 and 2^31 elements, and the last ones
    spans = [(0, 5000), ((1 << 30) - 1024, (1 << 30) + 1024), (far - 1024, n)]
    for a, b in spans:
        g[a:b] = torch.randn(b - a, generator=gen, device="cuda").to(BF)
    lst = tr.AdamWList([torch.zeros(4, dtype=BF, device="cuda"), p], [torch.zeros(4, dtype=BF, device="cuda"), g], [torch.zeros(4, device="cuda"), m],
                       [torch.zeros(4, device="cuda"), v], None, [None, ms], [None, vs])   # the tensor's place in the list is 1
    lr, step = torch.full((1,), 1e-3, device="cuda"), torch.full((1,), (1 << 32) + 6, dtype=torch.int64, device="cuda")
    tr.qt2_adamw(lst, lr, step, B1, B2, 1e-8, None, 1.0, SEED)
    f32 = lambda x: torch.tensor(x, dtype=torch.float64).float().cuda()  # noqa: E731
    for a, b in spans:
        a, b = a // 256 * 256, min(n, (b + 255) // 256 * 256)
        x = g[a:b].float()
        w = words(a, b - a, 1, 6, SEED)
        for value, draw, codes, scales, root in ((x * f32(1 - B1), w & 0xFFFF, m, ms, False),
                                                 ((x * x * f32(1 - B2)).sqrt(), w >> 16, v, vs, True)):
            want, scale = encode(value, draw, root)
            assert torch.equal(codes[a:b].double(), want) and torch.equal(scales[a // 256:(b + 255) // 256], scale), (a, root)
            # another draw would give other codes
            other, _ = encode(value, words(a + 4096 if a == 0 else a - 4096, b - a, 1, 6, SEED) & 0xFFFF, root)
            assert not torch.equal(codes[a:b].double(), other)
    assert (ms[20:1000] == 0).all() and tr.qt2_train_device_status() == 0
