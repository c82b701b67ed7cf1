"""AdamW's 8-bit states as include/qt2_train.h defines them: what a value's E4M3 code and a block's scale are, given
the element's draw."""
import numpy as np
import torch

from tests import block_ref as ref


def words(first, n, tensor, step, seed, device="cuda"):
    """The draws' words of elements [first, first + n) (first a multiple of 4)."""
    group = np.arange(first // 4, (first + n + 3) // 4, dtype=np.uint64)
    c = np.stack([group & np.uint64(0xFFFFFFFF), group >> np.uint64(32), np.full_like(group, tensor),
                  np.full_like(group, step & 0xFFFFFFFF)], 1)
    return torch.from_numpy(ref.philox(c, seed).reshape(-1)[:n].astype(np.int64)).to(device)


def encode(x, draw, root):
    """(codes' values, scales) of fp32 values x in blocks of 256 under 16-bit draws; root: of sqrt(v).  The products
    are fp32 operations, what follows is exact in 64 bits."""
    top = torch.stack([c.abs().max() for c in x.split(256)])
    most = torch.full_like(top, 448)   # an array: divided by a number, torch multiplies with its reciprocal
    zero = top < 2.0 ** -100
    inv = torch.where(zero, 0.0, most / top).repeat_interleave(256)[:x.numel()]
    a = x.abs() * inv
    lift = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)
    z = (a + lift).double()
    unit = (torch.frexp(z.clamp(min=2.0 ** -6))[1].long() - 4 + 1023 << 52).view(torch.float64)   # powers of two, exact
    k = (z / unit).floor()
    k += (z / unit - k) * 2 ** 20 + 16 * draw >= 2 ** 20
    y = (k * unit - lift.double()).clamp(max=448)
    if root:
        y = torch.where((a > 0) & (y == 0), 2.0 ** -9, y)
    return torch.where(x < 0, -y, y), torch.where(zero, 0.0, top / most)
