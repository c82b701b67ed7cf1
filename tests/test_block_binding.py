"""The binding of a transformer block's operators refuses arrays that are shorter than the call reads, or that hold
something else, without a GPU."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr

DEV, SHAPE = qt2.QT2_ERR_DEVICE, qt2.QT2_ERR_SHAPE
M, F, K = 256, 384, 128


def refused(call, status):
    with pytest.raises(qt2.QT2Error) as e:
        call()
    assert e.value.status == status


def view(R, C, scales=1):
    return qt2.View(torch.zeros(R, C // 2, dtype=torch.uint8), torch.zeros(R * C // 16, dtype=torch.uint8), torch.zeros(scales))


@pytest.mark.parametrize("arg", range(5))
def test_views_with_a_scale_for_128_rows_are_refused(arg, monkeypatch):
    """Their codes and scales are those of a view with one tensor scale."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    out = torch.zeros(M, F, dtype=torch.bfloat16)

    def call(k, scales=None):
        n = lambda i, R: scales(R) if scales and i == k else 1  # noqa: E731
        if k < 3:
            tr.qt2_gemm_nvfp4_gated(view(M, K, n(0, M)), view(F, K, n(1, F)), view(F, K, n(2, F)), M, F, K, 1.0, 0, None, None, F, out, F)
        else:
            tr.qt2_gemm_nvfp4_gated_bwd(view(M, K, n(3, M)), view(F, K, n(4, F)), M, F, K, 1.0, 0, out, out, F, out, out, F, None, F)
    refused(lambda: call(arg), DEV)   # nothing else is wrong: its tensors are the host's
    refused(lambda: call(arg, lambda R: R // 128), SHAPE)
    refused(lambda: call(arg, lambda R: 0), SHAPE)
