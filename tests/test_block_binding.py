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


# 5 tokens, 2 + 1 heads of 16, the first 8 elements turned by the tables' 9 rows
T, D, P, R = 5, 16, 9, 8
VECTORS = dict(wq=(D,), wk=(D,), pos=(T,), cos=(P, R // 2), sin=(P, R // 2), dwq=(D,), dwk=(D,))


def qk(backward, T=T, D=D, P=P, R=R, **shapes):
    v = {k: None if s is None else torch.zeros(s, dtype=torch.int64 if k == "pos" else torch.float32) for k, s in dict(VECTORS, **shapes).items()}
    x, ws = torch.zeros(5, 3, 16), torch.zeros(1 << 16, dtype=torch.uint8)
    rest = v["wq"], v["wk"], 1e-6, v["pos"], v["cos"], v["sin"], P, R, tr.QT2_ROPE_HALVES
    if backward:
        tr.qt2_qk_norm_rope_bwd(x, 48, 16, x, T, 2, 1, D, 48, 16, *rest, x, 48, 16, v["dwq"], v["dwk"], ws, 1 << 16)
    else:
        tr.qt2_qk_norm_rope_fwd(x, T, 2, 1, D, 48, 16, *rest, torch.zeros(5, 3, 16), 48, 16)


@pytest.mark.parametrize("backward", [False, True])
def test_rotations_vectors_have_the_calls_sizes(backward, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    # nothing else is wrong: the tensors are the host's; longer positions, more rows, other shapes of one size
    for right in (dict(), dict(pos=(T + 3,)), dict(pos=(1, T)), dict(cos=(P + 2, R // 2), sin=(P + 1, R // 2)), dict(cos=(P * R // 2,)),
                  dict(wq=(4, 4)), dict(cos=(P, 1, R // 2)), dict(wq=None, wk=None, pos=None, dwq=None), dict(R=0, cos=(3,), sin=None)):
        refused(lambda: qk(backward, **right), DEV)
    bad = [dict(wq=(D - 1,)), dict(wk=(D + 1,)), dict(wq=(3, D)), dict(wk=(0,)), dict(pos=(T - 1,)), dict(pos=(1,)), dict(R=0, pos=(T - 1,)),
           dict(cos=(P, R)), dict(sin=(P, R)), dict(cos=(P - 1, R // 2)), dict(sin=(P * R // 2 - 1,)), dict(cos=(P * R // 2 + 4,)), dict(sin=(1,))]
    for case in bad + ([dict(dwq=(D - 1,)), dict(dwk=(2 * D,))] if backward else []):
        refused(lambda: qk(backward, **case), SHAPE)
