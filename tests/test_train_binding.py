"""The binding of the training operators hands the library addresses: vectors that are not one element
after the other (expanded ones take one element of memory) are refused, without a GPU."""
import pytest
import torch

from nvfp4_quantized_b200 import qt2
from nvfp4_quantized_b200 import qt2_train as tr

R, C, V = 6, 16, 24
x, y, dy, dx = (torch.zeros(R, C, dtype=torch.bfloat16) for _ in range(4))
w, dw = (torch.zeros(V, C, dtype=torch.bfloat16) for _ in range(2))
ws = torch.zeros(1 << 20, dtype=torch.uint8)
f32 = lambda n: torch.zeros(n)  # noqa: E731
CALLS = {
    "qt2_layernorm_fwd": (lambda v: tr.qt2_layernorm_fwd(x, R, C, C, v["weight"], v["bias"], 1e-5, y, C, v["mean"],
                                                         v["rstd"]),
                          dict(weight=f32(C), bias=f32(C), mean=f32(R), rstd=f32(R))),
    "qt2_layernorm_bwd": (lambda v: tr.qt2_layernorm_bwd(dy, C, x, R, C, C, v["weight"], v["mean"], v["rstd"], dx, C,
                                                         v["dweight"], v["dbias"], v["ws"], 1 << 20),
                          dict(weight=f32(C), mean=f32(R), rstd=f32(R), dweight=f32(C), dbias=f32(C), ws=ws)),
    "qt2_linear_xent_fwd": (lambda v: tr.qt2_linear_xent_fwd(x, w, v["targets"], R, C, V, C, C, -100, v["loss"],
                                                             v["lse"], v["ws"], 1 << 20),
                            dict(targets=f32(R).long(), loss=f32(R), lse=f32(R), ws=ws)),
    "qt2_linear_xent_bwd": (lambda v: tr.qt2_linear_xent_bwd(x, w, v["targets"], v["lse"], v["dloss"], R, C, V, C, C,
                                                             -100, dx, C, dw, 0, C, v["ws"], 1 << 20),
                            dict(targets=f32(R).long(), lse=f32(R), dloss=f32(R), ws=ws))}


@pytest.mark.parametrize("name,arg", [(n, a) for n, (_, vs) in CALLS.items() for a in vs])
def test_vectors_that_are_not_contiguous_are_refused(name, arg, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    call, vectors = CALLS[name]
    with pytest.raises(qt2.QT2Error) as e:
        call(vectors)
    assert e.value.status == qt2.QT2_ERR_DEVICE   # nothing else is wrong with the call: its tensors are the host's
    t = vectors[arg]
    for bad in (t[:1].expand(t.numel()), torch.zeros(2 * t.numel(), dtype=t.dtype)[::2],
                torch.zeros(2, t.numel(), dtype=t.dtype).t()):
        with pytest.raises(qt2.QT2Error) as e:
            call(dict(vectors, **{arg: bad}))
        assert e.value.status == qt2.QT2_ERR_INVALID_ARG
    # several dimensions are one vector where they lie one behind the other
    with pytest.raises(qt2.QT2Error) as e:
        call(dict(vectors, **{arg: t.reshape(2, -1)}))
    assert e.value.status == qt2.QT2_ERR_DEVICE


def test_workspace_of_the_gradient_norm(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    grads = tr.GradList([torch.zeros(8)])
    for bad, status in ((ws, qt2.QT2_ERR_DEVICE), (ws[::2], qt2.QT2_ERR_INVALID_ARG)):
        with pytest.raises(qt2.QT2Error) as e:
            tr.qt2_grad_norm(grads, torch.zeros(1), bad, 1 << 20)
        assert e.value.status == status


@pytest.mark.parametrize("arg", ["ldx", "ldw"])
def test_leading_dimensions_that_no_tensor_map_holds(arg):
    """A row stride of 2^40 bytes is refused as a shape, with the device and the library's CUDA calls left out."""
    from tests.test_train_abi import _xent_bwd, _xent_fwd
    L = tr.lib()
    for call in (_xent_fwd, _xent_bwd):
        for ld, status in (((1 << 39) - 8, qt2.QT2_OK), (1 << 39, qt2.QT2_ERR_SHAPE), (1 << 42, qt2.QT2_ERR_SHAPE)):
            with tr.fault_hook(lambda site: qt2.FAULT_SKIP):
                assert call(L, **{arg: ld}) == status, ld
