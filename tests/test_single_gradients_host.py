"""What the Python calls refuse of gradients that are not wanted, without a GPU."""
import pytest
import torch

import grouped_int4_dequant_amd as moe
from grouped_int4_dequant_amd import binding as B


@pytest.fixture
def on_gpu(monkeypatch):
    """Checks run on CPU tensors as on the GPU's; the call itself is recorded."""
    calls = []

    class Call(B._Call):
        __slots__ = ()

        def __init__(self, lead, name, stream):
            self.lead, self.dtype, self.device, self.index, self.stream, self.given = lead, lead.dtype, lead.device, lead.get_device(), None, None
            self.code = B._CODES[lead.dtype]

        def __call__(self, what, *args):
            calls.append((what, args))
    monkeypatch.setattr(B, "_Call", Call)
    return calls


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_linear(on_gpu):
    dy, x, W = t(4, 6), t(4, 8), t(6, 8)
    for args, kw in (((dy, None, W), {}), ((dy, None, W), dict(dx=False)), ((dy, x, None), {}), ((dy, x, None), dict(dW=False)), ((dy, None, None), dict(dx=False, dW=False)),
                     ((dy, x, W), dict(dx=False, dW=False)), ((dy, x[0], W), dict(dW=False)), ((dy, x, W[0]), dict(dx=False)),
                     ((dy, x, W), dict(dx=False, accumulate=True)), ((dy, x, W), dict(dW=False, bias_grad=True, accumulate=True)),
                     ((dy, None, t(5, 8)), dict(dW=False)), ((dy, t(3, 8), None), dict(dx=False))):
        with pytest.raises(ValueError):
            moe.linear_backward(*args, **kw)
    assert not on_gpu
    assert moe.linear_backward(dy, None, W, dW=False)[1:] == (None, None) and moe.linear_backward(dy, x, None, dx=False)[0] is None
    # x and dW, then W and dx are NULL
    (_, first), (_, second) = on_gpu
    assert first[3] is None and first[15] is None and second[8] is None and second[12] is None
    assert moe.linear_backward(t(4, 6), t(4, 8), None, pre=t(4, 12), act="swiglu", dx=False)[1].shape == (12, 8)


def test_norm(on_gpu):
    o, w = t(4, 8), t(8)
    with pytest.raises(ValueError, match="wanted"):
        moe.residual_norm_backward(o, o, o, o, w_o=w, w_n=w, dx=False, d_o=False, dw_o=False, dw_n=False)
    with pytest.raises(ValueError, match="nothing"):
        moe.residual_norm_backward(o, None, None, None, d_o=o)
    got = moe.residual_norm_backward(o, o, o, o, w_o=w, w_n=w, dx=False, d_o=False, dw_o=False)
    assert got[:4] == (None, None, None, None) and got[4].shape == (8,)
    assert moe.residual_norm_backward(o, None, None, None, d_o=False, dw_o=False)[0].shape == (4, 8)
