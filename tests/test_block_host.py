"""Host-side checks of the operators of the block around the experts (no GPU): bad
arguments are rejected with their status before anything is enqueued, empty calls enqueue
nothing, and the 64-bit reference forms agree with autograd."""
import ctypes

import pytest
import torch

import block_reference as R
import grouped_int4_dequant_amd as moe
from grouped_int4_dequant_amd import binding as B

p = 0x1000
EINVAL, EUNSUP, EWS, OK = B.MOE_EINVAL, B.MOE_EUNSUPPORTED, B.MOE_EWORKSPACE, B.MOE_OK
LARGE = (1 << 30) + 1
NAN = float("nan")


def call(name, good, **change):
    args = dict(good, **change)
    return getattr(moe.load(), name)(*args.values(), None)


LINEAR = dict(dtype=0, x=p, ldx=64, T=8, N=32, K=64, W=p, bias=p, bias_dtype=0, act=2, res=p, ldres=32, pre=p, ldpre=32, y=p, y_dtype=0, ldy=32)
LGRAD = dict(dtype=0, dy=p, lddy=32, x=p, ldx=64, T=8, N=32, K=64, W=p, pre=p, ldpre=32, act=2, dx=p, dx_dtype=0, lddx=64, dW=p, db=p, g_dtype=2,
             acc=0, ws=p, ws_bytes=1 << 30)
NORM = dict(dtype=0, o=p, ldo=64, x=p, ldx=64, s_dtype=0, T=8, d=64, w_o=p, gate=p, gates=2, w_n=p, w_dtype=0, scale=1.0, eps=1e-6, y=p, ldy=64, n=p, ldn=64)
NGRAD = dict(dtype=0, dy=p, lddy=64, dn=p, lddn=64, o=p, ldo=64, y=p, ldy=64, s_dtype=0, T=8, d=64, w_o=p, gate=p, gates=2, w_n=p, w_dtype=0, scale=1.0,
             eps=1e-6, dx=p, lddx=64, d_o=p, lddo=64, dw_o=p, dgate=p, dw_n=p, g_dtype=2, acc=0, ws=p, ws_bytes=1 << 30)
LAYER = dict(dtype=0, d=64, f=32, E=16, k=2, f_sh=8, gu=p, dn=p, sh_gu=p, sh_dn=p)
FEW = dict(L=LAYER, x=p, ldx=64, logits=p, T=8, add=p, ldadd=64, y=p, y_dtype=0, ldy=64, ids=p, w=p, ws=p, ws_bytes=1 << 30)

REFUSED = [
    ("moe_linear", LINEAR, EINVAL, dict(dtype=2), dict(y_dtype=1), dict(bias_dtype=1), dict(act=-1), dict(act=7), dict(x=None), dict(W=None), dict(y=None),
     dict(x=p + 1), dict(W=p + 1), dict(y=p + 1), dict(bias=p + 1), dict(bias_dtype=2, bias=p + 2), dict(res=p + 1), dict(pre=p + 1), dict(T=-1), dict(N=0),
     dict(K=0), dict(ldx=63), dict(ldy=31), dict(ldres=31), dict(ldpre=31), dict(act=5, N=31), dict(act=5, ldpre=31), dict(act=5, ldy=15),
     dict(res=p, y=p, ldres=40), dict(y_dtype=2, y=p + 2)),
    ("moe_linear", LINEAR, EUNSUP, dict(T=1, N=1 << 30, ldy=1 << 30, ldres=1 << 30, ldpre=1 << 30), dict(T=1 << 30, N=1 << 20, ldy=1 << 20, ldres=1 << 20, ldpre=1 << 20),
     dict(T=LARGE), dict(N=LARGE, ldy=LARGE, ldres=LARGE, ldpre=LARGE), dict(K=LARGE, ldx=LARGE)),
    ("moe_linear_backward", LGRAD, EINVAL, dict(dtype=2), dict(dx_dtype=1), dict(g_dtype=1), dict(act=9), dict(dy=None), dict(x=None), dict(W=None),
     dict(pre=None), dict(dx=None, dW=None, db=None), dict(dy=p + 1), dict(x=p + 1), dict(W=p + 1), dict(pre=p + 1), dict(dW=p + 2), dict(db=p + 2), dict(dx=p + 1),
     dict(ws=None), dict(ws=p + 16), dict(T=-1), dict(N=0), dict(K=0), dict(lddy=31), dict(ldx=63), dict(ldpre=31), dict(lddx=63), dict(act=6, N=33)),
    ("moe_linear_backward", LGRAD, EUNSUP, dict(g_dtype=0, acc=1), dict(act=0, T=1, N=1 << 29, lddy=1 << 29, K=8, ws_bytes=1 << 40),
     dict(act=0, db=None, N=1 << 20, lddy=1 << 20, K=1 << 20, ldx=1 << 20, lddx=1 << 20), dict(act=0, db=None, dW=None, T=1, K=1 << 30, ldx=1 << 30, lddx=1 << 30), dict(T=LARGE), dict(N=LARGE, lddy=LARGE, ldpre=LARGE), dict(K=LARGE, ldx=LARGE, lddx=LARGE)),
    ("moe_linear_backward", LGRAD, EWS, dict(ws_bytes=8 * 32 * 2), dict(act=0, ws_bytes=0), dict(db=None, ws_bytes=8 * 32 * 2 - 1),
     dict(act=0, db=None, T=8192, N=512, K=512, lddy=512, ldx=512, lddx=512, ws_bytes=1 << 20)),
    ("moe_residual_norm", NORM, EINVAL, dict(dtype=2), dict(s_dtype=1), dict(w_dtype=1), dict(o=None, x=None), dict(y=None, n=None), dict(w_n=None), dict(o=p + 1),
     dict(x=p + 1), dict(w_o=p + 1), dict(gate=p + 1), dict(w_n=p + 1), dict(y=p + 1), dict(n=p + 1), dict(w_dtype=2, w_o=p + 2), dict(s_dtype=2, x=p + 2),
     dict(gates=0), dict(gates=3), dict(T=-1), dict(d=0), dict(ldo=63), dict(ldx=63), dict(ldy=63), dict(ldn=63), dict(eps=-1.0), dict(eps=NAN),
     dict(ldx=72), dict(ldo=72)),
    ("moe_residual_norm", NORM, EUNSUP, dict(d=16385, ldo=1 << 15, ldx=1 << 15, ldy=1 << 15, ldn=1 << 15), dict(T=LARGE + 1)),
    ("moe_residual_norm_backward", NGRAD, EINVAL, dict(dtype=2), dict(s_dtype=1), dict(w_dtype=1), dict(g_dtype=1), dict(dy=None, dn=None), dict(o=None), dict(y=None),
     dict(w_n=None), dict(w_o=None), dict(gate=None), dict(dn=None), dict(dx=None, d_o=None, dw_o=None, dgate=None, dw_n=None), dict(dy=p + 1), dict(dn=p + 1),
     dict(o=p + 1), dict(y=p + 1), dict(dx=p + 1), dict(d_o=p + 1), dict(dw_o=p + 2), dict(dgate=p + 2), dict(dw_n=p + 2), dict(ws=None), dict(ws=p + 16),
     dict(gates=3), dict(gates=0), dict(T=-1), dict(d=0), dict(lddy=63), dict(lddn=63), dict(ldo=63), dict(ldy=63), dict(lddx=63), dict(lddo=63), dict(eps=-1.0),
     dict(dx=p, dy=p, lddx=72)),
    ("moe_residual_norm_backward", NGRAD, EUNSUP, dict(g_dtype=0, acc=1), dict(T=LARGE + 1)),
    ("moe_residual_norm_backward", NGRAD, EWS, dict(ws_bytes=3 * 8 * 64 * 4 - 1)),
]


@pytest.mark.parametrize("name,good,expect,change", [(n, g, e, c) for n, g, e, *cs in REFUSED for c in cs],
                         ids=[f"{n[4:]}-{'-'.join(f'{k}={v}' for k, v in c.items())}" for n, _, _, *cs in REFUSED for c in cs])
def test_refusals(name, good, expect, change):
    assert call(name, good, **change) == expect


def few(layer=None, **change):
    args = dict(FEW, **change)
    L = None if layer is False else B.MoeLayer16T(*dict(LAYER, **(layer or {})).values())
    args["L"] = None if L is None else ctypes.byref(L)
    return moe.load().moe_few_tokens_layer(*args.values(), None)


@pytest.mark.parametrize("layer,change", [(dict(dtype=2), {}), (dict(d=0), {}), (dict(f=0), {}), (dict(E=0), {}), (dict(k=0), {}), (dict(k=17), {}), (dict(f_sh=-1), {}),
                                          (dict(gu=None), {}), (dict(dn=None), {}), (dict(sh_gu=None), {}), (dict(sh_dn=None), {}), (dict(gu=p + 1), {}),
                                          (dict(dn=p + 1), {}), (dict(sh_gu=p + 1), {}), (False, {}), ({}, dict(x=None)), ({}, dict(logits=None)), ({}, dict(y=None)),
                                          ({}, dict(x=p + 1)), ({}, dict(logits=p + 2)), ({}, dict(y=p + 1)), ({}, dict(add=p + 1)), ({}, dict(ids=p + 2)),
                                          ({}, dict(w=p + 2)), ({}, dict(T=-1)), ({}, dict(ldx=63)), ({}, dict(ldy=63)), ({}, dict(ldadd=63)), ({}, dict(y_dtype=1)),
                                          ({}, dict(ldadd=72)), ({}, dict(ws=None)), ({}, dict(ws=p + 16))], ids=str)
def test_few_layer_refusals(layer, change):
    assert few(layer, **change) == EINVAL


def test_few_layer_limits():
    wide = dict(ldx=1 << 21, ldy=1 << 21, ldadd=1 << 21)
    assert few(dict(E=1025)) == EUNSUP and few(dict(E=100, k=65)) == EUNSUP and few({}, T=65) == EUNSUP and few(dict(k=9), T=64) == EUNSUP
    assert few(dict(d=(1 << 20) + 1), **wide) == EUNSUP and few(dict(f=(1 << 20) + 1)) == EUNSUP and few(dict(f_sh=(1 << 20) + 1)) == EUNSUP
    need = moe.few_tokens_workspace_bytes(8, torch.bfloat16, 64, 32, 16, 2, 8)
    assert few({}, ws_bytes=need - 1) == EWS
    assert need >= 8 * 2 * 32 * 4 + 8 * 8 * 4 and moe.few_tokens_workspace_bytes(65, torch.bfloat16, 64, 32, 16, 2) == 0
    assert few({}, T=0, x=None, logits=None, y=None, ws=None, ws_bytes=0) == OK


def test_empty_calls_enqueue_nothing():
    assert call("moe_linear", LINEAR, T=0, x=None, y=None, W=None) == OK
    assert call("moe_linear_backward", LGRAD, T=0, acc=1, dy=None, x=None, dx=None) == OK
    assert call("moe_linear_backward", LGRAD, T=0, dW=None, db=None, ws=None, ws_bytes=0, act=0) == OK
    assert call("moe_residual_norm", NORM, T=0, o=None, x=None, y=None, n=None) == OK
    assert call("moe_residual_norm_backward", NGRAD, T=0, acc=1, dy=None, dn=None, o=None, y=None, dx=None, d_o=None) == OK


def test_workspace_bytes():
    f = moe.linear_backward_workspace_bytes
    assert f(100, 64, 64, "silu") >= 100 * 64 * 2 + 64 * 4 and f(0, 64, 64, "none") > 0 and f(100, 64, 64, "none") < 100 * 64 * 2
    assert f(8192, 512, 512) > 2 * 512 * 512 * 4 and f(1 << 20, 1 << 13, 1 << 13) < 1 << 28
    assert B.load().moe_linear_backward_workspace_bytes(-1, 64, 64, 0) == 0 and B.load().moe_linear_backward_workspace_bytes(4, 63, 64, 5) == 0
    g = moe.residual_norm_backward_workspace_bytes
    assert g(100, 64, 1) >= 3 * 64 * 4 and g(0, 64, 3) > 0 and g(100, 64, 3) == 0 and g(100, 16385, 1) == 0 and g(100, 64, 0) == 0


def test_tensors_and_arguments_are_checked():
    x, w, v = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    e = torch.zeros(3, 12, 8, dtype=torch.bfloat16)
    for f in (lambda: moe.linear(x, w), lambda: moe.linear_backward(x, x, w), lambda: moe.residual_norm(x, x, w_n=v), lambda: moe.residual_norm(None, x, w_n=v),
              lambda: moe.residual_norm_backward(x, None, None, None), lambda: moe.few_tokens_layer(x, x.float(), e, e, 1)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        moe.linear(x.float(), w)
    with pytest.raises(ValueError, match="given"):
        moe.residual_norm(None, None)
    with pytest.raises(ValueError, match="given"):
        moe.residual_norm_backward(None, None, None, None)
    with pytest.raises(ValueError, match="act"):
        moe.linear_backward_workspace_bytes(4, 8, 8, "softplus")
    with pytest.raises(ValueError, match="even"):
        moe.linear_backward_workspace_bytes(4, 7, 8, "geglu")


@pytest.mark.parametrize("act", list(moe.ACTIVATIONS))
def test_linear_reference_against_autograd(act):
    g = torch.Generator().manual_seed(0)
    x, W, b = (torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True) for s in ((5, 6), (8, 6), (8,)))
    z = x @ W.T + b
    y = R.curve(R.GATED[act], z[:, :4]) * z[:, 4:] if act in R.GATED else R.curve(act, z)
    assert torch.allclose(y, R.linear(x, W, b, act, None)[0])
    f = dict(relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu, gelu_tanh=lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
             none=lambda v: v)[R.GATED.get(act, act)]
    assert torch.allclose(R.curve(R.GATED.get(act, act), z), f(z))
    dy = torch.randn(y.shape, generator=g, dtype=torch.float64)
    y.backward(dy)
    (dx, _), (dW, _), (db, _) = R.linear_grad(dy, x, W, z, act, torch.float32)
    assert torch.allclose(dx, x.grad) and torch.allclose(dW, W.grad) and torch.allclose(db, b.grad)


def test_norm_reference_against_autograd():
    g = torch.Generator().manual_seed(1)
    o, x, wo, ga, wn = (torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True) for s in ((6, 5), (6, 5), (5,), (3, 5), (5,)))

    def normed(v, w):
        return v * (v * v).mean(1, keepdim=True).add(1e-6).rsqrt() * w
    y = 0.5 * x + ga.repeat_interleave(2, 0) * normed(o, wo)
    n = normed(y, wn)
    (v, _), (m, _) = R.norm(o, x, wo, ga, 0.5, wn, 1e-6)
    assert torch.allclose(v, y) and torch.allclose(m, n)
    dy, dn = (torch.randn(6, 5, generator=g, dtype=torch.float64) for _ in range(2))
    ((y * dy).sum() + (n * dn).sum()).backward()
    got = R.norm_grad(dy, dn, o, y, wo, ga, 0.5, wn, 1e-6)
    for name, t in dict(dx=x, d_o=o, dw_o=wo, dgate=ga, dw_n=wn).items():
        assert torch.allclose(got[name][0], t.grad), name
