"""Host-side checks of the 16-bit operators (no GPU): bad arguments are
rejected with their status before anything is enqueued, empty calls enqueue nothing,
and the 64-bit reference forms agree with autograd."""
import pytest
import torch

import grouped_int4_dequant_amd as moe
from grouped_int4_dequant_amd import binding as B
import grouped_reference as R

p = 0x1000
EINVAL, EUNSUP, EWS, OK = B.MOE_EINVAL, B.MOE_EUNSUPPORTED, B.MOE_EWORKSPACE, B.MOE_OK


def call(name, good, **change):
    args = dict(good, **change)
    return getattr(moe.load(), name)(*args.values(), None)


GEMM = dict(dtype=0, A=p, lda=64, a_rows=8, a_row=p, offsets=p, G=4, P=8, N=32, K=64, W=p, C=p, c_dtype=0, ldc=32)
DGRAD = dict(dtype=0, dC=p, lddc=32, offsets=p, G=4, P=8, N=32, K=64, W=p, dA=p, da_dtype=0, ldda=64)
WGRAD = dict(dtype=0, dC=p, lddc=32, A=p, lda=64, a_rows=8, a_row=p, offsets=p, G=4, P=8, N=32, K=64, dW=p, dw_dtype=2, acc=0)
COMBINE = dict(dtype=0, o=p, ldo=64, P=16, pos=p, w=p, T=8, k=2, d=64, add=p, add_dtype=0, ldadd=64, y=p, y_dtype=0, ldy=64)
CGRAD = dict(dtype=0, dy=p, lddy=64, o=p, ldo=64, P=16, pos=p, w=p, T=8, k=2, d=64, d_o=p, lddo=64, dw=p)
PLAN = dict(ids=p, T=8, n=4, rows=p, offsets=p)
ADAPTER = dict(dtype=0, x=p, ldx=64, T=8, K=64, N=32, r=16, n=4, A=p, B=p, scale=p, rows=p, offsets=p, base=p, ldbase=32, y=p,
               y_dtype=0, ldy=32)
AGRAD = dict(dtype=0, dy=p, lddy=32, x=p, ldx=64, T=8, K=64, N=32, r=16, n=4, A=p, B=p, scale=p, rows=p, offsets=p, dx_base=p,
             lddx_base=64, dx=p, dx_dtype=0, lddx=64, dA=p, dB=p, g_dtype=2, acc=0, ws=p, ws_bytes=1 << 20)

LARGE = (1 << 30) + 1
REFUSED = [
    ("moe_grouped_gemm", GEMM, EINVAL, dict(dtype=2), dict(dtype=3), dict(c_dtype=1), dict(A=None), dict(W=None), dict(C=None),
     dict(offsets=None), dict(A=p + 1), dict(W=p + 1), dict(C=p + 1), dict(a_row=p + 2), dict(offsets=p + 2), dict(G=0), dict(N=0),
     dict(K=0), dict(P=-1), dict(a_rows=-1), dict(lda=63), dict(ldc=31), dict(c_dtype=2, C=p + 2)),
    ("moe_grouped_gemm", GEMM, EUNSUP, dict(G=1025), dict(P=1 << 30, N=1 << 20, ldc=1 << 20)),
    ("moe_grouped_gemm_dgrad", DGRAD, EINVAL, dict(dtype=2), dict(da_dtype=1), dict(dC=None), dict(W=None), dict(dA=None),
     dict(offsets=None), dict(dC=p + 1), dict(G=0), dict(N=0), dict(K=0), dict(P=-1), dict(lddc=31), dict(ldda=63)),
    ("moe_grouped_gemm_dgrad", DGRAD, EUNSUP, dict(G=1025)),
    ("moe_grouped_gemm_wgrad", WGRAD, EINVAL, dict(dtype=2), dict(dw_dtype=1), dict(dC=None), dict(A=None), dict(dW=None),
     dict(dW=p + 2), dict(G=0), dict(P=-1), dict(a_rows=-1), dict(lda=63), dict(lddc=31), dict(P=0, dW=None)),
    ("moe_grouped_gemm_wgrad", WGRAD, EUNSUP, dict(G=1025), dict(dw_dtype=0, acc=1)),
    ("moe_combine", COMBINE, EINVAL, dict(dtype=2), dict(y_dtype=1), dict(add_dtype=1), dict(o=None), dict(pos=None), dict(y=None),
     dict(o=p + 1), dict(w=p + 2), dict(pos=p + 2), dict(add=p + 1), dict(T=-1), dict(k=0), dict(d=0), dict(P=-1), dict(ldo=63),
     dict(ldy=63), dict(ldadd=63)),
    ("moe_combine", COMBINE, EUNSUP, dict(T=(1 << 20) + 1), dict(k=1025)),
    ("moe_combine_backward", CGRAD, EINVAL, dict(dtype=2), dict(dy=None), dict(o=None), dict(pos=None), dict(d_o=None, dw=None),
     dict(dw=p + 2), dict(T=-1), dict(k=0), dict(d=0), dict(lddy=63), dict(ldo=63), dict(lddo=63)),
    ("moe_combine_backward", CGRAD, EUNSUP, dict(T=(1 << 20) + 1), dict(k=1025)),
    ("moe_adapter_plan", PLAN, EINVAL, dict(ids=None), dict(rows=None), dict(offsets=None), dict(T=-1), dict(n=0), dict(ids=p + 2)),
    ("moe_adapter_plan", PLAN, EUNSUP, dict(n=1025), dict(T=(1 << 20) + 1)),
    ("moe_adapter_forward", ADAPTER, EINVAL, dict(dtype=2), dict(y_dtype=1), dict(x=None), dict(A=None), dict(B=None), dict(rows=None),
     dict(offsets=None), dict(y=None), dict(x=p + 1), dict(scale=p + 2), dict(base=p + 1), dict(T=-1), dict(K=0), dict(N=0), dict(r=0),
     dict(n=0), dict(ldx=63), dict(ldy=31), dict(ldbase=31)),
    ("moe_adapter_forward", ADAPTER, EUNSUP, dict(r=129), dict(n=1025), dict(T=(1 << 20) + 1)),
    ("moe_adapter_backward", AGRAD, EINVAL, dict(dtype=2), dict(dx_dtype=1), dict(g_dtype=1), dict(dy=None), dict(x=None), dict(A=None),
     dict(B=None), dict(rows=None), dict(offsets=None), dict(dx=None, dA=None, dB=None), dict(dA=p + 2), dict(ws=None), dict(ws=p + 16),
     dict(lddy=31), dict(lddx=63), dict(lddx_base=63), dict(ldx=63)),
    ("moe_adapter_backward", AGRAD, EUNSUP, dict(r=129), dict(n=1025), dict(T=(1 << 20) + 1), dict(g_dtype=0, acc=1)),
    ("moe_combine", COMBINE, EINVAL, dict(y=p, add=p, y_dtype=2), dict(y=p, add=p, ldadd=72)),
    ("moe_adapter_forward", ADAPTER, EINVAL, dict(base=p, y=p, ldbase=40)),
    ("moe_adapter_backward", AGRAD, EINVAL, dict(dx_base=p, dx=p, lddx_base=72)),
    ("moe_grouped_gemm", GEMM, EUNSUP, dict(P=LARGE), dict(N=LARGE, ldc=LARGE), dict(K=LARGE, lda=LARGE)),
    ("moe_grouped_gemm_dgrad", DGRAD, EUNSUP, dict(P=LARGE), dict(N=LARGE, lddc=LARGE), dict(K=LARGE, ldda=LARGE)),
    ("moe_grouped_gemm_wgrad", WGRAD, EUNSUP, dict(P=LARGE), dict(N=LARGE, lddc=LARGE), dict(K=LARGE, lda=LARGE)),
    ("moe_combine", COMBINE, EUNSUP, dict(d=LARGE, ldo=LARGE, ldy=LARGE, ldadd=LARGE)),
    ("moe_combine_backward", CGRAD, EUNSUP, dict(d=LARGE, lddy=LARGE, ldo=LARGE, lddo=LARGE)),
    ("moe_adapter_forward", ADAPTER, EUNSUP, dict(K=LARGE, ldx=LARGE), dict(N=LARGE, ldy=LARGE, ldbase=LARGE)),
    ("moe_adapter_backward", AGRAD, EUNSUP, dict(K=LARGE, ldx=LARGE, lddx=LARGE, lddx_base=LARGE), dict(N=LARGE, lddy=LARGE)),
    ("moe_adapter_backward", AGRAD, EWS, dict(ws_bytes=2 * 8 * 16 * 4 - 1), dict(r=17, ws_bytes=2 * 8 * 32 * 4 - 1)),
]


@pytest.mark.parametrize("name,good,expect,change", [(n, g, e, c) for n, g, e, *cs in REFUSED for c in cs],
                         ids=[f"{n[4:]}-{'-'.join(f'{k}={v}' for k, v in c.items())}" for n, _, _, *cs in REFUSED for c in cs])
def test_refusals(name, good, expect, change):
    assert call(name, good, **change) == expect


def test_empty_calls_enqueue_nothing():
    assert call("moe_grouped_gemm", GEMM, P=0, A=None, C=None, W=None) == OK
    assert call("moe_grouped_gemm_dgrad", DGRAD, P=0, dC=None, dA=None, W=None) == OK
    assert call("moe_grouped_gemm_wgrad", WGRAD, P=0, acc=1, dC=None, A=None) == OK
    assert call("moe_combine", COMBINE, T=0, o=None, y=None) == OK
    assert call("moe_combine_backward", CGRAD, T=0, dy=None) == OK
    assert call("moe_adapter_forward", ADAPTER, T=0, x=None, rows=None, y=None) == OK
    assert call("moe_adapter_backward", AGRAD, T=0, acc=1, x=None, dy=None, rows=None) == OK


def test_workspace_bytes():
    f = moe.adapter_backward_workspace_bytes
    assert f(100, 16) == 2 * 100 * 16 * 4 and f(100, 17) == 2 * 100 * 32 * 4 and f(7, 128) == 2 * 7 * 128 * 4
    assert f(0, 4) > 0 and f(-1, 4) == 0 and f(4, 0) == 0 and f(4, 129) == 0


def test_tensors_off_the_gpu_are_refused():
    x, w, o = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for f in (lambda: moe.grouped_gemm(x, w, o), lambda: moe.grouped_gemm_dgrad(x, w, o), lambda: moe.grouped_gemm_wgrad(x, x, o),
              lambda: moe.combine(x, o.view(1, 3)), lambda: moe.combine_backward(x, x, o.view(1, 3)), lambda: moe.adapter_plan(o, 2),
              lambda: moe.adapter_forward(x, w, w, None, (o, o)), lambda: moe.adapter_backward(x, x, w, w, None, (o, o))):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(TypeError):
        moe.grouped_gemm(x.float(), w, o)


def test_reference_forms_against_autograd():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True)  # noqa: E731
    offsets, a_row = torch.tensor([0, 2, 2, 5]), torch.tensor([1, 3, 0, 3, 2])
    A, W, G = r(4, 6), r(3, 5, 6), torch.randn(5, 5, generator=g, dtype=torch.float64)
    C = torch.cat([A[a_row[a:b]] @ W[e].T for e, a, b in R.spans(offsets)])
    assert torch.allclose(C, R.grouped(A, W, offsets, a_row, 5)[0])
    C.backward(G)
    assert torch.allclose(W.grad, R.grouped_wgrad(G, A, offsets, a_row)[0])
    rows = R.grouped_dgrad(G, W, offsets)[0]
    assert torch.allclose(A.grad, torch.zeros(4, 6, dtype=torch.float64).index_add(0, a_row, rows))
    x, P, Q, base, dy = r(7, 6), r(3, 2, 6), r(3, 5, 2), r(7, 5), torch.randn(7, 5, generator=g, dtype=torch.float64)
    s, ids = torch.tensor([0.5, 2.0, 1.5], dtype=torch.float64), torch.tensor([2, 0, -1, 0, 1, 3, 2])
    y = torch.stack([base[t] + (s[e] * Q[e] @ (P[e] @ x[t]) if 0 <= e < 3 else 0) for t, e in enumerate(ids.tolist())])
    assert torch.allclose(y, R.adapter(x, P, Q, s, ids, base)[0])
    y.backward(dy)
    (dx, _), (dA, _), (dB, _) = R.adapter_grad(dy, x, P, Q, s, ids, None)
    assert torch.allclose(x.grad, dx) and torch.allclose(P.grad, dA) and torch.allclose(Q.grad, dB)
