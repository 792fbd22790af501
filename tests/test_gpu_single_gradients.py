"""One gradient alone at the C interface, as a program with a frozen weight or a first layer asks for it: NULL for the results that are
not wanted and for what only they are formed of. Against the plain 64-bit forms, element by element."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    return m.load()


@pytest.fixture(scope="module")
def codes():
    from grouped_int4_dequant_amd import binding
    return binding._CODES


def rnd(g, *shape, dtype=BF, scale=1.0, shift=0.0):
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).cuda()


def ptr(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


WANTED = [("dx",), ("dW",), ("db",), ("dx", "dW"), ("dx", "db"), ("dW", "db")]
SHAPES = {"few": (33, 264, 200), "small": (129, 200, 328), "odd": (77, 66, 131), "wide": (700, 264, 6672), "cut": (4100, 520, 776), "none": (0, 24, 16)}


@pytest.mark.parametrize("wanted", WANTED, ids="-".join)
@pytest.mark.parametrize("act,dtype,grad", [("none", BF, F4), ("none", FP, FP), ("swiglu", BF, BF), ("gelu", BF, F4), ("swiglu", FP, F4), ("silu", FP, FP)],
                         ids=lambda v: v if isinstance(v, str) else str(v)[6:])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(lib, codes, shape, act, dtype, grad, wanted):
    import grouped_int4_dequant_amd as m
    T, N, K = SHAPES[shape]
    g = torch.Generator().manual_seed(7)
    cols = N // 2 if act in R.GATED else N
    dy, x, W, pre = rnd(g, T, cols, dtype=dtype), rnd(g, T, K, dtype=dtype), rnd(g, N, K, dtype=dtype, scale=K ** -0.5), rnd(g, T, N, dtype=dtype)
    out = dict(dx=torch.full((T, K), 9.0, dtype=grad, device="cuda"), dW=torch.full((N, K), 9.0, dtype=grad, device="cuda"), db=torch.full((N,), 9.0, dtype=grad, device="cuda"))
    given = {k: v if k in wanted else None for k, v in out.items()}
    need = m.linear_backward_workspace_bytes(T, N, K, act)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda") if act != "none" or "dW" in wanted or "db" in wanted else None
    status = lib.moe_linear_backward(codes[dtype], ptr(dy), cols, ptr(x) if "dW" in wanted else None, K, T, N, K, ptr(W) if "dx" in wanted else None,
                                     ptr(pre) if act != "none" else None, N, m.ACTIVATIONS[act], ptr(given["dx"]), codes[grad], K, ptr(given["dW"]), ptr(given["db"]),
                                     codes[grad], 0, ptr(ws), 0 if ws is None else need, stream())
    assert status == 0
    for (name, v), (value, slack) in zip(out.items(), R.linear_grad(dy, x, W, pre, act, dtype)):
        if name in wanted:
            R.within(v, value, R.stored(value, slack, grad), name)
        else:
            assert (v == 9).all()
    assert ws is None or (ws[need:] == 255).all()


NORM = ["dx", "d_o", "dw_o", "dgate", "dw_n"]


@pytest.mark.parametrize("wanted", [(n,) for n in NORM] + [("dx", "d_o"), ("dw_o", "dw_n"), ("dgate", "dw_n"), ("dx", "dw_n")], ids="-".join)
@pytest.mark.parametrize("T,d,gates", [(1, 64, 1), (60, 520, 1), (60, 77, 5), (60, 2056, 60), (900, 264, 3), (1000, 4104, 250), (30, 9000, 2)])
@pytest.mark.parametrize("dtype,stream_type,weights", [(BF, BF, BF), (FP, F4, F4)], ids=["bf16", "fp16-fp32"])
def test_norm(lib, codes, T, d, gates, dtype, stream_type, weights, wanted):
    import grouped_int4_dequant_amd as m
    g = torch.Generator().manual_seed(8)
    o, dn, y, dy = rnd(g, T, d, dtype=dtype), rnd(g, T, d, dtype=dtype), rnd(g, T, d, dtype=stream_type), rnd(g, T, d, dtype=stream_type)
    w_o, w_n, gate = (rnd(g, *s, dtype=weights, scale=0.3, shift=1.0) for s in ((d,), (d,), (gates, d)))
    out = dict(dx=torch.empty_like(dy), d_o=torch.empty_like(o), dw_o=torch.empty_like(w_o), dgate=torch.empty_like(gate), dw_n=torch.empty_like(w_n))
    for v in out.values():
        v.fill_(9.0)
    given = {k: v if k in wanted else None for k, v in out.items()}
    sums = any(k in wanted for k in NORM[2:])
    need = m.residual_norm_backward_workspace_bytes(T, d, gates)
    ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda") if sums else None
    block = any(k in wanted for k in ("d_o", "dw_o", "dgate"))  # o is read for these alone
    status = lib.moe_residual_norm_backward(codes[dtype], ptr(dy), d, ptr(dn), d, ptr(o) if block else None, d, ptr(y), d, codes[stream_type], T, d, ptr(w_o), ptr(gate), gates,
                                            ptr(w_n), codes[weights], 0.75, 1e-6, ptr(given["dx"]), d, ptr(given["d_o"]), d, ptr(given["dw_o"]), ptr(given["dgate"]),
                                            ptr(given["dw_n"]), codes[weights], 0, ptr(ws), need if sums else 0, stream())
    assert status == 0
    expect = R.norm_grad(dy, dn, o, y, w_o, gate, 0.75, w_n, 1e-6)
    for name, v in out.items():
        if name in wanted:
            R.within(v, expect[name][0], R.stored(*expect[name], v.dtype), name)
        else:
            assert (v == 9).all()
    assert ws is None or (ws[need:] == 255).all()


@pytest.mark.parametrize("act,dtype,grad", [("none", BF, F4), ("swiglu", BF, BF), ("gelu", FP, F4)], ids=lambda v: v if isinstance(v, str) else str(v)[6:])
@pytest.mark.parametrize("shape", ["few", "small", "odd", "wide", "none"])
def test_linear_from_python(lib, shape, act, dtype, grad):
    import grouped_int4_dequant_amd as m
    T, N, K = SHAPES[shape]
    g = torch.Generator().manual_seed(9)
    cols = N // 2 if act in R.GATED else N
    dy, x, W, pre = rnd(g, T, cols, dtype=dtype), rnd(g, T, K, dtype=dtype), rnd(g, N, K, dtype=dtype, scale=K ** -0.5), rnd(g, T, N, dtype=dtype)
    want = [(v, R.stored(v, s, t)) for (v, s), t in zip(R.linear_grad(dy, x, W, pre, act, dtype), (dtype, grad, grad))]
    kw = dict(pre=pre, act=act, grad_dtype=grad)
    db = torch.full((N,), 2.0, device="cuda")
    for got, formed in ((m.linear_backward(dy, x, W, dW=False, **kw), (0,)), (m.linear_backward(dy, None, W, dW=False, bias_grad=True, **kw), (0, 2)),
                        (m.linear_backward(dy, x, W, dx=False, **kw), (1,)), (m.linear_backward(dy, x, None, dx=False, bias_grad=True, **kw), (1, 2)),
                        (m.linear_backward(dy, None, W, dx=False, dW=False, bias_grad=True, **kw), (2,))):
        for i, (v, (value, bound), name) in enumerate(zip(got, want, ("dx", "dW", "db"))):
            if i in formed:
                R.within(v, value, bound, name)
            else:
                assert v is None
    got = m.linear_backward(dy, None, W, pre=pre, act=act, dx=False, dW=False, db=db, accumulate=True)
    assert got[2] is db and got[:2] == (None, None)
    value, slack = R.linear_grad(dy, x, W, pre, act, dtype)[2]
    R.within(db, value + 2.0, R.stored(value + 2.0, slack, F4), "db added")


@pytest.mark.parametrize("T,d,gates", [(60, 520, 1), (60, 77, 5), (30, 4104, 2)])
def test_norm_from_python(lib, T, d, gates):
    import grouped_int4_dequant_amd as m
    g = torch.Generator().manual_seed(10)
    o, dn, y, dy = rnd(g, T, d), rnd(g, T, d), rnd(g, T, d), rnd(g, T, d)
    w_o, w_n, gate = (rnd(g, *s, scale=0.3, shift=1.0) for s in ((d,), (d,), (gates, d)))
    expect = R.norm_grad(dy, dn, o, y, w_o, gate, 0.75, w_n, 1e-6)
    for wanted in [(n,) for n in NORM] + [("dx", "d_o"), ("dgate", "dw_n")]:
        got = m.residual_norm_backward(dy, dn, o, y, w_o=w_o, gate=gate, scale=0.75, w_n=w_n, grad_dtype=F4, **{n: False for n in NORM if n not in wanted})
        for name, v in zip(NORM, got):
            if name in wanted:
                R.within(v, expect[name][0], R.stored(*expect[name], v.dtype), name)
            else:
                assert v is None
