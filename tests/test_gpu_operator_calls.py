"""Calls of the 16-bit operators that leave results out (NULL in the C interface) or
run on another stream give the full call's results bit for bit."""
import pytest
import torch

from test_gpu_adapters import problem
from test_gpu_grouped import BF, F4, FP, gen, moe, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

#        T, n, K, N, r: rows shared by the waves or not, 16 and 32 rows a workgroup, several column slices, odd sizes
FORMS = [(40, 2, 1100, 1100, 16), (300, 2, 72, 136, 16), (60, 4, 136, 200, 40), (61, 4, 77, 131, 30), (90, 64, 1100, 40, 5), (290, 1, 64, 131, 128)]


def ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("T,n,K,N,r", FORMS)
@pytest.mark.parametrize("dtype,grads", [(BF, F4), (FP, FP)])
def test_parts_of_the_adapter_gradients(moe, T, n, K, N, r, dtype, grads):  # noqa: F811
    g, ids, x, dy, A, B, scale = problem(T, n, K, N, r, dtype)
    rows, offsets = plan = moe.adapter_plan(ids, n)
    base = rnd(g, T, K, dtype=grads)
    full = moe.adapter_backward(dy, x, A, B, scale, plan, dx_base=base, grad_dtype=grads)
    code = {BF: 0, FP: 1, F4: 2}
    need = moe.adapter_backward_workspace_bytes(T, r)
    for want in ("x", "A", "B", "xA", "xB", "AB"):
        out = [torch.full_like(t, 7.0) if name in want else None for name, t in zip("xAB", full)]
        ws = None if want == "x" else torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN in every word
        status = moe.load().moe_adapter_backward(
            code[dtype], ptr(dy), N, ptr(x), K, T, K, N, r, n, ptr(A), ptr(B), ptr(scale), ptr(rows), ptr(offsets), ptr(base) if "x" in want else None, K,
            ptr(out[0]), code[grads], K, ptr(out[1]), ptr(out[2]), code[grads], 0, ptr(ws), 0 if ws is None else need, torch.cuda.current_stream().cuda_stream)
        assert status == 0, want
        for name, got, all_of_it in zip("xAB", out, full):
            assert got is None or torch.equal(got, all_of_it), (want, name)


@pytest.mark.parametrize("T,k,dim", [(33, 4, 520), (5, 3, 77)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_parts_of_the_combine_gradient(moe, T, k, dim, dtype):  # noqa: F811
    g = gen(T)
    P = T * k
    o, dy, w = rnd(g, P, dim, dtype=dtype), rnd(g, T, dim, dtype=dtype), torch.rand(T, k, generator=g).cuda()
    pos = torch.randperm(P, generator=g).reshape(T, k).to(torch.int32).cuda()
    d_o, dw = moe.combine_backward(dy, o, pos, w)
    code, s = {BF: 0, FP: 1}[dtype], torch.cuda.current_stream().cuda_stream
    f = moe.load().moe_combine_backward
    rows, gates = torch.full_like(d_o, 7.0), torch.full_like(dw, 7.0)
    assert f(code, ptr(dy), dim, None, 0, P, ptr(pos), ptr(w), T, k, dim, ptr(rows), dim, None, s) == 0
    assert f(code, ptr(dy), dim, ptr(o), dim, P, ptr(pos), None, T, k, dim, None, 0, ptr(gates), s) == 0
    assert torch.equal(rows, d_o) and torch.equal(gates, dw)


@pytest.mark.parametrize("T,n,K,N,r", FORMS[:3])
def test_on_another_stream(moe, T, n, K, N, r):  # noqa: F811
    """Every call on a side stream whose inputs were made there, while the current stream works."""
    _, ids, x, dy, A, B, scale = problem(T, n, K, N, r, BF)
    k = 2
    pos = torch.randperm(T * k, generator=gen(3)).reshape(T, k).to(torch.int32).cuda()
    gate, o = torch.rand(T, k, generator=gen(4)).cuda(), rnd(gen(5), T * k, K)

    def step(x, stream):
        plan = moe.adapter_plan(ids, n, stream=stream)
        return [*plan, moe.adapter_forward(x, A, B, scale, plan, stream=stream), *moe.adapter_backward(dy, x, A, B, scale, plan, stream=stream),
                moe.combine(o, pos, weights=gate, add=x, stream=stream), *moe.combine_backward(x, o, pos, gate, stream=stream)]

    want = step(x * 2, None)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(1024, 1024, device="cuda")
    for _ in range(3):
        with torch.cuda.stream(side):
            doubled = x * 2
        for _ in range(8):
            busy = busy @ busy * 1e-3
        got = step(doubled, side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
