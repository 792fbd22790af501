"""Adapters whose middle products h = scale A x and g = scale B^T dy spread over many
binary orders, are very large or very small: both stay fp32, so every result keeps to the bound
of a sum of exact products in fp32, whichever ranks it takes."""
import pytest
import torch

import grouped_reference as R
from test_gpu_grouped import BF, F4, FP, gen, moe, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

#       T, n, r: one, two, four and eight rank tiles, 32 rows a workgroup (8 to 24 rows an adapter) and 16
FORMS = [(40, 2, 5), (60, 4, 16), (40, 2, 17), (60, 4, 32), (40, 2, 64), (62, 5, 50), (40, 2, 128),
         (50, 1, 5), (30, 6, 16), (50, 1, 32), (30, 6, 17), (50, 1, 64), (30, 6, 40)]


def spread(r, orders):
    """Powers of two over `orders` binary orders around 1, in no order of size."""
    at = torch.linspace(-orders / 2, orders / 2, r) if r > 1 else torch.zeros(1)
    return 2.0 ** at[torch.randperm(r, generator=gen(r))].round()


def case(T, n, r, dtype):
    g = gen(T + r)
    ids = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda()
    return g, ids, (torch.rand(n, generator=g) + 0.5).cuda()


def picks(n, width, r):
    """[n][width][r] of ones that lets output `c` take rank c % r alone."""
    return torch.nn.functional.one_hot(torch.arange(width) % r, r).float().expand(n, width, r)


@pytest.mark.parametrize("T,n,r", FORMS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("orders", [6, 16, 30])
def test_ranks_of_unlike_size(moe, T, n, r, dtype, orders):  # noqa: F811
    """Most outputs take one rank, some of them a rank whose value is 2^-30 of the row's largest."""
    K, N = 72, 3 * r + 5
    g, ids, scale = case(T, n, r, dtype)
    plan, x = moe.adapter_plan(ids, n), rnd(g, T, K, dtype=dtype)
    A = (torch.randn(n, r, K, generator=g) * 0.25 * spread(r, orders)[:, None]).to(dtype).cuda()
    B = picks(n, N, r) * torch.randn(n, N, r, generator=g)
    B[:, ::7] = torch.randn(n, len(range(0, N, 7)), r, generator=g)
    B = B.to(dtype).cuda()
    y = moe.adapter_forward(x, A, B, scale, plan, out_dtype=F4)
    value, slack, _, _ = R.adapter(x, A, B, scale, ids, None)
    R.within(y, value, R.stored(value, slack, F4), "y")
    # the gradient's g is h's mirror image: A and B in each other's place
    A, B, dy = B.transpose(1, 2).contiguous(), A.transpose(1, 2).contiguous(), x
    x = rnd(g, T, N, dtype=dtype)
    dx = torch.empty(T, N, dtype=F4, device="cuda")
    grads = moe.adapter_backward(dy, x, A, B, scale, plan, dx=dx, grad_dtype=F4)
    for name, t, (value, slack) in zip(("dx", "dA", "dB"), grads, R.adapter_grad(dy, x, A, B, scale, ids, None)):
        R.within(t, value, R.stored(value, slack, F4), name)


@pytest.mark.parametrize("T,n,r", FORMS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_middle_products_keep_their_bits(moe, T, n, r, dtype):  # noqa: F811
    """With one input column and outputs that pick one rank each, y is h itself, the
    fp32 product of scale and the exact A x. fp16: equal. bf16: the three parts
    of h add up in two or three matrix instructions, each of which may round (2^-24) or
    cut off (2^-23) once: 3 * 2^-23."""
    g, ids, scale = case(T, n, r, dtype)
    N = 2 * r + 3
    plan, x = moe.adapter_plan(ids, n), rnd(g, T, 1, dtype=dtype)
    A = (torch.randn(n, r, 1, generator=g) * spread(r, 20)[:, None]).to(dtype).cuda()
    B = picks(n, N, r).contiguous().to(dtype).cuda()
    has, e = ids >= 0, ids.clamp(min=0).long()
    h = scale[e][:, None] * (A.float()[e, :, 0] * x.float())  # the product is exact in fp32, times scale rounds once
    want = torch.where(has[:, None], h[:, torch.arange(N, device="cuda") % r], 0.0)
    near = 0.0 if dtype == FP else 3 * 2.0 ** -23
    y = moe.adapter_forward(x, A, B, scale, plan, out_dtype=F4)
    assert ((y - want).abs() <= near * want.abs()).all()
    dx = torch.empty(T, N, dtype=F4, device="cuda")
    moe.adapter_backward(x, rnd(g, T, N, dtype=dtype), B.transpose(1, 2).contiguous(), A.transpose(1, 2).contiguous(), scale, plan, dx=dx)
    assert ((dx - want).abs() <= near * want.abs()).all()


@pytest.mark.parametrize("T,n,r", FORMS)
@pytest.mark.parametrize("dtype,orders", [(BF, 115), (FP, 115), (BF, -90), (FP, -90)])
def test_large_and_small_middle_products(moe, T, n, r, dtype, orders):  # noqa: F811
    """h and g of about 2^115 and 2^-90, within fp32's range and so are the results."""
    K, N = 72, 40
    g, ids, scale = case(T, n, r, dtype)
    scale *= 2.0 ** orders
    plan, x, A = moe.adapter_plan(ids, n), rnd(g, T, K, dtype=dtype), rnd(g, n, r, K, dtype=dtype, scale=K ** -0.5)
    B = rnd(g, n, N, r, dtype=dtype, scale=r ** -0.5)
    y = moe.adapter_forward(x, A, B, scale, plan, out_dtype=F4)
    value, slack, _, _ = R.adapter(x, A, B, scale, ids, None)
    R.within(y, value, R.stored(value, slack, F4), "y")
    dx, dy = torch.empty(T, K, dtype=F4, device="cuda"), rnd(g, T, N, dtype=dtype)
    moe.adapter_backward(dy, x, A, B, scale, plan, dx=dx)
    value, slack = R.adapter_grad(dy, x, A, B, scale, ids, None)[0]
    R.within(dx, value, R.stored(value, slack, F4), "dx")


@pytest.mark.parametrize("T,n,r", [f for f in FORMS if f[2] > 4])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_large_values_beside_an_infinity(moe, T, n, r, dtype):  # noqa: F811
    """A row with an infinite rank: its other ranks are large, finite and of the other
    sign in the sum, which stays the formula's infinity."""
    g, ids, _ = case(T, n, r, dtype)
    plan, x, N = moe.adapter_plan(ids, n), torch.ones(T, 2, dtype=dtype, device="cuda"), 24
    A = torch.zeros(n, r, 2)
    A[:, :, 0], A[:, 2, 1] = 60000.0, float("inf")
    B = -torch.ones(n, N, r)
    B[:, :, 2] = 1.0
    A, B, scale = A.to(dtype).cuda(), B.to(dtype).cuda(), torch.full((n,), 3.0, device="cuda")
    has = ids >= 0
    y = moe.adapter_forward(x, A, B, scale, plan, out_dtype=F4)
    assert (y[has] == float("inf")).all() and (y[~has] == 0).all()
    dx = torch.empty(T, N, dtype=F4, device="cuda")
    moe.adapter_backward(x, torch.ones(T, N, dtype=dtype, device="cuda"), B.transpose(1, 2).contiguous(), A.transpose(1, 2).contiguous(), scale, plan, dx=dx)
    assert (dx[has] == float("inf")).all() and (dx[~has] == 0).all()
