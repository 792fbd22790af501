"""Infinite and NaN adapters: every result is what the formula gives for its row and column,
and no other row, column or adapter is touched."""
import pytest
import torch

import grouped_reference as R
from test_gpu_adapter_range import FORMS
from test_gpu_grouped import BF, F4, FP, gen, moe, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def middle(x, A, scale, ids):
    """scale A x of every row in 64 bits (rows without an adapter: zeros)."""
    e = ids.cpu().long().clamp(min=0)
    return R.d(scale)[e][:, None] * (R.d(A)[e] * R.d(x)[:, None, :]).sum(2)


def same(got, want, finite_bound, what):
    got = R.d(got)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN"
    assert torch.equal(got == float("inf"), want == float("inf")) and torch.equal(got == -float("inf"), want == -float("inf")), f"{what}: infinities"
    ok = torch.isfinite(want)
    assert ((got - want).abs()[ok] <= finite_bound[ok]).all(), what


def outer(h, M, ids):
    """sum_j h[t][j] M[a][c][j] with the formula's infinities and NaN."""
    e = ids.cpu().long()
    out = (h[:, None, :] * R.d(M)[e.clamp(min=0)]).sum(2)
    return torch.where((e >= 0)[:, None], out, 0.0)


@pytest.mark.parametrize("T,n,r", [(40, 2, 1), *FORMS])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F4), (FP, FP), (FP, F4)])
def test_weights_that_are_not_finite(moe, T, n, r, dtype, out):  # noqa: F811
    """Infinite and NaN elements of B (forward) and of A (dx). x, dy and the other
    factor are small whole numbers and powers of two, so that many parts
    of the middle products are zero, and everything finite is exact."""
    g, K, N = gen(7 * T + r), 24, 40
    ids = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda()
    plan = moe.adapter_plan(ids, n)
    whole = lambda *s: (torch.randint(1, 4, s, generator=g) * (2 * torch.randint(0, 2, s, generator=g) - 1)).to(dtype).cuda()  # noqa: E731
    x, A, B, scale = whole(T, K), whole(n, r, K), whole(n, N, r), torch.full((n,), 0.5, device="cuda")
    for c, v in ((3, float("inf")), (11, -float("inf")), (30, float("nan")), (38, float("inf"))):
        B[n - 1, c, c % r] = v
    B[n - 1, 38, (38 + 1) % r] = float("inf")  # two in one sum
    want = outer(middle(x, A, scale, ids), B, ids)
    zero = torch.full_like(want, 0.0) + torch.finfo(out).eps / 2 * want.abs().nan_to_num(0.0, 0.0, 0.0)
    same(moe.adapter_forward(x, A, B, scale, plan, out_dtype=out), want, zero, "y")
    # the mirror image: A as B, dy as x
    x2 = whole(T, N)
    dx = torch.empty(T, N, dtype=out, device="cuda")
    moe.adapter_backward(x, x2, B.transpose(1, 2).contiguous(), A.transpose(1, 2).contiguous(), scale, plan, dx=dx)
    same(dx, want, zero, "dx")


@pytest.mark.parametrize("T,n,r", FORMS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinite_weight_meets_infinite_row(moe, T, n, r, dtype):  # noqa: F811
    """Both factors infinite in the same rank: infinity, of the product's sign."""
    g, K, N = gen(T + r), 24, 40
    ids = torch.randint(0, n, (T,), generator=g, dtype=torch.int32).cuda()
    plan = moe.adapter_plan(ids, n)
    x, A, B = (torch.ones(*s, dtype=dtype, device="cuda") for s in ((T, K), (n, r, K), (n, N, r)))
    x[T // 2, 5] = -float("inf")
    B[:, 9, 2], B[:, 10, 2] = float("inf"), -float("inf")
    want = outer(middle(x, A, torch.ones(n), ids), B, ids)
    bound = torch.zeros_like(want)
    for t in (moe.adapter_forward(x, A, B, None, plan, out_dtype=F4),):
        same(t, want, bound, "y")
    dx = torch.empty(T, N, dtype=F4, device="cuda")
    moe.adapter_backward(x, torch.ones(T, N, dtype=dtype, device="cuda"), B.transpose(1, 2).contiguous(), A.transpose(1, 2).contiguous(), None, plan, dx=dx)
    same(dx, want, bound, "dx")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("r", [5, 16, 40, 128])
def test_ordinary_values_beside_an_infinite_weight(moe, dtype, r):  # noqa: F811
    """Random rows: one infinite element of B or of A gives its column the sign of the middle product."""
    T, n, K, N = 70, 2, 72, 40
    g = gen(r)
    ids = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32).cuda()
    plan, scale = moe.adapter_plan(ids, n), (torch.rand(n, generator=g) + 0.5).cuda()
    x, A, B = rnd(g, T, K, dtype=dtype), rnd(g, n, r, K, dtype=dtype, scale=K ** -0.5), rnd(g, n, N, r, dtype=dtype, scale=r ** -0.5)
    dy = rnd(g, T, N, dtype=dtype)
    clean, dx0 = moe.adapter_forward(x, A, B, scale, plan), moe.adapter_backward(dy, x, A, B, scale, plan)[0]
    B2, A2 = B.clone(), A.clone()
    B2[1, 7, r - 1], A2[1, r // 2, 9] = float("inf"), -float("inf")
    y = moe.adapter_forward(x, A, B2, scale, plan)
    hit = torch.zeros(T, N, dtype=torch.bool)
    hit[ids.cpu() == 1, 7] = True
    h = middle(x, A, scale, ids)[:, r - 1]
    assert torch.equal(R.d(y)[hit], (h.sign() * float("inf"))[hit.any(1)]) and torch.equal(y.cpu()[~hit], clean.cpu()[~hit])
    dx = moe.adapter_backward(dy, x, A2, B, scale, plan)[0]
    hit = torch.zeros(T, K, dtype=torch.bool)
    hit[ids.cpu() == 1, 9] = True
    gm = middle(dy, B.transpose(1, 2), scale, ids)[:, r // 2]
    assert torch.equal(R.d(dx)[hit], (gm.sign() * -float("inf"))[hit.any(1)]) and torch.equal(dx.cpu()[~hit], dx0.cpu()[~hit])
