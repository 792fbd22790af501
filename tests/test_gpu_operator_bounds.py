"""Bounds of the grouped products that a result of fewer bits cannot keep: a weight
gradient's by its own group's rows, gradients against differences along the gradient,
and the few-row form's rounding. The first two are shown to reject such results on the CPU."""
import pytest
import torch

import grouped_reference as R
from test_gpu_grouped import BF, CASES, F4, FP, IDS, LAYOUTS, bounds, gen, moe, problem, rnd  # noqa: F401


def rows_of(offsets):
    o = offsets.cpu().long()
    return (o[1:] - o[:-1]).to(R.F8)[:, None, None]


def wgrad_bound(value, mag, offsets, out, start=None):
    """An element sums the rows of its own group: so many roundings and the joins."""
    slack = R.sums(rows_of(offsets), mag)
    return R.stored(value, slack if start is None else slack + 2 * R.U * start.abs(), out)


def test_weight_gradient_bound_rejects_fewer_bits():
    """Every layout's fp32 bound fails a value rounded to bf16 somewhere in every group of rows."""
    g = gen(2)
    for layout, (counts, tail) in LAYOUTS.items():
        o = torch.tensor([0, *counts]).cumsum(0).to(torch.int32)
        P = int(o[-1]) + tail
        A, dC = (torch.randn(P, w, generator=g).to(BF) for w in (24, 40))
        value, mag = R.grouped_wgrad(dC, A, o, None)
        over = (value.to(BF).to(R.F8) - value).abs() > wgrad_bound(value, mag, o, F4)
        used = torch.tensor(counts) > 1  # (one product alone may be a bf16 value)
        assert over.flatten(1).any(1)[used].all(), layout


@pytest.mark.gpu
@pytest.mark.parametrize("layout,size,dtype,out", CASES, ids=IDS)
def test_weight_gradient(moe, layout, size, dtype, out):  # noqa: F811
    offsets, P, A, a_row, _, dC = problem(layout, size, dtype)
    value, mag = R.grouped_wgrad(dC, A, offsets, a_row)
    D = moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out_dtype=out)
    R.within(D, value, wgrad_bound(value, mag, offsets, out), "dW")
    if out == F4:
        D = rnd(gen(9), *value.shape, dtype=F4)
        start = R.d(D)
        moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out=D, accumulate=True)
        R.within(D, value + start, wgrad_bound(value + start, mag, offsets, out, start), "dW added")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("P,N,K", [(5, 64, 64), (300, 40, 72), (300, 33, 70), (1200, 1024, 512)])
def test_weight_gradient_with_masked_rows(moe, dtype, P, N, K):  # noqa: F811
    g, G = gen(5), 70
    offsets = torch.linspace(0, P, G + 1).to(torch.int32).cuda()
    A, dC = rnd(g, 20, K, dtype=dtype), rnd(g, P, N, dtype=dtype)
    a_row = torch.randint(-3, 24, (P,), generator=g, dtype=torch.int32).cuda()
    value, mag = R.grouped_wgrad(dC, A, offsets, a_row)
    R.within(moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out_dtype=F4), value, wgrad_bound(value, mag, offsets, F4), "dW")


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,counts", [(1024, 2048, [300, 0, 41, 700]), (2048, 512, [64] * 16), (1024, 2048, [1] * 8 + [0] * 248)])
def test_weight_gradient_at_layer_sizes(moe, N, K, counts):  # noqa: F811
    offsets, P = bounds(counts)
    g = gen(6)
    A, dC = rnd(g, P, K), rnd(g, P, N)
    value, mag = R.grouped_wgrad(dC[:, ::17].contiguous(), A[:, ::33].contiguous(), offsets, None)
    D = moe.grouped_gemm_wgrad(dC, A, offsets, out_dtype=F4)
    R.within(D[:, ::17, ::33], value, wgrad_bound(value, mag, offsets, F4), "dW")


def along(t, gradient):
    """An argument of t's size and type in the direction of its 64-bit gradient, so that the
    change of the sum adds up instead of cancelling out."""
    return (gradient * float(R.d(t).norm() / gradient.norm())).to(t.dtype).to(t.device)


def differences(layout):
    offsets, P, A, a_row, W, dC = problem(layout, "mid", BF) if torch.cuda.is_available() else cpu_problem(layout)
    value, mag, used = R.grouped(A, W, offsets, a_row, P)
    gW, mW = R.grouped_wgrad(dC, A, offsets, a_row)
    rows, mr, _ = R.grouped_dgrad(dC, W, offsets)
    at = a_row.cpu().long()
    ok = used & (at >= 0) & (at < A.shape[0])
    gA, mA = (torch.zeros(A.shape, dtype=R.F8).index_add(0, at[ok], t[ok]) for t in (rows, R.sums(W.shape[1], mr)))
    W2, A2 = along(W, gW), along(A, gA)
    G = R.d(dC).abs()
    out = []
    for a, w, grad, slack in ((A, W2, gW, R.sums(rows_of(offsets), mW)), (A2, W, gA, mA)):
        change = R.d(w) - R.d(W) if w is W2 else R.d(a) - R.d(A)
        both = mag + R.grouped(a, w, offsets, a_row, P)[1]
        allowed = float((R.sums(W.shape[2], both)[used] * G[used]).sum()) + float((slack * change.abs()).sum()) + R.U * float((grad * change).abs().sum())
        out.append((a, w, change, float((grad * change).sum()), allowed))
    return offsets, P, A, a_row, W, dC, used, out


def cpu_problem(layout):
    counts, tail = LAYOUTS[layout]
    N, K = 264, 200
    o = torch.tensor([0, *counts]).cumsum(0).to(torch.int32)
    P, g = int(o[-1]) + tail, gen(1)
    rows = max(1, P // 3)
    A = torch.randn(rows, K, generator=g).to(BF)
    a_row = torch.randint(-1, rows + 1, (P,), generator=g, dtype=torch.int32)
    return o, P, A, a_row, (torch.randn(len(counts), N, K, generator=g) * K ** -0.5).to(BF), torch.randn(P, N, generator=g).to(BF)


@pytest.mark.parametrize("layout", ["edges", "many", "tail"])
def test_differences_are_large_beside_their_slack(layout):
    """So that a gradient that is lost, halved or of the wrong sign cannot pass."""
    for *_, expected, allowed in differences(layout)[-1]:
        assert expected > 20 * allowed


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["edges", "many", "tail"])
def test_gradients_against_differences(moe, layout):  # noqa: F811
    """<C, G> changes by an argument's gradient times its change, along the gradient."""
    offsets, P, A, a_row, W, dC, used, ((_, W2, changeW, eW, sW), (A2, _, changeA, eA, sA)) = differences(layout)
    G = R.d(dC)
    loss = lambda a, w: float((R.d(moe.grouped_gemm(a, w, offsets, a_row=a_row, out_dtype=F4))[used] * G[used]).sum())  # noqa: E731
    dW = R.d(moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out_dtype=F4))
    assert abs(loss(A, W2) - loss(A, W) - float((dW * changeW).sum())) <= sW < eW / 20
    rows = R.d(moe.grouped_gemm_dgrad(dC, W, offsets, out_dtype=F4))
    at = a_row.cpu().long()
    ok = used & (at >= 0) & (at < A.shape[0])
    dA = torch.zeros(A.shape, dtype=R.F8).index_add(0, at[ok], rows[ok])
    assert abs(loss(A2, W) - loss(A, W) - float((dA * changeA).sum())) <= sA < eA / 20


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,top,G,N,K", [(1, 8, 256, 1024, 2048), (1, 8, 256, 2048, 512), (4, 8, 256, 512, 2048), (7, 2, 16, 136, 264)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_few_rows_round_once_and_repeat(moe, tokens, top, G, N, K, dtype):  # noqa: F811
    """Few rows of many groups: the fp32 result keeps the bound of an fp32 sum, the
    16-bit one is its rounding, and repeated calls agree bit for bit."""
    g = gen(tokens + N)
    ids = torch.stack([torch.randperm(G, generator=g)[:top] for _ in range(tokens)]).flatten()
    order = torch.sort(ids, stable=True).indices
    a_row = (order // top).to(torch.int32).cuda()
    offsets = torch.zeros(G + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(ids, minlength=G).cumsum(0)
    offsets, P = offsets.cuda(), tokens * top
    x, W = rnd(g, tokens, K, dtype=dtype), rnd(g, G, N, K, dtype=dtype, scale=K ** -0.5)
    C = moe.grouped_gemm(x, W, offsets, a_row=a_row, out_dtype=F4)
    value, mag, _ = R.grouped(x, W, offsets, a_row, P)
    R.within(C, value, R.stored(value, R.sums(K, mag), F4), "C")
    dC = rnd(g, P, N, dtype=dtype)
    D = moe.grouped_gemm_dgrad(dC, W, offsets, out_dtype=F4)
    value, mag, _ = R.grouped_dgrad(dC, W, offsets)
    R.within(D, value, R.stored(value, R.sums(N, mag), F4), "dA")
    for _ in range(10):
        assert torch.equal(moe.grouped_gemm(x, W, offsets, a_row=a_row), C.to(dtype))
        assert torch.equal(moe.grouped_gemm(x, W, offsets, a_row=a_row, out_dtype=F4), C)
        assert torch.equal(moe.grouped_gemm_dgrad(dC, W, offsets), D.to(dtype))
