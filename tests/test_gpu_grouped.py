"""Grouped 16-bit products, their gradients and the combine on the GPU against
plain 64-bit forms, element by element."""
import pytest
import torch

import grouped_reference as R

pytestmark = pytest.mark.gpu

BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    m.load()
    return m


def rnd(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bounds(counts, tail=0):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.tensor(counts).cumsum(0)
    return o.cuda(), int(o[-1]) + tail


def strided(t, extra, fill):
    """The same values in a matrix of wider rows (extra columns hold `fill`)."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide, wide[:, :t.shape[1]]


LAYOUTS = {
    "one_row": ([1], 0), "one_of_many": ([0, 0, 1, 0], 0), "edges": ([0, 15, 16, 17, 0, 127, 128, 129, 0], 0),
    "all_in_one": ([0, 700, 0], 0), "tail": ([33, 0, 5], 9), "single_rows": ([1] * 70, 0), "all_empty": ([0, 0, 0], 4),
    "many": ([(7 * i) % 23 for i in range(130)], 0), "wide": ([(37 * i) % 301 for i in range(140)], 3), "wide_long": ([700, 0, 513, 1030] * 9, 0), "short_long": ([3, 513, 64, 2, 0, 255], 0),
}
#          N, K
SIZES = {"wide": (1032, 1160), "tile": (128, 64), "small": (8, 8), "mid": (264, 200), "odd": (77, 131), "one": (1, 1), "odd_n": (65, 128), "odd_k": (128, 67),
         "deep": (40, 1544)}
CASES = [(l, s, t, o) for l in LAYOUTS for s, t, o in (("mid", BF, BF), ("odd", FP, F4))]
CASES += [(l, s, t, o) for s in SIZES for l, t, o in (("edges", FP, FP), ("short_long", BF, F4))]
CASES += [("wide_long", "wide", BF, BF), ("wide_long", "wide", FP, F4), ("wide", "wide", BF, F4), ("single_rows", "wide", FP, FP), ("one_row", "wide", BF, F4)]
IDS = [f"{l}-{s}-{str(t)[6:]}-{str(o)[6:]}" for l, s, t, o in CASES]


def problem(layout, size, dtype, seed=1):
    counts, tail = LAYOUTS[layout]
    N, K = SIZES[size]
    offsets, P = bounds(counts, tail)
    g = gen(seed)
    rows = max(1, P // 3)
    A = rnd(g, rows, K, dtype=dtype)
    a_row = torch.randint(-1, rows + 1, (P,), generator=g, dtype=torch.int32).cuda()  # -1 and `rows`: masked
    W = rnd(g, len(counts), N, K, dtype=dtype, scale=K ** -0.5)
    dC = rnd(g, P, N, dtype=dtype)
    return offsets, P, A, a_row, W, dC


def check_rows(got, value, mag, used, terms, before, what):
    R.within(got[used.to(got.device)], value[used], R.stored(value[used], R.sums(terms, mag[used]), got.dtype), what)
    idle = ~used.to(got.device)
    assert torch.equal(got[idle], before[idle]), f"{what}: rows of no group were written"


@pytest.mark.parametrize("layout,size,dtype,out", CASES, ids=IDS)
def test_forward(moe, layout, size, dtype, out):
    offsets, P, A, a_row, W, _ = problem(layout, size, dtype)
    N, K = SIZES[size]
    wide, C = strided(torch.full((P, N), 7.0, dtype=out, device="cuda"), 4, 3.0)
    before = C.clone()
    assert moe.grouped_gemm(A, W, offsets, a_row=a_row, out=C) is C
    value, mag, used = R.grouped(A, W, offsets, a_row, P)
    check_rows(C, value, mag, used, K, before, "gathered")
    assert (wide[:, N:] == 3.0).all()
    if P <= A.shape[0] or P == 0:
        return
    A = rnd(gen(2), P, K + 8, dtype=dtype)[:, :K]
    C = torch.full((P, N), 7.0, dtype=out, device="cuda")
    moe.grouped_gemm(A, W, offsets, out=C)
    value, mag, used = R.grouped(A, W, offsets, None, P)
    check_rows(C, value, mag, used, K, torch.full_like(C, 7.0), "strided rows")


@pytest.mark.parametrize("layout,size,dtype,out", CASES, ids=IDS)
def test_input_gradient(moe, layout, size, dtype, out):
    offsets, P, _, _, W, dC = problem(layout, size, dtype)
    N, K = SIZES[size]
    wide, D = strided(torch.full((P, K), 7.0, dtype=out, device="cuda"), 4, 3.0)
    before = D.clone()
    moe.grouped_gemm_dgrad(strided(dC, 8, float("nan"))[1], W, offsets, out=D)
    value, mag, used = R.grouped_dgrad(dC, W, offsets)
    check_rows(D, value, mag, used, N, before, "dA")
    assert (wide[:, K:] == 3.0).all()


@pytest.mark.parametrize("layout,size,dtype,out", CASES, ids=IDS)
def test_weight_gradient(moe, layout, size, dtype, out):
    offsets, P, A, a_row, _, dC = problem(layout, size, dtype)
    value, mag = R.grouped_wgrad(dC, A, offsets, a_row)
    D = moe.grouped_gemm_wgrad(strided(dC, 8, float("nan"))[1], strided(A, 8, float("nan"))[1], offsets, a_row=a_row, out_dtype=out)
    bound = R.stored(value, R.sums(P, mag), out)
    R.within(D, value, bound, "dW")
    assert (D[[e for e, a, b in R.spans(offsets) if a == b]] == 0).all()
    if out == F4:
        start = rnd(gen(9), *value.shape, dtype=F4)
        D = start.clone()
        moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out=D, accumulate=True)
        total = value + R.d(start)
        R.within(D, total, R.stored(total, R.sums(P, mag) + 2 * R.U * R.d(start).abs(), out), "dW added")
        empty = [e for e, a, b in R.spans(offsets) if a == b]
        assert torch.equal(D[empty], start[empty])


def test_no_rows(moe):
    W, offsets = rnd(gen(1), 3, 8, 16), torch.zeros(4, dtype=torch.int32, device="cuda")
    A = torch.empty(0, 16, dtype=BF, device="cuda")
    assert moe.grouped_gemm(A, W, offsets).shape == (0, 8)
    assert moe.grouped_gemm_dgrad(torch.empty(0, 8, dtype=BF, device="cuda"), W, offsets).shape == (0, 16)
    D = moe.grouped_gemm_wgrad(torch.empty(0, 8, dtype=BF, device="cuda"), A, offsets)
    assert D.shape == (3, 8, 16) and (D == 0).all()


@pytest.mark.parametrize("P,N,K", [(5, 64, 64), (300, 40, 72), (300, 33, 70), (1200, 1024, 512)])
def test_no_row_of_the_input(moe, P, N, K):
    """An input without rows: every row is masked."""
    g, G = gen(16), 70
    offsets = torch.linspace(0, P, G + 1).to(torch.int32).cuda()
    A, W, dC = torch.empty(0, K, dtype=BF, device="cuda"), rnd(g, G, N, K), rnd(g, P, N)
    W[3], dC[2] = float("nan"), float("inf")
    a_row = torch.randint(-2, 3, (P,), generator=g, dtype=torch.int32).cuda()
    assert (moe.grouped_gemm(A, W, offsets, a_row=a_row) == 0).all()
    assert (moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row) == 0).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("K", [72, 75, 128])
def test_infinities_and_nan_stay_in_their_sums(moe, dtype, K):
    """A row, a weight row or a column that is not finite reaches the results
    whose sums it enters and no others: not other rows of the tile, other
    groups, the padding of the last step, or masked rows."""
    counts = [5, 0, 20, 3]
    offsets, P = bounds(counts)
    g, N = gen(3), 40
    A, W, dC = rnd(g, P, K, dtype=dtype), rnd(g, 4, N, K, dtype=dtype), rnd(g, P, N, dtype=dtype)
    clean = moe.grouped_gemm(A, W, offsets, out_dtype=F4)
    A2, W2 = A.clone(), W.clone()
    A2[7, 3], W2[2, 11] = float("nan"), float("inf")
    W2[1] = float("nan")  # the empty group's weights
    C = moe.grouped_gemm(A2, W2, offsets, out_dtype=F4)
    hit = torch.zeros(P, N, dtype=torch.bool, device="cuda")
    hit[7] = True
    hit[5:25, 11] = True
    assert torch.equal(C[~hit], clean[~hit]) and not torch.isfinite(C[hit]).any()
    D = moe.grouped_gemm_dgrad(dC, W2, offsets, out_dtype=F4)
    assert torch.equal(D[:5], moe.grouped_gemm_dgrad(dC, W, offsets, out_dtype=F4)[:5]) and torch.isfinite(D[25:]).all()
    dC2 = dC.clone()
    dC2[24, 0], A2 = float("nan"), A.clone()
    A2[4, 1] = float("inf")
    G0, G1 = (moe.grouped_gemm_wgrad(x, y, offsets, out_dtype=F4) for x, y in ((dC, A), (dC2, A2)))
    hit = torch.zeros(4, N, K, dtype=torch.bool, device="cuda")
    hit[2, 0], hit[0, :, 1] = True, True
    assert torch.equal(G0[~hit], G1[~hit]) and not torch.isfinite(G1[hit]).any()


@pytest.mark.parametrize("P,N,K", [(5, 64, 64), (300, 40, 72), (300, 33, 70), (1200, 1024, 512)])
def test_masked_rows_are_zeros(moe, P, N, K):
    """A masked row gives zeros whatever the weights hold, and no gradient."""
    g, G = gen(5), 70
    offsets = torch.linspace(0, P, G + 1).to(torch.int32).cuda()
    A, W, dC = rnd(g, 20, K), rnd(g, G, N, K, scale=0.1), rnd(g, P, N)
    a_row = torch.randint(0, 20, (P,), generator=g, dtype=torch.int32)
    a_row[::3], a_row[1::7] = -1, 20
    masked = ((a_row < 0) | (a_row >= 20)).cuda()
    a_row = a_row.cuda()
    value, mag, _ = R.grouped(A, W, offsets, a_row, P)
    C = moe.grouped_gemm(A, W, offsets, a_row=a_row)
    R.within(C, value, R.stored(value, R.sums(K, mag), BF), "C")
    W[:, 3] = float("inf")
    W[:, 5] = float("nan")
    assert (moe.grouped_gemm(A, W, offsets, a_row=a_row)[masked] == 0).all()
    kept = torch.where(masked[:, None], 0.0, dC.float()).to(BF)
    D = moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out_dtype=F4)
    value, mag = R.grouped_wgrad(kept, A, offsets, torch.where(masked, 0, a_row))
    R.within(D, value, R.stored(value, R.sums(P, mag), F4), "dW")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("P,N,K", [(300, 40, 72), (300, 33, 70), (1200, 1024, 512)])
def test_masked_rows_give_no_weight_gradient(moe, dtype, P, N, K):
    """dC's rows may hold anything where the row of A is masked."""
    g, G, rows = gen(15), 70, P - 30
    offsets = torch.linspace(0, P, G + 1).to(torch.int32).cuda()
    A, dC = rnd(g, rows, K, dtype=dtype), rnd(g, P, N, dtype=dtype)
    a_row = torch.randint(0, rows, (P,), generator=g, dtype=torch.int32)
    a_row[::3], a_row[1::7] = -1, rows
    masked = ((a_row < 0) | (a_row >= rows)).cuda()
    a_row = a_row.cuda()
    want = moe.grouped_gemm_wgrad(torch.where(masked[:, None], 0.0, dC.float()).to(dtype), A, offsets, a_row=a_row, out_dtype=F4)
    dC[masked] = float("nan")
    assert torch.equal(moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out_dtype=F4), want) and torch.isfinite(want).all()


@pytest.mark.parametrize("layout", ["edges", "many"])
def test_gradients_against_differences(moe, layout):
    """The product is linear in A and in W: the change of <C, G> under a change of
    one argument equals that argument's gradient times the change."""
    offsets, P, A, a_row, W, dC = problem(layout, "mid", BF)
    G = R.d(dC)
    used = R.grouped(A, W, offsets, a_row, P)[2]
    loss = lambda a, w: float((R.d(moe.grouped_gemm(a, w, offsets, a_row=a_row, out_dtype=F4))[used] * G[used]).sum())  # noqa: E731
    dW = R.d(moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, out_dtype=F4))
    W2 = rnd(gen(8), *W.shape)
    mag = R.grouped(A, W, offsets, a_row, P)[1] + R.grouped(A, W2, offsets, a_row, P)[1]
    slack = float((R.sums(W.shape[2], mag)[used] * G[used].abs()).sum()) + float((R.sums(P, R.grouped_wgrad(dC, A, offsets, a_row)[1]) * (R.d(W2) - R.d(W)).abs()).sum())
    assert abs(loss(A, W2) - loss(A, W) - float((dW * (R.d(W2) - R.d(W))).sum())) <= slack
    rows = moe.grouped_gemm_dgrad(dC, W, offsets, out_dtype=F4)
    at = a_row.cpu().long()
    ok = used & (at >= 0) & (at < A.shape[0])
    dA = torch.zeros(A.shape, dtype=R.F8).index_add(0, at[ok], R.d(rows)[ok])
    A2 = rnd(gen(9), *A.shape)
    mag = R.grouped(A, W, offsets, a_row, P)[1] + R.grouped(A2, W, offsets, a_row, P)[1]
    slack = float((R.sums(W.shape[2], mag)[used] * G[used].abs()).sum())
    diff = (R.d(A2) - R.d(A)).abs()
    slack += float((R.sums(W.shape[1], R.grouped_dgrad(dC, W, offsets)[1])[ok] * diff[at[ok]]).sum())
    assert abs(loss(A2, W) - loss(A, W) - float((dA * (R.d(A2) - R.d(A))).sum())) <= slack


def test_rows_past_32_bit_offsets(moe):
    """Rows that start more than 4 GiB and more than 2^32 elements apart."""
    step, K, N = 1_300_000_008, 64, 32
    store = torch.empty(3 * step + K, dtype=BF, device="cuda")
    A = store.as_strided((4, K), (step, 1))
    g = gen(4)
    A.copy_(rnd(g, 4, K))
    W, offsets = rnd(g, 2, N, K, scale=0.1), bounds([3, 1])[0]
    a_row = torch.tensor([3, 0, 2, 3], dtype=torch.int32, device="cuda")
    small = A.contiguous()
    assert torch.equal(moe.grouped_gemm(A, W, offsets, a_row=a_row), moe.grouped_gemm(small, W, offsets, a_row=a_row))
    dC = rnd(g, 4, N)
    assert torch.equal(moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row), moe.grouped_gemm_wgrad(dC, small, offsets, a_row=a_row))
    want = moe.grouped_gemm_dgrad(dC, W, offsets)
    moe.grouped_gemm_dgrad(dC, W, offsets, out=A)
    assert torch.equal(A, want)
    pos = torch.tensor([[3, 1], [2, 0]], dtype=torch.int32, device="cuda")
    assert torch.equal(moe.combine(A, pos), moe.combine(want, pos))


@pytest.mark.parametrize("N,K,counts", [(1024, 2048, [300, 0, 41, 700]), (2048, 512, [64] * 16), (1024, 2048, [1] * 8 + [0] * 248)])
def test_layer_sizes(moe, N, K, counts):
    """The layer's projections, checked at every 17th column and row sum of products."""
    offsets, P = bounds(counts)
    g = gen(6)
    A, W, dC = rnd(g, P, K), rnd(g, len(counts), N, K, scale=K ** -0.5), rnd(g, P, N)
    value, mag, _ = R.grouped(A, W[:, ::17].contiguous(), offsets, None, P)
    C = moe.grouped_gemm(A, W, offsets)
    R.within(C[:, ::17], value, R.stored(value, R.sums(K, mag), BF), "C")
    value, mag, _ = R.grouped_dgrad(dC, W[:, :, ::33].contiguous(), offsets)
    R.within(moe.grouped_gemm_dgrad(dC, W, offsets)[:, ::33], value, R.stored(value, R.sums(N, mag), BF), "dA")
    value, mag = R.grouped_wgrad(dC[:, ::17].contiguous(), A[:, ::33].contiguous(), offsets, None)
    D = moe.grouped_gemm_wgrad(dC, A, offsets, out_dtype=F4)
    R.within(D[:, ::17, ::33], value, R.stored(value, R.sums(P, mag), F4), "dW")


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("T,k,dim", [(1, 1, 8), (1, 8, 2048), (5, 3, 77), (64, 8, 264), (33, 11, 520), (130, 2, 1)])
@pytest.mark.parametrize("dtype,out,add", [(BF, BF, BF), (FP, F4, FP), (BF, F4, F4), (FP, FP, None)])
def test_combine(moe, T, k, dim, dtype, out, add):
    g = gen(T + k)
    P = T * k + 3
    o = strided(rnd(g, P, dim, dtype=dtype), 8, float("nan"))[1]
    pos = torch.randperm(P, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    pos[T // 2, 0], pos[T - 1, k - 1] = -1, P  # dropped pairs
    pos = pos.cuda()
    w = torch.rand(T, k, generator=g).cuda()
    more = None if add is None else rnd(g, T, dim, dtype=add)
    for weights in (w, None):
        y = moe.combine(o, pos, weights=weights, add=more, out_dtype=out)
        value, mag = R.combine(o, pos, weights, more)
        R.within(y, value, R.stored(value, R.sums(k, mag), out), "y")
    if add == out:
        y = more.clone()
        moe.combine(o, pos, weights=w, add=y, out=y)
        assert torch.equal(y, moe.combine(o, pos, weights=w, add=more, out_dtype=out))
    dy = rnd(g, T, dim, dtype=dtype)
    d_o = torch.full((P, dim), 5.0, dtype=dtype, device="cuda")
    _, dw = moe.combine_backward(dy, o, pos, w, d_o=d_o)
    want = torch.full((P, dim), 5.0, dtype=R.F8)
    named = torch.zeros(P, dtype=torch.bool)
    dwv, dwm = (torch.zeros(T, k, dtype=R.F8) for _ in range(2))
    for t in range(T):
        for j in range(k):
            at = int(pos[t, j])
            if 0 <= at < P:
                want[at], named[at] = R.d(w)[t, j] * R.d(dy)[t], True
                dwv[t, j], dwm[t, j] = (R.d(o)[at] * R.d(dy)[t]).sum(), (R.d(o)[at] * R.d(dy)[t]).abs().sum()
    R.within(d_o[named.cuda()], want[named], R.stored(want[named], R.U * want[named].abs(), dtype), "d_o")
    assert (d_o[~named.cuda()] == 5.0).all()
    R.within(dw, dwv, R.stored(dwv, R.sums(dim, dwm), F4), "dw")


# ------------------------------------------------- streams, graphs, devices
def test_repeats_are_equal_and_streams_work(moe):
    offsets, P, A, a_row, W, dC = problem("short_long", "mid", BF)
    first = [moe.grouped_gemm(A, W, offsets, a_row=a_row), moe.grouped_gemm_dgrad(dC, W, offsets), moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        again = [moe.grouped_gemm(A, W, offsets, a_row=a_row, stream=side), moe.grouped_gemm_dgrad(dC, W, offsets, stream=side),
                 moe.grouped_gemm_wgrad(dC, A, offsets, a_row=a_row, stream=side)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_and_replayed(moe):
    """Forward and backward of a routed pair of projections in one graph; every
    replay equals the eager calls on the same inputs, with eager work between."""
    T, k, E, dim, f = 48, 2, 6, 128, 64
    g = gen(11)
    x, dy = rnd(g, T, dim), rnd(g, T, dim)
    W1, W2 = rnd(g, E, f, dim, scale=0.1), rnd(g, E, dim, f, scale=0.1)
    logits = torch.randn(T, E, generator=g).cuda()
    ws = moe.alloc_workspace(moe.route_workspace_bytes(T, E))
    rt = moe.alloc_routing(T, E, k)

    def step():
        moe.route(logits, k, out=rt, ws=ws)
        pos = rt["pair_pos"].view(T, k)
        h = moe.grouped_gemm(x, W1, rt["offsets"], a_row=rt["sorted_token"])
        o = moe.grouped_gemm(h, W2, rt["offsets"])
        y = moe.combine(o, pos, weights=rt["topk_w"])
        d_o, dw = moe.combine_backward(dy, o, pos, rt["topk_w"])
        dh = moe.grouped_gemm_dgrad(d_o, W2, rt["offsets"])
        dW2 = moe.grouped_gemm_wgrad(d_o, h, rt["offsets"])
        dx = moe.combine(moe.grouped_gemm_dgrad(dh, W1, rt["offsets"]), pos)
        dW1 = moe.grouped_gemm_wgrad(dh, x, rt["offsets"], a_row=rt["sorted_token"])
        return y, dw, dx, dW1, dW2

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        logits.copy_(torch.randn(T, E, generator=gen(20 + i)))
        x.copy_(rnd(gen(30 + i), T, dim))
        want = [t.clone() for t in step()]
        for t in held:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), f"replay {i}"


def test_moe_layer_forward_and_backward(moe):
    """Route, gate/up, SwiGLU, down and combine as a program runs them, and the
    gradients of x, the weights and the gates, against 64-bit autograd. The
    bounds come from the 16-bit tensors in between: 16 roundings of eps / 2 (their
    root mean square is far below one) on each result's norm."""
    T, k, E, dim, f = 96, 4, 8, 256, 192
    g = gen(12)
    x, dy = rnd(g, T, dim), rnd(g, T, dim)
    Wg, Wd = rnd(g, E, 2 * f, dim, scale=dim ** -0.5), rnd(g, E, dim, f, scale=f ** -0.5)
    logits = torch.randn(T, E, generator=g)
    rt = moe.route(logits.cuda(), k)
    pos, off, tok = rt["pair_pos"].view(T, k), rt["offsets"], rt["sorted_token"]
    a = moe.grouped_gemm(x, Wg, off, a_row=tok, out_dtype=F4).requires_grad_(True)
    h = torch.nn.functional.silu(a[:, :f]) * a[:, f:]
    h16 = h.detach().to(BF)
    o = moe.grouped_gemm(h16, Wd, off)
    y = moe.combine(o, pos, weights=rt["topk_w"], out_dtype=F4)
    d_o, dw = moe.combine_backward(dy, o, pos, rt["topk_w"])
    h.backward(moe.grouped_gemm_dgrad(d_o, Wd, off, out_dtype=F4))
    da = a.grad.to(BF)
    got = dict(y=y, dw=dw, dWd=moe.grouped_gemm_wgrad(d_o, h16, off, out_dtype=F4), dWg=moe.grouped_gemm_wgrad(da, x, off, a_row=tok, out_dtype=F4),
               dx=moe.combine(moe.grouped_gemm_dgrad(da, Wg, off), pos, out_dtype=F4))
    xr, gr, dr = (R.d(t).requires_grad_(True) for t in (x, Wg, Wd))
    w = R.d(rt["topk_w"]).requires_grad_(True)
    ids = rt["topk_ids"].cpu().long()
    yr = torch.stack([sum(w[t, j] * (dr[e] @ (torch.nn.functional.silu(gr[e][:f] @ xr[t]) * (gr[e][f:] @ xr[t]))) for j, e in enumerate(ids[t]))
                      for t in range(T)])
    yr.backward(R.d(dy))
    want = dict(y=yr.detach(), dw=w.grad, dWd=dr.grad, dWg=gr.grad, dx=xr.grad)
    for name in want:
        rel = float((R.d(got[name]) - want[name]).norm() / want[name].norm())
        assert rel <= 16 * torch.finfo(BF).eps / 2, (name, rel)


def test_refused_tensors(moe):
    x, W, off = rnd(gen(1), 8, 16), rnd(gen(1), 2, 8, 16), bounds([3, 5])[0]
    bad = [(ValueError, lambda: moe.grouped_gemm(x, W, off[:2])), (TypeError, lambda: moe.grouped_gemm(x, W.half(), off)),
           (ValueError, lambda: moe.grouped_gemm(x.t(), W, off)), (ValueError, lambda: moe.grouped_gemm(x, W.transpose(1, 2), off)),
           (TypeError, lambda: moe.grouped_gemm(x, W, off, out_dtype=FP)), (TypeError, lambda: moe.grouped_gemm(x, W, off.long())),
           (TypeError, lambda: moe.grouped_gemm(x, W, off, a_row=torch.zeros(8, device="cuda"))),
           (ValueError, lambda: moe.grouped_gemm(x, W, off, out=torch.empty(8, 9, dtype=BF, device="cuda"))),
           (ValueError, lambda: moe.grouped_gemm(x[:1].expand(8, 16), W, off)),
           (ValueError, lambda: moe.grouped_gemm_wgrad(rnd(gen(1), 8, 8), x, off, accumulate=True)),
           (ValueError, lambda: moe.grouped_gemm_wgrad(rnd(gen(1), 7, 8), x, off)),
           (ValueError, lambda: moe.grouped_gemm_wgrad(rnd(gen(1), 8, 8), x, off, out=torch.zeros(2, 8, 16, dtype=BF, device="cuda"), accumulate=True)),
           (ValueError, lambda: moe.combine(x, off)), (ValueError, lambda: moe.combine(x, off.view(1, 3), weights=torch.ones(1, 2, device="cuda"))),
           (ValueError, lambda: moe.combine_backward(x, x[:, :8], off.view(1, 3)))]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
