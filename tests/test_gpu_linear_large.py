"""Products of one matrix beyond 2^30 elements of an operand: they take the tiles, and about the time, of those just below; results against 64 bits."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, F4 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    m.load()
    return m


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=BF, device="cuda").normal_(0.0, scale, generator=g)
    return t


def shortest(f):
    f()
    times = []
    for _ in range(4):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def test_forward(moe):
    T, N, K = 300, 131072, 8192
    x, W = rnd(1, T, K), rnd(2, N, K, scale=K ** -0.5)
    y = torch.empty(T, N, dtype=BF, device="cuda")
    below = shortest(lambda: moe.linear(x, W[:-8], out=y[:, :-8]))
    assert shortest(lambda: moe.linear(x, W, out=y)) < 1.7 * below
    for at in (0, N // 2 + 31, N - 40):
        value, slack, _, _ = R.linear(x, W[at:at + 40], None, "none", None)
        R.within(y[:, at:at + 40], value, R.stored(value, slack, BF), "y")


def test_input_gradient(moe):
    T, N, K = 520, 131072, 8192  # (dW of these rows is 2^30 elements too)
    dy, x, W = rnd(1, T, N), rnd(2, T, K), rnd(3, N, K, scale=N ** -0.5)
    dx, dW = torch.empty(T, K, dtype=F4, device="cuda"), torch.empty(N, K, dtype=BF, device="cuda")
    ws = torch.empty(moe.linear_backward_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    below = shortest(lambda: moe.linear_backward(dy[:, :-8], x, W[:-8], dx=dx, dW=dW[:-8], ws=ws))
    assert shortest(lambda: moe.linear_backward(dy, x, W, dx=dx, dW=dW, ws=ws)) < 1.7 * below
    for at in (0, K - 24):
        cols = W[:, at:at + 24].contiguous()
        (value, slack), _, _ = R.linear_grad(dy[:40], x[:40, :24], cols, None, "none", BF)
        R.within(dx[:40, at:at + 24], value, R.stored(value, slack, F4), "dx")
    _, (value, slack), _ = R.linear_grad(dy[:, -40:], x[:, -40:], W[-40:, -40:], None, "none", BF)
    R.within(dW[-40:, -40:], value, R.stored(value, slack, BF), "dW")


@pytest.mark.parametrize("T,N,K", [(131072, 8192, 2048), (131072, 1024, 8192)], ids=["dz", "x"])
def test_weight_gradient(moe, T, N, K):
    dy, x, W = rnd(1, T, N), rnd(2, T, K), rnd(3, N, K)
    dx, dW = torch.empty(T, K, dtype=BF, device="cuda"), torch.empty(N, K, dtype=F4, device="cuda")
    ws = torch.empty(moe.linear_backward_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    below = shortest(lambda: moe.linear_backward(dy[:-8], x[:-8], W, dx=dx[:-8], dW=dW, ws=ws))
    assert shortest(lambda: moe.linear_backward(dy, x, W, dx=dx, dW=dW, ws=ws)) < 1.7 * below
    _, (value, slack), _ = R.linear_grad(dy[:, -24:], x[:, -24:], W[-24:, -24:], None, "none", BF)
    R.within(dW[-24:, -24:], value, R.stored(value, slack, F4), "dW")


def test_weight_gradient_of_rows_far_apart(moe):
    """Rows whose distance alone makes 2^30 elements, in views of a wider matrix."""
    T, N, K, ld = 1100, 2824, 2824, 1 << 20
    dy, x, W = rnd(1, T, ld), rnd(2, T, ld), rnd(3, N, K)
    dx, dW, _ = moe.linear_backward(dy[:, 64:64 + N], x[:, 8:8 + K], W, grad_dtype=F4)
    ex, ew, _ = moe.linear_backward(dy[:, 64:64 + N].contiguous(), x[:, 8:8 + K].contiguous(), W, grad_dtype=F4)
    assert torch.equal(dW, ew) and torch.equal(dx, ex)
