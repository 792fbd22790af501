"""The forms for few rows of the product and of its gradients over sums of several rounds of their loops (2048 terms a round forward, 512 in
the input gradient), whole and ragged ones; against plain 64-bit forms, element by element."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

BF, FP, F4 = torch.bfloat16, torch.float16, torch.float32
#         T, N, K: sums of N terms in the input gradient, of K forward
SHAPES = [(1, 264, 4104), (1, 4104, 264), (5, 1024, 4096), (16, 520, 2056), (17, 1032, 2048), (20, 1544, 2056), (33, 512, 6152), (48, 2056, 1024), (64, 520, 4096), (64, 4096, 136)]


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_int4_dequant_amd as m
    m.load()
    return m


def rnd(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_forward(moe, T, N, K, dtype, act):
    g = torch.Generator().manual_seed(T + N)
    x, W, b = rnd(g, T, K, dtype=dtype), rnd(g, N, K, dtype=dtype, scale=K ** -0.5), rnd(g, N, dtype=F4)
    r = rnd(g, T, N // 2 if act == "swiglu" else N, dtype=F4)
    pre = torch.full((T, N), 5.0, dtype=dtype, device="cuda")
    y = moe.linear(x, W, bias=b, act=act, residual=r, pre=pre)
    value, slack, z, zs = R.linear(x, W, b, act, r)
    R.within(y, value, R.stored(value, slack, F4), "y")
    R.within(pre, z, R.stored(z, zs, dtype), "pre")


@pytest.mark.parametrize("act,rounded", [("none", False), ("swiglu", True), ("gelu", True)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_gradients(moe, T, N, K, dtype, act, rounded):
    g = torch.Generator().manual_seed(T + K)
    x, W = rnd(g, T, K, dtype=dtype), rnd(g, N, K, dtype=dtype, scale=K ** -0.5)
    dy, pre = rnd(g, T, N // 2 if act == "swiglu" else N, dtype=dtype), rnd(g, T, N, dtype=dtype)
    got = moe.linear_backward(dy, x, W, pre=pre, act=act, bias_grad=True, dx=torch.empty(T, K, device="cuda"), grad_dtype=F4, round_dz=rounded)
    for v, (value, slack), name in zip(got, R.linear_grad(dy, x, W, pre, act, dtype), ("dx", "dW", "db")):
        R.within(v, value, R.stored(value, slack, F4), name)


@pytest.mark.parametrize("results", ["16", "32"])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_gradients_of_a_whole_dz(moe, T, N, K, dtype, results):
    """dz in its parts: 2^-15 (fp16: 2^-22, or 2^-25) of it is lost for 16-bit results and nothing for fp32 ones; six pairs of parts at most."""
    g = torch.Generator().manual_seed(T + K + 1)
    x, W = rnd(g, T, K, dtype=dtype), rnd(g, N, K, dtype=dtype, scale=K ** -0.5)
    dy, pre = rnd(g, T, N // 2, dtype=dtype), rnd(g, T, N, dtype=dtype)
    t = F4 if results == "32" else dtype
    dx, dW, _ = moe.linear_backward(dy, x, W, pre=pre, act="geglu", dx=torch.empty(T, K, dtype=t, device="cuda"), grad_dtype=t)
    dz, s, _ = R.act_grad(dy, pre, "geglu", dtype)
    s = s + (0.0 if t is F4 else 2.0 ** -15 * dz.abs() if dtype is BF else 2.0 ** -22 * dz.abs() + 2.0 ** -25)
    X, V = R.d(x), R.d(W)
    for got, value, slack, name in ((dx, dz @ V, s @ V.abs() + R.sums(6 * N, dz.abs() @ V.abs()), "dx"), (dW, dz.T @ X, s.T @ X.abs() + R.sums(6 * T, dz.abs().T @ X.abs()), "dW")):
        R.within(got, value, R.stored(value, slack, t), name)
