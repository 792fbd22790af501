"""The rounding flag of the product's gradient at the C interface, without a GPU."""
import torch

import grouped_int4_dequant_amd as moe
from grouped_int4_dequant_amd import binding as B

ROUND = 0x100
EINVAL, EWORKSPACE = -1, -3


def backward(act, ws_bytes):
    dtype = B._CODES[torch.bfloat16]
    p = 1 << 20  # aligned, never read: the call is refused
    return B.load().moe_linear_backward(dtype, p, 64, p, 32, 4, 64, 32, p, p, 64, act, p, dtype, 32, p, None, dtype, 0, p, ws_bytes, None)


def test_flag_belongs_to_the_gradient():
    bf = B._CODES[torch.bfloat16]
    p = 1 << 20
    assert B.load().moe_linear(bf, p, 32, 4, 64, 32, p, None, bf, 2 | ROUND, None, 0, None, 0, p, bf, 64, None) == EINVAL
    for act in (7, 7 | ROUND, 0x200, 2 | 0x400, -1):
        assert backward(act, 1 << 30) == EINVAL and B.load().moe_linear_backward_workspace_bytes(4, 64, 32, act) == 0


def test_workspace_goes_by_the_flag():
    f = B.load().moe_linear_backward_workspace_bytes
    T, N, K = 100, 64, 40
    for act in (1, 2, 3, 4, 5, 6):
        whole, rounded = f(T, N, K, act), f(T, N, K, act | ROUND)
        # three parts of dz and W and x in two each, against dz
        assert whole >= 3 * T * N * 2 + 2 * (N + T) * K * 2 and T * N * 2 <= rounded < T * N * 4 + (1 << 15)
        assert backward(act, f(4, 64, 32, act) - 1) == EWORKSPACE and backward(act | ROUND, f(4, 64, 32, act | ROUND) - 1) == EWORKSPACE
    assert f(T, N, K, 0) == f(T, N, K, ROUND)  # nothing to round without activation
    assert moe.linear_backward_workspace_bytes(T, N, K, "silu", round_dz=True) == f(T, N, K, 2 | ROUND)
    assert moe.linear_backward_workspace_bytes(T, N, K, "silu") == f(T, N, K, 2)
