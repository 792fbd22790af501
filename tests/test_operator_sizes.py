"""Sizes that do not fit the C interface's 32 bits are refused, not cut off."""
import pytest
import torch

from test_gpu_grouped import BF, moe  # noqa: F401


def test_workspace_of_sizes_past_32_bits():
    import grouped_int4_dequant_amd as m
    for T, r in (((1 << 32) + 8, 4), (8, (1 << 32) + 4), (1 << 31, 4)):
        with pytest.raises(ValueError, match="2\\^31"):
            m.adapter_backward_workspace_bytes(T, r)
    assert m.adapter_backward_workspace_bytes((1 << 31) - 1, 4) == 0


@pytest.mark.gpu
def test_sizes_past_32_bits_are_refused(moe):  # noqa: F811
    store = torch.empty((1 << 32) + 8, dtype=BF, device="cuda")  # 8 GiB; as 32-bit sizes these would be 8
    long, three = store.view(-1, 1), store.view(-1, 1, 1)
    x, w, at = torch.ones(8, 1, dtype=BF, device="cuda"), torch.ones(2, 1, 1, dtype=BF, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    pos = at.view(4, 2)
    plan = (at, off)
    ids = store.view(torch.int32)  # 2^31 + 4 of them
    for f in (lambda: moe.grouped_gemm(long, w, off, a_row=at), lambda: moe.grouped_gemm(long, w, off), lambda: moe.grouped_gemm(x, three, off),
              lambda: moe.grouped_gemm(x, w, off, a_row=ids), lambda: moe.grouped_gemm_dgrad(long, w, off), lambda: moe.grouped_gemm_dgrad(x, three, off),
              lambda: moe.grouped_gemm_wgrad(x, long, off, a_row=at), lambda: moe.grouped_gemm_wgrad(long, x, off, a_row=at),
              lambda: moe.combine(long, pos), lambda: moe.combine(x, ids.view(-1, 1)), lambda: moe.combine_backward(x[:4], long, pos),
              lambda: moe.adapter_plan(ids, 2), lambda: moe.adapter_plan(at, (1 << 32) + 2), lambda: moe.adapter_forward(long, w, w, None, plan),
              lambda: moe.adapter_forward(x, three, w, None, plan), lambda: moe.adapter_backward(x, long, w, w, None, plan)):
        with pytest.raises(ValueError, match="2\\^31"):
            f()
