"""One token through the whole layer at every size of its top-k (up to 64, 256 and 1024 experts have code of their own), few picks and
many, with aligned and unaligned rows; against the plain 64-bit form, element by element."""
import pytest
import torch

import block_reference as R

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


#         k, E, d, f, f_sh
SHAPES = [(8, 65, 264, 40, 24), (8, 256, 264, 40, 0), (1, 256, 72, 520, 8), (16, 256, 136, 24, 0), (33, 100, 72, 16, 16), (64, 64, 40, 16, 0), (64, 256, 40, 24, 8),
          (8, 257, 264, 40, 24), (6, 1000, 136, 72, 0), (17, 1024, 72, 16, 8), (64, 1024, 40, 16, 0), (15, 300, 2056, 40, 0),
          (8, 65, 77, 33, 0), (8, 256, 1029, 35, 17), (16, 130, 67, 41, 0), (64, 200, 33, 9, 5), (8, 257, 131, 19, 0), (64, 1024, 31, 7, 3)]


def problem(shape, dtype, seed=1):
    k, E, d, f, sh = shape
    g = torch.Generator().manual_seed(seed)
    p = dict(x=rnd(g, 1, d, dtype=dtype), logits=rnd(g, 1, E, dtype=F4), gu=rnd(g, E, 2 * f, d, dtype=dtype, scale=d ** -0.5),
             dn=rnd(g, E, d, f, dtype=dtype, scale=f ** -0.5), k=k)
    p["sh_gu"] = rnd(g, 2 * sh, d, dtype=dtype, scale=d ** -0.5) if sh else None
    p["sh_dn"] = rnd(g, d, sh, dtype=dtype, scale=sh ** -0.5) if sh else None
    p["add"] = rnd(g, 1, d, dtype=F4)
    return p


def check(moe, p, exact_gates=False):
    k, E = p["k"], p["logits"].shape[1]
    ids, w = torch.full((1, k), -7, dtype=torch.int32, device="cuda"), torch.full((1, k), -7.0, device="cuda")
    y = moe.few_tokens_layer(**p, topk_ids=ids, topk_w=w)
    value, slack, rids, gates = R.layer(p["x"], p["logits"], p["gu"], p["dn"], k, p["sh_gu"], p["sh_dn"], p["add"])
    assert torch.equal(ids.cpu().long(), rids)
    R.within(w, gates, 64 * R.U * gates, "gates")
    R.within(y, value, R.stored(value, slack, F4), "y")
    assert torch.equal(y, moe.few_tokens_layer(**p))
    return y, ids, w


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF, FP])
def test_one_token(moe, shape, dtype):
    p = problem(shape, dtype)
    ws = torch.full((moe.few_tokens_workspace_bytes(1, dtype, *shape[2:4], shape[1], shape[0], shape[4]),), 255, dtype=torch.uint8, device="cuda")
    y, ids, w = check(moe, p)
    got_ids, got_w = torch.empty_like(ids), torch.empty_like(w)
    assert torch.equal(y, moe.few_tokens_layer(**p, ws=ws, topk_ids=got_ids, topk_w=got_w)) and torch.equal(ids, got_ids) and torch.equal(w, got_w)


@pytest.mark.parametrize("shape", [(8, 65, 72, 16, 0), (64, 256, 40, 16, 8), (16, 200, 67, 9, 0), (17, 1024, 40, 16, 0), (64, 600, 33, 9, 0)], ids=lambda s: "-".join(map(str, s)))
def test_equal_logits(moe, shape):
    """Equal logits go to the lower expert: within a lane's run of experts, across lanes, and among signed zeros."""
    k, E = shape[:2]
    p = problem(shape, BF, seed=2)
    p["logits"] = torch.full_like(p["logits"], 0.25)
    _, ids, w = check(moe, p)
    assert ids[0].tolist() == list(range(k)) and torch.allclose(w, torch.full_like(w, 1.0 / k))
    g = torch.Generator().manual_seed(3)
    for levels in (2, 3, 7):  # a few values, each of many experts
        p["logits"] = torch.randint(0, levels, (1, E), generator=g).float().cuda() - 1.0
        check(moe, p)
    p["logits"] = torch.where(torch.arange(E) % 3 == 0, -0.0, 0.0)[None].cuda()
    _, ids, _ = check(moe, p)
    assert ids[0].tolist() == list(range(k))


def test_masked_experts(moe):
    """Experts at -inf are picked last, in order, and weigh nothing."""
    for shape in ((8, 256, 72, 16, 0), (20, 700, 33, 9, 0)):
        k, E = shape[:2]
        p = problem(shape, BF, seed=4)
        p["logits"][:] = float("-inf")
        p["logits"][0, E - 1], p["logits"][0, 70] = 1.0, 2.0
        _, ids, w = check(moe, p)
        assert ids[0].tolist() == [70, E - 1] + list(range(k - 2)) and (w[0, 2:] == 0).all()
