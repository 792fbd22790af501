"""The whole layer with 16-bit weights for a few tokens on the GPU against its
plain 64-bit form, element by element."""
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


#          T, k, E, d, f, f_sh
SHAPES = {"one": (1, 1, 1, 1, 1, 1), "decode": (1, 8, 256, 520, 72, 40), "two": (2, 2, 16, 256, 128, 128), "odd": (3, 2, 5, 77, 131, 33), "batch": (16, 8, 256, 264, 40, 24),
          "crowd": (50, 2, 3, 136, 200, 0), "all": (64, 8, 8, 72, 24, 16), "most": (64, 8, 300, 40, 16, 8), "many_experts": (7, 6, 1000, 64, 16, 0), "wide": (5, 1, 4, 2312, 1544, 2056),
          "ks": (8, 64, 70, 64, 16, 0), "tail_d": (20, 4, 9, 129, 64, 64), "tail_f": (20, 4, 9, 128, 65, 0), "deep": (17, 2, 4, 4104, 24, 520),
          "broad_odd": (21, 2, 5, 1031, 65, 33), "forty_nine": (49, 3, 49, 72, 520, 8), "ten": (10, 16, 64, 40, 16, 0), "one_odd": (1, 3, 9, 1029, 35, 0)}


def problem(shape, dtype, out=None, seed=1, inner=1.0):
    T, k, E, d, f, sh = SHAPES[shape]
    g = torch.Generator().manual_seed(seed)
    p = dict(x=rnd(g, T, d, dtype=dtype), logits=rnd(g, T, E, dtype=F4), gu=rnd(g, E, 2 * f, d, dtype=dtype, scale=inner * d ** -0.5),
             dn=rnd(g, E, d, f, dtype=dtype, scale=f ** -0.5), k=k)
    p["sh_gu"] = rnd(g, 2 * sh, d, dtype=dtype, scale=inner * d ** -0.5) if sh else None
    p["sh_dn"] = rnd(g, d, sh, dtype=dtype, scale=sh ** -0.5) if sh else None
    p["add"] = rnd(g, T, d, dtype=out) if out is not None else None
    return p


CASES = [(s, t, o, a) for s in SHAPES for t, o, a in ((BF, BF, True), (FP, F4, False))] + [("batch", BF, F4, True), ("odd", FP, FP, True), ("crowd", BF, F4, False)]


@pytest.mark.parametrize("shape,dtype,out,add", CASES, ids=[f"{s}-{str(t)[6:]}-{str(o)[6:]}" for s, t, o, _ in CASES])
def test_layer(moe, shape, dtype, out, add):
    p = problem(shape, dtype, out if add else None)
    T, k = p["x"].shape[0], p["k"]
    ids, w = torch.full((T, k), -7, dtype=torch.int32, device="cuda"), torch.full((T, k), -7.0, device="cuda")
    y = moe.few_tokens_layer(**p, out_dtype=out, topk_ids=ids, topk_w=w)
    value, slack, rids, gates = R.layer(p["x"], p["logits"], p["gu"], p["dn"], k, p["sh_gu"], p["sh_dn"], p["add"])
    assert torch.equal(ids.cpu().long(), rids)
    R.within(w, gates, 64 * R.U * gates, "gates")
    R.within(y, value, R.stored(value, slack, out), "y")
    assert torch.equal(y, moe.few_tokens_layer(**p, out_dtype=out))


@pytest.mark.parametrize("shape", ["batch", "crowd", "tail_d", "deep", "wide"])
def test_rows_do_not_depend_on_each_other(moe, shape):
    p = problem(shape, BF, F4)
    y = moe.few_tokens_layer(**p)
    T = p["x"].shape[0]
    for a, b in ((0, 2), (T // 2, T), (T - 3, T)):
        part = dict(p, x=p["x"][a:b], logits=p["logits"][a:b], add=p["add"][a:b])
        assert torch.equal(moe.few_tokens_layer(**part), y[a:b])
    # a call of one token cuts its sums in other places
    one = dict(p, x=p["x"][-1:], logits=p["logits"][-1:], add=p["add"][-1:])
    value, slack, _, _ = R.layer(one["x"], one["logits"], p["gu"], p["dn"], p["k"], p["sh_gu"], p["sh_dn"], one["add"])
    got = moe.few_tokens_layer(**one)
    R.within(got, value, R.stored(value, slack, F4), "one")
    R.within(y[-1:], value, R.stored(value, slack, F4), "among others")


def test_strided_and_in_place(moe):
    for shape in ("batch", "odd", "tail_d"):
        p = problem(shape, BF, F4)
        T, d = p["x"].shape
        expect = moe.few_tokens_layer(**p, out_dtype=F4)
        xw = torch.full((T, d + 3), float("nan"), dtype=BF, device="cuda")
        xw[:, :d] = p["x"]
        yw = torch.full((T, d + 5), 4.0, device="cuda")
        yw[:, :d] = p["add"]
        v = yw[:, :d]
        got = moe.few_tokens_layer(**dict(p, x=xw[:, :d], add=v), out=v)
        assert got is v and torch.equal(v, expect) and (yw[:, d:] == 4).all()


def test_ties_and_masked_experts(moe):
    """Equal logits go to the lower expert; experts at -inf are picked last and weigh nothing."""
    p = problem("two", BF)
    p["logits"] = torch.full_like(p["logits"], 0.25)
    ids, w = torch.empty((2, 2), dtype=torch.int32, device="cuda"), torch.empty((2, 2), device="cuda")
    moe.few_tokens_layer(**p, topk_ids=ids, topk_w=w)
    assert ids.tolist() == [[0, 1]] * 2 and w.tolist() == [[0.5, 0.5]] * 2
    p["logits"][:] = float("-inf")
    p["logits"][0, 9] = 2.0
    p["logits"][1, 3] = -5.0
    y = moe.few_tokens_layer(**p, topk_ids=ids, topk_w=w, out_dtype=F4)
    assert ids.tolist() == [[9, 0], [3, 0]] and w.tolist() == [[1.0, 0.0]] * 2
    one = dict(p, k=1)
    assert torch.equal(y, moe.few_tokens_layer(**one, out_dtype=F4))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_inner_values_of_any_size(moe, dtype):
    """Inner values far apart (columns of W_gu scaled by powers of four) and beyond fp16 enter the second product whole."""
    p = problem("two", dtype, seed=3)
    f = p["dn"].shape[2]
    scale = (4.0 ** (torch.arange(f) % 9 - 2)).to(dtype).cuda()  # 1/16 .. 4096, on each factor of h
    p["gu"] = p["gu"] * scale.repeat(2)[None, :, None]
    p["dn"] = p["dn"] * (scale.double() ** -2).to(dtype)[None, None, :]
    p["sh_gu"] = p["sh_dn"] = None
    y = moe.few_tokens_layer(**p, out_dtype=F4)
    value, slack, _, _ = R.layer(p["x"], p["logits"], p["gu"], p["dn"], p["k"], None, None, None)
    R.within(y, value, R.stored(value, slack, F4), "y")


def test_infinities_and_nan_stay_in_their_rows(moe):
    p = problem("batch", BF)
    clean = moe.few_tokens_layer(**p)
    x = p["x"].clone()
    x[3, 5], x[9, 0] = float("nan"), float("inf")
    got = moe.few_tokens_layer(**dict(p, x=x))
    rest = [t for t in range(16) if t not in (3, 9)]
    assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[3]).all() and not torch.isfinite(got[9]).any()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", ["two", "batch", "crowd", "tail_f"])
def test_infinite_weights_and_inner_values(moe, dtype, shape):
    """Infinite weights of the second product and inner values beyond the type give the formula's infinities, and only there."""
    p = problem(shape, dtype, seed=6)
    p["sh_gu"] = p["sh_dn"] = None
    T, k = p["x"].shape[0], p["k"]
    clean = moe.few_tokens_layer(**p, out_dtype=F4)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    e = int(torch.argmax(p["logits"][0]))
    q = dict(p, dn=p["dn"].clone(), gu=p["gu"].clone())
    q["dn"][e, 3, 5] = float("inf")       # column 3 of y
    q["dn"][e, 8, 0] = -float("inf")      # column 8
    q["gu"][e, 0] = 0.0                   # inner value 0 is zero: zero times infinity
    got = moe.few_tokens_layer(**q, out_dtype=F4, topk_ids=ids)
    hit = (ids == e).any(1)
    base = moe.few_tokens_layer(**dict(q, dn=p["dn"]), out_dtype=F4)
    cols = [c for c in range(got.shape[1]) if c not in (3, 8)]
    assert torch.equal(got[:, cols], base[:, cols]) and torch.equal(got[~hit], clean[~hit])
    x, g = R.d(p["x"]), R.d(q["gu"][e])
    f = g.shape[0] // 2
    h5 = R.curve("silu", x @ g[5]) * (x @ g[f + 5])
    for t in hit.nonzero()[:, 0].tolist():
        assert torch.isinf(got[t, 3]) and torch.sign(got[t, 3]).item() == torch.sign(h5[t]).item() and torch.isnan(got[t, 8])
    # an infinite inner value against finite weights
    q = dict(p, gu=p["gu"].clone())
    q["gu"][e, 2], q["gu"][e, f + 2] = float("inf"), 0.5
    x1 = dict(q, x=p["x"].abs() + 1, dn=p["dn"].abs() + 1)
    got = moe.few_tokens_layer(**x1, out_dtype=F4)
    assert (got[hit] == float("inf")).all() and torch.isfinite(got[~hit]).all()


def test_no_rows(moe):
    p = problem("two", BF)
    y = moe.few_tokens_layer(**dict(p, x=p["x"][:0], logits=p["logits"][:0]))
    assert y.shape == (0, p["x"].shape[1])
