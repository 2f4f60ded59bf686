"""The attention half's operators on the GPU at values where a rounding, a
mask or a range can go wrong: NaN, infinities, numbers at both ends of fp32's
range, scales far apart, and entries that a call may not use."""

import math

import pytest
import torch

from tests import attn_reference as R
from tests.test_gpu_attn import (DT, check_append, check_attend, gen, i32, make_cache, make_weights, normal,
                                  within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def m():
    import moe_decode_layer_sm_b200
    return moe_decode_layer_sm_b200


def bits(t):
    return t.view(torch.uint8) if t.dtype == R.FP8 else t


# --------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot", [None, (64, 0, False), (32, 32, False), (32, 0, True), (6, 10, False)])
@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 128)])   # 1, 2 and 4 units of 16 values a thread
def test_append_nan_stays_nan(m, dtype, rot, d, page):
    """A NaN with no infinity beside it, in values, in keys that are rotated and
    in dimensions that are not; both signs; a head of nothing else."""
    rope = None if rot is None else m.Rope(rot[0], offset=rot[1], interleaved=rot[2])
    k, v = (normal((1, page, 4, d), DT[dtype], 300 + i) for i in (0, 1))
    for x in (k, v):
        x[0, 3, 0, 5] = math.nan
        x[0, page - 1, 1, d - 1], x[0, 0, 1, 40] = -math.nan, math.nan
        x[0, :, 2] = math.nan
    check_append(m, dtype, [page], [page], page, 4, d, page, rope, k=k, v=v)


def test_append_keeps_a_page_scale_that_is_nan(m):
    """The older codes of such a page are no numbers, and stay none."""
    d, page, heads = 64, 16, 3
    for dtype in ("bf16", "f32"):
        cache = make_cache(m, 3, heads, page, d, 310)
        cache.k_scale[1, 1], cache.v_scale[1, 2] = math.nan, math.nan
        before = {n: getattr(cache, n).clone() for n in ("k", "v")}
        k, v = (normal((1, 3, heads, d), DT[dtype], 311 + i) for i in (0, 1))
        plan = m.AttnPlan(heads, heads, d, page, 3, 1, 2, max_new=3, dtype=dtype)
        want = R.append(cache, k, v, [9], [[1, 2]], [3], None, page)
        plan.append(cache, k, v, i32([9]), i32([[1, 2]]))
        for name, bad in (("k", 1), ("v", 2)):
            code, scale = getattr(cache, name), getattr(cache, name + "_scale")
            assert math.isnan(scale[1, bad].item())
            assert torch.isnan(code[1, bad, 6:9].float()).all()
            assert torch.equal(bits(code)[1, bad, :6], bits(before[name])[1, bad, :6])
            for h in set(range(heads)) - {bad}:
                assert torch.equal(code[1, h].double(), want[name][1, h]) and scale[1, h] == want[name + "_scale"][1, h]


def check_rotated_keys(m, k, rot, il=False):
    """One page of fp32 keys, its codes and scales from the rotated keys in fp64."""
    _, page, heads, d = k.shape
    rope = m.Rope(rot, interleaved=il)
    plan = m.AttnPlan(heads, heads, d, page, 1, 1, 1, max_new=1, dtype="f32")
    cache = m.KVCache.empty(1, heads, page, d)
    plan.append(cache, k, k, i32([page]), i32([[0]]), rope=rope)
    y = R.rotate(k[0], torch.arange(page, device="cuda"), rope).transpose(0, 1)
    finite = torch.where(torch.isfinite(y), y.abs(), 0.0)
    scale = (finite.amax((1, 2)) / 448).float().clamp_min(2.0 ** -126)
    assert torch.equal(cache.k_scale[0], scale)
    want = R.nearest_fp8(y / scale.double()[:, None, None])
    got = cache.k[0].double()
    assert ((got == want) | (torch.isnan(got) & torch.isnan(want))).all(), (got != want).sum().item()


@pytest.mark.parametrize("rot,il", [(64, False), (64, True), (32, False), (10, False)])
def test_append_rotated_keys_at_the_ends_of_the_range(m, rot, il):
    """Rotated keys that lie beyond the largest fp32 number, which the inputs do
    not, and keys among the smallest, whose codes are of scale 2^-126."""
    page, d = 16, 64
    g = gen(320)
    big = (torch.rand((1, page, 8, d), device="cuda", generator=g) * 0.5 + 0.5) * 3.4e38
    check_rotated_keys(m, big, rot, il)
    big[0, 3, 2, 1] = math.inf
    check_rotated_keys(m, big, rot, il)
    tiny = ((torch.rand((1, page, 1024, d), device="cuda", generator=g, dtype=torch.float64) - 0.5) * 2.0 ** -126).float()
    check_rotated_keys(m, tiny, rot, il)
    tiny[0, :, 5] = 0
    tiny[0, 2, 7, 3] = math.inf
    check_rotated_keys(m, tiny[:, :, :16].contiguous(), rot, il)


# ------------------------------------------------------ entries out of range

@pytest.mark.parametrize("lens", [(20, 9), (20, 70)])
def test_more_new_tokens_than_rows_leave_a_sequence_out(m, lens):
    """Where row 0 would lie is not known to the caller's rows: nothing of the
    sequence is written, its rows stay, and the other sequence is served."""
    d, page, hk, hq = 64, 16, 2, 4
    cache = make_cache(m, 5, hk, page, d, 330)
    k, v = (normal((2, 2, hk, d), torch.bfloat16, 331 + i) for i in (0, 1))
    plan = m.AttnPlan(hq, hk, d, page, 5, 2, 4, max_new=2)
    table = [[0, 1, -1, -1], [2, 3, 4, -1]]
    want = R.append(cache, k, v, [lens[0], 0], table, [2, 0], None, page)
    plan.append(cache, k, v, i32(lens), i32(table), n_new=i32([2, 5]))
    assert plan.query_error()[0] == -9
    for n in ("k", "v"):
        assert torch.equal(getattr(cache, n).double(), want[n])
        assert torch.equal(getattr(cache, n + "_scale"), want[n + "_scale"])
    q = normal((2, 2, hq, d), torch.bfloat16, 333)
    out, lse = torch.full_like(q, 5.0), torch.full((2, 2, hq), 5.0, device="cuda")
    plan.attend(cache, q, i32(lens), i32(table), out, lse=lse, n_new=i32([2, 5]))
    rc, st = plan.query_error()
    assert (rc, st.seq) == (-9, 1)
    assert (out[1] == 5.0).all() and (lse[1] == 5.0).all()
    wo, wl, ob, lb = R.attend(cache, q, [lens[0], 0], table, [2, 0], page, 1 / math.sqrt(d))
    within(out[0], wo[0], ob[0])
    within(lse[0], wl[0], lb[0])


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (64, 24, 2), (128, 10, 2), (128, 24, 2), (256, 4, 2)])
@pytest.mark.parametrize("power", [24, 40, 90, -90])
def test_attend_page_that_other_rows_see(m, dtype, d, hq, hk, power):
    """A page of values far larger (or smaller) than the others, of which only
    the first of four rows sees a token: the other rows keep all their bits."""
    page, window, lens = 16, 20, [38]
    cache = make_cache(m, 4, hk, page, d, 340)
    table = [[2, 0, 3]]
    cache.v_scale[2] *= 2.0 ** power
    q = normal((1, 4, hq, d), DT[dtype], 341)
    plan = m.AttnPlan(hq, hk, d, page, 4, 1, 3, max_new=4, dtype=dtype, window=window)
    out = plan.attend(cache, q, i32(lens), i32(table), torch.empty_like(q))
    want, _, ob, _ = R.attend(cache, q, lens, table, [4], page, 1 / math.sqrt(d), window)
    within(out[:, 1:], want[:, 1:], ob[:, 1:])
    if power < 0:   # row 0's bound counts the largest value that it sees, which is one of the others here
        within(out, want, ob)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk,seqs,length", [(64, 4, 2, 1, 100), (128, 5, 1, 1, 9000), (64, 8, 4, 64, 1000),
                                                 (64, 64, 4, 50, 1000), (128, 10, 2, 100, 600), (256, 4, 2, 90, 500)])
@pytest.mark.parametrize("power", [24, 40, 90])
def test_attend_large_page_without_weight(m, dtype, d, hq, hk, seqs, length, power):
    """A page of values 2^power times as large whose tokens have no weight (logits
    200 below the others: exp(-200) 2^90 is 1e-60): the others keep their bits.
    The bound is that of a cache where the page holds zeros.  Many sequences: a
    warp goes on to other pages of the item."""
    page = 64
    per = -(-length // page)
    pages = per * seqs
    cache = make_cache(m, pages, hk, page, d, 350)
    q = normal((seqs, 1, hq, d), DT[dtype], 351)
    q[..., 0] = 8.0   # every row's first element; the large page's keys hold all they have there
    code = torch.zeros(d, device="cuda")
    code[0] = -448.0
    large = range(1, pages, per)   # the second page of each sequence
    for i in large:
        cache.k[i] = code.to(R.FP8)
        cache.k_scale[i] = 230 * math.sqrt(d) / (8 * 448)
        cache.v_scale[i] *= 2.0 ** power
    table = [list(range(s * per, (s + 1) * per)) for s in range(seqs)]
    plan = m.AttnPlan(hq, hk, d, page, pages, seqs, per, dtype=dtype)
    out = plan.attend(cache, q, i32([length] * seqs), i32(table), torch.empty_like(q))
    for i in large:
        cache.v[i] = torch.zeros(d, device="cuda").to(R.FP8)
    want, _, ob, _ = R.attend(cache, q, [length] * seqs, table, [1] * seqs, page, 1 / math.sqrt(d))
    within(out, want, ob)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_one_token_gives_its_value(m, dtype):
    """Its probability is 1: the value is rounded once, to the nearest.  Twice the
    argument's rounding, (|logit| + 24) 2^-23 with logits below 8, lies between
    the sum and the probability: 2^-17."""
    for d, hq, hk in ((64, 8, 8), (128, 40, 8), (256, 16, 8)):
        cache = make_cache(m, 1, hk, 64, d, 360)
        q = normal((1, 1, hq, d), DT[dtype], 361) * 0.25
        plan = m.AttnPlan(hq, hk, d, 64, 1, 1, 1, dtype=dtype)
        out = plan.attend(cache, q, i32([1]), i32([[0]]), torch.empty_like(q))
        v = (cache.v[0, :, 0].double() * cache.v_scale[0].double()[:, None]).repeat_interleave(hq // hk, 0)
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -100)))) * torch.finfo(DT[dtype]).eps
        assert ((out[0, 0].double() - v).abs() <= unit / 2 + v.abs() * 2.0 ** -17).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 24, 2), (256, 4, 2)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("scale", [math.nan, math.inf])
def test_attend_scale_that_is_no_number(m, dtype, d, hq, hk, which, scale):
    """Rows that see none of the page stay clean; with NaN all that see it are NaN."""
    page, lens, table = 16, [34], [[1, 3, 0]]   # rows 0 and 1 end at token 31
    cache, clean = (make_cache(m, 4, hk, page, d, 370) for _ in range(2))
    getattr(cache, which + "_scale")[0, 1] = scale
    q = normal((1, 4, hq, d), DT[dtype], 371)
    plan = m.AttnPlan(hq, hk, d, page, 4, 1, 3, max_new=4, dtype=dtype)
    out = plan.attend(cache, q, i32(lens), i32(table), torch.empty_like(q))
    want, _, ob, _ = R.attend(clean, q, lens, table, [4], page, 1 / math.sqrt(d))
    half = hq // hk
    within(out[:, :2], want[:, :2], ob[:, :2])
    within(out[:, :, :half], want[:, :, :half], ob[:, :, :half])
    if math.isnan(scale):
        assert torch.isnan(out[:, 2:, half:]).all()
    elif which == "v":
        assert not torch.isfinite(out[:, 2:, half:]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 24, 2), (256, 4, 2)])
@pytest.mark.parametrize("length", [1, 200, 9000])
@pytest.mark.parametrize("power", [112, -100])
def test_attend_values_at_the_ends_of_the_range(m, dtype, d, hq, hk, length, power):
    """Values up to 2^112 times the usual, whose sums over 9000 tokens fp32 still
    holds, and far below the usual."""
    page = 64
    pages = -(-length // page)
    cache = make_cache(m, pages, hk, page, d, 380)
    for s in (cache.v_scale,):
        s *= 2.0 ** power
    q = normal((1, 1, hq, d), DT[dtype], 381)
    table = [list(range(pages))]
    plan = m.AttnPlan(hq, hk, d, page, pages, 1, pages, dtype=dtype)
    out = plan.attend(cache, q, i32([length]), i32(table), torch.empty_like(q))
    want, _, ob, _ = R.attend(cache, q, [length], table, [1], page, 1 / math.sqrt(d))
    within(out, want, ob)


# ---------------------------------------------------------- 4-bit projections

INT4 = [(128, "bf16", False), (32, "f32", True), (64, "bf16", True), (96, "f32", False), (256, "f32", True)]


def near_zero_codes(n, k, group, zeros, span, seed):
    """Codes that lie within `span` of their zero point."""
    g = gen(seed)
    z = torch.randint(span, 16 - span, (n, k // group), device="cuda", generator=g) if zeros else \
        torch.full((n, k // group), 8, device="cuda")
    q = z.repeat_interleave(group, 1) + torch.randint(-span, span + 1, (n, k), device="cuda", generator=g)
    return (q[:, 0::2] | q[:, 1::2] << 4).to(torch.uint8), z.to(torch.uint8) if zeros else None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,scales,zeros", INT4)
@pytest.mark.parametrize("n,groups", [(64, 1), (70, 9), (1003, 40), (20000, 5)])
@pytest.mark.parametrize("span", [0, 1])
def test_project_codes_next_to_the_zero_point(m, dtype, group, scales, zeros, n, groups, span):
    """Weights that are zero give zero exactly, small ones lose nothing to the
    zero point's share of the sum; x has a mean."""
    k = group * groups
    codes, z = near_zero_codes(n, k, group, zeros, span, 400)
    s = (torch.rand((n, groups), device="cuda", generator=gen(401)) + 0.1).to(DT[scales])
    plan = m.Projection(n, k, group=group, scale_dtype=scales, zeros=zeros, dtype=dtype)
    plan.pack(codes, s, z)
    full = R.weights(codes, s, z, "int4", group)
    for rows in (1, 3, 8):
        x = (normal((rows, k), torch.float32, 402) + 3).to(DT[dtype])
        y = plan.step(x, torch.empty(rows, n, dtype=DT[dtype], device="cuda"))
        within(y, *R.project(x, full))
        assert span or (y == 0).all()


KINDS = [("int4", 64, "f32", True), ("int4", 128, "bf16", False), ("mxfp4", 32, "bf16", False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,group,scales,zeros", KINDS)
@pytest.mark.parametrize("n,k,shift", [(130, 512, 0), (130, 512, 1), (7, 1280, 0), (9500, 6400, 0)])
def test_project_infinities(m, dtype, fmt, group, scales, zeros, n, k, shift):
    """x of +-infinity gives what the sum of products gives: infinities of the
    weights' signs, NaN where a weight is zero or two of them meet; finite
    numbers beside them that no fp16 holds change nothing."""
    w = make_weights(n, k, fmt, group, scales, zeros, 410)
    plan = m.Projection(n, k, fmt=fmt, group=group, scale_dtype=scales, zeros=zeros, dtype=dtype)
    plan.pack(*w)
    full = R.weights(*w, fmt, group)
    x = normal((6, k + 8), DT[dtype], 411)[:, shift:shift + k]
    x[0, 5] = math.inf
    x[1, k - 1] = -math.inf
    x[2, 7], x[2, k - 9] = math.inf, math.inf
    x[3, 100], x[3, ::3] = math.inf, -1e20
    x[4, 6], x[4, 300] = math.inf, math.nan
    y = plan.step(x, torch.empty(6, n, dtype=DT[dtype], device="cuda"))
    prod = torch.stack([(x[r].double() * full).sum(1) for r in range(6)])   # (a product for each weight, then their sum)
    got = y.double()
    assert torch.equal(torch.isnan(got), torch.isnan(prod))
    assert torch.equal(torch.isposinf(got), torch.isposinf(prod)) and torch.equal(torch.isneginf(got), torch.isneginf(prod))
    assert torch.isposinf(prod).any() and torch.isneginf(prod).any() and torch.isfinite(prod[5]).all()
    within(y[5:], *R.project(x[5:], full))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,group,scales,zeros", KINDS)
def test_project_long_parts(m, dtype, fmt, group, scales, zeros):
    """More than 16 blocks of inputs a warp (bf16): x is read twice, not held."""
    n, k = 9500, 6400
    w = make_weights(n, k, fmt, group, scales, zeros, 415)
    plan = m.Projection(n, k, fmt=fmt, group=group, scale_dtype=scales, zeros=zeros, dtype=dtype)
    plan.pack(*w)
    for rows in (1, 8):
        x = normal((rows, k), DT[dtype], 416)
        y = plan.step(x, torch.empty(rows, n, dtype=DT[dtype], device="cuda"))
        within(y, *R.project(x, R.weights(*w, fmt, group)))


def check_project(m, dtype, fmt, codes, scales, zeros, xs, group=32, scale_dtype="f32", more=0.0):
    n, k = codes.shape[0], codes.shape[1] * 2
    plan = m.Projection(n, k, fmt=fmt, group=group, scale_dtype=scale_dtype, zeros=zeros is not None, dtype=dtype)
    plan.pack(codes, scales, zeros)
    full = R.weights(codes, scales, zeros, fmt, group)
    for x in xs:
        y = plan.step(x, torch.empty(x.shape[0], n, dtype=x.dtype, device="cuda"))
        want, bound = R.project(x, full)
        assert torch.isfinite(want.to(x.dtype)).all()
        within(y, want, bound + more)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(64, 64), (130, 4096), (9500, 256)])
def test_project_large_scales(m, dtype, n, k):
    """Scales up to 2^113 with rows whose results are finite, and scales of both
    ends in one plan.  Results among the subnormals: half their spacing for each
    sum, and for the output's own rounding."""
    g = gen(420)
    more = (k / 32 + 20) * 2.0 ** -149 + (2.0 ** -134 if dtype == "bf16" else 0.0)
    codes, _, _ = make_weights(n, k, "mxfp4", 32, None, False, 421)
    x = normal((4, k), DT[dtype], 422)
    mixed = x * torch.tensor([1e-18, 1e-8, 2.0 ** -20, 2.0 ** -12], device="cuda")[:, None].to(x.dtype)
    for lo, hi in ((236, 237), (230, 240), (1, 240), (238, 239)):
        s = torch.randint(lo, hi, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
        check_project(m, dtype, "mxfp4", codes, s, None, [mixed], more=more)
    s = torch.full((n, k // 32), 5, dtype=torch.uint8, device="cuda")
    s[0] = 230   # one output's are large, the others' results among the subnormals
    check_project(m, dtype, "mxfp4", codes, s, None, [mixed, x * 1e-3], more=more)
    for sd in ("f32", "bf16"):
        s = ((torch.rand((n, k // 32), device="cuda", generator=g) + 0.5) * 2.0 ** 108)
        s[:, ::2] *= 2.0 ** -200
        s = (s * torch.where(torch.rand((n, k // 32), device="cuda", generator=g) < 0.5, -1.0, 1.0)).to(DT[sd])
        z = torch.randint(0, 16, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
        for zeros in (None, z):
            check_project(m, dtype, "int4", codes, s, zeros, [mixed], scale_dtype=sd, more=more)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-100, -112, -120, -126, -132])
def test_project_rows_of_tiny_numbers(m, dtype, power):
    """Rows whose largest number is near or among fp32's subnormals.  x enters as
    fp16 after a factor of at most 2^126: halves of fp16's smallest step, 2^-25,
    are 2^-151 of x, for each weight; with scales of 2^100 the results are usual."""
    n, k = 130, 512
    x = (normal((4, k), torch.float64, 430) * 2.0 ** power).to(DT[dtype])
    for fmt in ("int4", "mxfp4"):
        codes, s, _ = make_weights(n, k, fmt, 32, "f32", False, 431)
        s = torch.full_like(s, 227 if fmt == "mxfp4" else 2.0 ** 100)
        full = R.weights(codes, s, None, fmt, 32)
        check_project(m, dtype, fmt, codes, s, None, [x], more=2.0 ** -151 * full.abs().sum(1))


# ------------------------------------------------- outputs that share storage

def test_outputs_that_share_storage_lazily(m):
    """A lazily cloned output is given storage of its own before it is written."""
    r, pos = m.Rope(64), i32([3, 9])
    x = normal((2, 2, 64), torch.float32, 440)
    want = m.rope(x, pos, r, out=torch.empty_like(x))
    base = torch.full_like(x, 3.0)
    out = torch._lazy_clone(base)
    m.rope(x, pos, r, out=out)
    assert (base == 3.0).all() and torch.equal(out, want)
    again = torch._lazy_clone(x)   # in place
    before = x.clone()
    m.rope(again, pos, r)
    assert torch.equal(x, before) and torch.equal(again, want)
    plan = m.Projection(64, 64, group=32)
    plan.pack(*make_weights(64, 64, "int4", 32, "bf16", False, 441))
    xb = normal((2, 64), torch.bfloat16, 442)
    base = torch.full((2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    y = plan.step(xb, torch._lazy_clone(base))
    assert (base == 3.0).all() and torch.equal(y, plan.step(xb, torch.empty_like(base)))
    cache = make_cache(m, 2, 2, 16, 64, 443)
    attn = m.AttnPlan(4, 2, 64, 16, 2, 1, 2)
    q = normal((1, 1, 4, 64), torch.bfloat16, 444)
    base, lbase = torch.full_like(q, 3.0), torch.full((1, 1, 4), 3.0, device="cuda")
    out, lse = torch._lazy_clone(base), torch._lazy_clone(lbase)
    attn.attend(cache, q, i32([20]), i32([[1, 0]]), out, lse=lse)
    assert (base == 3.0).all() and (lbase == 3.0).all() and not (out == 3.0).all() and not (lse == 3.0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk", [(64, 8, 8), (64, 64, 4), (128, 40, 8), (128, 24, 2), (256, 16, 8)])
def test_attend_one_token_is_exact(m, dtype, d, hq, hk):
    """Its probability is 1 whatever its logit: the output is the value, the
    product of its code and scale in fp32, also where that is a tie between two
    bf16 numbers (scales of 8 bits make many)."""
    for seed in range(6):
        cache = make_cache(m, 4, hk, 16, d, 450 + seed)
        cache.v_scale.copy_(cache.v_scale.bfloat16())
        q = normal((2, 1, hq, d), DT[dtype], 460 + seed) * 2.0 ** (seed - 2)
        plan = m.AttnPlan(hq, hk, d, 16, 4, 2, 2, dtype=dtype)
        out = plan.attend(cache, q, i32([1, 1]), i32([[0, 0], [3, 0]]), torch.empty_like(q))
        v = cache.v[[0, 3], :, 0].float() * cache.v_scale[[0, 3]][:, :, None]
        assert torch.equal(out[:, 0], v.repeat_interleave(hq // hk, 1).to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 24, 2), (256, 4, 2)])
def test_attend_smallest_scales(m, dtype, d, hq, hk):
    """Page scales from 2^-126 up beside usual ones that other rows see.  Beyond
    the usual bound: half of fp32's smallest step for each group of 16 tokens and
    the joins, the output's own smallest half step, and for bf16 rows a scale in
    steps of 2^-134, half of one times codes up to 448."""
    page, length = 64, 700
    pages = -(-length // page)
    cache = make_cache(m, pages + 1, hk, page, d, 470)
    cache.v_scale[:pages] = cache.v_scale[:pages] * 2.0 ** -119
    cache.v_scale[2] = 2.0 ** -126
    q = normal((2, 1, hq, d), DT[dtype], 471)
    table = [list(range(pages)), [pages] + [-1] * (pages - 1)]
    plan = m.AttnPlan(hq, hk, d, page, pages + 1, 2, pages, dtype=dtype)
    out = plan.attend(cache, q, i32([length, 50]), i32(table), torch.empty_like(q))
    want, _, ob, _ = R.attend(cache, q, [length, 50], table, [1, 1], page, 1 / math.sqrt(d))
    more = (length / 16 + 40) * 2.0 ** -150
    if dtype == "bf16":
        more += 2.0 ** -134 + 448 * 2.0 ** -135
    within(out, want, ob + more)


# ------------------------------------------------------- the largest calls

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_most_rows_and_most_sequences(m, dtype, d):
    """128 query heads a key head with 8 new tokens each (1024 rows of one item),
    and 4096 sequences, padding among them, in one call."""
    check_attend(m, dtype, [300, 9, 65], [8, 8, 3], 8, 128, 1, d, 16)
    lens = [1 + (7 * i) % 40 for i in range(4096)]
    new = [0 if i % 9 == 4 else 1 + i % 2 for i in range(4096)]
    check_attend(m, dtype, lens, new, 2, 2, 1, d, 16, window=30)
    check_append(m, dtype, lens, [min(n, ln) for n, ln in zip(new, lens)], 2, 1, d, 16, m.Rope(d))
