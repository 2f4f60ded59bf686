"""The attention half's operators on the GPU against plain fp64 statements
(attn_reference.py) at the sizes, masks, strides and orders where they can go
wrong, their refusals, and a run of them together with the FFN half-layer."""

import math

import pytest
import torch

from tests import attn_reference as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def m():
    import moe_decode_layer_sm_b200
    return moe_decode_layer_sm_b200


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, seed):
    return torch.empty(shape, device="cuda").normal_(generator=gen(seed)).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def within(got, want, bound):
    """Every finite value within its bound, the others equal."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin].nan_to_num(7.0), want[~fin].nan_to_num(7.0))
    over = (got - want).abs()[fin] - bound[fin]
    assert not over.numel() or over.max() <= 0, (over.max().item(), (got - want).abs()[fin].max().item())


# --------------------------------------------------------------------- rotary

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("head_dim,rot,offset,il", [
    (128, 128, 0, False), (128, 128, 0, True), (128, 64, 64, False), (64, 32, 32, True), (256, 256, 0, False),
    (128, 6, 10, False), (128, 6, 10, True), (2, 2, 0, True), (80, 24, 8, False), (100, 100, 0, False),
    (1024, 256, 512, False), (34, 16, 16, True)])
@pytest.mark.parametrize("tokens,heads", [(1, 1), (3, 5), (301, 3)])
def test_rope(m, dtype, head_dim, rot, offset, il, tokens, heads):
    r = m.Rope(rot, offset=offset, interleaved=il, scaling="yarn", factor=4.0)
    x = normal((tokens, heads, head_dim), DT[dtype], 1)
    pos = torch.randint(0, 1 << 20, (tokens,), dtype=torch.int32, device="cuda", generator=gen(2))
    pos[0] = 10_000_000
    for transpose in (False, True):
        want, bound = R.rotate(x, pos, r, transpose), R.rotate_bound(x, r, DT[dtype])
        bound = torch.where(bound > 0, bound + R.half_step(DT[dtype]) * want.abs(), bound)
        out = torch.full_like(x, 9.0)
        assert m.rope(x, pos, r, out=out, transpose=transpose) is out
        within(out, want, bound)
        y = x.clone()
        m.rope(y, pos, r, transpose=transpose)   # in place
        assert torch.equal(y, out)


def test_rope_strides_padding_and_alignment(m):
    r = m.Rope(64)
    big = normal((7, 9, 128), torch.bfloat16, 3)
    pos = i32([5, -1, 0, 77, -2 ** 31, 2 ** 31 - 1, 4])
    fused = normal((7, 4 * 64 + 2 * 64), torch.bfloat16, 4)   # q and k of a fused projection
    q = fused[:, :256].view(7, 4, 64)
    for x in (big[:, 1:8:2, 32:96], big[:, :, 3:67], big.transpose(0, 1)[:7, :7, :64], q):
        out = torch.full(x.shape, 3.0, device="cuda", dtype=x.dtype)
        m.rope(x, pos, r, out=out)
        live = pos >= 0
        live[5] = False   # the angle itself is off by 2^-53 of 3e8 turns there: only that it is written
        want, bound = R.rotate(x, pos, r), R.rotate_bound(x, r, x.dtype)
        within(out[live], want[live], (bound + R.half_step(x.dtype) * want.abs())[live])
        assert torch.equal(out[[1, 4]], torch.full_like(out[[1, 4]], 3.0))
        assert torch.isfinite(out[5]).all() and (out[5] != 3.0).any()
    before = fused.clone()
    m.rope(q, pos, r)   # in place inside the fused rows: the rest stays
    assert torch.equal(fused[:, 256:], before[:, 256:])
    assert not torch.equal(fused[0, :256], before[0, :256])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,d,rot,offset,il", [(1, 128, 128, 0, False), (3, 64, 64, 0, True), (2, 128, 64, 64, False),
                                                   (5, 80, 6, 10, True), (7, 256, 256, 0, False)])
def test_rope_many_tokens(m, dtype, heads, d, rot, offset, il):
    """Several tokens a CTA, padding among them, a last CTA that is not full."""
    tokens = 10007
    r = m.Rope(rot, offset=offset, interleaved=il)
    x = normal((tokens, heads, d), DT[dtype], 9)
    pos = torch.randint(-1000, 100000, (tokens,), dtype=torch.int32, device="cuda", generator=gen(10))
    out = torch.full_like(x, 3.0)
    m.rope(x, pos, r, out=out)
    live = pos >= 0
    want, bound = R.rotate(x, pos, r), R.rotate_bound(x, r, DT[dtype])
    bound = torch.where(bound > 0, bound + R.half_step(DT[dtype]) * want.abs(), bound)
    within(out[live], want[live], bound[live])
    assert (out[~live] == 3.0).all()
    m.rope(x, pos, r)
    assert torch.equal(x[live], out[live])


def test_rope_far_strides(m):
    """Rows further apart than 32 bits count."""
    store = torch.zeros(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((2, 3, 64), (2 ** 31, 64, 1))
    x.copy_(normal((2, 3, 64), torch.bfloat16, 14))
    r, pos = m.Rope(64), i32([7, 900])
    want, bound = R.rotate(x, pos, r), R.rotate_bound(x, r, x.dtype)
    out = torch.empty(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    m.rope(x, pos, r, out=out)
    within(out, want, bound + R.half_step(x.dtype) * want.abs())
    m.rope(x, pos, r)
    assert torch.equal(x, out)


def test_rope_gradient(m):
    """transpose is the gradient: <rope(x), y> = <x, rope^T(y)>, and the
    difference of the inner product along a direction is the same."""
    r = m.Rope(32, offset=16, interleaved=True, scaling="ntk", factor=2.0, attn_factor=1.25)
    x, y, d = (normal((6, 3, 64), torch.float32, s) for s in (5, 6, 7))
    pos = i32([0, 1, 9, 100, 4095, 100000])
    f = lambda t: (m.rope(t, pos, r, out=torch.empty_like(t)).double() * y.double()).sum()  # noqa: E731
    g = m.rope(y, pos, r, out=torch.empty_like(y), transpose=True)
    # the map is linear: the difference over any step is the derivative; each value is off by 12 x 2^-24 of its pair
    tol = 12 * 2.0 ** -24 * 1.25 * 2 * (x.abs().sum() + d.abs().sum()).item() * y.abs().max().item()
    assert abs(((f(x + d) - f(x)) - (g.double() * ((x + d).double() - x.double())).sum()).item()) <= 2 * tol
    z = normal((6, 3, 64), torch.float32, 8)
    one = m.Rope(32, offset=16)
    back = m.rope(m.rope(z, pos, one, out=torch.empty_like(z)), pos, one, out=torch.empty_like(z), transpose=True)
    assert (back - z).abs().max() <= 24 * 2.0 ** -24 * 2 * z.abs().max()


def test_rope_empty_and_refusals(m):
    r = m.Rope(64)
    x = normal((2, 2, 64), torch.float32, 1)
    pos = i32([0, 1])
    m.rope(x[:0], pos[:0], r)
    m.rope(x[:, :0], pos, r)
    for bad in (lambda: m.rope(x, pos.long(), r), lambda: m.rope(x, pos[:1], r), lambda: m.rope(x.half(), pos, r),
                lambda: m.rope(x, pos, r, out=x.bfloat16()), lambda: m.rope(x.cpu(), pos, r),
                lambda: m.rope(x.transpose(1, 2), pos, m.Rope(2)), lambda: m.rope(x[0], pos, r)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: m.rope(x, pos, r, out=x.flip(0)[:1].expand(2, 2, 64)), lambda: m.rope(x[:, :, :62], pos, r),
                lambda: m.rope(x[:1].expand(2, 2, 64), pos, r)):
        with pytest.raises(m.MonoError):
            bad()


# ------------------------------------------------------------------ the cache

def make_cache(m, pages, heads, page, d, seed, fill=True):
    c = m.KVCache.empty(pages, heads, page, d)
    if fill:
        for t, s, i in ((c.k, c.k_scale, 0), (c.v, c.v_scale, 1)):
            x = normal(tuple(t.shape), torch.float32, seed + i)
            x *= torch.rand((pages, heads, 1, 1), device="cuda", generator=gen(seed + 7)) + 0.25
            sc = x.abs().amax((2, 3)) / 448
            t.copy_((x / sc[:, :, None, None]).clamp(-448, 448).to(R.FP8))
            s.copy_(sc)
    return c


def make_table(lens, page, cols, pages, seed, fill=-1):
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    rows, at = [], 0
    for n in lens:
        k = -(-max(n, 0) // page)
        rows.append(order[at:at + k] + [fill] * (cols - k))
        at += k
    return rows


def check_append(m, dtype, lens, n_new, width, heads, d, page, rope, cache=None, k=None, v=None, seed=11, pass_new=True):
    seqs = len(lens)
    cols = max(-(-max(n, 1) // page) for n in lens) + 1
    pages = sum(-(-max(n, 0) // page) for n in lens) + 3
    table = make_table(lens, page, cols, pages, seed, fill=-7)
    cache = cache or make_cache(m, pages, heads, page, d, seed)
    k = normal((seqs, width, heads, d), DT[dtype], seed + 2) if k is None else k
    v = normal((seqs, width, heads, d), DT[dtype], seed + 3) * 2 if v is None else v
    plan = m.AttnPlan(heads, heads, d, page, pages, seqs, cols, max_new=min(width, 8), dtype=dtype)
    want = R.append(cache, k, v, lens, table, n_new, rope, page)
    plan.append(cache, k, v, i32(lens), i32(table), rope=rope, n_new=i32(n_new) if pass_new else None)
    assert plan.query_error()[0] == 0
    for name in ("k", "v"):
        got = getattr(cache, name).double()
        same = (got == want[name]) | (torch.isnan(got) & torch.isnan(want[name]))
        assert same.all(), (name, (~same).sum().item())
        assert torch.equal(getattr(cache, name + "_scale"), want[name + "_scale"]), name
    plan.close()
    return cache


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_ragged(m, dtype, d, page):
    """First tokens, page borders, several pages, padding sequences, sequences shorter than their rows."""
    lens = [1, page, page + 1, 3 * page - 1, 77, 2 * page + 3, 5, 3]
    new = [1, page, 2, 2 * page + 5, 0, 7, -1, 9]
    width = 2 * page + 5
    new = [min(n, width) for n in new]
    for rope in (None, m.Rope(d), m.Rope(d // 2, offset=d // 2, interleaved=True, scaling="linear", factor=3.0)):
        check_append(m, dtype, lens, new, width, 3, d, page, rope)


@pytest.mark.parametrize("rot,offset,il", [(6, 10, False), (10, 2, True), (24, 4, False), (48, 8, True), (128, 0, True)])
def test_append_odd_rotations(m, rot, offset, il):
    check_append(m, "bf16", [40, 9, 64], [40, 3, 2], 40, 2, 128, 32, m.Rope(rot, offset=offset, interleaved=il))
    check_append(m, "f32", [40, 9, 64], [40, 3, 2], 40, 2, 128, 32, m.Rope(rot, offset=offset, interleaved=il))


@pytest.mark.parametrize("heads", [1, 2, 5, 8, 12])
def test_append_decode_and_many_sequences(m, heads):
    """One token a sequence; enough of them that heads share a CTA."""
    lens = [1 + 37 * i for i in range(40)]
    check_append(m, "bf16", lens, [1] * 40, 1, heads, 128, 64, m.Rope(128), pass_new=False)


def test_append_long_prompt(m):
    check_append(m, "bf16", [3001, 1023], [3001, 1023], 3001, 8, 128, 64, m.Rope(128, theta=500000.0))


def test_append_strides_alignment_and_values(m):
    fused = normal((3, 5, 2 * 4 * 64 + 3), torch.float32, 21)
    k, v = fused[..., 1:257].view(3, 5, 4, 64), fused[..., 257:513].view(3, 5, 4, 64)
    check_append(m, "f32", [5, 21, 16], [5, 4, 5], 5, 4, 64, 16, m.Rope(64), k=k, v=v)
    k, v = (normal((3, 4, 5, 64), torch.bfloat16, s).transpose(1, 2) for s in (22, 23))
    check_append(m, "bf16", [5, 21, 16], [5, 4, 5], 5, 4, 64, 16, m.Rope(64), k=k, v=v)
    # rows of zeros, tiny and huge values, infinities and NaN; values on the borders between codes
    v = normal((1, 16, 8, 64), torch.float32, 24)
    v[0, :, 0] = 0
    v[0, :, 1] *= 1e-39
    v[0, :, 2] *= 1e37
    v[0, 3, 3, 5], v[0, 4, 3, 6], v[0, 5, 3, 7] = math.inf, -math.inf, math.nan
    v[0, :, 4] = math.inf
    v[0, :, 5] = torch.arange(16 * 64, device="cuda").view(16, 64) * 0.4375
    v[0, :, 6] = torch.arange(16 * 64, device="cuda").view(16, 64).float() / 1023 * 0.1
    v[0, :, 7] = 448.0 * 2.0 ** -torch.arange(64, device="cuda").float()
    check_append(m, "f32", [16], [16], 16, 8, 64, 16, None, v=v)
    check_append(m, "f32", [13], [13], 16, 8, 64, 16, None, k=v, v=v.flip(1))


def test_append_codes_and_borders_between_them(m):
    """Values that lie exactly on codes and on borders, and next to them, at many
    scales: the quotient's own rounding must not move one."""
    g = gen(190)
    heads = 64
    s = torch.randint(1 << 12, 1 << 13, (heads,), device="cuda", generator=g).double() * 2.0 ** -20   # 13 bits: exact products
    n = torch.arange(16 * 64, device="cuda")
    steps = torch.cat([n[:600], torch.randint(0, 448 * 1024, (16 * 64 - 600,), device="cuda", generator=g) & ~0x1FF])
    v = (s[:, None] * (steps.double() * 2.0 ** -10)).float()
    assert torch.equal(v.double(), s[:, None] * (steps.double() * 2.0 ** -10))
    v = torch.where(n % 3 == 0, v, torch.where(n % 3 == 1, torch.nextafter(v, v + 1), torch.nextafter(v, v - 1)))
    v = torch.where(n % 2 == 0, v, -v)
    v[:, 777] = 448.0 * s.float()
    v = v.view(heads, 16, 64).transpose(0, 1)[None].contiguous()
    check_append(m, "f32", [16], [16], 16, heads, 64, 16, None, k=v, v=v.flip(1))


def test_append_token_by_token_keeps_the_page(m):
    """A page filled in many calls: the scale grows with the values, the older
    codes follow, and the slots behind the sequence keep their bytes."""
    d, page, heads = 64, 16, 2
    cache = make_cache(m, 4, heads, page, d, 31)
    plan = m.AttnPlan(heads, heads, d, page, 4, 1, 4)
    rope = m.Rope(d)
    table = [[2, 0, 3, 1]]
    for t in range(40):
        k, v = (normal((1, 1, heads, d), torch.bfloat16, 100 + 2 * t + i) * (1 + 0.2 * t) for i in (0, 1))
        want = R.append(cache, k, v, [t + 1], table, [1], rope, page)
        plan.append(cache, k, v, i32([t + 1]), i32(table), rope=rope)
        for name in ("k", "v"):
            assert torch.equal(getattr(cache, name).double(), want[name])
            assert torch.equal(getattr(cache, name + "_scale"), want[name + "_scale"])


# ------------------------------------------------------------------ attention

def check_attend(m, dtype, lens, n_new, width, hq, hk, d, page, window=0, scale=0.0, seed=41, lse=True, spoil=True,
                 max_new=None, q=None, plan=None):
    seqs = len(lens)
    cols = max(-(-max(n, 1) // page) for n in lens) + 1
    pages = sum(-(-max(n, 0) // page) for n in lens) + 3
    table = make_table(lens, page, cols, pages, seed, fill=2 ** 30)
    cache = make_cache(m, pages, hk, page, d, seed)
    q = normal((seqs, width, hq, d), DT[dtype], seed + 5) * 2 if q is None else q
    sc = scale or 1 / math.sqrt(d)
    want, wl, ob, lb = R.attend(cache, q, lens, table, n_new, page, sc, window)
    if spoil:   # what no row sees holds NaN codes; pages in no table NaN scales too
        for s, row in enumerate(table):
            n, pos0 = lens[s], max(0, lens[s] - max(n_new[s], 0))
            lo = max(0, pos0 + 1 - window) if window else 0
            for i, pg in enumerate(row[:-(-max(n, 0) // page)]):
                for t in (cache.k, cache.v):
                    u = t.view(torch.uint8)
                    if (i + 1) * page > n:
                        u[pg, :, n - i * page:] = 0x7F
                    if i * page < lo:
                        u[pg, :, :max(0, min(page, lo - i * page))] = 0xFF
                if window and (i + 1) * page <= lo:
                    row[i] = -5   # before every window: any entry
        used = {p for row in table for p in row}
        free = [p for p in range(pages) if p not in used]
        cache.k_scale[free], cache.v_scale[free] = math.nan, math.nan
    plan = plan or m.AttnPlan(hq, hk, d, page, pages, seqs, cols, max_new=max_new or width, dtype=dtype, scale=scale,
                              window=window)
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device="cuda")
    ls = torch.full(q.shape[:3], 5.0, device="cuda") if lse else None
    args = (cache, q, i32(lens), i32(table), out)
    plan.attend(*args, lse=ls, n_new=i32(n_new))
    assert plan.query_error()[0] == 0
    dead = torch.tensor([[j >= max(n, 0) for j in range(width)] for n in n_new], device="cuda")
    assert (out[dead] == 5.0).all()
    live = ~dead
    within(out[live], want[live], ob[live])
    if lse:
        assert (ls[dead] == 5.0).all()
        within(ls[live], wl[live], lb[live])
    first = out.clone()
    for _ in range(3):   # the same bits every time, whatever order the CTAs arrive in
        plan.attend(*args, lse=ls, n_new=i32(n_new))
        assert torch.equal(out.view(torch.uint8), first.view(torch.uint8))
    return plan


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("hq,hk,width", [(1, 1, 1), (5, 1, 1), (8, 2, 3), (16, 2, 8), (24, 2, 8), (128, 1, 1)])
def test_attend(m, dtype, d, page, hq, hk, width):
    lens = [1, page, page + 1, 4 * page - 1, 200, 333, 2, 0]
    new = [1, width, width, max(1, width - 1), 0, width, width, width]   # 2, 0: rows that see nothing
    check_attend(m, dtype, lens, new, width, hq, hk, d, page)


@pytest.mark.parametrize("window", [1, 7, 16, 64, 100, 1000])
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (256, "bf16")])
def test_attend_window(m, window, d, dtype):
    check_attend(m, dtype, [1, 65, 300, 777, 3], [1, 4, 4, 2, 4], 4, 10, 2, d, 16, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 4), (128, 10, 2), (256, 8, 1)])
def test_attend_long(m, dtype, d, hq, hk):
    check_attend(m, dtype, [9001, 3, 5003], [1, 1, 1], 1, hq, hk, d, 64, spoil=False)


def test_attend_many_sequences(m):
    check_attend(m, "bf16", [1 + 13 * i for i in range(130)], [1] * 130, 1, 5, 1, 128, 16)
    check_attend(m, "f32", [7] * 200, [2] * 200, 2, 4, 4, 64, 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,hq,hk,width,window", [(64, 4, 2, 1, 0), (64, 16, 2, 3, 40), (128, 10, 2, 1, 0), (128, 8, 2, 4, 0),
                                                  (256, 4, 2, 2, 70), (256, 2, 2, 1, 0)])
def test_attend_more_items_than_sms(m, dtype, d, hq, hk, width, window):
    """Narrow CTAs: several items each, items over several CTAs, padding among them."""
    lens = [1 + (37 * i) % 600 for i in range(90)]
    new = [0 if i % 11 == 5 else 1 + i % width for i in range(90)]
    check_attend(m, dtype, lens, new, width, hq, hk, d, 16, window=window)


def test_attend_short_tables(m):
    """No sequence longer than a narrow CTA's round."""
    check_attend(m, "bf16", [1, 16, 9], [1, 1, 1], 1, 40, 8, 128, 16)
    check_attend(m, "f32", [1, 3, 2], [1, 3, 3], 3, 8, 8, 64, 16)
    check_attend(m, "bf16", [1], [1], 1, 1, 1, 256, 16)


def test_attend_large_logits_and_scales(m):
    """Logits of hundreds: the running maximum carries the sums; a scale of its own."""
    q = normal((2, 1, 8, 128), torch.bfloat16, 3) * 40
    check_attend(m, "bf16", [500, 900], [1, 1], 1, 8, 2, 128, 64, q=q, scale=0.125)
    q = normal((2, 1, 8, 128), torch.float32, 3) * 1e-30
    check_attend(m, "f32", [500, 900], [1, 1], 1, 8, 2, 128, 64, q=q)
    q = torch.zeros(2, 1, 8, 128, device="cuda")
    check_attend(m, "f32", [500, 900], [1, 1], 1, 8, 2, 128, 64, q=q)
    q = normal((2, 1, 8, 128), torch.float32, 3) * 1e-3
    q[..., 0] = 0.5   # small elements beside a large one
    check_attend(m, "f32", [500, 900], [1, 1], 1, 8, 2, 128, 64, q=q)


def test_attend_one_plan_many_widths(m):
    lens = [100, 50]
    plan = m.AttnPlan(40, 8, 128, 64, 6, 2, 3, max_new=8)
    for width in (1, 8, 2, 5):
        check_attend(m, "bf16", lens, [width] * 2, width, 40, 8, 128, 64, plan=plan)


def test_attend_strides_alignment_and_outputs_beside(m):
    d, hq, hk, page = 64, 6, 2, 16
    cache = make_cache(m, 8, hk, page, d, 51)
    table, lens = [[1, 2, 3], [4, 5, 6]], [40, 17]
    plan = m.AttnPlan(hq, hk, d, page, 8, 2, 3, max_new=2, dtype="bf16")
    store = normal((2, 2, hq * d + 2 * hk * d + 1), torch.bfloat16, 52)
    for q in (store[..., :hq * d].view(2, 2, hq, d), store[..., 1:1 + hq * d].view(2, 2, hq, d),
              normal((hq, 2, 2, d), torch.bfloat16, 53).permute(1, 2, 0, 3), normal((1, 1, hq, d), torch.bfloat16, 5).expand(2, 2, hq, d)):
        want, _, ob, _ = R.attend(cache, q, lens, table, [2, 2], page, 1 / math.sqrt(d))
        for kind in range(3):
            big = torch.full((hq, 2, 2, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
            out = big.permute(1, 2, 0, 3)[..., (0, 8, 3)[kind]:][..., :d]
            keep = torch.ones_like(big, dtype=torch.bool)
            keep[..., (0, 8, 3)[kind]:(0, 8, 3)[kind] + d] = False
            plan.attend(cache, q, i32(lens), i32(table), out)
            within(out, want, ob)
            assert (big[keep] == 7.0).all()


def test_attend_nan_reaches_only_rows_that_see_it(m):
    """A NaN among the drafted tokens' values: the rows before it stay clean."""
    d, page, hq, hk = 128, 64, 4, 2
    for dtype in ("bf16", "f32"):
        for length in (70, 64, 9):
            cache = make_cache(m, 3, hk, page, d, 61)
            table = [[2, 0]]
            q = normal((1, 4, hq, d), DT[dtype], 62)
            at = length - 2   # the third of four new tokens
            clean = make_cache(m, 3, hk, page, d, 61)
            cache.v.view(torch.uint8)[table[0][at // page], 1, at % page, 5] = 0x7F
            plan = m.AttnPlan(hq, hk, d, page, 3, 1, 2, max_new=4, dtype=dtype)
            out = torch.empty_like(q)
            plan.attend(cache, q, i32([length]), i32(table), out)
            want, _, ob, _ = R.attend(clean, q, [length], table, [4], page, 1 / math.sqrt(d))
            hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
            hit[0, 2:, 2:, 5] = True
            assert torch.equal(torch.isnan(out), hit)
            assert ((out.double() - want).abs() <= ob)[~hit].all()


def test_attend_far_offsets(m):
    """A cache of more than 2^32 bytes: pages at its end."""
    pages, hk, page, d = 70000, 8, 64, 128
    cache = m.KVCache.empty(pages, hk, page, d)
    small = make_cache(m, 4, hk, page, d, 71)
    ids = [pages - 1, 3, pages - 2, 65537]
    for name in ("k", "v", "k_scale", "v_scale"):
        src, dst = getattr(small, name), getattr(cache, name)
        if src.dtype == R.FP8:
            src, dst = src.view(torch.uint8), dst.view(torch.uint8)
        for i, p in enumerate(ids):
            dst[p] = src[i]
    q = normal((1, 2, 16, d), torch.bfloat16, 72)
    plan = m.AttnPlan(16, hk, d, page, pages, 1, 4, max_new=2)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    plan.attend(cache, q, i32([250]), i32([ids]), out)
    near = m.AttnPlan(16, hk, d, page, 4, 1, 4, max_new=2)
    near.attend(small, q, i32([250]), i32([[0, 1, 2, 3]]), ref)
    assert torch.equal(out, ref)
    k, v = (normal((1, 2, hk, d), torch.bfloat16, s) * 3 for s in (73, 74))
    plan.append(cache, k, v, i32([252]), i32([ids]), rope=m.Rope(d))
    near.append(small, k, v, i32([252]), i32([[0, 1, 2, 3]]), rope=m.Rope(d))
    for name in ("k", "v"):
        assert torch.equal(getattr(cache, name)[ids].view(torch.uint8), getattr(small, name).view(torch.uint8))


def test_bad_indices_are_recorded_and_touch_nothing(m):
    d, page, hk = 64, 16, 2
    cache = make_cache(m, 4, hk, page, d, 81)
    plan = m.AttnPlan(4, hk, d, page, 4, 2, 2, max_new=2)
    q = normal((2, 2, 4, d), torch.bfloat16, 82)
    out = torch.empty_like(q)
    k = normal((2, 2, hk, d), torch.bfloat16, 83)
    good = i32([[0, 1], [2, 3]])
    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")}

    def bad(what, seq, value, lens=(20, 20), table=good, new=(2, 2)):
        plan.attend(cache, q, i32(lens), table, out, n_new=i32(new))
        rc, st = plan.query_error()
        assert (rc, st.what, st.seq, st.value) == (-9, what, seq, value)
        assert plan.query_error()[0] == 0

    bad(1, 1, 4, table=i32([[0, 1], [2, 4]]))
    bad(1, 0, -1, table=i32([[-1, 1], [2, 3]]))
    bad(2, 1, 33, lens=(20, 33))
    bad(2, 0, -4, lens=(-4, 20))
    bad(3, 1, 3, new=(2, 3))
    # the tokens of a bad page are left out, the others count
    plan.attend(cache, q, i32([20, 20]), i32([[0, 9], [2, 3]]), out)
    want, _, ob, _ = R.attend(cache, q, [16, 20], [[0, 1], [2, 3]], [1, 2], page, 1 / math.sqrt(d))
    within(out[1], want[1], ob[1])
    assert plan.query_error()[0] == -9
    plan.append(cache, k, k, i32([18, 40]), i32([[0, 77], [2, 3]]))
    rc, st = plan.query_error()
    assert rc == -9 and st.what in (1, 2)
    for n, t in before.items():
        now = getattr(cache, n)
        assert torch.equal(now.view(torch.uint8) if t.dtype == R.FP8 else now, t.view(torch.uint8) if t.dtype == R.FP8 else t), n


def test_attn_refusals(m):
    plan = m.AttnPlan(4, 2, 64, 16, 4, 2, 2, max_new=2)
    cache = m.KVCache.empty(4, 2, 16, 64)
    q = normal((2, 2, 4, 64), torch.bfloat16, 1)
    kv = normal((2, 2, 2, 64), torch.bfloat16, 2)
    lens, table, out = i32([3, 4]), i32([[0, 1], [2, 3]]), torch.empty_like(q)
    for bad in (lambda: plan.attend(cache, q.float(), lens, table, out), lambda: plan.attend(cache, q[:, :, :2], lens, table, out),
                lambda: plan.attend(cache, q, lens.long(), table, out), lambda: plan.attend(cache, q, lens, table[:, :1], out),
                lambda: plan.attend(cache, q, lens, table, out[:1]), lambda: plan.attend(cache, q.cpu(), lens, table, out),
                lambda: plan.attend(cache, q, lens, table, out, n_new=i32([1])),
                lambda: plan.attend(cache, q, lens, table, out, lse=torch.empty(2, 2, 4, 1, device="cuda")),
                lambda: plan.attend(m.KVCache.empty(5, 2, 16, 64), q, lens, table, out),
                lambda: plan.append(cache, kv, kv[:, :1], lens, table), lambda: plan.append(cache, q, q, lens, table),
                lambda: m.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale.double()),
                lambda: m.KVCache(cache.k, cache.v[:, :, :8], cache.k_scale, cache.v_scale),
                lambda: m.KVCache(cache.k.float(), cache.v, cache.k_scale, cache.v_scale)):
        with pytest.raises(ValueError):
            bad()
    three = q[:, :1].expand(2, 3, 4, 64).contiguous()
    for bad in (lambda: plan.attend(cache, three, lens, table, torch.empty_like(three)),
                lambda: plan.attend(cache, q, lens, table, q), lambda: plan.attend(cache, q, lens, table, out[:1].expand(2, 2, 4, 64)),
                lambda: plan.attend(cache, torch.cat([q, q]), i32([1] * 4), i32([[0, 1]] * 4), torch.cat([q, q])),
                lambda: plan.append(cache, kv, kv, lens, table, rope=m.Rope(64, offset=2))):
        with pytest.raises(m.MonoError):
            bad()
    plan.attend(cache, q[:0], lens[:0], table[:0], out[:0])
    plan.attend(cache, q[:, :0], lens, table, out[:, :0])
    plan.append(cache, kv[:, :0], kv[:, :0], lens, table)
    assert plan.query_error()[0] == 0 and plan.info()["grid"] > 0


# ---------------------------------------------------------- 4-bit projections

def make_weights(n, k, fmt, group, scales, zeros, seed):
    g = gen(seed)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    if fmt == "mxfp4":
        return codes, torch.randint(110, 125, (n, k // group), dtype=torch.uint8, device="cuda", generator=g), None
    s = (torch.rand((n, k // group), device="cuda", generator=g) + 0.1).to(DT[scales])
    z = torch.randint(0, 16, (n, k // group), dtype=torch.uint8, device="cuda", generator=g) if zeros else None
    return codes, s, z


KINDS = [("int4", 128, "bf16", False), ("int4", 32, "f32", True), ("int4", 64, "bf16", True), ("int4", 96, "f32", False),
         ("mxfp4", 32, "bf16", False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,group,scales,zeros", KINDS)
@pytest.mark.parametrize("n,groups", [(1, 1), (63, 3), (64, 2), (200, 17), (1003, 40), (20000, 5)])
def test_project(m, dtype, fmt, group, scales, zeros, n, groups):
    k = group * groups
    w = make_weights(n, k, fmt, group, scales, zeros, 91)
    plan = m.Projection(n, k, fmt=fmt, group=group, scale_dtype=scales, zeros=zeros, dtype=dtype)
    plan.pack(*w)
    full = R.weights(*w, fmt, group)
    for rows in (1, 2, 3, 5, 8):
        x = normal((rows, k), DT[dtype], 92 + rows)
        y = torch.full((rows, n), 7.0, dtype=DT[dtype], device="cuda")
        assert plan.step(x, y) is y
        within(y, *R.project(x, full))
        again = torch.empty_like(y)
        plan.step(x, again)
        assert torch.equal(y, again)
    plan.step(x[:0], y[:0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_project_strides_alignment_and_values(m, dtype):
    n, k = 130, 512
    w = make_weights(n, k, "int4", 128, "f32", True, 93)
    plan = m.Projection(n, k, group=128, scale_dtype="f32", zeros=True, dtype=dtype)
    plan.pack(*w)
    full = R.weights(*w, "int4", 128)
    big = normal((6, 2 * k + 3), DT[dtype], 94)
    for x in (big[::2, :k], big[:3, 1:1 + k], big[:1, :k].expand(3, k), big[:3, 3:3 + k] * 1e-30, big[:3, :k] * 1e30):
        store = torch.full((3, n + 5), 7.0, dtype=DT[dtype], device="cuda")
        y = store[:, 1:1 + n]
        plan.step(x, y)
        within(y, *R.project(x, full))
        assert (store[:, 0] == 7).all() and (store[:, 1 + n:] == 7).all()
    x = big[:3, :k].clone()
    x[0, 5], x[1, 7] = math.nan, math.inf
    y = torch.empty(3, n, dtype=DT[dtype], device="cuda")
    plan.step(x, y)
    assert torch.isnan(y[0]).all() and not torch.isfinite(y[1][full[:, 7] != 0]).any() and torch.isfinite(y[2]).all()
    x = torch.zeros(2, k, dtype=DT[dtype], device="cuda")
    plan.step(x, y[:2])
    assert (y[:2] == 0).all()


def test_project_e8m0_extremes(m):
    codes, scales, _ = make_weights(64, 64, "mxfp4", 32, None, False, 95)
    scales[0], scales[1], scales[2, 0] = 0, 1, 255
    plan = m.Projection(64, 64, fmt="mxfp4", group=32, dtype="f32")
    plan.pack(codes, scales)
    x = normal((2, 64), torch.float32, 96) * 2.0 ** 20
    y = torch.empty(2, 64, device="cuda")
    plan.step(x, y)
    want, bound = R.project(x, R.weights(codes, scales, None, "mxfp4", 32))
    assert torch.isnan(y[:, 2]).all()
    keep = torch.arange(64, device="cuda") != 2
    # the smallest results lie among the subnormals: half of their spacing more
    within(y[:, keep], want[:, keep], bound[:, keep] + 40 * 2.0 ** -150)


def test_project_refusals(m):
    plan = m.Projection(64, 128)
    x = normal((2, 128), torch.bfloat16, 1)
    y = torch.empty(2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.MonoError, match="no packed"):
        plan.step(x, y)
    codes, scales, zeros = make_weights(64, 128, "int4", 128, "bf16", True, 97)
    for bad in (lambda: plan.pack(codes, scales, zeros), lambda: plan.pack(codes[:, :3], scales), lambda: plan.pack(codes, scales.float()),
                lambda: plan.pack(codes.cpu(), scales), lambda: plan.pack(codes.t().contiguous().t(), scales)):
        with pytest.raises(ValueError):
            bad()
    plan.pack(codes, scales)
    for bad in (lambda: plan.step(x.float(), y), lambda: plan.step(x[:, :64], y), lambda: plan.step(x, y[:1]),
                lambda: plan.step(x, y.t().contiguous().t()), lambda: plan.step(x.cpu(), y)):
        with pytest.raises(ValueError):
            bad()
    nine = normal((9, 128), torch.bfloat16, 2)
    store = normal((2, 256), torch.bfloat16, 3)
    for bad in (lambda: plan.step(nine, torch.empty(9, 64, dtype=torch.bfloat16, device="cuda")),
                lambda: plan.step(store[:, :128], store[:, 100:164]), lambda: plan.step(x, y[:1].expand(2, 64))):
        with pytest.raises(m.MonoError):
            bad()
    assert plan.info()["cluster"] >= 1 and plan.info()["packed_bytes"] >= 64 * 64


# --------------------------------------------- streams, graphs, the run of them

def test_other_streams_and_two_plans_at_once(m):
    d, page, hq, hk, n = 128, 64, 8, 2, 3000
    caches = [make_cache(m, 48, hk, page, d, 100 + i) for i in range(2)]
    plans = [m.AttnPlan(hq, hk, d, page, 48, 1, 47) for _ in range(2)]
    table = [list(range(47))]
    qs = [normal((1, 1, hq, d), torch.bfloat16, 110 + i) for i in range(2)]
    want = [torch.empty_like(q) for q in qs]
    for c, p, q, o in zip(caches, plans, qs, want):
        p.attend(c, q, i32([n]), i32(table), o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    lens, tab = i32([n]), i32(table)
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    torch.cuda.synchronize()
    for j in range(20):
        for c, p, q, o, st in zip(caches, plans, qs, outs, streams):
            if j % 2:
                p.attend(c, q, lens, tab, o[j], stream=st)
            else:
                with torch.cuda.stream(st):
                    p.attend(c, q, lens, tab, o[j])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for os, w in zip(outs, want) for o in os)


def test_projection_and_append_share_a_plan_across_streams(m):
    """Neither has scratch: calls on one plan that overlap in time."""
    plan = m.Projection(640, 512, group=64, zeros=True)
    w = make_weights(640, 512, "int4", 64, "bf16", True, 150)
    plan.pack(*w)
    xs = [normal((4, 512), torch.bfloat16, 151 + i) for i in range(2)]
    want = [plan.step(x, torch.empty(4, 640, dtype=torch.bfloat16, device="cuda")) for x in xs]
    attn = m.AttnPlan(2, 2, 64, 16, 8, 1, 4)
    caches = [make_cache(m, 8, 2, 16, 64, 160) for _ in range(4)]
    kv = [normal((1, 1, 2, 64), torch.bfloat16, 170 + i) for i in range(2)]
    lens, table, rope = i32([33]), i32([[0, 1, 2, 3]]), m.Rope(64)
    for c, k in zip(caches[:2], kv):
        attn.append(c, k, k, lens, table, rope=rope)
    ys = [[torch.empty_like(want[0]) for _ in range(10)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(10):
        for i, st in enumerate(streams):
            plan.step(xs[i], ys[i][j], stream=st)
            if j == 5:
                attn.append(caches[2 + i], kv[i], kv[i], lens, table, rope=rope, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in ys[i])
    for i in range(2):
        assert torch.equal(caches[i].k.view(torch.uint8), caches[2 + i].k.view(torch.uint8))
        assert torch.equal(caches[i].v_scale, caches[2 + i].v_scale)


def test_packing_again_replaces_the_weights(m):
    plan = m.Projection(100, 64, fmt="mxfp4", group=32)
    x, y = normal((2, 64), torch.bfloat16, 180), torch.empty(2, 100, dtype=torch.bfloat16, device="cuda")
    for seed, special in ((181, True), (182, False)):   # scales of 0 and 255 first, then none
        codes, scales, _ = make_weights(100, 64, "mxfp4", 32, None, False, seed)
        if special:
            scales[3, 0], scales[4, 1] = 255, 0
        plan.pack(codes, scales)
        plan.step(x, y)
        want, bound = R.project(x, R.weights(codes, scales, None, "mxfp4", 32))
        keep = torch.arange(100, device="cuda") != (3 if special else -1)
        within(y[:, keep], want[:, keep], bound[:, keep])
        assert torch.isnan(y[:, 3]).all() == special


def test_captured_decode_serves_growing_lengths(m):
    """One captured step replayed while the sequences grow on the device."""
    d, page, hq, hk, seqs = 64, 16, 8, 2, 3
    cols, pages = 12, 40
    cache, eager = (make_cache(m, pages, hk, page, d, 121) for _ in range(2))
    plan, plan2 = (m.AttnPlan(hq, hk, d, page, pages, seqs, cols) for _ in range(2))
    rope = m.Rope(d)
    lens = i32([1, 40, 100])
    table = i32([list(range(12)), list(range(12, 24)), list(range(24, 36))])
    k, v, q = (normal((seqs, 1, h, d), torch.bfloat16, 130 + h) for h in (hk, hk + 1, hq))
    k, v = k[:, :, :hk], v[:, :, :hk]
    qr, out = torch.empty_like(q), torch.empty_like(q)

    def step(plan, cache, qr, out, lens):
        plan.append(cache, k, v, lens, table, rope=rope)
        m.rope(q.view(seqs, hq, d), lens - 1, rope, out=qr.view(seqs, hq, d))
        plan.attend(cache, qr, lens, table, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    held = lens.clone()
    with torch.cuda.stream(side):
        step(plan, make_cache(m, pages, hk, page, d, 121), qr, out, lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(plan, cache, qr, out, held)
        held += 1
    qr2, out2 = torch.empty_like(q), torch.empty_like(q)
    for i in range(60):
        graph.replay()
        step(plan2, eager, qr2, out2, lens + i)
        assert torch.equal(out, out2)
        k.mul_(1.02)   # the scales of begun pages grow
    assert torch.equal(cache.k.view(torch.uint8), eager.k.view(torch.uint8))
    assert plan.query_error()[0] == 0


@pytest.mark.parametrize("rows,fmt", [(1, "int4"), (3, "mxfp4"), (8, "int4")])
def test_decode_layer_of_both_halves(m, rows, fmt):
    """x -> q, k, v projections -> append -> attend -> output projection ->
    mono_ffn_step_pending, as a decode step uses them; every operator against
    its statement on the inputs it was given, the FFN half against the oracle,
    and the whole step captured and replayed bit for bit."""
    from oracle import oracle as O
    from synth import configs as C
    from synth import synth as S
    from tests.gpu_harness import LayerRun, check_chain_layer, compare_rel_l2
    from tests.oracle_helpers import all_experts
    wl = C.scaled(C.FLASH_BF16_R8, seed=503).with_(rows=rows)
    run = LayerRun(wl)
    a = S.gpu_attn_pending(wl)
    H, hq, hk, d, page = wl.hidden, 8, 2, 64, 16
    lens = [17 + 31 * r for r in range(rows)]
    cols, pages = 20, 20 * rows
    table = make_table(lens, page, cols, pages, 140, fill=-1)
    cache = make_cache(m, pages, hk, page, d, 141)
    plan = m.AttnPlan(hq, hk, d, page, pages, rows, cols)
    rope = m.Rope(d)
    group = 32
    wq = make_weights((hq + 2 * hk) * d, H, fmt, group, "bf16", False, 142)
    wo = make_weights(H, hq * d, fmt, group, "bf16", False, 143)
    if fmt == "int4":
        wq, wo = ((c, s * (0.2 / math.sqrt(c.shape[1])), z) for c, s, z in (wq, wo))
    p_in = m.Projection((hq + 2 * hk) * d, H, fmt=fmt, group=group)
    p_out = m.Projection(H, hq * d, fmt=fmt, group=group)
    p_in.pack(*wq)
    p_out.pack(*wo)
    x = normal((rows, H), torch.bfloat16, 144)
    qkv = torch.empty(rows, (hq + 2 * hk) * d, dtype=torch.bfloat16, device="cuda")
    heads = qkv.view(rows, 1, hq + 2 * hk, d)
    q, k, v = heads[:, :, :hq], heads[:, :, hq:hq + hk], heads[:, :, hq + hk:]
    qr, out = (torch.empty(rows, 1, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    y_attn = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    ln, tab, pos = i32(lens), i32(table), i32(lens) - 1

    def step():
        p_in.step(x, qkv)
        plan.append(cache, k, v, ln, tab, rope=rope)
        m.rope(q[:, 0], pos, rope, out=qr[:, 0])
        plan.attend(cache, qr, ln, tab, out)
        p_out.step(out.view(rows, hq * d), y_attn)
        run.plan.step_pending(rows, a["x"], a["post"], a["comb"], y_attn, run.out)

    before = {n: getattr(cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")}
    step()
    assert plan.query_error()[0] == 0 and run.plan.query_error()[0] == 0
    within(qkv, *R.project(x, R.weights(*wq, fmt, group)))
    made = m.KVCache(before["k"].clone(), before["v"].clone(), before["k_scale"].clone(), before["v_scale"].clone())
    want = R.append(made, k, v, lens, table, [1] * rows, rope, page)
    assert torch.equal(cache.k.double(), want["k"]) and torch.equal(cache.v_scale, want["v_scale"])
    rq, rb = R.rotate(q[:, 0], pos, rope), R.rotate_bound(q[:, 0], rope, torch.bfloat16)
    within(qr[:, 0], rq, rb + R.half_step(torch.bfloat16) * rq.abs())
    wa, _, ob, _ = R.attend(cache, qr, lens, table, [1] * rows, page, 1 / math.sqrt(d))
    within(out, wa, ob)
    within(y_attn, *R.project(out.view(rows, -1), R.weights(*wo, fmt, group)))
    host = S.cpu_attn_pending(wl)
    lw = O.LayerWeights(wl, S.cpu_dense(wl, 0), all_experts(wl, 0))
    y_host = y_attn.cpu().view(torch.int16).numpy().view("uint16")
    _, streams, _ = O.layer_pending(wl, lw, host["x"], host["post"], host["comb"], y_host)
    compare_rel_l2(run.tap(0, "x"), O.decode_hc(wl, streams), "streams")
    check_chain_layer(wl, run, 0, lw, run.out_host())
    first = (y_attn.clone(), run.out.clone())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        for n, t in before.items():
            dst = getattr(cache, n)
            (dst.view(torch.uint8) if dst.dtype == R.FP8 else dst).copy_(t.view(torch.uint8) if t.dtype == R.FP8 else t)
        y_attn.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y_attn, first[0]) and torch.equal(run.out, first[1])
    run.close()
