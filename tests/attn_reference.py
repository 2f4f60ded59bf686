"""Plain fp64 statements of the attention half's operators, on the GPU, and
the error bounds that the kernels' arithmetic allows."""

import math

import torch

FP8 = torch.float8_e4m3fn
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def half_step(dtype):
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def rotate(x, pos, rope, transpose=False):
    """x [tokens][heads][head_dim] -> fp64; rope: the binding's Rope."""
    v = rope.value
    n = v.rot_dim // 2
    turns = torch.tensor(list(v.turns[:n]), dtype=torch.float64, device=x.device)
    a = pos.double()[:, None] * turns
    a = 2 * math.pi * (a - torch.round(a))
    c, s = torch.cos(a)[:, None] * v.factor, torch.sin(a)[:, None] * v.factor
    if transpose:
        s = -s
    y = x.double().clone()
    d = torch.arange(n, device=x.device)
    i1 = v.offset + (2 * d if v.interleaved else d)
    i2 = v.offset + (2 * d + 1 if v.interleaved else d + n)
    x1, x2 = x.double()[..., i1], x.double()[..., i2]
    y[..., i1] = c * x1 - s * x2
    y[..., i2] = s * x1 + c * x2
    return y


def rotate_bound(x, rope, dtype):
    """|error| of each rotated value.  The angle enters sincospi as 2 t in fp32:
    |2 pi t| <= pi, so it is off by pi 2^-24; sin and cos by one more unit
    (2^-23 for values up to 1), the factor (and its product), two products and a
    sum by a half unit each: below 11 x 2^-24 (|x1| + |x2|) factor.  Then one rounding."""
    v = rope.value
    n = v.rot_dim // 2
    d = torch.arange(n, device=x.device)
    i1 = v.offset + (2 * d if v.interleaved else d)
    i2 = v.offset + (2 * d + 1 if v.interleaved else d + n)
    b = torch.zeros_like(x, dtype=torch.float64)
    m = (x.double()[..., i1].abs() + x.double()[..., i2].abs()) * abs(v.factor) * 11 * 2.0 ** -24
    b[..., i1] = m
    b[..., i2] = m
    return b * (1 + half_step(dtype))


def nearest_fp8(q):
    """The nearest e4m3 value, ties to even, from fp64 in one rounding; NaN stays."""
    q = q.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(q / step) * step


def append(cache, k, v, lens, table, n_new, rope, page):
    """The cache after the call: dict of fp64 codes' values and fp32 scales (lists on the host are the integers)."""
    out = {"k": cache.k.double(), "v": cache.v.double(), "k_scale": cache.k_scale.clone(), "v_scale": cache.v_scale.clone()}
    for s, (ln, n) in enumerate(zip(lens, n_new)):
        for pg in range(max(ln - n, 0) // page, (ln - 1) // page + 1) if n > 0 and ln > 0 else ():
            a, b, i = max(ln - n, pg * page, 0), min(ln, (pg + 1) * page), table[s][pg]
            for name, x in (("k", k), ("v", v)):
                x = x[s, a - (ln - n):b - (ln - n)]
                x = rotate(x, torch.arange(a, b, device=x.device), rope) if rope is not None and name == "k" else x.double()
                x = x.transpose(0, 1)
                fin = torch.where(x.abs() <= 3.402823466e38, x.abs(), 0.0)
                scale = (fin.amax(dim=(1, 2)) / 448.0).float().clamp_min(2.0 ** -126)
                old = a - pg * page
                if old > 0:
                    was = out[name + "_scale"][i]
                    scale = torch.maximum(scale, was)
                    ratio = was.double() / scale.double()
                    out[name][i, :, :old] = nearest_fp8(out[name][i, :, :old] * ratio[:, None, None])
                out[name + "_scale"][i] = scale
                out[name][i, :, old:b - pg * page] = nearest_fp8(x / scale.double()[:, None, None])
    return out


def attend(cache, q, lens, table, n_new, page, scale, window=0):
    """(out, lse, bound of out, bound of lse) fp64; rows that are not live hold NaN in all four.

    Bounds.  A logit: q enters with 11 bits below the row's largest (22 for fp32)
    -- exact for bf16 -- and each of the D/16 matrix steps may cut 2^-22 of what
    it adds up, the scales and the softmax scale three more half units:
    e = S (D/16 + 4) 2^-22 with S the largest sum of |q_d k_d| scale that the row
    sees.  A probability: that, exp2's own 2^-22 and the argument's rounding
    (|logit| up to S and the 2^15 bias: (S + 24) 2^-23), then 11 bits (bf16) or
    22; values' scale ratio 2^-21.  So out is off by A (2 e + ...) with
    A = sum p |v|, and by one unit for each of the tiles that are added up; then
    its own rounding.  Probabilities below 2^-29 lose bits: 2^-40 max |v| a token."""
    seqs, width, hq, d = q.shape
    hk = cache.k.shape[1]
    g = hq // hk
    f32 = q.dtype == torch.float32
    nan = float("nan")
    out = torch.full(q.shape, nan, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:3], nan, dtype=torch.float64, device=q.device)
    ob, lb = out.clone(), lse.clone()
    for s in range(seqs):
        ln, n = lens[s], n_new[s]
        if n <= 0:
            continue
        ids = torch.tensor(table[s][:max(0, -(-ln // page))], dtype=torch.long, device=q.device)
        k, v = ((c[ids].double() * sc[ids].double()[:, :, None, None]).permute(1, 0, 2, 3).reshape(hk, -1, d)
                for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        for j in range(n):
            e = ln - n + j + 1
            b = max(0, e - window) if window else 0
            if e <= b:
                out[s, j], lse[s, j], ob[s, j], lb[s, j] = 0.0, -math.inf, 0.0, 0.0
                continue
            qq = q[s, j].double().view(hk, g, d)
            kk, vv = k[:, b:e], v[:, b:e]
            w = torch.einsum("hgd,htd->hgt", qq, kk) * scale
            big = torch.einsum("hgd,htd->hgt", qq.abs(), kk.abs()).amax(-1) * scale
            p = torch.softmax(w, -1)
            o = torch.einsum("hgt,htd->hgd", p, vv)
            a = torch.einsum("hgt,htd->hgd", p, vv.abs())
            tiles = (e - b) / 16 + 2
            err = big * (d / 16 + 4) * 2.0 ** -22 + (big + 24) * 2.0 ** -23 + 2.0 ** -22
            rel = 2 * err + (2.0 ** -22 if f32 else 2.0 ** -11) + 2.0 ** -21 + tiles * 2.0 ** -23
            low = (e - b) * 2.0 ** -40 * vv.abs().amax(1)[:, None, :]
            out[s, j] = o.reshape(hq, d)
            ob[s, j] = ((a * rel[..., None] + low) * (1 + half_step(q.dtype)) + half_step(q.dtype) * o.abs()).reshape(hq, d)
            lse[s, j] = torch.logsumexp(w, -1).reshape(hq)
            lb[s, j] = (err + tiles * 2.0 ** -23 + lse[s, j].view(hk, g).abs() * 2.0 ** -22 + 2.0 ** -22).reshape(hq)
    return out, lse, ob, lb


def weights(codes, scales, zeros, fmt, group):
    """W [n_out][n_in] fp64."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    rep = lambda t: t.repeat_interleave(group, 1)  # noqa: E731
    if fmt == "mxfp4":
        s = torch.where(scales == 255, float("nan"), torch.exp2(scales.double() - 127))
        return E2M1.to(codes.device)[c] * rep(s)
    z = 8.0 if zeros is None else rep((zeros & 15).double())
    return (c.double() - z) * rep(scales.double())


def project(x, w):
    """(y, bound) fp64.  Products are exact; a scale's 32 are added by two matrix
    steps that may cut 2^-22 each, then in fp32 over a warp's share (an eighth of
    the inputs at most), 8 warps and up to 8 CTAs; fp32 rows enter with 22 bits.
    x below 2^-14 of its row's largest (of the part that a CTA reads) loses bits:
    2^-39 of that largest (a second term takes fp32's there too)."""
    y = x.double() @ w.t()
    a = x.double().abs() @ w.abs().t()
    f32 = x.dtype == torch.float32
    k = w.shape[1]
    rel = 2 * 2.0 ** -22 + (k / 256 + 20) * 2.0 ** -23 + (2.0 ** -22 if f32 else 0)
    low = 2.0 ** -39 * x.double().abs().amax(1, keepdim=True) * w.abs().sum(1)
    return y, (a * rel + low) * (1 + half_step(x.dtype)) + half_step(x.dtype) * y.abs()
