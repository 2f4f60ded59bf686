"""The attention half's decode operators, as cases to measure: rotary positions,
the append to a paged 8-bit cache, attention over that cache and the 4-bit
projections.  Each case runs in a plain form (elementary torch operations) or,
with `own` set, through the framework's entry points."""

import math

import numpy as np
import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
SCALE_MIN = 2.0 ** -126
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step of 8 rows: the queries of 40 heads, every dimension rotated
        dict(name="rope_decode", op="rope", dtype="bf16", tokens=8, heads=40, head_dim=128, rot=128, offset=0,
             interleaved=False, scaling="none", factor=1.0, theta=10000.0, start=8191, transpose=False),
        # the gradient's direction over a prompt: fp32, the last half of the head, far positions of a stretched context
        dict(name="rope_prompt_transposed", op="rope", dtype="f32", tokens=8191, heads=40, head_dim=128, rot=64,
             offset=64, interleaved=True, scaling="yarn", factor=16.0, theta=10000.0, start=1000000, transpose=True),
        # one decode step: 8 sequences, one new token each
        dict(name="append_decode", op="append", dtype="bf16", seqs=8, new=1, max_len=8192, ragged=False, kv_heads=8,
             head_dim=128, page=64, rot=128, offset=0, interleaved=False, scaling="none", factor=1.0, theta=10000.0),
        # four prompts of ragged length written to the cache at once
        dict(name="append_prompts", op="append", dtype="bf16", seqs=4, new=4093, max_len=4093, ragged=True, kv_heads=8,
             head_dim=128, page=64, rot=128, offset=0, interleaved=False, scaling="none", factor=1.0, theta=10000.0),
        # drafted tokens of many sequences, some of them padding, small pages, part of the head rotated
        dict(name="append_drafts_f32", op="append", dtype="f32", seqs=64, new=5, max_len=2048, ragged=True, kv_heads=2,
             head_dim=64, page=16, rot=32, offset=32, interleaved=True, scaling="yarn", factor=4.0, theta=10000.0),
        # a sequence's first token: the smallest call
        dict(name="attend_first", op="attend", dtype="bf16", seqs=1, new=1, max_len=1, ragged=False, q_heads=40,
             kv_heads=8, head_dim=128, page=64, window=0, lse=False),
        # an ordinary decode step: 8 sequences of mixed length
        dict(name="attend_8x8k", op="attend", dtype="bf16", seqs=8, new=1, max_len=8192, ragged=True, q_heads=40,
             kv_heads=8, head_dim=128, page=64, window=0, lse=False),
        # one very long sequence
        dict(name="attend_long", op="attend", dtype="bf16", seqs=1, new=1, max_len=131071, ragged=False, q_heads=40,
             kv_heads=8, head_dim=128, page=64, window=0, lse=False),
        # drafted tokens checked at once: causal among themselves, a sliding window, fp32
        dict(name="attend_drafts_f32", op="attend", dtype="f32", seqs=16, new=4, max_len=4097, ragged=True, q_heads=32,
             kv_heads=4, head_dim=64, page=16, window=1500, lse=True),
        # the q, k and v projection of one row
        dict(name="project_qkv", op="project", dtype="bf16", rows=1, n_out=7168, n_in=5120, fmt="int4", group=128,
             scales="bf16", zeros=False),
        # an odd width with zero points, fp32
        dict(name="project_odd_f32", op="project", dtype="f32", rows=3, n_out=1003, n_in=1056, fmt="int4", group=32,
             scales="f32", zeros=True),
        # the output head over a large vocabulary at the widest step
        dict(name="project_vocab", op="project", dtype="bf16", rows=8, n_out=131072, n_in=5120, fmt="mxfp4", group=32,
             scales="e8m0", zeros=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "project"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "project":
        c.update(rows=rng.randint(1, 8), fmt=rng.choice(["int4", "int4", "mxfp4"]))
        c["group"] = 32 if c["fmt"] == "mxfp4" else rng.choice([32, 64, 128])
        c["scales"] = "e8m0" if c["fmt"] == "mxfp4" else rng.choice(["bf16", "f32"])
        c["zeros"] = c["fmt"] == "int4" and rng.random() < 0.5
        c["n_in"] = c["group"] * _spread(rng, max(1, 256 // c["group"]), 8192 // c["group"])
        c["n_out"] = _spread(rng, 100, 65536)
        return c
    c["head_dim"] = d = rng.choice([64, 128, 128, 256])
    if op != "attend":
        rot = rng.choice([d, d, d // 2])
        c.update(rot=rot, offset=rng.choice([0, d - rot]), interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), theta=rng.choice([10000.0, 500000.0]))
        c["factor"] = 1.0 if c["scaling"] == "none" else rng.choice([2.0, 4.0, 16.0])
    if op == "rope":
        c.update(heads=_spread(rng, 1, 64), start=_spread(rng, 1, 1000000), transpose=rng.random() < 0.3)
        c["tokens"] = _spread(rng, 1, max(1, (1 << 24) // (c["heads"] * d)))
        return c
    c.update(seqs=_spread(rng, 1, 64), page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
    if op == "append":
        c["kv_heads"] = rng.choice([1, 2, 4, 8])
        c["new"] = rng.choice([1, rng.randint(1, 8), _spread(rng, 1, max(1, (1 << 22) // (c["seqs"] * c["kv_heads"] * d)))])
        c["max_len"] = c["new"] + _spread(rng, 1, max(1, (1 << 23) // (c["seqs"] * c["kv_heads"] * d)))
        return c
    c["kv_heads"] = rng.choice([1, 2, 4, 8])
    c["q_heads"] = c["kv_heads"] * rng.choice([1, 4, 5, 8, 16])
    c["new"] = rng.choice([1, 1, rng.randint(2, 8)])
    rows = c["new"] * c["q_heads"] // c["kv_heads"]
    c["max_len"] = c["new"] + _spread(rng, 1, max(1, (1 << 26) // (c["seqs"] * c["kv_heads"] * d * max(1, rows // 32))))
    c["window"] = 0 if rng.random() < 0.7 else _spread(rng, 1, c["max_len"])
    c["lse"] = rng.random() < 0.5
    return c


def _lens(c):
    """Each sequence's length after the call and its new tokens.  Ragged: between
    one token and max_len; some hold fewer new tokens than the widest, one in
    sixteen none (a padding sequence)."""
    s = c["seqs"]
    if not c["ragged"]:
        return [c["max_len"]] * s, [c["new"]] * s
    lens = [max(1, int(c["max_len"] * ((0.6180339887 * (i + 1)) % 1.0))) if i else c["max_len"] for i in range(s)]
    if c["new"] > 8:   # prompts: everything that a sequence has is new
        return lens, [min(n, c["new"]) for n in lens]
    if c["new"] == 1:
        return lens, [1] * s
    new = [0 if i % 16 == 15 else min(n, 1 + (c["new"] - 1 + 3 * i) % c["new"]) for i, n in enumerate(lens)]
    return lens, new


def _freqs(c):
    """Radians a position for each rotated pair, and the factor on the result."""
    rot, theta, s = c["rot"], c["theta"], c["factor"]
    if c["scaling"] == "ntk" and rot > 2:
        theta *= s ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if c["scaling"] == "linear":
        return f / s, 1.0
    if c["scaling"] != "yarn":
        return f, 1.0
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
    return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0


def _own_rope(c):
    from moe_decode_layer_sm_b200 import Rope
    return Rope(c["rot"], theta=c["theta"], scaling=c["scaling"], factor=c["factor"], orig_context=4096,
                interleaved=c["interleaved"], offset=c["offset"])


def _pages(c, lens, g):
    """A page table over shuffled pages; entries behind a sequence's end are -1."""
    per = [-(-n // c["page"]) for n in lens]
    width, total = max(per), sum(per) + 3
    order = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
    live = torch.arange(width, device="cuda")[None, :] < torch.tensor(per, device="cuda")[:, None]
    table[live] = order[:sum(per)]
    return table, total


def _cache(c, total, g, fill):
    shape = (total, c["kv_heads"], c["page"], c["head_dim"])
    made = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s = x.abs().amax(dim=(2, 3)).float() / FP8_MAX
        made.append((x / s[:, :, None, None] if fill else x * 0).clamp_(-FP8_MAX, FP8_MAX).to(FP8))
        made.append(s if fill else torch.zeros_like(s))
    return dict(k=made[0], k_scale=made[1], v=made[2], v_scale=made[3])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    normal = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g).to(DTYPE[c["dtype"]])  # noqa: E731
    if c["op"] == "rope":
        st["x"] = normal(c["tokens"], c["heads"], c["head_dim"])
        st["pos"] = torch.arange(c["tokens"], dtype=torch.int32, device="cuda") + c["start"]
        if own:
            st["out"], st["rope"] = torch.empty_like(st["x"]), _own_rope(c)
        return st
    if c["op"] == "project":
        n, k, gr = c["n_out"], c["n_in"], c["group"]
        st["x"] = normal(c["rows"], k)
        st["codes"] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
        if c["fmt"] == "mxfp4":
            e = 125 - round(math.log2(k) / 2)
            st["scales"] = torch.randint(e - 2, e + 3, (n, k // gr), dtype=torch.uint8, device="cuda", generator=g)
        else:
            s = torch.rand((n, k // gr), device="cuda", generator=g) + 0.5
            st["scales"] = (s / (4.6 * math.sqrt(k))).to(DTYPE[c["scales"]])
        st["zeros"] = torch.randint(4, 12, (n, k // gr), dtype=torch.uint8, device="cuda", generator=g) if c["zeros"] else None
        if own:
            from moe_decode_layer_sm_b200 import Projection
            st["plan"] = Projection(n, k, fmt=c["fmt"], group=gr, scale_dtype=c["scales"], zeros=c["zeros"],
                                    dtype=c["dtype"])
            st["plan"].pack(st["codes"], st["scales"], st["zeros"])
            st["y"] = torch.empty((c["rows"], n), dtype=DTYPE[c["dtype"]], device="cuda")
        return st
    lens, new = _lens(c)
    st["table"], total = _pages(c, lens, g)
    st.update(_cache(c, total, g, fill=c["op"] == "attend" or c["new"] <= 8))
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if c["ragged"] and c["new"] > 1 else None
    if c["op"] == "attend":
        st["q"] = normal(c["seqs"], c["new"], c["q_heads"], c["head_dim"])
    else:
        st["k_new"] = normal(c["seqs"], c["new"], c["kv_heads"], c["head_dim"])
        st["v_new"] = normal(c["seqs"], c["new"], c["kv_heads"], c["head_dim"])
    if own:
        from moe_decode_layer_sm_b200 import AttnPlan, KVCache
        st["plan"] = AttnPlan(q_heads=c.get("q_heads", c["kv_heads"]), kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                              page_size=c["page"], num_pages=total, max_seqs=c["seqs"], max_pages=st["table"].shape[1],
                              max_new=min(c["new"], 8), dtype=c["dtype"], window=c.get("window", 0))
        st["cache"] = KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if c["op"] == "append":
            st["rope"] = _own_rope(c)
        else:   # rows that a padding sequence leaves as they were: zero
            st["out"] = torch.zeros_like(st["q"])
            st["lse"] = torch.zeros(st["q"].shape[:3], device="cuda") if c["lse"] else None
    return st


def _rotated(c, x, pos):
    """x [tokens][heads][head_dim] rotated by its tokens' positions: fp64 in, fp64 out."""
    f, m = _freqs(c)
    a = pos.double()[:, None, None] * torch.from_numpy(f).to(x.device)
    cos, sin = torch.cos(a) * m, torch.sin(a) * m
    if c.get("transpose"):
        sin = -sin
    lo, hi = c["offset"], c["offset"] + c["rot"]
    r = x[..., lo:hi]
    if c["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :c["rot"] // 2], r[..., c["rot"] // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((x[..., :lo], r, x[..., hi:]), -1)


def _plain_project(st):
    c = st["case"]
    n, k, gr = c["n_out"], c["n_in"], c["group"]
    q = torch.stack((st["codes"] & 15, st["codes"] >> 4), -1).reshape(n, k // gr, gr)
    if c["fmt"] == "mxfp4":
        w = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")[q.long()]
        s = torch.exp2(st["scales"].float() - 127)
    else:
        w = q.float() - (st["zeros"][:, :, None].float() if c["zeros"] else 8.0)
        s = st["scales"].float()
    w = (w * s[:, :, None]).reshape(n, k)
    return (st["x"].float() @ w.t()).to(DTYPE[c["dtype"]])


def _nearest_fp8(x):
    """The nearest e4m3 value of each, ties to even, rounded once from fp64 (a cast would go through fp32)."""
    x = x.clamp(-FP8_MAX, FP8_MAX)
    grid = (torch.frexp(x).exponent - 1).clamp_min(-6) - 3
    return torch.ldexp(torch.round(torch.ldexp(x, -grid)), grid).to(FP8)


def _plain_append(st):
    c = st["case"]
    s, n, h, d, p = c["seqs"], c["new"], c["kv_heads"], c["head_dim"], c["page"]
    new = st["new"].long() if st["new"] is not None else torch.full((s,), n, device="cuda")
    first = st["lens"].long() - new                                      # position of a sequence's first new token
    j = torch.arange(n, device="cuda")
    pos = first[:, None] + j
    live = (j < new[:, None]) & (pos >= 0)
    spans = (n - 1) // p + 2                                             # pages that new tokens can touch
    chunk = pos // p - (first // p)[:, None]
    row = (torch.arange(s, device="cuda")[:, None] * spans + chunk) * p + pos % p
    page_no = (first // p)[:, None] + torch.arange(spans, device="cuda")
    used = torch.zeros(s * spans, dtype=torch.bool, device="cuda").index_fill_(0, row[live] // p, True).view(s, spans)
    ids = st["table"].gather(1, page_no.clamp(0, st["table"].shape[1] - 1)).long()[used]
    begun = (used & (torch.arange(spans, device="cuda") == 0) & (first % p > 0)[:, None])[used]   # pages with older tokens
    for name, x in (("k", st["k_new"]), ("v", st["v_new"])):
        x = x.reshape(s * n, h, d).double()
        if name == "k":
            x = _rotated(c, x, pos.reshape(-1))
        dense = torch.zeros(s * spans * p, h, d, dtype=torch.float64, device="cuda")
        dense[row[live]] = x[live.reshape(-1)]
        dense = dense.view(s, spans, p, h, d)[used].transpose(1, 2)      # [pages][heads][page][head_dim]
        fresh = torch.zeros(s * spans * p, dtype=torch.bool, device="cuda").index_fill_(0, row[live], True)
        fresh = fresh.view(s, spans, p)[used][:, None, :, None]
        was = st[name + "_scale"][ids].double()
        scale = (dense.abs().amax(dim=(2, 3)) / FP8_MAX).clamp_min(SCALE_MIN)
        scale = torch.where(begun[:, None], torch.maximum(scale, was), scale).float().double()
        old = st[name][ids].double()
        older = torch.arange(p, device="cuda") < torch.where(begun, (first % p)[:, None].expand(s, spans)[used], 0)[:, None]
        kept = torch.where((scale > was)[:, :, None, None] & older[:, None, :, None],
                           old * (was / scale)[:, :, None, None], old)
        code = torch.where(fresh, dense / scale[:, :, None, None], kept)
        st[name][ids] = _nearest_fp8(code)
        st[name + "_scale"][ids] = scale.float()
    return {x: st[x] for x in ("k", "v", "k_scale", "v_scale")}


def _plain_attend(st):
    c = st["case"]
    s, n, hk, d, p = c["seqs"], c["new"], c["kv_heads"], c["head_dim"], c["page"]
    g = c["q_heads"] // hk
    new = st["new"].long() if st["new"] is not None else torch.full((s,), n, device="cuda")
    ids = st["table"].clamp_min(0).long()
    length = ids.shape[1] * p
    every = []
    for name in ("k", "v"):
        x = st[name][ids].float() * st[name + "_scale"][ids][:, :, :, None, None]
        x = x.transpose(1, 2).reshape(s, hk, length, d)
        gone = torch.arange(length, device="cuda") >= st["lens"][:, None]
        every.append(x.masked_fill(gone[:, None, :, None], 0.0))
    k, v = every
    q = st["q"].float().view(s, n, hk, g, d).permute(0, 2, 1, 3, 4).reshape(s, hk, n * g, d)
    logits = (q @ k.transpose(2, 3)).view(s, hk, n, g, length) / math.sqrt(d)
    j = torch.arange(n, device="cuda")
    pos = (st["lens"].long() - new)[:, None] + j                         # [seqs][new]
    at = torch.arange(length, device="cuda")
    seen = (at <= pos[:, :, None]) & (j < new[:, None])[:, :, None]
    if c["window"]:
        seen &= at > pos[:, :, None] - c["window"]
    seen = seen[:, None, :, None, :]
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    prob = torch.exp(logits - top.masked_fill(top == -math.inf, 0.0))
    total = prob.sum(-1, keepdim=True)
    out = (prob.view(s, hk, n * g, length) @ v).view(s, hk, n, g, d) / total.clamp_min(1e-30)
    out = out.permute(0, 2, 1, 3, 4).reshape(s, n, hk * g, d).to(DTYPE[c["dtype"]])
    if not c["lse"]:
        return {"out": out}
    lse = (top + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(s, n, hk * g)
    return {"out": out, "lse": torch.where((j < new[:, None])[:, :, None], lse, torch.zeros_like(lse))}


def run(state):
    st, c = state, state["case"]
    if own:
        if c["op"] == "rope":
            from moe_decode_layer_sm_b200 import rope
            return rope(st["x"], st["pos"], st["rope"], out=st["out"], transpose=c["transpose"])
        if c["op"] == "project":
            return st["plan"].step(st["x"], st["y"])
        if c["op"] == "append":
            st["plan"].append(st["cache"], st["k_new"], st["v_new"], st["lens"], st["table"], rope=st["rope"],
                              n_new=st["new"])
            return {x: st[x] for x in ("k", "v", "k_scale", "v_scale")}
        st["plan"].attend(st["cache"], st["q"], st["lens"], st["table"], st["out"], lse=st["lse"], n_new=st["new"])
        return {"out": st["out"], "lse": st["lse"]} if c["lse"] else {"out": st["out"]}
    if c["op"] == "rope":
        return _rotated(c, st["x"].double(), st["pos"]).to(DTYPE[c["dtype"]])
    return {"project": _plain_project, "append": _plain_append, "attend": _plain_attend}[c["op"]](st)


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["head_dim"]
        return {"bytes": 2 * n * e + 4 * c["tokens"], "flops": 3 * n}
    if c["op"] == "project":
        n, k, gr = c["n_out"], c["n_in"], c["group"]
        per = {"bf16": 2, "f32": 4, "e8m0": 1}[c["scales"]] + (1 if c["zeros"] else 0)
        return {"bytes": n * k // 2 + n * (k // gr) * per + e * c["rows"] * (n + k), "flops": 2 * n * k * c["rows"]}
    lens, new = _lens(c)
    hk, d, p = c["kv_heads"], c["head_dim"], c["page"]
    if c["op"] == "append":
        pages = sum((ln - 1) // p - (ln - n) // p + 1 for ln, n in zip(lens, new) if n)
        return {"bytes": 2 * sum(new) * hk * d * (e + 1) + 8 * pages * hk, "flops": 8 * sum(new) * hk * d}
    keys = pairs = pages = 0
    for ln, n in zip(lens, new):
        if n:
            lo = max(0, ln - n + 1 - c["window"]) if c["window"] else 0
            keys += ln - lo
            pages += (ln - 1) // p - lo // p + 1
            pairs += sum(min(ln - n + 1 + j, c["window"] or ln) for j in range(n))
    rows = sum(new) * c["q_heads"]
    return {"bytes": 2 * keys * hk * d + 8 * pages * hk + 2 * rows * d * e + (4 * rows if c["lse"] else 0),
            "flops": 4 * pairs * c["q_heads"] * d}


def _e4m3(x):
    """The nearest e4m3 value of each (ties to even), in fp64."""
    x = x.clamp(-FP8_MAX, FP8_MAX)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))).clamp_min(-6) - 3)
    return torch.round(x / step) * step


def _turned(c, x, pos):
    """x [tokens][heads][head_dim] rotated to its tokens' positions by complex products, in fp64."""
    f, m = _freqs(c)
    a = torch.outer(pos.double(), torch.from_numpy(f).to(x.device))
    z = torch.polar(torch.full_like(a, m), a)[:, None, :]
    z = z.conj() if c.get("transpose") else z
    y = x.double()
    part = y[..., c["offset"]:c["offset"] + c["rot"]]
    pair = part.unflatten(-1, (-1, 2)) if c["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    y[..., c["offset"]:c["offset"] + c["rot"]] = (w if c["interleaved"] else w.transpose(-1, -2)).flatten(-2)
    return y


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "rope":
        return _turned(c, st["x"], st["pos"])
    if c["op"] == "project":
        x, gr = st["x"].double(), c["group"]
        y = torch.empty((c["rows"], c["n_out"]), dtype=torch.float64, device="cuda")
        for a in range(0, c["n_out"], 16384):
            rows = slice(a, a + 16384)
            code = st["codes"][rows].long()
            w = torch.empty((code.shape[0], c["n_in"]), dtype=torch.float64, device="cuda")
            for half, v in ((0, code % 16), (1, code // 16)):
                if c["fmt"] == "mxfp4":
                    mag, e = v % 2, (v // 2) % 4
                    val = torch.where(e > 0, (1 + 0.5 * mag) * torch.exp2((e - 1).double()), 0.5 * mag)
                    w[:, half::2] = torch.where(v >= 8, -val, val)
                else:
                    w[:, half::2] = v.double()
            s = st["scales"][rows].double()
            s = (torch.exp2(s - 127) if c["fmt"] == "mxfp4" else s).repeat_interleave(gr, 1)
            if c["fmt"] == "int4":
                w -= st["zeros"][rows].double().repeat_interleave(gr, 1) if c["zeros"] else 8.0
            y[:, rows] = x @ (w * s).t()
        return y
    lens, new = _lens(c)
    p, d, hk = c["page"], c["head_dim"], c["kv_heads"]
    table = st["table"].cpu().tolist()
    if c["op"] == "append":
        out = {n: st[n].double() for n in ("k", "v", "k_scale", "v_scale")}
        for s in range(c["seqs"]):
            first = lens[s] - new[s]
            for page in range(first // p, (lens[s] - 1) // p + 1) if new[s] else ():
                a, b, i = max(first, page * p), min(lens[s], (page + 1) * p), table[s][page]
                for name in ("k", "v"):
                    x = st[name + "_new"][s, a - first:b - first]
                    x = _turned(c, x, torch.arange(a, b, device="cuda")) if name == "k" else x.double()
                    x = x.transpose(0, 1)
                    scale = (x.abs().amax(dim=(1, 2)) / FP8_MAX).clamp_min(SCALE_MIN).float().double()
                    if a > page * p:
                        was = out[name + "_scale"][i]
                        scale = torch.maximum(scale, was)
                        kept = out[name][i, :, :a - page * p]
                        out[name][i, :, :a - page * p] = _e4m3(kept * (was / scale)[:, None, None])
                    out[name + "_scale"][i] = scale
                    out[name][i, :, a - page * p:b - page * p] = _e4m3(x / scale[:, None, None])
        return out
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:3], dtype=torch.float64, device="cuda")
    g = c["q_heads"] // hk
    for s in range(c["seqs"]):
        if not new[s]:
            continue
        ids = torch.tensor(table[s][:-(-lens[s] // p)], device="cuda")
        k, v = ((st[n][ids].double() * st[n + "_scale"][ids].double()[:, :, None, None]).permute(1, 0, 2, 3)
                .reshape(hk, -1, d)[:, :lens[s]] for n in ("k", "v"))
        for j in range(new[s]):
            e = lens[s] - new[s] + j + 1
            b = max(0, e - c["window"]) if c["window"] else 0
            q = st["q"][s, j].double().view(hk, g, d)
            w = torch.einsum("hgd,htd->hgt", q, k[:, b:e]) / math.sqrt(d)
            out[s, j] = torch.einsum("hgt,htd->hgd", torch.softmax(w, -1), v[:, b:e]).reshape(-1, d)
            lse[s, j] = torch.logsumexp(w, -1).reshape(-1)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
