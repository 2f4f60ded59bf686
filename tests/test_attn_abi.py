"""The attention half's operators without a GPU: exported symbols, every
refusal, the prepared rotation's numbers, and the index arithmetic that the
kernels share with the host (csrc/kv_index.h), compiled here as plain C++."""

import ctypes
import math
import os
import random
import re
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_decode_layer_sm_b200", "csrc")


@pytest.fixture(scope="module")
def attn():
    from moe_decode_layer_sm_b200 import attn, build
    build.build()
    attn._lib()
    return attn


def test_library_exports_every_declared_symbol(attn):
    src = open(os.path.join(ROOT, "include", "mono_attn.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(mono_(?:attn|rope|proj)_\w+)\s*\(", src))
    L = attn._lib()
    assert all(hasattr(L, n) for n in names)
    assert names == set(attn.SYMBOLS)


def test_names_of_the_package():
    import moe_decode_layer_sm_b200 as m
    for n in ("Rope", "rope", "KVCache", "AttnPlan", "Projection", "Plan"):
        assert callable(getattr(m, n))
    with pytest.raises(AttributeError):
        m.nothing


GOOD_ATTN = dict(q_heads=8, kv_heads=2, head_dim=128, page_size=64, num_pages=16, max_seqs=4, max_pages=8, max_new=2,
                 dtype=1, scale=0.0, window=0, device=0)


def _plan_reasons(attn, **kw):
    L = attn._lib()
    h = ctypes.c_void_p()
    rc = L.mono_attn_plan(ctypes.byref(attn.AttnConfig(**{**GOOD_ATTN, **kw})), ctypes.byref(h))
    if rc == 0:
        L.mono_attn_destroy(h)
        return ""
    return L.mono_attn_last_error().decode()


@pytest.mark.parametrize("kw,frag", [
    (dict(kv_heads=0), "kv_heads"), (dict(q_heads=7), "q_heads"), (dict(q_heads=0), "q_heads"),
    (dict(q_heads=512, kv_heads=2), "q_heads"), (dict(head_dim=96), "head_dim"), (dict(page_size=48), "page_size"),
    (dict(page_size=256), "page_size"), (dict(num_pages=0), "num_pages"), (dict(max_seqs=0), "max_seqs"),
    (dict(max_seqs=4097), "max_seqs"), (dict(max_pages=0), "max_pages"), (dict(max_new=0), "max_new"),
    (dict(max_new=9), "max_new"), (dict(dtype=2), "dtype"), (dict(window=-1), "window"),
    (dict(scale=float("nan")), "scale"), (dict(scale=-1.0), "scale"),
    (dict(max_pages=1 << 26, page_size=64), "2^31"), (dict(max_pages=1 << 20, max_seqs=4096), "work partition"),
    (dict(device=-1), "device"),
])
def test_attn_plan_refuses(attn, kw, frag):
    why = _plan_reasons(attn, **kw)
    assert frag in why or (frag == "device" and why), why


def test_attn_plan_lists_every_reason(attn):
    why = _plan_reasons(attn, head_dim=96, page_size=5, max_new=0)
    assert all(f in why for f in ("head_dim", "page_size", "max_new"))
    assert "work partition" not in _plan_reasons(attn, max_seqs=64, max_pages=2048)


GOOD_PROJ = dict(n_out=64, n_in=256, format=4, group=128, scale_dtype=1, zeros=0, dtype=1, device=0)


@pytest.mark.parametrize("kw,frag", [
    (dict(n_out=0), "n_out"), (dict(n_out=(1 << 30) + 1), "n_out"), (dict(n_in=0), "n_in"), (dict(n_in=192), "n_in"), (dict(format=2), "format"),
    (dict(group=48), "group"), (dict(group=0), "group"), (dict(format=3, group=128), "group must be 32"),
    (dict(format=3, group=32, zeros=1), "zeros"), (dict(scale_dtype=2), "scale_dtype"), (dict(dtype=3), "dtype"),
    (dict(n_in=128 * 4096), "too large"),
])
def test_proj_plan_refuses(attn, kw, frag):
    L = attn._lib()
    h = ctypes.c_void_p()
    assert L.mono_proj_plan(ctypes.byref(attn.ProjConfig(**{**GOOD_PROJ, **kw})), ctypes.byref(h)) == -1
    assert frag in L.mono_attn_last_error().decode()
    assert not h


def test_null_handles_and_arguments(attn):
    L = attn._lib()
    h = ctypes.c_void_p()
    assert L.mono_attn_plan(None, ctypes.byref(h)) == -1
    assert L.mono_proj_plan(None, ctypes.byref(h)) == -1
    assert L.mono_rope_init(None, None) == -1
    assert L.mono_attn_append(None, None, None, None, None, None, None) == -1
    assert L.mono_attn_attend(None, None, None, None, None, None, None) == -1
    assert L.mono_attn_query_error(None, None) == -1
    assert L.mono_attn_get_info(None, None) == -1
    assert L.mono_proj_pack(None, None, None, None, None) == -1
    assert L.mono_proj_step(None, 1, None, 0, None, 0, None) == -1
    assert L.mono_proj_get_info(None, None) == -1
    L.mono_attn_destroy(None)
    L.mono_proj_destroy(None)


def _frequency(rot, theta, scaling, factor, orig=4096, fast=32.0, slow=1.0):
    """Radians a position, pair by pair, from the formulas."""
    out = []
    base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" else theta
    for i in range(rot // 2):
        f = 1.0 / base ** (2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            pair = lambda turns: rot / 2 * math.log(orig / (2 * math.pi * turns)) / math.log(theta)  # noqa: E731
            lo, hi = max(0, math.floor(pair(fast))), min(rot - 1, math.ceil(pair(slow)))
            keep = 1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0), ("yarn", 1.0)])
@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
def test_prepared_rotation(attn, rot, scaling, factor):
    if scaling == "ntk" and rot == 2:
        with pytest.raises(attn.MonoError, match="NTK"):
            attn.Rope(rot, scaling=scaling, factor=factor)
        return
    r = attn.Rope(rot, theta=10000.0, scaling=scaling, factor=factor).value
    got = np.array(r.turns[:rot // 2]) * 2 * math.pi
    # a power, a division and a blend, each rounded to binary64
    np.testing.assert_allclose(got, _frequency(rot, 10000.0, scaling, factor), rtol=1e-13)
    want = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    assert abs(r.factor - want) <= 2.0 ** -52 * 2 and r.rot_dim == rot
    assert not any(r.turns[rot // 2:])
    assert attn.Rope(rot, attn_factor=0.5).value.factor == 0.5


@pytest.mark.parametrize("kw,frag", [
    (dict(rot_dim=0), "rot_dim"), (dict(rot_dim=3), "rot_dim"), (dict(rot_dim=258), "rot_dim"),
    (dict(offset=1), "offset"), (dict(offset=-2), "offset"), (dict(theta=1.0), "theta"),
    (dict(theta=float("inf")), "theta"), (dict(scaling="linear", factor=0.5), "factor"),
    (dict(scaling="linear", factor=float("nan")), "factor"), (dict(scaling="yarn", factor=2.0, orig_context=0), "YaRN"),
    (dict(scaling="yarn", factor=2.0, beta_fast=1.0), "YaRN"), (dict(attn_factor=float("inf")), "attn_factor"),
])
def test_rope_init_refuses(attn, kw, frag):
    with pytest.raises(attn.MonoError, match=frag):
        attn.Rope(**{**dict(rot_dim=64), **kw})


def test_rope_unknown_scaling(attn):
    with pytest.raises(ValueError, match="scaling"):
        attn.Rope(64, scaling="other")
    with pytest.raises(ValueError, match="fmt"):
        attn.Projection(64, 64, fmt="int8")


def test_rope_apply_refuses(attn):
    """Refused before any launch: the pointers are never read."""
    L, r = attn._lib(), attn.Rope(64, offset=64)

    def call(tokens=2, heads=2, head_dim=128, dtype=1, x=4096, xs=(256, 128), pos=64, out=1 << 20, os=(256, 128), at=None):
        rc = L.mono_rope_apply(r._at if at is None else at, tokens, heads, head_dim, dtype, x, *xs, pos, out, *os, 0, None)
        return rc, L.mono_attn_last_error().decode()

    for kw, frag in [(dict(tokens=-1), "tokens"), (dict(heads=65536), "heads"), (dict(head_dim=1025), "head_dim"),
                     (dict(head_dim=126), "passes the head's end"), (dict(dtype=2), "dtype"), (dict(x=None), "NULL"),
                     (dict(pos=None), "NULL"), (dict(out=4096, os=(512, 128)), "in place"), (dict(out=4096 + 512), "overlap"),
                     (dict(os=(0, 128)), "rows of out"), (dict(os=(256, 64)), "rows of out"),
                     (dict(os=(128, 128)), "rows of out")]:
        rc, why = call(**kw)
        assert rc == -1 and frag in why, (kw, why)
    assert call(tokens=0)[0] == 0 and call(heads=0, x=None, pos=None, out=None)[0] == 0
    broken = attn.RopeValue(rot_dim=500)
    assert call(at=ctypes.addressof(broken))[0] == -1


# ------------------------------------------------------- kv_index.h, on the host

SHIM = r"""
#include "kv_index.h"
using namespace mono;
extern "C" {
void view(int len, int n_new, int width, int cap, int* o) {
  const SeqView v = view_seq(len, n_new, width, cap);
  o[0] = v.n, o[1] = v.first, o[2] = v.bad, o[3] = v.bad_value;
}
int hi(int len, int n_new, int width, int cap, int j) { return row_hi(view_seq(len, n_new, width, cap), j, cap); }
int lo(int len, int n_new, int width, int cap, int j, int w) { return row_lo(view_seq(len, n_new, width, cap), j, w); }
int tiles(int len, int n_new, int width, int cap, int w, int t, int lead) {
  return seq_tiles(view_seq(len, n_new, width, cap), w, cap, t, lead);
}
int ok(int page, int n) { return page_ok(page, n); }
long long row(int page, int heads, int h, int p, int tok) { return code_row(page, heads, h, p, tok); }
unsigned share(unsigned total, unsigned grid, unsigned least) { return share_of(total, grid, least); }
unsigned slot(unsigned c, unsigned base, unsigned share) { return part_slot(c, base, share); }
}
"""


@pytest.fixture(scope="module")
def idx(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_index")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-shared", "-fPIC", "-I",
                    CSRC, str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.row.restype = ctypes.c_longlong
    for f in (L.share, L.slot):
        f.argtypes = [ctypes.c_uint] * 3
        f.restype = ctypes.c_uint
    return L


def _view(L, *a):
    o = (ctypes.c_int * 4)()
    L.view(*a, o)
    return tuple(o)


def test_rows_of_a_sequence(idx):
    assert _view(idx, 100, 3, 4, 1024) == (3, 97, 0, 0)
    assert _view(idx, 2, 4, 4, 1024) == (4, -2, 0, 0)          # shorter than its new tokens
    assert _view(idx, 5, 0, 4, 1024)[0] == 0 and _view(idx, -9, -3, 4, 1024) == (0, 0, 0, 0)
    assert _view(idx, 50, 9, 4, 1024) == (4, 46, 3, 9)         # more new tokens than rows
    assert _view(idx, 1025, 1, 4, 1024)[2:] == (2, 1025)
    assert _view(idx, -1, 1, 4, 1024) == (1, -1, 2, -1)
    top = 2 ** 31 - 1
    assert _view(idx, top, 8, 8, 1024)[1] == top - 8
    assert idx.hi(top, 8, 8, 1024, 7) == 1024 and idx.lo(top, 8, 8, 1024, 7, 5) == top - 5
    assert idx.tiles(top, 8, 8, 1024, 5, 32, 0) == 1              # nothing seen: one tile, so that rows are written
    assert [idx.hi(2, 4, 4, 64, j) for j in range(4)] == [-1, 0, 1, 2]
    assert idx.tiles(0, 1, 1, 64, 0, 16, 0) == 1 and idx.tiles(64, 0, 1, 64, 0, 16, 3) == 0


def test_rows_see_what_the_definition_says(idx):
    rng = random.Random(1)
    for _ in range(3000):
        cap = 16 * rng.randint(1, 20)
        length, width = rng.randint(0, cap), rng.randint(1, 8)
        n, w, t = rng.randint(1, width), rng.choice([0, 0, 1, rng.randint(1, 2 * cap)]), rng.choice([16, 32, 64])
        seen = []
        for j in range(n):
            pos = length - n + j
            want = [x for x in range(cap) if x <= pos and (w == 0 or x > pos - w)]
            lo, hi = idx.lo(length, n, width, cap, j, w), idx.hi(length, n, width, cap, j)
            assert want == list(range(lo, max(lo, hi))), (length, n, j, w)
            assert hi <= cap and lo >= 0
            seen += want
        lead = rng.randint(0, 3)
        count = idx.tiles(length, n, width, cap, w, t, lead) - lead
        first = idx.lo(length, n, width, cap, 0, w) // t
        assert set(x // t for x in seen) <= set(range(first, first + count)) and count >= 1


def test_pages_and_code_rows(idx):
    assert [idx.ok(p, 5) for p in (-2 ** 31, -1, 0, 4, 5, 2 ** 31 - 1)] == [0, 0, 1, 1, 0, 0]
    assert idx.row(2 ** 30, 1024, 1023, 128, 127) == (2 ** 30 * 1024 + 1023) * 128 + 127


def test_equal_runs_cover_the_line_and_keep_their_slots(idx):
    """Every tile belongs to one CTA; an item that spans CTAs has a slot of its
    own in each, below 2 x grid, and a CTA never uses a slot for two items."""
    rng = random.Random(2)
    for _ in range(400):
        grid, least, lead = rng.randint(1, 40), rng.choice([1, 2, 4]), rng.randint(0, 3)
        items = [rng.choice([1, 1, 2, rng.randint(1, 60)]) for _ in range(rng.randint(1, 40))]
        total = sum(items) + lead * len(items)
        share = idx.share(total, grid, least)
        assert share >= least and share * grid >= total
        base, used = 0, set()
        for n in items:
            base += lead
            first, last = base // share, (base + n - 1) // share
            assert last < grid
            if first != last:
                for c in range(first, last + 1):
                    slot = idx.slot(c, base, share)
                    assert slot // 2 == c and slot not in used
                    used.add(slot)
            base += n


def test_more_new_tokens_than_rows_have_no_work(idx):
    """Such a sequence is left out: no tile of it, whatever else is wrong."""
    for length in (-1, 0, 50, 1024, 1025):
        for lead in (0, 3):
            assert idx.tiles(length, 9, 8, 1024, 0, 32, lead) == 0
            assert idx.tiles(length, 8, 8, 1024, 0, 32, lead) > lead


def test_get_info_says_what_is_wrong(attn):
    """Not the reason of the call before it."""
    L = attn._lib()
    assert L.mono_rope_init(None, None) == -1
    for f, frag in ((L.mono_attn_get_info, "attn_get_info"), (L.mono_proj_get_info, "proj_get_info")):
        assert f(None, None) == -1 and frag in L.mono_attn_last_error().decode()
