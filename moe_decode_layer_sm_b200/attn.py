"""Thin ctypes binding of the attention half's operators (include/mono_attn.h):
rotary positions, the append to a paged 8-bit cache, attention over it and the
4-bit projections.

Argument checks and marshalling only; every operator runs in the library's
CUDA kernels.  The calls of a decode step (rope, append, attend, step) check and
marshal in a compiled module (csrc/call.cpp); where it takes a call for wrong,
the reasons are found here.  Tensors are CUDA tensors of the plan's device, the last
dimension contiguous, other strides free where the text says so.  Calls run on
the current stream of that device unless `stream` is given.
"""

import ctypes

import torch

from .binding import BF16, ERRORS, F32, MXFP4, MonoError, lib

INT4 = 4
SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_CODE = {torch.float32: F32, torch.bfloat16: BF16}
_NAME = {"f32": torch.float32, "bf16": torch.bfloat16}
ERRORS.setdefault(-9, "BAD_INDEX")

SYMBOLS = ["mono_rope_init", "mono_rope_apply", "mono_attn_plan", "mono_attn_append", "mono_attn_attend",
           "mono_attn_query_error", "mono_attn_get_info", "mono_attn_destroy", "mono_proj_plan", "mono_proj_pack",
           "mono_proj_step", "mono_proj_get_info", "mono_proj_destroy", "mono_attn_last_error"]

_vp, _i32, _i64, _f32, _f64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double


class RopeConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("rot_dim", "offset", "interleaved", "scaling")] + \
               [(n, _f64) for n in ("theta", "factor", "beta_fast", "beta_slow")] + \
               [("orig_context", _i32), ("attn_factor", _f64)]


class RopeValue(ctypes.Structure):
    _fields_ = [("rot_dim", _i32), ("offset", _i32), ("interleaved", _i32), ("factor", _f64), ("turns", _f64 * 128)]


class AttnConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("q_heads", "kv_heads", "head_dim", "page_size", "num_pages", "max_seqs", "max_pages",
                                    "max_new", "dtype")] + [("scale", _f32), ("window", _i32), ("device", _i32)]


class CacheStruct(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "k_scale", "v_scale")]


class AttnInfo(ctypes.Structure):
    _fields_ = [("grid", _i32), ("scratch_bytes", _i64)]


class AttnStatus(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("code", "what", "seq", "value")]


class ProjConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n_out", "n_in", "format", "group", "scale_dtype", "zeros", "dtype", "device")]


class ProjInfo(ctypes.Structure):
    _fields_ = [("cluster", _i32), ("packed_bytes", _i64)]


_ready = None
_call = None   # the compiled module


def _lib():
    global _ready, _call
    if _ready is None:
        L = lib()
        P = ctypes.POINTER
        L.mono_rope_init.argtypes = [P(RopeConfig), P(RopeValue)]
        L.mono_rope_apply.argtypes = [_vp, _i32, _i32, _i32, _i32, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i32, _vp]
        L.mono_attn_plan.argtypes = [P(AttnConfig), P(_vp)]
        L.mono_attn_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.mono_attn_attend.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.mono_attn_query_error.argtypes = [_vp, P(AttnStatus)]
        L.mono_attn_get_info.argtypes = [_vp, P(AttnInfo)]
        L.mono_proj_plan.argtypes = [P(ProjConfig), P(_vp)]
        L.mono_proj_pack.argtypes = [_vp, _vp, _vp, _vp, _vp]
        L.mono_proj_step.argtypes = [_vp, _i32, _vp, _i64, _vp, _i64, _vp]
        L.mono_proj_get_info.argtypes = [_vp, P(ProjInfo)]
        for f in SYMBOLS:
            getattr(L, f).restype = _i32
        for f in ("mono_attn_destroy", "mono_proj_destroy"):
            getattr(L, f).argtypes = [_vp]
            getattr(L, f).restype = None
        L.mono_attn_last_error.argtypes = []
        L.mono_attn_last_error.restype = ctypes.c_char_p
        try:
            from . import _call as compiled
        except ImportError as e:
            raise RuntimeError("_call.so is missing: build it with __graft_entry__.build() (g++, Python's headers, "
                               "torch)") from e
        _call, _ready = compiled, L
    return _ready


def _check(rc):
    if rc != 0:
        raise MonoError(rc, _lib().mono_attn_last_error().decode())


def _stream_of(device, stream):
    return torch.cuda.current_stream(device).cuda_stream if stream is None else stream.cuda_stream


def _refuse(who, why):
    if why:
        raise ValueError(f"{who}: " + "; ".join(why))


class Rope:
    """A prepared rotation (mono_rope_init): a host value, usable on any device.

    rot_dim dimensions of a head from `offset` on, in pairs (i, i + rot_dim/2)
    or, interleaved, (2i, 2i+1).  scaling: "none", "linear", "ntk" or "yarn"
    with its `factor`; orig_context, beta_fast and beta_slow are YaRN's.
    attn_factor multiplies the rotated values (0: 1, for YaRN 0.1 ln(factor) + 1)."""

    def __init__(self, rot_dim, theta=10000.0, scaling="none", factor=1.0, orig_context=4096, beta_fast=32.0,
                 beta_slow=1.0, interleaved=False, offset=0, attn_factor=0.0):
        if scaling not in SCALING:
            raise ValueError(f"Rope: unknown scaling {scaling!r}")
        cfg = RopeConfig(rot_dim=rot_dim, offset=offset, interleaved=int(interleaved), scaling=SCALING[scaling],
                         theta=theta, factor=factor, beta_fast=beta_fast, beta_slow=beta_slow,
                         orig_context=orig_context, attn_factor=attn_factor)
        self.value = RopeValue()
        _check(_lib().mono_rope_init(ctypes.byref(cfg), ctypes.byref(self.value)))
        self._at = ctypes.addressof(self.value)


def rope(x, positions, rope, out=None, transpose=False, stream=None):
    """mono_rope_apply: x [tokens][heads][head_dim] (fp32 or bf16, token and head
    strides free) rotated to positions (int32 [tokens]; below zero: a padding
    row, left as it was).  out None rotates in place.  transpose applies the
    transposed map (the gradient's).  Returns out."""
    out = x if out is None else out
    rc = _call.rope(rope._at, x, positions, out, transpose, None if stream is None else stream.cuda_stream)
    if rc:
        if rc == _call.NOT_TAKEN:
            _refuse_rope(x, positions, out)
        _check(rc)
    return out


def _refuse_rope(x, positions, out):
    why = []
    if x.dim() != 3 or positions.dim() != 1 or out.shape != x.shape or positions.shape[0] != x.shape[0]:
        why.append("x and out [tokens][heads][head_dim], positions [tokens]")
    if x.dtype not in _CODE or out.dtype != x.dtype:
        why.append("x and out must both be fp32 or bf16")
    if positions.dtype != torch.int32 or not positions.is_contiguous():
        why.append("positions must be contiguous int32")
    dev = x.get_device()
    if dev < 0 or positions.get_device() != dev or out.get_device() != dev:
        why.append("every tensor must be on one CUDA device")
    _refuse("rope", why or ["the last dimension must be contiguous"])


class KVCache:
    """One layer's paged cache: k, v float8_e4m3fn [num_pages][kv_heads][page_size][head_dim],
    k_scale, v_scale fp32 [num_pages][kv_heads]; contiguous CUDA tensors that the caller owns."""

    def __init__(self, k, v, k_scale, v_scale):
        why = []
        if k.dim() != 4 or v.shape != k.shape:
            why.append("k and v [num_pages][kv_heads][page_size][head_dim]")
        elif tuple(k_scale.shape) != tuple(k.shape[:2]) or v_scale.shape != k_scale.shape:
            why.append("k_scale and v_scale [num_pages][kv_heads]")
        if k.dtype != torch.float8_e4m3fn or v.dtype != torch.float8_e4m3fn:
            why.append("k and v must be float8_e4m3fn")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            why.append("k_scale and v_scale must be fp32")
        ts = (k, v, k_scale, v_scale)
        if not all(t.is_contiguous() for t in ts):
            why.append("every tensor must be contiguous")
        if not all(t.is_cuda and t.device == k.device for t in ts):
            why.append("every tensor must be on one CUDA device")
        _refuse("KVCache", why)
        self.k, self.v, self.k_scale, self.v_scale = ts
        self.shape, self.device = tuple(k.shape), k.get_device()
        self.struct = CacheStruct(*[t.data_ptr() for t in ts])
        self._at = ctypes.addressof(self.struct)

    @classmethod
    def empty(cls, num_pages, kv_heads, page_size, head_dim, device=0):
        d = torch.device("cuda", device)
        shape = (num_pages, kv_heads, page_size, head_dim)
        return cls(*[torch.zeros(shape, dtype=torch.uint8, device=d).view(torch.float8_e4m3fn) for _ in range(2)],
                   *[torch.zeros(shape[:2], device=d) for _ in range(2)])


class AttnPlan:
    """mono_attn_plan: the shapes of one attention sublayer and the scratch of its
    calls.  One plan serves any number of layers' caches; calls that overlap in
    time need a plan each."""

    def __init__(self, q_heads, kv_heads, head_dim, page_size, num_pages, max_seqs, max_pages, max_new=1, dtype="bf16",
                 scale=0.0, window=0, device=0):
        self._lib = _lib()
        self.cfg = AttnConfig(q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size,
                              num_pages=num_pages, max_seqs=max_seqs, max_pages=max_pages, max_new=max_new,
                              dtype=_CODE[_NAME[dtype]], scale=scale, window=window, device=device)
        self.handle = None
        h = _vp()
        _check(self._lib.mono_attn_plan(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.handle = h
        self.dtype, self.device = _NAME[dtype], device
        self.shape = (num_pages, kv_heads, page_size, head_dim)
        self.q_heads, self.kv_heads, self.head_dim, self.max_pages = q_heads, kv_heads, head_dim, max_pages
        self._at, self._code = h.value, self.cfg.dtype

    def _refuse(self, who, names, cache, x, heads, y, lens, table, n_new):
        why, d = [], self.device
        for name, t in zip(names, (x, y)):
            if t.dim() != 4 or t.shape[2] != heads or t.shape[3] != self.head_dim:
                why.append(f"{name} must be [seqs][width][{heads}][{self.head_dim}]")
            elif t.stride(3) != 1:
                why.append(f"{name}: the last dimension must be contiguous")
            if t.dtype != self.dtype or t.get_device() != d:
                why.append(f"{name} must be {self.dtype} on the plan's device")
        if x.shape[:2] != y.shape[:2]:
            why.append(f"{names[0]} and {names[1]} must have the same rows")
        if cache.shape != self.shape or cache.device != d:
            why.append(f"the cache must be {list(self.shape)} on the plan's device")
        n = x.shape[0] if x.dim() else 0
        if lens.dtype != torch.int32 or tuple(lens.shape) != (n,) or lens.get_device() != d or not lens.is_contiguous():
            why.append("lens must be contiguous int32 [seqs] on the plan's device")
        if table.dtype != torch.int32 or tuple(table.shape) != (n, self.max_pages) or table.get_device() != d \
                or not table.is_contiguous():
            why.append(f"the page table must be contiguous int32 [seqs][{self.max_pages}] on the plan's device")
        if n_new is not None and (n_new.dtype != torch.int32 or tuple(n_new.shape) != (n,) or n_new.get_device() != d
                                  or not n_new.is_contiguous()):
            why.append("n_new must be contiguous int32 [seqs] on the plan's device")
        _refuse(who, why or ["wrong arguments"])

    def append(self, cache, k, v, lens, table, rope=None, n_new=None, stream=None):
        """mono_attn_append: k, v [seqs][width][kv_heads][head_dim] (strides free)
        into the pages of `table` [seqs][max_pages]; lens [seqs] counts the new
        tokens, n_new [seqs] says how many of the rows are new (None: all).
        rope: the keys are rotated to their positions on the way."""
        if cache.shape != self.shape or cache.device != self.device:
            self._refuse("append", ("k", "v"), cache, k, self.kv_heads, v, lens, table, n_new)
        rc = _call.append(self._at, cache._at, self.kv_heads, self.head_dim, self._code, self.device, self.max_pages,
                          k, v, lens, table, n_new, None if rope is None else rope._at,
                          None if stream is None else stream.cuda_stream)
        if rc:
            if rc == _call.NOT_TAKEN:
                self._refuse("append", ("k", "v"), cache, k, self.kv_heads, v, lens, table, n_new)
            _check(rc)

    def attend(self, cache, q, lens, table, out, lse=None, n_new=None, stream=None):
        """mono_attn_attend: out [seqs][width][q_heads][head_dim] of q (rotated; the
        same shape, strides free) over the cached tokens that each row sees.  lse:
        fp32 [seqs][width][q_heads], the log of the sum of exponentials.  Returns out."""
        if cache.shape != self.shape or cache.device != self.device:
            self._refuse("attend", ("q", "out"), cache, q, self.q_heads, out, lens, table, n_new)
        rc = _call.attend(self._at, cache._at, self.q_heads, self.head_dim, self._code, self.device, self.max_pages,
                          q, out, lens, table, n_new, lse, None if stream is None else stream.cuda_stream)
        if rc:
            if rc == _call.NOT_TAKEN:
                if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:3]
                                        or not lse.is_contiguous() or lse.get_device() != self.device):
                    raise ValueError("attend: lse must be contiguous fp32 [seqs][width][q_heads] on the plan's device")
                self._refuse("attend", ("q", "out"), cache, q, self.q_heads, out, lens, table, n_new)
            _check(rc)
        return out

    def query_error(self):
        """Synchronise; (code, status) of the first page id, length or number of
        new tokens that a kernel could not use since the last query."""
        st = AttnStatus()
        rc = self._lib.mono_attn_query_error(self.handle, ctypes.byref(st))
        if rc not in (0, -9):
            _check(rc)
        return rc, st

    def info(self):
        inf = AttnInfo()
        _check(self._lib.mono_attn_get_info(self.handle, ctypes.byref(inf)))
        return {f: getattr(inf, f) for f, _ in AttnInfo._fields_}

    def close(self):
        if getattr(self, "handle", None):
            self._lib.mono_attn_destroy(self.handle)
            self.handle, self._at = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Projection:
    """mono_proj_plan: y = x W^T for up to 8 rows, W [n_out][n_in] in 4 bits.

    fmt "int4": unsigned codes with a zero point (8, or given at packing with
    zeros=True) and a scale ("bf16" or "f32") for each `group` inputs; "mxfp4":
    e2m1 codes with an e8m0 scale for each 32."""

    def __init__(self, n_out, n_in, fmt="int4", group=128, scale_dtype="bf16", zeros=False, dtype="bf16", device=0):
        self._lib = _lib()
        if fmt not in ("int4", "mxfp4"):
            raise ValueError(f"Projection: unknown fmt {fmt!r}")
        mx = fmt == "mxfp4"
        self.cfg = ProjConfig(n_out=n_out, n_in=n_in, format=MXFP4 if mx else INT4, group=group,
                              scale_dtype=BF16 if mx else _CODE[_NAME[scale_dtype]], zeros=int(zeros),
                              dtype=_CODE[_NAME[dtype]], device=device)
        self.handle = None
        h = _vp()
        _check(self._lib.mono_proj_plan(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.handle = h
        self.dtype, self.device = _NAME[dtype], device
        self.scale_dtype = torch.uint8 if mx else _NAME[scale_dtype]
        self.n_out, self.n_in, self.group, self.zeros = n_out, n_in, group, bool(zeros)
        self._at = h.value

    def pack(self, codes, scales, zeros=None, stream=None):
        """codes uint8 [n_out][n_in / 2] (the even input in the low nibble), scales
        [n_out][n_in / group], zeros uint8 [n_out][n_in / group]; contiguous."""
        why, groups = [], (self.n_out, self.n_in // self.group)
        if codes.dtype != torch.uint8 or tuple(codes.shape) != (self.n_out, self.n_in // 2):
            why.append(f"codes must be uint8 [{self.n_out}][{self.n_in // 2}]")
        if scales.dtype != self.scale_dtype or tuple(scales.shape) != groups:
            why.append(f"scales must be {self.scale_dtype} {list(groups)}")
        if (zeros is not None) != self.zeros:
            why.append("zeros must be given exactly when the plan has them")
        elif zeros is not None and (zeros.dtype != torch.uint8 or tuple(zeros.shape) != groups):
            why.append(f"zeros must be uint8 {list(groups)}")
        ts = [t for t in (codes, scales, zeros) if t is not None]
        if not all(t.is_contiguous() and t.get_device() == self.device for t in ts):
            why.append("every tensor must be contiguous, on the plan's device")
        _refuse("pack", why)
        _check(self._lib.mono_proj_pack(self.handle, codes.data_ptr(), scales.data_ptr(),
                                        None if zeros is None else zeros.data_ptr(), _stream_of(self.device, stream)))

    def step(self, x, y, stream=None):
        """y [rows][n_out] = x [rows][n_in] W^T, up to 8 rows, row strides free.  Returns y."""
        rc = _call.step(self._at, self.n_out, self.n_in, self.cfg.dtype, self.device, x, y,
                        None if stream is None else stream.cuda_stream)
        if rc:
            if rc == _call.NOT_TAKEN:
                self._refuse_step(x, y)
            _check(rc)
        return y

    def _refuse_step(self, x, y):
        why = []
        if x.dim() != 2 or x.shape[1] != self.n_in or tuple(y.shape) != (x.shape[0], self.n_out):
            why.append(f"x must be [rows][{self.n_in}] and y [rows][{self.n_out}]")
        elif x.stride(1) != 1 or (y.stride(1) != 1 and self.n_out > 1):
            why.append("the last dimension must be contiguous")
        if x.dtype != self.dtype or y.dtype != self.dtype:
            why.append(f"x and y must be {self.dtype}")
        if x.get_device() != self.device or y.get_device() != self.device:
            why.append("x and y must be on the plan's device")
        _refuse("step", why or ["wrong arguments"])

    def info(self):
        inf = ProjInfo()
        _check(self._lib.mono_proj_get_info(self.handle, ctypes.byref(inf)))
        return {f: getattr(inf, f) for f, _ in ProjInfo._fields_}

    def close(self):
        if getattr(self, "handle", None):
            self._lib.mono_proj_destroy(self.handle)
            self.handle, self._at = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
