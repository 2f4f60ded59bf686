// Host side of the attention half's operators: the C ABI declared in
// include/mono_attn.h — checks, plans, packing and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "mono_attn.h"
#include "proj.cuh"

using namespace mono;

namespace {

thread_local std::string g_error;

int fail(int code, const std::string& msg) {
  g_error = msg;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(e == cudaErrorMemoryAllocation ? MONO_ERR_OOM : MONO_ERR_CUDA,
              std::string(what) + ": " + cudaGetErrorString(e));
}

// no exception leaves a C entry point
template <typename F>
int guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    g_error.clear();
    return MONO_ERR_OOM;   // the strings and vectors here fail for want of memory only
  }
}

struct OnDevice {
  int prev = 0;
  explicit OnDevice(int device) {
    cudaGetDevice(&prev);
    if (prev != device) cudaSetDevice(device);
    else prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

constexpr size_t kSmemMax = 227 * 1024;   // of a CTA

size_t elem(int dtype) { return dtype == MONO_BF16 ? 2 : 4; }

int check_device(int device, std::string* why, int* sms) {
  int n = 0, major = 0, minor = 0;
  if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) *why += "no CUDA device\n";
  else if (device < 0 || device >= n) *why += "device ordinal out of range\n";
  if (!why->empty()) return fail(MONO_ERR_INVALID_ARG, *why);
  cudaError_t e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return cuda_fail(e, "device attributes");
  if (major != 10 || minor != 0)
    return fail(MONO_ERR_UNSUPPORTED_ARCH, "device " + std::to_string(device) + " is sm_" + std::to_string(major) +
                                               std::to_string(minor) + "; this library is built for sm_100a only");
  return MONO_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// bytes [lo, hi) that `n` steps of each of three strides cover
struct Extent {
  const char *lo, *hi;
};
Extent extent(const void* p, size_t el, const int64_t* stride, const int64_t* count, int dims, int64_t inner) {
  int64_t lo = 0, hi = inner;
  for (int i = 0; i < dims; ++i) {
    const int64_t d = stride[i] * (count[i] - 1);
    if (d < 0) lo += d;
    else hi += d;
  }
  const char* b = static_cast<const char*>(p);
  return {b + lo * (int64_t)el, b + hi * (int64_t)el};
}
bool meet(const Extent& a, const Extent& b) { return a.lo < b.hi && b.lo < a.hi; }

// whether two rows of `inner` elements of an output may share one: its
// strides, from the smallest, must each step over all that lies within it
bool self_overlap(const int64_t* stride, const int64_t* count, int dims, int64_t inner) {
  std::vector<std::pair<int64_t, int64_t>> d;
  for (int i = 0; i < dims; ++i)
    if (count[i] > 1) d.emplace_back(std::abs(stride[i]), count[i]);
  std::sort(d.begin(), d.end());
  int64_t span = inner;
  for (const auto& x : d) {
    if (x.first < span) return true;
    span += x.first * (x.second - 1);
  }
  return false;
}

}  // namespace

extern "C" const char* mono_attn_last_error(void) { return g_error.c_str(); }

// ------------------------------------------------------ rotary positions --

extern "C" int mono_rope_init(const mono_rope_config* c, mono_rope* out) {
  return guarded([&] {
    if (!c || !out) return fail(MONO_ERR_INVALID_ARG, "rope_init: NULL argument");
    std::string why;
    if (c->rot_dim < 2 || c->rot_dim > 256 || c->rot_dim % 2) why += "rot_dim must be even, 2..256\n";
    if (c->offset < 0 || c->offset % 2) why += "offset must be even and not negative\n";
    if (c->scaling < MONO_ROPE_NONE || c->scaling > MONO_ROPE_YARN) why += "unknown scaling\n";
    if (!(c->theta > 1.0) || !std::isfinite(c->theta)) why += "theta must be above 1\n";
    if (c->scaling != MONO_ROPE_NONE && (!(c->factor >= 1.0) || !std::isfinite(c->factor))) why += "factor must be at least 1\n";
    if (c->scaling == MONO_ROPE_NTK && c->rot_dim == 2) why += "NTK scaling needs rot_dim above 2\n";
    if (c->scaling == MONO_ROPE_YARN && (c->orig_context < 1 || !(c->beta_slow > 0.0) || !(c->beta_fast > c->beta_slow)))
      why += "YaRN needs orig_context >= 1 and beta_fast > beta_slow > 0\n";
    if (!(std::fabs(c->attn_factor) <= 1e6)) why += "attn_factor must be between -1e6 and 1e6\n";
    if (!why.empty()) return fail(MONO_ERR_INVALID_ARG, "rope_init: " + why);
    const double two_pi = 6.283185307179586476925286766559;
    const int rot = c->rot_dim;
    double theta = c->theta;
    if (c->scaling == MONO_ROPE_NTK) theta *= std::pow(c->factor, (double)rot / (rot - 2));
    // YaRN's ramp: from the pair that makes beta_fast turns over the original
    // context (kept) to the one that makes beta_slow (interpolated)
    double lo = 0, hi = 0;
    if (c->scaling == MONO_ROPE_YARN) {
      auto at = [&](double turns) { return rot * std::log(c->orig_context / (turns * two_pi)) / (2 * std::log(theta)); };
      lo = std::max(std::floor(at(c->beta_fast)), 0.0);
      hi = std::min(std::ceil(at(c->beta_slow)), (double)(rot - 1));
    }
    *out = mono_rope{};
    out->rot_dim = rot;
    out->offset = c->offset;
    out->interleaved = c->interleaved != 0;
    out->factor = c->attn_factor != 0.0 ? c->attn_factor : c->scaling == MONO_ROPE_YARN ? 0.1 * std::log(c->factor) + 1.0 : 1.0;
    for (int i = 0; i < rot / 2; ++i) {
      double f = std::pow(theta, -2.0 * i / rot);
      if (c->scaling == MONO_ROPE_LINEAR) f /= c->factor;
      if (c->scaling == MONO_ROPE_YARN) {
        const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
        f = f / c->factor * ramp + f * (1.0 - ramp);
      }
      out->turns[i] = f / two_pi;
    }
    return (int)MONO_OK;
  });
}

namespace {

std::string rope_reasons(const mono_rope* r, int head_dim) {
  std::string why;
  if (r->rot_dim < 2 || r->rot_dim > 256 || r->rot_dim % 2 || r->offset < 0 || r->offset % 2)
    why += "rope is not one that mono_rope_init filled\n";
  else if ((int64_t)r->offset + r->rot_dim > head_dim) why += "the rotated part passes the head's end\n";
  return why;
}

template <typename T, int VEC>
void launch_rope(const RopeParams& p, dim3 grid, cudaStream_t st) {
  const size_t smem = (size_t)p.tokens_per_cta * (p.rope.rot_dim / 2) * sizeof(float2);
  if (p.rope.interleaved) rope_kernel<T, VEC, true><<<grid, kRopeThreads, smem, st>>>(p);
  else rope_kernel<T, VEC, false><<<grid, kRopeThreads, smem, st>>>(p);
}

}  // namespace

extern "C" int mono_rope_apply(const mono_rope* rope, int tokens, int heads, int head_dim, int dtype, const void* x,
                               int64_t x_token, int64_t x_head, const int* pos, void* out, int64_t out_token,
                               int64_t out_head, int transpose, void* stream) {
  return guarded([&] {
    std::string why;
    if (!rope) return fail(MONO_ERR_INVALID_ARG, "rope_apply: NULL rope");
    if (tokens < 0) why += "tokens must not be negative\n";
    if (heads < 0 || heads > 65535) why += "heads must be 0..65535\n";
    if (head_dim < 2 || head_dim > 1024) why += "head_dim must be 2..1024\n";
    if (dtype != MONO_F32 && dtype != MONO_BF16) why += "dtype must be MONO_F32 or MONO_BF16\n";
    why += rope_reasons(rope, head_dim);
    if (tokens > 0 && heads > 0 && (!x || !pos || !out)) why += "NULL tensor pointer\n";
    if (!why.empty()) return fail(MONO_ERR_INVALID_ARG, "rope_apply: " + why);
    if (tokens == 0 || heads == 0) return (int)MONO_OK;
    const size_t el = elem(dtype);
    const bool in_place = x == out;
    const int64_t count[2] = {tokens, heads}, xs[2] = {x_token, x_head}, os[2] = {out_token, out_head};
    if (self_overlap(os, count, 2, head_dim)) return fail(MONO_ERR_INVALID_ARG, "rope_apply: rows of out overlap");
    if (in_place) {
      if (x_token != out_token || x_head != out_head)
        return fail(MONO_ERR_INVALID_ARG, "rope_apply: in place with other strides");
    } else if (meet(extent(x, el, xs, count, 2, head_dim), extent(out, el, os, count, 2, head_dim))) {
      return fail(MONO_ERR_INVALID_ARG, "rope_apply: x and out overlap");
    }
    RopeParams p{*rope, x, out, pos, x_token, x_head, out_token, out_head, tokens, heads, head_dim, 1, heads,
                 transpose != 0, in_place};
    // 16-byte vectors where every one of them is aligned and holds whole pairs of one kind
    const int vec = (int)(16 / el);
    const int unit = rope->interleaved ? rope->rot_dim : rope->rot_dim / 2;
    const bool wide = unit % vec == 0 && rope->offset % vec == 0 && head_dim % vec == 0 && aligned(x, 16) &&
                      aligned(out, 16) && x_token % vec == 0 && x_head % vec == 0 && out_token % vec == 0 &&
                      out_head % vec == 0;
    // Ten vectors a thread: few heads bring more tokens into a CTA (16000 tokens
    // of one head, bf16: 37 us with one each, 12 with 16), as long as there are
    // four CTAs an SM; few tokens bring their heads into several CTAs.  8191 x 40
    // heads, bf16, with 1, 4, 8 and 16 tokens a CTA: 48, 35, 32 and 36 us.
    constexpr int kSms = 148;
    const int64_t row = (int64_t)heads * head_dim / (wide ? vec : 1);
    p.tokens_per_cta = (int)std::min<int64_t>({kRopeTokens, (2559 + row) / row, std::max(1, tokens / (4 * kSms))});
    int parts = 1;
    if (tokens < 2 * kSms) parts = std::min(heads, (2 * kSms + tokens - 1) / tokens);
    p.heads_per_cta = (heads + parts - 1) / parts;
    // places within a CTA are 32-bit; strides that pass that leave it one row
    const auto reach = [&](int64_t token, int64_t head) {
      return (double)p.tokens_per_cta * std::fabs((double)token) + (double)p.heads_per_cta * std::fabs((double)head) + head_dim;
    };
    if (std::max(reach(x_token, x_head), reach(out_token, out_head)) >= 1073741824.0) p.tokens_per_cta = p.heads_per_cta = 1;
    const dim3 grid((tokens + p.tokens_per_cta - 1) / p.tokens_per_cta, (heads + p.heads_per_cta - 1) / p.heads_per_cta);
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == MONO_BF16) {
      if (wide) launch_rope<__nv_bfloat16, 8>(p, grid, st);
      else launch_rope<__nv_bfloat16, 1>(p, grid, st);
    } else {
      if (wide) launch_rope<float, 4>(p, grid, st);
      else launch_rope<float, 1>(p, grid, st);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? (int)MONO_OK : cuda_fail(e, "rope_apply");
  });
}

// ------------------------------------------------------------- attention --

struct mono_attn_plan_s {
  mono_attn_config cfg{};
  int page_shift = 0, sms = 0;
  int grid[2][2] = {};   // CTAs of an attend launch with 8 rows a warp, and with 16; narrow and wide
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  unsigned int* arrived = nullptr;
  BadIndex* bad = nullptr;
  int64_t scratch = 0;
};

namespace {

// rows of the call -> row tiles a warp, warps side by side, row blocks.  A
// warp takes 8 rows (the MMA's n) or 16; more rows share the keys' trip to the
// SM between warps (they read the same lines at the same time), and beyond 4
// warps between row blocks.  head_dim 256 keeps 8 rows a warp: the output of
// 16 would not fit its registers.
struct RowPlan {
  int nt, wr, blocks;
};
RowPlan plan_rows(int head_dim, int rows) {
  RowPlan r{1, 1, 1};
  if (head_dim <= 128 && rows > 8) r.nt = 2;
  const int per = 8 * r.nt;
  while (r.wr < 4 && r.wr * per < rows) r.wr *= 2;
  r.blocks = (rows + r.wr * per - 1) / (r.wr * per);
  return r;
}

// A launch is narrow, CTAs of 4 warps with items of their own, or wide, one CTA
// an SM, whose warps share an item.
struct Launch {
  RowPlan rows;
  bool wide;
  int warps(int head_dim) const { return wide ? attend_wide_warps(head_dim, rows.nt) : 4; }
  // tokens of a round
  int round(int head_dim) const {
    return (head_dim == 256 ? 16 : head_dim == 64 && rows.nt == 1 ? 64 : 32) * (warps(head_dim) / rows.wr);
  }
};

constexpr unsigned kLeastRounds = 1;   // of an attend CTA
constexpr unsigned kLeadRounds = 3;    // that an item's start takes

using AttendFn = void (*)(AttendParams);
struct AttendKernel {
  AttendFn fn;
  size_t (*smem)(int, int);
};
template <int D, int NT, bool F32>
AttendKernel attend_pick(bool wide) {
  constexpr int W = attend_wide_warps(D, NT);
  if (wide) return {&attend_kernel<D, NT, F32, W>, &AttendShape<D, NT, F32, W>::smem};
  return {&attend_kernel<D, NT, F32, 4>, &AttendShape<D, NT, F32, 4>::smem};
}
template <bool F32>
AttendKernel attend_of(int head_dim, int nt, bool wide) {
  if (head_dim == 64) return nt == 1 ? attend_pick<64, 1, F32>(wide) : attend_pick<64, 2, F32>(wide);
  if (head_dim == 128) return nt == 1 ? attend_pick<128, 1, F32>(wide) : attend_pick<128, 2, F32>(wide);
  return attend_pick<256, 1, F32>(wide);
}
AttendKernel attend_for(int head_dim, bool f32, const Launch& l) {
  return f32 ? attend_of<true>(head_dim, l.rows.nt, l.wide) : attend_of<false>(head_dim, l.rows.nt, l.wide);
}

// Wide up to one item (sequence, key head, row block) an SM: the parts of an
// item to join are a third as many, and its phases have an SM's warps.  With
// more items narrow CTAs run theirs side by side.  5 query heads a key head, 8
// key heads, bf16, us wide and narrow, sequences x tokens:
//   heads of 128   1 x 8000 15.4 and 21.7, 1 x 16000 19.7 and 28.9, 8 x 1000 14.5
//                  and 15.6, 8 x 8000 37.7 and 38.2, 16 x 1000 16.3 and 21.0; but
//                  8 x 2000 21.2 and 19.1; beyond an item an SM 64 x 200 30.4
//                  and 22.1, 64 x 1000 53.3 and 40.4
//   heads of 256   1 x 8000 22.1 and 30.2, 8 x 8000 60.0 and 61.5
//   heads of 64    1 x 8000 12.9 and 14.5, 16 x 1000 13.7 and 17.3; but 1 x 1000
//                  12.0 and 10.3, 8 x 8000 30.7 and 27.8
// And where a sequence may be longer than a narrow CTA's round (the lengths are
// on the device, the table's width is what is known here): at one token 8.7 and 8.0.
bool attend_wide(int64_t items, int sms, int64_t tokens, int narrow_round) {
  return items <= sms && tokens > narrow_round;
}

using AppendFn = void (*)(AppendParams);
struct AppendKernel {
  AppendFn fn;
  size_t (*ring)(int);
};
template <typename T, int U>
AppendKernel append_pick(bool each) {
  return {each ? &append_kernel<T, U, true> : &append_kernel<T, U, false>, &append_ring<T, U>};
}
template <typename T>
AppendKernel append_pick(int units, bool each) {
  return units == 4 ? append_pick<T, 4>(each) : units == 2 ? append_pick<T, 2>(each) : append_pick<T, 1>(each);
}
AppendKernel append_for(bool f32, int units, bool each) {
  return f32 ? append_pick<float>(units, each) : append_pick<__nv_bfloat16>(units, each);
}

template <typename T>
cudaError_t dalloc(T** p, size_t bytes, int64_t* total) {
  const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(p), bytes);
  if (e == cudaSuccess) *total += (int64_t)bytes;
  return e;
}

}  // namespace

extern "C" void mono_attn_destroy(mono_attn_plan_t* p) {
  if (!p) return;
  {
    OnDevice on(p->cfg.device);
    cudaFree(p->part_o);
    cudaFree(p->part_ml);
    cudaFree(p->arrived);
    cudaFree(p->bad);
  }
  delete p;
}

extern "C" int mono_attn_plan(const mono_attn_config* c, mono_attn_plan_t** out) {
  return guarded([&] {
    if (!c || !out) return fail(MONO_ERR_INVALID_ARG, "attn_plan: NULL argument");
    *out = nullptr;
    std::string why;
    auto need = [&](bool ok, const std::string& m) {
      if (!ok) why += m + "\n";
    };
    need(c->kv_heads >= 1 && c->kv_heads <= 1024, "kv_heads must be 1..1024");
    need(c->q_heads >= 1 && (c->kv_heads < 1 || (c->q_heads % c->kv_heads == 0 && c->q_heads / c->kv_heads <= 128)),
         "q_heads must be a multiple of kv_heads, at most 128 times as many");
    need(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, "head_dim must be 64, 128 or 256");
    need(c->page_size == 16 || c->page_size == 32 || c->page_size == 64 || c->page_size == 128,
         "page_size must be 16, 32, 64 or 128");
    need(c->num_pages >= 1, "num_pages must be at least 1");
    need(c->max_seqs >= 1 && c->max_seqs <= 4096, "max_seqs must be 1..4096");
    need(c->max_pages >= 1, "max_pages must be at least 1");
    need(c->max_new >= 1 && c->max_new <= 8, "max_new must be 1..8");
    need(c->dtype == MONO_F32 || c->dtype == MONO_BF16, "dtype must be MONO_F32 or MONO_BF16");
    need(c->window >= 0, "window must not be negative");
    need(std::isfinite(c->scale) && c->scale >= 0.f, "scale must be finite and not negative");
    if (why.empty()) {
      need((int64_t)c->max_pages * c->page_size < (1ll << 31) - 65536, "max_pages x page_size must stay below 2^31 - 65536");
      const RowPlan r = plan_rows(c->head_dim, c->max_new * (c->q_heads / c->kv_heads));
      const double tiles = (double)c->max_seqs * c->kv_heads * r.blocks *
                           ((double)c->max_pages * c->page_size / Launch{r, false}.round(c->head_dim) + 2 + kLeadRounds);
      need(tiles < 2147483648.0, "max_seqs x kv_heads x max_pages x page_size too large for the 32-bit work partition");
    }
    int sms = 0;
    const int rc = check_device(c->device, &why, &sms);
    if (rc) return rc;
    OnDevice on(c->device);
    mono_attn_plan_t* p = new mono_attn_plan_s();
    p->cfg = *c;
    if (p->cfg.scale == 0.f) p->cfg.scale = (float)(1.0 / std::sqrt((double)c->head_dim));
    while ((1 << p->page_shift) < c->page_size) ++p->page_shift;
    p->sms = sms;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < 6 && e == cudaSuccess; ++i)
      e = cudaFuncSetAttribute(append_for(c->dtype == MONO_F32, 1 << i / 2, i % 2).fn,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax - 1024);
    size_t rows_max = 0;   // grid x rows of a CTA
    const int group = c->q_heads / c->kv_heads;
    int blocks = 1;
    for (int i = 2; i < 2 * c->max_new + 2 && e == cudaSuccess; ++i) {
      const Launch l{plan_rows(c->head_dim, i / 2 * group), i % 2 == 1};
      const RowPlan& r = l.rows;
      const AttendKernel k = attend_for(c->head_dim, c->dtype == MONO_F32, l);
      const size_t smem = k.smem(c->max_seqs, r.wr);
      int occ = 0;
      e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, k.fn, 32 * l.warps(c->head_dim), smem);
      if (e == cudaSuccess && occ < 1) e = cudaErrorInvalidConfiguration;
      int& g = p->grid[r.nt - 1][l.wide];
      g = g ? std::min(g, occ * p->sms) : occ * p->sms;
      rows_max = std::max(rows_max, (size_t)occ * p->sms * r.wr * 8 * r.nt);
      blocks = std::max(blocks, r.blocks);
    }
    const size_t items = (size_t)c->max_seqs * c->kv_heads * blocks;
    if (e == cudaSuccess) e = dalloc(&p->part_o, 2 * rows_max * c->head_dim * 4, &p->scratch);
    if (e == cudaSuccess) e = dalloc(&p->part_ml, 2 * rows_max * 8, &p->scratch);
    if (e == cudaSuccess) e = dalloc(&p->arrived, items * 4, &p->scratch);
    if (e == cudaSuccess) e = dalloc(&p->bad, sizeof(BadIndex), &p->scratch);
    if (e == cudaSuccess) e = cudaMemset(p->arrived, 0, items * 4);
    if (e == cudaSuccess) e = cudaMemset(p->bad, 0, sizeof(BadIndex));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
      cudaGetLastError();
      mono_attn_destroy(p);
      return cuda_fail(e, "attn_plan");
    }
    *out = p;
    return (int)MONO_OK;
  });
}

namespace {

bool has_rows(const mono_seqs* s) { return s && s->seqs > 0 && s->width > 0; }

std::string call_reasons(const mono_attn_plan_t* p, const mono_kv_cache* c, const mono_seqs* s) {
  std::string why;
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) why += "NULL cache pointer\n";
  else if (!aligned(c->k, 16) || !aligned(c->v, 16)) why += "cache codes must be 16-byte aligned\n";
  if (!s) return why + "NULL seqs\n";
  if (s->seqs < 0 || s->seqs > p->cfg.max_seqs)
    why += "seqs " + std::to_string(s->seqs) + " outside [0, max_seqs = " + std::to_string(p->cfg.max_seqs) + "]\n";
  if (s->width < 0) why += "width must not be negative\n";
  if (has_rows(s) && (!s->lens || !s->table)) why += "NULL lens or table\n";
  return why;
}

}  // namespace

extern "C" int mono_attn_append(mono_attn_plan_t* p, const mono_kv_cache* c, const mono_seqs* s, const mono_rows* k,
                                const mono_rows* v, const mono_rope* rope, void* stream) {
  return guarded([&] {
    if (!p) return fail(MONO_ERR_INVALID_ARG, "append: NULL plan");
    std::string why = call_reasons(p, c, s);
    if (!k || !v || (has_rows(s) && (!k->p || !v->p))) why += "NULL k or v\n";
    if (rope) why += rope_reasons(rope, p->cfg.head_dim);
    if (s && s->width > (1 << 20)) why += "width above 2^20\n";
    if (!why.empty()) return fail(MONO_ERR_INVALID_ARG, "append: " + why);
    if (s->seqs == 0 || s->width == 0) return (int)MONO_OK;
    OnDevice on(p->cfg.device);
    AppendParams a{};
    const int D = p->cfg.head_dim, P = p->cfg.page_size;
    const mono_rows* rows[2] = {k, v};
    const size_t el = elem(p->cfg.dtype);
    const int vec = (int)(16 / el);
    a.vec_ok = 1;
    for (int i = 0; i < 2; ++i) {
      a.x[i] = rows[i]->p;
      a.x_seq[i] = rows[i]->seq;
      a.x_tok[i] = rows[i]->token;
      a.x_head[i] = rows[i]->head;
      a.vec_ok = a.vec_ok && aligned(rows[i]->p, 16) && rows[i]->seq % vec == 0 && rows[i]->token % vec == 0 &&
                 rows[i]->head % vec == 0;
    }
    a.codes[0] = (uint8_t*)c->k;
    a.codes[1] = (uint8_t*)c->v;
    a.scales[0] = c->k_scale;
    a.scales[1] = c->v_scale;
    a.lens = s->lens;
    a.n_new = s->n_new;
    a.table = s->table;
    a.bad = p->bad;
    a.width = s->width;
    a.kv_heads = p->cfg.kv_heads;
    a.head_dim = D;
    a.head_log2 = D == 64 ? 6 : D == 128 ? 7 : 8;
    a.page_shift = p->page_shift;
    a.num_pages = p->cfg.num_pages;
    a.max_pages = p->cfg.max_pages;
    a.rotate = rope != nullptr;
    if (rope) a.rope = *rope;
    const int spans = std::min((s->width + P - 2) / P + 1, p->cfg.max_pages);
    // heads share a CTA's angles once there are CTAs enough without them
    int hpc = 1;
    while (hpc < p->cfg.kv_heads && hpc < 8 &&
           (int64_t)spans * s->seqs * 2 * ((p->cfg.kv_heads + 2 * hpc - 1) / (2 * hpc)) >= 8 * p->sms)
      hpc *= 2;
    a.heads_per_cta = hpc;
    const int groups = (p->cfg.kv_heads + hpc - 1) / hpc;
    const int most = std::min(P, s->width), total = most * D / 16;   // new tokens of a page, units of 16 values
    const int units = total <= append_threads(1) ? 1 : total <= 2 * append_threads(2) ? 2 : 4;
    const int threads = std::max(128, (total / units + 31) / 32 * 32);   // (older codes may have to be taken along)
    const bool each = rope && ((rope->offset | (rope->interleaved ? rope->rot_dim : rope->rot_dim / 2)) & 7);
    const AppendKernel kernel = append_for(p->cfg.dtype == MONO_F32, units, each);
    const size_t smem = kernel.ring(threads) + (rope ? append_angles(most, rope->rot_dim) : 0);
    kernel.fn<<<dim3(spans, 2 * groups, s->seqs), threads, smem, (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? (int)MONO_OK : cuda_fail(e, "append");
  });
}

extern "C" int mono_attn_attend(mono_attn_plan_t* p, const mono_kv_cache* c, const mono_seqs* s, const mono_rows* q,
                                const mono_rows* out, float* lse, void* stream) {
  return guarded([&] {
    if (!p) return fail(MONO_ERR_INVALID_ARG, "attend: NULL plan");
    std::string why = call_reasons(p, c, s);
    if (!q || !out || (has_rows(s) && (!q->p || !out->p))) why += "NULL q or out\n";
    if (s && s->width > p->cfg.max_new)
      why += "width " + std::to_string(s->width) + " above max_new = " + std::to_string(p->cfg.max_new) + "\n";
    if (!why.empty()) return fail(MONO_ERR_INVALID_ARG, "attend: " + why);
    if (s->seqs == 0 || s->width == 0) return (int)MONO_OK;
    const size_t el = elem(p->cfg.dtype);
    const int64_t count[3] = {s->seqs, s->width, p->cfg.q_heads}, qs[3] = {q->seq, q->token, q->head},
                  os[3] = {out->seq, out->token, out->head};
    if (meet(extent(q->p, el, qs, count, 3, p->cfg.head_dim), extent(out->p, el, os, count, 3, p->cfg.head_dim)))
      return fail(MONO_ERR_INVALID_ARG, "attend: q and out overlap");
    if (self_overlap(os, count, 3, p->cfg.head_dim)) return fail(MONO_ERR_INVALID_ARG, "attend: rows of out overlap");
    OnDevice on(p->cfg.device);
    const int group = p->cfg.q_heads / p->cfg.kv_heads;
    const int64_t tokens = (int64_t)p->cfg.max_pages * p->cfg.page_size;
    const RowPlan r = plan_rows(p->cfg.head_dim, s->width * group);
    const Launch l{r, attend_wide((int64_t)s->seqs * p->cfg.kv_heads * r.blocks, p->sms, tokens,
                                   Launch{r, false}.round(p->cfg.head_dim))};
    const AttendKernel k = attend_for(p->cfg.head_dim, p->cfg.dtype == MONO_F32, l);
    AttendParams a{};
    a.k = (const uint8_t*)c->k;
    a.v = (const uint8_t*)c->v;
    a.ks = c->k_scale;
    a.vs = c->v_scale;
    a.q = q->p;
    a.out = out->p;
    a.q_seq = q->seq, a.q_tok = q->token, a.q_head = q->head;
    a.o_seq = out->seq, a.o_tok = out->token, a.o_head = out->head;
    a.lse = lse;
    a.lens = s->lens;
    a.n_new = s->n_new;
    a.table = s->table;
    a.bad = p->bad;
    a.part_o = p->part_o;
    a.part_ml = p->part_ml;
    a.arrived = p->arrived;
    a.seqs = s->seqs;
    a.width = s->width;
    a.q_heads = p->cfg.q_heads;
    a.kv_heads = p->cfg.kv_heads;
    a.group = group;
    a.page_shift = p->page_shift;
    a.num_pages = p->cfg.num_pages;
    a.max_pages = p->cfg.max_pages;
    a.window = p->cfg.window;
    a.wr = r.wr;
    a.row_blocks = r.blocks;
    a.least = kLeastRounds;
    a.lead = kLeadRounds;
    a.q_vec = aligned(q->p, 4 * el) && q->seq % 4 == 0 && q->token % 4 == 0 && q->head % 4 == 0;
    a.o_vec = aligned(out->p, 4 * el) && out->seq % 4 == 0 && out->token % 4 == 0 && out->head % 4 == 0;
    a.scale_log2 = p->cfg.scale * 1.4426950408889634f;
    // no more CTAs than the call can have rounds
    const int64_t rounds = (tokens / l.round(p->cfg.head_dim) + 2 + kLeadRounds) * s->seqs * p->cfg.kv_heads * r.blocks;
    const int grid = (int)std::min<int64_t>(p->grid[r.nt - 1][l.wide], rounds);
    k.fn<<<grid, 32 * l.warps(p->cfg.head_dim), k.smem(s->seqs, r.wr), (cudaStream_t)stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? (int)MONO_OK : cuda_fail(e, "attend");
  });
}

extern "C" int mono_attn_query_error(mono_attn_plan_t* p, mono_attn_status* st) {
  return guarded([&] {
    if (!p) return fail(MONO_ERR_INVALID_ARG, "query_error: NULL plan");
    OnDevice on(p->cfg.device);
    BadIndex b{};
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&b, p->bad, sizeof(b), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && b.what) e = cudaMemset(p->bad, 0, sizeof(b));
    if (e == cudaSuccess && b.what) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "query_error");
    if (st) *st = mono_attn_status{b.what ? MONO_ERR_BAD_INDEX : 0, (int)b.what, b.seq, b.value};
    if (!b.what) return (int)MONO_OK;
    const char* what = b.what == kBadPage ? "page id" : b.what == kBadLen ? "length" : "number of new tokens";
    return fail(MONO_ERR_BAD_INDEX, std::string("bad ") + what + " " + std::to_string(b.value) + " in sequence " +
                                        std::to_string(b.seq));
  });
}

extern "C" int mono_attn_get_info(const mono_attn_plan_t* p, mono_attn_info* info) {
  if (!p || !info) return guarded([] { return fail(MONO_ERR_INVALID_ARG, "attn_get_info: NULL argument"); });
  info->grid = std::max(std::max(p->grid[0][0], p->grid[0][1]), std::max(p->grid[1][0], p->grid[1][1]));
  info->scratch_bytes = p->scratch;
  return MONO_OK;
}

// ----------------------------------------------------- 4-bit projections --

struct mono_proj_plan_s {
  mono_proj_config cfg{};
  int kblocks = 0, groups = 0, nblocks = 0, cluster = 1, teams = 1, sms = 0, sc = 0;
  uint8_t* codes = nullptr;
  uint8_t* scales = nullptr;
  uint8_t* zeros = nullptr;
  unsigned int* special = nullptr;
  int64_t packed = 0;
  bool is_packed = false;
};

namespace {

using ProjFn = void (*)(ProjParams);
template <bool F32>
ProjFn proj_pick(int sc, bool zp) {
  if (sc == kScaleE8m0) return &proj_kernel<F32, kScaleE8m0, false>;
  if (sc == kScaleF32) return zp ? &proj_kernel<F32, kScaleF32, true> : &proj_kernel<F32, kScaleF32, false>;
  return zp ? &proj_kernel<F32, kScaleBf16, true> : &proj_kernel<F32, kScaleBf16, false>;
}
ProjFn proj_for(bool f32, int sc, bool zp) { return f32 ? proj_pick<true>(sc, zp) : proj_pick<false>(sc, zp); }
using ProjSmemFn = size_t (*)(int, int);
template <bool F32>
ProjSmemFn proj_smem_pick(int sc, bool zp) {
  if (sc == kScaleE8m0) return &proj_smem<F32, kScaleE8m0, false>;
  if (sc == kScaleF32) return zp ? &proj_smem<F32, kScaleF32, true> : &proj_smem<F32, kScaleF32, false>;
  return zp ? &proj_smem<F32, kScaleBf16, true> : &proj_smem<F32, kScaleBf16, false>;
}
size_t proj_smem_of(bool f32, int sc, bool zp, int rows, int kb) {
  return (f32 ? proj_smem_pick<true>(sc, zp) : proj_smem_pick<false>(sc, zp))(rows, kb);
}

constexpr double kProjSumCost = 4, kProjPushCost = 7;   // of an output block's sums, in blocks of a warp
}  // namespace

extern "C" void mono_proj_destroy(mono_proj_plan_t* p) {
  if (!p) return;
  {
    OnDevice on(p->cfg.device);
    cudaFree(p->codes);
    cudaFree(p->scales);
    cudaFree(p->zeros);
    cudaFree(p->special);
  }
  delete p;
}

extern "C" int mono_proj_plan(const mono_proj_config* c, mono_proj_plan_t** out) {
  return guarded([&] {
    if (!c || !out) return fail(MONO_ERR_INVALID_ARG, "proj_plan: NULL argument");
    *out = nullptr;
    std::string why;
    auto need = [&](bool ok, const std::string& m) {
      if (!ok) why += m + "\n";
    };
    const bool mx = c->format == MONO_MXFP4, f32 = c->dtype == MONO_F32;
    need(c->n_out >= 1 && c->n_out <= 1 << 30, "n_out must be 1..2^30");
    need(mx || c->format == MONO_INT4, "format must be MONO_INT4 or MONO_MXFP4");
    need(c->group >= 32 && c->group % 32 == 0, "group must be a multiple of 32");
    need(!mx || c->group == 32, "group must be 32 for MONO_MXFP4");
    need(c->n_in >= 1 && (c->group < 1 || c->n_in % c->group == 0), "n_in must be a positive multiple of group");
    need(mx || c->scale_dtype == MONO_F32 || c->scale_dtype == MONO_BF16, "scale_dtype must be MONO_F32 or MONO_BF16");
    need(!mx || !c->zeros, "MONO_MXFP4 has no zeros");
    need(f32 || c->dtype == MONO_BF16, "dtype must be MONO_F32 or MONO_BF16");
    const int kblocks = c->n_in / 32;
    const int sc = mx ? kScaleE8m0 : c->scale_dtype == MONO_F32 ? kScaleF32 : kScaleBf16;
    int limit = 1;   // blocks of a CTA that fit its shared memory
    while (why.empty() && proj_smem_of(f32, sc, c->zeros != 0, 8, limit + 1) <= kSmemMax) ++limit;
    need((kblocks + 7) / 8 <= limit, "n_in too large: " + std::to_string(limit * 8 * 32) + " at most for this dtype");
    int sms = 0;
    const int rc = check_device(c->device, &why, &sms);
    if (rc) return rc;
    OnDevice on(c->device);
    mono_proj_plan_t* p = new mono_proj_plan_s();
    p->cfg = *c;
    p->sms = sms;
    p->kblocks = kblocks;
    p->groups = c->n_in / c->group;
    p->nblocks = (c->n_out + kProjN - 1) / kProjN;
    p->sc = sc;
    // The inputs are cut among a cluster, or a CTA's warps into teams, where that
    // shortens the longest run of a warp: rounds over the output blocks x (a
    // warp's blocks of each + what the sums of a round cost).
    double best = 1e30;
    auto offer = [&](int cluster, int teams) {
      const int kb = (kblocks + cluster - 1) / cluster, slots = p->sms / cluster * teams, tw = kProjWarps / teams;
      if (kb > limit) return;
      const double cost = (double)((p->nblocks + slots - 1) / slots) *
                          ((kb + tw - 1) / tw + (cluster > 1 ? kProjPushCost : kProjSumCost));
      if (cost < best) best = cost, p->cluster = cluster, p->teams = teams;
    };
    for (int x = 1; x <= 8; x *= 2) offer(x, 1);
    offer(1, 2);
    const size_t sb = p->sc == kScaleBf16 ? 2 : p->sc == kScaleF32 ? 4 : 1;
    const size_t n64 = (size_t)p->nblocks * p->groups * kProjN;
    cudaError_t e = dalloc(&p->codes, (size_t)p->nblocks * kblocks * 1024, &p->packed);
    if (e == cudaSuccess) e = dalloc(&p->scales, n64 * sb, &p->packed);
    if (e == cudaSuccess && c->zeros) e = dalloc(&p->zeros, n64, &p->packed);
    if (e == cudaSuccess) e = dalloc(&p->special, 4, &p->packed);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(proj_for(f32, p->sc, c->zeros != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kSmemMax);
    if (e != cudaSuccess) {
      cudaGetLastError();
      mono_proj_destroy(p);
      return cuda_fail(e, "proj_plan");
    }
    *out = p;
    return (int)MONO_OK;
  });
}

extern "C" int mono_proj_pack(mono_proj_plan_t* p, const void* codes, const void* scales, const void* zeros,
                              void* stream) {
  return guarded([&] {
    if (!p) return fail(MONO_ERR_INVALID_ARG, "proj_pack: NULL plan");
    std::string why;
    if (!codes || !scales) why += "NULL codes or scales\n";
    if (p->cfg.zeros && !zeros) why += "NULL zeros\n";
    if (!p->cfg.zeros && zeros) why += "zeros given to a plan without them\n";
    if (!why.empty()) return fail(MONO_ERR_INVALID_ARG, "proj_pack: " + why);
    OnDevice on(p->cfg.device);
    cudaStream_t st = (cudaStream_t)stream;
    const long long words = (long long)p->nblocks * p->kblocks * 256, n64 = (long long)p->nblocks * p->groups * kProjN;
    auto grid = [&](long long n) { return (unsigned)std::min<long long>((n + 255) / 256, 148LL * 64); };
    pack_proj_codes_kernel<<<grid(words), 256, 0, st>>>((const uint8_t*)codes, (uint32_t*)p->codes, p->cfg.n_out,
                                                         p->cfg.n_in, words, p->cfg.format == MONO_MXFP4);
    const cudaError_t cleared = cudaMemsetAsync(p->special, 0, 4, st);
    if (cleared != cudaSuccess) return cuda_fail(cleared, "proj_pack");
    if (p->sc == kScaleBf16)
      pack_proj_groups_kernel<<<grid(n64), 256, 0, st>>>((const uint16_t*)scales, (uint16_t*)p->scales, p->cfg.n_out,
                                                          p->groups, n64, 0, p->special, 0x7FFFu, (127u + 64u) << 7);
    else if (p->sc == kScaleF32)
      pack_proj_groups_kernel<<<grid(n64), 256, 0, st>>>((const uint32_t*)scales, (uint32_t*)p->scales, p->cfg.n_out,
                                                          p->groups, n64, 0, p->special, 0x7FFFFFFFu, (127u + 64u) << 23);
    else
      pack_proj_groups_kernel<<<grid(n64), 256, 0, st>>>((const uint8_t*)scales, p->scales, p->cfg.n_out, p->groups,
                                                          n64, 0, p->special, 0xFFu, 127u + 64u);
    if (zeros)
      pack_proj_groups_kernel<<<grid(n64), 256, 0, st>>>((const uint8_t*)zeros, p->zeros, p->cfg.n_out, p->groups, n64,
                                                          15, nullptr, 0u, 0u);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "proj_pack");
    p->is_packed = true;
    return (int)MONO_OK;
  });
}

extern "C" int mono_proj_step(mono_proj_plan_t* p, int rows, const void* x, int64_t x_row, void* y, int64_t y_row,
                              void* stream) {
  return guarded([&] {
    if (!p) return fail(MONO_ERR_INVALID_ARG, "proj_step: NULL plan");
    if (rows < 0 || rows > 8) return fail(MONO_ERR_INVALID_ARG, "proj_step: rows " + std::to_string(rows) + " outside 0..8");
    if (!p->is_packed) return fail(MONO_ERR_NOT_PACKED, "proj_step: no packed weights");
    if (rows == 0) return (int)MONO_OK;
    if (!x || !y) return fail(MONO_ERR_INVALID_ARG, "proj_step: NULL x or y");
    const bool f32 = p->cfg.dtype == MONO_F32;
    const size_t el = elem(p->cfg.dtype);
    const int64_t n = rows;
    if (meet(extent(x, el, &x_row, &n, 1, p->cfg.n_in), extent(y, el, &y_row, &n, 1, p->cfg.n_out)))
      return fail(MONO_ERR_INVALID_ARG, "proj_step: x and y overlap");
    if (self_overlap(&y_row, &n, 1, p->cfg.n_out)) return fail(MONO_ERR_INVALID_ARG, "proj_step: rows of y overlap");
    OnDevice on(p->cfg.device);
    ProjParams a{};
    a.codes = p->codes;
    a.scales = p->scales;
    a.zeros = p->zeros;
    a.special = p->special;
    a.x = x;
    a.y = y;
    a.x_row = x_row;
    a.y_row = y_row;
    a.rows = rows;
    a.n_out = p->cfg.n_out;
    a.kblocks = p->kblocks;
    a.blocks_per_group = p->cfg.group / 32;
    a.groups = p->groups;
    a.nblocks = p->nblocks;
    a.x_vec = aligned(x, 16) && x_row % (int64_t)(16 / el) == 0;
    auto log2_of = [](int v) {
      int l = 0;
      while ((1 << l) < v) ++l;
      return l;
    };
    a.teams_log2 = log2_of(p->teams);
    a.cluster_log2 = log2_of(p->cluster);
    const int clusters = std::min((p->nblocks + p->teams - 1) / p->teams, p->sms / p->cluster);
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3(clusters * p->cluster);
    lc.blockDim = dim3(kProjThreads);
    lc.dynamicSmemBytes = proj_smem_of(f32, p->sc, p->zeros != nullptr, rows, (p->kblocks + p->cluster - 1) / p->cluster);
    lc.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p->cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, proj_for(f32, p->sc, p->zeros != nullptr), a);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_fail(e, "proj_step");
    }
    return (int)MONO_OK;
  });
}

extern "C" int mono_proj_get_info(const mono_proj_plan_t* p, mono_proj_info* info) {
  if (!p || !info) return guarded([] { return fail(MONO_ERR_INVALID_ARG, "proj_get_info: NULL argument"); });
  info->cluster = p->cluster;
  info->packed_bytes = p->packed;
  return MONO_OK;
}
