// The append to the paged 8-bit cache: rotate the new keys, find each touched
// page's scale, encode, and re-encode a page's older codes where its scale grows.
#pragma once
#include "kv_index.h"
#include "rope.cuh"

namespace mono {

// the first index that a kernel could not use (mono_attn_query_error)
struct BadIndex {
  unsigned int what;   // 0: none
  int seq, value;
};

__device__ __forceinline__ void record_bad(BadIndex* e, int what, int seq, int value) {
  if (atomicCAS(&e->what, 0u, (unsigned)what) == 0u) {
    e->seq = seq;
    e->value = value;
  }
}

struct AppendParams {
  uint8_t* codes[2];   // k, v
  float* scales[2];
  const void* x[2];
  long long x_seq[2], x_tok[2], x_head[2];
  const int* lens;
  const int* n_new;
  const int* table;
  BadIndex* bad;
  int width, kv_heads, head_dim, head_log2, page_shift, num_pages, max_pages, heads_per_cta, rotate, vec_ok;
  mono_rope rope;
};

constexpr float kFp8Max = 448.0f;
constexpr int kAppendThreads = 512;   // of a CTA at most

// A float whose nearest e4m3 value is that of q: truncated, with its last bit
// set if anything was cut off, so that rounding twice cannot pass a border.
__device__ __forceinline__ float fp8_sticky(double q) {
  const float f = __double2float_rz(q);
  return (double)f != q && fabsf(f) < kFp8Max ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// whether q, a quotient that is off by less than 4 units in the last place,
// may lie on the other side of a border between two codes: halfway between two
// mantissas of 3 bits.  Below 2^-6 the codes are as far apart as above it.
__device__ __forceinline__ bool fp8_near_border(float q) {
  float m = fabsf(q);
  if (m < 0.015625f) m += 0.015625f;
  return ((__float_as_uint(m) + 0x80008u) & 0xFFFF0u) == 0u;
}

// q = x / s near a border: on the side of it where the exact quotient lies, or
// on it.  The border has 5 bits, so the sign of x - border x s is exact.
__device__ __forceinline__ float fp8_settle(float q, float x, float s) {
  const float low = fabsf(q) < 0.015625f ? 0.015625f : 0.f;
  const float b = __uint_as_float((__float_as_uint(fabsf(q) + low) & 0xFFF00000u) | 0x80000u) - low;
  const float r = fmaf(-b, s, fabsf(x));
  const uint32_t y = __float_as_uint(b) + (r > 0.f ? 1u : r < 0.f ? 0xFFFFFFFFu : 0u);
  return __uint_as_float(y | (__float_as_uint(q) & 0x80000000u));
}

__device__ __forceinline__ uint16_t fp8_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint2 fp8_pack8(const float* q) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = fp8_pair(q[2 * i], q[2 * i + 1]);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// eight values from a row, by one or two 16-byte loads where that is allowed
template <typename T>
__device__ __forceinline__ Vec<T, 8> load8(const T* p, bool wide) {
  Vec<T, 8> v;
  if (wide) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      const Vec<T, N> a = reinterpret_cast<const Vec<T, N>*>(p)[i];
#pragma unroll
      for (int j = 0; j < N; ++j) v.v[i * N + j] = a.v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = p[i];
  }
  return v;
}

__device__ __forceinline__ double2 turn_by(double2 a, double2 b) {   // angles added
  return make_double2(a.x * b.x - a.y * b.y, a.y * b.x + a.x * b.y);
}

__device__ __forceinline__ double2 turn_of(double turns) {
  double sn, cs;
  sincospi(2.0 * (turns - rint(turns)), &sn, &cs);
  return make_double2(cs, sn);
}

// cos and sin of the tokens of a page in two levels: token t of the new ones is
// turned by far[t / 8] and then by near[t % 8].  A level's pairs lie so that
// threads which take eight pairs each meet no bank conflict.
struct Turns {
  const double2* far;
  const double2* near;
  int half, off, step;   // step: (half + 7) / 8
  bool interleaved;
  __device__ __forceinline__ int slot(int i) const { return (i & 7) * step + (i >> 3); }
  __device__ __forceinline__ double2 at(int t, int i) const {
    return turn_by(far[(t >> 3) * 8 * step + slot(i)], near[(t & 7) * 8 * step + slot(i)]);
  }
  // dimension d (rotated) of a token's head
  template <typename T>
  __device__ double one(const T* row, int t, int d) const {
    const int r = d - off;
    const bool low = interleaved ? !(r & 1) : r < half;
    const int i = interleaved ? r >> 1 : low ? r : r - half;
    const int e = interleaved ? (low ? d + 1 : d - 1) : low ? d + half : d - half;
    const double2 cs = at(t, i);
    return cs.x * (double)to_f(row[d]) + (low ? -cs.y : cs.y) * (double)to_f(row[e]);
  }
};

// The code of dimension d of a token's head, from its exact value; out of
// line, since few values need it and the kernel's code would not fit the
// instruction cache with it at every place.
template <typename T>
__device__ __noinline__ uint8_t exact_code(const Turns& turns, bool rotated, const T* row, int t, int d, float s) {
  const double y = rotated ? turns.one(row, t, d) : (double)to_f(row[d]);
  return (uint8_t)fp8_pair(fp8_sticky(y / (double)s), 0.f);
}

// the largest finite magnitude of eight values of a token's head
template <typename T>
__device__ __noinline__ double finite_max8(const Turns& turns, bool rotate, const T* row, int t, int d) {
  double most = 0.0;
#pragma unroll 1
  for (int e = d; e < d + 8; ++e) {
    const double m =
        fabs(rotate && e >= turns.off && e < turns.off + 2 * turns.half ? turns.one(row, t, e) : (double)to_f(row[e]));
    if (m > most && m < 1e300) most = m;
  }
  return most;
}

// shared memory of `most` new tokens in a page
__host__ __device__ inline size_t append_smem(int most, int rot_dim) {
  return (size_t)((most + 7) / 8 + (most < 8 ? most : 8)) * 8 * ((rot_dim / 2 + 7) / 8) * sizeof(double2);
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const unsigned int hi = __reduce_max_sync(0xFFFFFFFFu, (unsigned int)(v >> 32));
  const unsigned int lo = __reduce_max_sync(0xFFFFFFFFu, (unsigned int)(v >> 32) == hi ? (unsigned int)v : 0u);
  return ((unsigned long long)hi << 32) | lo;
}

// One CTA: the new tokens of one page of one sequence, for a group of heads
// of k or of v.  grid (pages a sequence's new tokens can touch, 2 x head
// groups, sequences).  A page's head is held in registers between the two
// passes that its scale needs (largest magnitude, then the codes), so the
// input is read once, the next head's while this one's is reduced.
//
// The rotation is done in binary64 and a code near a border is found from it
// again, so codes and scales are those of the exact rotated values: a key's
// code does not depend on which call, or which neighbours, it was written
// with.  Two sines and cosines a pair and page, shared by its heads, give all
// the others by turning; a thread holds both halves of its pairs, so a value
// costs one conversion each way and four binary64 operations.
//
// U: units of 16 values that a thread holds of a page's head.  EACH: rotations
// whose offset or halves no vector of eight respects.
template <typename T, int U, bool EACH>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) unsigned char smem_append[];   // near [8][slots], far [tokens / 8][slots]
  __shared__ unsigned long long red[2][kAppendThreads / 32];
  const int s = blockIdx.z, which = blockIdx.y & 1, hg = blockIdx.y >> 1;
  const int P = 1 << p.page_shift, D = p.head_dim, cap = p.max_pages << p.page_shift;
  const int n_new = p.n_new ? __ldg(p.n_new + s) : p.width;
  if (n_new <= 0) return;
  const SeqView sv = view_seq(__ldg(p.lens + s), n_new, p.width, cap);
  const bool reporter = threadIdx.x == 0 && blockIdx.y == 0;
  if (sv.bad && reporter && blockIdx.x == 0) record_bad(p.bad, sv.bad, s, sv.bad_value);
  // tokens [a, b) of this page
  const int first = max(sv.first, 0);
  const int page_no = (first >> p.page_shift) + blockIdx.x;
  if (page_no >= p.max_pages) return;
  const int a = max(first, page_no << p.page_shift);
  const int b = min(sv.first + sv.n, (page_no + 1) << p.page_shift);
  if (a >= b) return;
  const int page = __ldg(p.table + (long long)s * p.max_pages + page_no);
  if (!page_ok(page, p.num_pages)) {
    if (reporter) record_bad(p.bad, kBadPage, s, page);
    return;
  }
  const int older = a - (page_no << p.page_shift);   // the page's tokens before the new ones
  const int rot = p.rope.rot_dim, half = rot >> 1, off = p.rope.offset;
  // how a token's head is cut into units: all rows as they come; (half layout)
  // eight pairs, the unrotated vectors two by two; (interleaved) 16 in a row
  enum { kPlain, kHalves, kInterleaved, kEach };
  const int mode = !p.rotate || which ? kPlain : EACH ? kEach : p.rope.interleaved ? kInterleaved : kHalves;
  const int upt_log2 = p.head_log2 - 4, nunits = (b - a) << upt_log2;
  const int h0 = hg * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.kv_heads);
  const T* x0 = reinterpret_cast<const T*>(p.x[which]) + (long long)s * p.x_seq[which] +
                (long long)(a - sv.first) * p.x_tok[which];

  int tok[U], da[U], db[U], pair[U];   // token, the two vectors' places, kHalves: first pair or -1
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int idx = threadIdx.x + u * blockDim.x, c = idx & ((1 << upt_log2) - 1);
    live[u] = idx < nunits;
    tok[u] = idx >> upt_log2;
    da[u] = c * 16, db[u] = da[u] + 8, pair[u] = -1;
    if (!EACH && mode == kHalves) {
      const int nh = half >> 3, j = 16 * (c - nh);
      if (c < nh) pair[u] = c * 8, da[u] = off + c * 8, db[u] = da[u] + half;
      else da[u] = j < off ? j : j + rot, db[u] = j + 8 < off ? j + 8 : j + 8 + rot;
    }
  }
  auto row_of = [&](int h, int u) { return x0 + (long long)h * p.x_head[which] + (long long)tok[u] * p.x_tok[which]; };
  Vec<T, 8> raw[U][2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (live[u]) {
        const T* row = row_of(h, u);
        raw[u][0] = load8(row + da[u], p.vec_ok);
        raw[u][1] = load8(row + db[u], p.vec_ok);
      }
  };
  constexpr bool kAhead = U * sizeof(T) <= 8;   // registers for the next head's values
  if (kAhead) fetch(h0);

  Turns turns{nullptr, nullptr, half, off, (half + 7) >> 3, p.rope.interleaved != 0};
  if (mode != kPlain) {
    const int n_far = (b - a + 7) >> 3, n_near = min(b - a, 8), slots = 8 * turns.step;
    double2* near = reinterpret_cast<double2*>(smem_append);
    double2* far = near + n_near * slots;
    for (int i = threadIdx.x; i < 2 * half; i += blockDim.x) {
      const bool is_far = i < half;
      const int pr = is_far ? i : i - half;
      const double f = p.rope.turns[pr];
      double2 w = make_double2(1.0, 0.0);
      if (is_far) {
        w = turn_of(f * (double)a);
        w.x *= (double)p.rope.factor, w.y *= (double)p.rope.factor;
      }
      const int n = is_far ? n_far : n_near;
      double2* to = (is_far ? far : near) + turns.slot(pr);
      if (n > 1) {
        const double2 by = turn_of(is_far ? 8.0 * f : f);
        for (int k = 0; k < n; ++k, w = turn_by(w, by)) to[k * slots] = w;
      } else {
        *to = w;
      }
    }
    turns.far = far;
    turns.near = near;
    __syncthreads();
  }

  int turn = 0;
  for (int h = h0; h < h1; ++h) {
    float* scale_at = p.scales[which] + (long long)page * p.kv_heads + h;
    const float was = older > 0 ? *scale_at : 0.f;
    if (!kAhead) fetch(h);
    float val[U][16];
    double amax = 0.0;
    float top = 0.f;   // of the values that are not rotated
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (live[u]) {
        if (!EACH && mode == kHalves && pair[u] >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const double2 cs = turns.at(tok[u], pair[u] + i);
            const double x1 = to_f(raw[u][0].v[i]), x2 = to_f(raw[u][1].v[i]);
            const double y1 = cs.x * x1 - cs.y * x2, y2 = cs.y * x1 + cs.x * x2;
            amax = fmax(amax, fabs(y1));   // NaN is left out
            amax = fmax(amax, fabs(y2));
            val[u][i] = (float)y1, val[u][8 + i] = (float)y2;
          }
        } else {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int d = v ? db[u] : da[u];
            if (!EACH && mode == kInterleaved && d >= off && d < off + rot) {
#pragma unroll
              for (int i = 0; i < 8; i += 2) {
                const double2 cs = turns.at(tok[u], (d - off + i) >> 1);
                const double x1 = to_f(raw[u][v].v[i]), x2 = to_f(raw[u][v].v[i + 1]);
                const double y1 = cs.x * x1 - cs.y * x2, y2 = cs.y * x1 + cs.x * x2;
                amax = fmax(amax, fabs(y1));   // NaN is left out
                amax = fmax(amax, fabs(y2));
                val[u][8 * v + i] = (float)y1, val[u][8 * v + i + 1] = (float)y2;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float x = to_f(raw[u][v].v[i]);
                if (EACH && mode == kEach && d + i >= off && d + i < off + rot) {
                  const double y = turns.one(row_of(h, u), tok[u], d + i);
                  amax = fmax(amax, fabs(y));
                  x = (float)y;
                } else {
                  top = fmaxf(top, fabsf(x));
                }
                val[u][8 * v + i] = x;
              }
            }
          }
        }
      }
    if (kAhead && h + 1 < h1) fetch(h + 1);
    // the largest of the page's head; positive doubles order as their bits do
    amax = fmax(amax, (double)top);
    auto block_max = [&](unsigned long long v) {
      v = warp_max(v);
      if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = v;
      __syncthreads();   // red has two places: the one after next writes here behind the next barrier
      v = warp_max((threadIdx.x & 31) < (blockDim.x >> 5) ? red[turn][threadIdx.x & 31] : 0ull);
      turn ^= 1;
      return __longlong_as_double((long long)v);
    };
    amax = block_max((unsigned long long)__double_as_longlong(amax));
    if (!(amax < 1e300)) {   // an infinity among them: once more, without
      amax = 0.0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (live[u]) {
          amax = fmax(amax, finite_max8(turns, mode != kPlain, row_of(h, u), tok[u], da[u]));
          amax = fmax(amax, finite_max8(turns, mode != kPlain, row_of(h, u), tok[u], db[u]));
        }
      amax = block_max((unsigned long long)__double_as_longlong(amax));
    }
    float sc = fmaxf((float)(amax / (double)kFp8Max), 1.175494351e-38f);
    if (older > 0) sc = fmaxf(sc, was);
    const float rs = __fdiv_rn(1.f, sc);
    uint8_t* dst = p.codes[which] + code_row(page, p.kv_heads, h, P, 0) * D;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (live[u]) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int d = v ? db[u] : da[u];
          uint8_t* to = dst + (older + tok[u]) * D + d;
          unsigned int near = 0u;
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y[i] = val[u][8 * v + i] * rs;
            if (fp8_near_border(y[i])) near |= 1u << i;
          }
          // (bf16 values meet borders often: 0.3 % of them, half of a warp's vectors)
          if (!EACH && near && !(mode == kHalves ? pair[u] >= 0 : mode == kInterleaved && d >= off && d < off + rot)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (near & (1u << i)) y[i] = fp8_settle(y[i], val[u][8 * v + i], sc);
            near = 0u;
          }
          *reinterpret_cast<uint2*>(to) = fp8_pack8(y);
#pragma unroll 1
          for (; near; near &= near - 1) {
            const int e = d + __ffs(near) - 1;
            to[e - d] = exact_code(turns, mode != kPlain && e >= off && e < off + rot, row_of(h, u), tok[u], e, sc);
          }
        }
      }
    if (older > 0 && sc > was) {
      const double ratio = (double)was / (double)sc;
      for (int idx = threadIdx.x; idx < older << (upt_log2 + 1); idx += blockDim.x) {
        uint2* at = reinterpret_cast<uint2*>(dst + idx * 8);
        const uint2 w = *at;
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = e4m3x2_to_f2((uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1))));
          v[2 * i] = fp8_sticky((double)f.x * ratio);
          v[2 * i + 1] = fp8_sticky((double)f.y * ratio);
        }
        *at = fp8_pack8(v);
      }
    }
    if (threadIdx.x == 0) *scale_at = sc;
  }
}

}  // namespace mono
