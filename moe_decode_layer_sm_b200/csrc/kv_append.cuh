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
  int width, kv_heads, head_dim, page_shift, num_pages, max_pages, heads_per_cta, rotate, vec_ok;
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
// may lie on the other side of a border between two codes
__device__ __forceinline__ bool fp8_near_border(float q) {
  const int low = (int)(__float_as_uint(q) & 0xFFFFFu) - 0x80000;
  return (low <= 4 && low >= -4) || fabsf(q) < 0.015625f;
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

template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float* v) {
  if (vec) {
    constexpr int N = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
      const Vec<T, N> a = reinterpret_cast<const Vec<T, N>*>(p)[i];
#pragma unroll
      for (int j = 0; j < N; ++j) v[i * N + j] = to_f(a.v[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f(p[i]);
  }
}

// cos and sin of the tokens of a page in two levels: token t of the new ones is
// turned by far[t / 8] and then by near[t % 8]
struct Turns {
  const double2* far;
  const double2* near;
  int half, off;
  bool interleaved;
  __device__ __forceinline__ double2 at(int t, int i) const {
    const double2 a = far[(t >> 3) * half + i], b = near[(t & 7) * half + i];
    return make_double2(a.x * b.x - a.y * b.y, a.y * b.x + a.x * b.y);
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

// One CTA: the new tokens of one page of one sequence, for a group of heads
// of k or of v.  grid (pages a sequence's new tokens can touch, 2 x head
// groups, sequences).  A page's head is held in registers between the two
// passes that its scale needs (largest magnitude, then the codes), so the
// input is read once.  The angles are computed once for all heads of the CTA.
// The rotation is done in binary64 and a code near a border is found from it
// again, so codes and scales are those of the exact rotated values: a key's
// code does not depend on which call, or which neighbours, it was written with.
// VECS: vectors of 8 values that a thread holds of a page's head.
template <typename T, int VECS>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) unsigned char smem_append[];   // far [tokens / 8][half], near [8][half]
  __shared__ double red[32];
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
  const int vpt = D >> 3;                            // vectors of 8 a token
  const int half = p.rope.rot_dim >> 1, off = p.rope.offset;
  const bool rotate = p.rotate && which == 0;
  Turns turns{nullptr, nullptr, half, off, p.rope.interleaved != 0};
  if (rotate) {
    const int n_far = (b - a + 7) >> 3, n_near = min(b - a, 8);
    double2* far = reinterpret_cast<double2*>(smem_append);
    double2* near = far + n_far * half;
    for (int i = threadIdx.x; i < (n_far + n_near) * half; i += blockDim.x) {
      const int t = i / half, pair = i - t * half;
      const bool is_far = t < n_far;
      double x = p.rope.turns[pair] * (double)(is_far ? a + 8 * t : t - n_far);
      x -= rint(x);
      double sn, cs;
      sincospi(2.0 * x, &sn, &cs);
      const double f = is_far ? (double)p.rope.factor : 1.0;
      far[i] = make_double2(f * cs, f * sn);
    }
    turns.far = far;
    turns.near = near;
    __syncthreads();
  }
  const int h0 = hg * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.kv_heads);
  const int nvec = (b - a) * vpt;
  for (int h = h0; h < h1; ++h) {
    const T* x = reinterpret_cast<const T*>(p.x[which]) + (long long)s * p.x_seq[which] +
                 (long long)h * p.x_head[which] + (long long)(a - sv.first) * p.x_tok[which];
    float* scale_at = p.scales[which] + (long long)page * p.kv_heads + h;
    const float was = older > 0 ? *scale_at : 0.f;
    float val[VECS][8];
    double amax = 0.0;
    auto turned = [&](int d) { return rotate && d >= off && d < off + 2 * half; };
#pragma unroll
    for (int q = 0; q < VECS; ++q) {
      const int idx = threadIdx.x + q * blockDim.x;
      if (idx < nvec) {
        const int t = idx / vpt, d0 = (idx - t * vpt) * 8;
        const T* row = x + (long long)t * p.x_tok[which];
        load8(row + d0, p.vec_ok, val[q]);
        float top = 0.f;   // of the values as they came
        if (!turned(d0) && !turned(d0 + 7) && (off < d0 || off >= d0 + 8 || !rotate)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(val[q][i]) <= 3.402823466e38f ? fabsf(val[q][i]) : 0.f);
          amax = fmax(amax, (double)top);
        } else if (p.vec_ok && half % 8 == 0 && off % 8 == 0) {
          const int r = d0 - off;
          double y[8];
          if (p.rope.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const double2 cs = turns.at(t, (r + i) >> 1);
              const double x1 = val[q][i], x2 = val[q][i + 1];
              y[i] = cs.x * x1 - cs.y * x2;
              y[i + 1] = cs.y * x1 + cs.x * x2;
            }
          } else {
            const bool low = r < half;
            float other[8];
            load8(row + (low ? d0 + half : d0 - half), true, other);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const double2 cs = turns.at(t, (low ? r : r - half) + i);
              y[i] = cs.x * (double)val[q][i] + (low ? -cs.y : cs.y) * (double)other[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const double m = fabs(y[i]);
            if (m > amax && m < 1e300) amax = m;
            val[q][i] = (float)y[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const double y = turned(d0 + i) ? turns.one(row, t, d0 + i) : (double)val[q][i];
            const double m = fabs(y);
            if (m > amax && m < 1e300) amax = m;
            val[q][i] = (float)y;
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmax(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    __syncthreads();   // red of the head before is read
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) amax = fmax(amax, red[w]);
    float sc = fmaxf((float)(amax / (double)kFp8Max), 1.175494351e-38f);
    if (older > 0) sc = fmaxf(sc, was);
    const float rs = __fdiv_rn(1.f, sc);
    uint8_t* dst = p.codes[which] + code_row(page, p.kv_heads, h, P, 0) * D;
#pragma unroll
    for (int q = 0; q < VECS; ++q) {
      const int idx = threadIdx.x + q * blockDim.x;
      if (idx < nvec) {
        bool near = false;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = val[q][i] * rs;
          near |= fp8_near_border(y[i]);
        }
        if (near) {
          const int t = idx / vpt, d0 = (idx - t * vpt) * 8;
          const T* row = x + (long long)t * p.x_tok[which];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fp8_near_border(y[i]))
              y[i] = fp8_sticky((turned(d0 + i) ? turns.one(row, t, d0 + i) : (double)val[q][i]) / (double)sc);
        }
        *reinterpret_cast<uint2*>(dst + (long long)older * D + idx * 8) = fp8_pack8(y);
      }
    }
    if (older > 0 && sc > was) {
      const double ratio = (double)was / (double)sc;
      for (int idx = threadIdx.x; idx < older * vpt; idx += blockDim.x) {
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
