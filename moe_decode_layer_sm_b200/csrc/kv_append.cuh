// The append to the paged 8-bit cache: rotate the new keys, find each touched
// page's scale, encode, and re-encode a page's older codes where its scale grows.
#pragma once
#include <type_traits>

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

// all but the N newest groups of asynchronous copies have arrived
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr float kFp8Max = 448.0f;
constexpr int kAppendThreads = 512;   // of a CTA at most
__host__ __device__ constexpr int append_threads(int units) { return units == 4 ? kAppendThreads : 256; }

__device__ __forceinline__ float rcp_approx(float x) {   // to one unit in the last place
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A float whose nearest e4m3 value is that of q: truncated, with its last bit
// set if anything was cut off, so that rounding twice cannot pass a border.
__device__ __forceinline__ float fp8_sticky(double q) {
  const float f = __double2float_rz(q);
  return (double)f != q && fabsf(f) < kFp8Max ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// whether q, a quotient that is off by less than 4 units in the last place,
// may lie on the other side of a border between two codes: halfway between two
// mantissas of 3 bits.  Below 2^-6 the codes are as far apart as above it.
__device__ __forceinline__ bool fp8_near_border(float q) {
  float m = fabsf(q);
  if (m < 0.015625f) m += 0.015625f;
  return ((__float_as_uint(m) + 0x80008u) & 0xFFFF0u) == 0u;
}

// q, an approximation of x / s (finite, s a normal number well above the
// smallest), moved next to the border between its two codes, to the side on
// which the exact quotient lies, or onto it.  The border has 5 bits, so the
// sign of x - border x s is exact.  A q that lies beyond a code ends next to
// that code's other border, on the side of the code.  low: 2^-6 where |q| is
// below it (codes are as far apart there as above), else 0; their sum is cut,
// so that it stays below 2^-5, where codes lie further apart.  x is a number:
// of NaN the step by bits would make a zero.
__device__ __forceinline__ float fp8_place(float q, float x, float s, float low) {
  const float b = __uint_as_float((__float_as_uint(__fadd_rz(fabsf(q), low)) & 0xFFF00000u) | 0x80000u) - low;
  const int r = __float_as_int(fmaf(-b, s, fabsf(x)));
  return __uint_as_float((__float_as_uint(b) + min(max(r, -1), 1)) | (__float_as_uint(q) & 0x80000000u));
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

// heads that a thread has in flight or in use, and their bytes in a CTA
template <typename T, int U>
__host__ __device__ constexpr int append_heads() {
  return U == 4 ? 4 / (int)sizeof(T) : sizeof(T) == 2 ? 3 : 2;
}
template <typename T, int U>
__host__ __device__ constexpr size_t append_ring(int threads) {
  return (size_t)append_heads<T, U>() * U * 16 * sizeof(T) * threads;
}

// shared memory of the angles of `most` new tokens in a page
__host__ __device__ inline size_t append_angles(int most, int rot_dim) {
  return (size_t)((most + 7) / 8 + (most < 8 ? most : 8)) * 8 * ((rot_dim / 2 + 7) / 8) * sizeof(double2);
}

// positive numbers order as their bits do
__device__ __forceinline__ unsigned int warp_max(unsigned int v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
  const unsigned int hi = __reduce_max_sync(0xFFFFFFFFu, (unsigned int)(v >> 32));
  const unsigned int lo = __reduce_max_sync(0xFFFFFFFFu, (unsigned int)(v >> 32) == hi ? (unsigned int)v : 0u);
  return ((unsigned long long)hi << 32) | lo;
}

// One CTA: the new tokens of one page of one sequence, for a group of heads
// of k or of v.  grid (pages a sequence's new tokens can touch, 2 x head
// groups, sequences).  A page's head is held in registers between the two
// passes that its scale needs (largest magnitude, then the codes), so the
// input is read once, and the next heads' are on their way meanwhile.
//
// The rotation is done in binary64 and a code near a border is found from it
// again, so codes and scales are those of the exact rotated values, rounded
// once.  (A page's scale goes by all the tokens that a call writes to it, and
// older codes are rounded again where it grows: a page filled token by token
// may hold other codes than one written at once.)  Two sines and cosines a pair
// and page, shared by its heads, give all the others by turning; a thread holds
// both halves of its pairs, so a value costs one conversion each way and four
// binary64 operations.
//
// Measured: 10486 tokens of 4 prompts, 8 heads of 128, bf16, rotated 43.5 us, not
// rotated 33, fp32 58 (64 and 107 MB: 10 and 16 us of memory); bound by
// instructions, of which a head's and a CTA's own are more than the values'.
// One token of 8 sequences 3.7 us.
//
// U: units of 16 values that a thread holds of a page's head.  EACH: rotations
// whose offset or halves no vector of eight respects.
template <typename T, int U, bool EACH>
__global__ void __launch_bounds__(append_threads(U), U == 4 ? 1 : 3) append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ __align__(16) unsigned char smem_append[];   // the ring, near [8][slots], far [tokens / 8][slots]
  __shared__ unsigned long long red[2][kAppendThreads / 32];
  const int s = blockIdx.z, which = blockIdx.y & 1, hg = blockIdx.y >> 1;
  const int P = 1 << p.page_shift, D = p.head_dim, cap = p.max_pages << p.page_shift;
  const int n_new = p.n_new ? __ldg(p.n_new + s) : p.width;
  if (n_new <= 0) return;
  const SeqView sv = view_seq(__ldg(p.lens + s), n_new, p.width, cap);
  const bool reporter = threadIdx.x == 0 && blockIdx.y == 0;
  if (sv.bad && reporter && blockIdx.x == 0) record_bad(p.bad, sv.bad, s, sv.bad_value);
  if (sv.left_out) return;
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

  // a unit's token, its first vector's place and the second's from there, its
  // first pair (kHalves; -1: not rotated), and where the first vector is read
  int tok[U], da[U], dx[U], pair[U];
  bool live[U];
  const T* from[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int idx = threadIdx.x + u * blockDim.x, c = idx & ((1 << upt_log2) - 1);
    live[u] = idx < nunits;
    tok[u] = idx >> upt_log2;
    da[u] = c * 16, dx[u] = 8, pair[u] = -1;
    if (!EACH && mode == kHalves) {
      const int nh = half >> 3, j = 16 * (c - nh);
      if (c < nh) {
        pair[u] = c * 8, da[u] = off + c * 8, dx[u] = half;
      } else {
        da[u] = j < off ? j : j + rot;
        dx[u] = (j + 8 < off ? j + 8 : j + 8 + rot) - da[u];
      }
    }
    from[u] = x0 + (long long)h0 * p.x_head[which] + (long long)tok[u] * p.x_tok[which] + da[u];
  }
  auto row_of = [&](int h, int u) { return x0 + (long long)h * p.x_head[which] + (long long)tok[u] * p.x_tok[which]; };
  // A thread's values of kHeads heads in shared memory, each asked for kHeads
  // heads before it is used; a thread reads only what it copied.  Rows that
  // 16-byte copies cannot take are read when they are needed.
  constexpr int kHeads = append_heads<T, U>(), kVecs = sizeof(T) / 2;   // 16-byte pieces of eight values
  auto place = [&](int head, int u, int v, int k) {
    return ((((head % kHeads) * U + u) * 2 + v) * kVecs + k) * blockDim.x + threadIdx.x;
  };
  uint4* ring = reinterpret_cast<uint4*>(smem_append);
  auto fetch = [&](int head) {
    if (p.vec_ok && head < h1 - h0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (live[u]) {
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
              cp_async16(ring + place(head, u, v, k), from[u] + v * dx[u] + k * (16 / (int)sizeof(T)));
          from[u] += p.x_head[which];
        }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kHeads - 1; ++i) fetch(i);

  Turns turns{nullptr, nullptr, half, off, (half + 7) >> 3, p.rope.interleaved != 0};
  if (mode != kPlain) {
    const int n_far = (b - a + 7) >> 3, n_near = min(b - a, 8), slots = 8 * turns.step;
    double2* near = reinterpret_cast<double2*>(smem_append + append_ring<T, U>(blockDim.x));
    double2* far = near + n_near * slots;
    for (int i = threadIdx.x; i < 2 * half; i += blockDim.x) {
      const bool is_far = i < half;
      const int pr = is_far ? i : i - half;
      const double f = p.rope.turns[pr];
      double2 w = make_double2(1.0, 0.0);
      if (is_far) {
        w = turn_of(f * (double)a);
        w.x *= p.rope.factor, w.y *= p.rope.factor;
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
  auto block_max = [&](auto v) {
    decltype(v)* at = reinterpret_cast<decltype(v)*>(red[turn]);   // red has two places: the one after next
    v = warp_max(v);                                               // writes here behind the next barrier
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_max((threadIdx.x & 31) < (blockDim.x >> 5) ? at[threadIdx.x & 31] : decltype(v)(0));
    turn ^= 1;
    return v;
  };
  float* scale_at = p.scales[which] + (long long)page * p.kv_heads + h0;
  uint8_t* dst = p.codes[which] + code_row(page, p.kv_heads, h0, P, 0) * D;
  auto heads = [&](auto plain) {
    constexpr bool PLAIN = decltype(plain)::value;   // nothing is rotated
    for (int h = h0; h < h1; ++h, ++scale_at, dst += P * D) {
      const float was = older > 0 ? *scale_at : 0.f;
      fetch(h - h0 + kHeads - 1);
      cp_async_wait<kHeads - 1>();
      float val[U][16];
      double amax = 0.0;
      float top = 0.f;   // of the values that are not rotated; NaN if one of them is
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (live[u]) {
          Vec<T, 8> raw[2];
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (p.vec_ok) {
#pragma unroll
              for (int k = 0; k < kVecs; ++k)
                reinterpret_cast<uint4*>(&raw[v])[k] = ring[place(h - h0, u, v, k)];
            } else {
              const T* at = row_of(h, u) + da[u] + v * dx[u];
#pragma unroll
              for (int i = 0; i < 8; ++i) raw[v].v[i] = at[i];
            }
          if (!PLAIN && !EACH && mode == kHalves && pair[u] >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const double2 cs = turns.at(tok[u], pair[u] + i);
              const double x1 = to_f(raw[0].v[i]), x2 = to_f(raw[1].v[i]);
              const double y1 = cs.x * x1 - cs.y * x2, y2 = cs.y * x1 + cs.x * x2;
              amax = fmax(amax, fmax(fabs(y1), fabs(y2)));   // NaN is left out
              val[u][i] = (float)y1, val[u][8 + i] = (float)y2;
            }
          } else {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int d = da[u] + v * dx[u];
              if (!PLAIN && !EACH && mode == kInterleaved && d >= off && d < off + rot) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                  const double2 cs = turns.at(tok[u], (d - off + i) >> 1);
                  const double x1 = to_f(raw[v].v[i]), x2 = to_f(raw[v].v[i + 1]);
                  const double y1 = cs.x * x1 - cs.y * x2, y2 = cs.y * x1 + cs.x * x2;
                  amax = fmax(amax, fmax(fabs(y1), fabs(y2)));
                  val[u][8 * v + i] = (float)y1, val[u][8 * v + i + 1] = (float)y2;
                }
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float x = to_f(raw[v].v[i]);
                  if (!PLAIN && EACH && d + i >= off && d + i < off + rot) {
                    const double y = turns.one(row_of(h, u), tok[u], d + i);
                    amax = fmax(amax, fabs(y));
                    x = (float)y;
                  } else {
                    top = max_nan(top, fabsf(x));
                  }
                  val[u][8 * v + i] = x;
                }
              }
            }
          }
        }
      // the largest of the page's head
      if (PLAIN) {
        amax = __uint_as_float(block_max(__float_as_uint(top)));
      } else {
        amax = top == top ? fmax(amax, (double)top) : (double)top;
        amax = __longlong_as_double((long long)block_max((unsigned long long)__double_as_longlong(amax)));
      }
      const bool special = !(amax < 1e300);   // (the bits of NaN order above infinity's)
      if (special) {   // an infinity or NaN among them: once more, without
        amax = 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (live[u]) {
            amax = fmax(amax, finite_max8(turns, !PLAIN, row_of(h, u), tok[u], da[u]));
            amax = fmax(amax, finite_max8(turns, !PLAIN, row_of(h, u), tok[u], da[u] + dx[u]));
          }
        amax = __longlong_as_double((long long)block_max((unsigned long long)__double_as_longlong(amax)));
      }
      // amax / 448, correctly rounded (one step from the product with the inverse), at least 2^-126
      const float af = (float)amax, q0 = af * (1.f / kFp8Max);
      float sc = fmaxf(PLAIN ? fmaf(fmaf(-q0, kFp8Max, af), 1.f / kFp8Max, q0) : (float)(amax * (1.0 / (double)kFp8Max)),
                       1.175494351e-38f);
      if (older > 0) sc = max_nan(sc, was);   // a page whose older values are none has none
      const float rs = rcp_approx(sc);
      // where fp8_place does not hold; and there a rotated value's fp32 form is not
      // good enough: beyond fp32's range, or among its subnormals
      const bool exact = special || !(sc >= 1e-27f) || !(af <= 3.402823466e38f);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (live[u]) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int d = da[u] + v * dx[u];
            uint8_t* to = dst + (older + tok[u]) * D + d;
            const bool turned = !PLAIN && (EACH || (mode == kHalves ? pair[u] >= 0 : d >= off && d < off + rot));
            unsigned int near = 0u;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = val[u][8 * v + i] * rs;
            if (!turned && !exact) {   // the values as they came: bf16's meet borders often
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = fp8_place(y[i], val[u][8 * v + i], sc, fabsf(y[i]) < 0.015625f ? 0.015625f : 0.f);
            } else if (turned && exact) {
              near = amax > 0.0 ? 0xFFu : 0u;
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (fp8_near_border(y[i])) near |= 1u << i;
            }
            *reinterpret_cast<uint2*>(to) = fp8_pack8(y);
#pragma unroll 1
            for (; near; near &= near - 1) {
              const int e = d + __ffs(near) - 1;
              to[e - d] = exact_code(turns, !PLAIN && e >= off && e < off + rot, row_of(h, u), tok[u], e, sc);
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
  };
  if (mode == kPlain) heads(std::true_type{});
  else heads(std::false_type{});
}

}  // namespace mono
