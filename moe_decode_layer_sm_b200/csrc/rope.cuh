// Rotary positions: (y1, y2) = (c x1 - s x2, s x1 + c x2) for each pair of a
// head, with c = factor cos a, s = factor sin a, a = 2 pi turns_i pos.
#pragma once
#include "mono_attn.h"
#include "ptx.cuh"

namespace mono {

// cos and sin of pair i at a position.  The angle is reduced to within half a
// revolution in binary64, so its error is 2^-53 of the revolutions passed
// (1e-7 of a turn after 1e9 turns); what is left is the fp32 sincospif.
__device__ __forceinline__ void rope_cs(const mono_rope& r, int i, int pos, bool transpose, float* c, float* s) {
  double t = r.turns[i] * (double)pos;
  t -= rint(t);
  float sn, cs;
  sincospif(2.0f * (float)t, &sn, &cs);
  const float f = (float)r.factor;
  *c = f * cs;
  *s = transpose ? -f * sn : f * sn;
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T v[VEC];
};

struct RopeParams {
  mono_rope rope;
  const void* x;
  void* out;
  const int* pos;
  long long x_token, x_head, o_token, o_head;
  int tokens, heads, head_dim, tokens_per_cta, heads_per_cta, transpose, in_place;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 16;   // of a CTA at most

// One CTA: tokens_per_cta tokens, heads_per_cta heads.  A token's angles are
// computed once and shared by its heads, while the first kAhead units of each
// thread are on their way.  A thread owns whole pairs (both vectors of a
// half-layout pair block), so x may be rotated in place.  Bound by memory: one
// read and one write of every value (not in place: of the unrotated ones too).
// Measured, 8191 x 40 heads of 128: fp32 53 us (6.3 TB/s; 61 with 64-bit places
// found for each unit), bf16 halves 32 and interleaved 34 (5 TB/s: there the
// instructions weigh as much as the bytes).
// VEC = 16 bytes of T where layout and alignment allow, else 1.
template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 && VEC > 1 ? 5 : 6) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float2 turn[];   // cos, sin: [token][pair of a unit / 2][unit][2], so that lanes lie side by side
  __shared__ int padding[kRopeTokens];
  const int tok0 = blockIdx.x * p.tokens_per_cta, tokens = min(p.tokens_per_cta, p.tokens - tok0);
  const int half = p.rope.rot_dim >> 1, off = p.rope.offset, rot = p.rope.rot_dim;
  const int h0 = blockIdx.y * p.heads_per_cta, heads = min(p.heads_per_cta, p.heads - h0);
  const T* x = reinterpret_cast<const T*>(p.x) + (long long)tok0 * p.x_token + (long long)h0 * p.x_head;
  T* o = reinterpret_cast<T*>(p.out) + (long long)tok0 * p.o_token + (long long)h0 * p.o_head;
  // units of a head: rotated ones, then (not in place) the dimensions to copy
  constexpr int kPairs = IL ? (VEC > 1 ? VEC / 2 : 1) : VEC;   // pairs a rotated unit holds
  constexpr bool kOne = IL && VEC > 1;                         // a rotated unit is one vector, not two
  constexpr int kAhead = kOne ? 2 : 1;                         // units that a thread has in flight
  const int nrot = half / kPairs;
  const int ncopy = p.in_place ? 0 : (p.head_dim - rot) / VEC;
  const int units = nrot + ncopy;
  // a thread's units are kRopeThreads apart: (token, head, unit) and the rows'
  // places, which fit 32 bits within a CTA, step on by sums with carries
  const int step = kRopeThreads / units, step_u = kRopeThreads - step * units, step_t = step / heads, step_h = step - step_t * heads;
  const int xt = (int)p.x_token, xh = (int)p.x_head, ot = (int)p.o_token, oh = (int)p.o_head;
  const int step_x = step_t * xt + step_h * xh, step_o = step_t * ot + step_h * oh;
  const int wrap_x = xt - heads * xh, wrap_o = ot - heads * oh;
  const int row = threadIdx.x / units;
  int t = row / heads, h = row - t * heads, u = threadIdx.x - row * units;
  int xo = t * xt + h * xh, oo = t * ot + h * oh;
  using V = Vec<T, VEC>;
  bool first = true;
  // every thread meets the barrier below, also one without a unit
  while (first || t < tokens) {
    V a[kAhead], b[kAhead];
    int at_t[kAhead], at_u[kAhead], to[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      at_t[k] = t, at_u[k] = u;
      // the first dimension of the unit
      const int c = (u - nrot) * VEC;
      const int d = u < nrot ? off + u * (kOne ? VEC : IL ? 2 : kPairs) : c >= off ? c + rot : c;
      to[k] = oo + d;
      if (t < tokens) {
        const T* from = x + (xo + d);
        a[k] = *reinterpret_cast<const V*>(from);
        if (!kOne && u < nrot) b[k] = *reinterpret_cast<const V*>(from + (IL ? 1 : half));
      }
      u += step_u, h += step_h, t += step_t, xo += step_x, oo += step_o;
      if (u >= units) u -= units, ++h, xo += xh, oo += oh;
      if (h >= heads) h -= heads, ++t, xo += wrap_x, oo += wrap_o;
    }
    if (first) {
      first = false;
      for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
        const int tt = i / half, pair = i - tt * half, pos = __ldg(p.pos + tok0 + tt);
        float2* to = turn + tt * half +
                     (kPairs == 1 ? pair : ((pair % kPairs / 2) * nrot + pair / kPairs) * 2 + (pair & 1));
        rope_cs(p.rope, pair, pos, p.transpose, &to->x, &to->y);
        if (pair == 0) padding[tt] = pos < 0;
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (at_t[k] < tokens && !padding[at_t[k]]) {
        const int v = at_u[k];
        if (v >= nrot) {
          *reinterpret_cast<V*>(o + to[k]) = a[k];
          continue;
        }
        const float2* cs = turn + at_t[k] * half + (kPairs == 1 ? v : v * 2);
        float4 two = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if (kPairs == 1) two.x = cs->x, two.y = cs->y;
          else if (i % 2 == 0) two = *reinterpret_cast<const float4*>(cs + i * nrot);
          const float c = i % 2 ? two.z : two.x, s = i % 2 ? two.w : two.y;
          T& t1 = a[k].v[kOne ? 2 * i : i];
          T& t2 = kOne ? a[k].v[(2 * i + 1) % VEC] : b[k].v[i % VEC];
          const float x1 = to_f(t1), x2 = to_f(t2);
          t1 = from_f<T>(c * x1 - s * x2);
          t2 = from_f<T>(s * x1 + c * x2);
        }
        *reinterpret_cast<V*>(o + to[k]) = a[k];
        if (!kOne) *reinterpret_cast<V*>(o + to[k] + (IL ? 1 : half)) = b[k];
      }
  }
}

}  // namespace mono
