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
  *c = r.factor * cs;
  *s = transpose ? -r.factor * sn : r.factor * sn;
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
  int heads, head_dim, heads_per_cta, transpose, in_place;
};

constexpr int kRopeThreads = 256;

// One CTA: one token, heads_per_cta heads.  The angles are computed once for
// the token and shared by its heads.  A thread owns whole pairs (both 16-byte
// halves of a half-layout pair block), so x may be rotated in place.
// VEC = 16 bytes of T where layout and alignment allow, else 1.
template <typename T, int VEC, bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float cs[128], sn[128];
  const int tok = blockIdx.x;
  const int pos = __ldg(p.pos + tok);
  if (pos < 0) return;
  const int half = p.rope.rot_dim >> 1, off = p.rope.offset, rot = p.rope.rot_dim;
  for (int i = threadIdx.x; i < half; i += kRopeThreads) rope_cs(p.rope, i, pos, p.transpose, &cs[i], &sn[i]);
  __syncthreads();
  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.heads);
  const T* x = reinterpret_cast<const T*>(p.x) + (long long)tok * p.x_token;
  T* o = reinterpret_cast<T*>(p.out) + (long long)tok * p.o_token;
  // units of a head: rotated ones, then (not in place) the dimensions to copy
  constexpr int kPairs = IL ? (VEC > 1 ? VEC / 2 : 1) : VEC;   // pairs a rotated unit holds
  const int nrot = half / kPairs;
  const int ncopy = p.in_place ? 0 : (p.head_dim - rot) / VEC;
  const int units = nrot + ncopy, total = units * (h1 - h0);
  using V = Vec<T, VEC>;
  for (int idx = threadIdx.x; idx < total; idx += kRopeThreads) {
    const int h = h0 + idx / units, u = idx % units;
    const T* xh = x + (long long)h * p.x_head;
    T* oh = o + (long long)h * p.o_head;
    if (u >= nrot) {
      int d = (u - nrot) * VEC;
      if (d >= off) d += rot;
      *reinterpret_cast<V*>(oh + d) = *reinterpret_cast<const V*>(xh + d);
    } else if (IL && VEC > 1) {
      const int d = off + u * VEC;
      V a = *reinterpret_cast<const V*>(xh + d);
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float c = cs[u * kPairs + i], s = sn[u * kPairs + i];
        const float x1 = to_f(a.v[2 * i]), x2 = to_f(a.v[(2 * i + 1) % VEC]);
        a.v[2 * i] = from_f<T>(c * x1 - s * x2);
        a.v[(2 * i + 1) % VEC] = from_f<T>(s * x1 + c * x2);
      }
      *reinterpret_cast<V*>(oh + d) = a;
    } else {
      const int i0 = u * kPairs;
      const int da = IL ? off + 2 * i0 : off + i0, db = IL ? da + 1 : da + half;
      V a = *reinterpret_cast<const V*>(xh + da), b = *reinterpret_cast<const V*>(xh + db);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float c = cs[i0 + i], s = sn[i0 + i];
        const float x1 = to_f(a.v[i]), x2 = to_f(b.v[i]);
        a.v[i] = from_f<T>(c * x1 - s * x2);
        b.v[i] = from_f<T>(s * x1 + c * x2);
      }
      *reinterpret_cast<V*>(oh + da) = a;
      *reinterpret_cast<V*>(oh + db) = b;
    }
  }
}

}  // namespace mono
