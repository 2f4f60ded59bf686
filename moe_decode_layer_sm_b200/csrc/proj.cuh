// 4-bit projections: y[r][n] = sum_k x[r][k] (q[n][k] - z[n][k/G]) s[n][k/G] for 1-8 rows.
#pragma once
#include <cooperative_groups.h>

#include "kv_attend.cuh"

namespace mono {

enum { kScaleBf16 = 0, kScaleF32 = 1, kScaleE8m0 = 2 };

struct ProjParams {
  const uint8_t* codes;    // packed, see pack_proj_codes_kernel
  const uint8_t* scales;   // packed
  const uint8_t* zeros;    // packed, or NULL
  const void* x;
  void* y;
  long long x_row, y_row;
  int rows, n_out, kblocks, blocks_per_group, groups, nblocks, x_vec;
};

constexpr int kProjWarps = 8, kProjThreads = 32 * kProjWarps;
constexpr int kProjN = 64;      // outputs a block
constexpr int kProjDepth = 4;   // 32-input blocks that a warp has in flight

// Packed codes: [nblock][kblock][tile pair 2][lane 32][16 bytes], a lane's 16
// bytes the words (tile 2h, step 0), (2h, 1), (2h + 1, 0), (2h + 1, 1).  For
// MMA tile i (outputs 16 i .. 16 i + 15 of the block) and step s, lane (g, t)
// takes outputs g and g + 8 and inputs k = 8 t + 4 s + {0, 1, 2, 3}: any
// assignment of inputs to the MMA's k indices will do as long as x follows it,
// and this one gives a lane 8 consecutive inputs of x (one 16-byte load).
//   int4:  nibble j + 4 u of the word = (output g + 8 (j & 1), input k + 2 (j >> 1) + u),
//          so that two masks and one shift leave the four fp16 pairs of the fragment
//   e2m1:  byte j = fragment register j, low nibble first (the pair converter's order)
__global__ void pack_proj_codes_kernel(const uint8_t* __restrict__ src, uint32_t* __restrict__ dst, int n_out, int n_in,
                                       long long words, int mx) {
  const int kblocks = n_in / 32;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < words;
       i += (long long)gridDim.x * blockDim.x) {
    const int word = i & 3, lane = (i >> 2) & 31, pair = (i >> 7) & 1;
    const long long blk = i >> 8;
    const int kb = (int)(blk % kblocks);
    const long long nb = blk / kblocks;
    const int g = lane >> 2, t = lane & 3, tile = 2 * pair + (word >> 1), s = word & 1;
    uint32_t w = 0;
    for (int j = 0; j < 4; ++j) {
      const long long n = nb * kProjN + tile * 16 + g + 8 * (j & 1);
      if (n >= n_out) continue;   // outputs behind the last: code 0 and scale 0
      const int k = kb * 32 + 8 * t + 4 * s + 2 * (j >> 1);
      const uint32_t two = src[n * (n_in / 2) + k / 2];
      if (mx) w |= two << (8 * j);
      else w |= (two & 15u) << (4 * j) | (two >> 4) << (4 * j + 16);
    }
    dst[i] = w;
  }
}

// Packed scales and zeros: [nblock][group][g 8][tile 4][output g, g + 8]: a
// lane's eight values of a group lie together.
template <typename T>
__global__ void pack_proj_groups_kernel(const T* __restrict__ src, T* __restrict__ dst, int n_out, int groups,
                                        long long total, int mask) {
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int e = i & 1, tile = (i >> 1) & 3, g = (i >> 3) & 7;
    const long long blk = i >> 6;
    const int gr = (int)(blk % groups);
    const long long n = blk / groups * kProjN + tile * 16 + g + 8 * e;
    T v = T(0);
    if (n < n_out) v = src[n * groups + gr];
    if (mask) v = T((int)v & mask);
    dst[i] = v;
  }
}

template <int SC>
struct ScaleRegs {
  uint32_t w[SC == kScaleBf16 ? 4 : SC == kScaleF32 ? 8 : 2];
  static constexpr int kBytes = SC == kScaleBf16 ? 2 : SC == kScaleF32 ? 4 : 1;
  __device__ __forceinline__ void load(const uint8_t* p) {
    if (SC == kScaleE8m0) {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = a.x, w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < (SC == kScaleBf16 ? 1 : 2); ++i) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = a.x, w[4 * i + 1] = a.y, w[(4 * i + 2) % (sizeof(w) / 4)] = a.z, w[(4 * i + 3) % (sizeof(w) / 4)] = a.w;
      }
    }
  }
  // of output g + 8 e of tile i
  __device__ __forceinline__ float get(int i, int e) const {
    if (SC == kScaleF32) return __uint_as_float(w[2 * i + e]);
    if (SC == kScaleBf16) return e ? bf16hi(w[i]) : bf16lo(w[i]);
    const uint32_t b = (w[i >> 1] >> (16 * (i & 1) + 8 * e)) & 0xFFu;
    return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
  }
};

template <bool F32>
size_t proj_smem(int rows, int kblocks) {
  return (size_t)kblocks * rows * 64 * (F32 ? 2 : 1) + 2 * kProjWarps * 32 * 16 * 4 + 512 * 4 + 64;
}

// A cluster of CTAs cuts the inputs; each CTA keeps its part of x in shared
// memory as fp16 (each row scaled by a power of two, fp32 rows as two terms)
// and walks over output blocks; its 8 warps cut the part again.  Weights go
// from global memory to registers, kProjDepth blocks ahead and across output
// blocks, and become exact fp16 operands (int4: the bits under the exponent of
// 1024 or 64; e2m1: the pair converter); a scale multiplies the fp32 sum of
// its 32 products.  The warps' sums are added in a fixed order, then the
// cluster's through distributed shared memory: no scratch, no atomics.
// Bound by the stream of weights: half a byte and 2 x rows operations each.
template <bool F32, int SC, bool ZP>
__global__ void __launch_bounds__(kProjThreads, 2) proj_kernel(const ProjParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  constexpr bool MX = SC == kScaleE8m0;
  constexpr int kSplit = F32 ? 2 : 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const int cs = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kb0 = (int)((long long)p.kblocks * rank / cs), kb1 = (int)((long long)p.kblocks * (rank + 1) / cs);
  const int kbs = kb1 - kb0, kb_max = (p.kblocks + cs - 1) / cs, R = p.rows;
  uint4* xs = reinterpret_cast<uint4*>(smem);   // [split][kb][row][t] 8 halves
  float* red = reinterpret_cast<float*>(smem + (size_t)kb_max * R * 64 * kSplit);   // [2][warp][lane][16]
  float* part = red + 2 * kProjWarps * 32 * 16;                                     // [512]
  float* unscale = part + 512;                                                      // [8]
  const int w0 = kbs * warp / kProjWarps, w1 = kbs * (warp + 1) / kProjWarps, wn = w1 - w0;
  const int nclusters = gridDim.x / cs, cl = blockIdx.x / cs;

  // the warp's blocks: output block cl, cl + nclusters, ..., input blocks
  // [w0, w1) of each, in rounds of kProjDepth (slots behind w1 stay empty)
  uint4 code[kProjDepth][2];
  ScaleRegs<SC> sc[kProjDepth];
  uint2 zp[kProjDepth];
  int ld_nb = cl, ld_kb = w0;   // the round that is loaded next
  auto load = [&](int slot) {
    if (ld_nb < p.nblocks && ld_kb + slot < w1) {
      const int kb = kb0 + ld_kb + slot;
      const uint4* at = reinterpret_cast<const uint4*>(p.codes) + ((long long)ld_nb * p.kblocks + kb) * 64 + lane;
      code[slot][0] = __ldcs(at);
      code[slot][1] = __ldcs(at + 32);
      const long long gr = ((long long)ld_nb * p.groups + kb / p.blocks_per_group) * 64 + g * 8;
      sc[slot].load(p.scales + gr * ScaleRegs<SC>::kBytes);
      if (ZP) zp[slot] = __ldg(reinterpret_cast<const uint2*>(p.zeros + gr));
    }
    if (slot == kProjDepth - 1) {
      ld_kb += kProjDepth;
      if (ld_kb >= w1) ld_kb = w0, ld_nb += nclusters;
    }
  };
#pragma unroll
  for (int i = 0; i < kProjDepth; ++i) load(i);

  // x: warp r takes row r
  for (int r = warp; r < R; r += kProjWarps) {
    const long long row = (long long)r * p.x_row + (long long)kb0 * 32;
    auto get = [&](int k) {
      return F32 ? __ldg(reinterpret_cast<const float*>(p.x) + row + k)
                 : __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16*>(p.x) + row + k));
    };
    auto get8 = [&](int k, float* v) {
      if (p.x_vec) {
        if (F32) {
          const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.x) + row + k);
          const float4 a = __ldg(q), b = __ldg(q + 1);
          v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.x) + row + k));
          v[0] = bf16lo(a.x), v[1] = bf16hi(a.x), v[2] = bf16lo(a.y), v[3] = bf16hi(a.y);
          v[4] = bf16lo(a.z), v[5] = bf16hi(a.z), v[6] = bf16lo(a.w), v[7] = bf16hi(a.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = get(k + i);
      }
    };
    float amax = 0.f;
    for (int q = lane; q < kbs * 4; q += 32) {
      float v[8];
      get8(q * 8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    int e = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
    e = amax > 0.f && amax <= 3.402823466e38f ? min(e, 100) : 0;
    const float up = __uint_as_float((uint32_t)(e + 127) << 23);
    if (lane == 0) unscale[r] = __uint_as_float((uint32_t)(127 - e) << 23);
    for (int q = lane; q < kbs * 4; q += 32) {
      float v[8];
      get8(q * 8, v);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i] * up, b = v[2 * i + 1] * up;
        hi[i] = pack_h2(a, b);
        const __half2 hh = *reinterpret_cast<const __half2*>(&hi[i]);
        lo[i] = F32 ? pack_h2(a - __low2float(hh), b - __high2float(hh)) : 0u;
      }
      const int at = ((q >> 2) * R + r) * 4 + (q & 3);
      xs[at] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (F32) xs[(size_t)kb_max * R * 4 + at] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncthreads();

  int turn = 0;
  for (int nb = cl; nb < p.nblocks; nb += nclusters, turn ^= 1) {
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    for (int kb = w0; kb < w1; kb += kProjDepth) {
#pragma unroll
      for (int u = 0; u < kProjDepth; ++u) {
        if (kb + u >= w1) {
          load(u);
          continue;
        }
        uint4 xv[kSplit];
#pragma unroll
        for (int sp = 0; sp < kSplit; ++sp) {
          xv[sp] = make_uint4(0u, 0u, 0u, 0u);
          if (g < R) xv[sp] = xs[(size_t)sp * kb_max * R * 4 + ((kb + u) * R + g) * 4 + t];
        }
        float sum[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.f;
          __half2 zlo[2], zhi[2];   // -(1024 + zero), -(64 + zero) of outputs g, g + 8
          if (!MX) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (ZP) {
                const uint32_t z = ((i < 2 ? zp[u].x : zp[u].y) >> (16 * (i & 1) + 8 * e)) & 15u;
                const uint32_t b = 0xE400E400u | z | (z << 16);   // -(1024 + z)
                zlo[e] = *reinterpret_cast<const __half2*>(&b);
                zhi[e] = __hadd2(zlo[e], __floats2half2_rn(960.f, 960.f));
              } else {
                zlo[e] = __floats2half2_rn(-1032.f, -1032.f);
                zhi[e] = __floats2half2_rn(-72.f, -72.f);
              }
            }
          }
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint4 cw = code[u][i >> 1];
            const uint32_t w = (i & 1) ? (st ? cw.w : cw.z) : (st ? cw.y : cw.x);
            uint32_t a[4];
            if (MX) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n}\n"
                    : "=r"(a[j])
                    : "r"(w >> (8 * j)));
            } else {
              const uint32_t v = w >> 8;
              const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
#pragma unroll
              for (int j = 0; j < 2; ++j) {   // outputs g (nibbles 0, 2) and g + 8 (1, 3)
                const uint32_t r0 = ((j ? w & 0x00F000F0u : w & 0x000F000Fu)) | 0x64006400u;
                const uint32_t r1 = ((j ? v & 0x00F000F0u : v & 0x000F000Fu)) | 0x64006400u;
                const __half2 h0 = *reinterpret_cast<const __half2*>(&r0), h1 = *reinterpret_cast<const __half2*>(&r1);
                const __half2 o0 = j ? __hfma2(h0, sixteenth, zhi[1]) : __hadd2(h0, zlo[0]);
                const __half2 o1 = j ? __hfma2(h1, sixteenth, zhi[1]) : __hadd2(h1, zlo[0]);
                a[j] = *reinterpret_cast<const uint32_t*>(&o0);
                a[2 + j] = *reinterpret_cast<const uint32_t*>(&o1);
              }
            }
#pragma unroll
            for (int sp = 0; sp < kSplit; ++sp)
              mma_f16(sum[i], a, st ? xv[sp].z : xv[sp].x, st ? xv[sp].w : xv[sp].y);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sc[u].get(i, j >> 1), sum[i][j], acc[i][j]);
        }
        load(u);
      }
    }
    // acc[i][j]: output 16 i + g + 8 (j >> 1), row 2 t + (j & 1)
    float4* mine = reinterpret_cast<float4*>(red + ((size_t)(turn * kProjWarps + warp) * 32 + lane) * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[(i + lane) & 3] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    __syncthreads();
    // thread: (lane ln, tile i) and two of its four values
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int idx = tid + half * kProjThreads;   // 512 sums: ln = idx / 16, slot of 4, j
      const int ln = idx >> 4, slot = (idx >> 2) & 3, j = idx & 3, i = (slot - ln) & 3;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kProjWarps; ++w) v += red[((size_t)(turn * kProjWarps + w) * 32) * 16 + idx];
      const int n = nb * kProjN + 16 * i + (ln >> 2) + 8 * (j >> 1), r = 2 * (ln & 3) + (j & 1);
      v *= r < R ? unscale[r] : 0.f;
      if (cs == 1) {
        if (r < R && n < p.n_out) {
          if (F32) reinterpret_cast<float*>(p.y)[(long long)r * p.y_row + n] = v;
          else reinterpret_cast<__nv_bfloat16*>(p.y)[(long long)r * p.y_row + n] = __float2bfloat16_rn(v);
        }
      } else {
        part[idx] = v;
      }
    }
    if (cs > 1) {
      cluster.sync();
      for (int idx = rank * kProjThreads + tid; idx < 512; idx += cs * kProjThreads) {
        const int ln = idx >> 4, slot = (idx >> 2) & 3, j = idx & 3, i = (slot - ln) & 3;
        const int n = nb * kProjN + 16 * i + (ln >> 2) + 8 * (j >> 1), r = 2 * (ln & 3) + (j & 1);
        float v = 0.f;
        for (int c = 0; c < cs; ++c) v += cluster.map_shared_rank(part, c)[idx];
        if (r < R && n < p.n_out) {
          if (F32) reinterpret_cast<float*>(p.y)[(long long)r * p.y_row + n] = v;
          else reinterpret_cast<__nv_bfloat16*>(p.y)[(long long)r * p.y_row + n] = __float2bfloat16_rn(v);
        }
      }
      cluster.sync();   // part is read
    }
  }
}

}  // namespace mono
