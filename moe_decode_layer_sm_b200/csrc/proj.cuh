// 4-bit projections: y[r][n] = sum_k x[r][k] (q[n][k] - z[n][k/G]) s[n][k/G] for 1-8 rows.
#pragma once
#include <cooperative_groups.h>

#include <type_traits>

#include "kv_attend.cuh"

namespace mono {

enum { kScaleBf16 = 0, kScaleF32 = 1, kScaleE8m0 = 2 };

// MXFP4: a scale byte is 0 or 255; a scale is 2^64 or more (or no number)
enum { kEnds = 1, kLarge = 2 };

struct ProjParams {
  const uint8_t* codes;    // packed, see pack_proj_codes_kernel
  const uint8_t* scales;   // packed
  const uint8_t* zeros;    // packed, or NULL
  const void* x;
  void* y;
  long long x_row, y_row;
  const unsigned int* special;   // kEnds, kLarge: what scales there are
  int rows, n_out, kblocks, blocks_per_group, groups, nblocks, x_vec;
  int teams_log2;     // output blocks that a CTA works on at once, each with kProjWarps / teams warps
  int cluster_log2;   // CTAs that share an output block's inputs
};

constexpr int kProjWarpsLog2 = 4, kProjWarps = 1 << kProjWarpsLog2, kProjThreads = 32 * kProjWarps;
constexpr int kProjN = 64;      // outputs a block
constexpr int kProjDepth = 4;   // 32-input blocks that a warp has in flight
constexpr int kProjRedRow = 68; // floats between the rows of a warp's sums: the lanes' banks 8 t + g

// Packed codes: [nblock][kblock][tile pair 2][lane 32][16 bytes], a lane's 16
// bytes the words (tile 2h, step 0), (2h, 1), (2h + 1, 0), (2h + 1, 1).  For
// MMA tile i (outputs 16 i .. 16 i + 15 of the block) and step s, lane (g, t)
// takes outputs g and g + 8 and inputs k = 8 t + 4 s + {0, 1, 2, 3}: any
// assignment of inputs to the MMA's k indices will do as long as x follows it,
// and this one gives a lane 8 consecutive inputs of x (one 16-byte load).
//   int4:  nibble j + 4 u of the word = (output g + 8 (j & 1), input k + 2 (j >> 1) + u),
//          so that masks and one shift leave the four fp16 pairs of the fragment
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
// lane's eight values of a group lie together.  special: kEnds and kLarge among
// the scales, by `magnitude` (all bits but a sign) and the bits of 2^64, `large`.
template <typename T>
__global__ void pack_proj_groups_kernel(const T* __restrict__ src, T* __restrict__ dst, int n_out, int groups,
                                        long long total, int mask, unsigned int* special, unsigned int magnitude,
                                        unsigned int large) {
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int e = i & 1, tile = (i >> 1) & 3, g = (i >> 3) & 7;
    const long long blk = i >> 6;
    const int gr = (int)(blk % groups);
    const long long n = blk / groups * kProjN + tile * 16 + g + 8 * e;
    T v = T(0);
    if (n < n_out) v = src[n * groups + gr];
    if (mask) v = T((int)v & mask);
    if (special && n < n_out) {
      const unsigned int found = (sizeof(T) == 1 && (v == T(0) || v == T(255)) ? kEnds : 0u) |
                                 (((unsigned int)v & magnitude) >= large ? kLarge : 0u);
      if (found) atomicOr(special, found);
    }
    dst[i] = v;
  }
}

// a lane's eight scales of a group: outputs g and g + 8 of each tile
template <int SC>
struct ScaleRegs {
  static constexpr int kBytes = SC == kScaleBf16 ? 2 : SC == kScaleF32 ? 4 : 1;
  uint32_t w[2 * kBytes];
  __device__ __forceinline__ void load(const unsigned char* p) {
    if (SC == kScaleE8m0) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x, w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 2; ++i) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[i];
        w[(4 * i) % (2 * kBytes)] = a.x, w[(4 * i + 1) % (2 * kBytes)] = a.y;
        w[(4 * i + 2) % (2 * kBytes)] = a.z, w[(4 * i + 3) % (2 * kBytes)] = a.w;
      }
    }
  }
  // of output g + 8 e of tile i; e8m0 by the exponent field alone, which is not what 0 and 255 stand for
  __device__ __forceinline__ float get(int i, int e) const {
    if (SC == kScaleF32) return __uint_as_float(w[(2 * i + e) % (2 * kBytes)]);
    if (SC == kScaleBf16) return e ? bf16hi(w[i % (2 * kBytes)]) : bf16lo(w[i % (2 * kBytes)]);
    const int at = 16 * (i & 1) + 8 * e;
    return __uint_as_float((at < 24 ? w[i >> 1] << (23 - at) : w[i >> 1] >> 1) & 0x7F800000u);
  }
};

__device__ __forceinline__ float e8m0_ends(float s) {   // 2^-127 and NaN
  const uint32_t b = __float_as_uint(s);
  return b == 0u ? __uint_as_float(0x00400000u) : b == 0x7F800000u ? __uint_as_float(0x7FC00000u) : s;
}

__device__ __forceinline__ float finite_max(float m, float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? fmaxf(m, a) : m;
}

// (w & mask) | 0x64006400, in one instruction (as two: 7168 x 5120 int4, 1 row, 9.4 us; 7.9 so)
__device__ __forceinline__ uint32_t under_1024(uint32_t w, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
  return r;
}

template <int SC, bool ZP>
__host__ __device__ constexpr int proj_slot() {   // bytes of a block in a warp's ring: codes, scales, zeros
  return 1024 + 64 * ScaleRegs<SC>::kBytes + (ZP ? 64 : 0);
}

// shared memory of a CTA with kb blocks of inputs
template <bool F32, int SC, bool ZP>
size_t proj_smem(int rows, int kb) {
  return (size_t)kProjWarps * kProjDepth * proj_slot<SC, ZP>() + (size_t)kb * rows * 64 * (F32 ? 2 : 1) +
         (size_t)kProjWarps * (rows * kProjRedRow + 8) * 4 + 2 * 512 * 4;
}

// A cluster of CTAs cuts the inputs and the warps of a team cut a CTA's part
// again; a CTA (one an SM) walks over output blocks, one for each team.  Each
// warp streams its weights through a ring of its own in shared memory by
// asynchronous copies, kProjDepth blocks ahead and across output blocks: in
// registers the same depth stalled, since a warp's few scoreboards tie the
// loads of different blocks together (131072 x 5120 MXFP4, 8 rows: 142 us, and
// 97 through the ring).
// x is converted once a CTA, each row of a warp's part scaled by a power of
// two to fp16's range (fp32 as two terms).  Codes become exact fp16 operands:
//   e2m1   by the pair converter
//   int4   q - z: masked under the exponent of 1024 a code is the half 1024 + q,
//          one nibble further up 1024 + 16 q, from which one exact operation
//          takes 1024 + z, or (with a 16th) 64 + z
// A group's scale multiplies the fp32 sum of its products.  (int4 codes as they
// lie, fp16 subnormals, save that operation, but then the zero point has to come
// off the sums, sum q x - z sum x, which loses weights near it: codes that equal
// their zero point gave 1e-6 of sum z |x| s for 0.)  The warps' sums are added
// in a fixed order, then the cluster's, pushed to the CTA that writes the
// output: no scratch, no atomics.
//
// Measured: 131072 x 5120 MXFP4, 8 rows, 74.5 us (4.8 TB/s; 156 instructions for
// 2048 codes; no pipe is full: issue 65 %, integer 55 %, tensor 27 %); 7168 x
// 5120 int4, 1 row 8.1 us, 8 rows 10.5 (the launch, x, the weights on the 112 SMs
// that have an output block, the sums: issue 62 % while a CTA runs); fp32 8 rows 14.3.
template <bool F32, int SC, bool ZP>
__global__ void __launch_bounds__(kProjThreads, 1) proj_kernel(const __grid_constant__ ProjParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  constexpr bool MX = SC == kScaleE8m0;
  constexpr int kSplit = F32 ? 2 : 1, kSlot = proj_slot<SC, ZP>(), SB = ScaleRegs<SC>::kBytes;
  extern __shared__ __align__(16) unsigned char smem[];
  const int cs = 1 << p.cluster_log2, rank = (int)cluster.block_rank(), teams = 1 << p.teams_log2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int tw_log2 = kProjWarpsLog2 - p.teams_log2, tw = 1 << tw_log2;   // warps of a team
  const int team = warp >> tw_log2, kw = warp & (tw - 1);
  const int kb0 = p.kblocks * rank >> p.cluster_log2, kb1 = p.kblocks * (rank + 1) >> p.cluster_log2;
  const int kbs = kb1 - kb0, kb_max = (p.kblocks + cs - 1) >> p.cluster_log2, R = p.rows;
  unsigned char* ring = smem + (size_t)warp * kProjDepth * kSlot;
  uint4* xs = reinterpret_cast<uint4*>(smem + (size_t)kProjWarps * kProjDepth * kSlot);   // [split][kb][row][t] 8 halves
  float* unscale = reinterpret_cast<float*>(xs + (size_t)kb_max * R * 4 * kSplit);        // [kw][8 rows]
  float* part = unscale + kProjWarps * 8;                 // [turn][rank][512 / cs]
  float* red = part + 2 * 512 + team * tw * R * kProjRedRow;   // [kw][row][output 64]
  const int w0 = kbs * kw >> tw_log2, w1 = kbs * (kw + 1) >> tw_log2, wn = w1 - w0;
  const int nclusters = gridDim.x >> p.cluster_log2, cl = blockIdx.x >> p.cluster_log2;
  const int nb0 = (cl << p.teams_log2) + team, nb_step = nclusters << p.teams_log2;
  if (cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // waited for before the first push
  const unsigned int special = __ldg(p.special);
  const bool large = (special & kLarge) != 0u;

  // the warp's blocks: output block nb0, nb0 + nb_step, ..., input blocks
  // [w0, w1) of each.  Zeros come with the first block of a group, or of the
  // part, scales with the last.
  const int bpg = MX ? 1 : p.blocks_per_group;
  const int gr0 = (kb0 + w0) / bpg, in0 = (kb0 + w0) - gr0 * bpg;   // the first block's group, and its place there
  int ld_nb = wn > 0 ? nb0 : p.nblocks, ld_kb = w0, ld_in = in0, ld_slot = 0;
  const uint4* ld_code = reinterpret_cast<const uint4*>(p.codes) + ((long long)nb0 * p.kblocks + kb0 + w0) * 64 + lane;
  // a lane's part of a group's scales: 2 SB bytes; of e8m0 scales and of zeros, 4 bytes by the first two t
  const int sc_lane = SB == 1 ? g * 8 + (t & 1) * 4 : lane * 2 * SB, zp_lane = g * 8 + (t & 1) * 4;
  const long long group_at = ((long long)nb0 * p.groups + gr0) * 64;
  const uint8_t* ld_sc = p.scales + group_at * SB + sc_lane;
  const uint8_t* ld_zp = p.zeros + group_at + zp_lane;
  const long long group_step = ((long long)nb_step * p.groups - ((kb0 + w1 - 1) / bpg - gr0)) * 64;   // from the part's last group
  const uint32_t ring_at = smem_u32(ring);
  auto issue = [&] {
    if (ld_nb < p.nblocks) {
      const uint32_t at = ring_at + ld_slot * kSlot;
      cp_async<16>(at + lane * 16, ld_code);
      cp_async<16>(at + 512 + lane * 16, ld_code + 32);
      const bool part_end = ld_kb == w1 - 1;
      if (ZP && (ld_in == 0 || ld_kb == w0) && t < 2) cp_async<4>(at + 1024 + 64 * SB + zp_lane, ld_zp);
      if (MX || ld_in == bpg - 1 || part_end) {
        if (SB > 1 || t < 2) cp_async<SB == 4 ? 8 : 4>(at + 1024 + sc_lane, ld_sc);
        if (!part_end) {
          ld_sc += 64 * SB;
          if (ZP) ld_zp += 64;
          ld_in = -1;
        }
      }
      ld_code += 64, ++ld_in, ++ld_kb;
      if (part_end) {
        ld_kb = w0, ld_nb += nb_step, ld_in = in0;
        ld_code += ((long long)nb_step * p.kblocks - wn) * 64;
        ld_sc += group_step * SB;
        if (ZP) ld_zp += group_step;
      }
    }
    if (++ld_slot == kProjDepth) ld_slot = 0;
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kProjDepth - 1; ++i) issue();

  // x of the warp's part; a team takes every p.teams-th row
  {
    const long long row0 = (long long)(kb0 + w0) * 32;
    auto get8 = [&](auto vec, int r, int q, float* v) {
      const long long at = (long long)r * p.x_row + row0 + q * 8;
      if (decltype(vec)::value) {
        if (F32) {
          const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.x) + at);
          const float4 a = __ldg(s), b = __ldg(s + 1);
          v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
          const uint4 a = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.x) + at));
          v[0] = bf16lo(a.x), v[1] = bf16hi(a.x), v[2] = bf16lo(a.y), v[3] = bf16hi(a.y);
          v[4] = bf16lo(a.z), v[5] = bf16hi(a.z), v[6] = bf16lo(a.w), v[7] = bf16hi(a.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = F32 ? __ldg(reinterpret_cast<const float*>(p.x) + at + i)
                     : __bfloat162float(__ldg(reinterpret_cast<const __nv_bfloat16*>(p.x) + at + i));
      }
    };
    // chunk q (8 inputs) of a row, scaled, to its place
    auto put = [&](int r, int q, bool there, const float* v, float up) {
      if (!there) return;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * up, b = v[2 * j + 1] * up;
        hi[j] = pack_h2(a, b);
        const __half2 hh = *reinterpret_cast<const __half2*>(&hi[j]);
        // (an infinity's second term, inf - inf, may be any number)
        lo[j] = F32 ? pack_h2(fmaxf(a - __low2float(hh), -64.f), fmaxf(b - __high2float(hh), -64.f)) : 0u;
      }
      const int at = ((w0 + (q >> 2)) * R + r) * 4 + (q & 3);
      xs[at] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (F32) xs[(size_t)kb_max * R * 4 + at] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
    // The power of two that takes a row's largest magnitude to [2^14, 2^15), 2^126
    // at most; its inverse is kept.  Beside infinities the largest finite one
    // counts, which `again` finds: the others must not become infinite too.
    auto scale_row = [&](int r, float most, auto again) {
      auto of_warp = [](float v) { return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v))); };
      most = of_warp(most);
      if (!(most <= 3.402823466e38f)) most = of_warp(again());
      int e = 14 - ((int)(__float_as_uint(most) >> 23) - 127);
      e = most > 0.f ? min(e, 126) : 0;   // 2^e and 2^-e are both normal
      if (lane == 0 && r < R) unscale[kw * 8 + r] = __uint_as_float((uint32_t)(127 - e) << 23);
      return __uint_as_float((uint32_t)(e + 127) << 23);
    };
    // A part that fits registers: its loads of four rows in flight at once (7168 x
    // 5120, 8 rows: 20 us where the loop below reads each row twice, 12 so).
    // Eight rows at a time cost MXFP4's loop registers and 4 %, and a single int4
    // row 0.4 us of code that runs once.
    auto convert_held = [&](auto rows) {
      constexpr int kRows = decltype(rows)::value;
      for (int r0 = team; r0 < R; r0 += kRows * teams) {
        uint4 raw[kRows][2][F32 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = r0 + i * teams, q = lane + 32 * k;
#pragma unroll
            for (int c = 0; c < (F32 ? 2 : 1); ++c) {
              raw[i][k][c] = make_uint4(0u, 0u, 0u, 0u);
              if (r < R && q < wn * 4)
                raw[i][k][c] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(p.x) +
                                                                    ((long long)r * p.x_row + row0 + q * 8) * (F32 ? 4 : 2)) + c);
            }
          }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int r = r0 + i * teams;
          if (r >= R) break;
          float v[2][8];
          float most = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 a = raw[i][k][0];
            if (F32) {
              const uint4 b = raw[i][k][F32 ? 1 : 0];
              const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
              for (int j = 0; j < 8; ++j) v[k][j] = __uint_as_float(w[j]);
            } else {
              const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) v[k][2 * j] = bf16lo(w[j]), v[k][2 * j + 1] = bf16hi(w[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[k][j]));
          }
          const float up = scale_row(r, most, [&] {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int j = 0; j < 8; ++j) m = finite_max(m, v[k][j]);
            return m;
          });
#pragma unroll
          for (int k = 0; k < 2; ++k) put(r, lane + 32 * k, lane + 32 * k < wn * 4, v[k], up);
        }
      }
    };
    // kRows: rows whose loads are in flight together
    auto convert = [&](auto vec, auto rows) {
      constexpr int kRows = decltype(rows)::value;
      for (int r0 = team; r0 < R; r0 += kRows * teams) {
        float amax[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) amax[i] = 0.f;
        for (int q = lane; q < wn * 4; q += 32)
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * teams;
            if (r < R) {
              float v[8];
              get8(vec, r, q, v);
#pragma unroll
              for (int j = 0; j < 8; ++j) amax[i] = fmaxf(amax[i], fabsf(v[j]));
            }
          }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          amax[i] = scale_row(r0 + i * teams, amax[i], [&] {
            float m = 0.f;
            for (int q = lane; q < wn * 4; q += 32) {
              float v[8];
              get8(vec, r0 + i * teams, q, v);
#pragma unroll
              for (int j = 0; j < 8; ++j) m = finite_max(m, v[j]);
            }
            return m;
          });
        for (int q0 = 0; q0 < wn * 4; q0 += 32) {
          const int q = q0 + lane;
#pragma unroll
          for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * teams;
            if (r < R) {
              float v[8];
              if (q < wn * 4) get8(vec, r, q, v);
              put(r, q, q < wn * 4, v, amax[i]);
            }
          }
        }
      }
    };
    if (p.x_vec && wn <= 16) convert_held(std::integral_constant<int, 4>{});
    else if (p.x_vec) convert(std::true_type{}, std::integral_constant<int, 4>{});
    else convert(std::false_type{}, std::integral_constant<int, 1>{});
    if (teams > 1) __syncthreads();
    else __syncwarp();
  }

  int turn = 0, slot = 0;
  bool waited = cs == 1;
  for (int nb = nb0; nb < p.nblocks; nb += nb_step, turn ^= 1) {
    float acc[4][4], sum[4][4];
    uint32_t zlo[4], zhi[4];   // int4: -(1024 + z) of outputs g, -(64 + z) of outputs g + 8, twice each
#pragma unroll
    for (int i = 0; i < 4; ++i) zlo[i] = 0xE408E408u, zhi[i] = 0xD480D480u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = sum[i][j] = 0.f;
    int in = in0;
#pragma unroll 1
    for (int kb = w0; kb < w1; ++kb) {
      cp_async_wait<kProjDepth - 2>();
      __syncwarp();   // the other lanes' copies of this block, and their reads of the slot that is filled next
      issue();
      const unsigned char* at = ring + slot * kSlot;
      if (++slot == kProjDepth) slot = 0;
      uint4 code[2];
      code[0] = *reinterpret_cast<const uint4*>(at + lane * 16);
      code[1] = *reinterpret_cast<const uint4*>(at + 512 + lane * 16);
      uint4 xv[kSplit];
#pragma unroll
      for (int sp = 0; sp < kSplit; ++sp) {
        xv[sp] = make_uint4(0u, 0u, 0u, 0u);
        if (g < R) xv[sp] = xs[(size_t)sp * kb_max * R * 4 + (kb * R + g) * 4 + t];
      }
      if (ZP && (in == 0 || kb == w0)) {
        const uint2 zp = *reinterpret_cast<const uint2*>(at + 1024 + 64 * SB + g * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t z = i < 2 ? zp.x : zp.y;
          zlo[i] = __byte_perm(z, 0xE4u, i & 1 ? 0x4242 : 0x4040);
          zhi[i] = __byte_perm(z << 4, 0xD4u, i & 1 ? 0x4343 : 0x4141);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint4 cw = code[i >> 1];
          const uint32_t w = (i & 1) ? (st ? cw.w : cw.z) : (st ? cw.y : cw.x);
          uint32_t a[4];
          if (MX) {
            asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n"
                " cvt.rn.f16x2.e2m1x2 %1, b1;\n cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
                : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                : "r"(w));
          } else {   // q - z of outputs g and g + 8 in turn
            const uint32_t v = w >> 8;
            a[0] = under_1024(w, 0x000F000Fu);
            a[1] = under_1024(w, 0x00F000F0u);
            a[2] = under_1024(v, 0x000F000Fu);
            a[3] = under_1024(v, 0x00F000F0u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 h = *reinterpret_cast<const __half2*>(&a[j]);
              const __half2 z = *reinterpret_cast<const __half2*>(j & 1 ? &zhi[i] : &zlo[i]);
              const __half2 q = j & 1 ? __hfma2(h, __floats2half2_rn(0.0625f, 0.0625f), z) : __hadd2(h, z);
              a[j] = *reinterpret_cast<const uint32_t*>(&q);
            }
          }
#pragma unroll
          for (int sp = 0; sp < kSplit; ++sp) {
            const uint32_t b0 = st ? xv[sp].z : xv[sp].x, b1 = st ? xv[sp].w : xv[sp].y;
            if (MX && st == 0 && sp == 0) mma_f16_first(sum[i], a, b0, b1);
            else mma_f16(sum[i], a, b0, b1);
          }
        }
      }
      const bool last = MX || ++in == bpg;
      if (MX || last || kb == w1 - 1) {
        ScaleRegs<SC> sc;
        sc.load(at + 1024 + g * 8 * SB);
        // The sums carry the rows' powers of two until the end.  With scales of
        // 2^64 or more in the plan they could pass fp32's end so; there a row's is
        // taken off first, after the scale where that is below 1.
        if (large) {
          const float un[2] = {unscale[kw * 8 + 2 * t], unscale[kw * 8 + 2 * t + 1]};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float s = MX ? e8m0_ends(sc.get(i, j >> 1)) : sc.get(i, j >> 1), u = un[j & 1];
              acc[i][j] = fabsf(s) >= 1.f ? fmaf(s, sum[i][j] * u, acc[i][j]) : fmaf(s * sum[i][j], u, acc[i][j]);
              sum[i][j] = 0.f;
            }
          in = 0;
        } else if (MX) {
          float s[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = sc.get(i >> 1, i & 1);
          if (special & kEnds) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = e8m0_ends(s[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s[2 * i + (j >> 1)], sum[i][j], acc[i][j]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[i][j] = fmaf(sc.get(i, j >> 1), sum[i][j], acc[i][j]);
              sum[i][j] = 0.f;
            }
          in = 0;
        }
      }
    }
    // acc[i][j]: output 16 i + g + 8 (j >> 1), row 2 t + (j & 1)
    auto team_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(tw * 32) : "memory"); };
    if (nb != nb0) team_sync();   // red of the block before is read
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (2 * t + r < R) {
        const float un = large ? 1.f : unscale[kw * 8 + 2 * t + r];
        float* to = red + (kw * R + 2 * t + r) * kProjRedRow + g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) to[16 * i + 8 * e] = acc[i][2 * e + r] * un;
      }
    team_sync();
    auto write = [&](int r, int n, float v) {
      if (n < p.n_out) {
        if (F32) reinterpret_cast<float*>(p.y)[(long long)r * p.y_row + n] = v;
        else reinterpret_cast<__nv_bfloat16*>(p.y)[(long long)r * p.y_row + n] = __float2bfloat16_rn(v);
      }
    };
    if (!waited) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      waited = true;
    }
    const int slice_log2 = 6 - p.cluster_log2, slice = 1 << slice_log2;   // of a block's outputs, for each CTA to finish
    for (int idx = tid - team * tw * 32; idx < R * kProjN; idx += tw * 32) {
      const int r = idx >> 6, n = idx & 63;
      float v = 0.f;
#pragma unroll 4
      for (int w = 0; w < tw; ++w) v += red[(w * R + r) * kProjRedRow + n];
      if (cs == 1) write(r, nb * kProjN + n, v);
      else *cluster.map_shared_rank(part + turn * 512 + (rank << (9 - p.cluster_log2)) + r * slice + (n & (slice - 1)), n >> slice_log2) = v;
    }
    if (cs > 1) {
      // one barrier a block: the other half of part is written before the next
      cluster.sync();
      for (int idx = tid; idx < R * slice; idx += kProjThreads) {
        float v = 0.f;
        for (int c = 0; c < cs; ++c) v += part[turn * 512 + (c << (9 - p.cluster_log2)) + idx];
        write(idx >> slice_log2, nb * kProjN + rank * slice + (idx & (slice - 1)), v);
      }
    }
  }
  cp_async_wait<0>();
  if (!waited) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace mono
