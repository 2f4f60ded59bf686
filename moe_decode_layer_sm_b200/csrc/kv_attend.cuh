// Attention of 1-8 new tokens a sequence over the paged 8-bit cache.
#pragma once
#include "kv_append.cuh"

namespace mono {

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit values across a warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// two e4m3 codes (a half of a word) -> two fp16 values, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w, int half) {
  uint32_t h;
  const uint16_t v = (uint16_t)(half ? w >> 16 : w & 0xFFFFu);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct AttendParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const void* q;
  void* out;
  long long q_seq, q_tok, q_head, o_seq, o_tok, o_head;
  float* lse;
  const int* lens;
  const int* n_new;
  const int* table;
  BadIndex* bad;
  float* part_o;          // [2 grid][rows of a CTA][D]
  float2* part_ml;        // [2 grid][rows of a CTA]
  unsigned int* arrived;  // [items], zero between calls
  int seqs, width, q_heads, kv_heads, group, page_shift, num_pages, max_pages, window;
  int wr, row_blocks;     // warps side by side over the rows; row blocks of a key head
  unsigned least;         // tiles a CTA takes at least
  float scale_log2;
};

constexpr int kAttendThreads = 128;
constexpr float kPBias = 15.f;   // probabilities are held as 2^15 p: fp16 keeps 11 bits down to p = 2^-29

template <int D, int NT, bool F32>
struct AttendShape {
  static constexpr int kSubs = D == 64 ? 4 : D == 128 ? 2 : 1;   // groups of 16 tokens a warp's tile holds
  static constexpr int kTile = 16 * kSubs;                       // tokens: 4 KB of keys
  static constexpr int kSplit = F32 ? 2 : 1;                     // fp16 terms that q and p are carried in
  static constexpr int kRows = 8 * NT;                           // rows of a warp
  static constexpr int kSteps = D / 16;
  static constexpr int kKeyWords = D / 8;                        // 32-bit words of keys a lane holds of 16 tokens
  static constexpr int kValWords = D / 32;                       // and of values, for each of its 4 tokens
  static size_t smem(int seqs, int wr) {
    const size_t q = (size_t)wr * NT * kSplit * kSteps * 256, merge = (size_t)4 * kRows * D * 4;
    return (size_t)(seqs + 1 + 3) / 4 * 16 + (q > merge ? q : merge) + 4 * kRows * 8 + 4 * kRows * 12 + 64;
  }
};

// One warp multiplies tiles of kTile tokens with 8 NT query rows: the scores
// S^T = K Q^T with the tokens as the m dimension, the output O^T = V^T P^T
// with the head's dimensions as m, so 8 rows fill an MMA's n and no lane
// works on padding at the usual group sizes.  Keys and values go from global
// memory straight to the lanes' registers (each byte is used by one warp, so
// shared memory would only add a trip), in the order in which a lane's 16
// bytes are its k indices of four MMAs; q is permuted to match.
//
// The work is the line of all (sequence, key head, row block, tile), cut into
// equal runs, one a CTA; the cut follows the lengths on the device, so one
// captured launch serves any lengths.  An item that spans CTAs leaves partial
// (O, m, l) in the scratch, and the CTA that arrives last adds them in the
// order of the line: results do not depend on the order of arrival.
template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kAttendThreads, (D == 128 && NT == 1) || D == 64 ? 3 : 2)
    attend_kernel(const AttendParams p) {
  using S = AttendShape<D, NT, F32>;
  constexpr int kSubs = S::kSubs, T = S::kTile, kRows = S::kRows, kSplit = S::kSplit;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned int* cum = reinterpret_cast<unsigned int*>(smem);
  unsigned char* big = smem + (size_t)(p.seqs + 1 + 3) / 4 * 16;
  const size_t qbytes = (size_t)p.wr * NT * kSplit * S::kSteps * 256, mbytes = (size_t)4 * kRows * D * 4;
  uint2* qf = reinterpret_cast<uint2*>(big);
  float* merge = reinterpret_cast<float*>(big);
  float2* ml = reinterpret_cast<float2*>(big + (qbytes > mbytes ? qbytes : mbytes));   // [4 warps][kRows]
  float* rowf = reinterpret_cast<float*>(ml + 4 * kRows);                             // [wr kRows]
  int* rlo = reinterpret_cast<int*>(rowf + 4 * kRows);
  int* rhi = rlo + 4 * kRows;
  unsigned int* wsum = reinterpret_cast<unsigned int*>(rhi + 4 * kRows);              // [4], then a flag
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int cap = p.max_pages << p.page_shift, P = 1 << p.page_shift;

  // tiles before each sequence
  {
    const int per = (p.seqs + kAttendThreads - 1) / kAttendThreads;
    const int s0 = min(tid * per, p.seqs), s1 = min(s0 + per, p.seqs);
    unsigned int sum = 0;
    for (int s = s0; s < s1; ++s)
      sum += seq_tiles(view_seq(__ldg(p.lens + s), p.n_new ? __ldg(p.n_new + s) : p.width, p.width, cap), p.window, cap, T);
    unsigned int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned int x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    unsigned int at = inc - sum;
    for (int w = 0; w < warp; ++w) at += wsum[w];
    for (int s = s0; s < s1; ++s) {
      const SeqView v = view_seq(__ldg(p.lens + s), p.n_new ? __ldg(p.n_new + s) : p.width, p.width, cap);
      if (v.bad && blockIdx.x == 0) record_bad(p.bad, v.bad, s, v.bad_value);
      cum[s] = at;
      at += seq_tiles(v, p.window, cap, T);
    }
    if (tid == kAttendThreads - 1) cum[p.seqs] = at;
    __syncthreads();
  }
  const unsigned int per_seq = (unsigned)(p.kv_heads * p.row_blocks);
  const unsigned int total = cum[p.seqs] * per_seq;
  const unsigned int share = share_of(total, gridDim.x, p.least);
  const unsigned int cta = blockIdx.x;
  if ((unsigned long long)cta * share >= total) return;
  const unsigned int end = min(total, cta * share + share);
  const int wt = warp / p.wr, wrow = warp - wt * p.wr, WT = 4 / p.wr;
  const int cta_rows = p.wr * kRows;

  for (unsigned int pos = cta * share; pos < end;) {
    // the item at pos
    int lo_s = 0, hi_s = p.seqs - 1;
    while (lo_s < hi_s) {
      const int mid = (lo_s + hi_s) >> 1;
      if (cum[mid + 1] * per_seq > pos) hi_s = mid;
      else lo_s = mid + 1;
    }
    const int s = lo_s;
    const unsigned int n_t = cum[s + 1] - cum[s], seq_base = cum[s] * per_seq;
    const unsigned int rel = pos - seq_base, hb = rel / n_t, tile0 = rel - hb * n_t;
    const unsigned int cnt = min(n_t - tile0, end - pos), base = seq_base + hb * n_t;
    const int h = (int)hb / p.row_blocks, rb = (int)hb - h * p.row_blocks;
    const SeqView sv = view_seq(__ldg(p.lens + s), p.n_new ? __ldg(p.n_new + s) : p.width, p.width, cap);
    const int live = sv.n * p.group - rb * cta_rows;   // live rows of this block (may pass cta_rows)
    const int tok_lo = row_lo(sv, 0, p.window), tok_hi = row_hi(sv, sv.n - 1, cap);
    const int all_lo = row_lo(sv, sv.n - 1, p.window), all_hi = row_hi(sv, 0, cap);
    const long long tok0 = (long long)(tok_lo / T + (int)tile0) * T;

    int pid[kSubs];
    uint32_t kw[kSubs][S::kKeyWords], vw[kSubs][4][S::kValWords];
    float ksc[kSubs], vsc[kSubs];
    auto find_pages = [&](unsigned int i) {
#pragma unroll
      for (int b = 0; b < kSubs; ++b) {
        const long long tok = tok0 + (long long)i * T + b * 16;
        pid[b] = -1;
        if (i < cnt && tok < tok_hi && tok + 16 > tok_lo) {
          pid[b] = __ldg(p.table + (long long)s * p.max_pages + (tok >> p.page_shift));
          if (!page_ok(pid[b], p.num_pages)) {
            if (lane == 0) record_bad(p.bad, kBadPage, s, pid[b]);
            pid[b] = -1;
          }
        }
      }
    };
    auto load_keys = [&](unsigned int i) {
#pragma unroll
      for (int b = 0; b < kSubs; ++b) {
        const int off = (int)((tok0 + (long long)i * T + b * 16) & (P - 1));
        ksc[b] = 0.f;
        if (pid[b] >= 0) {
          const uint8_t* at = p.k + (code_row(pid[b], p.kv_heads, h, P, off) + g) * D + t * 16;
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint4 w = __ldg(reinterpret_cast<const uint4*>(at + r * 8 * D + c * 64));
              uint32_t* d = &kw[b][(r * (D / 64) + c) * 4];
              d[0] = w.x, d[1] = w.y, d[2] = w.z, d[3] = w.w;
            }
          ksc[b] = __ldg(p.ks + (long long)pid[b] * p.kv_heads + h);
        } else {
#pragma unroll
          for (int j = 0; j < S::kKeyWords; ++j) kw[b][j] = 0;
        }
      }
    };
    auto load_vals = [&](unsigned int i) {
#pragma unroll
      for (int b = 0; b < kSubs; ++b) {
        const int off = (int)((tok0 + (long long)i * T + b * 16) & (P - 1));
        vsc[b] = 0.f;
        if (pid[b] >= 0) {
          const uint8_t* at = p.v + (code_row(pid[b], p.kv_heads, h, P, off) + 2 * t) * D + g * (D == 64 ? 8 : 16);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint8_t* row = at + ((r & 1) + (r >> 1) * 8) * D;
            if (D == 64) {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(row));
              vw[b][r][0] = w.x, vw[b][r][1] = w.y;
            } else {
#pragma unroll
              for (int c = 0; c < D / 128; ++c) {
                const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + c * 128));
                uint32_t* d = &vw[b][r][(c * 4) % S::kValWords];
                d[0] = w.x, d[1] = w.y, d[2 % S::kValWords] = w.z, d[3 % S::kValWords] = w.w;
              }
            }
          }
          vsc[b] = __ldg(p.vs + (long long)pid[b] * p.kv_heads + h);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < S::kValWords; ++j) vw[b][r][j] = 0;
        }
      }
    };
    unsigned int cur_ok = 0;   // which 16-token groups of the tile in registers have a page
    auto page_mask = [&] {
      unsigned int m = 0;
#pragma unroll
      for (int b = 0; b < kSubs; ++b) m |= (pid[b] >= 0 ? 1u : 0u) << b;
      return m;
    };
    find_pages(wt);
    load_keys(wt);
    load_vals(wt);
    cur_ok = page_mask();
    find_pages(wt + WT);

    // q: each row scaled by a power of two into fp16's range, in the B fragments' order
    for (int r = warp; r < cta_rows; r += 4) {
      const int m = rb * cta_rows + r, j = m / p.group, hq = h * p.group + (m - j * p.group);
      float qv[(D + 127) / 128][4];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < (D + 127) / 128; ++c) {
        const int d0 = (c * 32 + lane) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qv[c][i] = 0.f;
          if (r < live && d0 < D) {
            const long long at = (long long)s * p.q_seq + (long long)j * p.q_tok + (long long)hq * p.q_head + d0 + i;
            qv[c][i] = F32 ? reinterpret_cast<const float*>(p.q)[at]
                           : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q)[at]);
          }
          amax = fmaxf(amax, fabsf(qv[c][i]));
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      // 2^e takes the row's largest magnitude to [2^14, 2^15)
      int e = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
      e = amax > 0.f && amax <= 3.402823466e38f ? min(e, 100) : 0;
      const float up = __uint_as_float((uint32_t)(e + 127) << 23);
      if (lane == 0) {
        rowf[r] = p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
        rlo[r] = r < live ? row_lo(sv, j, p.window) : 0;
        rhi[r] = r < live ? row_hi(sv, j, cap) : 0;
      }
#pragma unroll
      for (int c = 0; c < (D + 127) / 128; ++c) {
        const int d0 = (c * 32 + lane) * 4;
        if (d0 < D) {
          const int step = (d0 >> 6) * 4 + ((d0 & 15) >> 2), tq = (d0 & 63) >> 4;
          const int slot = (r / kRows * NT + (r % kRows) / 8) * kSplit;
#pragma unroll
          for (int sp = 0; sp < kSplit; ++sp) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float a = qv[c][2 * i] * up, b = qv[c][2 * i + 1] * up;
              w[i] = pack_h2(a, b);
              if (sp == 1) {
                const __half2 hi = *reinterpret_cast<const __half2*>(&w[i]);
                w[i] = pack_h2(a - __low2float(hi), b - __high2float(hi));
              }
            }
            qf[((slot + sp) * S::kSteps + step) * 32 + (r % 8) * 4 + tq] = make_uint2(w[0], w[1]);
          }
        }
      }
    }
    __syncthreads();
    float rf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) rf[n][i] = rowf[wrow * kRows + n * 8 + 2 * t + i];

    float O[D / 16][NT][4], mx[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mx[n][0] = mx[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 16; ++w) O[w][n][0] = O[w][n][1] = O[w][n][2] = O[w][n][3] = 0.f;
    }
    const uint2* qw = qf + (size_t)wrow * NT * kSplit * S::kSteps * 32 + lane;

    for (unsigned int i = wt; i < cnt; i += WT) {
      const long long tile_tok = tok0 + (long long)i * T;
      const bool edge = tile_tok < all_lo || tile_tok + T > all_hi || cur_ok != (1u << kSubs) - 1u;
      // scores
      float c[kSubs][NT][4];
#pragma unroll
      for (int b = 0; b < kSubs; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) c[b][n][0] = c[b][n][1] = c[b][n][2] = c[b][n][3] = 0.f;
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) {
        uint32_t a[kSubs][4];
#pragma unroll
        for (int b = 0; b < kSubs; ++b) {
          const uint32_t w0 = kw[b][st], w1 = kw[b][S::kSteps + st];
          a[b][0] = e4m3x2_to_h2(w0, 0);
          a[b][1] = e4m3x2_to_h2(w1, 0);
          a[b][2] = e4m3x2_to_h2(w0, 1);
          a[b][3] = e4m3x2_to_h2(w1, 1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int sp = 0; sp < kSplit; ++sp) {
            const uint2 q2 = qw[((n * kSplit + sp) * S::kSteps + st) * 32];
#pragma unroll
            for (int b = 0; b < kSubs; ++b) mma_f16(c[b][n], a[b], q2.x, q2.y);
          }
      }
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
        for (int b = 0; b < kSubs; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[b][n][j] *= ksc[b] * rf[n][j & 1];
        if (edge) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = wrow * kRows + n * 8 + 2 * t + (j & 1), lo = rlo[row], hi = rhi[row];
#pragma unroll
            for (int b = 0; b < kSubs; ++b) {
              const long long tok = tile_tok + b * 16 + g + (j >> 1) * 8;
              if (tok < lo || tok >= hi || !((cur_ok >> b) & 1u)) c[b][n][j] = -INFINITY;
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kSubs; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[n][j & 1] = fmaxf(top[n][j & 1], c[b][n][j]);
      }
      const unsigned int next_ok = page_mask();
      if (i + WT < cnt) load_keys(i + WT);
      // running maximum and sum
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = top[n][r];
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
          top[n][r] = x;
          grew |= x > mx[n][r];
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float now = fmaxf(mx[n][r], top[n][r]);
            const float keep = now == -INFINITY ? 1.f : exp2_approx(mx[n][r] - now);
            mx[n][r] = now;
            l[n][r] *= keep;
#pragma unroll
            for (int w = 0; w < D / 16; ++w) O[w][n][r] *= keep, O[w][n][2 + r] *= keep;
          }
      }
      // probabilities, in units of the tile's largest value scale
      float vmax = 0.f;
#pragma unroll
      for (int b = 0; b < kSubs; ++b) vmax = fmaxf(vmax, vsc[b]);
      const float vinv = vmax > 0.f ? __fdividef(1.f, vmax) : 0.f;
      uint32_t pf[kSubs][NT][kSplit][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float off0 = mx[n][0] == -INFINITY ? 0.f : mx[n][0] - kPBias;
        const float off1 = mx[n][1] == -INFINITY ? 0.f : mx[n][1] - kPBias;
#pragma unroll
        for (int b = 0; b < kSubs; ++b) {
          const float r = kSubs > 1 ? vsc[b] * vinv : 1.f;
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[j] = exp2_approx(c[b][n][j] - (j & 1 ? off1 : off0));
            l[n][j & 1] += e[j];
            e[j] *= r;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t hi = pack_h2(e[2 * j], e[2 * j + 1]);
            pf[b][n][0][j] = movmatrix(hi);
            if (F32) {
              const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
              pf[b][n][kSplit - 1][j] = movmatrix(pack_h2(e[2 * j] - __low2float(hh), e[2 * j + 1] - __high2float(hh)));
            }
          }
        }
      }
      // a tile that some row does not see in full: values behind the sequence
      // (or before its window) read as zero; a NaN value reaches only the rows
      // that see its token
      if (edge) {
        bool nan = false;
#pragma unroll
        for (int b = 0; b < kSubs; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const long long tok = tile_tok + b * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
            const bool in = tok >= tok_lo && tok < tok_hi;
#pragma unroll
            for (int w = 0; w < S::kValWords; ++w) {
              if (!in) vw[b][r][w] = 0;
              nan |= (((vw[b][r][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
            }
          }
        if (__any_sync(0xFFFFFFFFu, nan)) {
          uint32_t sees[kSubs][NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < kSubs; ++b)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const long long tok = tile_tok + b * 16 + g + j * 8;
                const int row = wrow * kRows + n * 8 + 2 * t;
                sees[b][n][j] = movmatrix((tok >= rlo[row] && tok < rhi[row] ? 0x3C00u : 0u) |
                                          (tok >= rlo[row + 1] && tok < rhi[row + 1] ? 0x3C000000u : 0u));
              }
#pragma unroll
          for (int w = 0; w < 2 * S::kValWords; ++w) {
            float hit[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) hit[n][0] = hit[n][1] = hit[n][2] = hit[n][3] = 0.f;
#pragma unroll
            for (int b = 0; b < kSubs; ++b) {
              uint32_t x[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) {   // 1.0 (e4m3 0x38) where the code is NaN
                const uint32_t y = ((vw[b][r][w >> 1] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                x[r] = e4m3x2_to_h2((y >> 7) * 0x38u, w & 1);
              }
              const uint32_t a[4] = {__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                                     __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[2], x[3], 0x7632)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(hit[n], a, sees[b][n][0], sees[b][n][1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (hit[n][j] > 0.f) O[w][n][j] = __int_as_float(0x7FC00000);
          }
#pragma unroll
          for (int b = 0; b < kSubs; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int w = 0; w < S::kValWords; ++w) {
                const uint32_t y = ((vw[b][r][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                vw[b][r][w] &= ~((y >> 7) * 0xFFu);
              }
        }
      }
      // output
#pragma unroll
      for (int w = 0; w < 2 * S::kValWords; ++w) {
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
        for (int b = 0; b < kSubs; ++b) {
          uint32_t x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[r] = e4m3x2_to_h2(vw[b][r][w >> 1], w & 1);
          const uint32_t a[4] = {__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[0], x[1], 0x7632),
                                 __byte_perm(x[2], x[3], 0x5410), __byte_perm(x[2], x[3], 0x7632)};
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int sp = 0; sp < kSplit; ++sp) mma_f16(o[n], a, pf[b][n][sp][0], pf[b][n][sp][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) O[w][n][j] = fmaf(o[n][j], vmax, O[w][n][j]);
      }
      if (i + WT < cnt) {
        load_vals(i + WT);
        cur_ok = next_ok;
        find_pages(i + 2 * WT);
      }
    }

    // the CTA's warps together
    __syncthreads();   // q is read
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = l[n][r];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        const int row = n * 8 + 2 * t + r;
        if (g == 0) ml[warp * kRows + row] = make_float2(mx[n][r], x);
#pragma unroll
        for (int w = 0; w < S::kValWords; ++w) {
          const int d = D == 64 ? g * 8 + w * 4 : (w >> 2) * 128 + g * 16 + (w & 3) * 4;
          *reinterpret_cast<float4*>(merge + ((size_t)warp * kRows + row) * D + d) =
              make_float4(O[2 * w][n][r], O[2 * w][n][2 + r], O[2 * w + 1][n][r], O[2 * w + 1][n][2 + r]);
        }
      }
    __syncthreads();
    const unsigned int c_first = base / share, c_last = (base + n_t - 1) / share;
    const bool whole = c_first == c_last;
    auto finish = [&](int r, int d, float4 o, float m, float lsum) {
      const int row = rb * cta_rows + r, j = row / p.group, hq = h * p.group + (row - j * p.group);
      const float inv = lsum > 0.f || lsum != lsum ? __fdiv_rn(1.f, lsum) : 0.f;
      const float f[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
      const long long at = (long long)s * p.o_seq + (long long)j * p.o_tok + (long long)hq * p.o_head + d;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (F32) reinterpret_cast<float*>(p.out)[at + i] = f[i];
        else reinterpret_cast<__nv_bfloat16*>(p.out)[at + i] = __float2bfloat16_rn(f[i]);
      }
      if (p.lse && d == 0)
        p.lse[((long long)s * p.width + j) * p.q_heads + hq] =
            lsum == 0.f ? -INFINITY : (m + log2f(lsum) - kPBias) * 0.6931471805599453f;
    };
    const size_t slot = part_slot(cta, base, share);
    const int rows = min(live, cta_rows);
    for (int idx = tid; idx < rows * (D / 4); idx += kAttendThreads) {
      const int r = idx / (D / 4), d = (idx % (D / 4)) * 4, wq = r / kRows, rr = r % kRows;
      float m = -INFINITY;
      for (int w = 0; w < WT; ++w) m = fmaxf(m, ml[(w * p.wr + wq) * kRows + rr].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float lsum = 0.f;
      for (int w = 0; w < WT; ++w) {
        const int from = (w * p.wr + wq) * kRows + rr;
        const float2 y = ml[from];
        const float f = m == -INFINITY ? (y.y != y.y ? y.y : 0.f) : exp2_approx(y.x - m);
        const float4 z = *reinterpret_cast<const float4*>(merge + (size_t)from * D + d);
        o.x = fmaf(z.x, f, o.x), o.y = fmaf(z.y, f, o.y), o.z = fmaf(z.z, f, o.z), o.w = fmaf(z.w, f, o.w);
        lsum = fmaf(y.y, f, lsum);
      }
      if (whole) {
        finish(r, d, o, m, lsum);
      } else {
        __stcg(reinterpret_cast<float4*>(p.part_o + (slot * cta_rows + r) * D + d), o);
        if (d == 0) __stcg(p.part_ml + slot * cta_rows + r, make_float2(m, lsum));
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      unsigned int* cnt_at = p.arrived + (size_t)s * per_seq + hb;
      if (tid == 0) wsum[4] = atomicAdd(cnt_at, 1u) == c_last - c_first;
      __syncthreads();
      if (wsum[4]) {
        __threadfence();
        for (int idx = tid; idx < rows * (D / 4); idx += kAttendThreads) {
          const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
          float m = -INFINITY, lsum = 0.f;
          for (unsigned int x = c_first; x <= c_last; ++x)
            m = fmaxf(m, __ldcg(p.part_ml + (size_t)part_slot(x, base, share) * cta_rows + r).x);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (unsigned int x = c_first; x <= c_last; ++x) {
            const size_t from = (size_t)part_slot(x, base, share) * cta_rows + r;
            const float2 y = __ldcg(p.part_ml + from);
            const float4 z = __ldcg(reinterpret_cast<const float4*>(p.part_o + from * D + d));
            const float f = m == -INFINITY ? (y.y != y.y ? y.y : 0.f) : exp2_approx(y.x - m);
            o.x = fmaf(z.x, f, o.x), o.y = fmaf(z.y, f, o.y), o.z = fmaf(z.z, f, o.z), o.w = fmaf(z.w, f, o.w);
            lsum = fmaf(y.y, f, lsum);
          }
          finish(r, d, o, m, lsum);
        }
        if (tid == 0) *cnt_at = 0u;   // for the next call
      }
    }
    pos += cnt;
    __syncthreads();   // shared memory is read
  }
}

}  // namespace mono
