// Attention of 1-8 new tokens a sequence over the paged 8-bit cache.
#pragma once
#include <type_traits>

#include "kv_append.cuh"

namespace mono {

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A B, from zero
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 x 8 transpose of 16-bit values across a warp
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// four e4m3 codes -> two pairs of fp16 values, exactly
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
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
  int q_vec, o_vec;       // whether q and out take four values at a time
  int wr, row_blocks;     // warps side by side over the rows; row blocks of a key head
  unsigned least;         // rounds a CTA takes at least
  unsigned lead;          // rounds that an item's start stands for on the line
  float scale_log2;
};

constexpr int kQRows = 2;         // rows of q that a warp loads together
constexpr int kStages = 2;        // tiles that a warp has in flight or in use
constexpr float kPBias = 15.f;   // probabilities are held as 2^15 p: fp16 keeps 11 bits down to p = 2^-29;
constexpr float kPUnit = 1.f / 32768.f;   // sums of p times values come without it, or values above 2^113 would pass fp32's end

template <int D, int NT, bool F32, int W>
struct AttendShape {
  static constexpr int kThreads = 32 * W;
  static constexpr int kSubs = D == 64 ? (NT == 1 ? 4 : 2) : D == 128 ? 2 : 1;   // groups of 16 tokens a warp's tile holds
  static constexpr int kTile = 16 * kSubs;                       // tokens
  static constexpr int kSplit = F32 ? 2 : 1;                     // fp16 terms that q and p are carried in
  static constexpr int kRows = 8 * NT;                           // rows of a warp
  static constexpr int kSteps = D / 16;
  static constexpr int kValWords = D / 32;                       // 32-bit words of values a lane holds, for each of its 4 tokens
  static constexpr int kStage = 2 * kTile * D;                   // bytes of a tile's keys and values
  static constexpr int kRing = kStages * kStage + kStages * 32;  // a warp's tiles, and their scales
  static size_t smem(int seqs, int wr) {
    return (size_t)(seqs + 1 + 3) / 4 * 16 + (size_t)wr * NT * kSplit * kSteps * 256 + W * kRows * 8 + 4 * kRows * 12 +
           64 + W * kRing;
  }
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// warps of an SM: their registers, 168 or 255
__host__ __device__ constexpr int attend_wide_warps(int d, int nt) { return d == 64 || (d == 128 && nt == 1) ? 12 : 8; }

// where a 16-byte chunk of a token's row lies in a group of 16 tokens: keys are
// read by 8 lanes as 4 chunks of 2 rows next to each other, values as 2 chunks
// of 4 rows two apart; these places meet no bank twice
template <int D, bool VALUES>
__device__ __forceinline__ int kv_place(int row, int chunk) {
  if (D == 64) {
    if (!VALUES) return row * 64 + chunk * 16;
    return (row >> 1) * 128 + ((((row & 1) << 2) + chunk) ^ (((row >> 1) & 3) << 1)) * 16;
  }
  return row * D + (chunk ^ (VALUES ? ((row >> 1) & 3) << 1 : (row & 1) << 2)) * 16;
}

// where four dimensions of a row lie in a warp's results: apart for the 2 g x 4 t
// lanes that write together
template <int D>
__device__ __forceinline__ int merge_place(int row, int d) {
  const int t = (row >> 1) & 3;
  return d ^ (D == 64 ? (t & 1) | ((t & 2) << 1) : t) * 4;
}

// rows [first, first + rows) of a sequence and key head, of at most `stride` in a CTA
struct Item {
  int s, h, first, rows, stride;
};

template <bool F32>
__device__ __noinline__ void finish_row(const AttendParams& p, const Item& it, int r, int d, float4 o, float m, float l) {
  const int row = it.first + r, j = row / p.group, hq = it.h * p.group + (row - j * p.group);
  const float inv = l > 0.f || l != l ? __fdiv_rn(1.f / kPUnit, l) : 0.f;
  o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  const long long at = (long long)it.s * p.o_seq + (long long)j * p.o_tok + (long long)hq * p.o_head + d;
  if (F32) {
    float* to = reinterpret_cast<float*>(p.out) + at;
    if (p.o_vec) *reinterpret_cast<float4*>(to) = o;
    else to[0] = o.x, to[1] = o.y, to[2] = o.z, to[3] = o.w;
  } else {
    __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(p.out) + at;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    if (p.o_vec)
      *reinterpret_cast<uint2*>(to) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    else
      to[0] = lo.x, to[1] = lo.y, to[2] = hi.x, to[3] = hi.y;
  }
  if (p.lse && d == 0)
    p.lse[((long long)it.s * p.width + j) * p.q_heads + hq] =
        l == 0.f ? -INFINITY : (m + log2f(l) - kPBias) * 0.6931471805599453f;
}

// (O, m, l) of another part added
__device__ __forceinline__ void join_part(float4& o, float& m, float& l, const float4& z, const float2& y) {
  const float now = fmaxf(m, y.x);
  const float f = m == now ? 1.f : exp2_approx(m - now), e = y.x == now ? 1.f : exp2_approx(y.x - now);
  o.x = fmaf(z.x, e, o.x * f), o.y = fmaf(z.y, e, o.y * f), o.z = fmaf(z.z, e, o.z * f), o.w = fmaf(z.w, e, o.w * f);
  l = fmaf(y.y, e, l * f);
  m = now;
}

// An item's partial results of CTAs [c_first, c_last], in their order.  Out of
// line and in few instructions: a part of the kernel that runs once is fetched
// from memory, which took longer than its loads (7.7 us where this takes 3).
template <int D, bool F32>
__device__ __noinline__ void join_parts(const AttendParams& p, const Item& it, unsigned int base, unsigned int share,
                                        unsigned int c_first, unsigned int c_last) {
  constexpr int kBatch = 6;   // parts in flight
  for (int idx = threadIdx.x; idx < it.rows * (D / 4); idx += blockDim.x) {
    const int r = idx / (D / 4), d = (idx % (D / 4)) * 4;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (unsigned int x = c_first; x <= c_last; x += kBatch) {
      float4 z[kBatch];
      float2 y[kBatch];
#pragma unroll
      for (unsigned int k = 0; k < kBatch; ++k) {
        const size_t from = (size_t)part_slot(min(x + k, c_last), base, share) * it.stride + r;
        y[k] = __ldcg(p.part_ml + from);
        z[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + from * D + d));
      }
#pragma unroll
      for (unsigned int k = 0; k < kBatch; ++k)
        if (x + k <= c_last) join_part(o, m, l, z[k], y[k]);
    }
    finish_row<F32>(p, it, r, d, o, m, l);
  }
}

// a lane's elements of rows of q
template <int D>
struct QRows {
  float v[kQRows][(D + 127) / 128][4];
};

// One warp multiplies tiles of kTile tokens with 8 NT query rows: the scores
// S^T = K Q^T with the tokens as the m dimension, the output O^T = V^T P^T
// with the head's dimensions as m, so 8 rows fill an MMA's n and no lane
// works on padding at the usual group sizes.  A warp's tiles come through a
// ring of its own by asynchronous copies, keys and values each two tiles
// ahead, so no warp waits for another until its item ends; a lane's 16 bytes
// of keys are its k indices of four MMAs, and q is permuted to match.
//
// The work is the line of all (sequence, key head, row block, round), a round
// being a tile for each of the CTA's warps along the tokens, cut into equal
// runs, one a CTA; an item's start counts as some rounds more, which its pages,
// q, merge and the filling of the rings take.  The cut follows the lengths on
// the device, so one captured launch serves any lengths.  An item that spans CTAs leaves partial (O, m, l)
// in the scratch, and the CTA that arrives last joins them in a fixed order:
// results do not depend on the order of arrival.
//
// Measured, heads 40 / 8 of 128, bf16: one sequence of 131071 tokens 62 us
// (its rounds run at 7.0 TB/s; 3 us lie before the first copy, 10 behind the
// last), 8 sequences to 8192 tokens 29 us, one token 7.5 us.  With the rings in
// shared memory little L1 is left for spilled registers: 50 words that every
// tile stored and loaded took a third of the time.  bf16 kernels with 8 rows a
// warp spill none; with 16 rows of 128 dimensions a warp 9 to 13 words are
// spilled, elsewhere up to 3.
template <int D, int NT, bool F32, int W>
__global__ void __launch_bounds__(32 * W, W > 4 ? 1 : attend_wide_warps(D, NT) / 4)
    attend_kernel(const __grid_constant__ AttendParams p) {
  using S = AttendShape<D, NT, F32, W>;
  constexpr int kSubs = S::kSubs, T = S::kTile, kRows = S::kRows, kSplit = S::kSplit;
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned int* cum = reinterpret_cast<unsigned int*>(smem);
  unsigned char* big = smem + (size_t)(p.seqs + 1 + 3) / 4 * 16;
  uint2* qf = reinterpret_cast<uint2*>(big);
  float2* ml = reinterpret_cast<float2*>(big + (size_t)p.wr * NT * kSplit * S::kSteps * 256);   // [W warps][kRows]
  float* rowf = reinterpret_cast<float*>(ml + W * kRows);                             // [wr kRows]
  int* rlo = reinterpret_cast<int*>(rowf + 4 * kRows);
  int* rhi = rlo + 4 * kRows;
  unsigned int* wsum = reinterpret_cast<unsigned int*>(rhi + 4 * kRows);              // [W], then a flag
  unsigned char* rings = reinterpret_cast<unsigned char*>(wsum + 16);
  float* merge = reinterpret_cast<float*>(rings);   // once the rings are read
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int cap = p.max_pages << p.page_shift, P = 1 << p.page_shift;
  const int wt = warp / p.wr, wrow = warp - wt * p.wr, WT = W / p.wr;
  const int cta_rows = p.wr * kRows, round = T * WT;

  // rounds before each sequence
  {
    const int per = (p.seqs + S::kThreads - 1) / S::kThreads;
    const int s0 = min(tid * per, p.seqs), s1 = min(s0 + per, p.seqs);
    unsigned int sum = 0;
    for (int s = s0; s < s1; ++s)
      sum += seq_tiles(view_seq(__ldg(p.lens + s), p.n_new ? __ldg(p.n_new + s) : p.width, p.width, cap), p.window, cap, round, p.lead);
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
      at += seq_tiles(v, p.window, cap, round, p.lead);
    }
    if (tid == S::kThreads - 1) cum[p.seqs] = at;
    __syncthreads();
  }
  const unsigned int per_seq = (unsigned)(p.kv_heads * p.row_blocks);
  const unsigned int total = cum[p.seqs] * per_seq;
  const unsigned int share = share_of(total, gridDim.x, p.least);
  const unsigned int cta = blockIdx.x;
  if ((unsigned long long)cta * share >= total) return;
  const unsigned int end = min(total, cta * share + share);

  const unsigned char* ring = rings + warp * S::kRing;
  const uint32_t ring_at = smem_u32(ring);
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
    const unsigned int rel = pos - seq_base, hb = rel / n_t, at = rel - hb * n_t;
    if (at < p.lead) {
      pos += p.lead - at;
      continue;
    }
    const unsigned int tile0 = at - p.lead, cnt = min(n_t - at, end - pos), base = seq_base + hb * n_t + p.lead;
    const int h = (int)hb / p.row_blocks, rb = (int)hb - h * p.row_blocks;
    const SeqView sv = view_seq(__ldg(p.lens + s), p.n_new ? __ldg(p.n_new + s) : p.width, p.width, cap);
    const int live = sv.n * p.group - rb * cta_rows;   // live rows of this block (may pass cta_rows)
    const int tok_lo = row_lo(sv, 0, p.window), tok_hi = row_hi(sv, sv.n - 1, cap);
    const int all_lo = row_lo(sv, sv.n - 1, p.window), all_hi = row_hi(sv, 0, cap);
    const int tok0 = (tok_lo / round + (int)tile0) * round + wt * T;   // the warp's first tile

    // the page of each 16 tokens of the warp's i-th tile that some row sees
    int pid[2][kSubs];   // of the two tiles that are asked for next
    auto find_pages = [&](int i, int* to) {
#pragma unroll
      for (int b = 0; b < kSubs; ++b) {
        const int tok = tok0 + i * round + b * 16;
        to[b] = -1;
        if (i < (int)cnt && tok < tok_hi && tok + 16 > tok_lo)
          to[b] = __ldg(p.table + (long long)s * p.max_pages + (tok >> p.page_shift));
      }
    };
    // which of them can be used
    auto check_pages = [&](int i, const int* page) {
      unsigned int m = 0;
#pragma unroll
      for (int b = 0; b < kSubs; ++b) {
        const int tok = tok0 + i * round + b * 16;
        if (page_ok(page[b], p.num_pages)) m |= 1u << b;
        else if (lane == 0 && i < (int)cnt && tok < tok_hi && tok + 16 > tok_lo) record_bad(p.bad, kBadPage, s, page[b]);
      }
      return m;
    };
    // (groups that are not there keep whatever the ring holds; their scales read as zero)
    const long long head_at = (long long)h * P * D + lane * 16;
    auto issue = [&](int i, unsigned int ok, const int* page, auto values) {
      constexpr bool VALUES = decltype(values)::value;
      if (i < (int)cnt) {
        const uint32_t to = ring_at + i % kStages * S::kStage + (VALUES ? T * D : 0);
        constexpr int kChunks = D / 16, kPer = 32 / kChunks;   // chunks a row; rows that a warp copies at once
#pragma unroll
        for (int b = 0; b < kSubs; ++b)
          if ((ok >> b) & 1u) {
            const uint8_t* from = (VALUES ? p.v : p.k) + head_at + (long long)page[b] * (p.kv_heads * P * D) +
                                  ((tok0 + i * round + b * 16) & (P - 1)) * D;
#pragma unroll
            for (int j = 0; j < 16 / kPer; ++j)
              cp_async<16>(to + b * 16 * D + kv_place<D, VALUES>(lane / kChunks + j * kPer, lane % kChunks), from + j * 512);
            if (lane == b)
              cp_async<4>(ring_at + kStages * S::kStage + (i % kStages * 8 + (VALUES ? 4 : 0) + b) * 4,
                          (VALUES ? p.vs : p.ks) + (long long)page[b] * p.kv_heads + h);
          }
      }
      cp_async_commit();
    };
    const std::false_type keys;
    const std::true_type values;
    auto load_q = [&](int r0, QRows<D>& q) {
#pragma unroll
      for (int k = 0; k < kQRows; ++k) {
        const int r = r0 + W * k, m = rb * cta_rows + r, j = m / p.group, hq = h * p.group + (m - j * p.group);
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c) {
          const int d0 = (c * 32 + lane) * 4;
          const bool there = r < live && r < cta_rows && d0 < D;
          const long long at = (long long)s * p.q_seq + (long long)j * p.q_tok + (long long)hq * p.q_head + d0;
          if (there && p.q_vec) {
            if (F32) {
              const float4 w = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + at));
              q.v[k][c][0] = w.x, q.v[k][c][1] = w.y, q.v[k][c][2] = w.z, q.v[k][c][3] = w.w;
            } else {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(p.q) + at));
              q.v[k][c][0] = bf16lo(w.x), q.v[k][c][1] = bf16hi(w.x), q.v[k][c][2] = bf16lo(w.y), q.v[k][c][3] = bf16hi(w.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              q.v[k][c][i] = !there ? 0.f
                            : F32  ? reinterpret_cast<const float*>(p.q)[at + i]
                                   : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.q)[at + i]);
          }
        }
      }
    };
    unsigned int ok[kStages + 1];   // of tiles i, i + 1, ...
#pragma unroll
    for (int k = 0; k <= kStages; ++k) ok[k] = 0u;
    find_pages(0, pid[0]);
    find_pages(1, pid[1]);
    QRows<D> q;
    load_q(warp, q);

    float rf[NT][2];
    float O[D / 16][NT][4], mx[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mx[n][0] = mx[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 16; ++w) O[w][n][0] = O[w][n][1] = O[w][n][2] = O[w][n][3] = 0.f;
    }
    const uint2* qw = qf + (size_t)wrow * NT * kSplit * S::kSteps * 32 + lane;

    // the first kStages turns only ask for tiles
#pragma unroll 1
    for (int i = -kStages; i < (int)cnt; ++i) {
      if (i == 0) {
        // q: each row scaled by a power of two into fp16's range, in the B fragments' order
        for (int r0 = warp; r0 < cta_rows; r0 += W * kQRows) {
          if (r0 != warp) load_q(r0, q);
#pragma unroll
          for (int k = 0; k < kQRows; ++k) {
            const int r = r0 + W * k, j = (rb * cta_rows + r) / p.group;
            if (r >= cta_rows) break;
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < (D + 127) / 128; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(q.v[k][c][i]));
            amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax)));
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
                    const float a = q.v[k][c][2 * i] * up, b = q.v[k][c][2 * i + 1] * up;
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
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) rf[n][i] = rowf[wrow * kRows + n * 8 + 2 * t + i];
      }
      const int tile_tok = tok0 + i * round, next = i + kStages;
      const bool edge = tile_tok < all_lo || tile_tok + T > all_hi || ok[0] != (1u << kSubs) - 1u;
      const int at_stage = (i + kStages) % kStages;
      const unsigned char* kt = ring + at_stage * S::kStage;
      const float* sc = reinterpret_cast<const float*>(ring + kStages * S::kStage) + at_stage * 8;
      float c[kSubs][NT][4], top[NT][2];
      bool grew = false;
      if (i >= 0) {
        cp_async_wait<2 * kStages - 1>();
        __syncwarp();
        // scores
#pragma unroll
        for (int b = 0; b < kSubs; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n) c[b][n][0] = c[b][n][1] = c[b][n][2] = c[b][n][3] = 0.f;
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch) {
          uint4 k0[kSubs], k1[kSubs];   // rows g and g + 8
#pragma unroll
          for (int b = 0; b < kSubs; ++b) {
            const unsigned char* at = kt + b * 16 * D + kv_place<D, false>(g, ch * 4 + t);
            k0[b] = *reinterpret_cast<const uint4*>(at);
            k1[b] = *reinterpret_cast<const uint4*>(at + 8 * D);
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a[kSubs][4];
#pragma unroll
            for (int b = 0; b < kSubs; ++b) {
              const uint32_t w0 = w == 0 ? k0[b].x : w == 1 ? k0[b].y : w == 2 ? k0[b].z : k0[b].w;
              const uint32_t w1 = w == 0 ? k1[b].x : w == 1 ? k1[b].y : w == 2 ? k1[b].z : k1[b].w;
              e4m3x4_to_h2(w0, a[b][0], a[b][2]);
              e4m3x4_to_h2(w1, a[b][1], a[b][3]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int sp = 0; sp < kSplit; ++sp) {
                const uint2 q2 = qw[((n * kSplit + sp) * S::kSteps + ch * 4 + w) * 32];
#pragma unroll
                for (int b = 0; b < kSubs; ++b) mma_f16(c[b][n], a[b], q2.x, q2.y);
              }
          }
        }
        float ksc[kSubs];
#pragma unroll
        for (int b = 0; b < kSubs; ++b) ksc[b] = sc[b];
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
                const int tok = tile_tok + b * 16 + g + (j >> 1) * 8;
                if (tok < lo || tok >= hi || !((ok[0] >> b) & 1u)) c[b][n][j] = -INFINITY;
              }
            }
          }
#pragma unroll
          for (int b = 0; b < kSubs; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) top[n][j & 1] = fmaxf(top[n][j & 1], c[b][n][j]);
        }
        // the rows' maxima
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
      }
      __syncwarp();   // the keys are read
      ok[kStages] = check_pages(next, pid[0]);
      issue(next, ok[kStages], pid[0], keys);
      if (i >= 0) {
        cp_async_wait<2 * kStages - 1>();
        __syncwarp();
        float vsc[kSubs];
#pragma unroll
        for (int b = 0; b < kSubs; ++b) vsc[b] = (ok[0] >> b) & 1u ? sc[4 + b] : 0.f;
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
        uint32_t pf[kSubs][NT][kSplit][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // the difference first: it is 0 for the largest logit, whose probability is 1
          const float off0 = mx[n][0] == -INFINITY ? 0.f : mx[n][0];
          const float off1 = mx[n][1] == -INFINITY ? 0.f : mx[n][1];
#pragma unroll
          for (int b = 0; b < kSubs; ++b) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              e[j] = exp2_approx(c[b][n][j] - (j & 1 ? off1 : off0) + kPBias);
              l[n][j & 1] += e[j];
            }
            // a scale that is no finite number: only what sees the page's tokens meets it
            if (!(fabsf(vsc[b]) <= 3.402823466e38f)) {
#pragma unroll
              for (int j = 0; j < 4; ++j) e[j] = c[b][n][j] == -INFINITY ? 0.f : e[j] * vsc[b];
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
        // output, 16 tokens of a page at a time: their products by the matrix unit,
        // which cuts what it adds up, then times the page's scale in fp32.  With
        // the scale in the probabilities instead, a page of large values took the
        // others' bits, also from rows that do not see it.
#pragma unroll
        for (int b = 0; b < kSubs; ++b) {
          if (!(fabsf(vsc[b]) <= 3.402823466e38f)) vsc[b] = 1.f;
          // A scale times 2^-15 is inexact below 2^-111.  bf16 rows keep at least 8 bits
          // of it; fp32 rows take the 2^-15 off the products there (for every scale:
          // registers spilled, 3 %; the branch in bf16 rows 2 %).
          const bool low = F32 && fabsf(vsc[b]) < 0x1p-100f;
          const float vs = low ? vsc[b] : vsc[b] * kPUnit;
          uint32_t vw[4][S::kValWords];   // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + (r >> 1) * 8;
            const unsigned char* vt = kt + T * D + b * 16 * D;
            if (D == 64) {
              const uint2 w = *reinterpret_cast<const uint2*>(vt + kv_place<D, true>(row, g >> 1) + (g & 1) * 8);
              vw[r][0] = w.x, vw[r][1] = w.y;
            } else {
#pragma unroll
              for (int ch = 0; ch < D / 128; ++ch) {
                const uint4 w = *reinterpret_cast<const uint4*>(vt + kv_place<D, true>(row, ch * 8 + g));
                uint32_t* d = &vw[r][(ch * 4) % S::kValWords];
                d[0] = w.x, d[1] = w.y, d[2 % S::kValWords] = w.z, d[3 % S::kValWords] = w.w;
              }
            }
          }
          // a tile that some row does not see in full: values behind the sequence
          // (or before its window) read as zero; a NaN value reaches only the
          // rows that see its token
          if (edge) {
            bool nan = false;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int tok = tile_tok + b * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
              const bool in = tok >= tok_lo && tok < tok_hi && ((ok[0] >> b) & 1u);
#pragma unroll
              for (int w = 0; w < S::kValWords; ++w) {
                if (!in) vw[r][w] = 0;
                nan |= (((vw[r][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u;
              }
            }
            if (__any_sync(0xFFFFFFFFu, nan)) {
              uint32_t sees[NT][2];
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int tok = tile_tok + b * 16 + g + j * 8;
                  const int row = wrow * kRows + n * 8 + 2 * t;
                  sees[n][j] = movmatrix((tok >= rlo[row] && tok < rhi[row] ? 0x3C00u : 0u) |
                                         (tok >= rlo[row + 1] && tok < rhi[row + 1] ? 0x3C000000u : 0u));
                }
#pragma unroll
              for (int w = 0; w < 2 * S::kValWords; ++w) {
                uint32_t y[4];   // 1.0 (e4m3 0x38) where the code is NaN
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  y[r] = ((((vw[r][w >> 1] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0x38u;
                const uint32_t x0 = __byte_perm(y[0], y[1], w & 1 ? 0x7362 : 0x5140);
                const uint32_t x1 = __byte_perm(y[2], y[3], w & 1 ? 0x7362 : 0x5140);
                uint32_t a[4];
                e4m3x4_to_h2(x0, a[0], a[1]);
                e4m3x4_to_h2(x1, a[2], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float hit[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(hit, a, sees[n][0], sees[n][1]);
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (hit[j] > 0.f) O[w][n][j] = __int_as_float(0x7FC00000);
                }
              }
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int w = 0; w < S::kValWords; ++w) {
                  const uint32_t y = ((vw[r][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                  vw[r][w] &= ~((y >> 7) * 0xFFu);
                }
            }
          }
#pragma unroll
          for (int w = 0; w < 2 * S::kValWords; ++w) {
            // a dimension's codes of two tokens side by side, then two pairs of them at once
            const uint32_t x0 = __byte_perm(vw[0][w >> 1], vw[1][w >> 1], w & 1 ? 0x7362 : 0x5140);
            const uint32_t x1 = __byte_perm(vw[2][w >> 1], vw[3][w >> 1], w & 1 ? 0x7362 : 0x5140);
            uint32_t a[4];
            e4m3x4_to_h2(x0, a[0], a[1]);
            e4m3x4_to_h2(x1, a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float o[4];
              mma_f16_first(o, a, pf[b][n][0][0], pf[b][n][0][1]);
              if (F32) mma_f16(o, a, pf[b][n][kSplit - 1][0], pf[b][n][kSplit - 1][1]);
              if (low) o[0] *= kPUnit, o[1] *= kPUnit, o[2] *= kPUnit, o[3] *= kPUnit;
#pragma unroll
              for (int j = 0; j < 4; ++j) O[w][n][j] = fmaf(o[j], vs, O[w][n][j]);
            }
          }
        }
      }
      __syncwarp();   // the values are read
      issue(next, ok[kStages], pid[0], values);
#pragma unroll
      for (int b = 0; b < kSubs; ++b) pid[0][b] = pid[1][b];
      find_pages(next + 2, pid[1]);
#pragma unroll
      for (int k = 0; k < kStages; ++k) ok[k] = ok[k + 1];
    }

    // the CTA's warps together
    __syncthreads();   // q and the rings are read
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
          *reinterpret_cast<float4*>(merge + ((size_t)warp * kRows + row) * D + merge_place<D>(row, d)) =
              make_float4(O[2 * w][n][r], O[2 * w][n][2 + r], O[2 * w + 1][n][r], O[2 * w + 1][n][2 + r]);
        }
      }
    __syncthreads();
    const unsigned int c_first = base / share, c_last = (base + n_t - p.lead - 1) / share;
    const bool whole = c_first == c_last;
    const Item item{s, h, rb * cta_rows, min(live, cta_rows), cta_rows};
    const size_t slot = part_slot(cta, base, share);
    const int rows = item.rows;
    for (int idx = tid; idx < rows * (D / 4); idx += S::kThreads) {
      const int r = idx / (D / 4), d = (idx % (D / 4)) * 4, wq = r / kRows, rr = r % kRows;
      const int first = wq * kRows + rr, step = p.wr * kRows;
      float m = -INFINITY, lsum = 0.f;
#pragma unroll 4
      for (int w = 0; w < WT; ++w) m = fmaxf(m, ml[first + w * step].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < WT; ++w) {
        const float2 y = ml[first + w * step];
        const float4 z =
            *reinterpret_cast<const float4*>(merge + (size_t)(first + w * step) * D + merge_place<D>(rr, d));
        const float f = y.x == m ? 1.f : exp2_approx(y.x - m);
        o.x = fmaf(z.x, f, o.x), o.y = fmaf(z.y, f, o.y), o.z = fmaf(z.z, f, o.z), o.w = fmaf(z.w, f, o.w);
        lsum = fmaf(y.y, f, lsum);
      }
      if (whole) {
        finish_row<F32>(p, item, r, d, o, m, lsum);
      } else {
        __stcg(reinterpret_cast<float4*>(p.part_o + (slot * cta_rows + r) * D + d), o);
        if (d == 0) __stcg(p.part_ml + slot * cta_rows + r, make_float2(m, lsum));
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      unsigned int* cnt_at = p.arrived + (size_t)s * per_seq + hb;
      if (tid == 0) wsum[W] = atomicAdd(cnt_at, 1u) == c_last - c_first;
      __syncthreads();
      if (wsum[W]) {
        __threadfence();
        join_parts<D, F32>(p, item, base, share, c_first, c_last);
        if (tid == 0) *cnt_at = 0u;   // for the next call
      }
    }
    pos += cnt;
    __syncthreads();   // shared memory is read
  }
}

}  // namespace mono
