// Index arithmetic of the paged cache, shared by the kernels and the host
// tests: which positions a sequence's rows have and see, where a page's codes
// lie, and how attend's work is cut into equal shares.  Plain C++.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define MONO_HD __host__ __device__ __forceinline__
#else
#define MONO_HD inline
#endif

namespace mono {

enum { kBadPage = 1, kBadLen = 2, kBadNew = 3 };

// A sequence of a call: its live rows, the position of the first of them
// (below zero where the sequence is shorter than its new tokens), what was
// wrong with its entries (0 or kBad*), and whether it is left out: with more new
// tokens than rows, row j's position is not that of a token the caller gave.
struct SeqView {
  int n, first, bad, bad_value;
  bool left_out;
};

MONO_HD SeqView view_seq(int len, int n_new, int width, int cap) {
  SeqView v{n_new, 0, 0, 0, n_new > width};
  if (v.n <= 0) {
    v.n = 0;
    return v;
  }
  if (v.left_out) {
    v.n = width;
    v.bad = kBadNew;
    v.bad_value = n_new;
  }
  if (len < 0 || len > cap) {
    v.bad = kBadLen;
    v.bad_value = len;
  }
  v.first = (len < 0 ? 0 : len) - v.n;
  return v;
}

// tokens that row j of a sequence sees: [lo, hi), empty where hi <= lo
MONO_HD int row_hi(const SeqView& v, int j, int cap) {
  const int e = v.first + j + 1;   // no overflow: first <= INT_MAX - n and j < n
  return e < cap ? e : cap;
}

MONO_HD int row_lo(const SeqView& v, int j, int window) {
  const int e = v.first + j + 1;
  return window > 0 && e > window ? e - window : 0;
}

MONO_HD bool page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }

// row (of head_dim codes) of a token of a page; pages x heads x tokens may pass 32 bits
MONO_HD long long code_row(int page, int kv_heads, int h, int page_size, int tok) {
  return ((long long)page * kv_heads + h) * page_size + tok;
}

// length on the line of a sequence's item: `lead` for its start and the tiles
// of `tile` tokens that its rows read; at least one tile for a live sequence,
// whose rows have to be written even if they see nothing
MONO_HD int seq_tiles(const SeqView& v, int window, int cap, int tile, int lead) {
  if (v.n == 0 || v.left_out) return 0;
  const int lo = row_lo(v, 0, window), hi = row_hi(v, v.n - 1, cap);
  if (hi <= lo) return lead + 1;
  return lead + (hi - 1) / tile - lo / tile + 1;
}

// share of each CTA when `total` tiles are cut into at most `grid` equal runs of at least `least`
MONO_HD unsigned share_of(unsigned total, unsigned grid, unsigned least) {
  const unsigned u = (total + grid - 1) / grid;
  return u > least ? u : least;
}

// Partial results of an item (tiles [base, base + n) of the line, its start not
// among them): CTA c keeps at most two unfinished items, the one its run begins
// in (slot 2c) and the one that begins inside its run and goes on behind it
// (slot 2c + 1).
MONO_HD unsigned part_slot(unsigned c, unsigned base, unsigned share) {
  return 2u * c + (base > c * share ? 1u : 0u);
}

}  // namespace mono
