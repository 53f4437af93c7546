// Shared by the attention kernels: what a workgroup's rows see, and how the
// keys are split.
#pragma once

#include "serving.h"

namespace fcg {

constexpr float LN2 = 0.693147180559945309f;

// What a workgroup's rows see.  All members are the same in every lane.
struct RowTile {
  int s, hk, row0, rows;      // sequence, key head, first row, rows of the sequence
  int q0;                     // first token of the sequence in q
  int kv_len;                 // keys in the table
  int base;                   // position of the sequence's first new token
  int lo, hi;                 // positions of the tile's first and last row
  int beg, end;               // keys that some row sees: [beg, end)
};

// false: the tile has no rows, or its sequence is the other kernel's
__device__ __forceinline__ bool row_tile(const AttendArgs& a, int s, int hk, int tile, int tile_rows,
                                         int min_rows, int max_rows, int align, RowTile& t) {
  const int64_t c0 = a.cu_q[s], c1 = a.cu_q[s + 1];
  const int q0 = (int)(c0 < 0 ? 0 : (c0 > a.T ? a.T : c0));
  const int q1 = (int)(c1 < q0 ? q0 : (c1 > a.T ? a.T : c1));
  const int n = q1 - q0;
  t.s = s;
  t.hk = hk;
  t.q0 = q0;
  t.rows = (n < a.max_q ? n : a.max_q) * a.group;
  t.row0 = tile * tile_rows;
  if (t.row0 >= t.rows || t.rows < min_rows || t.rows > max_rows) return false;
  int len = a.kv_lens[s];
  const int64_t held = (int64_t)a.table_w << a.kv.page_shift;
  len = len < 0 ? 0 : len;
  t.base = len - n;
  t.kv_len = (int)(len < held ? len : held);
  const int last = t.row0 + tile_rows < t.rows ? t.row0 + tile_rows : t.rows;
  t.lo = t.base + t.row0 / a.group;
  t.hi = t.base + (last - 1) / a.group;
  t.end = t.hi + 1 < t.kv_len ? t.hi + 1 : t.kv_len;
  t.beg = a.window > 0 && t.lo - a.window + 1 > 0 ? (t.lo - a.window + 1) & -align : 0;
  return true;
}

// The tiles of tile_rows rows of all of the tile kernel's sequences, one after
// the other: the b-th.  Every wave finds it for itself, 64 sequences at a time.
// (A grid of max_q for each sequence would be mostly of workgroups without
// rows: 12 sequences of 1 .. 1031 tokens, 10 us more.)  false: there is none.
__device__ __forceinline__ bool find_tile(const AttendArgs& a, int b, int hk, int tile_rows, int align, RowTile& t) {
  const int lane = threadIdx.x & 63;
  int s = -1, tile = 0;
  for (int s0 = 0; s0 < a.seqs && s < 0; s0 += 64) {
    RowTile u;                                     // (of this lane's sequence; t is the same in every lane)
    const bool rows = s0 + lane < a.seqs && row_tile(a, s0 + lane, hk, 0, 1, a.stream_rows + 1, INT32_MAX, 1, u);
    const int each = rows ? (u.rows + tile_rows - 1) / tile_rows : 0;
    const int n = each < (1 << 24) ? each : 1 << 24;   // (no grid is that large: so that 64 of them add up in 32 bits)
    int sum = n;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
      const int up = __shfl_up(sum, k);
      if (lane >= k) sum += up;
    }
    const uint64_t past = __ballot(sum > b);
    if (past) {
      const int i = __builtin_ctzll(past);
      s = s0 + i;
      tile = __builtin_amdgcn_readlane(sum, i) - 1 - b;   // the last rows see the most keys: they come first
    } else {
      b -= __builtin_amdgcn_readlane(sum, 63);
    }
  }
  return s >= 0 && row_tile(a, s, hk, tile, tile_rows, a.stream_rows + 1, INT32_MAX, align, t);
}

// keys [c0, c1) of the tile's [beg, end) that split `split` takes: `per` of
// them each, so that the splits of all sequences cost the same
__device__ __forceinline__ void split_range(const RowTile& t, int split, int splits, int per, int& c0, int& c1) {
  const int64_t at = t.beg + (int64_t)split * per, to = at + per;
  c0 = at < t.end ? (int)at : t.end;
  c1 = split + 1 < splits && to < t.end ? (int)to : t.end;
}

// The larger of a and b, of three values: NaN loses.  (The library's maximum
// quiets its operands first; these values come from matrix instructions and
// are quiet already.)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

// The reference point of a row's exponentials: the largest score in powers of
// two, less LIFT.  (Not fused: the fused form keeps LIFT in a register.)
template <class E>
__device__ __forceinline__ float reference_of(float mx, float scale_log2) {
#pragma clang fp contract(off)
  const float z = mx * scale_log2;
  return z - Mat<E>::LIFT;
}

// ---- values in masked places ----
//
// A masked key's weight is 0, and 0 times an infinite or NaN value would be
// NaN.  Keys that no row may see (stale memory, no page) have their values
// cleared.  Where some rows of a tile see a key and others do not, its
// non-finite values are taken out of the product, and a second product counts
// them for each row and dimension: the codes 1, 2^7 and 2^14 for +inf, -inf
// and NaN against 1 for a key that the row sees; 64 keys at most, so that the
// sum is exact and says how many there are of each.

// all ones over the first n of a piece's 8 keys
__device__ __forceinline__ u32x4 keep_keys(int n) {
  u32x4 k;
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = n > 2 * j + 1 ? 0xFFFFFFFFu : (n == 2 * j + 1 ? 0xFFFFu : 0u);
  return k;
}
// not 0 if there are non-finite values
template <class E>
__device__ __forceinline__ uint32_t any_nonfinite(u32x4 v) {
  return nonfinite2<E>(v[0]) | nonfinite2<E>(v[1]) | nonfinite2<E>(v[2]) | nonfinite2<E>(v[3]);
}
// clears them; not 0 if there were any
template <class E>
__device__ __forceinline__ uint32_t take_nonfinite(u32x4& v) {
  uint32_t bad = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t f = nonfinite2<E>(v[j]);
    bad |= f;
    v[j] &= ~((f >> 15) * 0xFFFFu);
  }
  return bad;
}
template <class E>
__device__ __forceinline__ u32x4 nonfinite_codes(u32x4 v) {
  u32x4 c;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t y = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t x = v[j] >> (16 * e) & 0xFFFFu;
      const uint32_t code = (x & 0x7FFFu) > Mat<E>::INF ? Mat<E>::TWO14
                            : (x & 0x7FFFu) == Mat<E>::INF ? (x >> 15 ? Mat<E>::TWO7 : Mat<E>::ONE) : 0u;
      y |= code << (16 * e);
    }
    c[j] = y;
  }
  return c;
}
// what the counted values add up to
__device__ __forceinline__ float nonfinite_sum(float codes) {
  const uint32_t n = (uint32_t)codes, plus = n & 127u, minus = n >> 7 & 127u;
  if (n >> 14 || (plus && minus)) return __builtin_nanf("");
  return plus ? __builtin_inff() : (minus ? -__builtin_inff() : 0.f);
}

// the type's 1 for each of 8 keys from the one after `low` to `top`
template <class E>
__device__ __forceinline__ u32x4 seen_ones(int top, int low) {
  u32x4 one;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    one[j] = (2 * j <= top && 2 * j > low ? Mat<E>::ONE : 0u) | (2 * j + 1 <= top && 2 * j + 1 > low ? Mat<E>::ONE << 16 : 0u);
  return one;
}

// the value of lane + 32 or lane - 32
__device__ __forceinline__ float other_half(float x) {
  uint32_t a = __builtin_bit_cast(uint32_t, x), b = a;
  asm("" : "+v"(b));                            // (of two equal operands the compiler takes the results for equal too)
  const auto y = __builtin_amdgcn_permlane32_swap(a, b, false, false);   // {own low half twice, own high half twice}
  return __builtin_bit_cast(float, threadIdx.x & 32 ? y[0] : y[1]);
}

hipError_t launch_attend_tile(const AttendArgs& a, const AttendPlan& p, int dtype, hipStream_t st);

}  // namespace fcg
