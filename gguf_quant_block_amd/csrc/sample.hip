// The choice of the next token of each row of logits.
//
//   w_v = 2^(c x_v - top), c = log2(e) / temperature;  order: x descending, ties by id
//   kept: the beginning of that order that top_k, top_p and min_p leave
//   the first of the kept whose running sum of w passes u times the sum of the kept
//
// No row is sorted.  A token's weight is a whole number: with z = c x (f64), its
// octave floor(z) and M = 2^(z - octave) 2^33, rounded.  Quarters of octaves
// are the bins of a histogram, which are in the order of x and whose places do
// not depend on the row's largest, so that slices of a row are summed apart and
// joined later; sums of whole numbers do not depend on their order, and every
// level below adds up to the same.  A bin holds what top_k, top_p and u look for
// by its running sums, and only the tokens of such a bin are looked at again:
// 256 ways at a time, until few enough are left to be ranked against each other.
// (M is off by 2^-34 of itself; against sums of f64 a border moves by about
// 10^-10 of the sum, the rounding of u to f32 by 6 * 10^-8.)
//
// Tokens more than 64 octaves below the largest weigh less than 2^-40 together
// (vocab <= 2^24) and are never chosen; they are dropped from the histogram.
#include <math.h>

#include "serving.h"

namespace fcg {
namespace {

typedef unsigned long long u64;

constexpr int BINS = SAMPLE_BINS, QUARTERS = 4;
constexpr int COUNT_SHIFT = 49;                // a slice's bin: the sum of M below, the count of tokens from here on
constexpr int SLICE_MOST = 16384;              // 2^14 tokens of up to 2^34: 2^48
constexpr int LIST = 8192;                     // tokens that are looked at again from LDS
constexpr int FEW = 512;                       // that are ranked against each other

// N values at an address aligned to one of them
template <class T, int N> struct Some { typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T)))); };

// Where a logit stands: bin numbers fall with x.
struct Place {
  double octave;
  int quarter;
  u64 m;
};

// (No contraction: a token has the same place wherever it is computed.)
__device__ __forceinline__ Place place_of(double x, double c) {
#pragma clang fp contract(off)
  Place p;
  const double z = x * c;
  p.octave = __builtin_floor(z);
  const double f = z - p.octave;               // in [0, 1), but 1 for the least below 0
  const int q = (int)(f * QUARTERS);
  p.quarter = q < QUARTERS ? q : QUARTERS - 1;
  // 2^33 2^f about the middle: sqrt(2) 2^33 (ln 2)^n / n!, off by 2^-38
  const double g = f - 0.5;
  constexpr double L = 0.693147180559945309417;
  constexpr double C0 = 1.41421356237309504880 * 8589934592.0, C1 = C0 * L, C2 = C1 * L / 2, C3 = C2 * L / 3, C4 = C3 * L / 4,
                   C5 = C4 * L / 5, C6 = C5 * L / 6, C7 = C6 * L / 7, C8 = C7 * L / 8, C9 = C8 * L / 9;
  double y = C9;
  y = __builtin_fma(y, g, C8);
  y = __builtin_fma(y, g, C7);
  y = __builtin_fma(y, g, C6);
  y = __builtin_fma(y, g, C5);
  y = __builtin_fma(y, g, C4);
  y = __builtin_fma(y, g, C3);
  y = __builtin_fma(y, g, C2);
  y = __builtin_fma(y, g, C1);
  y = __builtin_fma(y, g, C0);
  p.m = __builtin_bit_cast(u64, y + 4503599627370496.0) & 0xFFFFFFFFFFFFFull;   // (2^52: the fraction's bits are the whole number)
  return p;
}
// bins between a place and one that is not below it; BINS where there are more
__device__ __forceinline__ int bins_below(double octave, int quarter, double top_octave, int top_quarter) {
  const double d = (top_octave - octave) * QUARTERS + (top_quarter - quarter);
  return d < BINS ? (int)d : BINS;
}
// An infinite logit has all the weight, and shares it with its like: its place
// is the top, whatever the others are.
__device__ __forceinline__ Place place_below(float x, float top, double c) {
  if (x == INFINITY) return {0.0, 0, 1ull << 33};
  Place p = place_of((double)x, c);
  if (top == INFINITY) p.octave = -INFINITY;
  return p;
}

struct Settings {
  double c;              // log2(e) / temperature
  int top_k;             // 0: all
  double top_p, min_p, u;
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t row) {
  Settings s;
  const float t = a.temperature ? a.temperature[row] : 1.f;
  s.c = 1.44269504088896340736 / (double)t;
  s.top_k = a.top_k ? a.top_k[row] : 0;
  s.top_p = a.top_p ? (double)a.top_p[row] : 1.0;
  s.min_p = a.min_p ? (double)a.min_p[row] : 0.0;
  s.u = (double)a.u[row];
  if (s.top_k < 0) s.top_k = 0;
  if (!(s.top_p < 1.0)) s.top_p = 1.0;
  if (!(t > 0.f)) {                            // the largest
    s.c = 1.44269504088896340736;
    s.top_k = 1;
  } else if (s.top_p <= 0.0 || s.min_p > 1.0) {
    s.top_k = 1;
  }
  if (s.top_k == 1) {
    s.top_p = 1.0;
    s.min_p = 0.0;
  }
  s.u = s.u > 0.0 ? s.u : 0.0;                 // (NaN too)
  return s;
}

__device__ __forceinline__ float larger(float a, float b) { return a > b ? a : b; }

// What a row's slice holds: the histogram of its tokens below its largest logit.
template <class I, int ROUNDS>
__global__ __launch_bounds__(512) void sample_slice_kernel(SampleArgs a) {
  constexpr int THREADS = 512, SLICE = THREADS * 4 * ROUNDS;
  static_assert(SLICE <= SLICE_MOST, "sums");
  __shared__ u64 hist[BINS];
  __shared__ float wave_top[THREADS / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y, v0 = (int64_t)blockIdx.x * SLICE;
  const int n = (int)(a.vocab - v0 < SLICE ? a.vocab - v0 : SLICE);
  const I* x = (const I*)a.x + row * a.x_stride + v0;
  typedef typename Some<I, 4>::vec IV;
  float z[ROUNDS * 4];
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int i = (k * THREADS + tid) * 4;
    if (i + 4 <= n) {
      const IV y = *(const IV*)(x + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[4 * k + e] = (float)y[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[4 * k + e] = i + e < n ? (float)x[i + e] : -INFINITY;
    }
  }
  if (tid < BINS) hist[tid] = 0;
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4 * ROUNDS; ++k) top = larger(z[k], top);     // (NaN is not larger)
#pragma unroll
  for (int k = 32; k; k /= 2) top = larger(__shfl_xor(top, k), top);
  if ((tid & 63) == 0) wave_top[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < THREADS / 64; ++k) top = larger(wave_top[k], top);
  const double c = settings_of(a, row).c;
  const Place t = place_below(top, top, c);
#pragma unroll
  for (int k = 0; k < 4 * ROUNDS; ++k) {
    if (!(z[k] > -INFINITY)) continue;
    const Place p = place_below(z[k], top, c);
    const int d = bins_below(p.octave, p.quarter, t.octave, t.quarter);
    if (d < BINS) atomicAdd(&hist[d], p.m | 1ull << COUNT_SHIFT);
  }
  __syncthreads();
  const int64_t slice = row * a.slices + blockIdx.x;
  if (tid < BINS) a.hist[slice * BINS + tid] = hist[tid];
  if (tid == 0) a.tops[slice] = top;
}

// The order of tokens: smaller is earlier.
__device__ __forceinline__ u64 order_of(float x, uint32_t id) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);          // (-0 as 0)
  return (u64)(b >> 31 ? b : ~b ^ 0x80000000u) << 32 | id;
}
__device__ __forceinline__ float logit_of(u64 order) {
  const uint32_t b = (uint32_t)(order >> 32);
  return __builtin_bit_cast(float, b >> 31 ? b : ~b ^ 0x80000000u);
}

// A beginning of the order: all bins before `bin`, and of that the first tokens.
struct Beginning {
  int bin;
  uint32_t count;        // tokens of the bin
  u64 sum;               // of their M
  u64 last;              // the last of them
};

template <class I>
struct RowChoice {
  static constexpr int THREADS = 1024;
  struct Shared {
    u64 sum[BINS];
    uint32_t count[BINS];
    double before[BINS + 1];                   // weight of the bins before, in units of 2^-33 of the top octave
    uint32_t count_before[BINS + 1];
    u64 part_sum[4][BINS];                     // (also the histogram of a bin's tokens)
    uint32_t part_count[4][BINS];
    u64 few[FEW], few_m[FEW], few_before[FEW];
    uint32_t few_rank[FEW];
    float wave_top[THREADS / 64];
    uint32_t n;                                // tokens of a list
    int found;
    Beginning got;
    u64 total_sum;
    uint32_t total_count;
    u64 list[LIST];
  };

  const SampleArgs& a;
  Shared& s;
  const int tid;
  const I* x;
  Settings set;
  float top;
  Place at;              // of the largest logit
  bool listed;
  int list_n;

  // bin of a token, BINS or more: of none
  __device__ __forceinline__ int bin_of(float v, u64& m) const {
    const Place p = place_below(v, top, set.c);
    m = p.m;
    return bins_below(p.octave, p.quarter, at.octave, at.quarter);
  }
  // 2^(octave of a bin - top octave)
  __device__ __forceinline__ double unit_of(int bin) const {
    const int q = at.quarter - bin;            // quarters above the top octave's begin
    const int octave = q >= 0 ? 0 : -((-q + QUARTERS - 1) / QUARTERS);
    return __builtin_ldexp(1.0, octave);
  }
  // No logit of bins up to `bin` is below this (and some that are not, are: bins are asked for).
  __device__ __forceinline__ float lowest_of(int bin) const {
    if (top == INFINITY) return INFINITY;
    const double z = at.octave + (at.quarter - bin) * (1.0 / QUARTERS), y = z / set.c;
    const float f = (float)(y - fabs(y) * 1e-6);
    return set.c > 0.0 && f == f ? f : -INFINITY;
  }

  // every token of bins first .. last that the row (or the list) has
  template <class F>
  __device__ __forceinline__ void each(int first, int last, F f) {
    auto look = [&](float v, uint32_t id) {
      u64 m;
      const int d = bin_of(v, m);
      if (d >= first && d <= last) f(v, id, m);
    };
    if (listed) {
      for (int i = tid; i < list_n; i += THREADS) look(logit_of(s.list[i]), (uint32_t)s.list[i]);
      return;
    }
    typedef typename Some<I, 4>::vec IV;
    const float low = lowest_of(last);
    const int n = (int)a.vocab, whole = n & ~3;
#pragma unroll 4
    for (int i = tid * 4; i < whole; i += THREADS * 4) {
      const IV y = *(const IV*)(x + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = (float)y[e];
        if (v >= low && v > -INFINITY) look(v, (uint32_t)(i + e));
      }
    }
    if (tid < n - whole) {
      const float v = (float)x[whole + tid];
      if (v >= low && v > -INFINITY) look(v, (uint32_t)(whole + tid));
    }
  }

  // The beginning of a bin that ends with its token `count` (where it is not
  // 0), or with the first whose running sum is `sum` or more.
  __device__ Beginning select(int bin, uint32_t count, u64 sum) {
    uint32_t had = 0, n = s.count[bin];        // tokens before those that are left, and how many these are
    u64 had_sum = 0, lo = 0, hi = ~0ull;       // sum before them, and their range
    if (n > FEW && top < INFINITY) {           // (a wide range of the bin's: what is outside goes to its ends)
      const float low = lowest_of(bin);
      const double z = at.octave + (at.quarter - bin + 1) * (1.0 / QUARTERS), y = z / set.c;
      const float high = (float)(y + fabs(y) * 1e-6);
      if (low > -INFINITY) hi = order_of(low, ~0u);
      if (set.c > 0.0 && high < INFINITY) lo = order_of(high, 0);
    }
    bool first = true;
    while (n > FEW) {
      // 256 ways
      const u64 range = hi - lo;
      const int bits = 64 - __builtin_clzll(range | 1), shift = bits > 8 ? bits - 8 : 0;
      if (tid < BINS) {
        s.part_sum[0][tid] = 0;
        s.part_count[0][tid] = 0;
      }
      __syncthreads();
      each(bin, bin, [&](float v, uint32_t id, u64 m) {
        const u64 o = order_of(v, id);
        if (!first && (o < lo || o > hi)) return;
        const int w = o < lo ? 0 : o > hi ? (int)(range >> shift) : (int)((o - lo) >> shift);
        atomicAdd(&s.part_sum[0][w], m);
        atomicAdd(&s.part_count[0][w], 1u);
      });
      __syncthreads();
      if (tid < 64) {
        // running sums, four ways a lane
        uint32_t c4 = 0;
        u64 s4 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c4 += s.part_count[0][4 * tid + k];
          s4 += s.part_sum[0][4 * tid + k];
        }
        uint32_t cs = c4;
        u64 ss = s4;
#pragma unroll
        for (int k = 1; k < 64; k *= 2) {
          const uint32_t cu = __shfl_up(cs, k);
          const u64 su = __shfl_up(ss, k);
          if (tid >= k) {
            cs += cu;
            ss += su;
          }
        }
        uint32_t cb = had + cs - c4;
        u64 sb = had_sum + ss - s4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t cn = s.part_count[0][4 * tid + k];
          const u64 sn = s.part_sum[0][4 * tid + k];
          if (count ? cb < count && count <= cb + cn : sb < sum && sum <= sb + sn) {
            s.found = 4 * tid + k;
            s.total_count = cb;
            s.total_sum = sb;
          }
          cb += cn;
          sb += sn;
        }
      }
      __syncthreads();
      const int w = s.found;
      had = s.total_count;
      had_sum = s.total_sum;
      n = s.part_count[0][w];
      // (at the first level the ends hold what is outside the range too)
      const u64 from = lo + ((u64)w << shift), to = shift ? from + (((u64)1 << shift) - 1) : from;
      if (!(first && w == 0)) lo = from; else lo = 0;
      hi = first && w == (int)(range >> shift) ? ~0ull : to;
      if (lo >> 32 == hi >> 32) {              // one logit: ids below vocab
        const u64 most = (lo >> 32) << 32 | (uint64_t)(a.vocab - 1);
        if (hi > most) hi = most;
      }
      first = false;
      __syncthreads();
    }
    // those that are left, each against all
    if (tid == 0) s.n = 0;
    if (tid < FEW) {
      s.few_before[tid] = 0;
      s.few_rank[tid] = 0;
    }
    __syncthreads();
    each(bin, bin, [&](float v, uint32_t id, u64 m) {
      const u64 o = order_of(v, id);
      if (o < lo || o > hi) return;
      const uint32_t i = atomicAdd(&s.n, 1u);
      if (i < FEW) {
        s.few[i] = o;
        s.few_m[i] = m;
      }
    });
    __syncthreads();
    const int few = (int)(s.n < FEW ? s.n : FEW);
    int parts = THREADS / (few > 0 ? few : 1);
    parts = parts < 1 ? 1 : (parts > 64 ? 64 : parts);
    if (tid < few * parts) {
      const int i = tid % few, from = tid / few;
      const u64 mine = s.few[i];
      uint32_t rank = 0;
      u64 before = 0;
      for (int j = from; j < few; j += parts)
        if (s.few[j] < mine) {
          ++rank;
          before += s.few_m[j];
        }
      atomicAdd(&s.few_rank[i], rank);
      atomicAdd(&s.few_before[i], before);
    }
    __syncthreads();
    if (tid < few) {
      const uint32_t r = had + s.few_rank[tid];
      const u64 b = had_sum + s.few_before[tid], m = s.few_m[tid];
      if (count ? r + 1 == count : b < sum && sum <= b + m) s.got = {bin, r + 1, b + m, s.few[tid]};
    }
    __syncthreads();
    const Beginning got = s.got;
    __syncthreads();
    return got;
  }

  // the bin in which the running weight reaches g > 0, or passes g >= 0
  __device__ int reach(double g, bool pass) {
    if (tid < BINS) {
      const double b = s.before[tid], e = s.before[tid + 1];
      if (pass ? b <= g && g < e : b < g && g <= e) s.found = tid;
    }
    __syncthreads();
    const int d = s.found;
    __syncthreads();
    return d;
  }
  __device__ __forceinline__ double weight(const Beginning& b) const { return s.before[b.bin] + (double)b.sum * unit_of(b.bin); }

  __device__ void run(int64_t row) {
    top = -INFINITY;
    for (int i = tid; i < a.slices; i += THREADS) top = larger(a.tops[row * a.slices + i], top);
#pragma unroll
    for (int k = 32; k; k /= 2) top = larger(__shfl_xor(top, k), top);
    if ((tid & 63) == 0) s.wave_top[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < THREADS / 64; ++k) top = larger(s.wave_top[k], top);
    if (!(top > -INFINITY)) {                  // nothing is left
      if (tid == 0) {
        a.out[row] = -1;
        if (a.logprobs) a.logprobs[row] = -INFINITY;
      }
      return;
    }
    at = place_below(top, top, set.c);

    // the slices' histograms, each moved by its largest logit's distance
    {
      const int d = tid % BINS, part = tid / BINS;
      u64 sum = 0;
      uint32_t count = 0;
      for (int i = part; i < a.slices; i += THREADS / BINS) {
        const float t = a.tops[row * a.slices + i];
        if (!(t > -INFINITY)) continue;
        const Place p = place_below(t, top, set.c);
        const int from = d - bins_below(p.octave, p.quarter, at.octave, at.quarter);
        if (from < 0) continue;
        const u64 h = a.hist[(row * a.slices + i) * BINS + from];
        sum += h & ((1ull << COUNT_SHIFT) - 1);
        count += (uint32_t)(h >> COUNT_SHIFT);
      }
      s.part_sum[part][d] = sum;
      s.part_count[part][d] = count;
    }
    __syncthreads();
    if (tid < BINS) {
      s.sum[tid] = s.part_sum[0][tid] + s.part_sum[1][tid] + s.part_sum[2][tid] + s.part_sum[3][tid];
      s.count[tid] = s.part_count[0][tid] + s.part_count[1][tid] + s.part_count[2][tid] + s.part_count[3][tid];
    }
    __syncthreads();
    if (tid < 64) {                            // running weights and counts, four bins a lane
      double w[4], w4 = 0.0;
      uint32_t c[4], c4 = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = (double)s.sum[4 * tid + k] * unit_of(4 * tid + k);
        c[k] = s.count[4 * tid + k];
        w4 += w[k];
        c4 += c[k];
      }
      double ws = w4;
      uint32_t cs = c4;
#pragma unroll
      for (int k = 1; k < 64; k *= 2) {
        const double wu = __shfl_up(ws, k);
        const uint32_t cu = __shfl_up(cs, k);
        if (tid >= k) {
          ws += wu;
          cs += cu;
        }
      }
      double wb = __shfl_up(ws, 1);
      uint32_t cb = cs - c4;
      if (tid == 0) wb = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s.before[4 * tid + k] = wb < ws ? wb : ws;   // (rises from lane to lane, whatever the order of the sum)
        s.count_before[4 * tid + k] = cb;
        wb = k == 3 ? ws : wb + w[k];
        cb += c[k];
      }
      if (tid == 63) {
        s.before[BINS] = wb;
        s.count_before[BINS] = cb;
      }
    }
    if (tid == 0) {
      s.found = 0;
      s.got = {0, 0, 0, 0};
    }
    __syncthreads();

    const uint32_t tokens = s.count_before[BINS];
    const double all = s.before[BINS];
    const bool by_count = set.top_k > 0 && (uint32_t)set.top_k < tokens, by_weight = set.top_p < 1.0;
    // the least logit that min_p leaves, and its bin
    double least = -INFINITY;
    int least_bin = BINS;
    if (set.min_p > 0.0 && top < INFINITY) {
      least = (double)top + log2(set.min_p) / set.c;
      const Place p = place_of(least, set.c);
      if (set.c > 0.0) least_bin = bins_below(p.octave, p.quarter, at.octave, at.quarter);
    }

    // the last bin that is looked into, and its tokens and those of the bins before in a list
    int last = BINS - 1;
    if (by_count) {
      if (tid < BINS && s.count_before[tid] < (uint32_t)set.top_k && (uint32_t)set.top_k <= s.count_before[tid + 1]) s.found = tid;
      __syncthreads();
      last = s.found;
      __syncthreads();
    } else {
      if (by_weight) last = reach(set.top_p * all, false);
      if (least_bin < last) last = least_bin;
    }
    const int count_bin = last;
    listed = false;
    list_n = 0;
    if (s.count_before[last + 1] <= LIST) {
      if (tid == 0) s.n = 0;
      __syncthreads();
      each(0, last, [&](float v, uint32_t id, u64) {
        const uint32_t i = atomicAdd(&s.n, 1u);
        if (i < LIST) s.list[i] = order_of(v, id);
      });
      __syncthreads();
      listed = true;
      list_n = (int)(s.n < LIST ? s.n : LIST);
    }

    // (a beginning that ends in no bin of its own: all of them)
    Beginning kept = {BINS - 1, s.count[BINS - 1], s.sum[BINS - 1], 0};
    if (by_count) {
      const uint32_t c = (uint32_t)set.top_k - s.count_before[count_bin];
      kept = c < s.count[count_bin] ? select(count_bin, c, 0) : Beginning{count_bin, c, s.sum[count_bin], 0};
    }
    if (by_weight) {
      const double g = set.top_p * (by_count ? weight(kept) : all);
      int d = reach(g < all ? g : all, false);
      if (d > kept.bin) d = kept.bin;
      if (d <= last) {                         // (past it min_p leaves less)
        const u64 most = d == kept.bin ? kept.sum : s.sum[d];
        double need = ceil((g - s.before[d]) / unit_of(d));
        need = need < 1.0 ? 1.0 : need;
        if (need < (double)most) kept = select(d, 0, (u64)need);
        else if (d < kept.bin) kept = {d, s.count[d], s.sum[d], 0};
      }
    }
    if (least_bin < kept.bin || (least_bin == kept.bin && least_bin < BINS)) {
      if (tid == 0) {
        s.total_count = 0;
        s.total_sum = 0;
      }
      __syncthreads();
      uint32_t c = 0;
      u64 m = 0;
      each(least_bin, least_bin, [&](float v, uint32_t, u64 w) {
        if ((double)v >= least) {
          ++c;
          m += w;
        }
      });
      if (c) {
        atomicAdd(&s.total_count, c);
        atomicAdd(&s.total_sum, m);
      }
      __syncthreads();
      if (least_bin < kept.bin || s.total_count < kept.count) kept = {least_bin, s.total_count, s.total_sum, 0};
      __syncthreads();
    }

    // the token
    const double sum = weight(kept);
    double t = set.u * sum;
    const double end = sum * (1.0 - 0x1p-52);
    t = t < end ? t : end;
    int d = reach(t, true);
    if (d > kept.bin) d = kept.bin;
    const u64 most = d == kept.bin ? kept.sum : s.sum[d];
    double g = floor((t - s.before[d]) / unit_of(d)) + 1.0;
    g = g < 1.0 ? 1.0 : (g < (double)most ? g : (double)most);
    const Beginning got = select(d, 0, (u64)g);
    if (tid == 0) {
      const Place p = place_below(logit_of(got.last), top, set.c);
      a.out[row] = (int32_t)(uint32_t)got.last;
      if (a.logprobs) a.logprobs[row] = (float)log((double)p.m * unit_of(d) / sum);
    }
  }
};

template <class I>
__global__ __launch_bounds__(1024) void sample_choose_kernel(SampleArgs a) {
  __shared__ typename RowChoice<I>::Shared shared;
  const int64_t row = blockIdx.x;
  RowChoice<I> r{a, shared, (int)threadIdx.x, (const I*)a.x + row * a.x_stride, settings_of(a, row)};
  r.run(row);
}

template <class I>
hipError_t launch_i(const SampleArgs& a, int slice, hipStream_t st) {
  const dim3 grid((unsigned)a.slices, (unsigned)a.rows);
  hipError_t e;
  switch (slice) {
    case 4096: e = launch_kernel(sample_slice_kernel<I, 2>, grid, 512, 0, st, a); break;
    case 8192: e = launch_kernel(sample_slice_kernel<I, 4>, grid, 512, 0, st, a); break;
    default: e = launch_kernel(sample_slice_kernel<I, 8>, grid, 512, 0, st, a); break;
  }
  if (e != hipSuccess) return e;
  return launch_kernel(sample_choose_kernel<I>, dim3((unsigned)a.rows), 1024, 0, st, a);
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int slice, int dtype, hipStream_t st) {
  if (dtype == DT_F32) return launch_i<float>(a, slice, st);
  return dtype == DT_F16 ? launch_i<f16>(a, slice, st) : launch_i<bf16>(a, slice, st);
}

}  // namespace fcg
