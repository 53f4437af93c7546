// The choice of the next token of each row of logits.
//
//   w_v = 2^(c x_v - top), c = log2(e) / temperature;  order: x descending, ties by id
//   kept: the beginning of that order that top_k, top_p and min_p leave
//   the first of the kept whose running sum of w passes u times the sum of the kept
//
// No row is sorted.  A token's weight is a whole number: with z = 4 c x (f64) and
// q the nearest whole number, M = 2^((z - q) / 4) 2^33, rounded.  Each q is a bin
// of a histogram: the bins stand in the order of x and do not depend on the row's
// largest, so that slices of a row are summed apart and joined later, and sums of
// whole numbers do not depend on their order.  Running sums say in which bins
// top_k, top_p, min_p and u end; only the tokens of those bins, or of the bins up
// to the last of them, are looked at again.
// (M is off by 2^-33 of itself: against sums of f64 a border moves by about
// 10^-10 of the sum, the rounding of u to f32 by 6 * 10^-8.)
//
// Tokens 256 bins and more below the largest, 63.75 octaves at least, weigh less
// than 2^-39.75 together (vocab <= 2^24) and are never chosen; they are dropped
// from the histogram.
//
// Two launches: slices of rows over the whole card, then a workgroup for each
// row.  A slice also writes down its first tokens, so that a row whose kept
// tokens are few, as they mostly are, is not read again.  Where it has to be,
// for the bins in which something ends, the workgroups that the rows leave idle
// read parts of it, and the one that is done last goes on with what they found.
//
// Measured, kernels alone: a row of 32064 with top_k, top_p and min_p 4.8 us and
// 11.3; 128 rows of 131073 f32 with top_p 24.0 and 18.9, where 67 MB are read
// once (2.8 TB/s) by 24 us of which reading is 13, weights and additions in LDS 6
// and first tokens 5; 33 rows of 131073 bf16, nearly flat, three quarters hidden
// 11.3 and 34.2, where the rows are read again.  The second kernel is bound by latency:
// joining 17 histograms, running sums, ranks, each behind a barrier.
// Both launches of a row of 131073 f32 (deviation 2.5, temperature 0.8): greedy 15
// us, top_k of 50 and top_p 18, temperature alone 28, top_p alone 35, for which the
// row is read again.
// Rows whose ends fall in bins of more than LIST tokens are read by one workgroup
// several times: 131073 logits about 0 with a deviation of 0.1 145 us, with top_p
// 211; 131073 equal ones 370 and 727.
#include <math.h>

#include "serving.h"

namespace fcg {
namespace {

typedef unsigned long long u64;

constexpr int BINS = SAMPLE_BINS;
constexpr int COUNT_SHIFT = 49;                // a slice's bin: the sum of M below, the count of tokens from here on
constexpr int SLICE_MOST = 16384;              // (2^14 tokens of less than 2^34 would be 2^48)
constexpr int FIRST = SAMPLE_FIRST;            // tokens that a slice writes down, at most
constexpr int FIRST_WANTED = FIRST - 16;
constexpr int LIST = 4096;                     // tokens that are looked at from LDS
constexpr int PART = SAMPLE_PART;              // of those that a workgroup of a row hands over
constexpr int FEW = 512;                       // tokens of a row that are ranked against each other at once,
constexpr int FEW_OF_BIN = 128;                // and of a bin, with their sums (each against all: 10 us for 512)

// N values at an address aligned to one of them
template <class T, int N> struct Some { typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T)))); };

// Where a logit stands.  (No contraction: a token has the same place wherever it
// is computed.)
struct Place {
  double q;              // bins fall with it
  u64 m;
};
// 2^33 2^(g / 4) for g from -1/2 to 1/2: a polynomial of degree 5, of itself off by
// -3.84 to 0.14 * 10^-11 (2^-34.6) with these coefficients, and 2^52, which leaves a
// whole number in the fraction's bits.  With that rounding M is off by 2^-33.1 at most.
struct Weigher {
  double c0 = 4503599627370496.0 + 8589934592.0, c1 = 8589934592.0 * 0.17328679512681341, c2 = 8589934592.0 * 0.015014155364465376,
         c3 = 8589934592.0 * 0.0008672518832954696, c4 = 8589934592.0 * 3.758491381301949e-05,
         c5 = 8589934592.0 * 1.3017562230028637e-06;
  // (in scalar registers: as literals they were moved to vector registers for every token, 10 instructions of 28)
  __device__ __forceinline__ void keep() {
    asm("" : "+s"(c0), "+s"(c1), "+s"(c2), "+s"(c3), "+s"(c4), "+s"(c5));
  }
  __device__ __forceinline__ u64 operator()(double g) const {
    double y = __builtin_fma(g, c5, c4);
    y = __builtin_fma(y, g, c3);
    y = __builtin_fma(y, g, c2);
    y = __builtin_fma(y, g, c1);
    y = __builtin_fma(y, g, c0);
    return __builtin_bit_cast(u64, y) & 0xFFFFFFFFFFFFFull;
  }
};
__device__ __forceinline__ Place place_of(double x, double c4, const Weigher& weigh) {
#pragma clang fp contract(off)
  const double z = x * c4, q = __builtin_rint(z), g = z - q;        // (exact)
  return {q, weigh(g)};
}
__device__ __forceinline__ double q_of(float x, double c4) {
#pragma clang fp contract(off)
  return __builtin_rint((double)x * c4);
}
// An infinite logit has all the weight, and shares it with its like: then its
// place is the top, and no other logit has one.
__device__ __forceinline__ Place place_below(float x, float top, double c4) {
  if (top == INFINITY) return {x == INFINITY ? 0.0 : -INFINITY, 1ull << 33};
  return place_of((double)x, c4, Weigher());
}
__device__ __forceinline__ double q_below(float x, float top, double c4) {
  if (top == INFINITY) return x == INFINITY ? 0.0 : -INFINITY;
  return q_of(x, c4);
}
// the bin of a place, BINS where it has none
__device__ __forceinline__ int bin_below(double q, double top_q) {
  const double d = top_q - q;
  return d < BINS ? (int)d : BINS;
}

// A bound of the logits of bins: all of bins up to `bin` are at least `out`, and
// those from `in` on are of these bins.  c4 is at least 10^-300.
struct Bound {
  float out, in;
};
__device__ __forceinline__ Bound lowest_of(int bin, float top, double top_q, double c4) {
  if (top == INFINITY) return {INFINITY, INFINITY};
  const double y = (top_q - bin - 0.5) / c4, e = fabs(y) * 1e-6;
  return {(float)(y - e), (float)(y + e)};
}

struct Settings {
  double c4;             // 4 log2(e) / temperature
  int top_k;             // 0: all
  double top_p, min_p, u;
};
__device__ __forceinline__ double c4_of(const SampleArgs& a, int64_t row) {
  const float t = a.temperature ? a.temperature[row] : 1.f;
  const double c4 = 4 * 1.44269504088896340736 / (t > 0.f ? (double)t : 1.0);
  return c4 > 1e-300 ? c4 : 1e-300;            // (of an infinite temperature: not 0 times -inf)
}
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t row) {
  Settings s;
  const float t = a.temperature ? a.temperature[row] : 1.f;
  s.c4 = c4_of(a, row);
  s.top_k = a.top_k ? a.top_k[row] : 0;
  s.top_p = a.top_p ? (double)a.top_p[row] : 1.0;
  s.min_p = a.min_p ? (double)a.min_p[row] : 0.0;
  s.u = (double)a.u[row];
  if (s.top_k < 0) s.top_k = 0;
  if (!(s.top_p < 1.0)) s.top_p = 1.0;
  if (!(t > 0.f) || s.top_p <= 0.0 || s.min_p > 1.0) s.top_k = 1;
  if (t == INFINITY) s.min_p = 0.0;            // (all finite logits weigh 1, however far below the top)
  if (s.top_k == 1) {
    s.top_p = 1.0;
    s.min_p = 0.0;
  }
  s.u = s.u > 0.0 ? s.u : 0.0;                 // (NaN too)
  return s;
}

// whether something but u ends the row's kept tokens: only then are the first ones of use
__device__ __forceinline__ bool ends_early(const SampleArgs& a, int64_t row) {
  return (a.temperature && !(a.temperature[row] > 0.f)) || (a.top_k && a.top_k[row] > 0) || (a.top_p && a.top_p[row] < 1.f) ||
         (a.min_p && a.min_p[row] > 0.f);
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

// The sum over this lane and those before it, by moves between lanes.
__device__ __forceinline__ uint32_t running_sum(uint32_t x) {
  x += __builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false);    // rows of 16 lanes: from 1, 2, 4 and 8 lanes before
  x += __builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);    // to rows 1 and 3 from the row before,
  x += __builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);    // to rows 2 and 3 from row 1
  return x;
}

__device__ __forceinline__ float larger(float a, float b) { return a > b ? a : b; }

// What a row's slice holds: the histogram of its tokens below its largest logit,
// and its first tokens, those of its first bins while they are FIRST_WANTED at most.
template <class I, int ROUNDS>
__global__ __launch_bounds__(512) void sample_slice_kernel(SampleArgs a) {
  constexpr int THREADS = 512, SLICE = THREADS * 4 * ROUNDS;
  static_assert(SLICE <= SLICE_MOST, "sums");
  __shared__ u64 hist[BINS];
  __shared__ float wave_top[THREADS / 64];
  __shared__ uint32_t first_n;
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
  const double c4 = c4_of(a, row);
  if (tid < BINS) hist[tid] = 0;
  if (tid == 0) first_n = 0;
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4 * ROUNDS; ++k) {
    z[k] = fmaxf(z[k], -INFINITY);             // NaN takes no part
    top = fmaxf(top, z[k]);
  }
#pragma unroll
  for (int k = 32; k; k /= 2) top = larger(__shfl_xor(top, k), top);
  if ((tid & 63) == 0) wave_top[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < THREADS / 64; ++k) top = larger(wave_top[k], top);
  const double top_q = q_below(top, top, c4);
  Weigher weigh;
  weigh.keep();
  if (top < INFINITY) {
    // (a place of -inf, and no top at all, convert to the largest number: none)
#pragma unroll
    for (int k = 0; k < 4 * ROUNDS; ++k) {
      const Place p = place_of((double)z[k], c4, weigh);
      const double d = top_q - p.q;
      if (d < BINS) atomicAdd(&hist[(int)d], p.m | 1ull << COUNT_SHIFT);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4 * ROUNDS; ++k)
      if (z[k] == INFINITY) atomicAdd(&hist[0], 1ull << 33 | 1ull << COUNT_SHIFT);
  }
  __syncthreads();
  const int64_t slice = row * a.slices + blockIdx.x;
  if (tid < BINS) a.hist[slice * BINS + tid] = hist[tid];
  // bins whose tokens are FIRST_WANTED at most, from the top on (every wave for itself)
  const bool of_use = ends_early(a, row);
  int bins = 0;
  if (of_use) {
    const int lane = tid & 63;
    uint32_t c[4], all4 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] = (uint32_t)(hist[4 * lane + k] >> COUNT_SHIFT);
      all4 += c[k];
    }
    uint32_t upto = running_sum(all4) - all4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      upto += c[k];
      bins += __builtin_popcountll(__ballot(upto <= (uint32_t)FIRST_WANTED));
    }
  }
  // What is below the bound of these bins is not in them; a few others that are
  // not may be written down too, while there is room.
  float low = INFINITY;
  if (bins > 0 && top > -INFINITY) low = fmaxf(lowest_of(bins - 1, top, top_q, c4).out, -3.4028234663852886e38f);
  if (bins > 0) {
    // (a place for all of a wave's at once; one for each token cost 5 us of 29 for 128 rows of 131073)
    u64 those[4 * ROUNDS];
    uint32_t many = 0;
#pragma unroll
    for (int k = 0; k < 4 * ROUNDS; ++k) {
      those[k] = __ballot(z[k] >= low);
      many += __builtin_popcountll(those[k]);
    }
    uint32_t at = 0;
    if ((tid & 63) == 0) at = atomicAdd(&first_n, many);
    at = __builtin_amdgcn_readfirstlane(at);
    uint2* first = a.first + slice * FIRST;
    const uint32_t id = (uint32_t)v0 + tid * 4;
    if (at + many <= (uint32_t)FIRST)
#pragma unroll
      for (int k = 0; k < 4 * ROUNDS; ++k)
        if (those[k]) {
          const uint32_t i = __builtin_amdgcn_mbcnt_hi((uint32_t)(those[k] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)those[k], at));
          if (__builtin_amdgcn_inverse_ballot_w64(those[k]))
            first[i] = make_uint2(__builtin_bit_cast(uint32_t, z[k]), id + k / 4 * THREADS * 4 + k % 4);
          at += __builtin_popcountll(those[k]);
        }
  }
  __syncthreads();
  if (tid == 0) {
    if (blockIdx.x == 0) a.arrived[row] = 0;
    const uint32_t n = first_n;
    a.slice_tops[slice] = n <= (uint32_t)FIRST ? SliceTop{top, (uint16_t)bins, (uint16_t)n} : SliceTop{top, 0, 0};
  }
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
  static constexpr int KNOWN = 64;             // slices whose places are kept in LDS
  static constexpr int AHEAD = 2;              // first tokens that a thread asks for before it knows whether they matter
  struct Shared {
    u64 sum[BINS];
    uint32_t count[BINS];
    double before[BINS + 1];                   // weight of the bins before, in units of M of the top bin
    uint32_t count_before[BINS + 1];
    u64 part_sum[BINS];                        // histogram of a bin's tokens
    uint32_t part_count[BINS];
    int its_bin[KNOWN];                        // of the slices: the bin of their largest logit,
    int its_end[KNOWN];                        // the first bin whose tokens they did not write down,
    int its_n[KNOWN];                          // and how many they wrote
    u64 few[FEW], few_m[FEW_OF_BIN], few_before[FEW_OF_BIN];
    uint32_t few_rank[FEW];
    float wave_top[THREADS / 64];
    uint32_t n;                                // tokens of a list
    uint32_t arrived;
    uint32_t part_n[SAMPLE_MOST_PARTS];
    int found;
    Beginning got;
    u64 total_sum;
    uint32_t total_count;
    u64 list[LIST];
  };

  const SampleArgs& a;
  Shared& s;
  const int tid;
  const int64_t row;
  const I* x;
  Settings set;
  float top;
  double top_q;          // of the largest logit
  int list_n;            // tokens of the list
  int list_from[2], list_to[2];   // the bins that it holds: two stretches
  uint2 ahead[AHEAD];

  // bin of a token, BINS: of none
  __device__ __forceinline__ int bin_of(float v, u64& m) const {
    const Place p = place_below(v, top, set.c4);
    m = p.m;
    return bin_below(p.q, top_q);
  }
  // of a bin's M against the top bin's: 2^(-bin / 4)
  __device__ __forceinline__ double unit_of(int bin) const {
    const int r = bin & 3;
    const double y = r == 0 ? 1.0 : r == 1 ? 0.84089641525371454303 : r == 2 ? 0.70710678118654752440 : 0.59460355750136053336;
    return __builtin_ldexp(y, -(bin >> 2));
  }

  // f(x, id) of the tokens of a stretch of the row whose logits are at least
  // `low`, 16 bytes a thread and load
  template <class F>
  __device__ __forceinline__ void each_above(int64_t from, int64_t to, float low, F f) {
    constexpr int V = 16 / sizeof(I);
    typedef typename Some<I, V>::vec IV;
    const int n = (int)(to - from), whole = n / V * V;
    const I* p = x + from;
#pragma unroll 4
    for (int i = tid * V; i < whole; i += THREADS * V) {
      const IV y = *(const IV*)(p + i);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float v = (float)y[e];
        if (v >= low && v > -INFINITY) f(v, (uint32_t)(from + i + e));
      }
    }
    if (tid < n - whole) {
      const float v = (float)p[whole + tid];
      if (v >= low && v > -INFINITY) f(v, (uint32_t)(from + whole + tid));
    }
  }

  // Of a slice: the bin of its largest logit (BINS: it has none that matters),
  // and the first bin whose tokens it did not write down.
  __device__ __forceinline__ void slice_bins(int i, int& bin, int& end, int& n) const {
    if (i < KNOWN) {
      bin = s.its_bin[i];
      end = s.its_end[i];
      n = s.its_n[i];
      return;
    }
    const SliceTop t = a.slice_tops[row * a.slices + i];
    bin = t.top > -INFINITY ? bin_below(q_below(t.top, top, set.c4), top_q) : BINS;
    end = bin + t.bins;
    n = t.n;
  }

  // The list: all tokens of bins from .. to, LIST at most.
  __device__ __forceinline__ void gather(int from, int to) {
    __syncthreads();
    if (tid == 0) s.n = 0;
    __syncthreads();
    auto take = [&](u64 order) {
      const uint32_t i = atomicAdd(&s.n, 1u);
      if (i < (uint32_t)LIST) s.list[i] = order;
    };
    // slices that wrote them all down
    constexpr int AT_ONCE = THREADS / FIRST;
    auto look = [&](int i, uint2 o) {
      const float v = __builtin_bit_cast(float, o.x);
      const int d = bin_below(q_below(v, top, set.c4), top_q);
      if (d >= from && d <= to) take(order_of(v, o.y));
    };
    int bin, end, many;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = tid / FIRST + k * AT_ONCE;
      if (i >= a.slices) break;
      slice_bins(i, bin, end, many);
      if (bin <= to && end > to && tid % FIRST < many) look(i, ahead[k]);
    }
    for (int i = tid / FIRST + AHEAD * AT_ONCE; i < a.slices; i += AT_ONCE) {
      slice_bins(i, bin, end, many);
      if (bin <= to && end > to && tid % FIRST < many) look(i, a.first[(row * a.slices + i) * FIRST + tid % FIRST]);
    }
    // the others, those next to each other as one stretch: nearly all tokens are told by two comparisons
    const Bound low = lowest_of(to, top, top_q, set.c4);
    const Bound high = from == 0 ? Bound{INFINITY, INFINITY} : lowest_of(from - 1, top, top_q, set.c4);
    for (int i0 = 0; i0 < a.slices; i0 += 64) {
      bool read = false;
      if (i0 + (tid & 63) < a.slices) {
        slice_bins(i0 + (tid & 63), bin, end, many);
        read = bin <= to && end <= to;
      }
      for (u64 left = __ballot(read); left;) {
        const int i = __builtin_ctzll(left);
        const u64 gap = ~(left >> i);          // (its first bit is the first after the stretch)
        const int n = gap ? __builtin_ctzll(gap) : 64;
        left = n + i < 64 ? left >> (n + i) << (n + i) : 0;
        const int64_t v0 = (int64_t)(i0 + i) * a.slice, v1 = v0 + (int64_t)n * a.slice;
        each_above(v0, v1 < a.vocab ? v1 : a.vocab, low.out, [&](float v, uint32_t id) {
          if (v > high.in) return;
          if (!(v >= low.in && (from == 0 || v < high.out))) {
            const int d = bin_below(q_below(v, top, set.c4), top_q);
            if (d < from || d > to) return;
          }
          take(order_of(v, id));
        });
      }
    }
    __syncthreads();
    list_n = (int)(s.n < (uint32_t)LIST ? s.n : (uint32_t)LIST);
    hold(from, to, 0, -1);
  }
  __device__ __forceinline__ void hold(int from, int to, int from2, int to2) {
    list_from[0] = from;
    list_to[0] = to;
    list_from[1] = from2;
    list_to[1] = to2;
  }
  __device__ __forceinline__ bool holds(int bin) const {
    return (list_from[0] <= bin && bin <= list_to[0]) || (list_from[1] <= bin && bin <= list_to[1]);
  }

  // whether the slices wrote down all tokens of bins up to `to`
  __device__ __forceinline__ bool written(int to) const {
    bool read = false;
    for (int i = tid & 63; i < a.slices; i += 64) {
      int bin, end, many;
      slice_bins(i, bin, end, many);
      read = read || (bin <= to && end <= to);
    }
    return !__any(read);
  }

  // The list of two stretches of bins, [from, to] before [from2, to2] (the latter
  // may be empty), each workgroup of the row reading a part of it: true in the one
  // that has the whole list, the last to be done.
  __device__ __forceinline__ bool gather_parts(int from, int to, int from2, int to2) {
    const int parts = gridDim.x, part = blockIdx.x;
    __syncthreads();
    if (tid == 0) s.n = 0;
    __syncthreads();
    const float low = lowest_of(to, top, top_q, set.c4).out, high = from == 0 ? INFINITY : lowest_of(from - 1, top, top_q, set.c4).in;
    const float low2 = to2 < from2 ? INFINITY : lowest_of(to2, top, top_q, set.c4).out;
    const float high2 = to2 < from2 ? -INFINITY : lowest_of(from2 - 1, top, top_q, set.c4).in;
    const int64_t each = ((a.vocab + parts - 1) / parts + 7) / 8 * 8, v0 = part * each, v1 = v0 + each;
    if (v0 < a.vocab)
      each_above(v0, v1 < a.vocab ? v1 : a.vocab, low < low2 ? low : low2, [&](float v, uint32_t id) {
        if (!((v >= low && v <= high) || (v >= low2 && v <= high2))) return;
        const int d = bin_below(q_below(v, top, set.c4), top_q);
        if (!((d >= from && d <= to) || (d >= from2 && d <= to2))) return;
        const uint32_t i = atomicAdd(&s.n, 1u);
        if (i < (uint32_t)LIST) s.list[i] = order_of(v, id);
      });
    __syncthreads();
    list_n = (int)s.n;
    if (parts > 1) {
      // handed over by stores and loads past the XCDs' caches; a part that found more than there is room for says so
      u64* mine = a.parts + (row * parts + part) * PART;
      for (int i = tid; i < list_n && i < PART; i += THREADS) __hip_atomic_store(mine + i, s.list[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (tid == 0) __hip_atomic_store(a.part_n + row * parts + part, (uint32_t)list_n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0) s.arrived = __hip_atomic_fetch_add(a.arrived + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      if (s.arrived != (uint32_t)parts - 1) return false;
      if (tid < parts) s.part_n[tid] = __hip_atomic_load(a.part_n + row * parts + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      for (int k = 0; k < parts; ++k) {
        const int n = (int)s.part_n[k];
        if (n > PART || (k != part && list_n + n > LIST)) {       // (bins will be gathered one by one)
          hold(0, -1, 0, -1);
          return true;
        }
        if (k == part) continue;
        const u64* its = a.parts + (row * parts + k) * PART;
        for (int i = tid; i < n; i += THREADS) s.list[list_n + i] = __hip_atomic_load(its + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        list_n += n;
      }
      __syncthreads();
    }
    hold(from, to, from2, to2);
    return true;
  }

  // f(x, id, M) of every token of a bin: from the list, into which its tokens go
  // if they fit it, or from the row, where those whose place in the order is
  // outside [lo, hi] may be passed over (their bin and M take 30 instructions)
  template <class F>
  __device__ __forceinline__ void each_of(int bin, u64 lo, u64 hi, F f) {
    if (holds(bin)) {
      for (int i = tid; i < list_n; i += THREADS) {
        const u64 o = s.list[i];
        u64 m;
        const float v = logit_of(o);
        if (bin_of(v, m) == bin) f(v, (uint32_t)o, m);
      }
      return;
    }
    // (an end of the order that no logit has is a NaN, which fmaxf and fminf leave out)
    const float low = fmaxf(lowest_of(bin, top, top_q, set.c4).out, logit_of(hi));
    const float high = fminf(bin == 0 ? INFINITY : lowest_of(bin - 1, top, top_q, set.c4).in, logit_of(lo));
    each_above(0, a.vocab, low, [&](float v, uint32_t id) {
      u64 m;
      if (v <= high && bin_of(v, m) == bin) f(v, id, m);
    });
  }
  __device__ __forceinline__ void see_to(int bin) {
    if (!holds(bin) && s.count[bin] <= LIST) gather(bin, bin);
  }

  // Ranks `few` tokens of s.few against each other: how many are before each, and, of SUMS, their M.
  template <bool SUMS>
  __device__ __forceinline__ void rank(int few) {
    int parts = THREADS / (few > 0 ? few : 1);
    parts = parts < 1 ? 1 : (parts > 64 ? 64 : parts);
    if (tid < few * parts) {
      const int i = tid % few, each = (few + parts - 1) / parts, from = tid / few * each, to = from + each < few ? from + each : few;
      const u64 mine = s.few[i];
      uint32_t r = 0;
      u64 before = 0;
#pragma unroll 8
      for (int j = from; j < to; ++j) {
        const bool b = s.few[j] < mine;
        r += b;
        if constexpr (SUMS) {
          const u64 m = s.few_m[j];
          before += b ? m : 0;
        }
      }
      if (r) atomicAdd(&s.few_rank[i], r);
      if constexpr (SUMS)
        if (before) atomicAdd(&s.few_before[i], before);
    }
  }

  // The beginning of a bin that ends with its token `count` (where it is not
  // 0), or with the first whose running sum is `sum` or more.
  __device__ __forceinline__ Beginning select(int bin, uint32_t count, u64 sum) {
    see_to(bin);
    uint32_t had = 0, n = s.count[bin];        // tokens before those that are left, and how many these are
    u64 had_sum = 0, lo = 0, hi = ~0ull;       // sum before them, and their range
    if (n > FEW_OF_BIN && top < INFINITY) {           // (at first all that is outside a narrower range goes to its ends)
      hi = order_of(lowest_of(bin, top, top_q, set.c4).out, ~0u);
      lo = order_of(lowest_of(bin - 1, top, top_q, set.c4).in, 0);
    }
    bool first = true;
    while (n > FEW_OF_BIN) {
      // 256 ways
      const u64 range = hi - lo;
      const int bits = 64 - __builtin_clzll(range | 1), shift = bits > 8 ? bits - 8 : 0;
      __syncthreads();
      if (tid < BINS) {
        s.part_sum[tid] = 0;
        s.part_count[tid] = 0;
      }
      __syncthreads();
      // A thread adds up while the way stays the same: 131073 equal logits went to one
      // counter one by one, 250 us a pass.
      int way = 0;
      u64 way_sum = 0;
      uint32_t way_count = 0;
      auto put = [&]() {
        if (!way_count) return;
        atomicAdd(&s.part_sum[way], way_sum);
        atomicAdd(&s.part_count[way], way_count);
        way_sum = 0;
        way_count = 0;
      };
      each_of(bin, first ? 0 : lo, first ? ~0ull : hi, [&](float v, uint32_t id, u64 m) {
        const u64 o = order_of(v, id);
        if (!first && (o < lo || o > hi)) return;
        const int w = o < lo ? 0 : o > hi ? (int)(range >> shift) : (int)((o - lo) >> shift);
        if (w != way) put();
        way = w;
        way_sum += m;
        ++way_count;
      });
      put();
      __syncthreads();
      if (tid < 64) {
        // running sums, four ways a lane
        uint32_t c4 = 0;
        u64 s4 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c4 += s.part_count[4 * tid + k];
          s4 += s.part_sum[4 * tid + k];
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
          const uint32_t cn = s.part_count[4 * tid + k];
          const u64 sn = s.part_sum[4 * tid + k];
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
      n = s.part_count[w];
      // (at first the ends hold what is outside the range too)
      const u64 from = lo + ((u64)w << shift), to = shift ? from + (((u64)1 << shift) - 1) : from;
      lo = first && w == 0 ? 0 : from;
      hi = first && w == (int)(range >> shift) ? ~0ull : to < hi ? to : hi;   // (the last way may reach past the range)
      if (lo >> 32 == hi >> 32) {              // one logit: ids below vocab
        const u64 most = (lo >> 32) << 32 | (uint64_t)(a.vocab - 1);
        if (hi > most) hi = most;
      }
      first = false;
    }
    // those that are left, each against all
    __syncthreads();
    if (tid == 0) s.n = 0;
    if (tid < FEW_OF_BIN) {
      s.few_before[tid] = 0;
      s.few_rank[tid] = 0;
    }
    __syncthreads();
    each_of(bin, lo, hi, [&](float v, uint32_t id, u64 m) {
      const u64 o = order_of(v, id);
      if (o < lo || o > hi) return;
      const uint32_t i = atomicAdd(&s.n, 1u);
      if (i < (uint32_t)FEW_OF_BIN) {
        s.few[i] = o;
        s.few_m[i] = m;
      }
    });
    __syncthreads();
    const int few = (int)(s.n < (uint32_t)FEW_OF_BIN ? s.n : (uint32_t)FEW_OF_BIN);
    rank<true>(few);
    __syncthreads();
    if (tid < few) {
      const uint32_t r = had + s.few_rank[tid];
      const u64 b = had_sum + s.few_before[tid], m = s.few_m[tid];
      if (count ? r + 1 == count : b < sum && sum <= b + m) s.got = {bin, r + 1, b + m, s.few[tid]};
    }
    __syncthreads();
    return s.got;
  }

  // the bin in which the running weight reaches g > 0, or passes g >= 0
  __device__ __forceinline__ int reach(double g, bool pass) {
    __syncthreads();
    if (tid < BINS) {
      const double b = s.before[tid], e = s.before[tid + 1];
      if (pass ? b <= g && g < e : b < g && g <= e) s.found = tid;
    }
    __syncthreads();
    return s.found;
  }
  __device__ __forceinline__ double weight(const Beginning& b) const { return s.before[b.bin] + (double)b.sum * unit_of(b.bin); }

  __device__ __forceinline__ void answer(u64 order, double weight, double sum) const {
    a.out[row] = (int32_t)(uint32_t)order;
    if (a.logprobs) a.logprobs[row] = (float)log(weight / sum);
  }

  // The choice where all tokens up to the last bin that matters are few: they
  // are ranked at once, and one wave sums their weights, 8 tokens a lane.
  __device__ __forceinline__ void choose_of_few(bool by_count, bool by_weight, double least, double all) {
    const int n = list_n;
    if (tid < n) {
      s.few_rank[tid] = 0;
      s.few[tid] = s.list[tid];
    }
    __syncthreads();
    rank<false>(n);
    __syncthreads();
    if (tid < n) s.list[FEW + s.few_rank[tid]] = s.few[tid];         // (in order)
    __syncthreads();
    if (tid >= 64) return;
    constexpr int EACH = FEW / 64;
    double w[EACH], e[EACH], mine = 0.0;       // weights, sums before
    float v[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = tid * EACH + k;
      w[k] = 0.0;
      v[k] = -INFINITY;
      if (i < n) {
        u64 m;
        v[k] = logit_of(s.list[FEW + i]);
        const int d = bin_of(v[k], m);
        w[k] = (double)m * unit_of(d);
      }
      mine += w[k];
    }
    double upto = mine;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
      const double up = __shfl_up(upto, k);
      if (tid >= k) upto += up;
    }
    double before = __shfl_up(upto, 1);
    if (tid == 0) before = 0.0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      e[k] = before < upto ? before : upto;    // (rises from lane to lane)
      before += w[k];
    }
    auto count_of = [&](auto holds) {          // tokens for which it holds
      int c = 0;
#pragma unroll
      for (int k = 0; k < EACH; ++k) c += __builtin_popcountll(__ballot(tid * EACH + k < n && holds(k)));
      return c;
    };
    auto before_token = [&](int i) {           // sum before token i, of all n where i is n
      double y = 0.0;
#pragma unroll
      for (int k = 0; k < EACH; ++k)
        if (k == i % EACH) y = e[k];
      const double last = __shfl(upto, 63);
      return i < n ? __shfl(y, i / EACH) : last;
    };
    int kept = n;
    if (by_count && set.top_k < kept) kept = set.top_k;
    if (by_weight) {
      const double g = set.top_p * (by_count ? before_token(kept) : all);
      const int c = count_of([&](int k) { return e[k] < g; });
      kept = c < kept ? c : kept;
    }
    const int c = count_of([&](int k) { return (double)v[k] >= least; });
    kept = c < kept ? c : kept;
    kept = kept < 1 ? 1 : kept;
    const double sum = before_token(kept), end = sum * (1.0 - 0x1p-52);
    double t = set.u * sum;
    t = t < end ? t : end;
    const int at = count_of([&](int k) { return e[k] <= t && tid * EACH + k < kept; }) - 1;
    double weight = 0.0;
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (k == at % EACH) weight = w[k];
    if (tid == at / EACH) answer(s.list[FEW + at], weight, sum);
  }

  __device__ __forceinline__ void run() {
    // All that is small is asked for before any of it is looked at.  A thread has
    // a bin of every fourth slice.
    constexpr int PARTS = THREADS / BINS, EACH = 4;
    u64 h[EACH];
    const SliceTop none = {-INFINITY, 0, 0};
    const SliceTop mine = tid < a.slices ? a.slice_tops[row * a.slices + tid] : none;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = tid / BINS + k * PARTS;
      h[k] = i < a.slices ? a.hist[(row * a.slices + i) * BINS + tid % BINS] : 0;
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = tid / FIRST + k * (THREADS / FIRST);
      ahead[k] = i < a.slices ? a.first[(row * a.slices + i) * FIRST + tid % FIRST] : make_uint2(0, 0);
    }
    set = settings_of(a, row);
    if (tid < BINS) {
      s.sum[tid] = 0;
      s.count[tid] = 0;
    }
    top = mine.top;
    for (int i = tid + THREADS; i < a.slices; i += THREADS) top = larger(a.slice_tops[row * a.slices + i].top, top);
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
    top_q = q_below(top, top, set.c4);
    if (tid < KNOWN) {
      const int bin = mine.top > -INFINITY ? bin_below(q_below(mine.top, top, set.c4), top_q) : BINS;
      s.its_bin[tid] = bin;
      s.its_end[tid] = bin + mine.bins;
      s.its_n[tid] = mine.n;
    }
    __syncthreads();

    // the slices' histograms, each moved by its largest logit's distance
    auto join = [&](int i, u64 h) {
      int bin, end, n;
      slice_bins(i, bin, end, n);
      const int d = tid % BINS + bin;
      if (h == 0 || d >= BINS) return;
      atomicAdd(&s.sum[d], h & ((1ull << COUNT_SHIFT) - 1));
      atomicAdd(&s.count[d], (uint32_t)(h >> COUNT_SHIFT));
    };
#pragma unroll
    for (int k = 0; k < EACH; ++k)
      if (tid / BINS + k * PARTS < a.slices) join(tid / BINS + k * PARTS, h[k]);
    for (int i = tid / BINS + EACH * PARTS; i < a.slices; i += PARTS) join(i, a.hist[(row * a.slices + i) * BINS + tid % BINS]);
    __syncthreads();
    if (tid < 64) {                            // running weights and counts, four bins a lane
      double w[4], w4 = 0.0;
      uint32_t c[4], c4 = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int d = 4 * tid + k;
        c[k] = s.count[d];
        w[k] = (double)s.sum[d] * unit_of(d);
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
      least = (double)top + 4 * log2(set.min_p) / set.c4;
      least_bin = bin_below(place_of(least, set.c4, Weigher()).q, top_q);
    }

    // the last bin that matters; the tokens up to it in a list
    int last = BINS - 1;
    if (by_count) {
      if (tid < BINS && s.count_before[tid] < (uint32_t)set.top_k && (uint32_t)set.top_k <= s.count_before[tid + 1]) s.found = tid;
      __syncthreads();
      last = s.found;
    } else {
      if (by_weight) last = reach(set.top_p * all, false);
      if (least_bin < last) last = least_bin;
    }
    list_n = 0;
    hold(0, -1, 0, -1);
    const uint32_t upto = s.count_before[last + 1];
    const bool in_slices = upto <= (uint32_t)LIST && written(last);
    if (in_slices) {
      if (blockIdx.x) return;
      gather(0, last);
    }
    if (upto <= (uint32_t)FEW) {
      if (!in_slices && !gather_parts(0, last, 0, -1)) return;
      if (!holds(last)) gather(0, last);
      choose_of_few(by_count, by_weight, least, all);
      return;
    }

    // The bins in which something ends, [b0, b1], and with them the range of the
    // kept weight, [least_sum, most_sum], and so of the bin of the token, [t0, t1].
    const int count_bin = last;
    bool for_count = by_count, for_weight = by_weight;
    int b0 = BINS, b1 = -1, end_bin = BINS - 1;
    double least_sum = all, most_sum = all;
    if (by_count) {
      b0 = b1 = end_bin = count_bin;
      least_sum = s.before[count_bin];
      most_sum = s.before[count_bin + 1];
    }
    if (by_weight) {
      const double g0 = set.top_p * least_sum, g1 = set.top_p * most_sum;
      int d0 = reach(g0 > 1e-300 ? g0 : 1e-300, false), d1 = reach(g1, false);
      d0 = d0 < end_bin ? d0 : end_bin;
      d1 = d1 < end_bin ? d1 : end_bin;
      b0 = d0 < b0 ? d0 : b0;
      b1 = d1 > b1 ? d1 : b1;
      end_bin = d1;
      least_sum = g0;
      most_sum = most_sum < s.before[d1 + 1] ? most_sum : s.before[d1 + 1];
    }
    const bool for_least = least_bin <= end_bin;
    if (for_least) {
      if (least_bin < b0) {                    // it leaves less than the others, wherever these end
        for_count = for_weight = false;
        b0 = b1 = least_bin;
      }
      b1 = least_bin > b1 ? least_bin : b1;
      end_bin = least_bin;
      least_sum = least_sum < s.before[least_bin] ? least_sum : s.before[least_bin];
      most_sum = most_sum < s.before[least_bin + 1] ? most_sum : s.before[least_bin + 1];
    }
    const double short_of_all = all * (1.0 - 0x1p-52), u1 = set.u * most_sum;
    int t0 = reach(set.u * least_sum < short_of_all ? set.u * least_sum : short_of_all, true);
    int t1 = reach(u1 < short_of_all ? u1 : short_of_all, true);
    t1 = t1 < end_bin ? t1 : end_bin;
    t0 = t0 < t1 ? t0 : t1;
    if (b1 >= 0 && t1 >= b0 - 1) {             // one stretch
      t0 = t0 < b0 ? t0 : b0;
      t1 = b1 > t1 ? b1 : t1;
      b0 = 0;
      b1 = -1;
    } else if (b1 < 0) {
      b0 = 0;
    }
    const uint32_t many = s.count_before[t1 + 1] - s.count_before[t0] + (b1 >= b0 ? s.count_before[b1 + 1] - s.count_before[b0] : 0);
    if (!in_slices) {
      if (many <= (uint32_t)LIST) {
        if (!gather_parts(t0, t1, b0, b1)) return;
      } else if (blockIdx.x) {
        return;
      }
    }

    // (a beginning that ends in no bin of its own: all of them)
    Beginning kept = {BINS - 1, s.count[BINS - 1], s.sum[BINS - 1], 0};
    if (for_count) {
      const uint32_t c = (uint32_t)set.top_k - s.count_before[count_bin];
      kept = c < s.count[count_bin] ? select(count_bin, c, 0) : Beginning{count_bin, c, s.sum[count_bin], 0};
    }
    if (for_weight) {
      const double g = set.top_p * (by_count ? weight(kept) : all);
      int d = reach(g < all ? g : all, false);
      if (d > kept.bin) d = kept.bin;
      const u64 most = d == kept.bin ? kept.sum : s.sum[d];
      double need = ceil((g - s.before[d]) / unit_of(d));
      need = need < 1.0 ? 1.0 : need;
      if (need < (double)most) kept = select(d, 0, (u64)need);
      else if (d < kept.bin) kept = {d, s.count[d], s.sum[d], 0};
    }
    if (for_least && least_bin <= kept.bin) {
      see_to(least_bin);
      __syncthreads();
      if (tid == 0) {
        s.total_count = 0;
        s.total_sum = 0;
      }
      __syncthreads();
      uint32_t c = 0;
      u64 m = 0;
      each_of(least_bin, 0, ~0ull, [&](float v, uint32_t, u64 w) {
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
    }

    // the token
    const double sum = weight(kept), end = sum * (1.0 - 0x1p-52);
    double t = set.u * sum;
    t = t < end ? t : end;
    int d = reach(t, true);
    if (d > kept.bin) d = kept.bin;
    const u64 most = d == kept.bin ? kept.sum : s.sum[d];
    double g = floor((t - s.before[d]) / unit_of(d)) + 1.0;
    g = g < 1.0 ? 1.0 : (g < (double)most ? g : (double)most);
    const Beginning got = select(d, 0, (u64)g);
    if (tid == 0) answer(got.last, (double)place_below(logit_of(got.last), top, set.c4).m * unit_of(d), sum);
  }
};

template <class I>
__global__ __launch_bounds__(1024) void sample_choose_kernel(SampleArgs a) {
  __shared__ typename RowChoice<I>::Shared shared;
  const int64_t row = blockIdx.y;
  RowChoice<I> r{a, shared, (int)threadIdx.x, row, (const I*)a.x + row * a.x_stride};
  r.run();
}

template <class I>
hipError_t launch_i(const SampleArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.slices, (unsigned)a.rows);
  hipError_t e;
  if (a.slice == 4096) e = launch_kernel(sample_slice_kernel<I, 2>, grid, 512, 0, st, a);
  else e = launch_kernel(sample_slice_kernel<I, 4>, grid, 512, 0, st, a);
  if (e != hipSuccess) return e;
  return launch_kernel(sample_choose_kernel<I>, dim3((unsigned)a.row_parts, (unsigned)a.rows), 1024, 0, st, a);
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t st) {
  if (dtype == DT_F32) return launch_i<float>(a, st);
  return dtype == DT_F16 ? launch_i<f16>(a, st) : launch_i<bf16>(a, st);
}

}  // namespace fcg
