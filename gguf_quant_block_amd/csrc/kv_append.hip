// Appending keys and values to the paged cache, with the rotation of queries
// and keys on the way.
//
//   angle(t, j) = position[axis[j]][t] * inv_freq[j]
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin)      for pair j of a head
//
// Bound by HBM: q, k and v are read once, the rotated q and the cache entries
// written once.  The angles are products in f64, reduced to a turn there:
// at position 10^5 an f32 product would be off by up to 0.004 rad.  They are
// taken once per token and pair into LDS and serve every head.  The rotation
// is in f32 with one rounding to the cache's type.  Measured: 4096 tokens, 32
// query and 8 key heads of 128: 22.3 us, 4.5 TB/s (a copy reaches 4.75; HBM
// writes 1.11 of the bytes, for cache lines that several workgroups fill), 29.6
// where nothing is cached; 2500 tokens on three axes 16.2 us, and 24.2; one
// token 5.3 us, most of it the launch.
//
// A workgroup takes tokens_per_wg consecutive tokens (1 for a decode step,
// where latency counts and the heads are spread over y_splits workgroups; up
// to 8 for a prompt).  Q and K are handled in units of 16 elements, the two
// pieces of 8 that hold 8 pairs.  V pieces hold 8 tokens of one dimension, so
// V is handled in runs: consecutive tokens whose slots follow each other
// inside one piece row.  A run belongs to the workgroup in whose tokens it
// begins; a thread reads 8 dimensions of its up to 8 tokens and turns them in
// registers, so that a whole piece is one 16-byte store wherever the prompt
// begins inside a page.
//
// With norms, a head is first divided by the root of its mean square and
// multiplied by weights; in 8 bits, keys (after norm and rotation, from f32)
// and values become codes under a scale of their own for each token and head
// (serving.h).  Both need a value of a whole head: its units stand in
// neighbouring lanes of a wave (of 96 dimensions 6 of 8), which exchange sums
// and maxima; of a run of V the largest of each of its 8 tokens.
// Measured, 4096 tokens of 32 query and 8 key heads of 128: with norms 22.3 us
// (101 MB, 4.5 TB/s: what the plain rotation takes), into 8 bits 22.2 (92 MB, 4.2
// TB/s, with HBM writing 47.7 of 41.9 MB, for cache lines that several workgroups
// fill); 128 tokens of a batch, norms and 8 bits, 6.9; one token with norms 4.5.
// Heads of 96 with norms or in 8 bits are further from that: the compiler keeps a
// unit that not every lane has in 48 bytes of scratch memory.  4096 tokens with
// norms 26.5 us (16.4 without; a copy of the bytes 16.2), into 8 bits 25 (14.9).
#include <type_traits>

#include "serving.h"

namespace fcg {
namespace {

constexpr int AP_MAX_TOKENS = 8;
constexpr int AP_MAX_HALF = 128;     // rotated pairs of a head

template <class E>
__device__ __forceinline__ void unpack16(const u32x4& a, const u32x4& b, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo2f<E>(a[i]);
    x[2 * i + 1] = hi2f<E>(a[i]);
    x[8 + 2 * i] = lo2f<E>(b[i]);
    x[8 + 2 * i + 1] = hi2f<E>(b[i]);
  }
}
template <class E>
__device__ __forceinline__ void pack16(const float* x, u32x4& a, u32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = pack2<E>(x[2 * i], x[2 * i + 1]);
    b[i] = pack2<E>(x[8 + 2 * i], x[8 + 2 * i + 1]);
  }
}
__device__ __forceinline__ void rotate16(float* x, const float2* cs, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 c = cs[i];
    const int i0 = interleaved ? 2 * i : i, i1 = interleaved ? 2 * i + 1 : i + 8;
    const float x0 = x[i0], x1 = x[i1];
    x[i0] = x0 * c.x - x1 * c.y;
    x[i1] = x1 * c.x + x0 * c.y;
  }
}
template <class E>
__device__ __forceinline__ void rotate8(u32x4& a, u32x4& b, const float2* cs, bool interleaved) {
  float x[16];
  unpack16<E>(a, b, x);
  rotate16(x, cs, interleaved);
  pack16<E>(x, a, b);
}

// An operation over 4, 8, 16 or 32 neighbouring lanes, its result in each: a
// quad's halves, its lanes, then the mirrored halves of 8 and of 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
template <int LANES, class F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, F f) {
  x = f(x, moved<0xB1>(x));
  x = f(x, moved<0x4E>(x));
  if constexpr (LANES >= 8) x = f(x, moved<0x141>(x));
  if constexpr (LANES >= 16) x = f(x, moved<0x140>(x));
  if constexpr (LANES >= 32) x = f(x, (uint32_t)__shfl_xor((int)x, 16));
  return x;
}
template <int LANES>
__device__ __forceinline__ float sum_lanes(float x) {
  return __builtin_bit_cast(float, over_lanes<LANES>(__builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }));
}
// (of magnitudes: their bits stand in the same order)
template <int LANES>
__device__ __forceinline__ float max_lanes(float x) {
  return __builtin_bit_cast(float, over_lanes<LANES>(__builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) { return a > b ? a : b; }));
}
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// A head's 16 values of this lane as codes under the head's scale: its stored
// exponent.  Infinite and NaN values become the NaN code and do not count for
// the scale.
template <class E, int LANES>
__device__ __forceinline__ int quantise16(const float* x, uint32_t* code) {
  float m = 0.f, odd = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    m = fmaxf(m, fabsf(x[i]));
    odd = fmaf(x[i], 0.f, odd);                  // NaN if there is an infinite or NaN value
  }
  bool special = !(odd == 0.f);
  if (__any(special)) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]) < INFINITY ? fabsf(x[i]) : 0.f);
  }
  const int e = exponent_of<E>(max_lanes<LANES>(m));
  const float by = __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
  special = special || e == Held<E>::HI;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = x[i] * by;
  if (__any(special)) {
    const float most = e == Held<E>::HI ? CODE_MOST_HI : CODE_MOST;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = fabsf(x[i]) < INFINITY ? fminf(fmaxf(y[i], -most), most) : __builtin_nanf("");
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
    code[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], lo, true);
  }
  return e;
}

// The mean square of a head, of which x are this lane's 16 values, and eps, whose
// root norms the head.  Squares of f16 are well inside the range of f32.  Those of
// bf16 are not from 2^64 on, nor are they precise below 2^-63: such a head, and
// eps with it, is first scaled by the power of two that takes the larger of its
// values and the root of eps below 1.  The scaled values have the same norm, and
// other heads keep their bits.  (A head with an infinite value, or of zeros without
// eps, stays what it is: by the formula NaN.)  The question costs 4096 bf16 tokens of
// 32 query and 8 key heads of 128 0.3 to 0.5 of 21.6 us.
template <class E, int LANES>
__device__ __forceinline__ float mean_square(float* x, float one_of, float eps) {
  auto mean = [&](float e) -> float {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) sum = fmaf(x[j], x[j], sum);
    return sum_lanes<LANES>(sum) * one_of + e;
  };
  float y = mean(eps);
  if constexpr (std::is_same<E, bf16>::value) {
    // (a mean of 2^-100: what squares lose below f32's normal range, 2^-150 each, is nothing to it)
    const bool odd = !(y >= 0x1p-100f && y < INFINITY);
    if (__any(odd)) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(x[j]));
      m = fmaxf(max_lanes<LANES>(m), sqrtf(eps));
      const int by = odd && m > 0.f && m < INFINITY ? -__builtin_amdgcn_frexp_expf(m) : 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = __builtin_ldexpf(x[j], by);
      y = mean(__builtin_ldexpf(eps, 2 * by));
    }
  }
  return y;
}

// A unit of 16 elements of a head: where it comes from and where it goes.
struct Unit {
  int t, h, u;         // token of the workgroup, head (queries, then keys), unit of the head
  int p0, p1;          // its two pieces: 8 pairs (halves or neighbours), or 16 elements that pass
};

// A run of V in 8 bits: 8 dimensions from d0 on of `len` tokens, N at most, whose
// slots begin at s, of head h; LANES lanes have the head.  (A decode step's runs
// are of one token: N = 1 instead of 8, one token of 32 query and 8 key heads of
// 128 5.3 us instead of 7.3, 128 tokens 6.9 instead of 8.6.)
template <class E, int D, int LANES, int N>
__device__ __forceinline__ void append_v8(const AppendArgs& a, const u32x4* v, int h, int d0, int len, int s) {
  const int ps = 1 << a.kv.page_shift;
  uint32_t bad = 0, top[(N + 1) / 2];            // the largest magnitudes of tokens 2j and 2j + 1, as bits of E
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= nonfinite2<E>(v[j][k]);
#pragma unroll
  for (int j = 0; j < (N + 1) / 2; ++j) {
    uint32_t m[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < (N > 1 ? 2 : 1); ++e) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w = v[2 * j + e][k];
        w &= ~((nonfinite2<E>(w) >> 15) * 0xFFFFu);
        m[e] = max16x2(m[e], w & 0x7FFF7FFFu);
      }
      m[e] = max16x2(m[e], m[e] >> 16) & 0xFFFFu;
    }
    top[j] = over_lanes<LANES>(m[0] | m[1] << 16, max16x2);
  }
  int e[N];
  float by[N];
  bool special = bad != 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    e[j] = exponent_of<E>(j & 1 ? hi2f<E>(top[j / 2]) : lo2f<E>(top[j / 2]));
    by[j] = __builtin_bit_cast(float, (uint32_t)(254 - e[j]) << 23);
    special = special || e[j] == Held<E>::HI;
  }
  const int64_t row = (int64_t)(s >> a.kv.page_shift) * a.kv.kv_heads + h;
  const int place = s & (ps - 1);
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (d0 == j * 8 && j < len) a.kv.v_scale[row * ps + place + j] = (uint8_t)e[j];
  if (LANES * 8 != D && d0 >= D) return;
  uint8_t* dst = (uint8_t*)a.kv.v + row * ps * D + ((int64_t)(place >> 3) * D + d0) * 8;
  const bool any = __any(special);
  uint32_t code[8][(N + 3) / 4];                 // of dimension d0 + i: the tokens' codes
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    float y[N > 1 ? N : 2];
    if constexpr (N == 1) y[1] = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float x = d & 1 ? hi2f<E>(v[j][d / 2]) : lo2f<E>(v[j][d / 2]);
      y[j] = x * by[j];
      if (any) {
        const float most = e[j] == Held<E>::HI ? CODE_MOST_HI : CODE_MOST;
        y[j] = fabsf(x) < INFINITY ? fminf(fmaxf(y[j], -most), most) : __builtin_nanf("");
      }
    }
    if constexpr (N == 1) {
      code[d][0] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j], y[4 * j + 1], 0, false);
        code[d][j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * j + 2], y[4 * j + 3], lo, true);
      }
    }
  }
  if constexpr (N == 8)
    if (len == 8) {
#pragma unroll
      for (int d = 0; d < 8; ++d) *(uint2*)(dst + d * 8) = make_uint2(code[d][0], code[d][1]);
      return;
    }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j < len)
#pragma unroll
      for (int d = 0; d < 8; ++d) dst[d * 8 + (s & 7) + j] = (uint8_t)(code[d][j / 4] >> (8 * (j & 3)));
}

template <class E, int D, int AP_THREADS, bool NORM, bool Q8>
__global__ __launch_bounds__(AP_THREADS) void kv_append_kernel(AppendArgs a) {
  __shared__ float2 cs[AP_MAX_TOKENS * AP_MAX_HALF];
  __shared__ int slot[AP_MAX_TOKENS + 8];      // [i + 1]: token i of the workgroup
  __shared__ int run_at[AP_MAX_TOKENS], run_len[AP_MAX_TOKENS], runs;
  const int tid = threadIdx.x;
  constexpr int units = D / 16, pieces = D / 8;
  // lanes of a head's units, and of 8 tokens of a head's V
  constexpr int lanes = (NORM || Q8) && D == 96 ? 8 : units, vlanes = Q8 && D == 96 ? 16 : pieces;
  const int ps = 1 << a.kv.page_shift;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_wg;
  const int nt = (int)(a.T - t0 < a.tokens_per_wg ? a.T - t0 : a.tokens_per_wg);
  const int half = a.inv_freq ? a.rot / 2 : 0, rot_units = half / 8;
  const int64_t top = a.kv.pages << a.kv.page_shift;
  const int per_token = (a.q_heads + a.kv.kv_heads) * lanes, all = nt * per_token;
  const int64_t page_elems = (int64_t)a.kv.kv_heads * ps * D;
  const int first = blockIdx.y * AP_THREADS + tid, step = a.y_splits * AP_THREADS;

  // the thread's next unit, requested ahead of its use
  u32x4 x0, x1;
  Unit w;
  int t_next = first / per_token, rest = first - t_next * per_token;
  auto request = [&]() {
    w.t = t_next;
    w.h = rest / lanes;
    w.u = rest - w.h * lanes;
    const bool apart = w.u < rot_units && !a.interleaved;
    w.p0 = apart ? w.u : 2 * w.u;
    w.p1 = apart ? w.u + rot_units : 2 * w.u + 1;
    const uint16_t* src = w.h < a.q_heads ? a.q + (t0 + w.t) * a.q_stride + w.h * D
                                          : a.k + (t0 + w.t) * a.k_stride + (w.h - a.q_heads) * D;
    if (lanes == units || w.u < units) {
      x0 = *(const u32x4*)(src + w.p0 * 8);
      x1 = *(const u32x4*)(src + w.p1 * 8);
    } else {                                     // (a lane without a unit)
      x0 = x1 = (u32x4){0, 0, 0, 0};
    }
    for (rest += step; rest >= per_token; rest -= per_token) ++t_next;
  };
  if (first < all) request();

  // the slots of the tokens, of the one before and of 7 after (-1 where a slot
  // names no place in the cache): a run of V may reach that far
  if (tid < nt + 8) {
    const int64_t t = t0 + tid - 1;
    const int64_t s = t >= 0 && t < a.T ? a.slots[t] : -1;
    slot[tid] = s >= 0 && s < top ? (int)s : -1;
  }
  for (int i = tid; i < nt * half; i += AP_THREADS) {
    const int t = i / half, j = i - t * half;
    int ax = a.pair_axis ? a.pair_axis[j] : 0;
    ax = ax < 0 || ax >= a.axes ? 0 : ax;
    const double turns = (double)a.positions[ax * a.T + t0 + t] * (double)a.inv_freq[j] * 0.15915494309189533577;
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c * a.rope_scale, s * a.rope_scale);
  }
  __syncthreads();
  if (tid < 64) {                              // the runs of V, a lane for each token
    bool begins = false;
    int len = 1;
    if (tid < nt) {
      const int s = slot[tid + 1], before = slot[tid];
      begins = s >= 0 && ((s & 7) == 0 || before < 0 || before != s - 1);
      bool on = true;
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        on = on && ((s + k) & 7) != 0 && slot[tid + 1 + k] == s + k;
        len += on;
      }
    }
    const uint64_t m = __ballot(begins);
    if (begins) {
      const int at = __builtin_popcountll(m & (((uint64_t)1 << tid) - 1));
      run_at[at] = tid;
      run_len[at] = len;
    }
    if (tid == 0) runs = __builtin_popcountll(m);
  }
  __syncthreads();

  // the first run of V, requested ahead of the units' stores
  const int per_run = a.kv.kv_heads * vlanes, vall = runs * per_run;
  u32x4 v[8];
  auto request_v = [&](int i) {
    const int r = i / per_run, rest = i - r * per_run, h = rest / vlanes, d0 = (rest - h * vlanes) * 8;
    const uint16_t* src = a.v + (t0 + run_at[r]) * a.v_stride + h * D + d0;
    const int len = vlanes == pieces || d0 < D ? run_len[r] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < len) v[j] = *(const u32x4*)(src + j * a.v_stride);
      else if (Q8) v[j] = (u32x4){0, 0, 0, 0};
  };
  if (first < vall) request_v(first);

  for (int i = first; i < all; i += step) {
    const Unit z = w;
    u32x4 y0 = x0, y1 = x1;
    if (i + step < all) request();
    const int s = slot[z.t + 1];
    uint32_t code[4];
    if constexpr (NORM || Q8) {
      float x[16];
      unpack16<E>(y0, y1, x);
      if constexpr (NORM) {
        const bool isq = z.h < a.q_heads;
        const float* weight = isq ? a.q_norm + (int64_t)z.h * a.q_norm_stride : a.k_norm + (int64_t)(z.h - a.q_heads) * a.k_norm_stride;
        if (isq ? a.q_norm != nullptr : a.k_norm != nullptr) {
          const float by = 1.f / sqrtf(mean_square<E, lanes>(x, 1.f / D, a.eps));
          if (lanes == units || z.u < units) {
            float g[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              *(floatx4*)(g + 4 * j) = *(const floatx4*)(weight + z.p0 * 8 + 4 * j);
              *(floatx4*)(g + 8 + 4 * j) = *(const floatx4*)(weight + z.p1 * 8 + 4 * j);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] *= by * g[j];
          }
        }
      }
      if (z.u < rot_units) rotate16(x, cs + z.t * half + z.u * 8, a.interleaved);
      pack16<E>(x, y0, y1);
      if constexpr (Q8)
        if (z.h >= a.q_heads) {
          const int e = quantise16<E, lanes>(x, code);
          if (z.u == 0 && s >= 0)
            a.kv.k_scale[((int64_t)(s >> a.kv.page_shift) * a.kv.kv_heads + (z.h - a.q_heads)) * ps + (s & (ps - 1))] = (uint8_t)e;
        }
      if (lanes != units && z.u >= units) continue;
    } else if (z.u < rot_units) rotate8<E>(y0, y1, cs + z.t * half + z.u * 8, a.interleaved);
    if (z.h < a.q_heads) {
      uint16_t* dst = a.q_out + (t0 + z.t) * a.o_stride + z.h * D;
      // (past the caches: whole lines that others read next, on other XCDs;
      // 31.7 -> 28.9 us for the 4096 tokens where nothing is in a cache yet)
      __builtin_nontemporal_store(y0, (u32x4*)(dst + z.p0 * 8));
      __builtin_nontemporal_store(y1, (u32x4*)(dst + z.p1 * 8));
    } else if (Q8) {
      if (s >= 0) {
        uint8_t* dst = (uint8_t*)a.kv.k + (int64_t)(s >> a.kv.page_shift) * page_elems +
                       (int64_t)(z.h - a.q_heads) * ps * D + (s & (ps - 1)) * 8;
        *(uint2*)(dst + (int64_t)z.p0 * ps * 8) = make_uint2(code[0], code[1]);
        *(uint2*)(dst + (int64_t)z.p1 * ps * 8) = make_uint2(code[2], code[3]);
      }
    } else if (s >= 0) {
      uint16_t* dst = (uint16_t*)a.kv.k + (int64_t)(s >> a.kv.page_shift) * page_elems +
                      (int64_t)(z.h - a.q_heads) * ps * D + (s & (ps - 1)) * 8;
      *(u32x4*)(dst + (int64_t)z.p0 * ps * 8) = y0;
      *(u32x4*)(dst + (int64_t)z.p1 * ps * 8) = y1;
    }
  }

  for (int i = first; i < vall; i += step) {
    if (i != first) request_v(i);
    const int r = i / per_run, rest = i - r * per_run, h = rest / vlanes, d0 = (rest - h * vlanes) * 8;
    const int len = run_len[r], s = slot[run_at[r] + 1];
    if constexpr (Q8) {
      if (__all(len == 1)) append_v8<E, D, vlanes, 1>(a, v, h, d0, len, s);
      else append_v8<E, D, vlanes, 8>(a, v, h, d0, len, s);
      continue;
    }
    uint16_t* dst = (uint16_t*)a.kv.v + (int64_t)(s >> a.kv.page_shift) * page_elems + (int64_t)h * ps * D +
                    (int64_t)(((s & (ps - 1)) >> 3) * D + d0) * 8;
    if (len == 8) {
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = v[2 * j][d / 2], hi = v[2 * j + 1][d / 2];
          y[j] = d & 1 ? (lo >> 16) | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | (hi << 16);
        }
        *(u32x4*)(dst + d * 8) = y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < len)
#pragma unroll
          for (int d = 0; d < 8; ++d)
            dst[d * 8 + (s & 7) + j] = (uint16_t)(d & 1 ? v[j][d / 2] >> 16 : v[j][d / 2]);
    }
  }
}

template <class E, int D, int THREADS>
hipError_t append_d(const AppendArgs& a, dim3 grid, hipStream_t st) {
  const bool norm = a.q_norm || a.k_norm;
  if (a.kv.k_scale)
    return norm ? launch_kernel(kv_append_kernel<E, D, THREADS, true, true>, grid, THREADS, 0, st, a)
                : launch_kernel(kv_append_kernel<E, D, THREADS, false, true>, grid, THREADS, 0, st, a);
  return norm ? launch_kernel(kv_append_kernel<E, D, THREADS, true, false>, grid, THREADS, 0, st, a)
              : launch_kernel(kv_append_kernel<E, D, THREADS, false, false>, grid, THREADS, 0, st, a);
}

template <class E, int THREADS>
hipError_t append_e(const AppendArgs& a, dim3 grid, hipStream_t st) {
  switch (a.kv.head_dim) {
    case 64: return append_d<E, 64, THREADS>(a, grid, st);
    case 96: return append_d<E, 96, THREADS>(a, grid, st);
    case 128: return append_d<E, 128, THREADS>(a, grid, st);
    default: return append_d<E, 256, THREADS>(a, grid, st);
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& args, int dtype, int num_cu, hipStream_t st) {
  AppendArgs a = args;
  // Tokens per workgroup: as many as leave a workgroup per CU.  Where that is
  // all 8, workgroups of 512 threads (2500 tokens, 40 heads of 128: 17.1 us,
  // 20.0 with 256 threads and 18.6 with 4 tokens); else of 256 (one token, 96
  // heads of 96: 4.9 us, 5.6 with 512).
  int tb = AP_MAX_TOKENS;
  while (tb > 1 && (a.T + tb - 1) / tb < num_cu) tb /= 2;
  const int threads = tb == AP_MAX_TOKENS ? 512 : 256;
  a.tokens_per_wg = tb;
  const int64_t wgs = (a.T + tb - 1) / tb;
  // a token's heads over several workgroups, one unit of 16 elements per thread, while CUs are idle
  const int64_t most = ((int64_t)tb * (a.q_heads + a.kv.kv_heads) * (a.kv.head_dim / 16) + threads - 1) / threads;
  int64_t y = num_cu / wgs;
  y = y < 1 ? 1 : (y > most ? most : y);
  a.y_splits = (int)y;
  const dim3 grid((unsigned)wgs, (unsigned)y);
  if (threads == 512) return dtype == DT_F16 ? append_e<f16, 512>(a, grid, st) : append_e<bf16, 512>(a, grid, st);
  return dtype == DT_F16 ? append_e<f16, 256>(a, grid, st) : append_e<bf16, 256>(a, grid, st);
}

}  // namespace fcg
