// Penalties for repeated tokens, biases and a grammar's mask on the logits of
// the output layer.  For token v of a row:
//
//   x = x > 0 ? x / repetition : x * repetition     if v is in the row's tokens
//   x = x - (frequency * n + presence * (n > 0))    n: times v was generated
//   x = x + bias[v]
//   x = -inf                                        if the mask's bit of v is 0
//
// in f32, one rounding to the output's type.  Bound by HBM for many rows (the
// logits in and out: 128 rows of 131073 f32 in 27.0 us, 5.0 TB/s where a copy
// reaches 4.75), by latency for one (32064 tokens: 4.1 us).
//
// A workgroup takes a slice of one row's tokens.  It counts the row's history
// in LDS (whole numbers, so that the order of the atomics changes nothing) and
// puts the row's biases beside them, then passes over its logits once, four
// values at a time (16 bytes of f32, 8 of f16 and bf16).  Its logits are read
// before the history, so that only one of the two waits is paid.  Entries of a
// bias list that name the same token are added in the list's order: one wave
// takes 64 entries at a time, and each lane first sums its token's entries among
// them in order.
#include <math.h>

#include "serving.h"

namespace fcg {
namespace {

constexpr uint32_t LG_SEEN = 0x80000000u;      // the token is in the row's tokens

// N values at an address aligned to one of them
template <class T, int N> struct Some { typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T)))); };

// A thread has V values next to each other, ROUNDS times: the slice is
// LG_THREADS * V * ROUNDS values.
template <class I, class O, int LG_THREADS, int V, int ROUNDS>
__global__ __launch_bounds__(LG_THREADS) void logits_kernel(LogitsArgs a) {
  constexpr int SLICE = LG_THREADS * V * ROUNDS;
  __shared__ uint32_t count[SLICE];
  __shared__ float bias[SLICE];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y;
  const int64_t v0 = (int64_t)blockIdx.x * SLICE;
  const int n = (int)(a.vocab - v0 < SLICE ? a.vocab - v0 : SLICE);
  const I* x = (const I*)a.x + row * a.x_stride + v0;
  O* y = (O*)a.out + row * a.o_stride + v0;

  typedef typename Some<I, V>::vec IV;
  typedef typename Some<O, V>::vec OV;
  IV z[ROUNDS];
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int i = (k * LG_THREADS + tid) * V;
    if (i + V <= n) z[k] = *(const IV*)(x + i);
    else
#pragma unroll
      for (int e = 0; e < V; ++e) z[k][e] = i + e < n ? x[i + e] : (I)0;
  }
  // 32 bits from the thread's first value's on (v0 is a multiple of 32, so is
  // a word's first value; the V values are in one word)
  uint32_t allow[ROUNDS];
#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int i = (k * LG_THREADS + tid) * V;
    allow[k] = a.mask && i < n ? a.mask[row * a.mask_stride + ((v0 + i) >> 5)] >> (i & 31) : ~0u;
  }

  int len = 0;
  int64_t b0 = 0, b1 = 0;
  if (a.tokens) {
    len = a.lens[row];
    len = len < 0 ? 0 : (len < a.tokens_stride ? len : (int)a.tokens_stride);
  }
  if (a.bias_offsets) {
    b0 = a.bias_offsets[row];
    b1 = a.bias_offsets[row + 1];
    b0 = b0 < 0 ? 0 : b0;
    b1 = b1 < a.bias_count ? b1 : a.bias_count;
  }
  const int prompt = a.prompt_lens && len > 0 ? a.prompt_lens[row] : 0;
  const float rep = a.repetition ? a.repetition[row] : 1.f;
  const float freq = a.frequency ? a.frequency[row] : 0.f;
  const float pres = a.presence ? a.presence[row] : 0.f;
  const bool counted = len > 0, biased = b0 < b1;
  for (int i = tid * 4; i < SLICE; i += LG_THREADS * 4) {
    if (counted) *(u32x4*)&count[i] = (u32x4){0, 0, 0, 0};
    if (biased) *(floatx4*)&bias[i] = (floatx4){0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();
  const int32_t* said = a.tokens + row * a.tokens_stride;
#pragma unroll 4
  for (int i = tid; i < len; i += LG_THREADS) {
    const int64_t v = said[i] - v0;
    if (v >= 0 && v < n) {
      atomicOr(&count[v], LG_SEEN);
      if (i >= prompt) atomicAdd(&count[v], 1u);
    }
  }
  if (tid < 64)
    for (int64_t e0 = b0; e0 < b1; e0 += 64) {
      const bool there = e0 + tid < b1;
      const int64_t v = there ? a.bias_ids[e0 + tid] - v0 : -1;
      const int id = v >= 0 && v < n ? (int)v : -1;
      const float b = there ? a.bias_values[e0 + tid] : 0.f;
      uint64_t here = __ballot(id >= 0);
      if (!here) continue;
      float sum = id >= 0 ? bias[id] : 0.f;
      for (; here; here &= here - 1) {
        const int j = __builtin_ctzll(here);
        const int idj = __builtin_amdgcn_readlane(id, j);
        const float bj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, b), j));
        if (idj == id) sum += bj;
      }
      if (id >= 0) bias[id] = sum;               // the same sum from every lane of a token
    }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < ROUNDS; ++k) {
    const int i = (k * LG_THREADS + tid) * V;
    if (i >= n) break;
    OV out;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float f = (float)z[k][e];
      if (counted) {
        const uint32_t c = count[i + e];
        if (c & LG_SEEN) {
          f = f > 0.f ? f / rep : f * rep;
          const uint32_t m = c & ~LG_SEEN;
          f -= freq * (float)m + (m ? pres : 0.f);
        }
      }
      if (biased) f += bias[i + e];
      out[e] = (O)(allow[k] >> e & 1 ? f : -INFINITY);
    }
    // (past the caches: 34.5 -> 32.5 us for 128 rows of which nothing is cached)
    if (i + V <= n) __builtin_nontemporal_store(out, (OV*)(y + i));
    else
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (i + e < n) y[i + e] = out[e];
  }
}

template <class I, class O>
hipError_t launch_io(const LogitsArgs& a, int num_cu, hipStream_t st) {
  // Slices of 4096 tokens, or of 1024 where those would leave CUs idle (one
  // row of 32064: 11 us and 4; 128 rows of 131073 f32 in slices of 4096, 512
  // threads: 27.9 us, 256 threads: 33.9, slices of 8192: 35.6, of 2048: 29.1).
  const int64_t wide = (a.vocab + 4095) / 4096, narrow = (a.vocab + 1023) / 1024;
  if (wide * a.rows >= 2 * num_cu)
    return launch_kernel(logits_kernel<I, O, 512, 4, 2>, dim3((unsigned)wide, (unsigned)a.rows), 512, 0, st, a);
  return launch_kernel(logits_kernel<I, O, 256, 4, 1>, dim3((unsigned)narrow, (unsigned)a.rows), 256, 0, st, a);
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, int in_dtype, int out_dtype, int num_cu, hipStream_t st) {
  if (in_dtype == DT_F32) return launch_io<float, float>(a, num_cu, st);
  if (in_dtype == DT_F16) return out_dtype == DT_F32 ? launch_io<f16, float>(a, num_cu, st) : launch_io<f16, f16>(a, num_cu, st);
  return out_dtype == DT_F32 ? launch_io<bf16, float>(a, num_cu, st) : launch_io<bf16, bf16>(a, num_cu, st);
}

}  // namespace fcg
