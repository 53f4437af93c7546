// Penalties for repeated tokens, biases and a grammar's mask on the logits of
// the output layer.  For token v of a row:
//
//   x = x > 0 ? x / repetition : x * repetition     if v is in the row's tokens
//   x = x - (frequency * n + presence * (n > 0))    n: times v was generated
//   x = x + bias[v]
//   x = -inf                                        if the mask's bit of v is 0
//
// in f32, one rounding to the output's type.  Bound by HBM for many rows (the
// logits in and out), by latency for one.
//
// A workgroup takes LG_SLICE tokens of one row.  It counts the row's history
// in LDS (whole numbers, so that the order of the atomics changes nothing) and
// puts the row's biases beside them, then passes over its logits once.
// Entries of a bias list that name the same token are added in the list's
// order: one wave takes 64 entries at a time, and each lane first sums its
// token's entries among them in order.
#include <math.h>

#include "serving.h"

namespace fcg {
namespace {

constexpr int LG_THREADS = 256;
constexpr uint32_t LG_SEEN = 0x80000000u;      // the token is in the row's tokens

template <class I> __device__ __forceinline__ float to_f(I x) { return (float)x; }

template <class I, class O, int SLICE>
__global__ __launch_bounds__(LG_THREADS) void logits_kernel(LogitsArgs a) {
  __shared__ uint32_t count[SLICE];
  __shared__ float bias[SLICE];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.y;
  const int64_t v0 = (int64_t)blockIdx.x * SLICE;
  const int n = (int)(a.vocab - v0 < SLICE ? a.vocab - v0 : SLICE);

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
  if (len > 0)
    for (int i = tid; i < n; i += LG_THREADS) count[i] = 0;
  if (b0 < b1)
    for (int i = tid; i < n; i += LG_THREADS) bias[i] = 0.f;
  __syncthreads();
  const int prompt = a.prompt_lens && len > 0 ? a.prompt_lens[row] : 0;
  for (int i = tid; i < len; i += LG_THREADS) {
    const int64_t v = a.tokens[row * a.tokens_stride + i] - v0;
    if (v < 0 || v >= n) continue;
    atomicOr(&count[v], LG_SEEN);
    if (i >= prompt) atomicAdd(&count[v], 1u);
  }
  if (tid < 64)
    for (int64_t e0 = b0; e0 < b1; e0 += 64) {
      const bool there = e0 + tid < b1;
      const int64_t v = there ? a.bias_ids[e0 + tid] - v0 : -1;
      const int id = v >= 0 && v < n ? (int)v : -1;
      if (!__any(id >= 0)) continue;
      const float x = there ? a.bias_values[e0 + tid] : 0.f;
      float sum = id >= 0 ? bias[id] : 0.f;
      for (int j = 0; j < 64; ++j) {
        const int idj = __shfl(id, j);
        const float xj = __shfl(x, j);
        if (idj == id) sum += xj;
      }
      if (id >= 0) bias[id] = sum;               // the same sum from every lane of a token
    }
  __syncthreads();

  const float rep = a.repetition ? a.repetition[row] : 1.f;
  const float freq = a.frequency ? a.frequency[row] : 0.f;
  const float pres = a.presence ? a.presence[row] : 0.f;
  const I* x = (const I*)a.x + row * a.x_stride + v0;
  O* y = (O*)a.out + row * a.o_stride + v0;
  const uint32_t* mask = a.mask ? a.mask + row * a.mask_stride + v0 / 32 : nullptr;
  for (int i = tid; i < n; i += LG_THREADS) {
    float z = to_f(x[i]);
    if (len > 0) {
      const uint32_t c = count[i];
      if (c & LG_SEEN) {
        z = z > 0.f ? z / rep : z * rep;
        const uint32_t k = c & ~LG_SEEN;
        z -= freq * (float)k + (k ? pres : 0.f);
      }
    }
    if (b0 < b1) z += bias[i];
    if (mask && !(mask[i >> 5] >> (i & 31) & 1)) z = -INFINITY;
    y[i] = (O)z;
  }
}

template <class I, class O>
hipError_t launch_io(const LogitsArgs& a, hipStream_t st) {
  constexpr int SLICE = 4096;
  const dim3 grid((unsigned)((a.vocab + SLICE - 1) / SLICE), (unsigned)a.rows);
  logits_kernel<I, O, SLICE><<<grid, LG_THREADS, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logits(const LogitsArgs& a, int in_dtype, int out_dtype, int num_cu, hipStream_t st) {
  (void)num_cu;
  if (in_dtype == DT_F32) return launch_io<float, float>(a, st);
  if (in_dtype == DT_F16) return out_dtype == DT_F32 ? launch_io<f16, float>(a, st) : launch_io<f16, f16>(a, st);
  return out_dtype == DT_F32 ? launch_io<bf16, float>(a, st) : launch_io<bf16, bf16>(a, st);
}

}  // namespace fcg
