// C-ABI of the choice of the next token (declarations and contract in
// include/fc_gguf.h).  Host logic only: argument checks and the division of the
// workspace.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fc_gguf.h"
#include "serving.h"

namespace {

constexpr int64_t kMaxRows = 65535, kMaxVocab = (int64_t)1 << 24;

bool on(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// bytes of `rows` rows in slices: their histograms, their first tokens, their largest logits
size_t workspace_of(int64_t rows, int64_t slices) {
  return (size_t)(rows * slices) * ((fcg::SAMPLE_BINS + fcg::SAMPLE_FIRST) * 8 + sizeof(fcg::SliceTop));
}

}  // namespace

extern "C" {

int64_t fc_gguf_sample_workspace(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab <= 0) return FC_GGUF_EINVAL;
  if (rows > kMaxRows || vocab > kMaxVocab) return FC_GGUF_ERANGE;
  const int cus = fcg::cus_of_current();
  if (cus <= 0) return FC_GGUF_EHIP;
  const int slice = fcg::sample_slice(rows, vocab, cus);
  return (int64_t)workspace_of(rows, (vocab + slice - 1) / slice);
}

int fc_gguf_sample(const void* x, int64_t x_stride, int dtype, int64_t rows, int64_t vocab, const float* u,
                   const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                   int32_t* out, float* logprobs, void* workspace, int64_t workspace_bytes, void* stream) {
  if (rows < 0 || vocab <= 0) return FC_GGUF_EINVAL;
  if (dtype != FC_GGUF_F16 && dtype != FC_GGUF_BF16 && dtype != FC_GGUF_F32) return FC_GGUF_EUNSUPPORTED;
  if (rows > kMaxRows || vocab > kMaxVocab) return FC_GGUF_ERANGE;
  if (rows == 0) return FC_GGUF_OK;
  if (!x || !on(x, dtype == FC_GGUF_F32 ? 4 : 2) || x_stride < vocab || !u || !on(u, 4) || !out || !on(out, 4) ||
      (temperature && !on(temperature, 4)) || (top_k && !on(top_k, 4)) || (top_p && !on(top_p, 4)) ||
      (min_p && !on(min_p, 4)) || (logprobs && !on(logprobs, 4)) || !workspace || !on(workspace, 8))
    return FC_GGUF_EINVAL;
  const int cus = fcg::cus_of_current();
  if (cus <= 0) return FC_GGUF_EHIP;
  const int slice = fcg::sample_slice(rows, vocab, cus);
  fcg::SampleArgs a = {};
  a.slice = slice;
  a.slices = (int)((vocab + slice - 1) / slice);
  if (workspace_bytes < 0 || (size_t)workspace_bytes < workspace_of(rows, a.slices)) return FC_GGUF_EINVAL;
  a.x = x;
  a.x_stride = x_stride;
  a.rows = rows;
  a.vocab = vocab;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.out = out;
  a.logprobs = logprobs;
  a.hist = (unsigned long long*)workspace;
  a.first = (uint2*)(a.hist + rows * a.slices * fcg::SAMPLE_BINS);
  a.slice_tops = (fcg::SliceTop*)(a.first + rows * a.slices * fcg::SAMPLE_FIRST);
  return fcg::launch_sample(a, dtype, (hipStream_t)stream) == hipSuccess ? FC_GGUF_OK : FC_GGUF_EHIP;
}

}  // extern "C"
