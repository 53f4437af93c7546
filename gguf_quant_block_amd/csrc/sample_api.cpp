// C-ABI of the choice of the next token (declarations and contract in
// include/fc_gguf.h).  Host logic only: argument checks and the division of the
// workspace.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fc_gguf.h"
#include "serving.h"

namespace {

constexpr int64_t kMaxRows = 65535, kMaxVocab = (int64_t)1 << 24;
constexpr int64_t kMaxSlices = (int64_t)1 << 23;      // a launch has under 2^32 threads: 512 for each

bool on(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// How a call's workspace is divided: the slices' histograms, first tokens and
// largest logits, then the lists that the parts of a row hand over, and counters.
// (All of 8 bytes but the counters, which come last.)
struct Division {
  int slice, slices, parts;
  size_t first, tops, lists, part_n, arrived, bytes;
  Division(int64_t rows, int64_t vocab, int cus) {
    slice = fcg::sample_slice(rows, vocab, cus);
    slices = (int)((vocab + slice - 1) / slice);
    parts = fcg::sample_parts(rows, vocab, cus);
    const size_t n = (size_t)rows * slices, lists_n = parts > 1 ? (size_t)rows * parts : 0;
    first = n * fcg::SAMPLE_BINS * 8;
    tops = first + n * fcg::SAMPLE_FIRST * sizeof(uint2);
    lists = tops + n * sizeof(fcg::SliceTop);
    part_n = lists + lists_n * fcg::SAMPLE_PART * 8;
    arrived = part_n + lists_n * 4;
    bytes = arrived + (size_t)rows * 4;
  }
};

}  // namespace

extern "C" {

int64_t fc_gguf_sample_workspace(int64_t rows, int64_t vocab) {
  if (rows < 0 || vocab <= 0) return FC_GGUF_EINVAL;
  if (rows > kMaxRows || vocab > kMaxVocab) return FC_GGUF_ERANGE;
  const int cus = fcg::cus_of_current();
  if (cus <= 0) return FC_GGUF_EHIP;
  const Division d(rows, vocab, cus);
  return rows * d.slices < kMaxSlices ? (int64_t)d.bytes : FC_GGUF_ERANGE;
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
  const Division d(rows, vocab, cus);
  if (rows * d.slices >= kMaxSlices) return FC_GGUF_ERANGE;
  if (workspace_bytes < 0 || (size_t)workspace_bytes < d.bytes) return FC_GGUF_EINVAL;
  fcg::SampleArgs a = {};
  a.slice = d.slice;
  a.slices = d.slices;
  a.row_parts = d.parts;
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
  char* const w = (char*)workspace;
  a.hist = (unsigned long long*)w;
  a.first = (uint2*)(w + d.first);
  a.slice_tops = (fcg::SliceTop*)(w + d.tops);
  a.parts = (unsigned long long*)(w + d.lists);
  a.part_n = (uint32_t*)(w + d.part_n);
  a.arrived = (uint32_t*)(w + d.arrived);
  return fcg::launch_sample(a, dtype, (hipStream_t)stream) == hipSuccess ? FC_GGUF_OK : FC_GGUF_EHIP;
}

}  // extern "C"
