// Host check of the C-ABI layer of the choice of the next token, without a GPU:
// the HIP runtime and the launcher are stand-ins.  Every refusal must launch
// nothing, and what is launched must fit the workspace that was asked for.
// Prints "ok" and returns 0, or the first line that does not hold.
#include <math.h>
#include <stdio.h>

#include "sample_api.cpp"

static int launches = 0, cus = 256;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 70; return hipSuccess; }   // (past the devices whose count is kept)
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = cus; return cus ? hipSuccess : hipErrorInvalidValue; }
}
namespace fcg {
static SampleArgs last;
hipError_t launch_sample(const SampleArgs& a, int, hipStream_t) {
  last = a;
  ++launches;
  return hipSuccess;
}
}  // namespace fcg

#define EXPECT(call, code, count)                                                             \
  do {                                                                                        \
    const int before = launches, got = (int)(call);                                           \
    if (got != (code) || launches - before != (count)) {                                      \
      printf("line %d: %s gave %d, %d launches\n", __LINE__, #call, got, launches - before);  \
      return 1;                                                                               \
    }                                                                                         \
  } while (0)

int main() {
  alignas(16) static unsigned char mem[1 << 16];
  void* p = mem;
  const int32_t* i = (const int32_t*)mem;
  const float* f = (const float*)mem;
  int32_t* o = (int32_t*)(mem + 1024);
  float* l = (float*)(mem + 2048);
  const int E = FC_GGUF_EINVAL, U = FC_GGUF_EUNSUPPORTED, R = FC_GGUF_ERANGE;
  const int64_t many = (int64_t)1 << 40;
  // x, xs, dtype, rows, vocab, u, temperature, top_k, top_p, min_p, out, logprobs, ws, bytes, stream
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), 0, 1);
  EXPECT(fc_gguf_sample(p, 41, 2, 2, 40, f, nullptr, nullptr, nullptr, nullptr, o, nullptr, p, many, nullptr), 0, 1);
  EXPECT(fc_gguf_sample(nullptr, 40, 1, 0, 40, nullptr, f, i, f, f, nullptr, l, nullptr, 0, nullptr), 0, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, -1, 40, f, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 0, f, f, i, f, f, o, l, p, many, nullptr), E, 0);
  for (int t : {-1, 3, 4}) EXPECT(fc_gguf_sample(p, 40, t, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), U, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 65536, 40, f, f, i, f, f, o, l, p, many, nullptr), R, 0);
  EXPECT(fc_gguf_sample(p, 1 << 25, 0, 2, (1 << 24) + 1, f, f, i, f, f, o, l, p, many, nullptr), R, 0);
  EXPECT(fc_gguf_sample(nullptr, 40, 0, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(mem + 1, 40, 0, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(mem + 2, 40, 2, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 39, 0, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, nullptr, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, nullptr, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, o, l, nullptr, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, o, l, mem + 4, many, nullptr), E, 0);
  const float* odd = (const float*)(mem + 2);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, odd, f, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, odd, i, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, (const int32_t*)odd, f, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, odd, f, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, odd, o, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, (int32_t*)odd, l, p, many, nullptr), E, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, o, (float*)odd, p, many, nullptr), E, 0);
  // the workspace: one byte less is refused, and all that is launched lies in it
  for (int n : {1, 64, 256, 304})
    for (int64_t rows : {1, 3, 128, 65535})
      for (int64_t vocab : {1, 4095, 4096, 4097, 32064, 131073, 1 << 24}) {
        cus = n;
        const int64_t need = fc_gguf_sample_workspace(rows, vocab);
        if (rows == 65535 && vocab == 1 << 24) {          // 2^27 workgroups
          if (need != R) return 2;
          EXPECT(fc_gguf_sample(p, vocab, 0, rows, vocab, f, f, i, f, f, o, l, p, many, nullptr), R, 0);
          continue;
        }
        EXPECT(fc_gguf_sample(p, vocab, 0, rows, vocab, f, f, i, f, f, o, l, p, need - 1, nullptr), E, 0);
        EXPECT(fc_gguf_sample(p, vocab, 0, rows, vocab, f, f, i, f, f, o, l, p, need, nullptr), 0, 1);
        const fcg::SampleArgs& a = fcg::last;
        const int64_t slices = a.slices;
        const int64_t parts = a.row_parts > 1 ? a.row_parts : 0;
        if ((char*)(a.arrived + rows) > (char*)p + need || (char*)a.hist != (char*)p ||
            (char*)(a.slice_tops + rows * slices) > (char*)a.parts || a.row_parts < 1 || a.row_parts > fcg::SAMPLE_MOST_PARTS ||
            (char*)(a.parts + rows * parts * fcg::SAMPLE_PART) > (char*)a.part_n || a.part_n + rows * parts > a.arrived ||
            (char*)(a.hist + rows * slices * fcg::SAMPLE_BINS) > (char*)a.first ||
            (char*)(a.first + rows * slices * fcg::SAMPLE_FIRST) > (char*)a.slice_tops || slices * a.slice < vocab ||
            (slices - 1) * a.slice >= vocab || slices * 512 * rows >= (int64_t)1 << 32) {
          printf("rows %lld, vocab %lld: workspace\n", (long long)rows, (long long)vocab);
          return 1;
        }
      }
  EXPECT(fc_gguf_sample_workspace(-1, 40), E, 0);
  EXPECT(fc_gguf_sample_workspace(1, 0), E, 0);
  EXPECT(fc_gguf_sample_workspace(65536, 40), R, 0);
  EXPECT(fc_gguf_sample_workspace(1, (1 << 24) + 1), R, 0);
  EXPECT(fc_gguf_sample_workspace(0, 40), 0, 0);
  cus = 0;
  EXPECT(fc_gguf_sample_workspace(1, 40), FC_GGUF_EHIP, 0);
  EXPECT(fc_gguf_sample(p, 40, 0, 2, 40, f, f, i, f, f, o, l, p, many, nullptr), FC_GGUF_EHIP, 0);
  printf("ok\n");
  return 0;
}
