// Host check of the C-ABI layer of the 8-bit cache and of append's head norms,
// without a GPU: the HIP runtime and the launchers are stand-ins, and every
// refusal must launch nothing.  Prints "ok" and returns 0, or the first line
// that does not hold.
#include <stdio.h>

#include "serving_api.cpp"

#include "attend_plan.cpp"

static int launches = 0, current = 0;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = current; return hipSuccess; }
hipError_t hipSetDevice(int d) { current = d; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) { *s = hipStreamCaptureStatusNone; return hipSuccess; }
hipError_t hipMallocAsync(void** p, size_t n, hipStream_t) { *p = malloc(n); return *p ? hipSuccess : hipErrorOutOfMemory; }
hipError_t hipFreeAsync(void* p, hipStream_t) { free(p); return hipSuccess; }
}
namespace fcg {
static AppendArgs appended;
static AttendArgs attended;
hipError_t launch_kv_append(const AppendArgs& a, int, int, hipStream_t) { appended = a; ++launches; return hipSuccess; }
hipError_t launch_attend(const AttendArgs& a, const AttendPlan&, int, hipStream_t) { attended = a; ++launches; return hipSuccess; }
hipError_t launch_logits(const LogitsArgs&, int, int, int, hipStream_t) { ++launches; return hipSuccess; }
}  // namespace fcg

#define EXPECT(call, code, count)                                                             \
  do {                                                                                        \
    const int before = launches, got = (call);                                                \
    if (got != (code) || launches - before != (count)) {                                      \
      printf("line %d: %s gave %d, %d launches\n", __LINE__, #call, got, launches - before);  \
      return 1;                                                                               \
    }                                                                                         \
  } while (0)
#define HOLDS(x)                                        \
  do {                                                  \
    if (!(x)) {                                         \
      printf("line %d: %s does not hold\n", __LINE__, #x); \
      return 1;                                         \
    }                                                   \
  } while (0)

int main() {
  alignas(16) static unsigned char mem[1 << 16];
  void* p = mem;
  void* odd = mem + 8;
  const int32_t* i = (const int32_t*)mem;
  const float* f = (const float*)mem;
  const int E = FC_GGUF_EINVAL, U = FC_GGUF_EUNSUPPORTED, R = FC_GGUF_ERANGE;
  fc_gguf_kv_t h = nullptr;
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 0, p, p, p, p, nullptr), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 0, p, p, nullptr, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 0, p, p, p, nullptr, &h), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 0, p, p, odd, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 0, p, p, p, odd, &h), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 0, odd, p, p, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 24, 2, 64, 0, p, p, p, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 80, 0, p, p, p, p, &h), U, 0);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 2, p, p, p, p, &h), U, 0);
  EXPECT(fc_gguf_kv_create8((int64_t)1 << 31, 16, 2, 64, 0, p, p, p, p, &h), R, 0);
  HOLDS(!h);
  EXPECT(fc_gguf_kv_create8(4, 16, 2, 64, 1, p, p, mem + 16, mem + 32, &h), 0, 0);

  // h, q, qs, hq, k, ks, v, vs, T, slots, qn, qns, kn, kns, eps, positions, axes, freq, axis, rot, inter, scale, out, os, stream
#define NORM(T, qn, qns, kn, kns, eps) \
  fc_gguf_kv_append_norm(h, p, 256, 4, p, 128, p, 128, T, i, qn, qns, kn, kns, eps, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr)
  EXPECT(NORM(5, f, 0, f, 64, 1e-6f), 0, 1);
  HOLDS(fcg::appended.kv.k_scale == mem + 16 && fcg::appended.kv.v_scale == mem + 32 && fcg::appended.q_norm == f &&
        fcg::appended.q_norm_stride == 0 && fcg::appended.k_norm_stride == 64 && fcg::appended.eps == 1e-6f);
  EXPECT(NORM(5, nullptr, 7, nullptr, 9, NAN), 0, 1);     // without norms none of it is read
  EXPECT(NORM(5, f, 64, nullptr, 0, 0.f), 0, 1);
  EXPECT(NORM(0, f, 64, nullptr, 0, 0.f), 0, 0);
  for (int64_t s : {-64, 1, 32, 65, 128}) {
    EXPECT(NORM(5, f, s, nullptr, 0, 1e-6f), E, 0);
    EXPECT(NORM(5, nullptr, 0, f, s, 1e-6f), E, 0);
  }
  for (float e : {-1e-6f, INFINITY, -INFINITY, NAN}) EXPECT(NORM(5, f, 0, nullptr, 0, e), E, 0);
  EXPECT(NORM(5, f + 1, 0, nullptr, 0, 1e-6f), E, 0);
  EXPECT(NORM(5, nullptr, 0, f + 2, 0, 1e-6f), E, 0);
  EXPECT(NORM(-1, f, 0, f, 0, 1e-6f), E, 0);
  EXPECT(NORM(((int64_t)1 << 25) + 1, f, 0, f, 0, 1e-6f), R, 0);
  current = 1;
  EXPECT(NORM(5, f, 0, f, 0, 1e-6f), FC_GGUF_EDEVICE, 0);
  current = 0;
  EXPECT(fc_gguf_kv_append_norm(nullptr, p, 256, 4, p, 128, p, 128, 5, i, f, 0, f, 0, 1e-6f, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(fc_gguf_kv_append(h, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), 0, 1);
  HOLDS(!fcg::appended.q_norm && !fcg::appended.k_norm && fcg::appended.kv.k_scale);
  EXPECT(fc_gguf_kv_attend(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), 0, 1);
  HOLDS(fcg::attended.kv.k_scale == mem + 16 && fcg::attended.kv.v_scale == mem + 32);
  EXPECT(fc_gguf_kv_destroy(h), 0, 0);
  EXPECT(fc_gguf_kv_create(4, 16, 2, 64, 1, p, p, &h), 0, 0);
  EXPECT(NORM(5, f, 0, f, 64, 1e-6f), 0, 1);
  HOLDS(!fcg::appended.kv.k_scale && !fcg::appended.kv.v_scale);
  EXPECT(fc_gguf_kv_destroy(h), 0, 0);
  printf("ok\n");
  return 0;
}
