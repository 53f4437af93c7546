// Host check of the serving operators' C-ABI layer, without a GPU: the HIP
// runtime calls and the launchers are stand-ins that count, so that every
// refusal can be seen to launch nothing.  Prints "ok" and returns 0, or the
// first line that does not hold.
#include <stdio.h>
#include <vector>

#include "serving_api.cpp"

static int launches = 0, current = 0;
static bool no_memory = false;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = current; return hipSuccess; }
hipError_t hipSetDevice(int d) { current = d; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipMallocAsync(void** p, size_t n, hipStream_t) {
  if (no_memory) return hipErrorOutOfMemory;
  *p = malloc(n);
  return hipSuccess;
}
hipError_t hipFreeAsync(void* p, hipStream_t) { free(p); return hipSuccess; }
}
namespace fcg {
static AttendArgs last;
hipError_t launch_kv_append(const AppendArgs&, int, int, hipStream_t) { ++launches; return hipSuccess; }
AttendPlan attend_plan(const AttendArgs&, int) { AttendPlan p = {}; p.splits = 3; return p; }
size_t attend_workspace_bytes(const AttendArgs&, const AttendPlan&) { return 4096; }
hipError_t launch_attend(const AttendArgs& a, const AttendPlan&, int, hipStream_t) { last = a; ++launches; return hipSuccess; }
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

int main() {
  alignas(16) static unsigned char mem[1 << 16];
  void* p = mem;
  void* odd = mem + 2;
  const int32_t* i = (const int32_t*)mem;
  const float* f = (const float*)mem;
  fc_gguf_kv_t h = nullptr;
  const int E = FC_GGUF_EINVAL, U = FC_GGUF_EUNSUPPORTED, R = FC_GGUF_ERANGE;
  EXPECT(fc_gguf_kv_create(4, 16, 2, 64, 0, p, p, nullptr), E, 0);
  EXPECT(fc_gguf_kv_create(0, 16, 2, 64, 0, p, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create(4, 16, 0, 64, 0, p, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create(4, 16, 2, 64, 0, nullptr, p, &h), E, 0);
  EXPECT(fc_gguf_kv_create(4, 16, 2, 64, 0, p, odd, &h), E, 0);
  for (int ps : {0, -16, 1, 8, 24, 48, 512}) EXPECT(fc_gguf_kv_create(4, ps, 2, 64, 0, p, p, &h), E, 0);
  for (int d : {0, -64, 16, 80, 112, 192, 512}) EXPECT(fc_gguf_kv_create(4, 16, 2, d, 0, p, p, &h), U, 0);
  for (int t : {-1, 2, 3}) EXPECT(fc_gguf_kv_create(4, 16, 2, 64, t, p, p, &h), U, 0);
  EXPECT(fc_gguf_kv_create((int64_t)1 << 31, 16, 2, 64, 0, p, p, &h), R, 0);
  EXPECT(fc_gguf_kv_create(4, 16, 1025, 64, 0, p, p, &h), R, 0);
  if (h) return 2;
  EXPECT(fc_gguf_kv_create(4, 16, 2, 64, 1, p, p, &h), 0, 0);

#define APPEND(...) fc_gguf_kv_append(__VA_ARGS__)
  // h, q, qs, hq, k, ks, v, vs, T, slots, positions, axes, freq, axis, rot, inter, scale, out, os, stream
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), 0, 1);
  EXPECT(APPEND(h, nullptr, 0, 0, p, 128, p, 128, 5, i, i, 3, f, i, 16, 1, 1.f, nullptr, 0, nullptr), 0, 1);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, nullptr, 0, nullptr, nullptr, 7, 9, 1.f, p, 256, nullptr), 0, 1);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 0, nullptr, nullptr, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), 0, 0);
  EXPECT(APPEND(nullptr, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, -1, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, -4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 248, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 260, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, odd, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, nullptr, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 120, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, nullptr, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, nullptr, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 0, f, nullptr, 64, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 17, f, nullptr, 64, 0, 1.f, p, 256, nullptr), R, 0);
  for (int rot : {0, -16, 8, 24, 80, 128})
    EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, rot, 0, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 2, 1.f, p, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, nullptr, 256, nullptr), E, 0);
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, ((int64_t)1 << 30) + 1, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), R, 0);
  current = 1;
  EXPECT(APPEND(h, p, 256, 4, p, 128, p, 128, 5, i, i, 1, f, nullptr, 64, 0, 1.f, p, 256, nullptr), FC_GGUF_EDEVICE, 0);
  current = 0;

#define ATTEND(...) fc_gguf_kv_attend(__VA_ARGS__)
  // h, q, qs, hq, T, cu, lens, seqs, table, ts, tw, max_q, scale, window, out, os, lse, stream
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), 0, 1);
  if (fcg::last.group != 2 || fcg::last.max_q != 4 || !fcg::last.part) return 3;
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 99, .125f, 0, p, 256, nullptr, nullptr), 0, 1);
  if (fcg::last.max_q != 6) return 4;
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, nullptr, 0, 0, 4, .125f, 0, p, 256, nullptr, nullptr), 0, 1);
  EXPECT(ATTEND(h, nullptr, 0, 4, 0, nullptr, nullptr, 2, nullptr, 3, 3, 4, .125f, 0, nullptr, 0, nullptr, nullptr), 0, 0);
  EXPECT(ATTEND(h, nullptr, 0, 4, 6, nullptr, nullptr, 0, nullptr, 3, 3, 4, .125f, 0, nullptr, 0, nullptr, nullptr), 0, 0);
  EXPECT(ATTEND(nullptr, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 3, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 0, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, nullptr, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, nullptr, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, nullptr, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 2, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, -1, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, -4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, -1, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 252, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, odd, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, (float*)odd, nullptr), E, 0);
  for (float s : {0.f, -1.f, INFINITY, NAN})
    EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, s, 0, p, 256, nullptr, nullptr), E, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 65536, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), R, 0);
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 1 << 28, 1 << 28, 4, .125f, 0, p, 256, nullptr, nullptr), R, 0);
  EXPECT(ATTEND(h, p, 256, 4, 1 << 30, i, i, 60000, i, 3, 3, 1 << 20, .125f, 0, p, 256, nullptr, nullptr), R, 0);
  current = 1;
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), FC_GGUF_EDEVICE, 0);
  current = 0;
  EXPECT(fc_gguf_kv_destroy(h), 0, 0);
  EXPECT(fc_gguf_kv_create(4, 16, 2, 64, 1, p, p, &h), 0, 0);
  no_memory = true;
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), FC_GGUF_ENOMEM, 0);
  no_memory = false;
  EXPECT(ATTEND(h, p, 256, 4, 6, i, i, 2, i, 3, 3, 4, .125f, 0, p, 256, nullptr, nullptr), 0, 1);
  EXPECT(fc_gguf_kv_destroy(h), 0, 0);
  EXPECT(fc_gguf_kv_destroy(nullptr), 0, 0);

#define LOGITS(...) fc_gguf_logits(__VA_ARGS__)
  // x, xs, dtype, rows, vocab, tokens, ts, lens, prompts, rep, freq, pres, offsets, ids, values, n, mask, ms, out, os, odt, stream
  const uint32_t* w = (const uint32_t*)mem;
  EXPECT(LOGITS(p, 40, 0, 2, 40, i, 5, i, i, f, f, f, i, i, f, 7, w, 2, p, 40, 0, nullptr), 0, 1);
  EXPECT(LOGITS(p, 40, 0, 2, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, mem + 64, 41, 2, nullptr), 0, 1);
  EXPECT(LOGITS(nullptr, 40, 0, 0, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, nullptr, 40, 0, nullptr), 0, 0);
  EXPECT(LOGITS(p, 40, 0, -1, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 0, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 39, 0, 2, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 41, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 2, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 2, 2, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, mem + 64, 40, 0, nullptr), U, 0);
  EXPECT(LOGITS(p, 40, 3, 2, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 3, nullptr), U, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, i, 5, nullptr, nullptr, f, f, f, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, i, -5, i, nullptr, f, f, f, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, nullptr, 0, nullptr, nullptr, f, f, f, i, nullptr, f, 3, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, nullptr, 0, nullptr, nullptr, f, f, f, i, i, f, -3, nullptr, 0, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 2, 40, nullptr, 0, nullptr, nullptr, f, f, f, nullptr, nullptr, nullptr, 0, w, 1, p, 40, 0, nullptr), E, 0);
  EXPECT(LOGITS(p, 40, 0, 65536, 40, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr, 0, p, 40, 0, nullptr), R, 0);
  printf("ok\n");
  return 0;
}
