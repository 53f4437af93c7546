// Host check of which sizes of an attention call are taken, without a GPU: the
// plan is the library's own.  Every call that is taken must launch grids of
// under 2^32 threads and tiles that the kernels can count in 32 bits; steps of
// a long chunk beside hundreds of single tokens must be taken.  An append takes
// 2^25 tokens and no more.  Prints "ok" and
// returns 0, or the first line that does not hold.
#include <stdio.h>
#include <random>

#include "serving_api.cpp"

#include "attend_plan.cpp"

extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) { *s = hipStreamCaptureStatusNone; return hipSuccess; }
hipError_t hipMallocAsync(void** p, size_t, hipStream_t) { *p = (void*)0x100000000; return hipSuccess; }
hipError_t hipFreeAsync(void*, hipStream_t) { return hipSuccess; }
}
static bool fits = true;
static int64_t tiles = 0;
namespace fcg {
hipError_t launch_kv_append(const AppendArgs&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_logits(const LogitsArgs&, int, int, int, hipStream_t) { return hipSuccess; }
// the grids of launch_attend
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, int, hipStream_t) {
  const int64_t hk = a.kv.kv_heads, top = (int64_t)1 << 32;
  auto threads = [&](int64_t wgs, int64_t each) { if (wgs < 1 || wgs * each >= top) fits = false; };
  tiles = 0;
  if (p.tile_rows) {
    tiles = tile_count(a, p.tile_rows) * hk * p.tile_splits;
    threads(tiles, p.tile_rows * 2);
    if (p.tile_splits > 1) threads(tile_count(a, 1024 / a.kv.head_dim) * hk, 256);
    // what find_tile adds up over 64 sequences
    if ((int64_t)a.max_q * a.group > (int64_t)1 << 30) fits = false;
  }
  if (p.stream_rows) threads((int64_t)p.splits * hk, at_waves(a.kv.head_dim) * 64);
  return hipSuccess;
}
}  // namespace fcg

int main() {
  alignas(16) static unsigned char mem[64];
  const int32_t* i = (const int32_t*)mem;
  fc_gguf_kv_t kv = nullptr;
  auto attend = [&](int64_t T, int64_t seqs, int64_t max_q, int64_t width, int heads) {
    const int64_t stride = (int64_t)heads * kv->kv.head_dim;
    return fc_gguf_kv_attend(kv, mem, stride, heads, T, i, i, seqs, i, width, width, max_q, .125f, 0, mem, stride, nullptr, nullptr);
  };
  // a chunk beside single tokens
  struct { int hk, heads; int64_t chunk, seqs; } mixed[] = {{8, 32, 8192, 512}, {8, 64, 8192, 256}, {8, 64, 16384, 4000}, {1, 16, 65536, 256}};
  for (auto& m : mixed) {
    if (fc_gguf_kv_create(100000, 64, m.hk, 128, 0, mem, mem, &kv)) return 1;
    const int rc = attend(m.chunk + m.seqs - 1, m.seqs, m.chunk, 1024, m.heads);
    if (rc != 0 || !fits || tiles > (m.chunk + m.seqs) * m.heads / 128 + (m.seqs + 1) * m.hk) {
      printf("%d heads, %d key heads, %ld tokens beside %ld: code %d, fits %d, %ld tiles\n", m.heads, m.hk, (long)m.chunk, (long)m.seqs - 1,
             rc, (int)fits, (long)tiles);
      return 1;
    }
    fc_gguf_kv_destroy(kv);
  }
  // tokens of an append: 2^25
  if (fc_gguf_kv_create(100000, 64, 2, 64, 0, mem, mem, &kv)) return 1;
  for (int64_t over : {0, 1}) {
    const int rc = fc_gguf_kv_append(kv, nullptr, 0, 0, mem, 128, mem, 128, ((int64_t)1 << 25) + over, i, nullptr, 1, nullptr, nullptr, 0, 0,
                                     1.f, nullptr, 0, nullptr);
    if (rc != (over ? FC_GGUF_ERANGE : 0)) {
      printf("2^25 + %ld tokens: code %d\n", (long)over, rc);
      return 1;
    }
  }
  fc_gguf_kv_destroy(kv);
  std::mt19937_64 g(1);
  auto up_to = [&](int64_t n) { return (int64_t)std::exp(std::uniform_real_distribution<>(0, std::log((double)n + .99))(g)); };
  const int dims[] = {64, 96, 128, 256};
  int taken = 0;
  for (int n = 0; n < 200000; ++n) {
    const int hk = (int)up_to(1024), dim = dims[g() % 4];
    if (fc_gguf_kv_create(100000, 16 << n % 5, hk, dim, 0, mem, mem, &kv)) return 1;
    const int heads = hk * (int)up_to(65536 / hk);
    const int64_t T = up_to((int64_t)1 << 30), seqs = up_to(65535), max_q = up_to(T);
    const int rc = attend(T, seqs, max_q, up_to(((int64_t)1 << 30) >> kv->kv.page_shift), heads);
    if ((rc != 0 && rc != FC_GGUF_ERANGE) || !fits) {
      printf("T %ld seqs %ld max_q %ld heads %d of %d, %d: code %d, fits %d\n", (long)T, (long)seqs, (long)max_q, heads, dim, hk, rc, (int)fits);
      return 1;
    }
    taken += rc == 0;
    fc_gguf_kv_destroy(kv);
  }
  if (taken < 20000) {
    printf("%d taken\n", taken);
    return 1;
  }
  printf("ok\n");
  return 0;
}
