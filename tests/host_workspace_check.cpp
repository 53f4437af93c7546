// Host check of the attention workspace, without a GPU: the plan is the
// library's own, the HIP runtime and the launchers are stand-ins.  Every launch
// must find its counters and partial sums in live memory, also those that a
// captured graph replays after later calls of any size; and after a call of
// given sizes no call of smaller ones may need more.  Prints "ok" and returns
// 0, or the first line that does not hold.
#include <stdio.h>
#include <map>
#include <random>
#include <vector>

#include "serving_api.cpp"

#include "attend_plan.cpp"

static std::map<char*, size_t> live;             // allocations of the stand-in
static int frees = 0, grown = 0;
static bool capturing = false, no_memory = false;
static int cus = 256;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = cus; return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
  *s = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
  return hipSuccess;
}
// (addresses only: nothing reads or writes there)
hipError_t hipMallocAsync(void** p, size_t n, hipStream_t) {
  static char* next = (char*)0x100000000;
  if (no_memory || capturing) return hipErrorOutOfMemory;
  *p = next;
  live[next] = n;
  next += (n + 4095) / 4096 * 4096;
  ++grown;
  return hipSuccess;
}
hipError_t hipFreeAsync(void* p, hipStream_t) {
  ++frees;
  return live.erase((char*)p) ? hipSuccess : hipErrorInvalidValue;
}
}

struct Launch {                                  // what a launch reads and writes of the workspace
  char* arrived;
  char* part;
  size_t counter_bytes, part_bytes;
};
static Launch last;
static bool fresh;
namespace fcg {
hipError_t launch_kv_append(const AppendArgs&, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_logits(const LogitsArgs&, int, int, int, hipStream_t) { return hipSuccess; }
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, int, hipStream_t) {
  const size_t bytes = attend_workspace_bytes(a, p);
  const bool counted = p.stream_rows > 0 && !p.whole;
  last = {(char*)a.arrived, (char*)a.part, counted ? (size_t)a.seqs * a.kv.kv_heads * 4 : 0, bytes};
  fresh = a.fresh;
  return hipSuccess;
}
}  // namespace fcg

static bool inside(char* p, size_t n) {
  if (n == 0) return true;
  auto it = live.upper_bound(p);
  if (it == live.begin()) return false;
  --it;
  return p + n <= it->first + it->second;
}
static bool sound(const Launch& x) {
  return inside(x.arrived, x.counter_bytes) && inside(x.part, x.part_bytes) &&
         (x.counter_bytes == 0 || x.part_bytes == 0 || x.arrived + x.counter_bytes <= x.part);
}

struct Size {
  int64_t T, seqs, max_q, width;
  int heads, window;
};
static fc_gguf_kv_t kv;
static int attend(const Size& s) {
  alignas(16) static unsigned char mem[64];
  const int32_t* i = (const int32_t*)mem;
  const int64_t stride = (int64_t)s.heads * kv->kv.head_dim;
  return fc_gguf_kv_attend(kv, mem, stride, s.heads, s.T, i, i, s.seqs, i, s.width, s.width, s.max_q, .125f, s.window, mem, stride,
                           nullptr, nullptr);
}

#define CHECK(x)                                                                                          \
  do {                                                                                                    \
    if (!(x)) {                                                                                           \
      printf("line %d: %s\n", __LINE__, #x);                                                              \
      return 1;                                                                                           \
    }                                                                                                     \
  } while (0)

int main() {
  alignas(16) static unsigned char mem[64];
  auto make = [&](int page, int kv_heads, int dim) { return fc_gguf_kv_create(100000, page, kv_heads, dim, 0, mem, mem, &kv) == 0; };
  // after the largest chunk, every smaller call stays in the memory that is there, also while a graph is captured
  CHECK(make(64, 8, 128));
  CHECK(attend({4096, 1, 4096, 512, 32, 0}) == 0 && sound(last));
  {
    const int before = grown;
    for (int64_t T = 1; T <= 4096; T += T < 300 ? 1 : 61)
      for (int64_t width : {1, 16, 100, 512})
        for (int window : {0, 1, 300, 3000}) {
          capturing = (T + width) & 1;
          CHECK(attend({T, 1, T, width, 32, window}) == 0 && sound(last));
        }
    capturing = false;
    CHECK(grown == before && frees == 0);
  }
  CHECK(fc_gguf_kv_destroy(kv) == 0 && live.empty());

  // a captured decode step, then calls that need more: the graph's memory stays
  CHECK(make(64, 8, 128));
  CHECK(attend({1, 1, 1, 512, 32, 0}) == 0);
  capturing = true;
  CHECK(attend({1, 1, 1, 512, 32, 0}) == 0);
  capturing = false;
  const Launch one = last;
  CHECK(sound(one) && one.part_bytes > 0);
  CHECK(attend({64, 1, 64, 512, 32, 0}) == 0 && sound(last) && sound(one));
  CHECK(attend({40, 40, 1, 512, 32, 0}) == 0 && sound(last) && sound(one));
  capturing = true;
  CHECK(attend({40, 40, 1, 512, 32, 0}) == 0);
  capturing = false;
  const Launch two = last;
  CHECK(attend({2000, 700, 1024, 512, 64, 0}) == 0 && sound(last) && sound(one) && sound(two));
  // growth in a capture and without memory is refused, and changes nothing
  capturing = true;
  CHECK(attend({4000, 900, 1000, 512, 64, 0}) == FC_GGUF_ENOMEM);
  capturing = false;
  no_memory = true;
  CHECK(attend({4000, 900, 1000, 512, 64, 0}) == FC_GGUF_ENOMEM);
  no_memory = false;
  CHECK(sound(one) && sound(two) && attend({1, 1, 1, 512, 32, 0}) == 0 && sound(last));
  CHECK(fc_gguf_kv_destroy(kv) == 0 && live.empty());

  // a call that splits nothing needs no workspace: also the first one, in a capture
  CHECK(make(16, 2, 64));
  capturing = true;
  CHECK(attend({3, 3, 1, 20, 4, 0}) == 0 && sound(last));
  CHECK(attend({3, 3, 1, 2000, 4, 0}) == FC_GGUF_ENOMEM);
  capturing = false;
  CHECK(attend({3, 3, 1, 2000, 4, 0}) == 0 && sound(last) && fresh);
  CHECK(attend({3, 3, 1, 2000, 4, 0}) == 0 && sound(last) && !fresh);
  CHECK(fc_gguf_kv_destroy(kv) == 0 && live.empty());

  // of two calls of which one is smaller in every size, the smaller never needs more
  std::mt19937_64 g(1);
  auto up_to = [&](int64_t n) { return (int64_t)std::exp(std::uniform_real_distribution<>(0, std::log((double)n + .99))(g)); };
  const int dims[] = {64, 96, 128, 256};
  for (int n = 0; n < 3000; ++n) {
    cus = n % 3 ? 256 : 32 << (n % 4);
    CHECK(make(16 << n % 5, (int)up_to(n % 2 ? 16 : 600), dims[g() % 4]));
    const int hk = kv->kv.kv_heads;
    Size big = {up_to(20000), up_to(300), 0, up_to((1 << 18) >> kv->kv.page_shift), hk * (int)up_to(20), 0};
    big.max_q = up_to(big.T);
    if (attend(big) != 0) {
      CHECK(fc_gguf_kv_destroy(kv) == 0);
      continue;
    }
    CHECK(sound(last));
    const int before = grown;
    for (int k = 0; k < 60; ++k) {
      Size s = {up_to(big.T), up_to(big.seqs), 0, up_to(big.width), hk * (int)up_to(big.heads / hk), 0};
      if (k % 4 == 0) s.heads = big.heads;
      if (k % 5 == 0) s.width = big.width;
      s.max_q = up_to(s.T < big.max_q ? s.T : big.max_q);
      s.window = k % 2 ? (int)up_to(10000) : 0;
      capturing = k % 3 == 0;
      CHECK(attend(s) == 0 && sound(last));
      capturing = false;
      CHECK(grown == before);
    }
    CHECK(fc_gguf_kv_destroy(kv) == 0 && live.empty());
  }
  printf("ok\n");
  return 0;
}
