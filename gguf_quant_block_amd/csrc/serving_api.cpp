// C-ABI of the serving operators (declarations and contracts in
// include/fc_gguf.h): the paged key/value cache, attention over it and the
// processing of logits.  Host logic only: argument checks and the workspace of
// the split sums.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <new>

#include "fc_gguf.h"
#include "serving.h"

// A workspace that a captured graph uses, kept until the handle goes.
struct KeptWorkspace {
  void* p;
  KeptWorkspace* next;
};

struct fc_gguf_kv {
  fcg::KvPages kv = {};
  int dtype = 0;
  int device = 0;
  int num_cu = 256;
  void* ws = nullptr;           // the attention's counters, then its partial sums
  size_t ws_bytes = 0;
  int64_t counters = 0;
  bool fresh = false;           // the counters are to be cleared by the next call
  bool graphed = false;         // a captured call uses it
  KeptWorkspace* kept = nullptr;
};

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;

bool on(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// FC_GGUF_TEST_FAIL_ALLOC: "workspace" or "all" makes the workspace's growth fail
bool fail_workspace() {
  const char* p = getenv("FC_GGUF_TEST_FAIL_ALLOC");
  return p && (!strcmp(p, "all") || !strcmp(p, "workspace"));
}

// CUs of the current device, asked for once per device (0: an error)
int cus_of_current() {
  static std::atomic<int> known[64];
  int dev = -1, n = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

int check_kv_device(const fc_gguf_kv* h) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return FC_GGUF_EHIP;
  return dev == h->device ? FC_GGUF_OK : FC_GGUF_EDEVICE;
}

size_t counter_bytes(int64_t counters) { return ((size_t)counters * 4 + 255) / 256 * 256; }

// Sees to a workspace of `counters` and `need` bytes.  Outside a capture it is
// made large enough for `bound` bytes, which no smaller call exceeds, so that
// smaller calls never move it.  It grows on the call's stream: released to and
// taken from the device's stream-ordered pool, so that the growth waits for
// that stream only.  One that a captured call uses is not released but kept for
// the graph, whose launches leave its counters at 0.  While the stream is
// captured nothing grows: the memory would belong to the graph.
int ensure_kv_ws(fc_gguf_kv* h, int64_t counters, size_t need, size_t bound, hipStream_t st, bool* in_capture) {
  *in_capture = false;
  if (bound == 0) return FC_GGUF_OK;
  auto holds = [&](size_t bytes) { return counters <= h->counters && counter_bytes(h->counters) + bytes <= h->ws_bytes; };
  hipStreamCaptureStatus captured = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(st, &captured) == hipSuccess && captured != hipStreamCaptureStatusNone) {
    *in_capture = true;
    if (need == 0) return FC_GGUF_OK;
    if (!holds(need)) return FC_GGUF_ENOMEM;
    h->graphed = true;
    return FC_GGUF_OK;
  }
  if (holds(bound)) return FC_GGUF_OK;
  if (fail_workspace()) return FC_GGUF_ENOMEM;
  if (counters < h->counters) counters = h->counters;
  if (counters < 1024) counters = 1024;
  const size_t had = h->ws ? h->ws_bytes - counter_bytes(h->counters) : 0;
  const size_t total = counter_bytes(counters) + (bound > had ? bound : had);
  KeptWorkspace* keep = nullptr;
  if (h->graphed && !(keep = new (std::nothrow) KeptWorkspace)) return FC_GGUF_ENOMEM;
  void* ws = nullptr;
  if (hipMallocAsync(&ws, total, st) != hipSuccess) {
    (void)hipGetLastError();     // (reported by the code: not left behind as well)
    delete keep;
    return FC_GGUF_ENOMEM;
  }
  hipError_t e = hipSuccess;
  if (keep) {
    *keep = {h->ws, h->kept};
    h->kept = keep;
  } else if (h->ws) {
    e = hipFreeAsync(h->ws, st);
  }
  h->ws = ws;
  h->ws_bytes = total;
  h->counters = counters;
  h->fresh = true;
  h->graphed = false;
  return e == hipSuccess ? FC_GGUF_OK : FC_GGUF_EHIP;
}

// a [tokens][heads][D] argument: 16-byte pieces, rows that do not overlap
bool rows_ok(const void* p, int64_t stride, int64_t width) {
  return p && on(p, 16) && stride >= width && stride % 8 == 0;
}

}  // namespace

extern "C" {

int fc_gguf_kv_create(int64_t pages, int page_size, int kv_heads, int head_dim, int dtype, void* k_pages,
                      void* v_pages, fc_gguf_kv_t* out) {
  if (!out) return FC_GGUF_EINVAL;
  *out = nullptr;
  if (pages <= 0 || kv_heads <= 0 || !k_pages || !v_pages || !on(k_pages, 16) || !on(v_pages, 16))
    return FC_GGUF_EINVAL;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return FC_GGUF_EINVAL;
  if (dtype != FC_GGUF_F16 && dtype != FC_GGUF_BF16) return FC_GGUF_EUNSUPPORTED;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 256) return FC_GGUF_EUNSUPPORTED;
  if (pages >= ((int64_t)1 << 31) || kv_heads > 1024) return FC_GGUF_ERANGE;
  fc_gguf_kv* h = new (std::nothrow) fc_gguf_kv();
  if (!h) return FC_GGUF_ENOMEM;
  h->kv.k = k_pages;
  h->kv.v = v_pages;
  h->kv.pages = pages;
  h->kv.page_shift = __builtin_ctz((unsigned)page_size);
  h->kv.kv_heads = kv_heads;
  h->kv.head_dim = head_dim;
  h->dtype = dtype;
  hipError_t e = hipGetDevice(&h->device);
  if (e == hipSuccess)
    e = hipDeviceGetAttribute(&h->num_cu, hipDeviceAttributeMultiprocessorCount, h->device);
  if (e != hipSuccess) {
    delete h;
    return FC_GGUF_EHIP;
  }
  *out = h;
  return FC_GGUF_OK;
}

int fc_gguf_kv_destroy(fc_gguf_kv_t h) {
  if (!h) return FC_GGUF_OK;
  if (h->ws) {
    // the handle's device, whichever is current: its work must end before the
    // workspaces are freed
    int cur = -1;
    const bool switched =
        hipGetDevice(&cur) == hipSuccess && cur != h->device && hipSetDevice(h->device) == hipSuccess;
    (void)hipDeviceSynchronize();                  // best effort: the handle goes anyway
    (void)hipFreeAsync(h->ws, nullptr);
    while (KeptWorkspace* k = h->kept) {
      (void)hipFreeAsync(k->p, nullptr);
      h->kept = k->next;
      delete k;
    }
    (void)hipStreamSynchronize(nullptr);
    if (switched) (void)hipSetDevice(cur);
  }
  delete h;
  return FC_GGUF_OK;
}

int fc_gguf_kv_append(fc_gguf_kv_t h, const void* q, int64_t q_stride, int q_heads, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, int64_t T, const int32_t* slots,
                      const int32_t* positions, int axes, const float* inv_freq, const int32_t* pair_axis,
                      int rot_dim, int interleaved, float rope_scale, void* q_out, int64_t q_out_stride,
                      void* stream) {
  if (!h || T < 0 || q_heads < 0) return FC_GGUF_EINVAL;
  if (const int rc = check_kv_device(h); rc != FC_GGUF_OK) return rc;
  const int D = h->kv.head_dim, hk = h->kv.kv_heads;
  // (a launch has under 2^32 threads: 512 for 8 tokens)
  if (q_heads > 65536 || T > ((int64_t)1 << 25)) return FC_GGUF_ERANGE;
  if (inv_freq) {
    if (rot_dim <= 0 || rot_dim > D || rot_dim % 16 || axes < 1 || (interleaved != 0 && interleaved != 1) ||
        !on(inv_freq, 4) || (pair_axis && !on(pair_axis, 4)))
      return FC_GGUF_EINVAL;
    if (axes > 16) return FC_GGUF_ERANGE;
  }
  if (T == 0) return FC_GGUF_OK;
  if (inv_freq && (!positions || !on(positions, 4))) return FC_GGUF_EINVAL;
  if (!slots || !on(slots, 4) || !rows_ok(k, k_stride, (int64_t)hk * D) || !rows_ok(v, v_stride, (int64_t)hk * D))
    return FC_GGUF_EINVAL;
  if (q_heads && (!rows_ok(q, q_stride, (int64_t)q_heads * D) || !rows_ok(q_out, q_out_stride, (int64_t)q_heads * D)))
    return FC_GGUF_EINVAL;
  fcg::AppendArgs a = {};
  a.kv = h->kv;
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.q_out = (uint16_t*)q_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.o_stride = q_out_stride;
  a.slots = slots;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.pair_axis = pair_axis;
  a.T = T;
  a.q_heads = q_heads;
  a.rot = inv_freq ? rot_dim : 0;
  a.axes = axes;
  a.interleaved = interleaved;
  a.rope_scale = rope_scale;
  return fcg::launch_kv_append(a, h->dtype, h->num_cu, (hipStream_t)stream) == hipSuccess ? FC_GGUF_OK
                                                                                         : FC_GGUF_EHIP;
}

int fc_gguf_kv_attend(fc_gguf_kv_t h, const void* q, int64_t q_stride, int q_heads, int64_t T,
                      const int32_t* cu_q, const int32_t* kv_lens, int64_t seqs, const int32_t* table,
                      int64_t table_stride, int64_t table_width, int64_t max_q, float scale, int window,
                      void* out, int64_t out_stride, float* lse, void* stream) {
  if (!h || T < 0 || seqs < 0 || q_heads <= 0 || q_heads % h->kv.kv_heads || max_q < 0 || table_width < 0 ||
      table_stride < table_width || window < 0 || !(scale > 0.f) || !isfinite(scale))
    return FC_GGUF_EINVAL;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634074);
  if (!isfinite(scale_log2) || window > kMaxTokens) return FC_GGUF_ERANGE;
  if (const int rc = check_kv_device(h); rc != FC_GGUF_OK) return rc;
  if (T > kMaxTokens || q_heads > 65536 || seqs > 65535 || max_q > kMaxTokens ||
      table_width > (kMaxTokens >> h->kv.page_shift))
    return FC_GGUF_ERANGE;
  if (T == 0 || seqs == 0 || max_q == 0) return FC_GGUF_OK;
  const int64_t width = (int64_t)q_heads * h->kv.head_dim;
  if (!rows_ok(q, q_stride, width) || !rows_ok(out, out_stride, width) || !cu_q || !kv_lens || !on(cu_q, 4) ||
      !on(kv_lens, 4) || (table_width && (!table || !on(table, 4))) || (lse && !on(lse, 4)))
    return FC_GGUF_EINVAL;
  fcg::AttendArgs a = {};
  a.kv = h->kv;
  a.q = (const uint16_t*)q;
  a.o = (uint16_t*)out;
  a.lse = lse;
  a.q_stride = q_stride;
  a.o_stride = out_stride;
  a.cu_q = cu_q;
  a.kv_lens = kv_lens;
  a.table = table;
  a.table_stride = table_stride;
  a.T = T;
  a.table_w = (int)table_width;
  a.seqs = (int)seqs;
  a.q_heads = q_heads;
  a.group = q_heads / h->kv.kv_heads;
  a.max_q = (int)(max_q < T ? max_q : T);
  a.window = window;
  a.scale_log2 = scale_log2;
  // A launch has under 2^32 threads: 512 for each tile of at least 128 rows
  // that T tokens of seqs sequences can have, and for each sequence that is not
  // split.  (The splits and their join are launched for few tiles only.)
  if ((int64_t)a.max_q * a.group > kMaxTokens || fcg::tile_count(a, 128) * h->kv.kv_heads >= fcg::kMaxWorkgroups)
    return FC_GGUF_ERANGE;
  const fcg::AttendPlan p = fcg::attend_plan(a, h->num_cu);
  const size_t need = fcg::attend_workspace_bytes(a, p), bound = fcg::attend_workspace_bound(a, h->num_cu);
  bool in_capture;
  const int rc = ensure_kv_ws(h, seqs * h->kv.kv_heads, need, bound > need ? bound : need, (hipStream_t)stream, &in_capture);
  if (rc != FC_GGUF_OK) return rc;
  if (need || (h->fresh && !in_capture)) {
    a.arrived = (uint32_t*)h->ws;
    a.counters = h->counters;
    a.fresh = h->fresh;
    a.part = (float*)((char*)h->ws + counter_bytes(h->counters));
  }
  if (fcg::launch_attend(a, p, h->dtype, (hipStream_t)stream) != hipSuccess) return FC_GGUF_EHIP;
  if (!in_capture) h->fresh = false;       // (what is captured has not run yet)
  return FC_GGUF_OK;
}

int fc_gguf_logits(const void* x, int64_t x_stride, int dtype, int64_t rows, int64_t vocab,
                   const int32_t* tokens, int64_t tokens_stride, const int32_t* lens,
                   const int32_t* prompt_lens, const float* repetition, const float* frequency,
                   const float* presence, const int32_t* bias_offsets, const int32_t* bias_ids,
                   const float* bias_values, int64_t bias_count, const uint32_t* mask, int64_t mask_stride,
                   void* out, int64_t out_stride, int out_dtype, void* stream) {
  if (rows < 0 || vocab <= 0) return FC_GGUF_EINVAL;
  if (dtype != FC_GGUF_F16 && dtype != FC_GGUF_BF16 && dtype != FC_GGUF_F32) return FC_GGUF_EUNSUPPORTED;
  if (out_dtype != dtype && out_dtype != FC_GGUF_F32) return FC_GGUF_EUNSUPPORTED;
  if (rows > 65535 || vocab > kMaxTokens || tokens_stride > kMaxTokens) return FC_GGUF_ERANGE;
  if (rows == 0) return FC_GGUF_OK;
  const size_t es = dtype == FC_GGUF_F32 ? 4 : 2, os = out_dtype == FC_GGUF_F32 ? 4 : 2;
  if (!x || !out || !on(x, es) || !on(out, os) || x_stride < vocab || out_stride < vocab) return FC_GGUF_EINVAL;
  if (x == out && (x_stride != out_stride || es != os)) return FC_GGUF_EINVAL;
  if (tokens) {
    if (!lens || tokens_stride < 0 || !on(tokens, 4) || !on(lens, 4) || (prompt_lens && !on(prompt_lens, 4)))
      return FC_GGUF_EINVAL;
  }
  if (bias_offsets) {
    if (bias_count < 0 || !on(bias_offsets, 4)) return FC_GGUF_EINVAL;
    if (bias_count && (!bias_ids || !bias_values || !on(bias_ids, 4) || !on(bias_values, 4))) return FC_GGUF_EINVAL;
  }
  if (mask && (!on(mask, 4) || mask_stride < (vocab + 31) / 32)) return FC_GGUF_EINVAL;
  if ((repetition && !on(repetition, 4)) || (frequency && !on(frequency, 4)) || (presence && !on(presence, 4)))
    return FC_GGUF_EINVAL;
  const int num_cu = cus_of_current();
  if (num_cu <= 0) return FC_GGUF_EHIP;
  fcg::LogitsArgs a = {};
  a.x = x;
  a.out = out;
  a.rows = rows;
  a.vocab = vocab;
  a.x_stride = x_stride;
  a.o_stride = out_stride;
  a.tokens = tokens;
  a.tokens_stride = tokens_stride;
  a.lens = lens;
  a.prompt_lens = prompt_lens;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_offsets = bias_offsets;
  a.bias_ids = bias_ids;
  a.bias_values = bias_values;
  a.bias_count = bias_count;
  a.mask = mask;
  a.mask_stride = mask_stride;
  return fcg::launch_logits(a, dtype, out_dtype, num_cu, (hipStream_t)stream) == hipSuccess ? FC_GGUF_OK
                                                                                            : FC_GGUF_EHIP;
}

}  // extern "C"
