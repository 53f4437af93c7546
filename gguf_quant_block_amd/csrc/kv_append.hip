// Appending keys and values to the paged cache, with the rotation of queries
// and keys on the way.
//
//   angle(t, j) = position[axis[j]][t] * inv_freq[j]
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin)      for pair j of a head
//
// Bound by HBM: q, k and v are read once, the rotated q and the cache entries
// written once.  The angles are products in f64, reduced to a turn there:
// at position 10^5 an f32 product would be off by up to 0.004 rad.  They are
// taken once per token and pair into LDS and serve every head.  The rotation
// is in f32 with one rounding to the cache's type.  Measured: 4096 tokens, 32
// query and 8 key heads of 128: 22.3 us, 4.5 TB/s (a copy reaches 4.75; HBM
// writes 1.11 of the bytes, for cache lines that several workgroups fill), 29.6
// where nothing is cached; 2500 tokens on three axes 16.2 us, and 24.2; one
// token 5.3 us, most of it the launch.
//
// A workgroup takes tokens_per_wg consecutive tokens (1 for a decode step,
// where latency counts and the heads are spread over y_splits workgroups; up
// to 8 for a prompt).  Q and K are handled in units of 16 elements, the two
// pieces of 8 that hold 8 pairs.  V pieces hold 8 tokens of one dimension, so
// V is handled in runs: consecutive tokens whose slots follow each other
// inside one piece row.  A run belongs to the workgroup in whose tokens it
// begins; a thread reads 8 dimensions of its up to 8 tokens and turns them in
// registers, so that a whole piece is one 16-byte store wherever the prompt
// begins inside a page.
#include "serving.h"

namespace fcg {
namespace {

constexpr int AP_MAX_TOKENS = 8;
constexpr int AP_MAX_HALF = 128;     // rotated pairs of a head

template <class E>
__device__ __forceinline__ void rotate8(u32x4& a, u32x4& b, const float2* cs, bool interleaved) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo2f<E>(a[i]);
    x[2 * i + 1] = hi2f<E>(a[i]);
    x[8 + 2 * i] = lo2f<E>(b[i]);
    x[8 + 2 * i + 1] = hi2f<E>(b[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 c = cs[i];
    const int i0 = interleaved ? 2 * i : i, i1 = interleaved ? 2 * i + 1 : i + 8;
    const float x0 = x[i0], x1 = x[i1];
    x[i0] = x0 * c.x - x1 * c.y;
    x[i1] = x1 * c.x + x0 * c.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = pack2<E>(x[2 * i], x[2 * i + 1]);
    b[i] = pack2<E>(x[8 + 2 * i], x[8 + 2 * i + 1]);
  }
}

// A unit of 16 elements of a head: where it comes from and where it goes.
struct Unit {
  int t, h, u;         // token of the workgroup, head (queries, then keys), unit of the head
  int p0, p1;          // its two pieces: 8 pairs (halves or neighbours), or 16 elements that pass
};

template <class E, int D, int AP_THREADS>
__global__ __launch_bounds__(AP_THREADS) void kv_append_kernel(AppendArgs a) {
  __shared__ float2 cs[AP_MAX_TOKENS * AP_MAX_HALF];
  __shared__ int slot[AP_MAX_TOKENS + 8];      // [i + 1]: token i of the workgroup
  __shared__ int run_at[AP_MAX_TOKENS], run_len[AP_MAX_TOKENS], runs;
  const int tid = threadIdx.x;
  constexpr int units = D / 16, pieces = D / 8;
  const int ps = 1 << a.kv.page_shift;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_wg;
  const int nt = (int)(a.T - t0 < a.tokens_per_wg ? a.T - t0 : a.tokens_per_wg);
  const int half = a.inv_freq ? a.rot / 2 : 0, rot_units = half / 8;
  const int64_t top = a.kv.pages << a.kv.page_shift;
  const int per_token = (a.q_heads + a.kv.kv_heads) * units, all = nt * per_token;
  const int64_t page_elems = (int64_t)a.kv.kv_heads * ps * D;
  const int first = blockIdx.y * AP_THREADS + tid, step = a.y_splits * AP_THREADS;

  // the thread's next unit, requested ahead of its use
  u32x4 x0, x1;
  Unit w;
  int t_next = first / per_token, rest = first - t_next * per_token;
  auto request = [&]() {
    w.t = t_next;
    w.h = rest / units;
    w.u = rest - w.h * units;
    const bool apart = w.u < rot_units && !a.interleaved;
    w.p0 = apart ? w.u : 2 * w.u;
    w.p1 = apart ? w.u + rot_units : 2 * w.u + 1;
    const uint16_t* src = w.h < a.q_heads ? a.q + (t0 + w.t) * a.q_stride + w.h * D
                                          : a.k + (t0 + w.t) * a.k_stride + (w.h - a.q_heads) * D;
    x0 = *(const u32x4*)(src + w.p0 * 8);
    x1 = *(const u32x4*)(src + w.p1 * 8);
    for (rest += step; rest >= per_token; rest -= per_token) ++t_next;
  };
  if (first < all) request();

  // the slots of the tokens, of the one before and of 7 after (-1 where a slot
  // names no place in the cache): a run of V may reach that far
  if (tid < nt + 8) {
    const int64_t t = t0 + tid - 1;
    const int64_t s = t >= 0 && t < a.T ? a.slots[t] : -1;
    slot[tid] = s >= 0 && s < top ? (int)s : -1;
  }
  for (int i = tid; i < nt * half; i += AP_THREADS) {
    const int t = i / half, j = i - t * half;
    int ax = a.pair_axis ? a.pair_axis[j] : 0;
    ax = ax < 0 || ax >= a.axes ? 0 : ax;
    const double turns = (double)a.positions[ax * a.T + t0 + t] * (double)a.inv_freq[j] * 0.15915494309189533577;
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[i] = make_float2(c * a.rope_scale, s * a.rope_scale);
  }
  __syncthreads();
  if (tid < 64) {                              // the runs of V, a lane for each token
    bool begins = false;
    int len = 1;
    if (tid < nt) {
      const int s = slot[tid + 1], before = slot[tid];
      begins = s >= 0 && ((s & 7) == 0 || before < 0 || before != s - 1);
      bool on = true;
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        on = on && ((s + k) & 7) != 0 && slot[tid + 1 + k] == s + k;
        len += on;
      }
    }
    const uint64_t m = __ballot(begins);
    if (begins) {
      const int at = __builtin_popcountll(m & (((uint64_t)1 << tid) - 1));
      run_at[at] = tid;
      run_len[at] = len;
    }
    if (tid == 0) runs = __builtin_popcountll(m);
  }
  __syncthreads();

  // the first run of V, requested ahead of the units' stores
  const int per_run = a.kv.kv_heads * pieces, vall = runs * per_run;
  u32x4 v[8];
  auto request_v = [&](int i) {
    const int r = i / per_run, rest = i - r * per_run, h = rest / pieces, d0 = (rest - h * pieces) * 8;
    const uint16_t* src = a.v + (t0 + run_at[r]) * a.v_stride + h * D + d0;
    const int len = run_len[r];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < len) v[j] = *(const u32x4*)(src + j * a.v_stride);
  };
  if (first < vall) request_v(first);

  for (int i = first; i < all; i += step) {
    const Unit z = w;
    u32x4 y0 = x0, y1 = x1;
    if (i + step < all) request();
    const int s = slot[z.t + 1];
    if (z.u < rot_units) rotate8<E>(y0, y1, cs + z.t * half + z.u * 8, a.interleaved);
    if (z.h < a.q_heads) {
      uint16_t* dst = a.q_out + (t0 + z.t) * a.o_stride + z.h * D;
      // (past the caches: whole lines that others read next, on other XCDs;
      // 31.7 -> 28.9 us for the 4096 tokens where nothing is in a cache yet)
      __builtin_nontemporal_store(y0, (u32x4*)(dst + z.p0 * 8));
      __builtin_nontemporal_store(y1, (u32x4*)(dst + z.p1 * 8));
    } else if (s >= 0) {
      uint16_t* dst = (uint16_t*)a.kv.k + (int64_t)(s >> a.kv.page_shift) * page_elems +
                      (int64_t)(z.h - a.q_heads) * ps * D + (s & (ps - 1)) * 8;
      *(u32x4*)(dst + (int64_t)z.p0 * ps * 8) = y0;
      *(u32x4*)(dst + (int64_t)z.p1 * ps * 8) = y1;
    }
  }

  for (int i = first; i < vall; i += step) {
    if (i != first) request_v(i);
    const int r = i / per_run, rest = i - r * per_run, h = rest / pieces, d0 = (rest - h * pieces) * 8;
    const int len = run_len[r], s = slot[run_at[r] + 1];
    uint16_t* dst = (uint16_t*)a.kv.v + (int64_t)(s >> a.kv.page_shift) * page_elems + (int64_t)h * ps * D +
                    (int64_t)(((s & (ps - 1)) >> 3) * D + d0) * 8;
    if (len == 8) {
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = v[2 * j][d / 2], hi = v[2 * j + 1][d / 2];
          y[j] = d & 1 ? (lo >> 16) | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | (hi << 16);
        }
        *(u32x4*)(dst + d * 8) = y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < len)
#pragma unroll
          for (int d = 0; d < 8; ++d)
            dst[d * 8 + (s & 7) + j] = (uint16_t)(d & 1 ? v[j][d / 2] >> 16 : v[j][d / 2]);
    }
  }
}

template <class E, int THREADS>
hipError_t append_e(const AppendArgs& a, dim3 grid, hipStream_t st) {
  switch (a.kv.head_dim) {
    case 64: return launch_kernel(kv_append_kernel<E, 64, THREADS>, grid, THREADS, 0, st, a);
    case 96: return launch_kernel(kv_append_kernel<E, 96, THREADS>, grid, THREADS, 0, st, a);
    case 128: return launch_kernel(kv_append_kernel<E, 128, THREADS>, grid, THREADS, 0, st, a);
    default: return launch_kernel(kv_append_kernel<E, 256, THREADS>, grid, THREADS, 0, st, a);
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& args, int dtype, int num_cu, hipStream_t st) {
  AppendArgs a = args;
  // Tokens per workgroup: as many as leave a workgroup per CU.  Where that is
  // all 8, workgroups of 512 threads (2500 tokens, 40 heads of 128: 17.1 us,
  // 20.0 with 256 threads and 18.6 with 4 tokens); else of 256 (one token, 96
  // heads of 96: 4.9 us, 5.6 with 512).
  int tb = AP_MAX_TOKENS;
  while (tb > 1 && (a.T + tb - 1) / tb < num_cu) tb /= 2;
  const int threads = tb == AP_MAX_TOKENS ? 512 : 256;
  a.tokens_per_wg = tb;
  const int64_t wgs = (a.T + tb - 1) / tb;
  // a token's heads over several workgroups, one unit of 16 elements per thread, while CUs are idle
  const int64_t most = ((int64_t)tb * (a.q_heads + a.kv.kv_heads) * (a.kv.head_dim / 16) + threads - 1) / threads;
  int64_t y = num_cu / wgs;
  y = y < 1 ? 1 : (y > most ? most : y);
  a.y_splits = (int)y;
  const dim3 grid((unsigned)wgs, (unsigned)y);
  if (threads == 512) return dtype == DT_F16 ? append_e<f16, 512>(a, grid, st) : append_e<bf16, 512>(a, grid, st);
  return dtype == DT_F16 ? append_e<f16, 256>(a, grid, st) : append_e<bf16, 256>(a, grid, st);
}

}  // namespace fcg
