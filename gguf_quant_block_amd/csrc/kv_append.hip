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
// is in f32 with one rounding to the cache's type.
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

constexpr int AP_THREADS = 256;
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

template <class E>
__global__ __launch_bounds__(AP_THREADS) void kv_append_kernel(AppendArgs a) {
  __shared__ float2 cs[AP_MAX_TOKENS * AP_MAX_HALF];
  __shared__ int slot[AP_MAX_TOKENS + 8];      // [i + 1]: token i of the workgroup
  __shared__ int run_at[AP_MAX_TOKENS], run_len[AP_MAX_TOKENS], runs;
  const int tid = threadIdx.x;
  const int D = a.kv.head_dim, ps = 1 << a.kv.page_shift;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_wg;
  const int nt = (int)(a.T - t0 < a.tokens_per_wg ? a.T - t0 : a.tokens_per_wg);
  const int half = a.inv_freq ? a.rot / 2 : 0;
  const int64_t top = a.kv.pages << a.kv.page_shift;

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
  if (tid == 0) {
    int n = 0;
    for (int i = 0; i < nt; ++i) {
      const int s = slot[i + 1];
      // does a run begin with token i?
      if (s < 0 || ((s & 7) != 0 && slot[i] >= 0 && slot[i] == s - 1)) continue;
      int len = 1;
      while (((s + len) & 7) != 0 && slot[i + 1 + len] == s + len) ++len;
      run_at[n] = i;
      run_len[n++] = len;
    }
    runs = n;
  }
  __syncthreads();

  const int units = D / 16, heads = a.q_heads + a.kv.kv_heads;
  const int per_token = heads * units;
  const int64_t page_elems = (int64_t)a.kv.kv_heads * ps * D;
  const int rot_units = half / 8;
  const int first = blockIdx.y * AP_THREADS + tid, step = a.y_splits * AP_THREADS;
  for (int i = first; i < nt * per_token; i += step) {
    const int t = i / per_token, rest = i - t * per_token;
    const int h = rest / units, u = rest - h * units;
    const bool is_q = h < a.q_heads;
    const int s = slot[t + 1];
    if (!is_q && s < 0) continue;
    // the unit's two pieces: 8 pairs (halves or neighbours), or 16 elements that pass
    const int p0 = u < rot_units && !a.interleaved ? u : 2 * u;
    const int p1 = u < rot_units && !a.interleaved ? u + rot_units : 2 * u + 1;
    const uint16_t* src = is_q ? a.q + (t0 + t) * a.q_stride + h * D
                               : a.k + (t0 + t) * a.k_stride + (h - a.q_heads) * D;
    u32x4 x0 = *(const u32x4*)(src + p0 * 8), x1 = *(const u32x4*)(src + p1 * 8);
    if (u < rot_units) rotate8<E>(x0, x1, cs + t * half + u * 8, a.interleaved);
    if (is_q) {
      uint16_t* dst = a.q_out + (t0 + t) * a.o_stride + h * D;
      *(u32x4*)(dst + p0 * 8) = x0;
      *(u32x4*)(dst + p1 * 8) = x1;
    } else {
      uint16_t* dst = (uint16_t*)a.kv.k + (int64_t)(s >> a.kv.page_shift) * page_elems +
                      (int64_t)(h - a.q_heads) * ps * D + (s & (ps - 1)) * 8;
      *(u32x4*)(dst + (int64_t)p0 * ps * 8) = x0;
      *(u32x4*)(dst + (int64_t)p1 * ps * 8) = x1;
    }
  }

  const int pieces = D / 8, per_run = a.kv.kv_heads * pieces;
  for (int i = first; i < runs * per_run; i += step) {
    const int r = i / per_run, rest = i - r * per_run;
    const int h = rest / pieces, d0 = (rest - h * pieces) * 8;
    const int t = run_at[r], len = run_len[r], s = slot[t + 1];
    const uint16_t* src = a.v + (t0 + t) * a.v_stride + h * D + d0;
    uint16_t* dst = (uint16_t*)a.kv.v + (int64_t)(s >> a.kv.page_shift) * page_elems +
                    (int64_t)h * ps * D + (int64_t)(((s & (ps - 1)) >> 3) * D + d0) * 8;
    if (len == 8) {
      u32x4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = *(const u32x4*)(src + j * a.v_stride);
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = x[2 * j][d / 2], hi = x[2 * j + 1][d / 2];
          y[j] = d & 1 ? (lo >> 16) | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | (hi << 16);
        }
        *(u32x4*)(dst + d * 8) = y;
      }
    } else {
      for (int j = 0; j < len; ++j) {
        const u32x4 x = *(const u32x4*)(src + j * a.v_stride);
#pragma unroll
        for (int d = 0; d < 8; ++d)
          dst[d * 8 + (s & 7) + j] = (uint16_t)(d & 1 ? x[d / 2] >> 16 : x[d / 2]);
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& args, int dtype, int num_cu, hipStream_t st) {
  AppendArgs a = args;
  // tokens per workgroup: as many as leave two workgroups per CU
  int tb = AP_MAX_TOKENS;
  while (tb > 1 && (a.T + tb - 1) / tb < 2 * num_cu) tb /= 2;
  a.tokens_per_wg = tb;
  const int64_t wgs = (a.T + tb - 1) / tb;
  // a token's heads over several workgroups, one unit of 16 elements per thread, while CUs are idle
  const int64_t most = ((int64_t)tb * (a.q_heads + a.kv.kv_heads) * (a.kv.head_dim / 16) + AP_THREADS - 1) / AP_THREADS;
  int64_t y = num_cu / wgs;
  y = y < 1 ? 1 : (y > most ? most : y);
  a.y_splits = (int)y;
  const dim3 grid((unsigned)wgs, (unsigned)y);
  if (dtype == DT_F16) kv_append_kernel<f16><<<grid, AP_THREADS, 0, st>>>(a);
  else kv_append_kernel<bf16><<<grid, AP_THREADS, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace fcg
