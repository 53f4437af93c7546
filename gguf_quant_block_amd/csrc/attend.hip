// Attention of new tokens over the paged cache: the streaming kernel (few
// query rows for each key head) and the joining of split sums.
//
//   row (token i of sequence s, head): position p = kv_len - q_len + i
//   o = sum_j 2^(c q.k_j - m) v_j / l,   m = max_j c q.k_j,  l = sum_j 2^(c q.k_j - m)
// over the keys j <= p, j > p - window, on pages of the pool; c = scale log2(e).
// One pass: m and l run along, and the sums are scaled when m grows.
//
// The rows of one key head are the tokens times the group of query heads that
// share it, token by token, so that K and V are read once for all of them.
// With 16 .. 64 rows the kernel is bound by HBM (the keys and values); the
// matrix instructions cost less than the loads even with one row of 16 in use.
//
// S^T = K Q^T and O^T = V^T P^T: with the keys as rows of the first product,
// a lane holds its scores for one query row (column lane % 16) and 4 keys of
// each 16.  The rows of the two 16-key operands of a 32-key tile are dealt so
// that lane group g = lane / 16 ends with keys 8g .. 8g + 7, which are the
// elements of its operand in the second product: the weights go from one
// product to the next without leaving their registers, and maxima and totals
// need two exchanges between lanes.  Both cache operands are loaded from HBM
// straight into registers in 16-byte pieces; the next tile's keys are
// requested as soon as this tile's scores exist, its values after the sums.
//
// The weights are rounded to the cache's type for the second product (f16 or
// bf16 matrix instructions); the totals are summed in f32 from the unrounded
// weights, and products, sums and statistics are f32.
#include <math.h>

#include "serving.h"

namespace fcg {
namespace {

constexpr int AT_WAVES = 4;
constexpr int AT_TILE = 32;                      // keys per wave and step
constexpr int AT_STEP = AT_WAVES * AT_TILE;
constexpr float LN2 = 0.693147180559945309f;

// What a workgroup's rows see.  All members are the same in every lane.
struct RowTile {
  int s, hk, row0, rows;      // sequence, key head, first row, rows of the sequence
  int q0;                     // first token of the sequence in q
  int kv_len;                 // keys in the table
  int base;                   // position of the sequence's first new token
  int lo, hi;                 // positions of the tile's first and last row
  int beg, end;               // keys that some row sees: [beg, end)
};

// false: the tile has no rows
__device__ __forceinline__ bool row_tile(const AttendArgs& a, int s, int hk, int tile, int tile_rows,
                                         RowTile& t) {
  const int64_t c0 = a.cu_q[s], c1 = a.cu_q[s + 1];
  const int q0 = (int)(c0 < 0 ? 0 : (c0 > a.T ? a.T : c0));
  const int q1 = (int)(c1 < q0 ? q0 : (c1 > a.T ? a.T : c1));
  const int n = q1 - q0;
  t.s = s;
  t.hk = hk;
  t.q0 = q0;
  t.rows = (n < a.max_q ? n : a.max_q) * a.group;
  t.row0 = tile * tile_rows;
  if (t.row0 >= t.rows) return false;
  int len = a.kv_lens[s];
  const int64_t held = (int64_t)a.table_w << a.kv.page_shift;
  len = len < 0 ? 0 : len;
  t.base = len - n;
  t.kv_len = (int)(len < held ? len : held);
  const int last = t.row0 + tile_rows < t.rows ? t.row0 + tile_rows : t.rows;
  t.lo = t.base + t.row0 / a.group;
  t.hi = t.base + (last - 1) / a.group;
  t.end = t.hi + 1 < t.kv_len ? t.hi + 1 : t.kv_len;
  t.beg = a.window > 0 && t.lo - a.window + 1 > 0 ? (t.lo - a.window + 1) & ~(AT_TILE - 1) : 0;
  return true;
}

// keys [c0, c1) of the tile's [beg, end) that split `split` of `splits` takes
__device__ __forceinline__ void split_range(int beg, int end, int split, int splits, int unit, int& c0,
                                            int& c1) {
  const int n = end - beg;
  int per = (n + splits - 1) / splits;
  per = (per + unit - 1) / unit * unit;
  const int64_t at = beg + (int64_t)split * per;
  c0 = at < end ? (int)at : end;
  c1 = at + per < end ? (int)(at + per) : end;
}

template <class E, int D, int RT>
__global__ __launch_bounds__(AT_WAVES * 64, D * RT <= 256 ? 2 : 1) void attend_stream_kernel(AttendArgs a) {
  constexpr int KS = D / 32, DT = D / 16;
  constexpr int PITCH = D + 4;                    // floats of a row in LDS
  __shared__ float sums[AT_WAVES * 16 * PITCH];
  __shared__ float ml[AT_WAVES][RT * 16][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;

  int b = blockIdx.x;
  const int hk = b % a.kv.kv_heads;
  b /= a.kv.kv_heads;
  const int split = b % a.splits;
  b /= a.splits;
  RowTile t;
  if (!row_tile(a, b % a.seqs, hk, b / a.seqs, RT * 16, t)) return;
  int c0, c1;
  split_range(t.beg, t.end, split, a.splits, AT_STEP, c0, c1);

  const int ps = 1 << a.kv.page_shift;
  const int64_t page_bytes = (int64_t)a.kv.kv_heads * ps * D * 2;
  const uint8_t* kbase = (const uint8_t*)a.kv.k + (int64_t)hk * ps * D * 2;
  const uint8_t* vbase = (const uint8_t*)a.kv.v + (int64_t)hk * ps * D * 2;
  const int32_t* table = a.table + t.s * a.table_stride;

  u32x4 q[RT][KS];
  int pos[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = t.row0 + i * 16 + r;
    const bool there = row < t.rows;
    const int tok = row / a.group;
    pos[i] = there ? t.base + tok : -1;
    const uint16_t* p = a.q + (t.q0 + tok) * a.q_stride + (hk * a.group + row - tok * a.group) * D + g * 8;
#pragma unroll
    for (int k = 0; k < KS; ++k) q[i][k] = there ? *(const u32x4*)(p + k * 32) : (u32x4){0, 0, 0, 0};
  }

  floatx4 o[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[i][d] = (floatx4){0.f, 0.f, 0.f, 0.f};
  }

  // The page of the 16 keys that hold a lane's key rows (r / 8) and of those
  // that hold its values (g / 2); a page never ends inside 16 keys.  -1: no
  // page of the pool, its keys take no part.
  auto page_at = [&](int key) -> int {
    if (key >= c1) return -1;
    const int p = table[key >> a.kv.page_shift];
    return (unsigned)p < (uint64_t)a.kv.pages ? p : -1;
  };
  u32x4 kr[2][KS], vr[DT];
  // key of row r of half h of a tile: 8 (r / 4) + 4 h + r % 4
  auto load_k = [&](int tok0, int page) {
    const uint8_t* p = kbase + (page < 0 ? 0 : page) * page_bytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = tok0 + 8 * (r >> 2) + 4 * h + (r & 3);
      const uint8_t* x = p + ((key & (ps - 1)) + g * ps) * 16;
#pragma unroll
      for (int k = 0; k < KS; ++k) kr[h][k] = *(const u32x4*)(x + k * 4 * ps * 16);
    }
  };
  auto load_v = [&](int tok0, int page) {
    const uint8_t* p = vbase + (page < 0 ? 0 : page) * page_bytes +
                       ((((tok0 + 8 * g) & (ps - 1)) >> 3) * D + r) * 16;
#pragma unroll
    for (int d = 0; d < DT; ++d) vr[d] = *(const u32x4*)(p + d * 256);
  };

  int tok0 = c0 + wave * AT_TILE;
  int pk = page_at(tok0 + (r >> 3) * 16), pv = page_at(tok0 + (g >> 1) * 16);
  if (tok0 < c1) {
    load_k(tok0, pk);
    load_v(tok0, pv);
  }
  for (; tok0 < c1; tok0 += AT_STEP) {
    const int next = tok0 + AT_STEP;
    const int npk = page_at(next + (r >> 3) * 16), npv = page_at(next + (g >> 1) * 16);
    floatx4 sc[RT][2];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) c = Mat<E>::mfma16(kr[h][k], q[i][k], c);
        sc[i][h] = c;
      }
    if (next < c1) load_k(next, npk);

    // every row sees every key of the tile: no mask
    const int key0 = tok0 + 8 * g;                 // keys of this lane: key0 .. key0 + 7
    const bool open = tok0 + AT_TILE <= c1 && tok0 + AT_TILE - 1 <= t.lo &&
                      (a.window <= 0 || tok0 > t.hi - a.window) && __all(pv >= 0);
    bool hard = false;                             // values of masked keys that are not finite
    if (!open) {
      uint32_t odd = 0, some = 0;                  // keys no row of the tile sees / some rows see
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + j;
        const bool gone = key >= c1 || pv < 0;
        odd |= (uint32_t)gone << j;
        some |= (uint32_t)(!gone && (key > t.lo || (a.window > 0 && key <= t.hi - a.window))) << j;
      }
      u32x4 keep, part;                            // dword j: keys 2j, 2j + 1
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        keep[j] = (odd >> (2 * j) & 1 ? 0u : 0xFFFFu) | (odd >> (2 * j + 1) & 1 ? 0u : 0xFFFF0000u);
        part[j] = (some >> (2 * j) & 1 ? 0xFFFFu : 0u) | (some >> (2 * j + 1) & 1 ? 0xFFFF0000u : 0u);
      }
      uint32_t bad = 0;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        vr[d] &= keep;                             // stale values must not meet a weight of 0 as NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) bad |= nonfinite2<E>(vr[d][j]) & part[j];
      }
      hard = __any(bad != 0);
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = key0 + j;
          if (key > pos[i] || (a.window > 0 && key <= pos[i] - a.window) || (odd >> j & 1))
            sc[i][j >> 2][j & 3] = -INFINITY;
        }
    }

#pragma unroll
    for (int i = 0; i < RT; ++i) {
      float mx = sc[i][0][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, sc[i][j >> 2][j & 3]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m[i], mx * a.scale_log2);
      const float ms = mn == -INFINITY ? 0.f : mn;
      const float al = __builtin_amdgcn_exp2f(m[i] - ms);
      m[i] = mn;
      float p[8], sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = __builtin_amdgcn_exp2f(sc[i][j >> 2][j & 3] * a.scale_log2 - ms);
        sum += p[j];
      }
      l[i] = l[i] * al + sum;
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack2<E>(p[2 * j], p[2 * j + 1]);
      if (!hard) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[i][d] *= al;
          o[i][d] = Mat<E>::mfma16(vr[d], w, o[i][d]);
        }
      } else {
        // a value that is infinite or NaN in a row that another row masks:
        // each row's sum is taken with its own masked keys' values at 0
#pragma unroll
        for (int d = 0; d < DT; ++d) o[i][d] *= al;
        for (int x = 0; x < 16; ++x) {
          const int px = __shfl(pos[i], x);
          u32x4 keep;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t k = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = key0 + 2 * j + e;
              if (key <= px && !(a.window > 0 && key <= px - a.window)) k |= 0xFFFFu << (16 * e);
            }
            keep[j] = k;
          }
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            floatx4 c = {0.f, 0.f, 0.f, 0.f};
            c = Mat<E>::mfma16(vr[d] & keep, w, c);
            if (r == x) o[i][d] += c;
          }
        }
      }
    }
    if (next < c1) load_v(next, npv);
    pv = npv;
  }

  // join the waves
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    l[i] += __shfl_xor(l[i], 16);
    l[i] += __shfl_xor(l[i], 32);
    if (g == 0) {
      ml[wave][i * 16 + r][0] = m[i];
      ml[wave][i * 16 + r][1] = l[i];
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *(floatx4*)&sums[(wave * 16 + r) * PITCH + d * 16 + g * 4] = o[i][d];
    __syncthreads();
    for (int x = tid; x < 16 * (D / 8); x += AT_WAVES * 64) {
      const int rr = x / (D / 8), d0 = (x - rr * (D / 8)) * 8, row = t.row0 + i * 16 + rr;
      if (row >= t.rows) continue;
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < AT_WAVES; ++w) mt = fmaxf(mt, ml[w][i * 16 + rr][0]);
      const float ms = mt == -INFINITY ? 0.f : mt;
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < AT_WAVES; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][i * 16 + rr][0] - ms);
        lt += ml[w][i * 16 + rr][1] * f;
        const float* p = &sums[(w * 16 + rr) * PITCH + d0];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] += p[j] * f;
      }
      const int tok = row / a.group, head = hk * a.group + row - tok * a.group;
      const int64_t orow = (int64_t)(t.q0 + tok) * a.q_heads + head;
      if (a.splits > 1) {
        const int64_t at = (int64_t)split * a.T * a.q_heads + orow;
        floatx4* p = (floatx4*)(a.part + at * D + d0);
        p[0] = (floatx4){y[0], y[1], y[2], y[3]};
        p[1] = (floatx4){y[4], y[5], y[6], y[7]};
        if (d0 == 0) *(float2*)(a.part_ml + at * 2) = make_float2(mt, lt);
      } else {
        const float f = lt == 0.f ? 0.f : 1.f / lt;
        u32x4 z;
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = pack2<E>(y[2 * j] * f, y[2 * j + 1] * f);
        *(u32x4*)(a.o + (t.q0 + tok) * a.o_stride + head * D + d0) = z;
        if (a.lse && d0 == 0) a.lse[orow] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * LN2;
      }
    }
  }
}

// Joins the splits of a row: a wave per row, D / 64 dimensions per lane.
template <class E, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t rr = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);   // row of the sequence
  const int s = blockIdx.y;
  RowTile t;
  if (!row_tile(a, s, 0, 0, 1, t)) return;
  const int tok = (int)(rr / a.q_heads), head = (int)(rr - (int64_t)tok * a.q_heads);
  if ((int64_t)tok * a.group >= t.rows) return;
  const int64_t rows = a.T * a.q_heads, orow = (int64_t)(t.q0 + tok) * a.q_heads + head;
  float mt = -INFINITY;
  for (int x = lane; x < a.splits; x += 64) mt = fmaxf(mt, a.part_ml[(x * rows + orow) * 2]);
#pragma unroll
  for (int k = 1; k < 64; k *= 2) mt = fmaxf(mt, __shfl_xor(mt, k));
  const float ms = mt == -INFINITY ? 0.f : mt;
  float lt = 0.f, y[(D + 63) / 64];
#pragma unroll
  for (int j = 0; j < (D + 63) / 64; ++j) y[j] = 0.f;
  for (int x = 0; x < a.splits; ++x) {
    const float2 v = *(const float2*)(a.part_ml + (x * rows + orow) * 2);
    const float f = __builtin_amdgcn_exp2f(v.x - ms);
    lt += v.y * f;
    const float* p = a.part + (x * rows + orow) * D;
#pragma unroll
    for (int j = 0; j < (D + 63) / 64; ++j) {
      const int d = j * 64 + lane;
      if (D % 64 == 0 || d < D) y[j] += p[d] * f;
    }
  }
  const float f = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
  for (int j = 0; j < (D + 63) / 64; ++j) {
    const int d = j * 64 + lane;
    if (D % 64 == 0 || d < D)
      a.o[(t.q0 + tok) * a.o_stride + head * D + d] = __builtin_bit_cast(uint16_t, (E)(y[j] * f));
  }
  if (a.lse && lane == 0) a.lse[orow] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * LN2;
}

template <class E, int D, int RT>
hipError_t stream_launch(const AttendArgs& a, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_q * a.group, tiles = (rows + RT * 16 - 1) / (RT * 16);
  const int64_t wgs = tiles * a.seqs * a.splits * a.kv.kv_heads;
  attend_stream_kernel<E, D, RT><<<dim3((unsigned)wgs), AT_WAVES * 64, 0, st>>>(a);
  return hipGetLastError();
}

template <class E, int D>
hipError_t launch_d(const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  hipError_t e;
  if (p.row_tiles == 1) e = stream_launch<E, D, 1>(a, st);
  else e = stream_launch<E, D, 2>(a, st);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.max_q * a.q_heads;
  attend_join_kernel<E, D><<<dim3((unsigned)((rows + 3) / 4), (unsigned)a.seqs), 256, 0, st>>>(a);
  return hipGetLastError();
}

template <class E>
hipError_t launch_e(const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  switch (a.kv.head_dim) {
    case 64: return launch_d<E, 64>(a, p, st);
    case 96: return launch_d<E, 96>(a, p, st);
    case 128: return launch_d<E, 128>(a, p, st);
    default: return launch_d<E, 256>(a, p, st);
  }
}

}  // namespace

AttendPlan attend_plan(const AttendArgs& a, int num_cu) {
  AttendPlan p;
  const int64_t rows = (int64_t)a.max_q * a.group;
  p.row_tiles = rows <= 16 ? 1 : 2;
  const int64_t wgs = (rows + p.row_tiles * 16 - 1) / (p.row_tiles * 16) * a.seqs * a.kv.kv_heads;
  const int64_t keys = (int64_t)a.table_w << a.kv.page_shift;
  // a part has at least 512 keys, and there are parts enough for 4 workgroups per CU
  int64_t most = (keys + 511) / 512, want = (4 * num_cu + wgs - 1) / wgs;
  p.splits = (int)(want < most ? want : most);
  if (p.splits < 1) p.splits = 1;
  return p;
}

size_t attend_workspace_bytes(const AttendArgs& a, const AttendPlan& p) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * a.T * a.q_heads * (a.kv.head_dim + 2) * sizeof(float);
}

hipError_t launch_attend(const AttendArgs& args, const AttendPlan& p, int dtype, hipStream_t st) {
  AttendArgs a = args;
  a.splits = p.splits;
  a.part_ml = a.part + (size_t)p.splits * a.T * a.q_heads * a.kv.head_dim;
  return dtype == DT_F16 ? launch_e<f16>(a, p, st) : launch_e<bf16>(a, p, st);
}

}  // namespace fcg
