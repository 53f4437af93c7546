// Attention of new tokens over the paged cache: the streaming kernel (few
// query rows for each key head), the join of split tiles, and the launches.
//
//   row (token i of sequence s, head): position p = kv_len - q_len + i
//   o = sum_j 2^(c q.k_j - m) v_j / l,   m = max_j c q.k_j - LIFT,  l = sum_j 2^(c q.k_j - m)
// over the keys j <= p, j > p - window, on pages of the pool; c = scale log2(e).
// One pass: m and l run along, and the sums are scaled when m grows.
//
// The rows of one key head are the tokens times the group of query heads that
// share it, token by token, so that K and V are read once for all of them.
// With up to 32 rows the kernel is bound by HBM (the keys and values); the
// matrix instructions cost less than the loads even with one row of 16 in use.
// Measured: one token over 131072 keys (32 heads of 128 on 8 key heads) 99 us,
// 5.4 TB/s; 64 tokens over up to 8192 keys each 137 us, 5.4 TB/s, of 6.1 that
// a plain read of 1 GiB reaches; bytes from HBM 1.005 of the keys and values.
// Short calls are bound by latency: 8 x 5 drafted tokens over up to 6001 keys
// 28 us (15 us at 5.3 TB/s, then 7 us for the pieces to be joined), one token
// over 1003 keys 9 us.
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
// bf16 matrix instructions): off by half a step, 2^-8 of a bf16 weight, 2^-11 of
// an f16 one or 2^-33 of the row's largest (LIFT in serving.h).  The totals are
// summed in f32 from the unrounded weights, and products, sums and statistics
// are f32.
#include <math.h>

#include "attend.h"

namespace fcg {
namespace {

// Keys [c0, c1) of a sequence's rows: the sums and statistics of this wave.
//
// Q8: a cache of 8 bits.  A 16-byte load is then two pieces, the same 8
// dimensions of keys 2r and 2r + 1 of the tile for lane row r, or the same 8
// keys of dimensions 2r and 2r + 1 of 32.  One of the two goes to each of a pair
// of operands, so that row r of half h of the first product is key 2r + h, and
// of the second dimension 32 (d / 2) + 2r + d % 2.  A lane still ends with the
// scores of keys 8g .. 8g + 7, in another order.  Codes become values of E
// where they are used, exactly (serving.h): what follows is the same.
//
// Measured: 64 tokens over up to 8192 keys each 81 us (372 MB, 4.6 TB/s; of 16
// bits 137); about 12 us of it are the call's begin and end and 10 the changes
// from sequence to sequence, and longer caches come to 6.1 TB/s.  One token over
// 131072 keys 56.4 us, or 49 with pages that the last-level cache holds in part
// (270 MB; of 16 bits 98); 8 x 5 drafted tokens over up to 6001 keys 26, one over
// 1003 keys 9.6.  A second tile in flight gained nothing (85 us instead of 82).
template <class E, int D, int RT, bool Q8, int WAVES>
struct Piece {
  static constexpr int KS = D / 32, DT = D / 16, AT_STEP = WAVES * AT_TILE;
  // where the score of the lane's key j stands: half, and element of it
  static constexpr int half_of(int j) { return Q8 ? j & 1 : j >> 2; }
  static constexpr int row_of(int j) { return Q8 ? j >> 1 : j & 3; }
  floatx4 o[RT][DT];
  float m[RT], l[RT];

  __device__ __forceinline__ void run(const AttendArgs& a, const RowTile& t, int c0, int c1) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const int ps = 1 << a.kv.page_shift, hk = t.hk;
    constexpr int B = Q8 ? 1 : 2;                // bytes of an element
    const int64_t page_bytes = (int64_t)a.kv.kv_heads * ps * D * B;
    const uint8_t* kbase = (const uint8_t*)a.kv.k + (int64_t)hk * ps * D * B;
    const uint8_t* vbase = (const uint8_t*)a.kv.v + (int64_t)hk * ps * D * B;
    const int32_t* table = a.table + t.s * a.table_stride;

    // The page of the 16 keys that hold a lane's key rows (r / 8) and of those
    // that hold its values (g / 2); a page never ends inside 16 keys.  -1: no
    // page of the pool, its keys take no part.
    // Entries of the table are read a step before they are looked at.
    auto entry_at = [&](int key) -> int { return table[(key < c1 ? key : c1 - 1) >> a.kv.page_shift]; };
    auto page_of = [&](int key, int entry) -> int { return key < c1 && (unsigned)entry < (uint64_t)a.kv.pages ? entry : -1; };
    constexpr int KH = Q8 ? 1 : 2, VT = Q8 ? DT / 2 : DT;
    u32x4 kr[KH][KS], vr[VT];
    uint32_t ke = 0;                               // Q8: the stored exponents of the lane's two keys,
    uint2 ve = {0, 0};                             // and of the 8 whose values it has
    auto scales_at = [&](const uint8_t* scales, int page, int key) -> const uint8_t* {
      return scales + ((int64_t)(page < 0 ? 0 : page) * a.kv.kv_heads + hk) * ps + (key & (ps - 1));
    };
    // key of row r of half h of a tile: 8 (r / 4) + 4 h + r % 4
    auto load_k = [&](int tok0, int page) {
      const uint8_t* p = kbase + (page < 0 ? 0 : page) * page_bytes;
      if constexpr (Q8) {
        const int key = tok0 + 2 * r;
        ke = *(const uint16_t*)scales_at(a.kv.k_scale, page, key);
        const uint8_t* x = p + ((key & (ps - 1)) + g * ps) * 8;
#pragma unroll
        for (int k = 0; k < KS; ++k) kr[0][k] = *(const u32x4*)(x + k * 4 * ps * 8);
      } else {
#pragma unroll
        for (int h = 0; h < KH; ++h) {
          const int key = tok0 + 8 * (r >> 2) + 4 * h + (r & 3);
          const uint8_t* x = p + ((key & (ps - 1)) + g * ps) * 16;
#pragma unroll
          for (int k = 0; k < KS; ++k) kr[h][k] = *(const u32x4*)(x + k * 4 * ps * 16);
        }
      }
    };
    auto v_at = [&](int tok0, int page) -> const uint8_t* {
      return vbase + (page < 0 ? 0 : page) * page_bytes + ((((tok0 + 8 * g) & (ps - 1)) >> 3) * D + (Q8 ? 2 * r : r)) * 8 * B;
    };
    auto load_v = [&](int tok0, int page) {
      const uint8_t* p = v_at(tok0, page);
      if constexpr (Q8) ve = *(const uint2*)scales_at(a.kv.v_scale, page, tok0 + 8 * g);
#pragma unroll
      for (int d = 0; d < VT; ++d) vr[d] = *(const u32x4*)(p + d * 256);
    };
    // every row sees every key of the tile: no mask
    auto is_open = [&](int tok0, int page) {
      return tok0 + AT_TILE <= c1 && tok0 + AT_TILE - 1 <= t.lo && (a.window <= 0 || tok0 > t.hi - a.window) &&
             __all(page >= 0);
    };
    // how many of the lane's keys tok0 + 8g .. + 7 are there
    auto have = [&](int tok0, int page) -> int {
      const int left = c1 - (tok0 + 8 * g);
      return page >= 0 ? (left < 8 ? left : 8) : 0;
    };

    const int first = c0 + wave * AT_TILE, ko = (r >> 3) * 16, vo = (g >> 1) * 16;
    int tok0 = first;
    int ek = 0, ev = 0, pv = -1;                   // entries of the next tile, page of this one's values
    if (tok0 < c1) {
      ek = entry_at(tok0 + ko);
      ev = entry_at(tok0 + vo);
      const int pk = page_of(tok0 + ko, ek);
      pv = page_of(tok0 + vo, ev);
      ek = entry_at(tok0 + AT_STEP + ko);
      ev = entry_at(tok0 + AT_STEP + vo);
      load_k(tok0, pk);
      load_v(tok0, pv);
    }
    u32x4 q[RT][KS];
    int pos[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int row = i * 16 + r;
      const bool there = row < t.rows;
      const int tok = row / a.group;
      pos[i] = there ? t.base + tok : -1;
      const uint16_t* p = a.q + (t.q0 + tok) * a.q_stride + (hk * a.group + row - tok * a.group) * D + g * 8;
#pragma unroll
      for (int k = 0; k < KS; ++k) q[i][k] = there ? *(const u32x4*)(p + k * 32) : (u32x4){0, 0, 0, 0};
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[i][d] = (floatx4){0.f, 0.f, 0.f, 0.f};
    }

    uint32_t bad = 0;                              // values were taken out of a masked tile
    for (; tok0 < c1; tok0 += AT_STEP) {
      const int next = tok0 + AT_STEP;
      floatx4 sc[RT][2];
      if constexpr (Q8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float by = __builtin_bit_cast(float, held_exponent<E>(ke >> (8 * h) & 0xFFu) << 23);
#pragma unroll
          for (int i = 0; i < RT; ++i) sc[i][h] = (floatx4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const u32x4 x = codes8<E>(kr[0][k][2 * h], kr[0][k][2 * h + 1], by);
#pragma unroll
            for (int i = 0; i < RT; ++i) sc[i][h] = Mat<E>::mfma16(x, q[i][k], sc[i][h]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KS; ++k) c = Mat<E>::mfma16(kr[h][k], q[i][k], c);
            sc[i][h] = c;
          }
      }
      // (past the last tile the loads are of the pool's first page, for nothing)
      load_k(next, page_of(next + ko, ek));
      ek = entry_at(next + AT_STEP + ko);

      u32x4 decoded[Q8 ? DT : 1];
      auto pick = [&]() -> auto& { if constexpr (Q8) return decoded; else return vr; };
      auto& vals = pick();                         // the tile's values
      if constexpr (Q8) {
        const ValueScales<E> scales(ve);
#pragma unroll
        for (int d = 0; d < DT; ++d) vals[d] = scales.values(vr[d / 2][2 * (d & 1)], vr[d / 2][2 * (d & 1) + 1]);
      }
      if (!is_open(tok0, pv)) {
        const int key0 = tok0 + 8 * g, n = have(tok0, pv);
        const u32x4 keep = keep_keys(n);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          vals[d] &= keep;                         // stale values must not meet a weight of 0 as NaN
          bad |= take_nonfinite<E>(vals[d]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int top = pos[i] - key0 < n ? pos[i] - key0 : n - 1;       // last key that the row sees
          const int low = a.window > 0 ? pos[i] - a.window - key0 : -1;    // last before its window
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j > top || j <= low) sc[i][half_of(j)][row_of(j)] = -INFINITY;
        }
      }

#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float mx = fmaxf(sc[i][0][0], sc[i][1][0]);
#pragma unroll
        for (int j = 1; j < 4; ++j) mx = max3(mx, sc[i][0][j], sc[i][1][j]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m[i], reference_of<E>(mx, a.scale_log2));
        const float ms = mn == -INFINITY ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f(m[i] - ms);
        m[i] = mn;
        float p[8], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = __builtin_amdgcn_exp2f(fmaf(sc[i][half_of(j)][row_of(j)], a.scale_log2, -ms));
          sum += p[j];
        }
        l[i] = l[i] * al + sum;
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack2<E>(p[2 * j], p[2 * j + 1]);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[i][d] *= al;
          o[i][d] = Mat<E>::mfma16(vals[d], w, o[i][d]);
        }
      }
      pv = page_of(next + vo, ev);
      load_v(next, pv);
      ev = entry_at(next + AT_STEP + vo);
    }

    if (__any(bad != 0))                           // counts of the values taken out
      for (tok0 = first; tok0 < c1; tok0 += AT_STEP) {
        const int page = page_of(tok0 + vo, entry_at(tok0 + vo));
        if (is_open(tok0, page)) continue;
        const int key0 = tok0 + 8 * g, n = have(tok0, page);
        const uint8_t* p = v_at(tok0, page);
        auto values_of = [&](int d) -> u32x4 {
          if constexpr (Q8) {
            const u32x4 x = *(const u32x4*)(p + (d / 2) * 256);
            return ValueScales<E>(*(const uint2*)scales_at(a.kv.v_scale, page, key0)).values(x[2 * (d & 1)], x[2 * (d & 1) + 1]);
          } else {
            return *(const u32x4*)(p + d * 256);
          }
        };
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const u32x4 one = seen_ones<E>(pos[i] - key0 < n ? pos[i] - key0 : n - 1, a.window > 0 ? pos[i] - a.window - key0 : -1);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            floatx4 c = {0.f, 0.f, 0.f, 0.f};
            c = Mat<E>::mfma16(nonfinite_codes<E>(values_of(d) & keep_keys(n)), one, c);
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][d][x] += nonfinite_sum(c[x]);
          }
        }
      }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      l[i] += __shfl_xor(l[i], 16);
      l[i] += __shfl_xor(l[i], 32);
    }
  }
};

// steps of WAVES tiles of keys of sequence s; 1 where its rows see no key or
// sequences are not split, 0 where it has no rows here
template <int WAVES>
__device__ __forceinline__ int seq_steps(const AttendArgs& a, int s, int hk, RowTile& t) {
  constexpr int AT_STEP = WAVES * AT_TILE;
  if (s >= a.seqs || !row_tile(a, s, hk, 0, a.stream_rows, 1, a.stream_rows, AT_TILE, t)) return 0;
  return t.end > t.beg && !a.whole ? (t.end - t.beg + AT_STEP - 1) / AT_STEP : 1;
}

// a / c, a >= 0, c > 0
__device__ __forceinline__ int64_t div64(int64_t a, int64_t c) {
  return a < ((int64_t)1 << 32) && c < ((int64_t)1 << 32) ? (int64_t)((uint32_t)a / (uint32_t)c) : a / c;
}

// ceil(a * b / c), all of them > 0
__device__ __forceinline__ int64_t mul_div_up(int64_t a, int b, int64_t c) { return div64(a * b - 1, c) + 1; }

// The workspace's pieces travel between workgroups of one launch, on any XCD:
// stores and loads at the device's scope (aux bit 4, sc1: written through the
// XCD's L2, read past it), so that no fence has to write back or drop all of
// an L2, which cost 190 us for one token over 131072 keys instead of 100.
constexpr int SC1 = 16;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t pieces_of(const float* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, -1, 0x00027000);
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Joins the pieces of a sequence's rows that workgroups x0 .. x1 left in the
// workspace.  Four columns of a row are a thread's, in one pass with a running
// maximum; while there are threads left the pieces are dealt to several.
template <class E, int D, int WAVES>
__device__ __forceinline__ void join_pieces(const AttendArgs& a, int q0, int rows, int hk, int x0, int x1, float* lds) {
  const __amdgpu_buffer_rsrc_t part = pieces_of(a.part), part_ml = pieces_of(a.part_ml);
  constexpr int THREADS = WAVES * 64, C4 = D / 4, AHEAD = 16;
  const int tid = threadIdx.x, n = x1 - x0 + 1;
  // row `row` of piece i
  auto at = [&](int i, int row) -> uint32_t { return ((hk * a.shares + x0 + i) * 2 + (i == 0)) * a.stream_rows + row; };
  const int cols = rows * C4, groups = cols <= THREADS / 2 ? THREADS / cols : 1;
  for (int c0 = 0; c0 < cols; c0 += THREADS) {
    const int grp = groups > 1 ? tid / cols : 0, c = groups > 1 ? tid - grp * cols : c0 + tid;
    const bool on = grp < groups && c < cols;
    const int row = on ? c / C4 : 0, d = on ? (c - row * C4) * 4 : 0;
    floatx4 y = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    for (int i0 = on ? grp : n; i0 < n; i0 += AHEAD * groups) {
      floatx4 z[AHEAD];
      float2 v[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = i0 + k * groups < n ? i0 + k * groups : i0;
        const uint32_t zr = at(i, row);
        v[k] = __builtin_bit_cast(float2, __builtin_amdgcn_raw_buffer_load_b64(part_ml, zr * 8, 0, SC1));
        z[k] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(part, (zr * D + d) * 4, 0, SC1));
      }
      float to = m;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) to = fmaxf(to, v[k].x);
      const float ms = to == -INFINITY ? 0.f : to, al = __builtin_amdgcn_exp2f(m - ms);
      m = to;
      l *= al;
      y *= al;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        if (i0 + k * groups < n) {
          const float f = __builtin_amdgcn_exp2f(v[k].x - ms);
          l += v[k].y * f;
          y += z[k] * f;
        }
    }
    if (groups > 1) {
      float* mine = lds + tid * 8;
      *(floatx4*)mine = y;
      mine[4] = m;
      mine[5] = l;
      __syncthreads();
      if (on && grp == 0) {
        float to = m;
        for (int k = 1; k < groups; ++k) to = fmaxf(to, lds[(tid + k * cols) * 8 + 4]);
        const float ms = to == -INFINITY ? 0.f : to, al = __builtin_amdgcn_exp2f(m - ms);
        m = to;
        l *= al;
        y *= al;
        for (int k = 1; k < groups; ++k) {
          const float* o = lds + (tid + k * cols) * 8;
          const float f = __builtin_amdgcn_exp2f(o[4] - ms);
          l += o[5] * f;
          y += *(const floatx4*)o * f;
        }
      }
      __syncthreads();
    }
    if (on && grp == 0) {
      const float f = l == 0.f ? 0.f : 1.f / l;
      const int tok = row / a.group, head = hk * a.group + row - tok * a.group;
      *(uint2*)(a.o + (q0 + tok) * a.o_stride + head * D + d) = make_uint2(pack2<E>(y[0] * f, y[1] * f), pack2<E>(y[2] * f, y[3] * f));
      if (a.lse && d == 0)
        a.lse[(int64_t)(q0 + tok) * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
    }
  }
}

// The steps of all sequences, one after the other, are dealt to the
// workgroups of a key head in equal shares, whatever the sequences' lengths.
// A share is made of pieces, one for each sequence that it touches: a piece
// that is all of its sequence goes straight to the output; of the others a
// workgroup has two at most, the end of a sequence (or its middle; slot 0) and
// the beginning of one (slot 1).  They go to the workspace, and the workgroup
// that brings a sequence's last piece joins them.
template <class E, int D, int RT, bool Q8, int AT_WAVES>
__global__ __launch_bounds__(AT_WAVES * 64, at_waves(D) / 4) void attend_stream_kernel(AttendArgs a) {
  constexpr int DT = D / 16, AT_STEP = AT_WAVES * AT_TILE;
  constexpr int PITCH = D + 4;                    // floats of a row in LDS
  __shared__ __attribute__((aligned(16))) float sums[AT_WAVES * 16 * PITCH];
  __shared__ float ml[AT_WAVES][RT * 16][2];
  __shared__ int last_piece[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
  const int hk = blockIdx.x % a.kv.kv_heads, x = blockIdx.x / a.kv.kv_heads;

  // The steps of all sequences, and this workgroup's share [at, to).  Every
  // wave finds them for itself, 64 sequences at a time.
  RowTile t;
  int64_t total = a.whole ? a.seqs : 0;
  int mine = 0;                                   // steps of sequence `lane`
  for (int s0 = a.whole ? a.seqs : 0; s0 < a.seqs; s0 += 64) {
    int n = seq_steps<AT_WAVES>(a, s0 + lane, hk, t);
    if (s0 == 0) mine = n;
    if (a.seqs > 1)
#pragma unroll
      for (int k = 1; k < 64; k *= 2) n += __shfl_xor(n, k);
    total += __builtin_amdgcn_readfirstlane(n);   // (64 times 2^23 at most)
  }
  const int shares = (int)(total < a.shares ? total : a.shares);
  if (x >= shares) return;
  int64_t at = div64(total * x, shares);
  const int64_t to = div64(total * (x + 1), shares);

  // the sequence of step `at`, and its first step (total > at: there is one)
  int s = a.whole ? x : (a.seqs > 1 ? a.seqs : 0);
  int64_t g0 = a.whole ? x : 0;
  for (int s0 = 0; s0 < a.seqs && s == a.seqs; s0 += 64) {
    const int n = s0 == 0 ? mine : seq_steps<AT_WAVES>(a, s0 + lane, hk, t);
    int sum = n;
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
      const int up = __shfl_up(sum, k);
      if (lane >= k) sum += up;
    }
    const uint64_t past = __ballot(g0 + sum > at);
    if (past) {
      const int i = __builtin_ctzll(past);
      s = s0 + i;
      g0 += __builtin_amdgcn_readlane(sum - n, i);
    } else {
      g0 += __builtin_amdgcn_readlane(sum, 63);
    }
  }
  // the pieces that are to be joined with others' (0: a sequence's end or middle, 1: its beginning)
  int64_t piece_g0[2] = {0, 0};
  int piece_s[2] = {-1, -1}, piece_n[2] = {0, 0}, piece_q0[2] = {0, 0}, piece_rows[2] = {0, 0};
  const __amdgpu_buffer_rsrc_t part = pieces_of(a.part), part_ml = pieces_of(a.part_ml);

  for (; at < to && s < a.seqs; ++s) {
    const int n = seq_steps<AT_WAVES>(a, s, hk, t);
    if (n == 0) {
      at += a.whole;                              // (a share of its own)
      continue;
    }
    const int off = (int)(at - g0), take = (int)(to - at < n - off ? to - at : n - off);
    const bool whole = take == n;
    const int c0 = t.beg + off * AT_STEP, c1 = off + take == n ? t.end : c0 + take * AT_STEP;
    Piece<E, D, RT, Q8, AT_WAVES> p;
    p.run(a, t, c0, c1);

    // join the waves
    if (g == 0)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        ml[wave][i * 16 + r][0] = p.m[i];
        ml[wave][i * 16 + r][1] = p.l[i];
      }
    const uint32_t slot = (hk * a.shares + x) * 2 + (off == 0);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      __syncthreads();
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        float* to = &sums[(wave * 16 + r) * PITCH];
        if constexpr (Q8) {                        // dimensions 8g .. of 32, from two operands in turn
          const floatx4 x = p.o[i][d & ~1], y = p.o[i][d | 1];
          const int e = 2 * (d & 1);
          *(floatx4*)&to[d / 2 * 32 + g * 8 + 2 * e] = (floatx4){x[e], y[e], x[e + 1], y[e + 1]};
        } else {
          *(floatx4*)&to[d * 16 + g * 4] = p.o[i][d];
        }
      }
      __syncthreads();
      for (int y0 = tid; y0 < 16 * (D / 8); y0 += AT_WAVES * 64) {
        const int rr = y0 / (D / 8), d0 = (y0 - rr * (D / 8)) * 8, row = i * 16 + rr;
        if (row >= t.rows) continue;
        float mt = -INFINITY, lt = 0.f;
#pragma unroll
        for (int w = 0; w < AT_WAVES; ++w) mt = fmaxf(mt, ml[w][row][0]);
        const float ms = mt == -INFINITY ? 0.f : mt;
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < AT_WAVES; ++w) {
          const float f = __builtin_amdgcn_exp2f(ml[w][row][0] - ms);
          lt += ml[w][row][1] * f;
          const float* z = &sums[(w * 16 + rr) * PITCH + d0];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] += z[j] * f;
        }
        if (!whole) {
          const uint32_t z = slot * a.stream_rows + row;
          const floatx4 lo = {y[0], y[1], y[2], y[3]}, hi = {y[4], y[5], y[6], y[7]};
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), part, (z * D + d0) * 4, 0, SC1);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), part, (z * D + d0) * 4 + 16, 0, SC1);
          if (d0 == 0)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, make_float2(mt, lt)), part_ml, z * 8, 0, SC1);
        } else {
          const int tok = row / a.group, head = hk * a.group + row - tok * a.group;
          const float f = lt == 0.f ? 0.f : 1.f / lt;
          u32x4 z;
#pragma unroll
          for (int j = 0; j < 4; ++j) z[j] = pack2<E>(y[2 * j] * f, y[2 * j + 1] * f);
          *(u32x4*)(a.o + (t.q0 + tok) * a.o_stride + head * D + d0) = z;
          if (a.lse && d0 == 0)
            a.lse[(int64_t)(t.q0 + tok) * a.q_heads + head] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * LN2;
        }
      }
    }

    if (!whole) {
      const int which = off == 0;
      piece_s[which] = s;
      piece_g0[which] = g0;
      piece_n[which] = n;
      piece_q0[which] = t.q0;
      piece_rows[which] = t.rows;
    }
    __syncthreads();
    at += take;
    g0 += n;
  }

  if (piece_s[0] < 0 && piece_s[1] < 0) return;
  // the pieces of the two sequences are those of workgroups x0 .. x1
  int x0[2], x1[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    x0[k] = piece_s[k] < 0 ? 0 : (int)mul_div_up(piece_g0[k] + 1, shares, total) - 1;
    x1[k] = piece_s[k] < 0 ? 0 : (int)mul_div_up(piece_g0[k] + piece_n[k], shares, total) - 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this thread's parts of the pieces are there for all
  __syncthreads();
  if (tid < 2) {
    const int ps = tid ? piece_s[1] : piece_s[0], others = tid ? x1[1] - x0[1] : x1[0] - x0[0];
    bool last = false;
    if (ps >= 0) {
      uint32_t* there = &a.arrived[(int64_t)ps * a.kv.kv_heads + hk];
      last = __hip_atomic_fetch_add(there, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)others;
      if (last) __hip_atomic_store(there, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);   // for the next call
    }
    last_piece[tid] = last;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k)
    if (last_piece[k]) join_pieces<E, D, AT_WAVES>(a, piece_q0[k], piece_rows[k], hk, x0[k], x1[k], sums);
}

// Joins the splits of the tile kernel: four columns of a row are a thread's,
// in one pass with a running maximum.  Bound by latency (5 us for 1193 tokens
// of 16 heads of 64 in two splits).
constexpr int join_rows(int D) { return 1024 / D; }   // of a workgroup
template <class E, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  constexpr int C4 = D / 4, AHEAD = 4, JOIN_ROWS = join_rows(D);
  const int hk = blockIdx.x % a.kv.kv_heads;
  RowTile t;
  if (!find_tile(a, blockIdx.x / a.kv.kv_heads, hk, JOIN_ROWS, 1, t)) return;
  const int64_t step = a.T * a.q_heads;                      // rows of a split
  const int i = threadIdx.x, row = t.row0 + i / C4, d = i % C4 * 4;
  if (i >= JOIN_ROWS * C4 || row >= t.rows) return;
  const int tok = row / a.group, head = hk * a.group + row - tok * a.group;
  const int64_t orow = (int64_t)(t.q0 + tok) * a.q_heads + head;
  floatx4 y = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  for (int x0 = 0; x0 < a.splits; x0 += AHEAD) {
    floatx4 z[AHEAD];
    float2 v[AHEAD];
    float to = m;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int64_t at = orow + (x0 + k < a.splits ? x0 + k : x0) * step;
      v[k] = *(const float2*)(a.part_ml + at * 2);
      z[k] = *(const floatx4*)(a.part + at * D + d);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) to = fmaxf(to, v[k].x);
    const float ms = to == -INFINITY ? 0.f : to, al = __builtin_amdgcn_exp2f(m - ms);
    m = to;
    l *= al;
    y *= al;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      // (a split without keys for the row leaves its sums unwritten)
      if (x0 + k >= a.splits || (v[k].x == -INFINITY && v[k].y == 0.f)) continue;
      const float f = __builtin_amdgcn_exp2f(v[k].x - ms);
      l += v[k].y * f;
      y += z[k] * f;
    }
  }
  const float f = l == 0.f ? 0.f : 1.f / l;
  *(uint2*)(a.o + (t.q0 + tok) * a.o_stride + head * D + d) = make_uint2(pack2<E>(y[0] * f, y[1] * f), pack2<E>(y[2] * f, y[3] * f));
  if (a.lse && d == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

template <class E, int D>
hipError_t join_launch(const AttendArgs& a, hipStream_t st) {
  if (a.splits == 1) return hipSuccess;
  return launch_kernel(attend_join_kernel<E, D>, dim3((unsigned)(tile_count(a, join_rows(D)) * a.kv.kv_heads)), 256, 0, st, a);
}

template <class E, int D, bool Q8, int WAVES>
hipError_t stream_w(const AttendArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.shares * a.kv.kv_heads));
  if constexpr (D < 256)
    if (a.stream_rows > 16) return launch_kernel(attend_stream_kernel<E, D, 2, Q8, WAVES>, grid, WAVES * 64, 0, st, a);
  return launch_kernel(attend_stream_kernel<E, D, 1, Q8, WAVES>, grid, WAVES * 64, 0, st, a);
}

template <class E, int D>
hipError_t stream_d(const AttendArgs& a, hipStream_t st) {
  if (!a.kv.k_scale) return stream_w<E, D, false, at_waves(D)>(a, st);
  if constexpr (at_waves(D) != 4)
    if (a.halved) return stream_w<E, D, true, 4>(a, st);
  return stream_w<E, D, true, at_waves(D)>(a, st);
}

template <class E>
hipError_t launch_e(const AttendArgs& a, bool join, hipStream_t st) {
  switch (a.kv.head_dim) {
    case 64: return join ? join_launch<E, 64>(a, st) : stream_d<E, 64>(a, st);
    case 96: return join ? join_launch<E, 96>(a, st) : stream_d<E, 96>(a, st);
    case 128: return join ? join_launch<E, 128>(a, st) : stream_d<E, 128>(a, st);
    default: return join ? join_launch<E, 256>(a, st) : stream_d<E, 256>(a, st);
  }
}

__global__ __launch_bounds__(256) void zero_kernel(AttendArgs a) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.counters; i += (int64_t)gridDim.x * 256) a.arrived[i] = 0;
}

}  // namespace

hipError_t launch_attend(const AttendArgs& args, const AttendPlan& p, int dtype, hipStream_t st) {
  AttendArgs a = args;
  a.part_ml = a.part + attend_part_rows(a, p) * a.kv.head_dim;
  a.stream_rows = p.stream_rows;
  a.shares = p.splits;
  a.whole = p.whole;
  a.halved = p.halved;
  if (a.fresh) {
    const int64_t wgs = (a.counters + 255) / 256;
    const hipError_t e = launch_kernel(zero_kernel, dim3((unsigned)(wgs < 1024 ? wgs : 1024)), 256, 0, st, a);
    if (e != hipSuccess) return e;
  }
  if (p.tile_rows) {
    a.splits = p.tile_splits;
    a.per_split = p.tile_per;
    hipError_t e = launch_attend_tile(a, p, dtype, st);
    if (e == hipSuccess) e = dtype == DT_F16 ? launch_e<f16>(a, true, st) : launch_e<bf16>(a, true, st);
    if (e != hipSuccess) return e;
  }
  if (p.stream_rows == 0) return hipSuccess;
  return dtype == DT_F16 ? launch_e<f16>(a, false, st) : launch_e<bf16>(a, false, st);
}

}  // namespace fcg
