// Attention of chunks over the paged cache (many query rows for each key
// head): tiles of rows against tiles of 64 keys in LDS.
//
// The rows of one key head are the tokens times the group of query heads that
// share it, token by token; a wave has 32 of them, a workgroup 32 WAVES, and
// the keys and values of a tile are read once for all.
//
// S^T = K Q^T and O^T = V^T P^T on 32x32x16 matrix instructions: a lane holds
// scores of one query row (column lane % 32).  Operand row 8a + 4h + b of the
// first product is key 16 (a / 2) + 8h + 4 (a % 2) + b of 32, so that lane
// half h ends with keys 16s + 8h .. 16s + 8h + 7, the elements of its operand
// in the second product: the weights stay in their registers, and the maximum
// needs one exchange between lanes.  The cache's 16-byte pieces are the
// operands' shape, so a tile is a plain copy of pieces ([D/8][64] of keys,
// [8][D] of values) whatever the page size, and every LDS read is a
// contiguous 1024 bytes.
//
// The reference point m of a row's exponentials is LIFT below a maximum of some
// earlier tile.  A tile's weights are taken against it as it stands; only if
// their sum then passes MOST (or m is still -inf) is the tile's maximum looked
// for, m moved and the weights taken again.  Weights stay below MOST, in range
// of f16, and most tiles cost no maximum and leave the sums as they are (f16:
// 32 equal weights of a lane make 2^13, so that scores may grow by 3 to 8
// powers of two before m moves).
//
// Bound by the matrix and vector instructions of a wave's 32 rows, and by the
// clock that the card holds under them: 4096 tokens over 8192 keys (32 heads
// of 128 on 8 key heads, f16) take 398 to 431 us on different cards, 960 to
// 1040 TFLOP/s, where a product of two 8192 x 8192 matrices reaches 1200; the
// matrix cores are busy for 397 of 798 thousand cycles, at about 2 GHz.  4
// waves of 64 rows spilled (454 TFLOP/s).  The weights are rounded to the
// cache's type for the second product (off by 2^-8 of a bf16 weight, by 2^-11 of
// an f16 one or 2^-33 of the row's largest); totals, products and statistics
// are f32, the totals of the unrounded weights.
#include <math.h>

#include <type_traits>

#include "attend.h"

namespace fcg {
namespace {

constexpr int KT = 64;                           // keys of a tile

template <int D, int WAVES>
struct TileCfg {
  static constexpr int ROWS = WAVES * 32;
  static constexpr int KB = KT * D * 2;          // bytes of a tile's keys, and of its values
  static constexpr int STAGE = 2 * KB;           // values of a tile, then keys of the next
  static constexpr int STAGES = WAVES > 4 ? 3 : 2;   // (a wave that runs behind needs a third)
  static constexpr int LDS = STAGES * STAGE + 16;
  static constexpr int NI = D / 8 / WAVES;       // 1 KB pieces of keys per wave
};

// the workgroup's LDS accesses are done; loads from memory stay in flight
__device__ __forceinline__ void half_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// half_barrier() of the waves for which `on`, the same in every lane, holds (a
// branch in the source, with the sums live across it, costs registers).
__device__ __forceinline__ void barrier_if(bool on) {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 1f\n\ts_barrier\n1:" ::"s"(__builtin_amdgcn_readfirstlane((int)on)) : "memory", "scc");
  __builtin_amdgcn_sched_barrier(0);
}

// BIG: pages of KT keys or more, so that a tile is in one page and where it
// begins is the same in every lane.
// Q8: a cache of 8 bits.  Its codes become values of E on their way to LDS, once
// for all waves (exactly: serving.h), and nothing after that knows of them.
template <class E, int D, int WAVES, bool BIG, bool Q8>
__global__ __launch_bounds__(WAVES * 64, D <= 128 ? 2 : 1) void attend_tile_kernel(AttendArgs a) {
  using C = TileCfg<D, WAVES>;
  static_assert(D / 8 % WAVES == 0, "pieces per wave");
  constexpr int KS = D / 16, DB = D / 32, NI = C::NI, READS = 2 * KS + 4 * DB, AHEAD = 6;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  int b = blockIdx.x;
  const int hk = b % a.kv.kv_heads;
  b /= a.kv.kv_heads;
  const int split = b % a.splits;
  b /= a.splits;
  RowTile t;
  if (!find_tile(a, b, hk, C::ROWS, KT, t)) return;
  int c0, c1;
  split_range(t, split, a.splits, a.per_split, c0, c1);

  const int ps = 1 << a.kv.page_shift;
  constexpr int B = Q8 ? 1 : 2;                  // bytes of an element
  typedef typename std::conditional<Q8, uint2, u32x4>::type Raw;   // a piece in memory
  const int64_t page_bytes = (int64_t)a.kv.kv_heads * ps * D * B;
  const uint8_t* kbase = (const uint8_t*)a.kv.k + (int64_t)hk * ps * D * B;
  const uint8_t* vbase = (const uint8_t*)a.kv.v + (int64_t)hk * ps * D * B;
  const int32_t* table = a.table + t.s * a.table_stride;

  // rows of this wave
  const int wrow0 = t.row0 + wave * 32;
  const int wlast = (wrow0 + 32 < t.rows ? wrow0 + 32 : t.rows) - 1;
  const bool any_rows = wrow0 < t.rows;
  const int wlo = t.base + wrow0 / a.group, whi = any_rows ? t.base + wlast / a.group : -1;

  // this lane's row
  const int row = wrow0 + r;
  const bool there = row < t.rows;
  const int tok = row / a.group, pos = there ? t.base + tok : -1;
  float m = there ? -INFINITY : 0.f, l = 0.f;    // reference point, total (of the lane half's keys)
  u32x4 q[KS];
  const uint16_t* p = a.q + (t.q0 + tok) * a.q_stride + (hk * a.group + row - tok * a.group) * D + h * 8;
#pragma unroll
  for (int k = 0; k < KS; ++k) q[k] = there ? *(const u32x4*)(p + k * 16) : (u32x4){0, 0, 0, 0};

  floatx16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[d][x] = 0.f;

  // Key tok0 + lane (BIG: all of the tile's): its entry in the table (read a
  // tile before it is looked at, so that nothing waits for it), its page, -1
  // for none of the pool (its keys take no part), where the page begins in
  // bytes, and which of the tile's keys have a page.
  auto entry_at = [&](int tok0) -> int {
    const int at = BIG ? tok0 : tok0 + lane, key = at < c1 ? at : c1 - 1;
    return *(const int32_t*)((const uint8_t*)table + (uint32_t)(key >> a.kv.page_shift) * 4u);
  };
  auto page_of = [&](int tok0, int entry) -> int {
    if constexpr (BIG) entry = __builtin_amdgcn_readfirstlane(entry);
    return tok0 + (BIG ? 0 : lane) < c1 && (unsigned)entry < (uint64_t)a.kv.pages ? entry : -1;
  };
  auto start_of = [&](int page) -> uint64_t { return (uint32_t)(page < 0 ? 0 : page) * (uint64_t)(uint32_t)page_bytes; };
  auto paged = [&](int tok0, int page) -> uint64_t {
    if constexpr (!BIG) return __ballot(page >= 0);
    return page < 0 ? 0 : (c1 - tok0 < KT ? ((uint64_t)1 << (c1 - tok0)) - 1 : ~0ull);
  };
  // pieces of keys and of values on their way to LDS
  Raw kraw[NI], vraw[NI];
  u32x4 vst[NI];
  // Q8: the stored exponents of the lane's key, and of the 8 keys of each piece
  // of values.  A wave's pieces are of 8 / WAVES times 8 keys, so that but for 96
  // dimensions these are the same in every lane and taken apart once, by scalar
  // instructions (by vector instructions for each piece: 4096 tokens over 8192
  // keys 444 us instead of 402).
  constexpr bool SAME = D % 64 == 0;
  constexpr int VG = SAME ? 8 / WAVES : NI;
  uint32_t ke = 0;
  uint2 ve[VG];
  // where the scales of a page that begins `start` bytes into the pool begin: a byte for D
  auto scales_at = [&](const uint8_t* scales, uint64_t start, int key) -> const uint8_t* {
    return scales + start / D + (uint32_t)(hk * ps + (key & (ps - 1)));
  };
  auto load_k = [&](int tok0, uint64_t start) {
    if constexpr (BIG) {
      const uint8_t* kp = kbase + start + (uint32_t)((tok0 & (ps - 1)) * 8 * B + wave * NI * ps * 8 * B);
#pragma unroll
      for (int i = 0; i < NI; ++i) kraw[i] = *(const Raw*)(kp + (uint32_t)(i * ps * 8 * B) + (uint32_t)lane * 8 * B);
    } else {
      const uint8_t* kp = kbase + start + (((tok0 + lane) & (ps - 1)) * 8 * B + wave * NI * ps * 8 * B);
#pragma unroll
      for (int i = 0; i < NI; ++i) kraw[i] = *(const Raw*)(kp + (uint32_t)(i * ps * 8 * B));
    }
    if constexpr (Q8) ke = *scales_at(a.kv.k_scale, start, tok0 + lane);
  };
  auto load_v = [&](int tok0, uint64_t start) {
    if constexpr (Q8 && SAME)
#pragma unroll
      for (int i = 0; i < VG; ++i) {
        const int k8 = wave * VG + i;
        uint64_t at = start;
        if constexpr (!BIG)
          at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(start >> 32), k8 * 8) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)start, k8 * 8);
        ve[i] = *(const uint2*)scales_at(a.kv.v_scale, at, tok0 + k8 * 8);
      }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if constexpr (BIG) {                       // pieces of a page follow each other
        vraw[i] = *(const Raw*)(vbase + start + (uint32_t)((tok0 & (ps - 1)) * (D * B) + (wave * NI + i) * 512 * B) + (uint32_t)lane * 8 * B);
        if constexpr (Q8 && !SAME) ve[i] = *(const uint2*)scales_at(a.kv.v_scale, start, tok0 + ((wave * NI + i) * 64 + lane) / D * 8);
      } else if constexpr (D % 64 == 0) {        // the wave's 64 pieces are of the same 8 keys
        const int p = (wave * NI + i) * 64, k8 = p / D, d = p - k8 * D;
        const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(start >> 32), k8 * 8) << 32 |
                            (uint32_t)__builtin_amdgcn_readlane((int)start, k8 * 8);
        const uint8_t* vp = vbase + at + (uint32_t)(((tok0 + k8 * 8) & (ps - 1)) * (D * B) + d * 8 * B);
        vraw[i] = *(const Raw*)(vp + (uint32_t)lane * 8 * B);
      } else {
        const int p = (wave * NI + i) * 64 + lane, k8 = p / D, d = p - k8 * D;
        const uint64_t at = __shfl(start, k8 * 8);
        vraw[i] = *(const Raw*)(vbase + at + (uint32_t)(((tok0 + k8 * 8) & (ps - 1)) * (D * B) + d * 8 * B));
        if constexpr (Q8) ve[i] = *(const uint2*)scales_at(a.kv.v_scale, at, tok0 + k8 * 8);
      }
    }
  };
  int* const flag = (int*)(smem + C::STAGES * C::STAGE);   // some value was taken out
  if (tid == 0) *flag = 0;
  __syncthreads();
  uint8_t* const mine = smem + (wave * NI * 64 + lane) * 16;
  auto store_v = [&](int at) {                   // at: where the tile's pieces begin
#pragma unroll
    for (int i = 0; i < NI; ++i) *(u32x4*)(mine + at + i * 1024) = vst[i];
  };
  auto store_k = [&](int at) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if constexpr (Q8) {
        const float by = __builtin_bit_cast(float, held_exponent<E>(ke) << 23);
        *(u32x4*)(mine + at + i * 1024) = codes8<E>(kraw[i].x, kraw[i].y, by);
      } else {
        *(u32x4*)(mine + at + i * 1024) = kraw[i];
      }
    }
  };
  auto piece_of = [&](const Raw& x, const uint2& e) -> u32x4 {   // of values
    if constexpr (Q8) return ValueScales<E>(e).values(x.x, x.y);
    else return x;
  };
  // the key of operand row r, in pieces
  const int krow = ((r >> 4) & 1) * 16 + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3);
  const uint8_t* const kop = smem + C::KB + (h * KT + krow) * 16;
  const uint8_t* const vop = smem + (h * D + r) * 16;

  // ok: bit j: key tok0 + j has a page
  // every row from position lo to hi sees every key of the tile: no mask
  auto is_open = [&](int tok0, uint64_t ok, int lo, int hi) {
    return ok == ~0ull && tok0 <= lo - (KT - 1) && tok0 > (a.window > 0 ? hi - a.window : -1);
  };
  // how many of the tile's keys 8x .. 8x + 7 are there (the first ones)
  auto have = [&](int tok0, uint64_t ok, int x) -> int {
    const int left = c1 - (tok0 + 8 * x);
    return (ok >> (8 * x) & 1) ? (left < 8 ? left : 8) : 0;
  };
  // A masked key's weight is 0, which must not meet an infinite or NaN value:
  // of tiles with masked keys those are stored as 0 and added at the end.
  auto clean = [&](int tok0, uint64_t ok) {
    if constexpr (Q8 && SAME) {
#pragma unroll
      for (int g = 0; g < VG; ++g) {
        const ValueScales<E> scales(make_uint2(__builtin_amdgcn_readfirstlane(ve[g].x), __builtin_amdgcn_readfirstlane(ve[g].y)));
#pragma unroll
        for (int i = g * NI / VG; i < (g + 1) * NI / VG; ++i) vst[i] = scales.values(vraw[i].x, vraw[i].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) vst[i] = piece_of(vraw[i], ve[SAME ? 0 : i]);
    }
    if (is_open(tok0, ok, t.lo, t.hi)) return;
    if (ok != ~0ull)
#pragma unroll
      for (int i = 0; i < NI; ++i) vst[i] &= keep_keys(have(tok0, ok, ((wave * NI + i) * 64 + lane) / D));
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) bad |= any_nonfinite<E>(vst[i]);
    if (__any(bad != 0)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) take_nonfinite<E>(vst[i]);
      *flag = 1;
    }
  };

  floatx16 sc[2];                            // scores
  u32x4 w[4];                                // weights
  auto scores = [&](int stage) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 16; ++x) sc[n][x] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const u32x4 kk = *(const u32x4*)(kop + stage + k * 2 * KT * 16 + n * 32 * 16);
        sc[n] = Mat<E>::mfma32(kk, q[k], sc[n]);
      }
  };
  auto weights = [&](int tok0, uint64_t ok) {
    if (!is_open(tok0, ok, wlo, whi)) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int key0 = tok0 + s * 16 + 8 * h, n = have(tok0, ok, 2 * s + h);
        const int top = pos - key0 < n ? pos - key0 : n - 1;       // last key that the row sees
        const int low = a.window > 0 ? pos - a.window - key0 : -1;    // last before its window
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j > top || j <= low) sc[s >> 1][(s & 1) * 8 + j] = -INFINITY;
      }
    }
    auto take = [&](float ms) -> float {       // weights against the reference point ms, their sum
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = sc[s >> 1][(s & 1) * 8 + 2 * j], y = sc[s >> 1][(s & 1) * 8 + 2 * j + 1];
          const float px = __builtin_amdgcn_exp2f(fmaf(x, a.scale_log2, -ms)), py = __builtin_amdgcn_exp2f(fmaf(y, a.scale_log2, -ms));
          w[s][j] = pack2<E>(px, py);
          sum[0] += px;
          sum[1] += py;
        }
      return sum[0] + sum[1];
    };
    float sum = take(m);
    if (__any(!(sum <= Mat<E>::MOST))) {               // (m = -inf makes it infinite or NaN)
      float mx = fmaxf(sc[0][0], sc[1][0]);
#pragma unroll
      for (int x = 1; x < 16; ++x) mx = max3(mx, sc[0][x], sc[1][x]);
      mx = fmaxf(mx, other_half(mx));
      const float to = fmaxf(m, reference_of<E>(mx, a.scale_log2)), ms = to == -INFINITY ? 0.f : to;
      const float al = __builtin_amdgcn_exp2f(m - ms);
      m = to;
      l *= al;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[d][x] *= al;
      sum = take(ms);
    }
    l += sum;
  };
  auto values = [&](int stage) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const u32x4 v = *(const u32x4*)(vop + stage + (s * 2 * D + d * 32) * 16);
        o[d] = Mat<E>::mfma32(v, w[s], o[d]);
      }
  };

  // Stage n of the ring has the values of tile n - 1 and the keys of tile n.
  // Of the loop's two halves one is vector work (weights), one matrix work.
  // With 8 waves, waves 4 to 7 run one half behind waves 0 to 3, their
  // neighbours on the SIMDs, so that one of the two kinds of work is always
  // next to the other.  Stage n is stored at the end of the first halves of tile
  // n - 2 and read in the second halves of tile n - 1.
  if (c0 < c1) {
    const int p0 = page_of(c0, entry_at(c0)), p1 = page_of(c0 + KT, entry_at(c0 + KT));
    const int p2 = page_of(c0 + 2 * KT, entry_at(c0 + 2 * KT));
    int e3 = entry_at(c0 + 3 * KT);
    uint64_t ok = paged(c0, p0), ok1 = paged(c0 + KT, p1), ok2 = paged(c0 + 2 * KT, p2), start2 = start_of(p2);
    load_k(c0, start_of(p0));
    store_k(C::KB);
    load_v(c0, start_of(p0));
    load_k(c0 + KT, start_of(p1));
    clean(c0, ok);
    store_v(C::STAGE);
    store_k(C::STAGE + C::KB);
    load_v(c0 + KT, start_of(p1));
    load_k(c0 + 2 * KT, start2);
    half_barrier();
    scores(0);
    if constexpr (WAVES > 4) barrier_if(wave >= 4);
    if constexpr (C::STAGES == 2) half_barrier();
    int cur = C::STAGE, next = C::STAGES == 2 ? 0 : 2 * C::STAGE;
    for (int tok0 = c0; tok0 < c1; tok0 += KT) {
      const int p3 = page_of(tok0 + 3 * KT, e3);
      const uint64_t ok3 = paged(tok0 + 3 * KT, p3), start3 = start_of(p3);
      weights(tok0, ok);
      __builtin_amdgcn_sched_barrier(0);
      clean(tok0 + KT, ok1);
      store_v(next);
      store_k(next + C::KB);
      half_barrier();
      // (past the last tile the loads are of keys without a page, never read)
      load_v(tok0 + 2 * KT, start2);
      load_k(tok0 + 3 * KT, start3);
      e3 = entry_at(tok0 + 4 * KT);
      values(cur);
      scores(cur);
      // LDS reads run AHEAD operands before the matrix instructions that use
      // them (left alone, two: every pair then waits for the LDS)
#pragma unroll
      for (int x = 0; x < READS + AHEAD; ++x) {
        if (x >= AHEAD) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (x < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      half_barrier();
      cur = next;
      next = next + C::STAGE == C::STAGES * C::STAGE ? 0 : next + C::STAGE;
      ok = ok1;
      ok1 = ok2;
      ok2 = ok3;
      start2 = start3;
    }
    if constexpr (WAVES > 4) barrier_if(wave < 4);
  }

  if (c0 < c1 && *flag) {                        // (all waves have passed the loop's last barrier)
    for (int tok0 = c0; tok0 < c1; tok0 += KT) {
      const int page = page_of(tok0, entry_at(tok0));
      const uint64_t ok = paged(tok0, page);
      if (is_open(tok0, ok, t.lo, t.hi)) continue;
      const int in_page = tok0 & (ps - 1);
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        floatx16 c;
#pragma unroll
        for (int x = 0; x < 16; ++x) c[x] = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int key0 = tok0 + s * 16 + 8 * h, n = have(tok0, ok, 2 * s + h);
          const u32x4 one = seen_ones<E>(pos - key0 < n ? pos - key0 : n - 1, a.window > 0 ? pos - a.window - key0 : -1);
          const int pg = BIG ? page : __shfl(page, s * 16 + 8 * h);
          const Raw x = *(const Raw*)(vbase + start_of(pg) +
                                      ((((in_page + s * 16 + 8 * h) & (ps - 1)) >> 3) * D + d * 32 + r) * 8 * B);
          uint2 e = {0, 0};
          if constexpr (Q8) e = *(const uint2*)scales_at(a.kv.v_scale, start_of(pg), key0);
          const u32x4 v = piece_of(x, e);
          c = Mat<E>::mfma32(nonfinite_codes<E>(v & keep_keys(n)), one, c);
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) o[d][x] += nonfinite_sum(c[x]);
      }
    }
  }

  const float lt = l + __shfl_xor(l, 32);
  const int head = hk * a.group + row - tok * a.group;
  const int64_t orow = (int64_t)(t.q0 + tok) * a.q_heads + head;
  if (a.splits > 1) {
    if (there) {
      const int64_t at = (int64_t)split * a.T * a.q_heads + orow;
      if (h == 0) *(float2*)(a.part_ml + at * 2) = make_float2(m, lt);
      if (c0 < c1) {
        float* p = a.part + at * D + 4 * h;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *(floatx4*)(p + d * 32 + 8 * x) =
                (floatx4){o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
      }
    }
    return;
  }
  // rows out: through LDS (the loop's last barrier has passed: no wave reads
  // the tiles any more)
  const float f = lt == 0.f ? 0.f : 1.f / lt;
  // 16-byte chunk c of row r at place c ^ (r & SWZ) of the row, for the banks
  constexpr int SWZ = D == 96 ? 3 : 7;
  static_assert(WAVES * 32 * D * 2 <= C::STAGES * C::STAGE, "rows fit");
  uint8_t* mem = smem + wave * 32 * D * 2;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint2 z;
      z.x = pack2<E>(o[d][4 * x] * f, o[d][4 * x + 1] * f);
      z.y = pack2<E>(o[d][4 * x + 2] * f, o[d][4 * x + 3] * f);
      *(uint2*)(mem + r * (D * 2) + ((d * 4 + x) ^ (r & SWZ)) * 16 + h * 8) = z;
    }
  if (a.lse && h == 0 && there) a.lse[orow] = lt == 0.f ? -INFINITY : (m + log2f(lt)) * LN2;
  // (within a wave: LDS operations complete in order)
  __builtin_amdgcn_wave_barrier();
  for (int x = lane; x < 32 * (D / 8); x += 64) {
    const int rr = x / (D / 8), c = x - rr * (D / 8), row2 = wrow0 + rr;
    if (row2 < t.rows) {
      const int tok2 = row2 / a.group, head2 = hk * a.group + row2 - tok2 * a.group;
      *(u32x4*)(a.o + (t.q0 + tok2) * a.o_stride + head2 * D + c * 8) =
          *(const u32x4*)(mem + rr * (D * 2) + (c ^ (rr & SWZ)) * 16);
    }
  }
}

template <class E, int D, int WAVES, bool BIG, bool Q8>
hipError_t tile_launch(const AttendArgs& a, hipStream_t st) {
  using C = TileCfg<D, WAVES>;
  static std::atomic<uint64_t> raised{0};
  const hipError_t e = raise_lds_limit((const void*)attend_tile_kernel<E, D, WAVES, BIG, Q8>, C::LDS, raised);
  if (e != hipSuccess) return e;
  const int64_t wgs = tile_count(a, C::ROWS) * a.splits * a.kv.kv_heads;
  return launch_kernel(attend_tile_kernel<E, D, WAVES, BIG, Q8>, dim3((unsigned)wgs), WAVES * 64, C::LDS, st, a);
}

template <class E, int D, int WAVES>
hipError_t tile_w(const AttendArgs& a, hipStream_t st) {
  const bool big = (1 << a.kv.page_shift) >= KT;
  if (a.kv.k_scale) return big ? tile_launch<E, D, WAVES, true, true>(a, st) : tile_launch<E, D, WAVES, false, true>(a, st);
  return big ? tile_launch<E, D, WAVES, true, false>(a, st) : tile_launch<E, D, WAVES, false, false>(a, st);
}

template <class E, int D>
hipError_t tile_d(const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  if constexpr (D == 64 || D == 128)
    if (p.tile_rows == 256) return tile_w<E, D, 8>(a, st);
  return tile_w<E, D, 4>(a, st);
}

template <class E>
hipError_t tile_e(const AttendArgs& a, const AttendPlan& p, hipStream_t st) {
  switch (a.kv.head_dim) {
    case 64: return tile_d<E, 64>(a, p, st);
    case 96: return tile_d<E, 96>(a, p, st);
    case 128: return tile_d<E, 128>(a, p, st);
    default: return tile_d<E, 256>(a, p, st);
  }
}

}  // namespace

hipError_t launch_attend_tile(const AttendArgs& a, const AttendPlan& p, int dtype, hipStream_t st) {
  return dtype == DT_F16 ? tile_e<f16>(a, p, st) : tile_e<bf16>(a, p, st);
}

}  // namespace fcg
