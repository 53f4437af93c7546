// Shared by the serving operators (paged key/value cache, attention over it,
// logits processing): kernel arguments, launchers and device helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "common.h"
#include "internal.h"

namespace fcg {

typedef __bf16 bf16;
typedef float floatx16 __attribute__((ext_vector_type(16)));

// Element types of the C-ABI (FC_GGUF_F16, FC_GGUF_BF16, FC_GGUF_F32).
constexpr int DT_F16 = 0;
constexpr int DT_BF16 = 1;
constexpr int DT_F32 = 2;

// The paged cache.  K page: [kv_heads][D/8][ps][8], V page: [kv_heads][ps/8][D][8]
// elements.  Both are made of 16-byte pieces, 8 head dimensions of one token
// (K) and 8 tokens of one head dimension (V): the two shapes in which the
// matrix instructions' operands hold 8 consecutive values of the summed index
// in one lane, for K.Q^T (summed over dimensions) and V^T.P^T (over tokens).
// In 8 bits the shapes are the same with e4m3 codes as elements, pieces of 8
// bytes, and each token and key head has two scales, [kv_heads][ps] bytes of a
// page: the exponents of powers of two, biased by 127.
struct KvPages {
  void* k;
  void* v;
  uint8_t* k_scale;    // null: 16 bits
  uint8_t* v_scale;
  int64_t pages;
  int page_shift;      // log2(tokens per page), 4 .. 8
  int kv_heads;
  int head_dim;
};

// Launches kernel(args) and returns this launch's own status, which is then not
// left behind as well.  (After <<<>>> there is only the thread's last error,
// which an earlier call of anyone may have left: the launch would be reported
// as failed.)
template <class Args>
hipError_t launch_kernel(void (*kernel)(Args), dim3 grid, int threads, size_t lds, hipStream_t st, const Args& args) {
  void* p[] = {const_cast<Args*>(&args)};
  const hipError_t e = hipLaunchKernel((const void*)kernel, grid, dim3(threads), p, lds, st);
  if (e != hipSuccess) (void)hipGetLastError();
  return e;
}

struct AppendArgs {
  KvPages kv;
  const uint16_t* q;   // [T][q_heads][D], row strides in elements
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const int32_t* slots;       // [T]
  const int32_t* positions;   // [axes][T]
  const float* inv_freq;      // [rot/2] or null: no rotation
  const int32_t* pair_axis;   // [rot/2] or null: axis 0
  int64_t T;
  int q_heads, rot, axes, interleaved;
  float rope_scale;
  const float* q_norm;        // [D], or [heads][D] with stride D; null: none
  const float* k_norm;
  int q_norm_stride, k_norm_stride;   // from head to head: 0 or D
  float eps;
  int tokens_per_wg, y_splits;
};
hipError_t launch_kv_append(const AppendArgs& a, int dtype, int num_cu, hipStream_t st);

struct AttendArgs {
  KvPages kv;
  const uint16_t* q;
  uint16_t* o;
  float* lse;                 // [T][q_heads] or null
  int64_t q_stride, o_stride;
  const int32_t* cu_q;        // [seqs + 1]
  const int32_t* kv_lens;     // [seqs]
  const int32_t* table;       // [seqs][table_stride], table_w entries used
  int64_t table_stride;
  int64_t T;
  int table_w, seqs, q_heads, group, max_q, window;
  float scale_log2;           // scale * log2(e)
  float* part;                // partial sums, and
  float* part_ml;             // their reference points and totals
  int splits, per_split;      // splits of the tile kernel; keys of a split
  int stream_rows;            // most rows of a streamed sequence; 0: none is streamed
  int shares;                 // workgroups of the streaming kernel for each key head
  bool whole;                 // each of them has a sequence of its own
  bool halved;                // and has 4 waves (of 8 bits)
  uint32_t* arrived;          // [seqs][kv_heads] pieces of a sequence that are there; 0 between calls
  int64_t counters;           // entries of `arrived`
  bool fresh;                 // they are to be cleared first
};
// Sequences with at most stream_rows rows (tokens times the group) for each
// key head are the streaming kernel's, the others the tile kernel's; the
// lengths are known on the device only, so where max_q allows both, both are
// launched and a workgroup without rows of its kind ends at once.
constexpr int at_stream_rows(int D) { return D == 256 ? 16 : 32; }   // at most (two row tiles of 256 dimensions do not fit a wave's registers)
// The streaming kernel: keys per wave and step, and waves of a workgroup, 8
// (two on each SIMD, of 256 registers) or 4 where a wave needs more.
constexpr int AT_TILE = 32;
constexpr int at_waves(int D) { return D == 256 ? 4 : 8; }
constexpr int at_step(int D) { return at_waves(D) * AT_TILE; }
constexpr int64_t kMaxWorkgroups = (int64_t)1 << 23;   // of 512 threads: fewer than these
struct AttendPlan {
  int stream_rows;            // most rows of a streamed sequence
  int splits;                 // shares of the streaming kernel
  bool whole;                 // of one sequence each
  bool halved;                // by 4 waves instead of 8
  int tile_rows;              // rows of a workgroup of the tile kernel; 0: not launched
  int tile_splits, tile_per;
};
AttendPlan attend_plan(const AttendArgs& a, int num_cu);
size_t attend_part_rows(const AttendArgs& a, const AttendPlan& p);
size_t attend_workspace_bytes(const AttendArgs& a, const AttendPlan& p);
hipError_t launch_attend(const AttendArgs& a, const AttendPlan& p, int dtype, hipStream_t st);

// most tiles of `rows` rows that the sequences of a key head have
inline int64_t tile_count(const AttendArgs& a, int rows) {
  const int64_t by_rows = a.T * a.group / rows + a.seqs, each = ((int64_t)a.max_q * a.group + rows - 1) / rows * a.seqs;
  return by_rows < each ? by_rows : each;
}

// A bound of attend_workspace_bytes over this call and all that are smaller in
// T, seqs, max_q, table width and heads, whatever their windows: a workspace
// of these bytes serves them all, though a smaller call may need more than a
// larger one (4096 tokens fill the CUs unsplit, 64 need 34 MB).
inline size_t attend_workspace_bound(const AttendArgs& a, int num_cu) {
  const int64_t D = a.kv.head_dim, hk = a.kv.kv_heads, held = (int64_t)a.table_w << a.kv.page_shift;
  const int64_t rows = (int64_t)a.max_q * a.group, step = at_step((int)D), few = at_stream_rows((int)D);
  int64_t stream = 0, tile = 0;
  if (held > 4 * step) {                         // shares of the streaming kernel: one a CU, one a step
    const int64_t steps = (held + step - 1) / step * a.seqs;
    int64_t shares = num_cu / hk < steps ? num_cu / hk : steps;
    shares = shares < 1 ? 1 : shares;
    stream = shares * hk * 2 * (rows < few ? rows : few);
  }
  // Splits of the tile kernel: of 256 keys at least; about num_cu / tiles,
  // rounded, of 2 tiles for 3 CUs at most, so that all splits have 4/3 num_cu
  // tiles at most; tiles of 256 rows only where the plan may split those.
  const int64_t most = (num_cu + hk / 2) / hk, by_keys = (held + 255) / 256;
  const int64_t splits = most < by_keys ? most : by_keys;
  if (rows > few && splits > 1) {
    const int64_t by_rows = splits * a.T * a.q_heads;
    const int64_t by_tiles = (num_cu + num_cu / 3) * (int64_t)((D == 64 || D == 128) && rows >= 192 && held >= 3600 ? 256 : 128);
    tile = by_rows < by_tiles ? by_rows : by_tiles;
  }
  return (size_t)(stream > tile ? stream : tile) * (D + 2) * sizeof(float);
}

struct LogitsArgs {
  const void* x;              // [rows][x_stride]
  void* out;                  // [rows][o_stride]
  int64_t rows, vocab, x_stride, o_stride;
  const int32_t* tokens;      // [rows][tokens_stride] or null
  int64_t tokens_stride;
  const int32_t* lens;        // [rows]
  const int32_t* prompt_lens; // [rows] or null: 0
  const float* repetition;    // [rows] or null: 1
  const float* frequency;     // [rows] or null: 0
  const float* presence;      // [rows] or null: 0
  const int32_t* bias_offsets;  // [rows + 1] or null
  const int32_t* bias_ids;
  const float* bias_values;
  int64_t bias_count;         // entries of bias_ids and bias_values
  const uint32_t* mask;       // [rows][mask_stride] words or null
  int64_t mask_stride;
};
hipError_t launch_logits(const LogitsArgs& a, int in_dtype, int out_dtype, int num_cu, hipStream_t st);

constexpr int SAMPLE_BINS = 256;                  // of a slice's histogram
constexpr int SAMPLE_FIRST = 128;                 // tokens that a slice writes down
constexpr int SAMPLE_PART = 2048;                 // tokens that a part of a row hands over
constexpr int SAMPLE_MOST_PARTS = 16;
struct SliceTop {
  float top;                  // its largest logit
  uint16_t bins;              // bins whose tokens are all among those written down
  uint16_t n;                 // how many these are
};
struct SampleArgs {
  const void* x;              // [rows][x_stride]
  int64_t rows, vocab, x_stride;
  const float* u;             // [rows]
  const float* temperature;   // [rows] or null: 1
  const int32_t* top_k;       // [rows] or null: all
  const float* top_p;         // [rows] or null: 1
  const float* min_p;         // [rows] or null: 0
  int32_t* out;               // [rows]
  float* logprobs;            // [rows] or null
  unsigned long long* hist;   // [rows][slices][SAMPLE_BINS]
  uint2* first;               // [rows][slices][SAMPLE_FIRST]: logits and ids
  SliceTop* slice_tops;       // [rows][slices]
  unsigned long long* parts;  // [rows][row_parts][SAMPLE_PART]: tokens that a part of a row holds
  uint32_t* part_n;           // [rows][row_parts]: how many
  uint32_t* arrived;          // [rows]: parts that are done
  int slice, slices;          // tokens of a slice, slices of a row
  int row_parts;              // workgroups that choose a row's token
};
// Tokens of a slice: few where larger ones would leave CUs idle.  (Both launches,
// slices of 4096 and of 8192: 128 rows of 131073 f32 50.0 us and 43.1; a row of
// 32064 16.0 and 16.0, of which the first launch 4.8 and 5.4.)
inline int sample_slice(int64_t rows, int64_t vocab, int num_cu) {
  return rows * ((vocab + 8191) / 8192) < 2 * (int64_t)num_cu ? 4096 : 8192;
}
// Workgroups that choose a row's token: those that would be idle, a slice's
// tokens for each at least.
inline int sample_parts(int64_t rows, int64_t vocab, int num_cu) {
  int64_t n = num_cu / (rows > 0 ? rows : 1);
  const int64_t most = (vocab + 8191) / 8192;
  n = n < most ? n : most;
  return (int)(n < 1 ? 1 : n < SAMPLE_MOST_PARTS ? n : SAMPLE_MOST_PARTS);
}
hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t st);

// ---- device helpers ----

template <class E> struct Mat;
template <> struct Mat<f16> {
  typedef f16 x8 __attribute__((ext_vector_type(8)));
  static constexpr uint32_t EXP1 = 0x04000400u;   // one exponent step in both halves of a dword
  static constexpr uint32_t INF = 0x7C00u, ONE = 0x3C00u, TWO7 = 0x5800u, TWO14 = 0x7400u;
  // Attention's weights are taken against the largest score less LIFT: up to
  // 2^LIFT, so that the rounding to f16, absolute below its normal range,
  // keeps what many small weights beside a large one hold (2^-33 of the
  // largest; of 2^-25, 2500 keys of 2^-25 each lost all of it).  Sums of
  // several weights stay finite.
  static constexpr float LIFT = 8.f;
  static constexpr float MOST = 65504.f;          // largest finite value
  static __device__ __forceinline__ floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
};
template <> struct Mat<bf16> {
  typedef bf16 x8 __attribute__((ext_vector_type(8)));
  static constexpr uint32_t EXP1 = 0x00800080u;
  static constexpr uint32_t INF = 0x7F80u, ONE = 0x3F80u, TWO7 = 0x4300u, TWO14 = 0x4680u;
  static constexpr float LIFT = 0.f;              // (f32's exponents: 2^-133)
  static constexpr float MOST = 4096.f;
  static __device__ __forceinline__ floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
};

// ---- the cache of 8 bits ----
//
// A head of a token is e4m3 codes times 2^e, e = ceil(log2(amax / 448)): a
// power of two costs a code with an exponent of its own no precision, unlike
// amax / 448 itself, and what the codes stand for is exact in E.  So that it is
// finite and exact for every code, e is held to [LO, HI] and codes at HI to 240
// (448 otherwise): the smallest code, 2^-9, at LO is 2^-23 in f16, where a
// normal value of the head keeps its three bits down to 2^-20.
template <class E> struct Held;
template <> struct Held<f16> { static constexpr int LO = 127 - 14, HI = 127 + 8; };
template <> struct Held<bf16> { static constexpr int LO = 127 - 110, HI = 127 + 120; };
constexpr float CODE_MOST = 448.f, CODE_MOST_HI = 240.f;
constexpr uint32_t CODE_NAN = 0x7F;

// a stored exponent as one that append writes: what stale memory holds is taken
// as the nearest, so that no scale is infinite
template <class E>
__device__ __forceinline__ uint32_t held_exponent(uint32_t b) {
  const uint32_t x = b < (uint32_t)Held<E>::LO ? (uint32_t)Held<E>::LO : b;
  return x < (uint32_t)Held<E>::HI ? x : (uint32_t)Held<E>::HI;
}
// the stored exponent of a largest magnitude: 448 = 1.75 * 2^8, and a fraction
// above .75 carries into the exponent
template <class E>
__device__ __forceinline__ int exponent_of(float amax) {
  const int e = (int)((__builtin_bit_cast(uint32_t, amax) + 0x1FFFFFu) >> 23) - 8;
  return e < Held<E>::LO ? Held<E>::LO : (e < Held<E>::HI ? e : Held<E>::HI);
}

// Four codes of a dword as E, times the power of two `scale`.
template <class E> __device__ __forceinline__ void codes4(uint32_t w, float scale, uint32_t& a, uint32_t& b);
template <>
__device__ __forceinline__ void codes4<f16>(uint32_t w, float scale, uint32_t& a, uint32_t& b) {
  a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false));
  b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true));
}
template <>
__device__ __forceinline__ void codes4<bf16>(uint32_t w, float scale, uint32_t& a, uint32_t& b) {
  a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
  b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true));
}
template <class E>
__device__ __forceinline__ u32x4 codes8(uint32_t lo, uint32_t hi, float scale) {
  uint32_t a, b, c, d;
  codes4<E>(lo, scale, a, b);
  codes4<E>(hi, scale, c, d);
  return (u32x4){a, b, c, d};
}

// two f32 -> two E in a dword, round to nearest even
template <class E>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef E x2 __attribute__((ext_vector_type(2)));
  const x2 v = {(E)a, (E)b};
  return __builtin_bit_cast(uint32_t, v);
}
template <class E>
__device__ __forceinline__ float lo2f(uint32_t w) { return (float)__builtin_bit_cast(E, (uint16_t)w); }
template <class E>
__device__ __forceinline__ float hi2f(uint32_t w) { return (float)__builtin_bit_cast(E, (uint16_t)(w >> 16)); }

// bits 15 and 31: whether the low and the high half are infinite or NaN
// (an exponent of all ones carries into the sign's place when one step is added)
template <class E>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + Mat<E>::EXP1) & 0x80008000u;
}

}  // namespace fcg
