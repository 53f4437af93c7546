// The split of attention's work between kernels, workgroups and parts of the
// keys, and the workspace that it takes.  Host code only: the device's lengths
// are not known here, so it goes by T, max_q and the table's width.
#include "attend.h"

namespace fcg {
namespace {

// splits of `keys` keys, at least `least` (a multiple of `unit`) each, for
// about `want` of them; *per is what each takes
int split_plan(int64_t keys, int64_t want, int least, int unit, int* per) {
  const int64_t most = (keys + least - 1) / least;
  int64_t n = want < most ? want : most;
  if (n < 1) n = 1;
  int64_t p = ((keys + n - 1) / n + unit - 1) / unit * unit;
  if (p < unit) p = unit;
  *per = (int)p;
  const int64_t splits = (keys + p - 1) / p;
  return splits < 1 ? 1 : (int)splits;
}

}  // namespace

AttendPlan attend_plan(const AttendArgs& a, int num_cu) {
  AttendPlan p = {};
  const int D = a.kv.head_dim, hk = a.kv.kv_heads;
  const int64_t rows = (int64_t)a.max_q * a.group;
  const int64_t held = (int64_t)a.table_w << a.kv.page_shift;
  const int most = at_stream_rows(D);
  p.stream_rows = (int)(rows < most ? rows : most);
  // keys from the first that a row of a tile of n rows sees to the last
  auto span = [&](int64_t n, int align) {
    const int64_t seen = (int64_t)a.window + (n + a.group - 1) / a.group + align;
    return a.window > 0 && seen < held ? seen : held;
  };
  // Shares: what the CUs hold at once, but no more than there are steps.  A
  // step takes a workgroup about 1 us and joining pieces 5, so that sequences
  // of up to 4 steps are not split: a share is one of them.
  const int64_t steps = (span(p.stream_rows, AT_TILE) + at_step(D) - 1) / at_step(D) * a.seqs;
  int64_t shares = num_cu / hk;
  shares = shares < steps ? shares : steps;
  p.splits = (int)(shares < 1 ? 1 : shares);
  p.whole = span(p.stream_rows, AT_TILE) <= 4 * at_step(D);
  if (p.whole) p.splits = a.seqs;
  if (rows > most) {
    // All sequences are the tile kernel's where each has max_q rows (if cu_q
    // says so too), and where so few keys are seen that a tile of few rows ends
    // as soon as the others: one launch less (7 short sequences beside chunks,
    // 2047 keys: 13 us).
    if (a.T >= a.max_q * (int64_t)a.seqs || span(128, 64) <= 4096) p.stream_rows = 0;
    // Tiles of 256 rows take half the LDS traffic of two of 128, but fill
    // fewer CUs: where there is one for every CU, or where the keys are long
    // enough to be split (128 rows and 256, us: 64 tokens over 30000 keys, 4
    // query heads for each of 8: 69 and 61; twice 2048 over 4096, one query
    // head: 99 and 91; 2000 over 2000: 67 and 67; 600 over 600: 24 and 26).
    // Not of 96 dimensions, whose pieces cannot be dealt to 8 waves, nor of
    // 256, which take the registers of two waves.
    const int64_t all = a.T * a.group;
    const bool wide = all / 256 * hk >= num_cu || (rows >= 192 && span(256, 64) >= 3600);
    p.tile_rows = (D == 64 || D == 128) && wide ? 256 : 128;
    const int64_t tiles = ((all + p.tile_rows - 1) / p.tile_rows) * hk;
    // Splits for a workgroup per CU (two: chunks beside single tokens with a
    // window 47 us instead of 41, 8 sequences of up to 1000 keys 29 instead of
    // 25, 30000 keys 68 instead of 69), of 768 keys or more: joining takes 5 to
    // 10 us, a tile of 64 keys 1.5 (600 over 600: 24 us, in two splits 28);
    // of 256 where those would leave half of the CUs idle (twice 11 tokens
    // over 5645 keys of 256 dimensions: 49 us and 36).
    // The grid holds them all, those without rows among them.
    const int64_t room = (kMaxWorkgroups - 1) / (tile_count(a, p.tile_rows) * hk);
    int64_t want = (num_cu + tiles / 2) / tiles;
    if (want > room) want = room;
    const int64_t few = tiles * ((span(p.tile_rows, 64) + 767) / 768) < num_cu / 2;
    p.tile_splits = split_plan(span(p.tile_rows, 64), want, few ? 256 : 768, 64, &p.tile_per);
  }
  return p;
}

// rows of partial sums in the workspace: the streaming kernel's pieces, or the
// splits of the tile kernel, which is done with them before the other starts
size_t attend_part_rows(const AttendArgs& a, const AttendPlan& p) {
  const size_t s = p.whole ? 0 : (size_t)p.splits * a.kv.kv_heads * 2 * p.stream_rows;
  const size_t t = p.tile_rows && p.tile_splits > 1 ? (size_t)p.tile_splits * a.T * a.q_heads : 0;
  return s > t ? s : t;
}

size_t attend_workspace_bytes(const AttendArgs& a, const AttendPlan& p) {
  return attend_part_rows(a, p) * (a.kv.head_dim + 2) * sizeof(float);
}

}  // namespace fcg
