// Launches of the top-k kernel (topk.cuh), for its own operation and for the beams'.
#include <stdio.h>

#include <algorithm>

#include "ops.h"
#include "topk.h"

namespace mlpk {

namespace {

using namespace lg;
using namespace tk;

// A beam's row of at most so many bytes is read by one block where rows leave SMs
// idle, longer ones by several, with a merge of its own (us, one block a row and several: bf16
// 1 x 4 x 32000 7.6 and 7.9, x 65536 8.8 and 9.6; fp32 1 x 4 x 50001 9.7 and 10.8, 7 x 5 x 50001 11.9 and 12.2;
// bf16 8 x 4 x 100003 12.1 and 12.6.  From about 220 KB on it turns: bf16 x 131072 1 x 4 11.0 and 10.3,
// 8 x 4 13.1 and 11.6).
constexpr int64_t kFusedRow = 256 * 1024;

// Blocks of a row and their threads.
//   A third more threads than entries at least, whose largest elements set the threshold
// (where the row has that many units: see topk.cuh), which leaves up to 1.9 k candidates so (16384 x 4000 bf16, k = 96: 142 us with 128 threads,
// 194 with 256; k = 32: 58 with 64, 201 with 32, too few).  One warp for short rows, which
// a block's barriers would hold up (16384 x 2000, k = 10: 52 us with 64 threads, 33 with
// 32; 16384 x 8000, k = 16: 73 and 65).
//   Fewer and larger blocks where the rows under way would not stay in L2 until they are
// read again (fp32 4096 x 32000, k = 64: 131 us with 1216 rows under way, 107 with 608).
//   More threads where rows are few (one row of 32000 bf16, k = 50: 5.8 us with 512).
//   A row is shared only where rows leave SMs idle and its parts are long, for what the
// blocks of a cluster tell one another takes microseconds (48 x 262144 bf16, k = 256:
// 19.7 us with two blocks a row, 24.4 with four).
struct TopkCut {
  int cluster, per, threads;
};
TopkCut topk_cut(int64_t rows, int64_t C, int es, int k, bool whole) {
  constexpr int64_t kThreads = kSMs * 1024;    // under way at a time (64 registers each)
  constexpr int64_t kKept = 96 << 20;          // bytes of L2 that rows may take
  constexpr int64_t kOneWarp = 1024;           // 16-byte units
  TopkCut c;
  c.cluster = 1;
  while (!whole && c.cluster < 8 && rows * c.cluster * 2 <= kSMs && ceil_div(C, c.cluster * 2) * es >= 64 * 1024)
    c.cluster *= 2;
  c.per = (int)round_up(ceil_div(C, c.cluster), 16 / es);
  const int64_t blocks = rows * c.cluster, units = c.per * es / 16;
  c.threads = k <= 24 && units <= kOneWarp ? 32 : k <= 48 ? 64 : k <= 96 ? 128 : k <= 192 ? 256 : 512;
  while (c.threads < 512 && std::min(blocks, kThreads / c.threads) * units * 16 > kKept) c.threads *= 2;
  while (c.threads < 512 && blocks * c.threads * 2 <= kThreads && units > c.threads * 4) c.threads *= 2;
  return c;
}

void topk_launch(int dtype, int64_t rows, const TopkParams& q, LaunchRec* rec) {
  const int es = dtype == DT_F32 ? 4 : 2, beams = q.out.beams;   // (0: rows of their own)
  const TopkCut cut = topk_cut(rows, q.C, es, q.k, beams > 0);
  TopkParams p = q;
  p.per = cut.per;
  const bool small = es == 2 && cut.per <= 65535;
  const int blocks = beams > 4 ? 8 : beams > 2 ? 4 : beams > 0 ? 2 : cut.cluster;
  const int mode = beams > 0 ? BEAMS : blocks > 1 ? SLICES : ALONE;
  rec->grid = dim3((unsigned)(beams > 0 ? rows / beams : rows), 1, (unsigned)blocks);
  rec->block = dim3((unsigned)cut.threads);
  rec->cluster = (unsigned)blocks;
  rec->smem = (unsigned)(topk_room(cut.threads) * ((small ? 4 : 8) + 4) +
                         (mode == ALONE ? 0 : 9 * 8 * p.k + (mode == BEAMS ? merge_bytes(beams, p.k) : 0)));
  rec->func = es == 4 ? topk_func_f32(mode, cut.threads) : small ? topk_func_bf16(mode, cut.threads) : topk_func_bf16_wide(mode, cut.threads);
  rec->name = mode == BEAMS ? "beam_select" : "topk";
  rec->set_args(p);
}

}  // namespace

int topk_plan(const TopkOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (op.B < 1 || op.B > INT32_MAX || op.C < 1 || op.C > kMaxC || op.k < 1 || op.k > kMaxK || op.k > op.C ||
      op.ldz < op.C || op.ldv < op.k || op.ldi < op.k) {
    snprintf(err, errlen, "topk: bad shape B=%lld C=%lld k=%lld or leading dimension", (long long)op.B,
             (long long)op.C, (long long)op.k);
    return -1;
  }
  TopkParams p{};
  p.z = op.z; p.ldz = op.ldz; p.C = (int)op.C; p.k = (int)op.k;
  p.T = op.temperature; p.c = kLog2e / op.temperature;
  p.values = op.values; p.ldv = op.ldv; p.indices = op.indices; p.ldi = op.ldi; p.lse = op.lse; p.tail = op.tail;
  topk_launch(op.dtype, op.B, p, rec);
  return 1;
}

bool beam_rows_plan(const BeamSelectOp& op, int entries, uint64_t* lists, float* stats, LaunchRec* rec) {
  TopkParams p{};
  p.z = op.z; p.ldz = op.ldz; p.C = (int)op.C; p.k = entries;
  p.T = 1.f; p.c = kLog2e;
  p.scores = op.scores; p.done = op.done;
  const int64_t rows = op.batch * op.beams;
  // the beams as a cluster's blocks, where they are few and a block is enough for a row
  const bool merge = op.beams <= 8 && (rows >= kSMs || op.C * (op.dtype == DT_F32 ? 4 : 2) <= kFusedRow);
  if (merge) {
    p.out = BeamOut{(int)op.beams, (int)op.m, entries, op.eos, op.scores_out, op.parents, op.tokens, op.done_out};
  } else {
    p.entries = lists; p.stats = reinterpret_cast<float2*>(stats);
  }
  topk_launch(op.dtype, rows, p, rec);
  if (!merge) rec->name = "beam_rows";
  return merge;
}

}  // namespace mlpk
