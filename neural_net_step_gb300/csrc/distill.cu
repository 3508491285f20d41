// Launches of the distillation kernel (distill.cuh).
#include <stdio.h>

#include <algorithm>

#include "distill.h"
#include "ops.h"

namespace mlpk {

namespace {

using namespace lg;
using namespace ds;

// How rows are cut: `cluster` blocks of `threads` threads (at least k) share a
// row, `per` columns each; a slice of at most 64 KB leaves room for three blocks on
// an SM.  Fewer threads for shorter slices, of which more fit: a block's sums and
// barriers cost each warp the same, however little of a row it has (bf16, k = 16:
// 16384 x 4000 208 us with 256 threads, 125 with 128, 90 with 64, 75 with one warp; 8192 x 14000 92 with
// 128 and 83 with 64).  More where rows are few, 512 where one slice fits.
struct Cut {
  int cluster, per, threads;
};
Cut cut_rows(int64_t rows, int64_t C, int es, int k) {
  int cs = 1;
  while (cs < 8 && ceil_div(C, cs) * es > kSliceBytes) cs *= 2;
  Cut c;
  c.cluster = cs;
  c.per = (int)round_up(ceil_div(C, cs), 16 / es);
  const int64_t bytes = (int64_t)c.per * es;
  c.threads = cs == 1 && bytes <= 8 * 1024 && k <= 32 ? 32
              : bytes <= 32 * 1024 && k <= 64         ? 64
              : bytes <= 48 * 1024 && k <= 128        ? 128
              : bytes <= 100 * 1024                   ? 256
                                                      : 512;
  while (c.threads < 256 && rows * cs * c.threads * 2 <= kSMs * 512 && bytes > c.threads * 64) c.threads *= 2;
  return c;
}

}  // namespace

int distill_plan(const DistillOp& op, LaunchRec* rec, char* err, size_t errlen) {
  if (op.B < 1 || op.B > INT32_MAX || op.C < 1 || op.C > kMaxC || op.k < 1 || op.k > kMaxK || op.k > op.C ||
      op.ldz < op.C || (op.dz && op.lddz < op.C) || op.ldtv < op.k || op.ldti < op.k) {
    snprintf(err, errlen, "distill: bad shape B=%lld C=%lld k=%lld or leading dimension", (long long)op.B,
             (long long)op.C, (long long)op.k);
    return -1;
  }
  const int es = op.dtype == DT_F32 ? 4 : 2;
  const Cut cut = cut_rows(op.B, op.C, es, (int)op.k);
  DistillParams p{};
  p.z = op.z; p.ldz = op.ldz; p.dz = op.dz; p.lddz = op.lddz;
  p.tv = op.t_values; p.ldtv = op.ldtv; p.ti = op.t_indices; p.ldti = op.ldti; p.tail = op.t_tail;
  p.labels = op.ce_weight != 0.f ? op.labels : nullptr; p.w = op.row_weights; p.loss = op.loss_rows;
  p.C = (int)op.C; p.k = (int)op.k; p.per = cut.per;
  p.T = op.temperature; p.inv_T = 1.f / op.temperature; p.c = kLog2e / op.temperature;
  p.a = op.ce_weight; p.b = op.kd_weight; p.g = op.grad_scale;
  p.err = op.err;
  const int hard = !p.labels || op.temperature == 1.f ? SAME : op.temperature == 2.f ? SQUARE : OTHER;
  rec->grid = dim3((unsigned)op.B, 1, (unsigned)cut.cluster);
  rec->block = dim3((unsigned)cut.threads);
  rec->cluster = (unsigned)cut.cluster;
  rec->smem = (unsigned)((op.k * 4 + 15) / 16 * 16 + slice_buffer(cut.per, es, cut.threads));
  rec->func = op.dtype == DT_F32 ? distill_func_f32(cut.cluster > 1, hard, cut.threads)
                                 : distill_func_bf16(cut.cluster > 1, hard, cut.threads);
  rec->name = "distill";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
