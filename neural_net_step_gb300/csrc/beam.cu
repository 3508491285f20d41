// Beam search: which (beam, token) pairs go on, and the reordering of the states
// that belong to the beams.
//
// Selection.  Only the m best tokens of a beam can be among the m best pairs: the
// top-k kernel (topk.cu) finds them, and, where a batch entry's beams are the blocks of
// a cluster, merges them as well.  Otherwise (more than eight beams, or rows that are shared
// by blocks) it leaves them in the workspace with the rows' largest logits and sums of
// exponentials, and one block per batch entry merges the lists here.
//
// Reordering.  Bound by DRAM.  A thread owns a column of all beams: it reads the
// columns of the parents and then writes, so that source and destination may be
// the same memory, and rows that stay are not written there.  A parent's row is read
// from DRAM once for all its children (24 planes of 16 x 4 rows of 512 KB: 190 us, 86 % of
// DRAM's peak).
#include <stdio.h>

#include <algorithm>

#include "beam.cuh"
#include "ops.h"

namespace mlpk {

namespace {

using namespace lg;

struct BeamMergeParams {
  const uint64_t* entries; const float2* stats;   // [batch * beams][per], [batch * beams]
  const float* scores; const uint8_t* in_done;
  BeamOut out;
};

// Bound by latency: a few KB of a batch entry, the same steps as in the fused kernel
// (2 x 16 beams of 32000 bf16, m = 32: 10.9 us with the rows' kernel before it).
__global__ void __launch_bounds__(512) beam_merge_kernel(const __grid_constant__ BeamMergeParams p) {
  pdl_enter();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BeamBase base[kMaxBeams];
  const int64_t r0 = (int64_t)blockIdx.x * p.out.beams;
  if ((int)threadIdx.x < p.out.beams) {
    const int64_t r = r0 + threadIdx.x;
    const float score = p.scores[r];
    const bool done = p.in_done && p.in_done[r];
    const float2 st = beam_reads_row(score, done) ? p.stats[r] : make_float2(0.f, 0.f);
    base[threadIdx.x] = beam_base(score, done, st.x, st.y);
  }
  __syncthreads();
  merge_beams(p.out, blockIdx.x, p.entries + r0 * p.out.per, base, reinterpret_cast<uint64_t*>(smem));
}

struct ReorderParams {
  const unsigned char* src; int64_t src_pitch, src_plane;
  unsigned char* dst; int64_t dst_pitch, dst_plane;
  const int32_t* parents; int64_t ldp;
  int batch, beams_in, beams_out;
  int64_t units;                // of U bytes in a row
  int64_t chunks;               // blocks along a row
  uint32_t* err;
};

// One block: blockDim.x units of all beams of one batch entry in one plane.
template <typename U, int W>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  pdl_enter();
  __shared__ int from[W];
  const int64_t row = blockIdx.x / p.chunks, chunk = blockIdx.x - row * p.chunks;   // row: (plane, batch entry)
  const int64_t plane = row / p.batch, b = row - plane * p.batch;
  if (threadIdx.x < W) {
    int f = -1;
    if ((int)threadIdx.x < p.beams_out) {
      f = p.parents[b * p.ldp + threadIdx.x];
      if (f < 0 || f >= p.beams_in) {
        if (p.err && plane == 0 && chunk == 0) atomicOr(p.err, ERRBIT_LABEL_RANGE);
        f = -1;
      }
      if (p.dst == p.src && f == (int)threadIdx.x) f = -1;   // (stays)
    }
    from[threadIdx.x] = f;
  }
  __syncthreads();
  const unsigned char* src = p.src + plane * p.src_plane + b * p.beams_in * p.src_pitch;
  unsigned char* dst = p.dst + plane * p.dst_plane + b * p.beams_out * p.dst_pitch;
  const int64_t u = chunk * blockDim.x + threadIdx.x;
  if (u >= p.units) return;
  U v[W];
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (from[i] >= 0) v[i] = *reinterpret_cast<const U*>(src + from[i] * p.src_pitch + u * (int64_t)sizeof(U));
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (from[i] >= 0) *reinterpret_cast<U*>(dst + i * p.dst_pitch + u * (int64_t)sizeof(U)) = v[i];
}

template <typename U>
const void* reorder_func(int W) {
  if (W <= 4) return (const void*)beam_reorder_kernel<U, 4>;
  if (W <= 8) return (const void*)beam_reorder_kernel<U, 8>;
  if (W <= 16) return (const void*)beam_reorder_kernel<U, 16>;
  return (const void*)beam_reorder_kernel<U, 32>;
}

}  // namespace

size_t beam_select_workspace(int64_t batch, int64_t beams, int64_t C, int64_t m) {
  if (batch < 1 || beams < 1 || beams > kMaxBeams || C < 1 || C > kMaxC || m < 1 || m > kMaxOut || m > beams * C ||
      batch > INT32_MAX / beams)
    return 0;
  return (size_t)(batch * beams) * (8 * (size_t)std::min(m, C) + 8);
}

int beam_select_plan(const BeamSelectOp& op, LaunchRec* recs, char* err, size_t errlen) {
  if (beam_select_workspace(op.batch, op.beams, op.C, op.m) == 0 || op.ldz < op.C) {
    snprintf(err, errlen, "beam_select: bad shape batch=%lld beams=%lld C=%lld m=%lld or leading dimension",
             (long long)op.batch, (long long)op.beams, (long long)op.C, (long long)op.m);
    return -1;
  }
  const int per = (int)std::min(op.m, op.C);
  const int64_t rows = op.batch * op.beams;
  uint64_t* entries = reinterpret_cast<uint64_t*>(op.ws);
  float* stats = reinterpret_cast<float*>(entries + rows * per);
  if (beam_rows_plan(op, per, entries, stats, &recs[0])) return 1;   // (merged there)
  BeamMergeParams p{};
  p.entries = entries; p.stats = reinterpret_cast<const float2*>(stats);
  p.scores = op.scores; p.in_done = op.done;
  p.out = BeamOut{(int)op.beams, (int)op.m, per, op.eos, op.scores_out, op.parents, op.tokens, op.done_out};
  const int all = p.out.beams * merge_stride(per);
  recs[1].func = (const void*)beam_merge_kernel;
  recs[1].grid = dim3((unsigned)op.batch);
  recs[1].block = dim3(all <= 128 ? 128 : all <= 256 ? 256 : 512);
  recs[1].smem = (unsigned)merge_bytes(p.out.beams, per);
  recs[1].name = "beam_merge";
  recs[1].set_args(p);
  return 2;
}

int beam_reorder_plan(const BeamReorderOp& op, LaunchRec* rec, char* err, size_t errlen) {
  const auto bad = [&](const char* what) {
    snprintf(err, errlen, "beam_reorder: %s", what);
    return -1;
  };
  if (op.planes < 1 || op.batch < 1 || op.beams_in < 1 || op.beams_out < 1 || op.beams_in > kMaxBeams ||
      op.beams_out > kMaxBeams || op.row_bytes < 1 || op.batch > INT32_MAX)
    return bad("bad shape");
  if (op.ldp < op.beams_out || op.src_pitch < op.row_bytes || op.dst_pitch < op.row_bytes)
    return bad("pitch too small");
  if (op.src == op.dst &&
      (op.beams_in != op.beams_out || op.src_pitch != op.dst_pitch || (op.planes > 1 && op.src_plane != op.dst_plane)))
    return bad("in place, source and destination have the same layout");
  const uint64_t any = (uint64_t)(uintptr_t)op.src | (uint64_t)(uintptr_t)op.dst | (uint64_t)op.src_pitch |
                       (uint64_t)op.dst_pitch | (uint64_t)op.row_bytes |
                       (op.planes > 1 ? (uint64_t)op.src_plane | (uint64_t)op.dst_plane : 0);
  // a thread's units stay in registers: 16 bytes for up to 8 beams, 8 for up to 16, 4 beyond
  const int W = (int)op.beams_out;
  const int widest = W <= 8 ? 16 : W <= 16 ? 8 : 4;
  const int ub = any % 16 == 0 && widest == 16 ? 16 : any % 8 == 0 && widest >= 8 ? 8 : any % 4 == 0 ? 4 : any % 2 == 0 ? 2 : 1;
  ReorderParams p{};
  p.src = static_cast<const unsigned char*>(op.src); p.src_pitch = op.src_pitch; p.src_plane = op.src_plane;
  p.dst = static_cast<unsigned char*>(op.dst); p.dst_pitch = op.dst_pitch; p.dst_plane = op.dst_plane;
  p.parents = op.parents; p.ldp = op.ldp;
  p.batch = (int)op.batch; p.beams_in = (int)op.beams_in; p.beams_out = W;
  p.units = op.row_bytes / ub;
  p.err = op.err;
  const int threads = p.units >= 256 ? 256 : p.units >= 128 ? 128 : 64;
  p.chunks = ceil_div(p.units, threads);
  if (op.planes > INT32_MAX / op.batch || p.chunks > INT32_MAX / (op.planes * op.batch)) return bad("too many bytes");
  rec->grid = dim3((unsigned)(op.planes * op.batch * p.chunks));
  rec->block = dim3((unsigned)threads);
  rec->smem = 0;
  rec->func = ub == 16 ? reorder_func<uint4>(W) : ub == 8 ? reorder_func<uint2>(W) : ub == 4 ? reorder_func<uint32_t>(W)
              : ub == 2 ? reorder_func<uint16_t>(W) : reorder_func<uint8_t>(W);
  rec->name = "beam_reorder";
  rec->set_args(p);
  return 1;
}

}  // namespace mlpk
