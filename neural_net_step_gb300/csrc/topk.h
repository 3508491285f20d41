// What the top-k kernel (topk.cuh) is launched with, and its instances: one
// translation unit per type of logits and of candidates.
#pragma once
#include "beam.cuh"

namespace mlpk {
namespace tk {

using lg::BeamOut;

struct TopkParams {
  const void* z; int64_t ldz;
  int C, k, per;
  float T, c;                       // temperature, log2(e) / T
  float* values; int64_t ldv;
  int32_t* indices; int64_t ldi;
  float* lse; float* tail;          // nullable
  // beam selection instead of the outputs above: entries [B, k] and
  // {largest logit, sum of exp(z - largest)} of each row
  uint64_t* entries; float2* stats;
  const float* scores; const uint8_t* done;
  BeamOut out;                      // or the selection itself (BEAMS)
};

// What the blocks of a cluster are.
enum TopkMode { ALONE, SLICES, BEAMS };   // (no cluster), slices of a row, the beams of a batch entry

// Candidates of a slice at most, and units listed at most, shared out to the warps.
constexpr int topk_room(int threads) { return threads < 64 ? 256 : threads < 256 ? 512 : 1024; }
template <int NT> constexpr int kRoom = topk_room(NT);

const void* topk_func_f32(int mode, int threads);
const void* topk_func_bf16(int mode, int threads);        // slices of at most 65535 elements
const void* topk_func_bf16_wide(int mode, int threads);

}  // namespace tk
}  // namespace mlpk
