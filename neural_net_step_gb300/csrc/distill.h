// What the distillation kernel (distill.cuh) is launched with, and its instances:
// one translation unit per type of logits.
#pragma once
#include "logits.cuh"

namespace mlpk {
namespace ds {

struct DistillParams {
  const void* z; int64_t ldz;
  void* dz; int64_t lddz;           // nullable
  const float* tv; int64_t ldtv;
  const int32_t* ti; int64_t ldti;
  const float* tail;                // nullable: nothing else
  const int32_t* labels;            // nullable: a is 0
  const float* w;                   // nullable: 1
  float* loss;
  int C, k, per;
  float T, inv_T, c, a, b, g;       // c: log2(e) / T
  uint32_t* err;
};

// The hard labels' softmax next to the soft ones': of the same temperature, at any
// other (a second exponential an element), or at half of it (T = 2: the square of
// the first, at twice its relative error, a few 2^-22; 8192 x 32000 bf16, k = 32: 219 us with a second
// exponential, 190 so).
enum Hard { SAME, OTHER, SQUARE };

const void* distill_func_f32(bool cluster, int hard, int threads);
const void* distill_func_bf16(bool cluster, int hard, int threads);

}  // namespace ds
}  // namespace mlpk
