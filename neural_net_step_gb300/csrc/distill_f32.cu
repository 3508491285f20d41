#include "distill.cuh"

namespace mlpk {
namespace ds {

const void* distill_func_f32(bool cluster, int hard, int threads) { return distill_func<float>(cluster, hard, threads); }

}  // namespace ds
}  // namespace mlpk
