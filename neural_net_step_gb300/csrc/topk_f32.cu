#include "topk.cuh"

namespace mlpk {
namespace tk {

const void* topk_func_f32(int mode, int threads) { return topk_func<float, uint64_t>(mode, threads); }

}  // namespace tk
}  // namespace mlpk
