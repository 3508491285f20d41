#include "topk.cuh"

namespace mlpk {
namespace tk {

const void* topk_func_bf16_wide(int mode, int threads) { return topk_func<__nv_bfloat16, uint64_t>(mode, threads); }

}  // namespace tk
}  // namespace mlpk
