#include "distill.cuh"

namespace mlpk {
namespace ds {

const void* distill_func_bf16(bool cluster, int hard, int threads) { return distill_func<__nv_bfloat16>(cluster, hard, threads); }

}  // namespace ds
}  // namespace mlpk
