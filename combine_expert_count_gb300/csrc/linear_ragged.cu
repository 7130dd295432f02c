// linear_ragged.cu -- products of many rows with any number of outputs.
#include "linear_tiles.cuh"

namespace moe {

cudaError_t launch_linear_ragged(const Linear &p, bool pair, const LinearPlan &plan,
                                 cudaStream_t st) {
    return launch_all<false>(p, pair, plan, st);
}

}  // namespace moe
