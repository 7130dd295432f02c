// linear_tiles.cu -- products of many rows whose outputs' rows start on 16 bytes.
#include "linear_tiles.cuh"

namespace moe {

cudaError_t launch_linear_tiles(const Linear &p, bool pair, const LinearPlan &plan,
                                cudaStream_t st) {
    return p.n % 8 == 0 ? launch_all<true>(p, pair, plan, st)
                        : launch_linear_ragged(p, pair, plan, st);
}

}  // namespace moe
