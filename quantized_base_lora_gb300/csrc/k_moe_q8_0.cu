// The experts' products over q8_0 weights.
#include "moe_rows.cuh"

namespace ovl {
namespace moe {

cudaError_t launch_products_q8_0(const MoeDev& m, cudaStream_t st) { return launch_products<OVL_Q8_0>(m, st); }

}  // namespace moe
}  // namespace ovl
