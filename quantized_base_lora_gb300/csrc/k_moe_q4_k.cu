// The experts' products over q4_K weights.
#include "moe_rows.cuh"

namespace ovl {
namespace moe {

cudaError_t launch_products_q4_k(const MoeDev& m, cudaStream_t st) { return launch_products<OVL_Q4_K>(m, st); }

}  // namespace moe
}  // namespace ovl
