#include "tree.h"
namespace dflash {
bool tree_tc_supports(const dflash_dims*) { return false; }
cudaError_t launch_tree_attn_tc(const TreeAttnParams&, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace dflash
