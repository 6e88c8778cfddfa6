// One head dim of the tree kernel (FD_TREE_D) and one way of loading the cache
// (FD_TREE_LOAD), for both element types; built once per combination so that
// they compile in parallel.
#include "fd_tree_kernel.cuh"

namespace fd {

#define FD_TREE_INST(F16, KV, LOAD)                                                                               \
    template cudaError_t launch_tree_variant<FD_TREE_D, F16, KV, LOAD>(const TreeParams &, const CUtensorMap &,   \
                                                                       const CUtensorMap &, const TreeLaunch &);
#if FD_TREE_LOAD == 0
FD_TREE_INST(false, kKvBf16, kTreeTma)
FD_TREE_INST(true, kKvF16, kTreeTma)
#elif FD_TREE_LOAD == 1
FD_TREE_INST(true, kKvE4m3, kTreeConvert)
FD_TREE_INST(true, kKvE5m2, kTreeConvert)
#elif FD_TREE_LOAD == 2
FD_TREE_INST(false, kKvBf16, kTreeCopy)
FD_TREE_INST(true, kKvF16, kTreeCopy)
#else
FD_TREE_INST(true, kKvE4m3, kTreeCopy)
FD_TREE_INST(true, kKvE5m2, kTreeCopy)
#endif

}  // namespace fd
