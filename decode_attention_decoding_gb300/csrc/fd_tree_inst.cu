// One head dim and loader of the tree kernel (FD_TREE_D, FD_TREE_LOAD), for
// bf16 and fp16 queries; built once per combination so that they compile in
// parallel.
#include "fd_tree_kernel.cuh"

namespace fd {

#define FD_TREE_INST(F16, KV, TMA)                                                                                \
    template cudaError_t launch_tree_variant<FD_TREE_D, F16, KV, TMA>(const TreeParams &, const CUtensorMap &,    \
                                                                      const CUtensorMap &, const TreeLaunch &);
#if FD_TREE_LOAD == 0
FD_TREE_INST(false, kKvBf16, true)
FD_TREE_INST(true, kKvF16, true)
#elif FD_TREE_LOAD == 1
FD_TREE_INST(false, kKvBf16, false)
FD_TREE_INST(true, kKvF16, false)
#elif FD_TREE_LOAD == 2
FD_TREE_INST(false, kKvE4m3, false)
FD_TREE_INST(true, kKvE4m3, false)
#else
FD_TREE_INST(false, kKvE5m2, false)
FD_TREE_INST(true, kKvE5m2, false)
#endif

}  // namespace fd
