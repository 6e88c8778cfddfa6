// One head dim (FD_WINDOW_D) and cache type (FD_WINDOW_KV) of the window
// attention; built once per combination so that they compile in parallel.
#include "fd_window_kernel.cuh"

#if !defined(FD_WINDOW_D) || !defined(FD_WINDOW_KV)
#error "define FD_WINDOW_D and FD_WINDOW_KV"
#endif

namespace fd {

template cudaError_t launch_window_variant<FD_WINDOW_D, FD_WINDOW_KV>(const WindowParams &, const WindowLaunch &);

}  // namespace fd
