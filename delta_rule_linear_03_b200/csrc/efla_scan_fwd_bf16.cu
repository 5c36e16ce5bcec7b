// efla_scan_fwd_bf16.cu - the forward kernels of the scan for bfloat16.
#include "efla_scan_launch.cuh"

namespace efla {
namespace scan {

template <> efla_status_t launch_forward<__nv_bfloat16>(Mode mode, const Args &a, const Plan &p, cudaStream_t st) {
    return for_shape(a.N, p, Forward<__nv_bfloat16>{mode, a, p, st});
}

}  // namespace scan
}  // namespace efla
