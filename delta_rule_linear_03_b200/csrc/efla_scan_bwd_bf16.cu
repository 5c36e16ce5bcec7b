// efla_scan_bwd_bf16.cu - the backward kernels of the scan for bfloat16.
#include "efla_scan_launch.cuh"

namespace efla {
namespace scan {

template <> efla_status_t launch_backward<__nv_bfloat16>(const Args &a, const Plan &p, cudaStream_t st) {
    return for_shape(a.N, p, Backward<__nv_bfloat16>{a, p, st});
}

}  // namespace scan
}  // namespace efla
