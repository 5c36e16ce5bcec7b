// efla_scan_bwd_f32.cu - the backward kernels of the scan for float.
#include "efla_scan_launch.cuh"

namespace efla {
namespace scan {

template <> efla_status_t launch_backward<float>(const Args &a, const Plan &p, cudaStream_t st) {
    return for_shape(a.N, p, Backward<float>{a, p, st});
}

}  // namespace scan
}  // namespace efla
