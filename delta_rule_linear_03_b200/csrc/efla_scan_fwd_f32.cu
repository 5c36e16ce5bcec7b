// efla_scan_fwd_f32.cu - the forward kernels of the scan for float.
#include "efla_scan_launch.cuh"

namespace efla {
namespace scan {

template <> efla_status_t launch_forward<float>(Mode mode, const Args &a, const Plan &p, cudaStream_t st) {
    return for_shape(a.N, p, Forward<float>{mode, a, p, st});
}

}  // namespace scan
}  // namespace efla
