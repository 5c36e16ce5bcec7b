// efla_scan_launch.cuh - how a scan's work is cut into blocks, and the
// launches of its kernels, which are compiled by type and direction in
// efla_scan_*.cu (they are many, and take minutes in one unit).
#pragma once
#include <utility>

#include "efla_host.cuh"
#include "efla_scan.cuh"

namespace efla {
namespace scan {

struct Plan {
    int ns, cp;        // state values of a lane in each channel, channels of a lane
    int nseg, seg;     // segments, tokens of one
    int tpg;           // channel tiles of a group
    long long blocks;  // of one segment
    int sub() const { return ns * cp >= 4 ? 4 : 8; }  // tokens from one checkpoint of the backward pass to the next
};

constexpr int tile_channels(int N, int ns, int cp) { return kThreads * ns / N * cp; }

// Tiles are long where the channels of a block are few, so that their rows
// keep the preparing warps busy; the backward pass, which has many buffers,
// has short ones, so that two blocks fit an SM.
constexpr int tile_tokens(int N, int ct, bool bwd) { return bwd || ct > 32 || N == 64 ? 16 : 32; }

template <typename T> efla_status_t launch_forward(Mode mode, const Args &a, const Plan &p, cudaStream_t st);
template <typename T> efla_status_t launch_backward(const Args &a, const Plan &p, cudaStream_t st);

// F.template run<Shape>() for the plan's shape.
template <typename F> efla_status_t for_shape(int N, const Plan &p, const F &f) {
#define EFLA_CASE(N_, NS, CP)                                             \
    if constexpr (!(F::kBackward && CP == 2 && N_ < 32)) /* not planned */ \
        if (N == N_ && p.ns == NS && p.cp == CP)                          \
    return f.template run<Shape<N_, NS, CP, tile_tokens(N_, tile_channels(N_, NS, CP), F::kBackward)>>()
    EFLA_CASE(8, 2, 1);
    EFLA_CASE(8, 4, 1);
    EFLA_CASE(8, 2, 2);
    EFLA_CASE(16, 2, 1);
    EFLA_CASE(16, 4, 1);
    EFLA_CASE(16, 4, 2);
    EFLA_CASE(32, 2, 1);
    EFLA_CASE(32, 4, 1);
    EFLA_CASE(32, 4, 2);
    EFLA_CASE(64, 4, 1);
    EFLA_CASE(64, 4, 2);
#undef EFLA_CASE
    return EFLA_ERR_UNSUPPORTED;
}

// Whether rows can be read in vectors of `vec` elements.
inline bool rows_in_vectors(const void *p, long long ld, int vec, size_t e) {
    return host::aligned_to(p, std::min<size_t>(16, vec * e)) && ld % vec == 0;
}

template <typename T, typename S> bool in_vectors(const Args &a) {
    const size_t e = sizeof(T);
    bool v = a.C / a.G % S::EPT == 0;
    for (const auto &q : {std::make_pair(a.x, a.ldx), std::make_pair(a.dt, a.lddt), std::make_pair(a.z, a.ldz)})
        v = v && rows_in_vectors(q.first, q.second, S::EPT, e);
    for (const auto &q : {std::make_pair(a.Bm, a.ldb), std::make_pair(a.Cm, a.ldc)})
        v = v && rows_in_vectors(q.first, q.second, S::BPT, e);
    return v;
}

template <typename T> struct Forward {
    static constexpr bool kBackward = false;
    Mode mode;
    const Args &a;
    const Plan &p;
    cudaStream_t st;

    template <typename S, bool VEC, Mode MODE> efla_status_t launch() const {
        constexpr size_t smem = sizeof(FwdSmem<S>);
        if (!ensure_smem<scan_fwd_kernel<T, S, VEC, MODE>>(smem)) return EFLA_ERR_CUDA;
        scan_fwd_kernel<T, S, VEC, MODE><<<(unsigned)(p.blocks * p.nseg), 2 * kThreads, smem, st>>>(a);
        return host::launched();
    }
    template <typename S> efla_status_t run() const {
        const bool vec = in_vectors<T, S>(a);
        if (mode == FULL) return vec ? launch<S, true, FULL>() : launch<S, false, FULL>();
        if constexpr (S::NS == 4 && S::CP == 1) {  // the shape of segments
            if (mode == STATE) return vec ? launch<S, true, STATE>() : launch<S, false, STATE>();
            return vec ? launch<S, true, BACK>() : launch<S, false, BACK>();
        }
        return EFLA_ERR_UNSUPPORTED;
    }
};

template <typename T> struct Backward {
    static constexpr bool kBackward = true;
    const Args &a;
    const Plan &p;
    cudaStream_t st;

    template <typename S, bool VEC> efla_status_t launch() const {
        constexpr size_t smem = sizeof(BwdSmem<S>);
        if (!ensure_smem<scan_bwd_kernel<T, S, VEC>>(smem)) return EFLA_ERR_CUDA;
        scan_bwd_kernel<T, S, VEC><<<(unsigned)(p.blocks * p.nseg), 2 * kThreads, smem, st>>>(a);
        return host::launched();
    }
    template <typename S> efla_status_t run() const {
        return in_vectors<T, S>(a) ? launch<S, true>() : launch<S, false>();
    }
};

}  // namespace scan
}  // namespace efla
