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

// Channels of one access to a row of activations: a thread's EPT, four of
// eight, or single ones (1), as the rows' alignment and the groups' width
// allow.  The last also where a row of Bm or Cm is not aligned for whole vectors.
template <typename T, typename S> int row_vector(const Args &a) {
    const size_t e = sizeof(T);
    for (const auto &q : {std::make_pair(a.Bm, a.ldb), std::make_pair(a.Cm, a.ldc)})
        if (!rows_in_vectors(q.first, q.second, S::BPT, e)) return 1;
    for (int v = S::EPT; v > 1; v /= 2) {
        if (v != S::EPT && v != 4) continue;
        bool fits = a.C / a.G % v == 0;
        for (const auto &q : {std::make_pair(a.x, a.ldx), std::make_pair(a.dt, a.lddt), std::make_pair(a.z, a.ldz)})
            fits = fits && rows_in_vectors(q.first, q.second, v, e);
        if (fits) return v;
    }
    return 1;
}

template <typename T> struct Forward {
    static constexpr bool kBackward = false;
    Mode mode;
    const Args &a;
    const Plan &p;
    cudaStream_t st;

    template <typename S, int V, Mode MODE> efla_status_t launch() const {
        constexpr size_t smem = sizeof(FwdSmem<S>);
        if (!ensure_smem<scan_fwd_kernel<T, S, V, MODE>>(smem)) return EFLA_ERR_CUDA;
        scan_fwd_kernel<T, S, V, MODE><<<(unsigned)(p.blocks * p.nseg), 2 * kThreads, smem, st>>>(a);
        return host::launched();
    }
    template <typename S, Mode MODE> efla_status_t pick() const {
        const int v = row_vector<T, S>(a);
        if constexpr (S::EPT == 1) return launch<S, 1, MODE>();
        else if (v == S::EPT) return launch<S, S::EPT, MODE>();
        if constexpr (S::EPT > 4)
            if (v == 4) return launch<S, 4, MODE>();
        return launch<S, 1, MODE>();
    }
    template <typename S> efla_status_t run() const {
        if (mode == FULL) return pick<S, FULL>();
        if constexpr (S::NS == 4 && S::CP == 1)  // the shape of segments
            return mode == STATE ? pick<S, STATE>() : pick<S, BACK>();
        return EFLA_ERR_UNSUPPORTED;
    }
};

template <typename T> struct Backward {
    static constexpr bool kBackward = true;
    const Args &a;
    const Plan &p;
    cudaStream_t st;

    template <typename S, int V> efla_status_t launch() const {
        constexpr size_t smem = sizeof(BwdSmem<S>);
        if (!ensure_smem<scan_bwd_kernel<T, S, V>>(smem)) return EFLA_ERR_CUDA;
        scan_bwd_kernel<T, S, V><<<(unsigned)(p.blocks * p.nseg), 2 * kThreads, smem, st>>>(a);
        return host::launched();
    }
    template <typename S> efla_status_t run() const {
        const int v = row_vector<T, S>(a);
        if constexpr (S::EPT == 1) return launch<S, 1>();
        else if (v == S::EPT) return launch<S, S::EPT>();
        if constexpr (S::EPT > 4)
            if (v == 4) return launch<S, 4>();
        return launch<S, 1>();
    }
};

}  // namespace scan
}  // namespace efla
