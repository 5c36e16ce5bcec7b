// efla_scan.cuh - the selective state space scan with a diagonal state of N
// values a channel, its backward pass and its one-token step.
//
//   D_t = softplus(dt_t + dt_bias)   (or dt_t + dt_bias)
//   h_t = exp(D_t A) h_{t-1} + D_t x_t B_t          per channel and state index
//   y_t = (<C_t, h_t> + D x_t) silu(z_t)
//   backward, g_t = dy_t silu(z_t), p_t the adjoint of h_t from t on:
//     p_t = C_t g_t + exp(D_{t+1} A) p_{t+1}
//     dB_t = sum_c p_t D_t x_t,  dC_t = sum_c g_t h_t,  dx_t = D_t <p_t, B_t> + D g_t
//     dD_t = <p_t exp(D_t A) h_{t-1}, A> + x_t <p_t, B_t>,  ddt_t = dD_t softplus'
//     dA = sum_t D_t p_t exp(D_t A) h_{t-1},  dD = sum g x,  dz = dy (<C, h> + D x) silu'(z)
//
// All of it is fp32 on the CUDA cores: nothing here is a product of
// matrices, because every (token, channel, index) has a decay of its own.
// That exponential bounds the forward pass: 16 a clock and SM.
//
// A block of 128 threads takes CT channels of one sequence; LN lanes share a
// channel, NS state values each, in registers.  The sequence goes by in
// tiles of TC tokens.  While a tile is worked on, the next one's rows are on
// their way into registers.  Each (token, channel) is prepared once, by the
// thread that loaded it (softplus, D x, gates), and passed to the lanes of
// its channel through shared memory, as are B and C in fp32.  Sums over the
// state index are taken for TB tokens at once: at each halving step a lane
// sends the half of its values that its partner keeps, so TB sums over TB
// lanes cost TB - 1 shuffles.
//
// Few channels leave SMs idle, so the sequence can be cut into segments that
// run side by side: one pass finds each segment's final state from zero and
// its sum of D (the decay over a segment is exp(A sum D)), and the pass that
// writes outputs starts each segment from the states so composed.  The extra
// pass repeats the exponentials, so it is taken only where it fills SMs that
// would idle.
#pragma once
#include "efla_vec.cuh"

namespace efla {
namespace scan {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.44269504088896340736f;

struct Args {
    const void *x, *dt, *z, *Bm, *Cm;
    long long ldx, lddt, ldz, ldb, ldc;  // elements from one token to the next
    const float *A, *D, *dt_bias, *h0;
    const int *lengths;
    void *y;
    float *h_L;
    int softplus, vec;  // vec: every row can be read and written in whole vectors
    int B, L, C, G, N;
    int tpg;            // channel tiles of a group
    int nseg, seg;      // segments, and tokens of one (a multiple of the tile)
    float *seg_h;       // [nseg][B][C][N]: final states from zero (the first: from h0)
    float *seg_d;       // [nseg][B][C]: sums of D
    float *seg_0;       // [B][C][N]: copy of h0, so that h_L may be h0
    // backward
    const void *dy;
    const float *dh_L;
    float *seg_p;       // [nseg][B][C][N]: adjoints that leave a segment at its start, from zero
    float *ckpt;        // per block: states at every kSub-th token
    float *part_bc;     // [G tpg tiles: tile within group][B][L][G][2][N]
    float *part;        // [B * nseg][C][N + 2]: dA, dD, ddt_bias
    void *dx, *ddt, *dz;
    float *dh0;
};

template <int N_, int NS_> struct Shape {
    static constexpr int N = N_, NS = NS_;
    static constexpr int LN = N / NS;                  // lanes of a channel
    static constexpr int LC = 32 / LN;                 // channels of a warp
    static constexpr int CT = kThreads / LN;           // channels of a block
    static constexpr int TC = CT > 32 ? 16 : 32;       // tokens of a tile
    static constexpr int EPT = TC * CT / kThreads;     // neighbouring channels of one token that a thread prepares
    static constexpr int VPR = CT / EPT;               // threads a token's row takes
    static constexpr int BPT = TC * N / kThreads;      // values of B (and of C) that a thread loads
    static constexpr int TB = LN < 8 ? LN : 8;         // tokens whose sums are taken together
    static constexpr int PAD = CT % 32 == 0 ? 8 : CT / 4;  // sums of TB tokens go to different banks
};

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// softplus(v) = max(v, 0) + log1p(e^-|v|), log1p(e) = 2 atanh(e / (2 + e)) by
// its series: the argument is at most 1/3, so eight terms leave less than
// 2^-29 of the result.
__device__ __forceinline__ float softplus_f32(float v) {
    const float e = __expf(-fabsf(v));
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaxf(v, 0.f) + 2.f * s * p;
}

// Sums v[0..V) over the 2^k lanes that differ in the bits of [STEP, LIM).
// At each step a lane keeps one half of the values and sends the other, so
// that afterwards v[0..max(1, V LIM^-1..)) hold the sums of the values whose
// index starts with the lane's bits; once one value is left, steps add it.
template <int V, int STEP, int LIM> __device__ __forceinline__ void halve(float *v, int lane) {
    if constexpr (STEP < LIM) {
        if constexpr (V > 1) {
            const bool up = lane & STEP;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float give = up ? v[i] : v[i + V / 2], keep = up ? v[i + V / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, STEP);
            }
            halve<V / 2, STEP * 2, LIM>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], STEP);
            halve<1, STEP * 2, LIM>(v, lane);
        }
    }
}
// Index of the first value that halve<V, STEP, LIM> leaves in a lane.
template <int V, int STEP, int LIM> __device__ __forceinline__ int halved_index(int lane) {
    if constexpr (STEP < LIM && V > 1)
        return ((lane & STEP) ? V / 2 : 0) + halved_index<V / 2, STEP * 2, LIM>(lane);
    else
        return 0;
}

__device__ __forceinline__ int length_of(const Args &a, int b) {
    if (!a.lengths) return a.L;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// Where a block works.
struct Where {
    int b, g, seg;       // sequence, group, segment
    int c0, nc;          // first channel, channels
    int tile;            // channel tile within the group
    int t0, t1, len;     // the segment's tokens, the sequence's length
    __device__ __forceinline__ Where(const Args &a, int CT) {
        const int tiles = a.tpg * a.G;
        const int ct = blockIdx.x % tiles, r = blockIdx.x / tiles;
        b = r % a.B;
        seg = r / a.B;
        g = ct / a.tpg;
        tile = ct % a.tpg;
        const int cg = a.C / a.G;
        c0 = g * cg + tile * CT;
        nc = min(CT, cg - tile * CT);
        t0 = seg * a.seg;
        t1 = min(a.L, t0 + a.seg);
        len = length_of(a, b);
    }
};

// EPT neighbouring channels of one token; zeros where the token or channel is none.
template <typename T, int EPT>
__device__ __forceinline__ Raw<T, EPT> load_row(const void *base, long long ld, long long row, int c, int n, bool on,
                                                bool vec) {
    if (!on || n <= 0) return zero_raw<T, EPT>();
    const T *p = static_cast<const T *>(base) + row * ld + c;
    return vec ? load_raw<T, EPT>(p) : load_raw_any<T, EPT>(p, n);
}

// BPT values of a token's B or C of one group, as they lie in memory.
template <typename T, typename S>
__device__ __forceinline__ Raw<T, S::BPT> load_bc(const void *base, long long ld, long long row, int off, bool on,
                                                  bool vec) {
    if (!on) return zero_raw<T, S::BPT>();
    const T *p = static_cast<const T *>(base) + row * ld + off;
    return vec ? load_raw<T, S::BPT>(p) : load_raw_any<T, S::BPT>(p, S::BPT);
}

// The composed state before segment `seg`, for one lane's values.
template <typename S>
__device__ __forceinline__ void start_state(const Args &a, const Where &w, int c, int n0, const float (&A2)[S::NS],
                                            float (&h)[S::NS]) {
    const long long bc = (long long)w.b * a.C + c, stride = (long long)a.B * a.C;
#pragma unroll
    for (int j = 0; j < S::NS; ++j) h[j] = 0.f;
    const float *h0 = a.nseg > 1 ? a.seg_0 : a.h0;
    if (w.seg == 0) {
        if (a.h0)
#pragma unroll
            for (int j = 0; j < S::NS; ++j) h[j] = h0[bc * S::N + n0 + j];
        return;
    }
    for (int s = 0; s < w.seg; ++s) {
        const float d = a.seg_d[s * stride + bc];
#pragma unroll
        for (int j = 0; j < S::NS; ++j) h[j] = fmaf(ex2(d * A2[j]), h[j], a.seg_h[(s * stride + bc) * S::N + n0 + j]);
    }
}

// ---------------------------------------------------------------- one segment's own maps
// REV = false: the final state from zero (the first segment: from h0) and the
// sum of D.  REV = true: the adjoint that leaves the segment at its start
// when none enters at its end (u_t = C_t g_t, p <- exp(D_t A) (p + u_t)).
template <typename T, typename S, bool REV>
__global__ void __launch_bounds__(kThreads) segment_kernel(Args a) {
    __shared__ float2 sd[S::TC][S::CT + S::PAD];  // D, D x (or g)
    __shared__ __align__(16) float sb[S::TC][S::N];
    const Where w(a, S::CT);
    const int tid = threadIdx.x, lane = tid & 31, ln = lane % S::LN, cl = (tid >> 5) * S::LC + lane / S::LN;
    const int c = w.c0 + cl, n0 = ln * S::NS;
    const bool on = cl < w.nc;
    float A2[S::NS], h[S::NS], sum = 0.f;
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
        A2[j] = on ? a.A[(long long)c * S::N + n0 + j] * kLog2e : 0.f;
        h[j] = 0.f;
    }
    const long long bc = (long long)w.b * a.C + c;
    if (!REV && w.seg == 0 && a.h0 && on)
#pragma unroll
        for (int j = 0; j < S::NS; ++j) {
            h[j] = a.h0[bc * S::N + n0 + j];
            a.seg_0[bc * S::N + n0 + j] = h[j];
        }
    const int end = min(w.t1, w.len);
    const int pt = tid / S::VPR, pc = (tid % S::VPR) * S::EPT;  // this thread's token and channels of a tile
    const int bt = tid * S::BPT / S::N, bn = tid * S::BPT % S::N;
    const int tiles = end > w.t0 ? (end - w.t0 + S::TC - 1) / S::TC : 0;
    float bias[S::EPT];
#pragma unroll
    for (int i = 0; i < S::EPT; ++i) bias[i] = a.dt_bias && pc + i < w.nc ? a.dt_bias[w.c0 + pc + i] : 0.f;

    Raw<T, S::EPT> rx, rd, rz;
    Raw<T, S::BPT> rb;
    const auto load = [&](int k) {
        const int t = w.t0 + k * S::TC;
        const long long row = (long long)w.b * a.L + t + pt, rowb = (long long)w.b * a.L + t + bt;
        const bool in = t + pt < end;
        rx = load_row<T, S::EPT>(REV ? a.dy : a.x, REV ? (long long)a.C : a.ldx, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rd = load_row<T, S::EPT>(a.dt, a.lddt, row, w.c0 + pc, w.nc - pc, in, a.vec);
        if (REV && a.z) rz = load_row<T, S::EPT>(a.z, a.ldz, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rb = load_bc<T, S>(REV ? a.Cm : a.Bm, REV ? a.ldc : a.ldb, rowb, w.g * S::N + bn, t + bt < end, a.vec);
    };
    if (tiles) load(REV ? tiles - 1 : 0);
    for (int i = 0; i < tiles; ++i) {
        const int k = REV ? tiles - 1 - i : i;
        const bool in = w.t0 + k * S::TC + pt < end;
#pragma unroll
        for (int e = 0; e < S::EPT; ++e) {
            const float v = to_f32(rd.e[e]) + bias[e];
            const float d = in ? (a.softplus ? softplus_f32(v) : v) : 0.f;
            const float u = to_f32(rx.e[e]);
            sd[pt][pc + e] = make_float2(d, REV ? (a.z ? u * silu_f32(to_f32(rz.e[e])) : u) : d * u);
        }
#pragma unroll
        for (int e = 0; e < S::BPT; ++e) sb[bt][bn + e] = to_f32(rb.e[e]);
        __syncthreads();
        if (i + 1 < tiles) load(REV ? k - 1 : k + 1);
#pragma unroll 8
        for (int s = 0; s < S::TC; ++s) {
            const int t = REV ? S::TC - 1 - s : s;
            const float2 d = sd[t][cl];
            sum += d.x;
#pragma unroll
            for (int j = 0; j < S::NS; ++j) {
                const float e = ex2(d.x * A2[j]), u = d.y * sb[t][n0 + j];
                h[j] = REV ? e * (h[j] + u) : fmaf(e, h[j], u);
            }
        }
        __syncthreads();
    }
    if (!on) return;
    const long long at = (long long)w.seg * a.B * a.C + bc;
    float *out = (REV ? a.seg_p : a.seg_h) + at * S::N + n0;
#pragma unroll
    for (int j = 0; j < S::NS; ++j) out[j] = h[j];
    if (!REV && ln == 0) a.seg_d[at] = sum;
}

// ---------------------------------------------------------------- forward
template <typename T, typename S> __global__ void __launch_bounds__(kThreads) scan_fwd_kernel(Args a) {
    __shared__ float2 sd[S::TC][S::CT + S::PAD];  // D, D x
    __shared__ float sy[S::TC][S::CT + S::PAD];   // <C, h>
    __shared__ __align__(16) float sb[S::TC][S::N], sc[S::TC][S::N];
    const Where w(a, S::CT);
    const int tid = threadIdx.x, lane = tid & 31, ln = lane % S::LN, cl = (tid >> 5) * S::LC + lane / S::LN;
    const int c = w.c0 + cl, n0 = ln * S::NS;
    const bool on = cl < w.nc;
    float A2[S::NS], h[S::NS];
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
        A2[j] = on ? a.A[(long long)c * S::N + n0 + j] * kLog2e : 0.f;
        h[j] = 0.f;
    }
    if (on) start_state<S>(a, w, c, n0, A2, h);
    const int end = min(w.t1, w.len);
    const int pt = tid / S::VPR, pc = (tid % S::VPR) * S::EPT;
    const int bt = tid * S::BPT / S::N, bn = tid * S::BPT % S::N;
    float bias[S::EPT], dskip[S::EPT];
#pragma unroll
    for (int i = 0; i < S::EPT; ++i) {
        bias[i] = a.dt_bias && pc + i < w.nc ? a.dt_bias[w.c0 + pc + i] : 0.f;
        dskip[i] = a.D && pc + i < w.nc ? a.D[w.c0 + pc + i] : 0.f;
    }
    Raw<T, S::EPT> rx, rd, rz;
    Raw<T, S::BPT> rb, rc;
    const auto load = [&](int t) {
        const long long row = (long long)w.b * a.L + t + pt, rowb = (long long)w.b * a.L + t + bt;
        const bool in = t + pt < end, inb = t + bt < end;
        rx = load_row<T, S::EPT>(a.x, a.ldx, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rd = load_row<T, S::EPT>(a.dt, a.lddt, row, w.c0 + pc, w.nc - pc, in, a.vec);
        if (a.z) rz = load_row<T, S::EPT>(a.z, a.ldz, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rb = load_bc<T, S>(a.Bm, a.ldb, rowb, w.g * S::N + bn, inb, a.vec);
        rc = load_bc<T, S>(a.Cm, a.ldc, rowb, w.g * S::N + bn, inb, a.vec);
    };
    load(w.t0);
    for (int t = w.t0; t < w.t1; t += S::TC) {
        const Raw<T, S::EPT> cx = rx, cz = rz;
        const bool in = t + pt < end;
#pragma unroll
        for (int e = 0; e < S::EPT; ++e) {
            const float v = to_f32(rd.e[e]) + bias[e];
            const float d = in ? (a.softplus ? softplus_f32(v) : v) : 0.f;
            sd[pt][pc + e] = make_float2(d, d * to_f32(rx.e[e]));
        }
#pragma unroll
        for (int e = 0; e < S::BPT; ++e) {
            sb[bt][bn + e] = to_f32(rb.e[e]);
            sc[bt][bn + e] = to_f32(rc.e[e]);
        }
        __syncthreads();
        if (t + S::TC < w.t1) load(t + S::TC);
        if (t < end) {
#pragma unroll 1
            for (int s = 0; s < S::TC; s += S::TB) {
                float p[S::TB];
#pragma unroll
                for (int u = 0; u < S::TB; ++u) {
                    const float2 d = sd[s + u][cl];
                    p[u] = 0.f;
#pragma unroll
                    for (int j = 0; j < S::NS; ++j) {
                        h[j] = fmaf(ex2(d.x * A2[j]), h[j], d.y * sb[s + u][n0 + j]);
                        p[u] = fmaf(h[j], sc[s + u][n0 + j], p[u]);
                    }
                }
                halve<S::TB, 1, S::LN>(p, lane);
                if (S::LN <= S::TB || ln < S::TB) sy[s + halved_index<S::TB, 1, S::LN>(lane)][cl] = p[0];
            }
        }
        __syncthreads();
        if (t + pt < w.t1 && pc < w.nc) {
            float o[S::EPT];
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) {
                o[e] = 0.f;
                if (in) {
                    o[e] = fmaf(dskip[e], to_f32(cx.e[e]), sy[pt][pc + e]);
                    if (a.z) o[e] *= silu_f32(to_f32(cz.e[e]));
                }
            }
            T *y = static_cast<T *>(a.y) + ((long long)w.b * a.L + t + pt) * a.C + w.c0 + pc;
            if (a.vec) store_raw<T, S::EPT>(y, narrow<T, S::EPT>(o));
            else store_raw_any<T, S::EPT>(y, narrow<T, S::EPT>(o), w.nc - pc);
        }
    }
    if (a.h_L && on && w.seg == a.nseg - 1)
#pragma unroll
        for (int j = 0; j < S::NS; ++j) a.h_L[((long long)w.b * a.C + c) * S::N + n0 + j] = h[j];
}

// ---------------------------------------------------------------- backward
// Two walks over the segment.  The first repeats the forward recurrence and
// leaves the state before every kSub-th token in the workspace, one float
// vector a thread, where the second finds it in reverse order.  The second
// goes backwards: for kSub tokens at a time it recomputes decays and states
// into registers from that state, and then runs the adjoint down through
// them.  Sums over channels (dB, dC) are taken by halving over a warp's
// channel lanes, then over the block's warps in shared memory, and reach the
// workspace as one partial row a block; those and the sums over sequences
// (dA, dD, ddt_bias) are added by kernels of their own in a fixed order.
constexpr int kSub = 8;

template <typename T, typename S> struct BwdSmem {
    float sdx[S::TC][S::CT + S::PAD], sdd[S::TC][S::CT + S::PAD], sg[S::TC][S::CT + S::PAD];  // D x, D, g
    float s1[S::TC][S::CT + S::PAD], s2[S::TC][S::CT + S::PAD], s3[S::TC][S::CT + S::PAD];    // <p,B>, <p e h,A>, <C,h>
    alignas(16) float sb[S::TC][S::N];
    alignas(16) float sc[S::TC][S::N];
    float bc[kThreads / 32][S::TC][2][S::N];  // a warp's sums over its channels
};

template <typename T, typename S> __global__ void __launch_bounds__(kThreads) scan_bwd_kernel(Args a) {
    extern __shared__ __align__(16) unsigned char raw_smem[];
    BwdSmem<T, S> &sm = *reinterpret_cast<BwdSmem<T, S> *>(raw_smem);
    constexpr int NS = S::NS, LN = S::LN, TC = S::TC;
    const Where w(a, S::CT);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ln = lane % LN, cl = warp * S::LC + lane / LN;
    const int c = w.c0 + cl, n0 = ln * NS;
    const bool on = cl < w.nc;
    const long long bc = (long long)w.b * a.C + c;
    float A2[NS], A1[NS], h[NS], p[NS], dA[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        A1[j] = on ? a.A[(long long)c * S::N + n0 + j] : 0.f;
        A2[j] = A1[j] * kLog2e;
        h[j] = p[j] = dA[j] = 0.f;
    }
    if (on) start_state<S>(a, w, c, n0, A2, h);
    const int end = min(w.t1, w.len);
    const int tiles = end > w.t0 ? (end - w.t0 + TC - 1) / TC : 0;
    const int pt = tid / S::VPR, pc = (tid % S::VPR) * S::EPT;
    const int bt = tid * S::BPT / S::N, bn = tid * S::BPT % S::N;
    float bias[S::EPT], dskip[S::EPT], aD[S::EPT], ab[S::EPT];
#pragma unroll
    for (int i = 0; i < S::EPT; ++i) {
        bias[i] = a.dt_bias && pc + i < w.nc ? a.dt_bias[w.c0 + pc + i] : 0.f;
        dskip[i] = a.D && pc + i < w.nc ? a.D[w.c0 + pc + i] : 0.f;
        aD[i] = ab[i] = 0.f;
    }
    float *ck = a.ckpt + ((long long)blockIdx.x * (a.seg / kSub) * kThreads + tid) * NS;
    const auto put = [&](int k, const float(&v)[NS]) {
        store_raw<float, NS>(ck + (long long)k * kThreads * NS, narrow<float, NS>(v));
    };

    Raw<T, S::EPT> rx, rd, rz, ry;
    Raw<T, S::BPT> rb, rc;
    const auto load_fwd = [&](int t) {
        const long long row = (long long)w.b * a.L + t + pt, rowb = (long long)w.b * a.L + t + bt;
        const bool in = t + pt < end;
        rx = load_row<T, S::EPT>(a.x, a.ldx, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rd = load_row<T, S::EPT>(a.dt, a.lddt, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rb = load_bc<T, S>(a.Bm, a.ldb, rowb, w.g * S::N + bn, t + bt < end, a.vec);
    };
    if (tiles) load_fwd(w.t0);
    for (int i = 0; i < tiles; ++i) {
        const int t = w.t0 + i * TC;
        const bool in = t + pt < end;
#pragma unroll
        for (int e = 0; e < S::EPT; ++e) {
            const float v = to_f32(rd.e[e]) + bias[e];
            const float d = in ? (a.softplus ? softplus_f32(v) : v) : 0.f;
            sm.sdd[pt][pc + e] = d;
            sm.sdx[pt][pc + e] = d * to_f32(rx.e[e]);
        }
#pragma unroll
        for (int e = 0; e < S::BPT; ++e) sm.sb[bt][bn + e] = to_f32(rb.e[e]);
        __syncthreads();
        if (i + 1 < tiles) load_fwd(t + TC);
#pragma unroll 1
        for (int s = 0; s < TC; s += kSub) {
            put((i * TC + s) / kSub, h);
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const float d = sm.sdd[s + u][cl], v = sm.sdx[s + u][cl];
#pragma unroll
                for (int j = 0; j < NS; ++j) h[j] = fmaf(ex2(d * A2[j]), h[j], v * sm.sb[s + u][n0 + j]);
            }
        }
        __syncthreads();
    }

    // the adjoint that enters at the segment's end
    if (on) {
        if (a.dh_L)
#pragma unroll
            for (int j = 0; j < NS; ++j) p[j] = a.dh_L[bc * S::N + n0 + j];
        const long long stride = (long long)a.B * a.C;
        for (int s = a.nseg - 1; s > w.seg; --s) {
            const float d = a.seg_d[s * stride + bc];
#pragma unroll
            for (int j = 0; j < NS; ++j) p[j] = fmaf(ex2(d * A2[j]), p[j], a.seg_p[(s * stride + bc) * S::N + n0 + j]);
        }
    }
    const auto load_bwd = [&](int t) {
        const long long row = (long long)w.b * a.L + t + pt, rowb = (long long)w.b * a.L + t + bt;
        const bool in = t + pt < end, inb = t + bt < end;
        rx = load_row<T, S::EPT>(a.x, a.ldx, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rd = load_row<T, S::EPT>(a.dt, a.lddt, row, w.c0 + pc, w.nc - pc, in, a.vec);
        ry = load_row<T, S::EPT>(a.dy, a.C, row, w.c0 + pc, w.nc - pc, in, a.vec);
        if (a.z) rz = load_row<T, S::EPT>(a.z, a.ldz, row, w.c0 + pc, w.nc - pc, in, a.vec);
        rb = load_bc<T, S>(a.Bm, a.ldb, rowb, w.g * S::N + bn, inb, a.vec);
        rc = load_bc<T, S>(a.Cm, a.ldc, rowb, w.g * S::N + bn, inb, a.vec);
    };
    const int all = (w.t1 - w.t0 + TC - 1) / TC;  // tiles with padding: their outputs are zeros
    if (tiles) load_bwd(w.t0 + (tiles - 1) * TC);
    for (int i = all - 1; i >= 0; --i) {
        const int t = w.t0 + i * TC;
        const bool in = t + pt < end;
        const Raw<T, S::EPT> cx = rx, cd = rd, cz = rz, cy = ry;
        if (i < tiles) {
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) {
                const float v = to_f32(rd.e[e]) + bias[e];
                const float d = in ? (a.softplus ? softplus_f32(v) : v) : 0.f;
                const float y = to_f32(ry.e[e]);
                sm.sdd[pt][pc + e] = d;
                sm.sdx[pt][pc + e] = d * to_f32(rx.e[e]);
                sm.sg[pt][pc + e] = a.z ? y * silu_f32(to_f32(rz.e[e])) : y;
            }
#pragma unroll
            for (int e = 0; e < S::BPT; ++e) {
                sm.sb[bt][bn + e] = to_f32(rb.e[e]);
                sm.sc[bt][bn + e] = to_f32(rc.e[e]);
            }
            __syncthreads();
            if (i > 0) load_bwd(t - TC);
#pragma unroll 1
            for (int s = TC - kSub; s >= 0; s -= kSub) {
                float hs[kSub + 1][NS], es[kSub][NS];
                widen<float, NS>(load_raw<float, NS>(ck + (long long)((i * TC + s) / kSub) * kThreads * NS), hs[0]);
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const float d = sm.sdd[s + u][cl], v = sm.sdx[s + u][cl];
#pragma unroll
                    for (int j = 0; j < NS; ++j) {
                        es[u][j] = ex2(d * A2[j]);
                        hs[u + 1][j] = fmaf(es[u][j], hs[u][j], v * sm.sb[s + u][n0 + j]);
                    }
                }
#pragma unroll
                for (int u0 = kSub - S::TB; u0 >= 0; u0 -= S::TB) {
                    float q1[S::TB], q2[S::TB], q3[S::TB];
#pragma unroll
                    for (int uu = S::TB - 1; uu >= 0; --uu) {
                        const int u = u0 + uu;
                        const float d = sm.sdd[s + u][cl], v = sm.sdx[s + u][cl], g = sm.sg[s + u][cl];
                        float m[2 * NS];  // dB, dC
                        q1[uu] = q2[uu] = q3[uu] = 0.f;
#pragma unroll
                        for (int j = 0; j < NS; ++j) {
                            const float cc = sm.sc[s + u][n0 + j];
                            p[j] = fmaf(cc, g, p[j]);
                            m[j] = p[j] * v;
                            m[NS + j] = hs[u + 1][j] * g;
                            q1[uu] = fmaf(p[j], sm.sb[s + u][n0 + j], q1[uu]);
                            q3[uu] = fmaf(hs[u + 1][j], cc, q3[uu]);
                            p[j] *= es[u][j];
                            const float q = p[j] * hs[u][j];
                            q2[uu] = fmaf(q, A1[j], q2[uu]);
                            dA[j] = fmaf(q, d, dA[j]);
                            if (!on) m[j] = m[NS + j] = 0.f;  // no channel: 0 even beside an infinite B or C
                        }
                        halve<2 * NS, LN, 32>(m, lane);
                        constexpr int left = 2 * NS > S::LC ? 2 * NS / S::LC : 1;
                        const int first = halved_index<2 * NS, LN, 32>(lane);
#pragma unroll
                        for (int k = 0; k < left; ++k)
                            sm.bc[warp][s + u][(first + k) / NS][n0 + (first + k) % NS] = m[k];
                    }
                    halve<S::TB, 1, LN>(q1, lane);
                    halve<S::TB, 1, LN>(q2, lane);
                    if (a.z) halve<S::TB, 1, LN>(q3, lane);
                    if (LN <= S::TB || ln < S::TB) {
                        const int tt = s + u0 + halved_index<S::TB, 1, LN>(lane);
                        sm.s1[tt][cl] = q1[0];
                        sm.s2[tt][cl] = q2[0];
                        sm.s3[tt][cl] = q3[0];
                    }
                }
            }
            __syncthreads();
        }
        if (t + pt < w.t1 && pc < w.nc) {
            float ox[S::EPT], od[S::EPT], oz[S::EPT];
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) {
                ox[e] = od[e] = oz[e] = 0.f;
                if (!in) continue;
                const float x = to_f32(cx.e[e]), v = to_f32(cd.e[e]) + bias[e];
                const float d = sm.sdd[pt][pc + e], g = sm.sg[pt][pc + e], q1 = sm.s1[pt][pc + e];
                ox[e] = fmaf(d, q1, dskip[e] * g);
                od[e] = fmaf(x, q1, sm.s2[pt][pc + e]);
                if (a.softplus) {
                    const float ev = __expf(-fabsf(v));
                    od[e] *= __fdividef(v >= 0.f ? 1.f : ev, 1.f + ev);
                }
                ab[e] += od[e];
                aD[e] = fmaf(g, x, aD[e]);
                if (a.z)
                    oz[e] = to_f32(cy.e[e]) * fmaf(dskip[e], x, sm.s3[pt][pc + e]) * dsilu_f32(to_f32(cz.e[e]));
            }
            const long long at = ((long long)w.b * a.L + t + pt) * a.C + w.c0 + pc;
            T *o[3] = {static_cast<T *>(a.dx) + at, static_cast<T *>(a.ddt) + at, a.z ? static_cast<T *>(a.dz) + at : nullptr};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (!o[k]) continue;
                const Raw<T, S::EPT> r = narrow<T, S::EPT>(k == 0 ? ox : k == 1 ? od : oz);
                if (a.vec) store_raw<T, S::EPT>(o[k], r);
                else store_raw_any<T, S::EPT>(o[k], r, w.nc - pc);
            }
        }
        // the block's share of dB and dC
        for (int k = tid; k < TC * 2 * S::N; k += kThreads) {
            const int tt = k / (2 * S::N), r = k % (2 * S::N);
            if (t + tt >= w.t1) break;
            float v = 0.f;
            if (t + tt < end)
#pragma unroll
                for (int u = 0; u < kThreads / 32; ++u) v += (&sm.bc[u][tt][0][0])[r];
            a.part_bc[((((long long)w.tile * a.B + w.b) * a.L + t + tt) * a.G + w.g) * (2 * S::N) + r] = v;
        }
        __syncthreads();
    }

    float *part = a.part + (long long)(w.seg * a.B + w.b) * a.C * (S::N + 2);
    if (on) {
        if (w.seg == 0 && a.dh0)
#pragma unroll
            for (int j = 0; j < NS; ++j) a.dh0[bc * S::N + n0 + j] = p[j];
        float *pa = part + (long long)c * S::N + n0;
#pragma unroll
        for (int j = 0; j < NS; ++j) pa[j] = dA[j];
    }
    // dD and ddt_bias: over the tokens that each thread prepared
    float *red = &sm.s1[0][0], *red2 = &sm.s2[0][0];
#pragma unroll
    for (int e = 0; e < S::EPT; ++e) {
        red[pt * (S::CT + S::PAD) + pc + e] = aD[e];
        red2[pt * (S::CT + S::PAD) + pc + e] = ab[e];
    }
    __syncthreads();
    for (int k = tid; k < S::CT; k += kThreads)
        if (k < w.nc) {
            float u = 0.f, v = 0.f;
            for (int tt = 0; tt < TC; ++tt) {
                u += sm.s1[tt][k];
                v += sm.s2[tt][k];
            }
            part[(long long)a.C * S::N + w.c0 + k] = u;
            part[(long long)a.C * (S::N + 1) + w.c0 + k] = v;
        }
}

// dB and dC from the blocks' shares: part[tile][rows][G][2][N] over the tiles of a group.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(const float *__restrict__ part, T *__restrict__ dB,
                                                      T *__restrict__ dC, long long rows_g, int N, int tpg) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4, n = rows_g * 2 * N;  // N is a multiple of 4
    if (i >= n) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < tpg; ++k) {
        const float4 v = *reinterpret_cast<const float4 *>(part + k * n + i);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const long long row = i / (2 * N);
    const int r = (int)(i - row * 2 * N);
    store4((r < N ? dB : dC) + row * N + (r < N ? r : r - N), s);
}

// ---------------------------------------------------------------- one token
// Four state values a thread, the state read and written once.  HBM bound
// (8 N bytes a channel); a thread takes ROWS sequences of the same channel,
// so that A is loaded once for them and several states are in flight.
template <typename T, int N, int ROWS>
__global__ void __launch_bounds__(128) scan_step_kernel(Args a) {
    constexpr int LN = N / 4;
    const int i = blockIdx.x * 128 + threadIdx.x, c = i / LN, n0 = (i % LN) * 4;
    const bool on = c < a.C;
    const int b0 = blockIdx.y * ROWS;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f), h[ROWS];
    float bias = 0.f, dskip = 0.f, xv[ROWS], dv[ROWS], zv[ROWS];
    float4 bv[ROWS], cv[ROWS];
    const int g = on ? c / (a.C / a.G) : 0;
    const auto four = [&](const void *base, long long ld, int b) {
        const T *p = static_cast<const T *>(base) + b * ld + g * N + n0;
        return a.vec ? load4(p) : make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
    };
    if (on) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (b0 + r < a.B) {
                const int b = b0 + r;
                h[r] = *reinterpret_cast<const float4 *>(a.h_L + ((long long)b * a.C + c) * N + n0);
                xv[r] = to_f32(static_cast<const T *>(a.x)[b * a.ldx + c]);
                dv[r] = to_f32(static_cast<const T *>(a.dt)[b * a.lddt + c]);
                zv[r] = a.z ? to_f32(static_cast<const T *>(a.z)[b * a.ldz + c]) : 0.f;
                bv[r] = four(a.Bm, a.ldb, b);
                cv[r] = four(a.Cm, a.ldc, b);
            }
        A = *reinterpret_cast<const float4 *>(a.A + (long long)c * N + n0);
        bias = a.dt_bias ? a.dt_bias[c] : 0.f;
        dskip = a.D ? a.D[c] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int b = b0 + r;
        float p = 0.f;
        if (on && b < a.B) {
            const float d = a.softplus ? softplus_f32(dv[r] + bias) : dv[r] + bias, u = d * xv[r], e = d * kLog2e;
            float4 v;
            v.x = fmaf(ex2(e * A.x), h[r].x, u * bv[r].x);
            v.y = fmaf(ex2(e * A.y), h[r].y, u * bv[r].y);
            v.z = fmaf(ex2(e * A.z), h[r].z, u * bv[r].z);
            v.w = fmaf(ex2(e * A.w), h[r].w, u * bv[r].w);
            *reinterpret_cast<float4 *>(a.h_L + ((long long)b * a.C + c) * N + n0) = v;
            p = fmaf(v.x, cv[r].x, fmaf(v.y, cv[r].y, fmaf(v.z, cv[r].z, v.w * cv[r].w)));
        }
#pragma unroll
        for (int o = LN / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
        if (on && b < a.B && n0 == 0) {
            float y = fmaf(dskip, xv[r], p);
            if (a.z) y *= silu_f32(zv[r]);
            static_cast<T *>(a.y)[(long long)b * a.C + c] = from_f32<T>(y);
        }
    }
}

}  // namespace scan
}  // namespace efla
