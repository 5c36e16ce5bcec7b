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
// A block takes CT channels of one sequence, which goes by in tiles of TC
// tokens.  Four of its warps run the recurrence: LN lanes share a channel, a
// lane has NS state values of each of CP channels in registers.  Four others
// prepare the next tile and finish the one before: softplus, gates and
// conversions of each (token, channel) are done once, by the thread that
// loads it, and passed on through shared memory, as are B and C in fp32.
//
// Shared memory is the second bound: what a lane reads a token goes through
// 128 bytes a clock and SM, broadcast or not.  A lane with one channel and four
// state values reads 10 bytes a value (D and D x, B, C), and its four warps
// take longer to read than to exponentiate; with two channels they share B
// and C, 6 bytes a value.
//
// Measured (bf16, gate, N = 16): 4 x 4096 x 2048 forward 269 us, where the 0.54
// 10^9 exponentials alone take 118 and the preparation's another 30; the special
// function units are busy 59% of the time, shared memory 64%.  Its 256 blocks
// leave 40 of the SMs with one where registers allow two.  Four warps that
// prepare for themselves took 513.  1 x 65536 x 2048, 128 blocks, 1.55 to 1.58
// ms: 45 clocks a token of one warp a scheduler, whose loads, exponentials and
// shuffles go one after another.  8 x 2048 x 1024 backward 548 us.
//
// Sums over the state index are taken for TB tokens at once: at each halving
// step a lane sends the half of its values that its partner keeps, so TB sums
// over TB lanes cost TB - 1 shuffles.
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

struct Args {
    const void *x, *dt, *z, *Bm, *Cm;
    long long ldx, lddt, ldz, ldb, ldc;  // elements from one token to the next
    const float *A, *D, *dt_bias, *h0;
    const int *lengths;
    void *y;
    float *h_L;
    int softplus, vec;  // vec: scan_step_kernel reads B and C in vectors
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
    float *ckpt;        // per block: states before every SUB-th token
    float *part_bc;     // [G tpg tiles: tile within group][B][L][G][2][N]
    float *part;        // [B * nseg][C][N + 2]: dA, dD, ddt_bias
    void *dx, *ddt, *dz;
    float *dh0;
};

template <int N_, int NS_, int CP_, int TC_> struct Shape {
    static constexpr int N = N_, NS = NS_, CP = CP_, TC = TC_;  // TC: tokens of a tile
    static constexpr int NP = NS / 2;                  // register pairs of a channel's state in a lane
    static constexpr int LN = N / NS;                  // lanes of a channel
    static constexpr int LC = 32 / LN;                 // channel groups (of CP) of a warp
    static constexpr int CT = kThreads / LN * CP;      // channels of a block
    static constexpr int EPT = TC * CT / kThreads;     // neighbouring channels of one token that a thread prepares
    static constexpr int VPR = CT / EPT;               // threads a token's row takes
    static constexpr int BPT = TC * N / kThreads;      // values of B (and of C) that a thread loads
    static constexpr int TB = LN < 8 ? LN : 8;         // tokens whose sums are taken together
    static constexpr int CS = CT + (CT % 32 == 0 ? 8 : CT / 4);  // a row of sums: those of TB tokens in different banks

    // Place of channel c of token t in the rows of (D, D x): a thread writes
    // EPT neighbours, two at a time, so neighbouring threads' pairs are put
    // into different banks.
    __device__ static __forceinline__ int place(int c, int t) {
        const int p = c >> 1;
        return ((p ^ (p >> 3 & 7) ^ ((t & 1) * (EPT / 4))) << 1) | (c & 1);
    }
};

// exp(D A) as 2^(D A2), A2 = A log2 e.  The approximate 2^v is on average too
// small for v from -1 to 0, by 0.6 to 2.6 10^-8 of itself (measured on this GPU
// over ranges of v), and a state of a thousand tokens' memory multiplies that by a
// thousand.  Adding 2.0 10^-8 to the argument, which costs nothing beside its
// product, leaves -1.2 to 0.9 10^-8; a step of 0 still gives exactly 1.
constexpr float kCentre = 2.0e-8f;
__device__ __forceinline__ f32x2 decay_2(f32x2 d, f32x2 A2) { return ex2_2(fma2(d, A2, twice(kCentre))); }

// softplus(v) = max(v, 0) + log1p(e), e = e^-|v|, by log1p(e) = 2 atanh(s),
// s = e / (2 + e) <= 1/3, whose series s + s^3/3 + ... + s^13/13 leaves less
// than 2^-26 of it.  A step's error goes into every decay of its token, so e
// and s are taken to the last bits: what the argument's product with log2 e
// and the rounding of log2 e lose is put back to first order, and the
// quotient has one Newton step.  Two values at once.
__device__ __forceinline__ f32x2 softplus_2(f32x2 v2) {
    const float2 v = unpack2(v2);
    const f32x2 a = pack2(fminf(fabsf(v.x), 126.f), fminf(fabsf(v.y), 126.f));  // e is 0 from there on
    const f32x2 t = mul2(a, twice(-kLog2e));
    const f32x2 lo = fma2(a, twice(-1.925963e-8f), fma2(a, twice(-kLog2e), mul2(a, twice(kLog2e))));
    f32x2 e = ex2_2(t);
    e = fma2(mul2(e, lo), twice(0.6931472f), e);
    const f32x2 w = fma2(e, twice(-1.f), twice(-2.f)), r = rcp_2(w);  // -(2 + e)
    f32x2 s = mul2(mul2(e, twice(-1.f)), r);
    s = fma2(fma2(s, w, e), mul2(r, twice(-1.f)), s);
    const f32x2 q = mul2(s, s);
    f32x2 p = fma2(twice(1.f / 13.f), q, twice(1.f / 11.f));
    p = fma2(p, q, twice(1.f / 9.f));
    p = fma2(p, q, twice(1.f / 7.f));
    p = fma2(p, q, twice(1.f / 5.f));
    p = fma2(p, q, twice(1.f / 3.f));
    const f32x2 s2 = add2(s, s);
    float2 top;  // max(v, 0), a NaN stays one
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top.x) : "f"(v.x));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(top.y) : "f"(v.y));
    return add2(pack2(top.x, top.y), fma2(mul2(p, q), s2, s2));
}
__device__ __forceinline__ float softplus_f32(float v) { return unpack2(softplus_2(twice(v))).x; }
template <int N> __device__ __forceinline__ void softplus_all(float (&v)[N]) {
    if constexpr (N == 1) {
        v[0] = softplus_f32(v[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 t = unpack2(softplus_2(pack2(v[i], v[i + 1])));
            v[i] = t.x;
            v[i + 1] = t.y;
        }
    }
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

// EPT neighbouring channels, from channel pc on, of a row of nc; what lies past
// the row's end repeats a channel of it.  V: channels of one access, for which
// rows are aligned and nc is a multiple (1: any row).  Rows are read whether
// or not their token counts: a load without a condition can be issued a tile
// ahead.
template <typename T, int EPT, int V>
__device__ __forceinline__ Raw<T, EPT> load_row(const T *row, int pc, int nc) {
    Raw<T, EPT> r;
#pragma unroll
    for (int i = 0; i < EPT; i += V) {
        const Raw<T, V> q = load_raw<T, V>(row + (pc + i < nc ? pc + i : 0));
#pragma unroll
        for (int j = 0; j < V; ++j) r.e[i + j] = q.e[j];
    }
    return r;
}
template <typename T, int EPT, int V>
__device__ __forceinline__ void store_row(T *at, const float (&o)[EPT], int pc, int nc) {
#pragma unroll
    for (int i = 0; i < EPT; i += V) {
        float q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = o[i + j];
        if (pc + i < nc) store_raw<T, V>(at + i, narrow<T, V>(q));
    }
}
template <typename T, int BPT, bool VEC> __device__ __forceinline__ Raw<T, BPT> load_bc(const T *p) {
    if constexpr (VEC) {
        return load_raw<T, BPT>(p);
    } else {
        Raw<T, BPT> r;
#pragma unroll
        for (int i = 0; i < BPT; ++i) r.e[i] = p[i];
        return r;
    }
}

// A lane's state values as register pairs, from and to shared or global memory.
template <int NP> __device__ __forceinline__ void load_pairs(const float *p, f32x2 (&v)[NP]) {
    if constexpr (NP == 2) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(p);
        v[0] = u.x;
        v[1] = u.y;
    } else {
        v[0] = *reinterpret_cast<const f32x2 *>(p);
    }
}
template <int NP> __device__ __forceinline__ void store_pairs(float *p, const f32x2 (&v)[NP]) {
    if constexpr (NP == 2) *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(v[0], v[1]);
    else *reinterpret_cast<f32x2 *>(p) = v[0];
}

// Register j of a lane holds state n0 + (j ^ x); x is 0 but in the backward pass.
template <typename S> __device__ __forceinline__ void gather(const float *p, int x, f32x2 (&v)[S::NP]) {
#pragma unroll
    for (int j = 0; j < S::NP; ++j) v[j] = pack2(p[(2 * j) ^ x], p[(2 * j + 1) ^ x]);
}
template <typename S> __device__ __forceinline__ void scatter(float *p, int x, const f32x2 (&v)[S::NP]) {
#pragma unroll
    for (int j = 0; j < S::NP; ++j) {
        const float2 t = unpack2(v[j]);
        p[(2 * j) ^ x] = t.x;
        p[(2 * j + 1) ^ x] = t.y;
    }
}

// h exp(d A) + own: what a segment whose steps sum to d makes of the state (or
// adjoint) that enters it.  By halves, for over many tokens the decay alone may
// leave fp32's range where its product with h does not; a zero stays zero.
template <int NP>
__device__ __forceinline__ void pass_segment(f32x2 (&h)[NP], float d, const f32x2 (&A2)[NP], const f32x2 (&own)[NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const float2 t = unpack2(ex2_2(mul2(twice(0.5f * d), A2[j])));
        const f32x2 e = pack2(fminf(t.x, 3e38f), fminf(t.y, 3e38f));
        h[j] = fma2(e, mul2(e, h[j]), own[j]);
    }
}

// The state before the block's segment, composed of the segments before it.
template <typename S>
__device__ __forceinline__ void start_state(const Args &a, const Where &w, int c, int n0, int x,
                                            const f32x2 (&A2)[S::NP], f32x2 (&h)[S::NP]) {
    const long long bc = (long long)w.b * a.C + c, stride = (long long)a.B * a.C;
    if (w.seg == 0) {
        if (a.h0) gather<S>((a.nseg > 1 ? a.seg_0 : a.h0) + bc * S::N + n0, x, h);
        return;
    }
    for (int s = 0; s < w.seg; ++s) {
        const float d = a.seg_d[s * stride + bc];
        f32x2 own[S::NP];
        gather<S>(a.seg_h + (s * stride + bc) * S::N + n0, x, own);
        pass_segment<S::NP>(h, d, A2, own);
    }
}

// A preparing thread's part in a tile: the token and channels it prepares,
// the token and indices of B and C it loads.
template <typename S> struct Part {
    int pt, pc, bt, bn;
    __device__ __forceinline__ Part(int tid)
        : pt(tid / S::VPR), pc(tid % S::VPR * S::EPT), bt(tid * S::BPT / S::N), bn(tid * S::BPT % S::N) {}
};

// D and D x (or g) of a token's channels.
template <typename S>
__device__ __forceinline__ void put_steps(float2 (*sd)[S::CT], int pt, int pc, const float (&d)[S::EPT],
                                          const float (&u)[S::EPT]) {
    if constexpr (S::EPT == 1) {
        sd[pt][S::place(pc, pt)] = make_float2(d[0], u[0]);
    } else {
#pragma unroll
        for (int e = 0; e + 1 < S::EPT; e += 2)
            *reinterpret_cast<float4 *>(&sd[pt][S::place(pc + e, pt)]) = make_float4(d[e], u[e], d[e + 1], u[e + 1]);
    }
}
// The same of a lane's channels, as its paired operations take them.
template <typename S> struct Steps {
    f32x2 d[S::CP], u[S::CP];
    __device__ __forceinline__ void get(const float2 *p) {
        if constexpr (S::CP == 2) {
            const float4 t = *reinterpret_cast<const float4 *>(p);
            d[0] = twice(t.x);
            u[0] = twice(t.y);
            d[1] = twice(t.z);
            u[1] = twice(t.w);
        } else {
            const float2 t = *p;
            d[0] = twice(t.x);
            u[0] = twice(t.y);
        }
    }
};

__device__ __forceinline__ void tile_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Where a lane of the recurrence works: first state index, channels.
template <typename S> struct Lane {
    int lane, ln, n0, cl;
    bool on[S::CP];
    __device__ __forceinline__ Lane(int tid, const Where &w)
        : lane(tid & 31), ln(lane % S::LN), n0(ln * S::NS), cl(((tid >> 5) * S::LC + lane / S::LN) * S::CP) {
#pragma unroll
        for (int i = 0; i < S::CP; ++i) on[i] = cl + i < w.nc;
    }
};

// ---------------------------------------------------------------- forward
// FULL: outputs, from the composed state.  STATE: a segment's final state
// from zero (the first segment's from h0) and its sum of D.  BACK: the
// adjoint that leaves a segment at its start when none enters at its end
// (p <- exp(D_t A) (p + C_t g_t), from the last token to the first).
enum Mode { FULL, STATE, BACK };

template <typename S> struct FwdSmem {
    alignas(16) float2 sd[2][S::TC][S::CT];  // D, D x (or g)
    alignas(16) float sy[2][S::TC][S::CS];   // <C, h>
    alignas(16) float sb[2][S::TC][S::N], sc[2][S::TC][S::N];
};

template <typename T, typename S, int V, Mode MODE>
__global__ void __launch_bounds__(2 * kThreads, 2) scan_fwd_kernel(Args a) {
    extern __shared__ __align__(16) unsigned char raw_smem[];
    FwdSmem<S> &sm = *reinterpret_cast<FwdSmem<S> *>(raw_smem);
    constexpr int NP = S::NP, TC = S::TC, TB = S::TB, CP = S::CP;
    const Where w(a, S::CT);
    const int end = min(w.t1, w.len);
    const int tiles = end > w.t0 ? (end - w.t0 + TC - 1) / TC : 0;               // those with tokens that count
    const int all = MODE == FULL ? (w.t1 - w.t0 + TC - 1) / TC : tiles;          // those with outputs
    const auto tile_of = [&](int k) { return MODE == BACK ? tiles - 1 - k : k; };  // the k-th that is worked on
    if (threadIdx.x < kThreads) {  // the recurrence
        const Lane<S> me(threadIdx.x, w);
        f32x2 A2[CP][NP], h[CP][NP];
        float sum[CP];
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < NP; ++j) A2[i][j] = h[i][j] = 0ull;
            const int c = w.c0 + me.cl + i;
            const long long at = ((long long)w.b * a.C + c) * S::N + me.n0;
            if (me.on[i]) gather<S>(a.A + (long long)c * S::N + me.n0, 0, A2[i]);
#pragma unroll
            for (int j = 0; j < NP; ++j) A2[i][j] = mul2(A2[i][j], twice(kLog2e));
            if (MODE == FULL && me.on[i]) start_state<S>(a, w, c, me.n0, 0, A2[i], h[i]);
            if (MODE == STATE && me.on[i] && w.seg == 0 && a.h0) {
                gather<S>(a.h0 + at, 0, h[i]);
                scatter<S>(a.seg_0 + at, 0, h[i]);
            }
        }
        const int k0 = S::place(me.cl, 0), k1 = S::place(me.cl, 1), o = halved_index<TB, 1, S::LN>(me.lane) * S::CS + me.cl;
        tile_barrier();
        for (int k = 0; k < all; ++k) {
            const int f = k & 1;
            const float2 *d0 = &sm.sd[f][0][k0], *d1 = &sm.sd[f][0][k1];
            const float *sb = &sm.sb[f][0][me.n0], *sc = &sm.sc[f][0][me.n0];
            float *out = &sm.sy[f][0][0] + o;
            if (k < tiles) {
                // Decays and terms of the next PB tokens are fetched and computed beside the chain of
                // these, and a batch's sums over the lanes wait until the next one's work is there to
                // hide them: there may be no more than one such warp a scheduler.
                constexpr int PB = 2;
                f32x2 e[2][PB][CP][NP], v[2][PB][CP][NP];
                const auto terms = [&](int s, f32x2(&e)[PB][CP][NP], f32x2(&v)[PB][CP][NP]) {
#pragma unroll
                    for (int u = 0; u < PB; ++u) {
                        const int t = MODE == BACK ? TC - 1 - s - u : s + u;
                        Steps<S> d;
                        d.get((t & 1 ? d1 : d0) + t * S::CT);
                        f32x2 b[NP];
                        load_pairs<NP>(sb + t * S::N, b);
#pragma unroll
                        for (int i = 0; i < CP; ++i) {
                            if (MODE == STATE) sum[i] += unpack2(d.d[i]).x;
#pragma unroll
                            for (int j = 0; j < NP; ++j) {
                                e[u][i][j] = decay_2(d.d[i], A2[i][j]);
                                v[u][i][j] = mul2(d.u[i], b[j]);
                            }
                        }
                    }
                };
                // The sums stay in registers until the tile's end: a store between would keep the loads
                // behind it from being issued ahead.
                float p[CP][TB], done[TC / TB][CP];
                const auto reduce = [&](int s) {
#pragma unroll
                    for (int i = 0; i < CP; ++i) {
                        halve<TB, 1, S::LN>(p[i], me.lane);
                        done[s / TB][i] = p[i][0];
                    }
                };
                terms(0, e[0], v[0]);
#pragma unroll
                for (int s = 0; s < TC; s += PB) {
                    const int g = s / PB & 1;
                    f32x2 q[PB][NP];
                    if (MODE == FULL)
#pragma unroll
                        for (int u = 0; u < PB; ++u) load_pairs<NP>(sc + (s + u) * S::N, q[u]);
                    if (s + PB < TC) terms(s + PB, e[g ^ 1], v[g ^ 1]);
                    if (MODE == FULL && s % TB == 0 && s > 0) reduce(s - TB);
#pragma unroll
                    for (int u = 0; u < PB; ++u)
#pragma unroll
                        for (int i = 0; i < CP; ++i) {
                            f32x2 y = 0ull;
#pragma unroll
                            for (int j = 0; j < NP; ++j) {
                                if (MODE == BACK) h[i][j] = mul2(e[g][u][i][j], add2(h[i][j], v[g][u][i][j]));
                                else h[i][j] = fma2(e[g][u][i][j], h[i][j], v[g][u][i][j]);
                                if (MODE == FULL) y = j ? fma2(h[i][j], q[u][j], y) : mul2(h[i][j], q[u][j]);
                            }
                            if (MODE == FULL) p[i][(s + u) % TB] = sum2(y);
                        }
                }
                if constexpr (MODE == FULL) {
                    reduce(TC - TB);
                    if (S::LN <= TB || me.ln < TB)
#pragma unroll
                        for (int s = 0; s < TC; s += TB) {
                            if constexpr (CP == 2) *reinterpret_cast<float2 *>(out + s * S::CS) = make_float2(done[s / TB][0], done[s / TB][1]);
                            else out[s * S::CS] = done[s / TB][0];
                        }
                }
            }
            tile_barrier();
        }
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            if (!me.on[i]) continue;
            const long long bc = (long long)w.b * a.C + w.c0 + me.cl + i, at = (long long)w.seg * a.B * a.C + bc;
            if (MODE == FULL) {
                if (a.h_L && w.seg == a.nseg - 1) scatter<S>(a.h_L + bc * S::N + me.n0, 0, h[i]);
            } else {
                scatter<S>((MODE == BACK ? a.seg_p : a.seg_h) + at * S::N + me.n0, 0, h[i]);
                if (MODE == STATE && me.ln == 0) a.seg_d[at] = sum[i];
            }
        }
    } else {  // preparation and outputs
        const Part<S> part(threadIdx.x - kThreads);
        const int pt = part.pt, pc = part.pc;
        float bias[S::EPT], dskip[S::EPT];
#pragma unroll
        for (int i = 0; i < S::EPT; ++i) {
            bias[i] = a.dt_bias && pc + i < w.nc ? a.dt_bias[w.c0 + pc + i] : 0.f;
            dskip[i] = a.D && pc + i < w.nc ? a.D[w.c0 + pc + i] : 0.f;
        }
        const long long ldx = MODE == BACK ? a.C : a.ldx, ldz = a.z ? a.ldz : ldx, ldb = MODE == BACK ? a.ldc : a.ldb;
        const T *px = static_cast<const T *>(MODE == BACK ? a.dy : a.x) + w.c0, *pd = static_cast<const T *>(a.dt) + w.c0;
        const T *pz = a.z ? static_cast<const T *>(a.z) + w.c0 : px;
        const T *pb = static_cast<const T *>(MODE == BACK ? a.Cm : a.Bm) + w.g * S::N + part.bn;
        const T *pq = static_cast<const T *>(a.Cm) + w.g * S::N + part.bn;
        Raw<T, S::EPT> rx, rd, rz, mx, mz, ox, oz;  // of the tile that comes in, the one worked on, the one to finish
        Raw<T, S::BPT> rb, rc;
        const auto load = [&](int k) {
            const int t = w.t0 + max(tile_of(k), 0) * TC;
            const long long row = (long long)w.b * a.L + min(t + pt, a.L - 1), rowb = (long long)w.b * a.L + min(t + part.bt, a.L - 1);
            rx = load_row<T, S::EPT, V>(px + row * ldx, pc, w.nc);
            rd = load_row<T, S::EPT, V>(pd + row * a.lddt, pc, w.nc);
            if (MODE != STATE) rz = load_row<T, S::EPT, V>(pz + row * ldz, pc, w.nc);
            rb = load_bc<T, S::BPT, (V > 1)>(pb + rowb * ldb);
            if (MODE == FULL) rc = load_bc<T, S::BPT, (V > 1)>(pq + rowb * a.ldc);
        };
        const auto prepare = [&](int k) {
            const int t = w.t0 + tile_of(k) * TC, f = k & 1;
            const bool in = t + pt < end, inb = t + part.bt < end;
            float x[S::EPT], d[S::EPT], b[S::BPT], q[S::BPT];
            widen<T, S::EPT>(rx, x);
            widen<T, S::EPT>(rd, d);
            widen<T, S::BPT>(rb, b);
            if constexpr (MODE == BACK) {
                float z[S::EPT];
                widen<T, S::EPT>(rz, z);
                if (a.z)
#pragma unroll
                    for (int e = 0; e < S::EPT; ++e) x[e] *= silu_f32(z[e]);
            }
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) d[e] += bias[e];
            if (a.softplus) softplus_all<S::EPT>(d);
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) {
                d[e] = in ? d[e] : 0.f;
                x[e] = in ? (MODE == BACK ? x[e] : d[e] * x[e]) : 0.f;
            }
            put_steps<S>(sm.sd[f], pt, pc, d, x);
#pragma unroll
            for (int e = 0; e < S::BPT; ++e) b[e] = inb ? b[e] : 0.f;
            store_raw<float, S::BPT>(&sm.sb[f][part.bt][part.bn], narrow<float, S::BPT>(b));
            if constexpr (MODE == FULL) {
                widen<T, S::BPT>(rc, q);
#pragma unroll
                for (int e = 0; e < S::BPT; ++e) q[e] = inb ? q[e] : 0.f;
                store_raw<float, S::BPT>(&sm.sc[f][part.bt][part.bn], narrow<float, S::BPT>(q));
            }
        };
        const auto finish = [&](int k) {
            const int t = w.t0 + k * TC, f = k & 1;
            if (t + pt >= w.t1 || pc >= w.nc) return;
            float x[S::EPT], z[S::EPT], o[S::EPT];
            widen<T, S::EPT>(ox, x);
            widen<T, S::EPT>(oz, z);
            widen<float, S::EPT>(load_raw<float, S::EPT>(&sm.sy[f][pt][pc]), o);
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) {
                o[e] = fmaf(dskip[e], x[e], o[e]);
                if (a.z) o[e] *= silu_f32(z[e]);
                o[e] = t + pt < end ? o[e] : 0.f;
            }
            T *y = static_cast<T *>(a.y) + ((long long)w.b * a.L + t + pt) * a.C + w.c0 + pc;
            store_row<T, S::EPT, V>(y, o, pc, w.nc);
        };
        load(0);
        prepare(0);
        mx = rx;
        mz = rz;
        load(1);
        tile_barrier();
        for (int k = 0; k < all; ++k) {
            if (MODE != BACK || k + 1 < all) prepare(k + 1);  // past the last tile: zeros that nothing reads
            const Raw<T, S::EPT> nx = rx, nz = rz;
            load(k + 2);
            if (MODE == FULL && k > 0) finish(k - 1);
            ox = mx;
            oz = mz;
            mx = nx;
            mz = nz;
            tile_barrier();
        }
        if (MODE == FULL) finish(all - 1);
    }
}

// ---------------------------------------------------------------- backward
// Two walks over the segment, each with four warps that run the recurrence
// and four that prepare and finish, as in the forward pass.  The first walk
// repeats the forward recurrence and leaves the state before every SUB-th
// token in the workspace, one vector a thread, where the second finds it in
// reverse order.  The second goes backwards: for SUB tokens at a time it
// recomputes decays and states into registers from that state, and then runs
// the adjoint down through them.
//
// dB and dC are sums over channels: a lane's 2 NS products of a token (its
// channels' added) are halved over the warp's channel lanes, then added over
// the block's warps in shared memory, and reach the workspace as one partial
// row a block; those and the sums over sequences (dA, dD, ddt_bias) are added
// by kernels of their own in a fixed order.  So that halving needs no
// selection, a lane whose channel bit says "keep the upper half" has its state
// values in the registers in swapped order (register j: state n0 + (j ^ x)),
// and reads B and C from a copy in that order.
//
// Bound by what four recurrence warps a block can issue: 2.2 instructions a
// clock and SM on two blocks, FMA pipes 41%, special functions 32%, shared
// memory 53%, while the preparing warps wait for them 40% of their time.
// Checkpoints every four tokens cost 8 bytes a value of traffic (13% of the copy
// rate); every eighth token would need twice the registers of the recurrence's half.

template <typename S> struct BwdSmem {
    // One order's copy of B or C, so long that the copies which neighbouring lanes read at once lie in
    // different banks (lanes of one access differ in the upper state bit first).
    static constexpr int COPY = S::TC * S::N + (S::NS == 4 ? 8 : 16);
    alignas(16) float2 sd[2][S::TC][S::CT];         // D, D x
    alignas(16) float sg[2][S::TC][S::CS];          // g
    alignas(16) float s1[2][S::TC][S::CS];          // <p, B>
    alignas(16) float s2[2][S::TC][S::CS];          // <p e h, A>
    alignas(16) float s3[2][S::TC][S::CS];          // <C, h>
    alignas(16) float sb[2][S::NS + 1][COPY];       // the last: zeros, for lanes without a channel
    alignas(16) float sc[2][S::NS + 1][COPY];
    alignas(16) float bc[2][kThreads / 32][S::TC][2][S::N];  // a warp's sums over its channels
};

template <typename T, typename S, int V>
__global__ void __launch_bounds__(2 * kThreads, S::N == 64 && S::CP == 2 ? 1 : 2) scan_bwd_kernel(Args a) {
    extern __shared__ __align__(16) unsigned char raw_smem[];
    BwdSmem<S> &sm = *reinterpret_cast<BwdSmem<S> *>(raw_smem);
    constexpr int NS = S::NS, NP = S::NP, LN = S::LN, TC = S::TC, TB = S::TB, CP = S::CP, SUB = NS * CP >= 4 ? 4 : 8;
    constexpr int QB = TB < SUB ? TB : SUB;  // tokens whose sums over the state index are taken together
    const Where w(a, S::CT);
    const int end = min(w.t1, w.len);
    const int tiles = end > w.t0 ? (end - w.t0 + TC - 1) / TC : 0;
    const int all = (w.t1 - w.t0 + TC - 1) / TC;  // tiles with padding: their outputs are zeros
    float *sums = a.part + (long long)(w.seg * a.B + w.b) * a.C * (S::N + 2);
    if (threadIdx.x < kThreads) {  // the recurrences
        const int tid = threadIdx.x, warp = tid >> 5;
        const Lane<S> me(tid, w);
        const int lane = me.lane, n0 = me.n0, ox = halved_index<NS, LN, 32>(lane);  // the order of this lane's states
        const int copy = me.on[0] ? ox : NS;
        f32x2 A2[CP][NP], h[CP][NP];
#pragma unroll
        for (int i = 0; i < CP; ++i) {
#pragma unroll
            for (int j = 0; j < NP; ++j) A2[i][j] = h[i][j] = 0ull;
            if (me.on[i]) gather<S>(a.A + (long long)(w.c0 + me.cl + i) * S::N + n0, ox, A2[i]);
#pragma unroll
            for (int j = 0; j < NP; ++j) A2[i][j] = mul2(A2[i][j], twice(kLog2e));
            if (me.on[i]) start_state<S>(a, w, w.c0 + me.cl + i, n0, ox, A2[i], h[i]);
        }
        constexpr int CKS = kThreads * NS * CP;  // floats of one checkpoint of the block
        float *ck = a.ckpt + (long long)blockIdx.x * (a.seg / SUB) * CKS + tid * NS;
        const int k0 = S::place(me.cl, 0), k1 = S::place(me.cl, 1);
        tile_barrier();
        for (int k = 0; k < tiles; ++k) {
            const int f = k & 1;
            const float2 *d0 = &sm.sd[f][0][k0], *d1 = &sm.sd[f][0][k1];
            const float *lb = &sm.sb[f][copy][n0];
#pragma unroll
            for (int s = 0; s < TC; s += SUB) {
#pragma unroll
                for (int i = 0; i < CP; ++i) store_pairs<NP>(ck + (long long)((k * TC + s) / SUB) * CKS + i * kThreads * NS, h[i]);
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    Steps<S> d;
                    d.get((u & 1 ? d1 : d0) + (s + u) * S::CT);
                    f32x2 b[NP];
                    load_pairs<NP>(lb + (s + u) * S::N, b);
#pragma unroll
                    for (int i = 0; i < CP; ++i)
#pragma unroll
                        for (int j = 0; j < NP; ++j) h[i][j] = fma2(decay_2(d.d[i], A2[i][j]), h[i][j], mul2(d.u[i], b[j]));
                }
            }
            tile_barrier();
        }

        // the adjoint that enters at the segment's end
        f32x2 A1[CP][NP], p[CP][NP], dA[CP][NP], lost[CP][NP], next[CP][NP];
#pragma unroll
        for (int i = 0; i < CP; ++i) {
#pragma unroll
            for (int j = 0; j < NP; ++j) A1[i][j] = p[i][j] = dA[i][j] = lost[i][j] = 0ull;
            if (!me.on[i]) continue;
            const long long bc = (long long)w.b * a.C + w.c0 + me.cl + i, stride = (long long)a.B * a.C;
            gather<S>(a.A + (long long)(w.c0 + me.cl + i) * S::N + n0, ox, A1[i]);
            if (a.dh_L) gather<S>(a.dh_L + bc * S::N + n0, ox, p[i]);
            for (int s = a.nseg - 1; s > w.seg; --s) {
                const float d = a.seg_d[s * stride + bc];
                f32x2 own[NP];
                gather<S>(a.seg_p + (s * stride + bc) * S::N + n0, ox, own);
                pass_segment<NP>(p[i], d, A2[i], own);
            }
        }
        if (tiles)
#pragma unroll
            for (int i = 0; i < CP; ++i)
                load_pairs<NP>(ck + (long long)(tiles * TC / SUB - 1) * CKS + i * kThreads * NS, next[i]);
        tile_barrier();
        for (int i0 = all - 1; i0 >= 0; --i0) {
            const int f = i0 & 1;
            const float2 *d0 = &sm.sd[f][0][k0], *d1 = &sm.sd[f][0][k1];
            const float *sg = &sm.sg[f][0][me.cl], *lb = &sm.sb[f][copy][n0], *lc = &sm.sc[f][copy][n0];
            if (i0 < tiles) {
#pragma unroll 1
                for (int s = TC - SUB; s >= 0; s -= SUB) {
                    f32x2 hs[SUB + 1][CP][NP], es[SUB][CP][NP], part_dA[CP][NP];
#pragma unroll
                    for (int i = 0; i < CP; ++i)
#pragma unroll
                        for (int j = 0; j < NP; ++j) {
                            hs[0][i][j] = next[i][j];
                            part_dA[i][j] = 0ull;
                        }
                    const int before = max((i0 * TC + s) / SUB - 1, 0);
#pragma unroll
                    for (int i = 0; i < CP; ++i) load_pairs<NP>(ck + (long long)before * CKS + i * kThreads * NS, next[i]);
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        Steps<S> d;
                        d.get((u & 1 ? d1 : d0) + (s + u) * S::CT);
                        f32x2 b[NP];
                        load_pairs<NP>(lb + (s + u) * S::N, b);
#pragma unroll
                        for (int i = 0; i < CP; ++i)
#pragma unroll
                            for (int j = 0; j < NP; ++j) {
                                es[u][i][j] = decay_2(d.d[i], A2[i][j]);
                                hs[u + 1][i][j] = fma2(es[u][i][j], hs[u][i][j], mul2(d.u[i], b[j]));
                            }
                    }
                    constexpr int SB = NS == 4 ? (S::LC >= 4 ? 2 : 1) : 1;  // state bits that are halved
                    constexpr int V1 = 2 * NS >> SB, ST = LN << SB;          // what that leaves in a lane; the next lane bit
                    // sums stay in registers until the end: a store between would keep the loads behind it
                    // from being issued ahead
                    float left[SUB][ST < 32 ? 1 : V1], q1[SUB / QB][CP][QB], q2[SUB / QB][CP][QB], q3[SUB / QB][CP][QB];
#pragma unroll
                    for (int u0 = SUB - QB; u0 >= 0; u0 -= QB) {
#pragma unroll
                        for (int r = QB - 1; r >= 0; --r) {
                            const int u = u0 + r;
                            Steps<S> d;
                            d.get((u & 1 ? d1 : d0) + (s + u) * S::CT);
                            f32x2 b[NP], q[NP], gg[CP];
                            load_pairs<NP>(lb + (s + u) * S::N, b);
                            load_pairs<NP>(lc + (s + u) * S::N, q);
                            if constexpr (CP == 2) {
                                const float2 t = *reinterpret_cast<const float2 *>(sg + (s + u) * S::CS);
                                gg[0] = twice(t.x);
                                gg[1] = twice(t.y);
                            } else {
                                gg[0] = twice(sg[(s + u) * S::CS]);
                            }
                            f32x2 mb[NP], mc[NP];
#pragma unroll
                            for (int j = 0; j < NP; ++j) mb[j] = mc[j] = 0ull;
#pragma unroll
                            for (int i = 0; i < CP; ++i) {
                                f32x2 y1 = 0ull, y2 = 0ull, y3 = 0ull;
                                // Half a pair's channels may be none where rows are not whole vectors: those
                                // add nothing, even beside an infinite B or C.
                                const bool add = V > 1 || i == 0 || me.on[i];
#pragma unroll
                                for (int j = 0; j < NP; ++j) {
                                    f32x2 &pj = p[i][j];
                                    pj = fma2(q[j], gg[i], pj);
                                    if (add) {
                                        mb[j] = i ? fma2(pj, d.u[i], mb[j]) : mul2(pj, d.u[i]);
                                        mc[j] = i ? fma2(hs[u + 1][i][j], gg[i], mc[j]) : mul2(hs[u + 1][i][j], gg[i]);
                                    }
                                    y1 = j ? fma2(pj, b[j], y1) : mul2(pj, b[j]);
                                    y3 = j ? fma2(hs[u + 1][i][j], q[j], y3) : mul2(hs[u + 1][i][j], q[j]);
                                    pj = mul2(pj, es[u][i][j]);
                                    const f32x2 back = mul2(pj, hs[u][i][j]);
                                    y2 = j ? fma2(back, A1[i][j], y2) : mul2(back, A1[i][j]);
                                    part_dA[i][j] = fma2(back, d.d[i], part_dA[i][j]);
                                }
                                q1[u0 / QB][i][r] = sum2(y1);
                                q2[u0 / QB][i][r] = sum2(y2);
                                q3[u0 / QB][i][r] = sum2(y3);
                            }
                            float m[2 * NS];  // of each register j: dB, dC
#pragma unroll
                            for (int j = 0; j < NP; ++j) {
                                const float2 tb = unpack2(mb[j]), tc = unpack2(mc[j]);
                                m[4 * j] = tb.x;
                                m[4 * j + 1] = tc.x;
                                m[4 * j + 2] = tb.y;
                                m[4 * j + 3] = tc.y;
                            }
                            // over the channel lanes: first the state bits, by the lanes' orders, then dB from dC
#pragma unroll
                            for (int k = 0; k < NS; ++k) m[k] += __shfl_xor_sync(0xffffffffu, m[k + NS], LN);
                            if constexpr (SB == 2)
#pragma unroll
                                for (int k = 0; k < NS / 2; ++k) m[k] += __shfl_xor_sync(0xffffffffu, m[k + NS / 2], 2 * LN);
                            if constexpr (ST < 32) {
                                static_assert(V1 == 2, "one state is left where lanes are");
                                halve<2, ST, 32>(m, lane);
                                left[u][0] = m[0];
                            } else {
#pragma unroll
                                for (int k = 0; k < V1; ++k) left[u][k] = m[k];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < CP; ++i) {
                            halve<QB, 1, LN>(q1[u0 / QB][i], lane);
                            halve<QB, 1, LN>(q2[u0 / QB][i], lane);
                            if (a.z) halve<QB, 1, LN>(q3[u0 / QB][i], lane);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        if constexpr (ST < 32) {
                            sm.bc[f][warp][s + u][(lane & ST) ? 1 : 0][n0 + ox] = left[u][0];
                        } else {  // V1 / 2 states (registers 0 ..), dB and dC of each
#pragma unroll
                            for (int k = 0; k < V1; ++k) sm.bc[f][warp][s + u][k & 1][n0 + ((k >> 1) ^ ox)] = left[u][k];
                        }
                    }
                    if (LN <= QB || me.ln < QB)
#pragma unroll
                        for (int u0 = 0; u0 < SUB; u0 += QB) {
                            const int tt = s + u0 + halved_index<QB, 1, LN>(lane);
#pragma unroll
                            for (int i = 0; i < CP; ++i) {
                                sm.s1[f][tt][me.cl + i] = q1[u0 / QB][i][0];
                                sm.s2[f][tt][me.cl + i] = q2[u0 / QB][i][0];
                                sm.s3[f][tt][me.cl + i] = q3[u0 / QB][i][0];
                            }
                        }
                    // the long sum over tokens, with what its additions lose carried on
#pragma unroll
                    for (int i = 0; i < CP; ++i)
#pragma unroll
                        for (int j = 0; j < NP; ++j) {
                            const f32x2 add = add2(part_dA[i][j], lost[i][j]), to = add2(dA[i][j], add);
                            lost[i][j] = add2(add, fma2(to, twice(-1.f), dA[i][j]));
                            dA[i][j] = to;
                        }
                }
            }
            tile_barrier();
        }
#pragma unroll
        for (int i = 0; i < CP; ++i)
            if (me.on[i]) {
                const int c = w.c0 + me.cl + i;
                if (w.seg == 0 && a.dh0) scatter<S>(a.dh0 + ((long long)w.b * a.C + c) * S::N + n0, ox, p[i]);
                scatter<S>(sums + (long long)c * S::N + n0, ox, dA[i]);
            }
    } else {  // preparation and outputs
        const int tid = threadIdx.x - kThreads;
        const Part<S> part(tid);
        const int pt = part.pt, pc = part.pc;
        float bias[S::EPT], dskip[S::EPT], aD[S::EPT], ab[S::EPT];
#pragma unroll
        for (int i = 0; i < S::EPT; ++i) {
            bias[i] = a.dt_bias && pc + i < w.nc ? a.dt_bias[w.c0 + pc + i] : 0.f;
            dskip[i] = a.D && pc + i < w.nc ? a.D[w.c0 + pc + i] : 0.f;
            aD[i] = ab[i] = 0.f;
        }
        const T *px = static_cast<const T *>(a.x) + w.c0, *pd = static_cast<const T *>(a.dt) + w.c0;
        const T *py = static_cast<const T *>(a.dy) + w.c0, *pz = a.z ? static_cast<const T *>(a.z) + w.c0 : px;
        const long long ldz = a.z ? a.ldz : a.ldx;
        const T *pb = static_cast<const T *>(a.Bm) + w.g * S::N + part.bn, *pq = static_cast<const T *>(a.Cm) + w.g * S::N + part.bn;
        // lanes without a channel meet zeros alone, so that they add zeros to dB and dC
        for (int k = tid; k < 2 * BwdSmem<S>::COPY; k += kThreads) {
            sm.sb[k & 1][NS][k >> 1] = 0.f;
            sm.sc[k & 1][NS][k >> 1] = 0.f;
        }
        struct Rows {
            Raw<T, S::EPT> x, d, y, z;
        };
        Rows in_, mid, old;  // of the tile that comes in, the one worked on, the one to finish
        Raw<T, S::BPT> rb, rc;
        const auto load = [&](int i, bool back) {
            const int t = w.t0 + max(i, 0) * TC;
            const long long row = (long long)w.b * a.L + min(t + pt, a.L - 1), rowb = (long long)w.b * a.L + min(t + part.bt, a.L - 1);
            in_.x = load_row<T, S::EPT, V>(px + row * a.ldx, pc, w.nc);
            in_.d = load_row<T, S::EPT, V>(pd + row * a.lddt, pc, w.nc);
            rb = load_bc<T, S::BPT, (V > 1)>(pb + rowb * a.ldb);
            if (back) {
                in_.y = load_row<T, S::EPT, V>(py + row * a.C, pc, w.nc);
                in_.z = load_row<T, S::EPT, V>(pz + row * ldz, pc, w.nc);
                rc = load_bc<T, S::BPT, (V > 1)>(pq + rowb * a.ldc);
            }
        };
        // B or C of the tile, zeros past the end, in every lane's order
        const auto put_bc = [&](float (*to)[BwdSmem<S>::COPY], const Raw<T, S::BPT> &r, bool inb) {
            float v[S::BPT];
            widen<T, S::BPT>(r, v);
#pragma unroll
            for (int e = 0; e < S::BPT; ++e) v[e] = inb ? v[e] : 0.f;
            const int at = part.bt * S::N + part.bn;
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                if constexpr (S::BPT % 4 == 0) {
#pragma unroll
                    for (int e = 0; e < S::BPT; e += 4)
                        *reinterpret_cast<float4 *>(&to[k][at + e]) = make_float4(v[e ^ k], v[(e + 1) ^ k], v[(e + 2) ^ k], v[(e + 3) ^ k]);
                } else {
#pragma unroll
                    for (int e = 0; e < S::BPT; ++e) to[k][(at + e) ^ k] = v[e];
                }
            }
        };
        const auto prepare = [&](int i, bool back) {
            const int t = w.t0 + i * TC, f = i & 1;
            const bool inb = t + part.bt < end;
            bool in[S::EPT];
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) in[e] = t + pt < end && pc + (e & -V) < w.nc;
            float x[S::EPT], d[S::EPT];
            widen<T, S::EPT>(in_.x, x);
            widen<T, S::EPT>(in_.d, d);
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) d[e] += bias[e];
            if (a.softplus) softplus_all<S::EPT>(d);
#pragma unroll
            for (int e = 0; e < S::EPT; ++e) {
                d[e] = in[e] ? d[e] : 0.f;
                x[e] = in[e] ? d[e] * x[e] : 0.f;
            }
            put_steps<S>(sm.sd[f], pt, pc, d, x);
            put_bc(sm.sb[f], rb, inb);
            if (back) {
                float g[S::EPT], z[S::EPT];
                widen<T, S::EPT>(in_.y, g);
                widen<T, S::EPT>(in_.z, z);
#pragma unroll
                for (int e = 0; e < S::EPT; ++e) {
                    if (a.z) g[e] *= silu_f32(z[e]);
                    g[e] = in[e] ? g[e] : 0.f;
                }
                store_raw<float, S::EPT>(&sm.sg[f][pt][pc], narrow<float, S::EPT>(g));
                put_bc(sm.sc[f], rc, inb);
            }
        };
        const auto finish = [&](int i) {
            const int t = w.t0 + i * TC, f = i & 1;
            const bool in = t + pt < end;
            if (t + pt < w.t1 && pc < w.nc) {
                float x[S::EPT], v[S::EPT], y[S::EPT], z[S::EPT], g[S::EPT], q1[S::EPT], q2[S::EPT], q3[S::EPT];
                widen<T, S::EPT>(old.x, x);
                widen<T, S::EPT>(old.d, v);
                widen<T, S::EPT>(old.y, y);
                widen<T, S::EPT>(old.z, z);
                widen<float, S::EPT>(load_raw<float, S::EPT>(&sm.sg[f][pt][pc]), g);
                widen<float, S::EPT>(load_raw<float, S::EPT>(&sm.s1[f][pt][pc]), q1);
                widen<float, S::EPT>(load_raw<float, S::EPT>(&sm.s2[f][pt][pc]), q2);
                widen<float, S::EPT>(load_raw<float, S::EPT>(&sm.s3[f][pt][pc]), q3);
#pragma unroll
                for (int e = 0; e < S::EPT; ++e) {
                    const float d = sm.sd[f][pt][S::place(pc + e, pt)].x;
                    q2[e] = fmaf(x[e], q1[e], q2[e]);
                    if (a.softplus) q2[e] *= sigmoid_f32(v[e] + bias[e]);
                    q1[e] = fmaf(d, q1[e], dskip[e] * g[e]);
                    if (a.z) z[e] = y[e] * fmaf(dskip[e], x[e], q3[e]) * dsilu_f32(z[e]);
                    q1[e] = in ? q1[e] : 0.f;
                    q2[e] = in ? q2[e] : 0.f;
                    z[e] = in ? z[e] : 0.f;
                    ab[e] += q2[e];
                    aD[e] += in ? g[e] * x[e] : 0.f;
                }
                const long long at = ((long long)w.b * a.L + t + pt) * a.C + w.c0 + pc;
                store_row<T, S::EPT, V>(static_cast<T *>(a.dx) + at, q1, pc, w.nc);
                store_row<T, S::EPT, V>(static_cast<T *>(a.ddt) + at, q2, pc, w.nc);
                if (a.z) store_row<T, S::EPT, V>(static_cast<T *>(a.dz) + at, z, pc, w.nc);
            }
            // the block's share of dB and dC
            for (int k = tid * 4; k < TC * 2 * S::N; k += kThreads * 4) {
                const int tt = k / (2 * S::N), r = k % (2 * S::N);
                if (t + tt >= w.t1) break;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t + tt < end)
#pragma unroll
                    for (int u = 0; u < kThreads / 32; ++u) {
                        const float4 o = *reinterpret_cast<const float4 *>(&sm.bc[f][u][tt][0][0] + r);
                        v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
                    }
                *reinterpret_cast<float4 *>(a.part_bc + ((((long long)w.tile * a.B + w.b) * a.L + t + tt) * a.G + w.g) * (2 * S::N) + r) = v;
            }
        };
        load(0, false);
        prepare(0, false);
        load(1, false);
        tile_barrier();
        for (int k = 0; k < tiles; ++k) {
            if (k + 1 < tiles) prepare(k + 1, false);
            load(k + 2, false);
            tile_barrier();
        }
        load(all - 1, true);
        prepare(all - 1, true);
        mid = in_;
        load(all - 2, true);
        tile_barrier();
        for (int i = all - 1; i >= 0; --i) {
            if (i + 1 < all) finish(i + 1);  // reads D and g where the next line puts those of tile i - 1
            if (i > 0) prepare(i - 1, true);
            const Rows now = in_;
            load(i - 2, true);
            old = mid;
            mid = now;
            tile_barrier();
        }
        finish(0);
        // dD and ddt_bias: over the tokens that each thread prepared
        asm volatile("bar.sync 2, 128;" ::: "memory");  // every finish is done with s1 and s2
#pragma unroll
        for (int e = 0; e < S::EPT; ++e) {
            sm.s1[0][pt][pc + e] = aD[e];
            sm.s2[0][pt][pc + e] = ab[e];
        }
        asm volatile("bar.sync 2, 128;" ::: "memory");
        if (tid < w.nc) {
            float u = 0.f, v = 0.f;
            for (int tt = 0; tt < TC; ++tt) {
                u += sm.s1[0][tt][tid];
                v += sm.s2[0][tt][tid];
            }
            sums[(long long)a.C * S::N + w.c0 + tid] = u;
            sums[(long long)a.C * (S::N + 1) + w.c0 + tid] = v;
        }
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
// The state is read and written once: HBM bound, 8 N bytes a channel.  A
// thread has eight values of a channel's state: with four, the step's
// softplus and the loads of single values weigh more (256 x 8192 x 16: 61 us
// against 89, the state's bytes at the copy rate 41), with sixteen, or two
// sequences, fewer threads are resident (69, 64).  64 x 4096 x 16: 10.2 to 10.8 us
// from HBM, 8.0 where L2 holds the states: 4096 blocks in 1.7 waves.
template <typename T, int N> __global__ void __launch_bounds__(128) scan_step_kernel(Args a) {
    constexpr int NS = 8, LN = N / NS;
    const int i = blockIdx.x * 128 + threadIdx.x, c = i / LN, n0 = (i % LN) * NS, b = blockIdx.y;
    const bool on = c < a.C;
    float p = 0.f, x = 0.f, z = 0.f, dskip = 0.f;
    if (on) {
        const int off = c / (a.C / a.G) * N + n0;
        const auto eight = [&](const void *base, long long ld) {
            const T *q = static_cast<const T *>(base) + b * ld + off;
            return a.vec ? load_raw<T, NS>(q) : load_bc<T, NS, false>(q);
        };
        float *at = a.h_L + ((long long)b * a.C + c) * N + n0;
        float h[NS], A[NS], bv[NS], cv[NS];
        widen<float, NS>(load_raw<float, NS>(at), h);
        widen<float, NS>(load_raw<float, NS>(a.A + (long long)c * N + n0), A);
        widen<T, NS>(eight(a.Bm, a.ldb), bv);
        widen<T, NS>(eight(a.Cm, a.ldc), cv);
        x = to_f32(static_cast<const T *>(a.x)[b * a.ldx + c]);
        if (a.z) z = to_f32(static_cast<const T *>(a.z)[b * a.ldz + c]);
        if (a.D) dskip = a.D[c];
        float d = to_f32(static_cast<const T *>(a.dt)[b * a.lddt + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
        if (a.softplus) d = softplus_f32(d);
        const float u = d * x, e = d * kLog2e;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            h[j] = fmaf(ex2(fmaf(e, A[j], kCentre)), h[j], u * bv[j]);
            p = fmaf(h[j], cv[j], p);
        }
        store_raw<float, NS>(at, narrow<float, NS>(h));
    }
#pragma unroll
    for (int o = LN / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
    if (on && n0 == 0) {
        float y = fmaf(dskip, x, p);
        if (a.z) y *= silu_f32(z);
        static_cast<T *>(a.y)[(long long)b * a.C + c] = from_f32<T>(y);
    }
}

}  // namespace scan
}  // namespace efla
