// efla_conv.cuh - the short causal convolution along the sequence, one
// filter of K taps a channel, with an optional SiLU; its backward pass and
// its one-token step.  (The pages' layer has one of width 4 in front of the
// mixer: jsqmd.com blog, section 4.1.)
//
//   pre_t = bias + sum_j w_j x_{t-K+1+j},  y = pre or silu(pre)
//   x_{-K+1} .. x_{-1} = state (or 0);  state_out = the last K-1 inputs
//   backward: d_t = dy_t silu'(pre_t),  dx_t = sum_j w_j d_{t+K-1-j},
//             dw_j = sum d_t x_{t-K+1+j},  dbias = sum d_t
//
// HBM bound.  A thread owns VEC neighbouring channels and walks TT tokens
// with the last K-1 inputs in registers, so x is read once but for the K-1
// rows where its run begins (those lie in the L1 or L2 of the run before).
// Eight runs make a block; 32 lanes side by side cover 32 VEC channels.
// y may go to [B][H][L][d] directly, the layout the mixer reads.
#pragma once
#include "efla_vec.cuh"

namespace efla {
namespace conv {

constexpr int kWarps = 8;
constexpr int kRunFwd = 32, kRunBwd = 32;  // tokens of one thread's run

struct Args {
    const void *x;
    long long ldx;  // elements from one token's row of x to the next
    const float *w, *bias;
    const void *state;
    const int *lengths;
    int silu, head;  // head: channels of a head where y (or dy) is [B][H][L][head], 0 where it is [B][L][C]
    int B, L, C, tiles;
    // forward
    void *y, *state_out;
    // backward
    const void *dy, *dstate_out;
    void *dx, *dstate;
    float *part_w, *part_b;  // [B * tiles][C * K], [B * tiles][C]
};

__device__ __forceinline__ int length_of(const Args &a, int b) {
    if (!a.lengths) return a.L;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.L ? a.L : n;
}

// Element offset of (b, t, c) in y or dy.
__device__ __forceinline__ long long out_at(const Args &a, int b, long long t, int c) {
    if (!a.head) return ((long long)b * a.L + t) * a.C + c;
    return (((long long)b * (a.C / a.head) + c / a.head) * a.L + t) * a.head + c % a.head;
}

// Filters w[j][i] of VEC channels from channel c on.
template <int K, int VEC> __device__ __forceinline__ void load_filters(const float *p, int c, float (&w)[K][VEC]) {
    float v[VEC * K];
    p += (long long)c * K;
    if constexpr (VEC * K % 4 == 0) {  // c is a multiple of VEC, so the filters begin on 16 bytes
#pragma unroll
        for (int i = 0; i < VEC * K; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i);
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC * K; ++i) v[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = v[i * K + j];
}

template <typename T, int K, int VEC>
__global__ void __launch_bounds__(32 * kWarps) conv_fwd_kernel(Args a) {
    constexpr int U = 4;  // rows in flight
    const int b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int c = (blockIdx.y * 32 + (threadIdx.x & 31)) * VEC, warp = threadIdx.x >> 5;
    const int t0 = (tile * kWarps + warp) * kRunFwd;
    if (c >= a.C || (t0 >= a.L && t0 > 0)) return;
    const int len = length_of(a, b);
    const T *x = static_cast<const T *>(a.x) + (long long)b * a.L * a.ldx + c;
    const T *st = a.state ? static_cast<const T *>(a.state) + (long long)b * (K - 1) * a.C + c : nullptr;
    T *y = static_cast<T *>(a.y) + out_at(a, b, 0, c);
    const long long ldy = a.head ? a.head : a.C;

    float w[K][VEC], bias[VEC], win[K - 1][VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.f;
    load_filters<K, VEC>(a.w, c, w);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int t = t0 - (K - 1) + j;
        Raw<T, VEC> r = zero_raw<T, VEC>();
        if (t >= 0) {
            if (t < len) r = load_raw<T, VEC>(x + t * a.ldx);
        } else if (st) {
            r = load_raw<T, VEC>(st + (long long)(t + K - 1) * a.C);
        }
        widen<T, VEC>(r, win[j]);
    }
    const int t1 = min(t0 + kRunFwd, a.L);
    for (int t = t0; t < t1; t += U) {
        Raw<T, VEC> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = t + u < len && t + u < t1 ? load_raw<T, VEC>(x + (t + u) * a.ldx) : zero_raw<T, VEC>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= t1) break;
            float v[VEC], o[VEC];
            widen<T, VEC>(r[u], v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float s = bias[i];
#pragma unroll
                for (int j = 0; j < K - 1; ++j) s = fmaf(w[j][i], win[j][i], s);
                s = fmaf(w[K - 1][i], v[i], s);
                o[i] = t + u < len ? (a.silu ? silu_f32(s) : s) : 0.f;
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) win[j][i] = win[j + 1][i];
                win[K - 2][i] = v[i];
            }
            store_raw<T, VEC>(y + (t + u) * ldy, narrow<T, VEC>(o));
        }
    }
    if (a.state_out && t0 == 0) {
        // last: this thread is the only reader of these channels' state, so state_out may be the state itself
        Raw<T, VEC> keep[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int t = len - (K - 1) + j;
            keep[j] = t >= 0 ? load_raw<T, VEC>(x + t * a.ldx)
                      : st   ? load_raw<T, VEC>(st + (long long)(t + K - 1) * a.C)
                             : zero_raw<T, VEC>();
        }
        T *so = static_cast<T *>(a.state_out) + (long long)b * (K - 1) * a.C + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) store_raw<T, VEC>(so + (long long)j * a.C, keep[j]);
    }
}

// The run of a thread computes d for its own tokens and the K-1 after them,
// which its last dx need; dw and dbias count its own tokens alone.  The
// eight runs of a block add theirs up in shared memory and the block writes
// one partial row, which colsum_kernel adds in a fixed order.
template <typename T, int K, int VEC>
__global__ void __launch_bounds__(32 * kWarps) conv_bwd_kernel(Args a) {
    constexpr int U = 4;
    __shared__ float red[kWarps][32 * VEC * (K + 1)];
    const int b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const int t0 = (tile * kWarps + warp) * kRunBwd;
    const bool on = c < a.C && (t0 < a.L || t0 == 0);
    float dw[K][VEC], db[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = 0.f;
    }
    if (on) {
        const int len = length_of(a, b);
        const T *x = static_cast<const T *>(a.x) + (long long)b * a.L * a.ldx + c;
        const T *st = a.state ? static_cast<const T *>(a.state) + (long long)b * (K - 1) * a.C + c : nullptr;
        const T *dso = a.dstate_out ? static_cast<const T *>(a.dstate_out) + (long long)b * (K - 1) * a.C + c : nullptr;
        const T *dy = static_cast<const T *>(a.dy) + out_at(a, b, 0, c);
        const long long ldy = a.head ? a.head : a.C;
        T *dx = static_cast<T *>(a.dx) + (long long)b * a.L * a.C + c;
        T *ds = a.dstate ? static_cast<T *>(a.dstate) + (long long)b * (K - 1) * a.C + c : nullptr;

        float w[K][VEC], bias[VEC], win[K][VEC], dwin[K][VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) dwin[j][i] = 0.f;
        }
        load_filters<K, VEC>(a.w, c, w);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {  // x_{t0-K+1} .. x_{t0-1}, moved down by one when t0 itself comes in
            const int t = t0 - (K - 1) + j;
            Raw<T, VEC> r = zero_raw<T, VEC>();
            if (t >= 0) {
                if (t < len) r = load_raw<T, VEC>(x + t * a.ldx);
            } else if (st) {
                r = load_raw<T, VEC>(st + (long long)(t + K - 1) * a.C);
            }
            widen<T, VEC>(r, win[j + 1]);
        }
        const int te = t0 + kRunBwd + K - 1;
        for (int t = t0; t < te; t += U) {
            Raw<T, VEC> rx[U], ry[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = t + u < len && t + u < te;
                rx[u] = in ? load_raw<T, VEC>(x + (t + u) * a.ldx) : zero_raw<T, VEC>();
                ry[u] = in ? load_raw<T, VEC>(dy + (t + u) * ldy) : zero_raw<T, VEC>();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u;
                if (tt >= te) break;
                const int to = tt - (K - 1);  // the token whose dx is complete now
                float xv[VEC], yv[VEC], o[VEC];
                widen<T, VEC>(rx[u], xv);
                widen<T, VEC>(ry[u], yv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) {
                        win[j][i] = win[j + 1][i];
                        dwin[j][i] = dwin[j + 1][i];
                    }
                    win[K - 1][i] = xv[i];
                    float d = 0.f;
                    if (tt < len) {
                        d = yv[i];
                        if (a.silu) {
                            float s = bias[i];
#pragma unroll
                            for (int j = 0; j < K; ++j) s = fmaf(w[j][i], win[j][i], s);
                            d *= dsilu_f32(s);
                        }
                    }
                    dwin[K - 1][i] = d;
                    if (tt < t0 + kRunBwd) {
                        db[i] += d;
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][i] = fmaf(d, win[j][i], dw[j][i]);
                    }
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) s = fmaf(w[K - 1 - j][i], dwin[j][i], s);
                    o[i] = s;
                }
                if (to >= a.L || (to < t0 && to >= 0) || (to < 0 && t0 > 0)) continue;
                const int at = to - len + K - 1;  // the row of state_out that holds x_to
                if (dso && at >= 0 && at < K - 1) {
                    float g[VEC];
                    widen<T, VEC>(load_raw<T, VEC>(dso + (long long)at * a.C), g);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o[i] += g[i];
                }
                if (to >= 0)
                    store_raw<T, VEC>(dx + (long long)to * a.C, narrow<T, VEC>(o));
                else if (ds)
                    store_raw<T, VEC>(ds + (long long)(to + K - 1) * a.C, narrow<T, VEC>(o));
            }
        }
    }
    float *mine = &red[warp][0];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) mine[(lane * VEC + i) * K + j] = dw[j][i];
        mine[32 * VEC * K + lane * VEC + i] = db[i];
    }
    __syncthreads();
    const int c0 = blockIdx.y * 32 * VEC, n = min(32 * VEC, a.C - c0);
    for (int i = threadIdx.x; i < 32 * VEC * (K + 1); i += 32 * kWarps) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += red[k][i];
        if (i < 32 * VEC * K) {
            if (i < n * K) a.part_w[((long long)blockIdx.x * a.C + c0) * K + i] = s;
        } else if (i - 32 * VEC * K < n) {
            a.part_b[(long long)blockIdx.x * a.C + c0 + i - 32 * VEC * K] = s;
        }
    }
}

// One token: y from the state and x, then the state moved up by one.  A
// thread owns its channels' state, so the update is in place.
template <typename T, int K, int VEC>
__global__ void __launch_bounds__(128) conv_step_kernel(const T *x, long long ldx, T *state, const float *w,
                                                        const float *bias, T *y, int silu, int C) {
    const int c = (blockIdx.y * 128 + threadIdx.x) * VEC;
    if (c >= C) return;
    const long long b = blockIdx.x;
    T *st = state + b * (K - 1) * C + c;
    Raw<T, VEC> r[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j] = load_raw<T, VEC>(st + (long long)j * C);
    r[K - 1] = load_raw<T, VEC>(x + b * ldx + c);
    float o[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float s = bias ? bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) s = fmaf(w[(long long)(c + i) * K + j], to_f32(r[j].e[i]), s);
        o[i] = silu ? silu_f32(s) : s;
    }
    store_raw<T, VEC>(y + b * C + c, narrow<T, VEC>(o));
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_raw<T, VEC>(st + (long long)j * C, r[j + 1]);
}

}  // namespace conv
}  // namespace efla
