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
// Bound by HBM and by the special function units nearly alike: the SiLU's
// exponential and reciprocal are two of their 16 results a clock and SM, 15 us
// for 4 x 4096 x 2048 elements whose bytes in bf16 take 20.5, and the schedulers
// have some 14 instructions an element of which sum, SiLU and conversions are
// 10.  So elements are worked on in pairs, and runs of tokens that lie wholly inside their sequence have
// no conditions in them.  A thread owns VEC neighbouring channels and walks a run
// of tokens with the last K-1 inputs in registers, kAhead rows on their way
// while as many are worked on; x is read once but for the K-1 rows where a
// run begins (those lie in the L1 or L2 of the run before).  Four runs make a
// block; 32 lanes side by side cover 32 VEC channels.  y may go to
// [B][H][L][d] directly, the layout the mixer reads.
//
// Measured: 4 x 4096 x 2048, bf16, K = 4, 29.7 us (48 with one channel a thread's
// operation, 129 one element at a time); 8 x 2047 x 1001 backward, fp32, odd
// rows, random lengths, 38 to 41 us (all its bytes 30); one token of 64 x 2048 2.3
// us, a launch.
#pragma once
#include "efla_vec.cuh"

namespace efla {
namespace conv {

constexpr int kWarps = 4;
constexpr int kAhead = 8;
constexpr int kShortRun = 8, kLongRun = 256, kLongFwdRun = 128;  // tokens of one thread's run; multiples of kAhead

struct Args {
    const void *x;
    long long ldx;  // elements from one token's row of x to the next
    const float *w, *bias;
    const void *state;
    const int *lengths;
    int silu, head;  // head: channels of a head where y (or dy) is [B][H][L][head], 0 where it is [B][L][C]
    int B, L, C, run, tiles;
    // forward
    void *y, *state_out;
    // backward
    const void *dy, *dstate_out;
    void *dx, *dstate;
    float *part;  // [B * tiles] rows of dw [C][K], dbias [C]
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

// VEC channels' values: pairs, or one float.
template <int VEC> struct Vals {
    static constexpr int NE = VEC / 2;
    f32x2 v[NE];
};
template <> struct Vals<1> {
    static constexpr int NE = 1;
    float v[1];
};
__device__ __forceinline__ float mad(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f32x2 mad(f32x2 a, f32x2 b, f32x2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float times(float a, float b) { return a * b; }
__device__ __forceinline__ f32x2 times(f32x2 a, f32x2 b) { return mul2(a, b); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ f32x2 plus(f32x2 a, f32x2 b) { return add2(a, b); }
__device__ __forceinline__ float silu_of(float v) { return silu_f32(v); }
__device__ __forceinline__ f32x2 silu_of(f32x2 v) { return silu_2(v); }
__device__ __forceinline__ float dsilu_of(float v) { return dsilu_f32(v); }
__device__ __forceinline__ f32x2 dsilu_of(f32x2 v) { return dsilu_2(v); }

template <int VEC> __device__ __forceinline__ Vals<VEC> vals_of(const float (&f)[VEC]) {
    Vals<VEC> r;
    if constexpr (VEC == 1) r.v[0] = f[0];
    else
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) r.v[i] = pack2(f[2 * i], f[2 * i + 1]);
    return r;
}
template <int VEC> __device__ __forceinline__ void floats_of(const Vals<VEC> &x, float (&f)[VEC]) {
    if constexpr (VEC == 1) f[0] = x.v[0];
    else
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 t = unpack2(x.v[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
}
template <typename T, int VEC> __device__ __forceinline__ Vals<VEC> vals(const Raw<T, VEC> &r) {
    float f[VEC];
    widen<T, VEC>(r, f);
    return vals_of<VEC>(f);
}
template <typename T, int VEC> __device__ __forceinline__ Raw<T, VEC> raw(const Vals<VEC> &x) {
    float f[VEC];
    floats_of<VEC>(x, f);
    return narrow<T, VEC>(f);
}
template <int VEC> __device__ __forceinline__ Vals<VEC> none() { return vals<float, VEC>(zero_raw<float, VEC>()); }

// Filters w[j] of VEC channels from channel c on, and their bias.
template <int K, int VEC>
__device__ __forceinline__ void load_filters(const Args &a, int c, Vals<VEC> (&w)[K], Vals<VEC> &bias) {
    float v[VEC * K], f[VEC];
    const float *p = a.w + (long long)c * K;
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
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = v[i * K + j];
        w[j] = vals_of<VEC>(f);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = a.bias ? a.bias[c + i] : 0.f;
    bias = vals_of<VEC>(f);
}

// The K-1 inputs before token t0 (t0 = 0: the state's).
template <typename T, int K, int VEC>
__device__ __forceinline__ void load_window(const Args &a, const T *x, const T *st, int t0, int len, Vals<VEC> *win) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int t = t0 - (K - 1) + j;
        Raw<T, VEC> r = zero_raw<T, VEC>();
        if (t >= 0) {
            if (t < len) r = load_raw<T, VEC>(x + t * a.ldx);
        } else if (st) {
            r = load_raw<T, VEC>(st + (long long)(t + K - 1) * a.C);
        }
        win[j] = vals<T, VEC>(r);
    }
}

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

template <typename T, int K, int VEC>
__global__ void __launch_bounds__(32 * kWarps) conv_fwd_kernel(Args a) {
    constexpr int U = kAhead, NE = Vals<VEC>::NE;
    const int b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int c = (blockIdx.y * 32 + (threadIdx.x & 31)) * VEC, warp = threadIdx.x >> 5;
    const int t0 = (tile * kWarps + warp) * a.run;
    if (c >= a.C || (t0 >= a.L && t0 > 0)) return;
    const int len = length_of(a, b);
    const T *x = static_cast<const T *>(a.x) + (long long)b * a.L * a.ldx + c;
    const T *st = a.state ? static_cast<const T *>(a.state) + (long long)b * (K - 1) * a.C + c : nullptr;
    const long long ldy = a.head ? a.head : a.C;
    if (t0 >= len && t0 > 0) {  // padding alone
        T *y = static_cast<T *>(a.y) + out_at(a, b, t0, c);
        for (int t = t0; t < min(t0 + a.run, a.L); ++t, y += ldy) store_raw<T, VEC>(y, zero_raw<T, VEC>());
        return;
    }

    Vals<VEC> w[K], bias, win[K - 1 + U];  // win: the K-1 inputs before a batch, and the batch
    load_filters<K, VEC>(a, c, w, bias);
    load_window<T, K, VEC>(a, x, st, t0, len, win);
    const int t1 = min(t0 + a.run, a.L), tl = min(t1, len);
    const auto walk = [&](auto whole) {  // whole: every token of the run counts
        constexpr bool kWhole = decltype(whole)::value;
        const T *in = x + t0 * a.ldx;
        T *y = static_cast<T *>(a.y) + out_at(a, b, t0, c);
        Raw<T, VEC> next[U];
        const auto load = [&](int t) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (kWhole || t + u < tl) next[u] = load_raw<T, VEC>(in + u * a.ldx);
                else next[u] = zero_raw<T, VEC>();
            }
            in += U * a.ldx;
        };
        load(t0);
        for (int t = t0; t < t1; t += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) win[K - 1 + u] = vals<T, VEC>(next[u]);
            if (!kWhole || t + U < t1) load(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!kWhole && t + u >= t1) break;
                Vals<VEC> o = bias;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
#pragma unroll
                    for (int j = 0; j < K; ++j) o.v[i] = mad(w[j].v[i], win[u + j].v[i], o.v[i]);
                    if (a.silu) o.v[i] = silu_of(o.v[i]);
                }
                if (!kWhole && t + u >= len) o = none<VEC>();
                store_raw<T, VEC>(y, raw<T, VEC>(o));
                y += ldy;
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) win[j] = win[j + U];
        }
    };
    if (t0 + a.run <= len) walk(Yes{});
    else walk(No{});

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
// which its last dx need; dw and dbias count its own tokens alone.  The runs
// of a block add theirs up in shared memory and the block writes one partial
// row, which colsum_kernel adds in a fixed order.  Four blocks an SM, five of
// single channels: with three, of 142 registers, 4 x 4096 x 2048 in fp32 takes 97
// us, not 72, and with four of single channels 8 x 4096 x 1001 105, not 95.
template <typename T, int K, int VEC>
__global__ void __launch_bounds__(32 * kWarps, VEC == 1 ? 5 : 4) conv_bwd_kernel(Args a) {
    constexpr int U = kAhead, NE = Vals<VEC>::NE;
    __shared__ float red[kWarps][32 * VEC * (K + 1)];
    const int b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const int t0 = (tile * kWarps + warp) * a.run;
    Vals<VEC> dw[K], db = none<VEC>();
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j] = none<VEC>();
    const int len = length_of(a, b);
    if (c < a.C && t0 >= len && t0 > 0) {  // padding alone
        T *dx = static_cast<T *>(a.dx) + ((long long)b * a.L + t0) * a.C + c;
        for (int t = t0; t < min(t0 + a.run, a.L); ++t, dx += a.C) store_raw<T, VEC>(dx, zero_raw<T, VEC>());
    } else if (c < a.C) {
        const T *x = static_cast<const T *>(a.x) + (long long)b * a.L * a.ldx + c;
        const T *st = a.state ? static_cast<const T *>(a.state) + (long long)b * (K - 1) * a.C + c : nullptr;
        const T *dso = a.dstate_out ? static_cast<const T *>(a.dstate_out) + (long long)b * (K - 1) * a.C + c : nullptr;
        T *ds = a.dstate ? static_cast<T *>(a.dstate) + (long long)b * (K - 1) * a.C + c : nullptr;
        const long long ldy = a.head ? a.head : a.C;

        Vals<VEC> w[K], bias, win[K - 1 + U], d[K - 1 + U];  // the K-1 before a batch, and the batch
        load_filters<K, VEC>(a, c, w, bias);
        load_window<T, K, VEC>(a, x, st, t0, len, win);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) d[j] = none<VEC>();
        const int tl = min(t0 + a.run + K - 1, len);
        const T *in = x + t0 * a.ldx, *dy = static_cast<const T *>(a.dy) + out_at(a, b, t0, c);
        T *dx = static_cast<T *>(a.dx) + ((long long)b * a.L + t0 - (K - 1)) * a.C + c;  // of token t - (K-1)
        Raw<T, VEC> nx[U], ny[U];
        // inside: every token of the batch counts, every dx that it completes is the run's own and gets nothing else
        const auto load = [&](int t, auto inside) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (decltype(inside)::value || t + u < tl) {
                    nx[u] = load_raw<T, VEC>(in + u * a.ldx);
                    ny[u] = load_raw<T, VEC>(dy + u * ldy);
                } else {
                    nx[u] = zero_raw<T, VEC>();
                    ny[u] = zero_raw<T, VEC>();
                }
            }
            in += U * a.ldx;
            dy += U * ldy;
        };
        const auto batch = [&](int t, auto inside) {
            constexpr bool kInside = decltype(inside)::value;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                win[K - 1 + u] = vals<T, VEC>(nx[u]);
                d[K - 1 + u] = vals<T, VEC>(ny[u]);
            }
            if (t + U < t0 + a.run + K - 1) {
                if (t + 2 * U <= tl) load(t + U, Yes{});
                else load(t + U, No{});
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u, to = tt - (K - 1);  // to: the token whose dx is complete now
                Vals<VEC> &dn = d[K - 1 + u];
                if (a.silu) {
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        auto s = bias.v[i];
#pragma unroll
                        for (int j = 0; j < K; ++j) s = mad(w[j].v[i], win[u + j].v[i], s);
                        dn.v[i] = times(dn.v[i], dsilu_of(s));
                    }
                }
                if (!kInside && tt >= len) dn = none<VEC>();
                if (kInside || tt < t0 + a.run)
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        db.v[i] = plus(db.v[i], dn.v[i]);
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j].v[i] = mad(dn.v[i], win[u + j].v[i], dw[j].v[i]);
                    }
                Vals<VEC> o;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    o.v[i] = times(w[K - 1].v[i], d[u].v[i]);
#pragma unroll
                    for (int j = 1; j < K; ++j) o.v[i] = mad(w[K - 1 - j].v[i], d[u + j].v[i], o.v[i]);
                }
                if (kInside) {
                    store_raw<T, VEC>(dx, raw<T, VEC>(o));
                } else if (to < a.L && to < t0 + a.run && (to >= t0 || (to < 0 && t0 == 0))) {
                    const int at = to - len + K - 1;  // the row of state_out that holds x_to
                    if (dso && at >= 0 && at < K - 1) {
                        const Vals<VEC> g = vals<T, VEC>(load_raw<T, VEC>(dso + (long long)at * a.C));
#pragma unroll
                        for (int i = 0; i < NE; ++i) o.v[i] = plus(o.v[i], g.v[i]);
                    }
                    if (to >= 0) store_raw<T, VEC>(dx, raw<T, VEC>(o));
                    else if (ds) store_raw<T, VEC>(ds + (long long)(to + K - 1) * a.C, raw<T, VEC>(o));
                }
                dx += a.C;
            }
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                win[j] = win[j + U];
                d[j] = d[j + U];
            }
        };
        load(t0, No{});
        for (int t = t0; t < t0 + a.run + K - 1; t += U) {
            if (t >= a.L + K - 1) break;  // no token's dx is left
            // the first batch completes tokens before the run, the last those behind it; state_out's rows end at len
            if (t >= t0 + K - 1 && t + U <= t0 + a.run && t + U <= len - (K - 1)) batch(t, Yes{});
            else batch(t, No{});
        }
    }
    float f[VEC], *mine = &red[warp][0];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        floats_of<VEC>(dw[j], f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) mine[(lane * VEC + i) * K + j] = f[i];
    }
    floats_of<VEC>(db, f);
#pragma unroll
    for (int i = 0; i < VEC; ++i) mine[32 * VEC * K + lane * VEC + i] = f[i];
    __syncthreads();
    const int c0 = blockIdx.y * 32 * VEC, n = min(32 * VEC, a.C - c0);
    float *part = a.part + (long long)blockIdx.x * a.C * (K + 1);
    for (int i = threadIdx.x; i < 32 * VEC * (K + 1); i += 32 * kWarps) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += red[k][i];
        if (i < 32 * VEC * K) {
            if (i < n * K) part[(long long)c0 * K + i] = s;
        } else if (i - 32 * VEC * K < n) {
            part[(long long)a.C * K + c0 + i - 32 * VEC * K] = s;
        }
    }
}

// One token: y from the state and x, then the state moved up by one.  A
// thread owns its channels' state, so the update is in place.  The sum is
// taken as the forward kernel takes it, so that tokens one by one give the
// same bits as a prompt.
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
