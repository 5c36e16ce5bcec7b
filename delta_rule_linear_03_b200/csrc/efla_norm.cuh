// efla_norm.cuh - root-mean-square norm of rows with the residual's addition
// and an optional 8-bit output with scales, and its backward pass.
//
//   h = x + res,  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd w,  res_out = h
//   8 bits: scale = max(max |y| / 448, 2^-126) over a group of 128 columns or
//   the row, y8 = e4m3(y / scale)
//   backward: u = w dy,  dh = rstd (u - h rstd^2 mean(u h)) + dres_out,
//             dw = sum over rows of dy h rstd
//
// HBM bound: a handful of flops an element.  A row stays in registers
// between the sum of its squares and its output, so each tensor crosses HBM
// once.  TPR threads, or a block, share a row with 16-byte accesses, IT of them
// each, and RPI rows are in flight a thread; the row's sums go through shuffles
// and, past a warp, one exchange in shared memory for all RPI rows.  h is
// the unrounded fp32 sum for the norm; res_out is its rounding.
//
// Measured, of a copy's 6.57 TB/s: 65536 x 2048, bf16 with residual to 8 bits
// 137 us (all of it; element by element in fp32 it took 272, bound by the ALUs,
// which now stand at 62%, hence paired operations and conversions); 131008
// x 128, fp32, 23.2 us (88%); 16384 x 2048 backward, bf16 with an fp32
// residual, 90.6 us (90%).  64 rows are a launch: 2.7 us.
#pragma once
#include <cuda_fp8.h>

#include "efla_vec.cuh"

namespace efla {
namespace norm {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: no scale is 0 or subnormal
constexpr int kGroup = 128;
constexpr int kMaxC = 16384;

// Threads of a block whose rows have TPR threads each; TPR < 0: the block is
// the row's, as large as the row needs, up to -TPR threads.
template <int TPR> constexpr int kThreadsOf = TPR < 0 ? -TPR : TPR > 256 ? TPR : 256;

// The larger magnitude; a NaN stays one.
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
    return r;
}

// Sums or maxima of V values over the TPR threads of a row.
template <int TPR, int V> struct RowReduce {
    static constexpr bool kWarps = TPR < 0 || TPR > 32;  // a row has several
    static constexpr int NW = kThreadsOf<TPR> / 32, LANES = kWarps ? 32 : TPR;
    float red[kWarps ? V : 1][kWarps ? NW : 1];

    template <typename F> __device__ __forceinline__ void reduce(float (&v)[V], F f) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = f(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
        if constexpr (kWarps) {
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) red[i][warp] = v[i];
            __syncthreads();
            if constexpr (TPR < 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = lane < blockDim.x / 32 ? red[i][lane] : 0.f;  // no more than NW
#pragma unroll
                for (int o = NW / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = f(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
            } else {
                const int w0 = warp / (TPR / 32) * (TPR / 32);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float s = red[i][w0];
#pragma unroll
                    for (int k = 1; k < TPR / 32; ++k) s = f(s, red[i][w0 + k]);
                    v[i] = s;
                }
            }
        }
    }
    __device__ __forceinline__ void sum(float (&v)[V]) {
        reduce(v, [](float a, float b) { return a + b; });
    }
    // largest of values that are magnitudes; a NaN stays one
    __device__ __forceinline__ void max_abs(float (&v)[V]) {
        reduce(v, [](float a, float b) { return norm::max_abs(a, b); });
    }
};

// 1 / sqrt(m): the approximate root's 2 ulp with one Newton step; 0 for an infinite m.
__device__ __forceinline__ float rstd_of(float m) {
    const float r = rsqrtf(m);
    return m < __int_as_float(0x7f800000) ? r * fmaf(-0.5f * m * r, r, 1.5f) : m != m ? m : 0.f;
}
// A group's scale from its largest |y|; a NaN stays one.
__device__ __forceinline__ float scale_of(float top) {
    const float a = top * (1.f / kE4m3Max);
    return a < kScaleMin ? kScaleMin : a;
}
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
template <int N> __device__ __forceinline__ void widen2(const float (&v)[N], f32x2 (&o)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) o[i] = pack2(v[2 * i], v[2 * i + 1]);
}
template <typename T, int N> __device__ __forceinline__ void widen2(const Raw<T, N> &r, f32x2 (&o)[N / 2]) {
    float v[N];
    widen<T, N>(r, v);
    widen2<N>(v, o);
}
template <typename T, int N> __device__ __forceinline__ Raw<T, N> narrow2(const f32x2 (&p)[N / 2]) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 t = unpack2(p[i]);
        v[2 * i] = t.x;
        v[2 * i + 1] = t.y;
    }
    return narrow<T, N>(v);
}

struct FwdArgs {
    const void *x, *res;
    const float *w;
    void *y, *res_out;
    unsigned char *y8;
    float *scale;
    float eps, inv_c;  // inv_c = 1 / C
    int group;  // columns of one scale: 128, or 0 for the row
    int C;
    long long rows;
};

// VEC columns from c on; ANY: those of them that are columns of the row, each
// vector aligned although the row is not.
template <bool ANY, typename T, int VEC> __device__ __forceinline__ Raw<T, VEC> load_cols(const T *row, int c, int C, bool on) {
    if constexpr (ANY) {
        Raw<T, VEC> r = zero_raw<T, VEC>();
        if (on && c >= 0 && c + VEC <= C) return load_raw<T, VEC>(row + c);
        if (on && c < C)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (c + j >= 0 && c + j < C) r.e[j] = row[c + j];
        return r;
    } else {
        return on && c < C ? load_raw<T, VEC>(row + c) : zero_raw<T, VEC>();
    }
}
template <bool ANY, typename T, int VEC>
__device__ __forceinline__ void store_cols(T *row, int c, int C, bool on, const Raw<T, VEC> &r) {
    if (!on || c >= C) return;
    if (!ANY || (c >= 0 && c + VEC <= C)) {
        store_raw<T, VEC>(row + c, r);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (c + j >= 0 && c + j < C) row[c + j] = r.e[j];
    }
}

// Rows in 16-byte vectors.  ANY: the width is no multiple of them, so a row's
// vectors begin at the 16-byte boundary before it, and one vector of a group of
// 128 columns begins in the group before; the groups' maxima meet in shared
// memory.  Element by element instead, as norm_fwd_any_kernel has it, 33520 x
// 1001 took 259 us in fp32 (82 with vectors) and 166 in bf16 (98); up to 128
// columns, with two cut vectors in every few, it is the faster (74 against 159).
template <typename T, typename R, int TPR, int IT, int RPI, bool ANY>
__global__ void __launch_bounds__(kThreadsOf<TPR>) norm_fwd_kernel(FwdArgs a) {
    constexpr int VEC = 16 / sizeof(T), SLOTS = TPR > 0 ? kThreadsOf<TPR> / TPR : 1;
    constexpr int LPG = TPR > 0 && kGroup / VEC > TPR ? TPR : kGroup / VEC;  // lanes of one group of 128 columns
    const int tpr = TPR > 0 ? TPR : blockDim.x;
    __shared__ RowReduce<TPR, RPI> rs, rm;
    const int slot = TPR > 0 ? threadIdx.x / tpr : 0, l = TPR > 0 ? threadIdx.x % tpr : threadIdx.x, C = a.C;
    const long long row0 = (long long)blockIdx.x * (SLOTS * RPI) + slot;
    const T *x = static_cast<const T *>(a.x);
    const R *res = static_cast<const R *>(a.res);
    const int off = ANY ? (int)(row0 * C & (VEC - 1)) : 0;
    static_assert(!ANY || RPI == 1, "one row, one offset");
    constexpr int NG = ANY ? (TPR > 0 ? TPR : -TPR) * IT * VEC / kGroup + 2 : 1;
    __shared__ int gmax[ANY ? SLOTS : 1][NG];  // maxima as bits, whose order is the values'; a NaN is the largest
    if (ANY) {
        for (int g = threadIdx.x; g < SLOTS * NG; g += blockDim.x) (&gmax[0][0])[g] = 0;
        __syncthreads();
    }
    const auto col = [&](int k) { return (k * tpr + l) * VEC - off; };

    Raw<T, VEC> xr[RPI][IT];
    Raw<R, VEC> rr[RPI][IT];
#pragma unroll
    for (int i = 0; i < RPI; ++i)
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const long long row = row0 + i * SLOTS;
            xr[i][k] = load_cols<ANY, T, VEC>(x + row * C, col(k), C, row < a.rows);
            if (res) rr[i][k] = load_cols<ANY, R, VEC>(res + row * C, col(k), C, row < a.rows);
        }
    f32x2 h[RPI][IT][VEC / 2];
    float ss[RPI];
#pragma unroll
    for (int i = 0; i < RPI; ++i) {
        f32x2 s2 = 0ull;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            widen2<T, VEC>(xr[i][k], h[i][k]);
            if (res) {
                f32x2 r[VEC / 2];
                widen2<R, VEC>(rr[i][k], r);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) h[i][k][j] = add2(h[i][k][j], r[j]);
            }
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) s2 = fma2(h[i][k][j], h[i][k][j], s2);
        }
        ss[i] = sum2(s2);
    }
    f32x2 w[IT][VEC / 2];
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int c = col(k);
        if constexpr (ANY) {
            Raw<float, VEC> r;
#pragma unroll
            for (int j = 0; j < VEC; ++j) r.e[j] = a.w[min(max(c + j, 0), C - 1)];
            // 0 outside the row: an infinite weight at its end would make NaN of the zeros there, and of a scale.  In a
            // branch of its own, for few vectors: selected at every load, 8190 x 4097 in bf16 to 8 bits takes 147 us, so 110.
            if (a.y8 && (c < 0 || c + VEC > C))
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (c + j < 0 || c + j >= C) r.e[j] = 0.f;
            widen2<float, VEC>(r, w[k]);
        } else {
            widen2<float, VEC>(c < C ? load_raw<float, VEC>(a.w + c) : zero_raw<float, VEC>(), w[k]);
        }
    }
    rs.sum(ss);
    // columns outside the row hold zeros, their weights too, so that they add nothing to a maximum
    // (the product with an infinite or absent root is kept out where a vector has no column)
    float top[RPI];
#pragma unroll
    for (int i = 0; i < RPI; ++i) {
        const long long row = row0 + i * SLOTS;
        const float rstd = rstd_of(fmaf(ss[i], a.inv_c, a.eps));
        top[i] = 0.f;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = col(k);
            const bool in = row < a.rows && c < C;
            if (a.res_out) store_cols<ANY, R, VEC>(static_cast<R *>(a.res_out) + row * C, c, C, in, narrow2<R, VEC>(h[i][k]));
            const f32x2 r2 = in ? pack2(rstd, rstd) : 0ull;
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) h[i][k][j] = mul2(mul2(h[i][k][j], r2), w[k][j]);
            if (a.y) store_cols<ANY, T, VEC>(static_cast<T *>(a.y) + row * C, c, C, in, narrow2<T, VEC>(h[i][k]));
        }
    }
    if (!a.y8) return;
    if (!a.group) {
#pragma unroll
        for (int i = 0; i < RPI; ++i)
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const float2 t = unpack2(h[i][k][j]);
                    top[i] = max_abs(max_abs(top[i], t.x), t.y);
                }
        rm.max_abs(top);
    }
    const int ng = a.group ? (C + kGroup - 1) / kGroup : 1;
    if (ANY && a.group) {
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int v0 = col(k) + off, g = v0 / kGroup, cut = v0 % kGroup ? 0 : off;  // columns before `cut` are group g - 1's
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                const float2 t = unpack2(h[0][k][j]);
                if (2 * j < cut) lo = max_abs(lo, t.x); else hi = max_abs(hi, t.x);
                if (2 * j + 1 < cut) lo = max_abs(lo, t.y); else hi = max_abs(hi, t.y);
            }
#pragma unroll
            for (int o = LPG / 2; o > 0; o >>= 1) hi = max_abs(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            if (l % LPG == 0) atomicMax(&gmax[slot][g], __float_as_int(hi));
            if (cut && g > 0) atomicMax(&gmax[slot][g - 1], __float_as_int(lo));
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < RPI; ++i) {
        const long long row = row0 + i * SLOTS;
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = col(k);
            float m = top[i];
            const int g = (c + off) / kGroup, cut = ANY && a.group && (c + off) % kGroup == 0 ? off : 0;
            if (ANY && a.group) {
                m = __int_as_float(gmax[slot][g]);
            } else if (a.group) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const float2 t = unpack2(h[i][k][j]);
                    m = max_abs(max_abs(m, t.x), t.y);
                }
#pragma unroll
                for (int o = LPG / 2; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            const float s = scale_of(m), inv = rcp(s);
            if (row >= a.rows || c >= C) continue;
            if (a.group ? l % LPG == 0 && g < ng : l == 0 && k == 0) a.scale[row * ng + (a.group ? g : 0)] = s;
            const float low = cut && g > 0 ? rcp(scale_of(__int_as_float(gmax[slot][g - 1]))) : inv;
            uint16_t q[VEC / 2];
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                const float2 t = unpack2(mul2(h[i][k][j], ANY ? pack2(2 * j < cut ? low : inv, 2 * j + 1 < cut ? low : inv) : pack2(inv, inv)));
                q[j] = e4m3x2(t.x, t.y);
            }
            unsigned char *p = a.y8 + row * C + c;
            if constexpr (ANY) {
                if (c < 0 || c + VEC > C) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (c + j >= 0 && c + j < C) p[j] = (unsigned char)(q[j / 2] >> (j % 2 * 8));
                    continue;
                }
            }
            if constexpr (VEC == 8)
                *reinterpret_cast<uint2 *>(p) =
                    make_uint2(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16);
            else
                *reinterpret_cast<uint32_t *>(p) = q[0] | (uint32_t)q[1] << 16;
        }
    }
}

// Few columns, or a width that the vectors of norm_fwd_kernel do not reach:
// WPR warps share a row, each takes whole groups of 128 columns,
// IT of them, four single elements a lane, so that a group's maximum stays
// within one warp.
template <typename T, typename R, int WPR, int IT>
__global__ void __launch_bounds__(kThreadsOf<WPR * 32>) norm_fwd_any_kernel(FwdArgs a) {
    constexpr int TPR = WPR * 32, SLOTS = kThreadsOf<TPR> / TPR;
    __shared__ RowReduce<TPR, 1> rs, rm;
    const int slot = threadIdx.x / TPR, wr = threadIdx.x % TPR / 32, lane = threadIdx.x & 31, C = a.C;
    const long long row = (long long)blockIdx.x * SLOTS + slot;
    const bool on = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + row * C;
    const R *res = a.res ? static_cast<const R *>(a.res) + row * C : nullptr;
    // all loads before the first store: one behind a store would wait for it, as far as the compiler can tell
    float h[IT][4], w[IT][4], ss[1] = {0.f};
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
            h[k][j] = on && c < C ? to_f32(x[c]) : 0.f;
            w[k][j] = c < C ? a.w[c] : 0.f;
        }
    if (res)
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
                if (on && c < C) h[k][j] += to_f32(res[c]);
            }
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) ss[0] = fmaf(h[k][j], h[k][j], ss[0]);
    rs.sum(ss);
    const float rstd = rstd_of(fmaf(ss[0], a.inv_c, a.eps));
    float top[1] = {0.f};
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
            if (!on || c >= C) {
                h[k][j] = 0.f;
                continue;
            }
            if (a.res_out) static_cast<R *>(a.res_out)[row * C + c] = from_f32<R>(h[k][j]);
            h[k][j] = h[k][j] * rstd * w[k][j];
            if (a.y) static_cast<T *>(a.y)[row * C + c] = from_f32<T>(h[k][j]);
            top[0] = max_abs(top[0], h[k][j]);
        }
    if (!a.y8) return;
    if (!a.group) rm.max_abs(top);
    const int ng = a.group ? (C + kGroup - 1) / kGroup : 1;
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        float m = top[0];
        if (a.group) {
            m = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max_abs(m, h[k][j]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        const float s = scale_of(m), inv = rcp(s);
        const int g = k * WPR + wr;
        if (!on || g * kGroup >= C) continue;
        if (lane == 0 && (a.group || g == 0)) a.scale[row * ng + (a.group ? g : 0)] = s;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = g * kGroup + j * 32 + lane;
            if (c < C) a.y8[row * C + c] = (unsigned char)(e4m3x2(h[k][j] * inv, 0.f) & 0xffu);
        }
    }
}

struct BwdArgs {
    const void *dy, *h, *dres_out;
    const float *w;
    void *dx, *dres;  // dx in the type of dy, dres in the type of h; either may be NULL
    float *part;      // [blocks][C]
    float eps, inv_c;
    int C;
    long long rows;
};

// A persistent block keeps its columns' share of dw in registers over all of
// its rows; the shares of its row slots meet in shared memory at the end.  Two
// blocks an SM, so that one's loads cover the other's sums (57% of a warp's
// wait is for loads, 20% for its block): one of 255 registers took 93 us where
// two of 128 take 91 (16384 x 2048), in fp32 with rows in pairs 122 against 88.
template <typename T, typename R, int TPR, int IT, int RPI>
__global__ void __launch_bounds__(kThreadsOf<TPR>, TPR <= 256 ? 2 : 1) norm_bwd_kernel(BwdArgs a) {
    constexpr int VEC = 16 / sizeof(T), NT = kThreadsOf<TPR>, SLOTS = NT / TPR;
    __shared__ RowReduce<TPR, 2 * RPI> rs[2];
    __shared__ float cols[SLOTS > 1 ? SLOTS : 1][SLOTS > 1 ? TPR * IT * VEC : 1];
    const int slot = threadIdx.x / TPR, l = threadIdx.x % TPR, C = a.C;
    const T *dy = static_cast<const T *>(a.dy);
    const R *h = static_cast<const R *>(a.h), *dr = static_cast<const R *>(a.dres_out);
    float w[IT][VEC], acc[IT][VEC];
#pragma unroll
    for (int k = 0; k < IT; ++k) {
        const int c = (k * TPR + l) * VEC;
        widen<float, VEC>(c < C ? load_raw<float, VEC>(a.w + c) : zero_raw<float, VEC>(), w[k]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[k][j] = 0.f;
    }
    int par = 0;
    for (long long base = (long long)blockIdx.x * (SLOTS * RPI); base < a.rows;
         base += (long long)gridDim.x * (SLOTS * RPI), par ^= 1) {
        Raw<T, VEC> yr[RPI][IT];
        Raw<R, VEC> hr[RPI][IT], rr[RPI][IT];
#pragma unroll
        for (int i = 0; i < RPI; ++i)
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const long long row = base + i * SLOTS + slot;
                const int c = (k * TPR + l) * VEC;
                const bool in = row < a.rows && c < C;
                yr[i][k] = in ? load_raw<T, VEC>(dy + row * C + c) : zero_raw<T, VEC>();
                hr[i][k] = in ? load_raw<R, VEC>(h + row * C + c) : zero_raw<R, VEC>();
                rr[i][k] = in && dr ? load_raw<R, VEC>(dr + row * C + c) : zero_raw<R, VEC>();
            }
        float s[2 * RPI];  // sum h^2, sum u h
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            s[2 * i] = s[2 * i + 1] = 0.f;
#pragma unroll
            for (int k = 0; k < IT; ++k)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float hv = to_f32(hr[i][k].e[j]);
                    s[2 * i] = fmaf(hv, hv, s[2 * i]);
                    s[2 * i + 1] = fmaf(to_f32(yr[i][k].e[j]) * w[k][j], hv, s[2 * i + 1]);
                }
        }
        rs[par].sum(s);
#pragma unroll
        for (int i = 0; i < RPI; ++i) {
            const long long row = base + i * SLOTS + slot;
            const float rstd = rstd_of(fmaf(s[2 * i], a.inv_c, a.eps));
            const float m = rstd * (rstd * (s[2 * i + 1] * a.inv_c));  // the square alone may overflow
#pragma unroll
            for (int k = 0; k < IT; ++k) {
                const int c = (k * TPR + l) * VEC;
                if (row >= a.rows || c >= C) continue;
                float d[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float hv = to_f32(hr[i][k].e[j]), yv = to_f32(yr[i][k].e[j]);
                    acc[k][j] = fmaf(yv, hv * rstd, acc[k][j]);
                    d[j] = fmaf(rstd, yv * w[k][j] - hv * m, to_f32(rr[i][k].e[j]));
                }
                if (a.dx) store_raw<T, VEC>(static_cast<T *>(a.dx) + row * C + c, narrow<T, VEC>(d));
                if (a.dres) store_raw<R, VEC>(static_cast<R *>(a.dres) + row * C + c, narrow<R, VEC>(d));
            }
        }
    }
    float *part = a.part + (long long)blockIdx.x * C;
    if constexpr (SLOTS > 1) {
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) cols[slot][(k * TPR + l) * VEC + j] = acc[k][j];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += NT) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) t += cols[i][c];
            part[c] = t;
        }
    } else {
#pragma unroll
        for (int k = 0; k < IT; ++k) {
            const int c = (k * TPR + l) * VEC;
            if (c < C) store_raw<float, VEC>(part + c, narrow<float, VEC>(acc[k]));
        }
    }
}

// Any width, as norm_fwd_any_kernel lays rows out.
template <typename T, typename R, int WPR, int IT>
__global__ void __launch_bounds__(kThreadsOf<WPR * 32>, WPR <= 8 ? 2 : 1) norm_bwd_any_kernel(BwdArgs a) {
    constexpr int TPR = WPR * 32, NT = kThreadsOf<TPR>, SLOTS = NT / TPR;
    __shared__ RowReduce<TPR, 2> rs[2];
    __shared__ float cols[SLOTS > 1 ? SLOTS : 1][SLOTS > 1 ? WPR * IT * kGroup : 1];
    const int slot = threadIdx.x / TPR, wr = threadIdx.x % TPR / 32, lane = threadIdx.x & 31, C = a.C;
    const T *dy = static_cast<const T *>(a.dy);
    const R *h = static_cast<const R *>(a.h), *dr = static_cast<const R *>(a.dres_out);
    float w[IT][4], acc[IT][4];
#pragma unroll
    for (int k = 0; k < IT; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
            w[k][j] = c < C ? a.w[c] : 0.f;
            acc[k][j] = 0.f;
        }
    int par = 0;
    for (long long base = (long long)blockIdx.x * SLOTS; base < a.rows; base += (long long)gridDim.x * SLOTS, par ^= 1) {
        const long long row = base + slot;
        const bool on = row < a.rows;
        float hv[IT][4], yv[IT][4], rv[IT][4], s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
                const bool in = on && c < C;
                hv[k][j] = in ? to_f32(h[row * C + c]) : 0.f;
                yv[k][j] = in ? to_f32(dy[row * C + c]) : 0.f;
                rv[k][j] = in && dr ? to_f32(dr[row * C + c]) : 0.f;
            }
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[0] = fmaf(hv[k][j], hv[k][j], s[0]);
                s[1] = fmaf(yv[k][j] * w[k][j], hv[k][j], s[1]);
            }
        rs[par].sum(s);
        const float rstd = rstd_of(fmaf(s[0], a.inv_c, a.eps));
        const float m = rstd * (rstd * (s[1] * a.inv_c));
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
                if (!on || c >= C) continue;
                acc[k][j] = fmaf(yv[k][j], hv[k][j] * rstd, acc[k][j]);
                const float d = fmaf(rstd, yv[k][j] * w[k][j] - hv[k][j] * m, rv[k][j]);
                if (a.dx) static_cast<T *>(a.dx)[row * C + c] = from_f32<T>(d);
                if (a.dres) static_cast<R *>(a.dres)[row * C + c] = from_f32<R>(d);
            }
    }
    float *part = a.part + (long long)blockIdx.x * C;
    if constexpr (SLOTS > 1) {
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) cols[slot][(k * WPR + wr) * kGroup + j * 32 + lane] = acc[k][j];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += NT) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) t += cols[i][c];
            part[c] = t;
        }
    } else {
#pragma unroll
        for (int k = 0; k < IT; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = (k * WPR + wr) * kGroup + j * 32 + lane;
                if (c < C) part[c] = acc[k][j];
            }
    }
}

}  // namespace norm
}  // namespace efla
