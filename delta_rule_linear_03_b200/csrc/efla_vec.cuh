// efla_vec.cuh - loads and stores of N consecutive elements, widened to and
// rounded from fp32, for the kernels whose rows may be strided, odd or not
// aligned for 16-byte accesses.
#pragma once
#include <string.h>

#include "efla_common.cuh"

namespace efla {

// N elements of T as they lie in memory, in registers: a load kept in this
// form can be issued long before its use.
template <typename T, int N> struct alignas(N * sizeof(T) > 16 ? 16 : N * sizeof(T)) Raw { T e[N]; };

// One access of min(16, N * sizeof(T)) bytes each; p must be aligned to that.
template <typename T, int N> __device__ __forceinline__ Raw<T, N> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, N> *>(p);
}
template <typename T, int N> __device__ __forceinline__ Raw<T, N> zero_raw() {
    Raw<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = from_f32<T>(0.f);
    return r;
}
// bf16 is widened and rounded by pairs: one shift or mask, and half a
// conversion, an element.
template <typename T, int N> __device__ __forceinline__ void widen(const Raw<T, N> &r, float (&v)[N]) {
    if constexpr (sizeof(T) == 2 && N % 2 == 0) {
        uint32_t u[N / 2];
        memcpy(u, r.e, sizeof(u));
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = to_f32(r.e[i]);
    }
}
template <typename T, int N> __device__ __forceinline__ Raw<T, N> narrow(const float (&v)[N]) {
    Raw<T, N> r;
    if constexpr (sizeof(T) == 2 && N % 2 == 0) {
        __nv_bfloat162 p[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        memcpy(r.e, p, sizeof(p));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.e[i] = from_f32<T>(v[i]);
    }
    return r;
}
template <typename T, int N> __device__ __forceinline__ void store_raw(T *p, const Raw<T, N> &r) {
    *reinterpret_cast<Raw<T, N> *>(p) = r;
}
constexpr float kLog2e = 1.44269504088896340736f;

// 2^v and 1 / v, approximate (2 and 1 ulp); subnormals count as zeros.
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + e^-v) and v / (1 + e^-v); where e^-v overflows they are 0 and -0.
__device__ __forceinline__ float sigmoid_f32(float v) { return rcp(1.f + ex2(-kLog2e * v)); }
__device__ __forceinline__ float silu_f32(float v) { return v * sigmoid_f32(v); }
// d silu(v) / dv = s + s v (1 - s), s = sigmoid(v); 1 - s loses what is under
// 2^-24 of 1, which v makes no more than |v| such steps of the result.
__device__ __forceinline__ float dsilu_f32(float v) {
    const float s = sigmoid_f32(v);
    return fmaf(s, fmaf(-v, s, v), s);
}

// Two fp32 operations in one instruction, on a register pair.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
    const float2 t = unpack2(v);
    return t.x + t.y;
}

__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
    const float2 t = unpack2(v);
    return pack2(ex2(t.x), ex2(t.y));
}
__device__ __forceinline__ f32x2 rcp_2(f32x2 v) {
    const float2 t = unpack2(v);
    return pack2(rcp(t.x), rcp(t.y));
}
__device__ __forceinline__ f32x2 twice(float v) { return pack2(v, v); }
__device__ __forceinline__ f32x2 sigmoid_2(f32x2 v) { return rcp_2(add2(twice(1.f), ex2_2(mul2(v, twice(-kLog2e))))); }
__device__ __forceinline__ f32x2 silu_2(f32x2 v) { return mul2(v, sigmoid_2(v)); }
__device__ __forceinline__ f32x2 dsilu_2(f32x2 v) {
    const f32x2 s = sigmoid_2(v);
    return fma2(s, fma2(mul2(v, twice(-1.f)), s, v), s);
}

// Column sums of partial results, in a fixed order: out[i] = sum_p part[p][i].
// The columns may be spread over up to three outputs.  One block of 32 x 32
// threads per 32 columns; row group r adds rows r, r + 32, ...
struct ColsumOut {
    float *out[3];
    long long end[3];  // columns before end[i] (and from end[i-1] on) belong to out[i], which may be NULL
};
static __global__ void __launch_bounds__(1024) colsum_kernel(const float *__restrict__ part, ColsumOut o, long long M,
                                                             int P) {
    __shared__ float red[32][33];
    const int x = threadIdx.x & 31, r = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + x;
    float s = 0.f;
    if (i < M) {
        const float *p = part + i;
#pragma unroll 4
        for (int k = r; k < P; k += 32) s += p[(long long)k * M];
    }
    red[r][x] = s;
    __syncthreads();
    const float t = warp_sum(red[x][r]);  // warp r: column r of the block, one row group a lane
    const long long col = (long long)blockIdx.x * 32 + r;
    if (x == 0 && col < M) {
        const int k = col < o.end[0] ? 0 : col < o.end[1] ? 1 : 2;
        if (o.out[k]) o.out[k][col - (k ? o.end[k - 1] : 0)] = t;
    }
}

}  // namespace efla
