// efla_vec.cuh - loads and stores of N consecutive elements, widened to and
// rounded from fp32, for the kernels whose rows may be strided, odd or not
// aligned for 16-byte accesses.
#pragma once
#include "efla_common.cuh"

namespace efla {

// N elements of T as they lie in memory, in registers: a load kept in this
// form can be issued long before its use.
template <typename T, int N> struct alignas(N * sizeof(T) > 16 ? 16 : N * sizeof(T)) Raw { T e[N]; };

// One access of min(16, N * sizeof(T)) bytes each; p must be aligned to that.
template <typename T, int N> __device__ __forceinline__ Raw<T, N> load_raw(const T *p) {
    return *reinterpret_cast<const Raw<T, N> *>(p);
}
// Element accesses: any p, and the first n elements alone (the others are 0).
template <typename T, int N> __device__ __forceinline__ Raw<T, N> load_raw_any(const T *p, int n) {
    Raw<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = i < n ? p[i] : from_f32<T>(0.f);
    return r;
}
template <typename T, int N> __device__ __forceinline__ Raw<T, N> zero_raw() {
    Raw<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = from_f32<T>(0.f);
    return r;
}
template <typename T, int N> __device__ __forceinline__ void widen(const Raw<T, N> &r, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(r.e[i]);
}
template <typename T, int N> __device__ __forceinline__ Raw<T, N> narrow(const float (&v)[N]) {
    Raw<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = from_f32<T>(v[i]);
    return r;
}
template <typename T, int N> __device__ __forceinline__ void store_raw(T *p, const Raw<T, N> &r) {
    *reinterpret_cast<Raw<T, N> *>(p) = r;
}
template <typename T, int N> __device__ __forceinline__ void store_raw_any(T *p, const Raw<T, N> &r, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) p[i] = r.e[i];
}

// 1 / (1 + e^-v) and v / (1 + e^-v).  The division is the approximate one
// (2 ulp); for v below -87 its result is 0 instead of a value under 2^-120.
__device__ __forceinline__ float sigmoid_f32(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
__device__ __forceinline__ float silu_f32(float v) { return __fdividef(v, 1.f + __expf(-v)); }
// d silu(v) / dv = s (1 + v (1 - s)), s = sigmoid(v); 1 - s as e^-v s.
__device__ __forceinline__ float dsilu_f32(float v) {
    const float e = __expf(-v);
    const float s = __fdividef(1.f, 1.f + e);
    return v < -80.f ? 0.f : s * fmaf(v * e, s, 1.f);
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
