// Shared by the kernels that normalise rows: 16-byte pieces as fp32 values, groups of 8 values,
// sums over a group of lanes, and the sum of the CTAs' parts of a weight's gradient.
#pragma once

#include "kda_internal.cuh"

namespace kda {

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &r, float *x);
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4 &r, float *x) {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void unpack16<float>(const uint4 &r, float *x) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float *x);
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float *x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
template <>
__device__ __forceinline__ uint4 pack16<float>(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
}

// 8 consecutive values as they lie in memory, and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw8<float> {
    uint4 a, b;
};
__device__ __forceinline__ Raw8<__nv_bfloat16> load8(const __nv_bfloat16 *p) {
    return {*reinterpret_cast<const uint4 *>(p)};
}
__device__ __forceinline__ Raw8<float> load8(const float *p) {
    return {*reinterpret_cast<const uint4 *>(p), *reinterpret_cast<const uint4 *>(p + 4)};
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float *x) {
    unpack16<__nv_bfloat16>(r.a, x);
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float *x) {
    unpack16<float>(r.a, x);
    unpack16<float>(r.b, x + 4);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x) {
    *reinterpret_cast<uint4 *>(p) = pack16<__nv_bfloat16>(x);
}
__device__ __forceinline__ void store8(float *p, const float *x) {
    *reinterpret_cast<uint4 *>(p) = pack16<float>(x);
    *reinterpret_cast<uint4 *>(p + 4) = pack16<float>(x + 4);
}

// How a CTA holds a row of D > 512 values: groups of 8 a thread, and whole warps.
struct RowThreads {
    int threads, groups;
};
inline RowThreads row_threads(int D, bool backward) {
    const auto warps = [D](int groups) { return ((D / 8 + groups - 1) / groups + 31) / 32; };
    // Two groups a thread; four where two would take more than 512 threads. The backward pass takes one where that
    // leaves fewer lanes idle (60000 x 1032, bf16: 94 us, and 111 with two; the forward pass 85 and 87, but with an
    // 8-bit output 102 and 85), and three up to the width where that takes 512 threads, which leaves registers for
    // fp32 rows (4000 x 12288, fp32: 149 us, and 179 with four; 4000 x 8200: 104 and 152).
    const int groups = D > 8192 ? (backward && D <= 12288 ? 3 : 4) : backward && D <= 4096 && warps(1) < 2 * warps(2) ? 1 : 2;
    return {32 * warps(groups), groups};
}

// Sum over `kLanes` neighbouring lanes (a power of two), in all of them.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// dweight[c] = sum over `parts` rows of part [parts][D], in a fixed order.
cudaError_t launch_sum_parts(const float *part, int parts, int D, float *dweight, cudaStream_t stream);

}  // namespace kda
