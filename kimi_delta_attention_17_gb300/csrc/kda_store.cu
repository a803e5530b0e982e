// States kept in 8 bits: slots of a pool of fp32 states into a store of codes with one fp32 scale for
// each block of 32, 64 or 128 consecutive values, and back. With m the largest magnitude of a block and
// top = 127 (int8) or 448 (e4m3):
//     scale = m * (1 / top),   code = round(x * (top / m)),   value = code * scale,
// the factor top / m and the products rounded to fp32, codes to the nearest, ties to even; blocks with
// m < 2^-100, whose factor could overflow, are stored as zeros.
//
// A CTA takes one piece of one entry's slot in one layer. A warp reads 128 values at a time, four a
// lane, so that a block is 8, 16 or 32 lanes and its largest magnitude comes from one reduction over
// them; codes leave as four bytes a lane, a full 128-byte line per warp. The loads of a piece are issued
// before the entry is looked up among the later ones (the last of those that name one destination
// holds), by every CTA: with 4096 entries, the most, of 64 KiB quantising takes 69 us (4.9 TB/s), where 256 of 1 MiB
// take 58 (5.8 TB/s). Bound by HBM: 4 bytes a value one way, 1 the other.
#include <cuda_fp8.h>

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kStoreThreads = 256;
constexpr int kStoreUnroll = 4;  // 2: quantising 256 slots of 1 MiB takes 64 us for 58; 8: no change
constexpr int kStorePiece = kStoreThreads * 4 * kStoreUnroll;  // values

// Whether entry i writes: its destination and source are in range, and no later entry that writes names
// the same destination. Uniform over the CTA.
__device__ __forceinline__ bool entry_holds(const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n, int i,
                                            int src_slots, int dst_slots) {
    const int d = dst[i];
    if (d < 0 || d >= dst_slots || src[i] >= src_slots) return false;
    int later = 0;
    for (int j = i + 1 + threadIdx.x; j < n; j += kStoreThreads) later |= dst[j] == d && src[j] < src_slots;
    return !__syncthreads_or(later);
}

__device__ __forceinline__ uint32_t top_bits(uint32_t bits, int block) {
    const unsigned lane = threadIdx.x & 31u;
    const unsigned mask = block == 128 ? 0xffffffffu : block == 64 ? 0xffffu << (lane & 16u) : 0xffu << (lane & 24u);
    return __reduce_max_sync(mask, bits);
}

template <bool kInt8>
__device__ __forceinline__ uint32_t encode(const float4 &x, float inv) {
    if (kInt8) {
        // Added to 1.5 2^23 a product is rounded to a whole number, ties to even, whose two's complement are the
        // sum's low bits.
        constexpr float kWhole = 12582912.f;
        const uint32_t a = __float_as_uint(__fadd_rn(__fmul_rn(x.x, inv), kWhole)), b = __float_as_uint(__fadd_rn(__fmul_rn(x.y, inv), kWhole));
        const uint32_t c = __float_as_uint(__fadd_rn(__fmul_rn(x.z, inv), kWhole)), d = __float_as_uint(__fadd_rn(__fmul_rn(x.w, inv), kWhole));
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x * inv, x.y * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z * inv, x.w * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

template <bool kInt8>
__device__ __forceinline__ float4 decode(uint32_t c, float scale) {
    if (kInt8)
        return make_float4((float)(int8_t)c * scale, (float)(int8_t)(c >> 8) * scale, (float)(int8_t)(c >> 16) * scale,
                           (float)((int32_t)c >> 24) * scale);
    const __half2 lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
    const __half2 hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3);
    const float2 a = __half22float2(lo), b = __half22float2(hi);
    return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

template <bool kInt8>
__global__ void __launch_bounds__(kStoreThreads)
quantize_kernel(const float *__restrict__ pool, int num_slots, uint8_t *__restrict__ store, float *__restrict__ scales,
                int store_slots, const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n,
                long long slot_values, int block, int shift) {  // block = 1 << shift
    const int entry = blockIdx.y;
    const size_t layer = blockIdx.z;
    const int s = src[entry];
    const long long at = (long long)blockIdx.x * kStorePiece + 4 * threadIdx.x;
    float4 x[kStoreUnroll];
    const float *from = pool + (layer * num_slots + (size_t)max(min(s, num_slots - 1), 0)) * slot_values;
#pragma unroll
    for (int k = 0; k < kStoreUnroll; ++k) {
        const long long c = at + (long long)k * 4 * kStoreThreads;
        x[k] = s >= 0 && c < slot_values ? __ldcs(reinterpret_cast<const float4 *>(from + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (!entry_holds(src, dst, n, entry, num_slots, store_slots)) return;
    const size_t to = layer * store_slots + dst[entry];
#pragma unroll
    for (int k = 0; k < kStoreUnroll; ++k) {
        const long long c = at + (long long)k * 4 * kStoreThreads;
        const uint32_t abs_mask = 0x7fffffffu;
        uint32_t m = max(max(__float_as_uint(x[k].x) & abs_mask, __float_as_uint(x[k].y) & abs_mask),
                         max(__float_as_uint(x[k].z) & abs_mask, __float_as_uint(x[k].w) & abs_mask));
        m = top_bits(m, block);  // the bits of magnitudes are ordered as they are, NaN above all
        const float most = __uint_as_float(m), top = kInt8 ? 127.f : 448.f;
        const bool none = most < kStoreTiny;
        const float inv = none ? 0.f : __fdiv_rn(top, most);
        if (c >= slot_values) continue;
        *reinterpret_cast<uint32_t *>(store + to * slot_values + c) = encode<kInt8>(x[k], inv);
        if ((c & (block - 1)) == 0)
            scales[to * (slot_values >> shift) + (c >> shift)] =
                none                       ? 0.f
                : m < 0x7f800000u ? most * (float)(kInt8 ? 1.0 / 127.0 : 1.0 / 448.0)
                                  : __uint_as_float(0x7fffffffu);  // not finite: the block comes back as NaN
    }
}

template <bool kInt8>
__global__ void __launch_bounds__(kStoreThreads)
dequantize_kernel(const uint8_t *__restrict__ store, const float *__restrict__ scales, int store_slots,
                  float *__restrict__ pool, int num_slots, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                  int n, long long slot_values, int shift) {
    const int entry = blockIdx.y;
    const size_t layer = blockIdx.z;
    const int s = src[entry];
    const long long at = (long long)blockIdx.x * kStorePiece + 4 * threadIdx.x;
    const size_t from = layer * store_slots + (size_t)max(min(s, store_slots - 1), 0);
    uint32_t x[kStoreUnroll];
    float f[kStoreUnroll];
#pragma unroll
    for (int k = 0; k < kStoreUnroll; ++k) {
        const long long c = at + (long long)k * 4 * kStoreThreads;
        const bool in = s >= 0 && c < slot_values;
        x[k] = in ? *reinterpret_cast<const uint32_t *>(store + from * slot_values + c) : 0u;
        f[k] = in ? scales[from * (slot_values >> shift) + (c >> shift)] : 0.f;
    }
    if (!entry_holds(src, dst, n, entry, store_slots, num_slots)) return;
    float *to = pool + (layer * num_slots + dst[entry]) * slot_values;
#pragma unroll
    for (int k = 0; k < kStoreUnroll; ++k) {
        const long long c = at + (long long)k * 4 * kStoreThreads;
        if (c < slot_values) __stcs(reinterpret_cast<float4 *>(to + c), decode<kInt8>(x[k], f[k]));
    }
}

dim3 store_grid(const StoreArgs &a) {
    return dim3((unsigned)((a.slot_values + kStorePiece - 1) / kStorePiece), (unsigned)a.n, (unsigned)a.layers);
}
int store_shift(const StoreArgs &a) { return a.block == 32 ? 5 : a.block == 64 ? 6 : 7; }

}  // namespace

cudaError_t launch_state_quantize(const StoreArgs &a, cudaStream_t stream) {
    if (a.n == 0) return cudaSuccess;
    (a.int8 ? quantize_kernel<true> : quantize_kernel<false>)<<<store_grid(a), kStoreThreads, 0, stream>>>(
        a.pool, a.num_slots, a.store, a.scales, a.store_slots, a.src, a.dst, a.n, a.slot_values, a.block, store_shift(a));
    return cudaGetLastError();
}

cudaError_t launch_state_dequantize(const StoreArgs &a, cudaStream_t stream) {
    if (a.n == 0) return cudaSuccess;
    (a.int8 ? dequantize_kernel<true> : dequantize_kernel<false>)<<<store_grid(a), kStoreThreads, 0, stream>>>(
        a.store, a.scales, a.store_slots, a.pool, a.num_slots, a.src, a.dst, a.n, a.slot_values, store_shift(a));
    return cudaGetLastError();
}

}  // namespace kda
