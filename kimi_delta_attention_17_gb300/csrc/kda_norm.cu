// Root-mean-square norm of rows, with the residual's addition before it:
//     h = x + residual (as stored),   y = w o h / sqrt(mean(h^2) + eps),
// y in x's type, or in e4m3 with one fp32 scale per row or per 128 values.
//
// A row is read once and kept in registers: `kTpr` threads of a row hold kGroups groups of 8 values
// each, the sum of squares (and the largest magnitude, for the scales) goes over the row's lanes by
// shuffles and over its warps through shared memory. Rows of up to 32 lanes share a CTA of 128
// threads. Bound by HBM: x and the residual in, h and y out, nothing twice.
#include <cuda_fp8.h>

#include "kda_rows.cuh"

namespace kda {
namespace {

struct NoResidual {};

constexpr int kRowCta = 128;  // threads of a CTA whose rows take a warp or less

template <int kTpr>
struct RowShape {
    static constexpr int threads = kTpr > 32 ? kTpr : kRowCta;
    static constexpr int rows = threads / kTpr;  // per CTA
    static constexpr int lanes = kTpr > 32 ? 32 : kTpr;
    static constexpr int warps = kTpr > 32 ? kTpr / 32 : 1;  // per row
};

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <typename X, typename R, bool kQuant, int kTpr, int kGroups>
__global__ void __launch_bounds__(RowShape<kTpr>::threads)
rmsnorm_kernel(const X *__restrict__ x, const R *residual, const float *__restrict__ w, float eps,
               X *__restrict__ out, uint8_t *__restrict__ q, float *__restrict__ scales, int scale_block,
               R *residual_out, float *__restrict__ rstd, long long rows, int D) {
    using S = RowShape<kTpr>;
    constexpr bool kRes = !std::is_same<R, NoResidual>::value;
    __shared__ float sums[32];
    __shared__ uint32_t tops[32];
    const int lane = threadIdx.x % kTpr, warp = threadIdx.x >> 5;
    const long long row = (long long)blockIdx.x * S::rows + threadIdx.x / kTpr;
    const bool live = row < rows;
    const size_t base = (size_t)(live ? row : 0) * D;
    float h[kGroups][8];
    Raw8<X> rx[kGroups];
    const int groups = D / 8;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int c = lane + i * kTpr;
        if (live && c < groups) rx[i] = load8(x + base + 8 * c);
    }
    if constexpr (kRes) {
        Raw8<R> rr[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (live && c < groups) rr[i] = load8(residual + base + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (!(live && c < groups)) continue;
            float r[8];
            unpack8(rx[i], h[i]);
            unpack8(rr[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = to_f32<R>(from_f32<R>(h[i][j] + r[j]));
            store8(residual_out + base + 8 * c, h[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) unpack8(rx[i], h[i]);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        if (!(live && lane + i * kTpr < groups)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += h[i][j] * h[i][j];
    }
    ss = lanes_sum<S::lanes>(ss);
    if constexpr (S::warps > 1) {
        if ((threadIdx.x & 31) == 0) sums[warp] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < S::warps; ++i) ss += sums[i];
    }
    const float r = rsqrtf(ss / (float)D + eps);
    if (rstd && live && lane == 0) rstd[row] = r;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int c = lane + i * kTpr;
        if (c >= groups) continue;
        float wv[8];
        if (w) {
            unpack8(load8(w + 8 * c), wv);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) wv[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = wv[j] * (h[i][j] * r);
        if (!kQuant && live) store8(out + base + 8 * c, h[i]);
    }
    if constexpr (kQuant) {
        // The largest magnitude by its bits, whose order is the magnitudes' with NaN above all.
        uint32_t top[kGroups], most = 0;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            top[i] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) top[i] = umax(top[i], __float_as_uint(h[i][j]) & 0x7fffffffu);
            most = umax(most, top[i]);
        }
        const int nblocks = scale_block ? (D + scale_block - 1) / scale_block : 1;
        if (scale_block) {  // 128 values: 16 lanes of one group each, or a whole row of 64
            constexpr int kBlockLanes = kTpr < 16 ? kTpr : 16;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int m = kBlockLanes / 2; m > 0; m >>= 1)
                    top[i] = umax(top[i], __shfl_xor_sync(0xffffffffu, top[i], m));
        } else {
#pragma unroll
            for (int m = S::lanes / 2; m > 0; m >>= 1) most = umax(most, __shfl_xor_sync(0xffffffffu, most, m));
            if constexpr (S::warps > 1) {
                if ((threadIdx.x & 31) == 0) tops[warp] = most;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < S::warps; ++i) most = umax(most, tops[i]);
            }
#pragma unroll
            for (int i = 0; i < kGroups; ++i) top[i] = most;
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (!(live && c < groups)) continue;
            const float m = __uint_as_float(top[i]);
            const bool none = m < kStoreTiny;
            const float inv = none ? 0.f : __fdiv_rn(448.f, m);
            uint32_t code[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                code[p] = 0;
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float2 v = make_float2(h[i][4 * p + j] * inv, h[i][4 * p + j + 1] * inv);
                    code[p] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (8 * j);
                }
            }
            *reinterpret_cast<uint2 *>(q + base + 8 * c) = make_uint2(code[0], code[1]);
            if (scale_block ? c % 16 == 0 : c == 0)
                scales[(size_t)row * nblocks + (scale_block ? c / 16 : 0)] = none ? 0.f : m * (float)(1.0 / 448.0);
        }
    }
}

template <typename X, typename R, bool kQuant, int kTpr, int kGroups>
cudaError_t launch_fwd_k(const NormArgs &a, cudaStream_t stream) {
    using S = RowShape<kTpr>;
    const unsigned blocks = (unsigned)((a.rows + S::rows - 1) / S::rows);
    rmsnorm_kernel<X, R, kQuant, kTpr, kGroups><<<blocks, S::threads, 0, stream>>>(
        static_cast<const X *>(a.x), static_cast<const R *>(a.residual), a.w, a.eps, static_cast<X *>(a.out),
        static_cast<uint8_t *>(a.q), a.scales, a.scale_block, static_cast<R *>(a.residual_out), a.rstd, a.rows, a.D);
    return cudaGetLastError();
}

template <typename X, typename R, bool kQuant>
cudaError_t launch_fwd_q(const NormArgs &a, cudaStream_t stream) {
    if (a.D <= 64) return launch_fwd_k<X, R, kQuant, 8, 1>(a, stream);
    if (a.D <= 128) return launch_fwd_k<X, R, kQuant, 16, 1>(a, stream);
    if (a.D <= 512) return launch_fwd_k<X, R, kQuant, 32, 2>(a, stream);
    if (a.D <= 1024) return launch_fwd_k<X, R, kQuant, 64, 2>(a, stream);
    if (a.D <= 2048) return launch_fwd_k<X, R, kQuant, 128, 2>(a, stream);
    if (a.D <= 4096) return launch_fwd_k<X, R, kQuant, 256, 2>(a, stream);
    if (a.D <= 8192) return launch_fwd_k<X, R, kQuant, 512, 2>(a, stream);
    if (a.D <= 16384) return launch_fwd_k<X, R, kQuant, 1024, 2>(a, stream);
    return launch_fwd_k<X, R, kQuant, 1024, 4>(a, stream);
}

template <typename X, typename R>
cudaError_t launch_fwd_r(const NormArgs &a, cudaStream_t stream) {
    return a.q ? launch_fwd_q<X, R, true>(a, stream) : launch_fwd_q<X, R, false>(a, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs &a, cudaStream_t stream) {
    if (a.rows == 0) return cudaSuccess;
    const bool res = a.residual != nullptr;
    if (a.dtype == KDA_DTYPE_F32)
        return res ? launch_fwd_r<float, float>(a, stream) : launch_fwd_r<float, NoResidual>(a, stream);
    if (!res) return launch_fwd_r<__nv_bfloat16, NoResidual>(a, stream);
    return a.residual_dtype == KDA_DTYPE_F32 ? launch_fwd_r<__nv_bfloat16, float>(a, stream)
                                             : launch_fwd_r<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace kda
