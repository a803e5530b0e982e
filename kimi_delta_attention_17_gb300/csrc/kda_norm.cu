// Root-mean-square norm of rows, with the residual's addition before it:
//     h = x + residual (as stored),   y = w o h / sqrt(mean(h^2) + eps),
// y in x's type, or in e4m3 with one fp32 scale per row or per 128 values.
//
// A row is read once and kept in registers: the threads of a row hold kGroups groups of 8 values each, the
// sum of squares (and the largest magnitude, for the scales) goes over the row's lanes by shuffles and over
// its warps through shared memory. Rows of up to 512 values take a warp or less, several a CTA; wider ones a
// CTA of as many warps as they need. Bound by HBM: x and the residual in, h and y out, nothing twice.
#include <cuda_fp8.h>

#include "kda_rows.cuh"

namespace kda {
namespace {

struct NoResidual {};

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Threads of a row: kTpr lanes (8, 16 or 32; a CTA of 128 threads then has 128 / kTpr rows a pass), or the
// whole CTA (0), whose warps meet in shared memory.
template <int kTpr>
struct RowShape {
    static constexpr int lanes = kTpr ? kTpr : 32;
    static constexpr int threads = 128;              // of a CTA, kTpr > 0
    static constexpr int rows = kTpr ? threads / kTpr : 1;  // a pass
};

template <typename X, typename R, bool kQuant, int kTpr, int kGroups, int kPasses, int kThreads>
__global__ void __launch_bounds__(kThreads)
rmsnorm_kernel(const X *x, const R *residual, const float *__restrict__ w, float eps,
               X *__restrict__ out, uint8_t *__restrict__ q, float *__restrict__ scales, int scale_block,
               R *residual_out, float *__restrict__ rstd, long long rows, int D) {
    using S = RowShape<kTpr>;
    constexpr bool kRes = !std::is_same<R, NoResidual>::value;
    __shared__ __align__(16) float sums[32];
    __shared__ __align__(16) uint32_t tops[32];
    const int tpr = kTpr ? kTpr : blockDim.x, lane = kTpr ? threadIdx.x % kTpr : threadIdx.x;
    const int warp = threadIdx.x >> 5, warps = kTpr ? 1 : (int)blockDim.x >> 5;
    const int groups = D / 8;
    const long long row0 = (long long)blockIdx.x * (S::rows * kPasses) + (kTpr ? threadIdx.x / tpr : 0);
    if (!kTpr && warp == 0) {  // what no warp writes counts as nothing
        sums[threadIdx.x] = 0.f;
        tops[threadIdx.x] = 0;
    }
    if (!kTpr) __syncthreads();
    auto inside = [&](int p, int i) { return row0 + p * S::rows < rows && lane + i * tpr < groups; };
    auto place = [&](int p, int i) { return (size_t)(row0 + p * S::rows) * D + 8 * (lane + i * tpr); };
    float h[kPasses][kGroups][8];
    {
        Raw8<X> rx[kPasses][kGroups];
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                if (inside(p, i)) rx[p][i] = load8(x + place(p, i));
        if constexpr (kRes) {
            Raw8<R> rr[kPasses][kGroups];
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    if (inside(p, i)) rr[p][i] = load8(residual + place(p, i));
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    if (!inside(p, i)) continue;
                    float r[8];
                    unpack8(rx[p][i], h[p][i]);
                    unpack8(rr[p][i], r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[p][i][j] = to_f32<R>(from_f32<R>(h[p][i][j] + r[j]));
                    store8(residual_out + place(p, i), h[p][i]);
                }
        } else {
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    if (inside(p, i)) unpack8(rx[p][i], h[p][i]);
        }
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const long long row = row0 + p * S::rows;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!inside(p, i)) h[p][i][j] = 0.f;
                ss += h[p][i][j] * h[p][i][j];
            }
        }
        ss = lanes_sum<S::lanes>(ss);
        if constexpr (kTpr == 0) {
            if ((threadIdx.x & 31) == 0) sums[warp] = ss;
            __syncthreads();
            ss = 0.f;
            for (int i = 0; i < warps; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&sums[i]);
                ss += (v.x + v.y) + (v.z + v.w);
            }
        }
        const float r = rsqrtf(ss / (float)D + eps);
        if (rstd && row < rows && lane == 0) rstd[row] = r;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * tpr;
            if (c >= groups) continue;
            float wv[8];
            if (w) {
                unpack8(load8(w + 8 * c), wv);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) wv[j] = 1.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[p][i][j] = wv[j] * (h[p][i][j] * r);
            if (!kQuant && row < rows) store8(out + place(p, i), h[p][i]);
        }
        if constexpr (kQuant) {
            // The largest magnitude by its bits, whose order is the magnitudes' with NaN above all.
            uint32_t top[kGroups], most = 0;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                top[i] = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top[i] = umax(top[i], __float_as_uint(h[p][i][j]) & 0x7fffffffu);
                most = umax(most, top[i]);
            }
            const int nblocks = scale_block ? (D + scale_block - 1) / scale_block : 1;
            if (scale_block) {  // 128 values: 16 lanes of one group each, or a whole row of 64
                constexpr int kBlockLanes = S::lanes < 16 ? S::lanes : 16;
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
#pragma unroll
                    for (int m = kBlockLanes / 2; m > 0; m >>= 1)
                        top[i] = umax(top[i], __shfl_xor_sync(0xffffffffu, top[i], m));
            } else {
#pragma unroll
                for (int m = S::lanes / 2; m > 0; m >>= 1) most = umax(most, __shfl_xor_sync(0xffffffffu, most, m));
                if constexpr (kTpr == 0) {
                    if ((threadIdx.x & 31) == 0) tops[warp] = most;
                    __syncthreads();
                    for (int i = 0; i < warps; i += 4) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(&tops[i]);
                        most = umax(most, umax(umax(v.x, v.y), umax(v.z, v.w)));
                    }
                }
#pragma unroll
                for (int i = 0; i < kGroups; ++i) top[i] = most;
            }
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int c = lane + i * tpr;
                if (!inside(p, i)) continue;
                const float m = __uint_as_float(top[i]);
                const bool none = m < kStoreTiny;
                const float inv = none ? 0.f : __fdiv_rn(448.f, m);
                uint32_t code[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    code[k] = 0;
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float2 v = make_float2(h[p][i][4 * k + j] * inv, h[p][i][4 * k + j + 1] * inv);
                        code[k] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (8 * j);
                    }
                }
                *reinterpret_cast<uint2 *>(q + place(p, i)) = make_uint2(code[0], code[1]);
                if (scale_block ? c % 16 == 0 : c == 0)
                    scales[(size_t)row * nblocks + (scale_block ? c / 16 : 0)] = none ? 0.f : m * (float)(1.0 / 448.0);
            }
        }
    }
}

template <typename X, typename R, bool kQuant, int kTpr, int kGroups, int kPasses, int kThreads>
cudaError_t launch_fwd_k(const NormArgs &a, int threads, cudaStream_t stream) {
    const long long per = RowShape<kTpr>::rows * kPasses;
    rmsnorm_kernel<X, R, kQuant, kTpr, kGroups, kPasses, kThreads><<<(unsigned)((a.rows + per - 1) / per), threads, 0, stream>>>(
        static_cast<const X *>(a.x), static_cast<const R *>(a.residual), a.w, a.eps, static_cast<X *>(a.out),
        static_cast<uint8_t *>(a.q), a.scales, a.scale_block, static_cast<R *>(a.residual_out), a.rstd, a.rows, a.D);
    return cudaGetLastError();
}

template <typename X, typename R, bool kQuant>
cudaError_t launch_fwd_q(const NormArgs &a, cudaStream_t stream) {
    constexpr int T = RowShape<8>::threads;
    if (a.D <= 64) return launch_fwd_k<X, R, kQuant, 8, 1, 2, T>(a, T, stream);
    if (a.D <= 128) return launch_fwd_k<X, R, kQuant, 16, 1, 2, T>(a, T, stream);
    if (a.D <= 256) return launch_fwd_k<X, R, kQuant, 32, 1, 2, T>(a, T, stream);
    if (a.D <= 512) return launch_fwd_k<X, R, kQuant, 32, 2, 1, T>(a, T, stream);
    const RowThreads s = row_threads(a.D, false);
    if (s.groups == 2) return launch_fwd_k<X, R, kQuant, 0, 2, 1, 512>(a, s.threads, stream);
    if (s.threads <= 512) return launch_fwd_k<X, R, kQuant, 0, 4, 1, 512>(a, s.threads, stream);
    return launch_fwd_k<X, R, kQuant, 0, 4, 1, 1024>(a, s.threads, stream);
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
