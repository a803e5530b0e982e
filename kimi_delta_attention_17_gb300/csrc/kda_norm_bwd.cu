// Gradients of the row norms. With r = 1/sqrt(mean(h^2) + eps), n = h r:
//     rmsnorm (y = w o n):              u = w o dy,
//                                       dh = dh_in + r (u - n mean(u o n)),  dw = sum_rows dy o n
//     output gate (y = w o n o s(z)):   u = w o dy o s(z),
//                                       do = r (u - n mean(u o n)),  dw = sum_rows dy o s(z) o n,
//                                       dz = u o n o (1 - s(z))
// Bound by HBM: every row is read once, its sums go over its lanes, and its gradients are written.
// The weight's gradient is summed in registers over the rows a thread takes (each thread keeps to its
// columns), over a CTA's rows through shared memory, and over the CTAs by a second small launch, in a
// fixed order.
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int kBwdCta = 256;  // threads of a CTA whose rows take a warp or less

template <int kTpr>
struct BwdShape {
    static constexpr int threads = kTpr > 32 ? kTpr : kBwdCta;
    static constexpr int rows = threads / kTpr;
    static constexpr int lanes = kTpr > 32 ? 32 : kTpr;
    static constexpr int warps = kTpr > 32 ? kTpr / 32 : 1;
};

template <typename X, typename Hh, int kTpr, int kGroups>
__global__ void __launch_bounds__(BwdShape<kTpr>::threads)
rmsnorm_bwd_kernel(const X *dy, const Hh *__restrict__ h, const float *__restrict__ rstd,
                   const float *__restrict__ w, const Hh *dh, X *dx, Hh *dres,  // may be in place
                   float *__restrict__ part, long long rows, int D) {
    using S = BwdShape<kTpr>;
    extern __shared__ float smem[];  // the rows' weight gradients, where a CTA has several rows
    __shared__ float sums[2][32];
    const int lane = threadIdx.x % kTpr, warp = threadIdx.x >> 5, sub = threadIdx.x / kTpr;
    const int groups = D / 8;
    float wv[kGroups][8], dw[kGroups][8];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int c = lane + i * kTpr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            wv[i][j] = c < groups ? (w ? w[8 * c + j] : 1.f) : 0.f;
            dw[i][j] = 0.f;
        }
    }
    int flip = 0;
    const float inv_d = 1.f / (float)D;
    for (long long first = (long long)blockIdx.x * S::rows; first < rows; first += (long long)gridDim.x * S::rows) {
        const long long row = first + sub;
        const bool live = row < rows;
        const size_t base = (size_t)(live ? row : 0) * D;
        Raw8<X> ry[kGroups];
        Raw8<Hh> rh[kGroups], rd[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (live && c < groups) {
                ry[i] = load8(dy + base + 8 * c);
                rh[i] = load8(h + base + 8 * c);
                if (dh) rd[i] = load8(dh + base + 8 * c);
            }
        }
        const float r = live ? rstd[row] : 0.f;
        float un = 0.f;
        float u[kGroups][8], n[kGroups][8];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const bool in = live && lane + i * kTpr < groups;
            unpack8(ry[i], u[i]);
            unpack8(rh[i], n[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!in) u[i][j] = n[i][j] = 0.f;
                n[i][j] *= r;
                dw[i][j] += u[i][j] * n[i][j];
                u[i][j] *= wv[i][j];
                un += u[i][j] * n[i][j];
            }
        }
        un = lanes_sum<S::lanes>(un);
        if constexpr (S::warps > 1) {
            if ((threadIdx.x & 31) == 0) sums[flip][warp] = un;
            __syncthreads();  // the other half of `sums` is read no more: one barrier a row
            un = 0.f;
#pragma unroll
            for (int i = 0; i < S::warps; ++i) un += sums[flip][i];
            flip ^= 1;
        }
        un *= inv_d;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (!(live && c < groups)) continue;
            float d[8];
            if (dh) {
                unpack8(rd[i], d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] += r * (u[i][j] - n[i][j] * un);
            store8(dx + base + 8 * c, d);
            if (dres) store8(dres + base + 8 * c, d);
        }
    }
    if (!part) return;
    if constexpr (S::rows > 1) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (c < groups) store8(smem + (size_t)sub * D + 8 * c, dw[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += S::threads) {
            float t = 0.f;
            for (int s = 0; s < S::rows; ++s) t += smem[(size_t)s * D + c];
            part[(size_t)blockIdx.x * D + c] = t;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * kTpr;
            if (c < groups) store8(part + (size_t)blockIdx.x * D + 8 * c, dw[i]);
        }
    }
}

template <typename X, typename Hh, int kTpr, int kGroups>
cudaError_t launch_bwd_k(const NormBwdArgs &a, cudaStream_t stream) {
    using S = BwdShape<kTpr>;
    const long long want = (a.rows + S::rows - 1) / S::rows;
    const unsigned blocks = (unsigned)(want < kNormParts ? want : kNormParts);
    const size_t smem = a.dweight && S::rows > 1 ? (size_t)S::rows * a.D * sizeof(float) : 0;
    rmsnorm_bwd_kernel<X, Hh, kTpr, kGroups><<<blocks, S::threads, smem, stream>>>(
        static_cast<const X *>(a.dy), static_cast<const Hh *>(a.h), a.rstd, a.w, static_cast<const Hh *>(a.dh),
        static_cast<X *>(a.dx), static_cast<Hh *>(a.dres), a.dweight ? a.part : nullptr, a.rows, a.D);
    const cudaError_t err = cudaGetLastError();
    return err != cudaSuccess || !a.dweight ? err : launch_sum_parts(a.part, (int)blocks, a.D, a.dweight, stream);
}

template <typename X, typename Hh>
cudaError_t launch_bwd_t(const NormBwdArgs &a, cudaStream_t stream) {
    if (a.D <= 64) return launch_bwd_k<X, Hh, 8, 1>(a, stream);
    if (a.D <= 128) return launch_bwd_k<X, Hh, 16, 1>(a, stream);
    if (a.D <= 256) return launch_bwd_k<X, Hh, 32, 1>(a, stream);
    if (a.D <= 512) return launch_bwd_k<X, Hh, 64, 1>(a, stream);
    if (a.D <= 1024) return launch_bwd_k<X, Hh, 128, 1>(a, stream);
    if (a.D <= 2048) return launch_bwd_k<X, Hh, 256, 1>(a, stream);
    if (a.D <= 4096) return launch_bwd_k<X, Hh, 512, 1>(a, stream);
    if (a.D <= 8192) return launch_bwd_k<X, Hh, 1024, 1>(a, stream);
    if (a.D <= 16384) return launch_bwd_k<X, Hh, 1024, 2>(a, stream);
    return launch_bwd_k<X, Hh, 1024, 4>(a, stream);
}

// ---- the output gate

constexpr int kGateWarps = 8;

template <int D, typename T>
__global__ void __launch_bounds__(32 * kGateWarps)
gate_bwd_kernel(const T *dout, const T *o, const T *z, const float *__restrict__ w, float eps, T *d_o,
                T *dz,  // either may be in place
                float *__restrict__ part, long long rows) {
    constexpr int E = 16 / (int)sizeof(T), L = D / E, RPW = 32 / L, kRows = kGateWarps * RPW;
    __shared__ float sums[kRows][D];
    const int lane = threadIdx.x & 31, sub = (threadIdx.x >> 5) * RPW + lane / L, li = lane % L;
    float wv[E], dw[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        wv[j] = w ? w[E * li + j] : 1.f;
        dw[j] = 0.f;
    }
    for (long long first = (long long)blockIdx.x * kRows; first < rows; first += (long long)gridDim.x * kRows) {
        const long long row = first + sub;
        const bool live = row < rows;
        const size_t at = (size_t)(live ? row : 0) * D + E * li;
        float x[E], g[E], dy[E];
        unpack16<T>(*reinterpret_cast<const uint4 *>(o + at), x);
        unpack16<T>(*reinterpret_cast<const uint4 *>(z + at), g);
        unpack16<T>(*reinterpret_cast<const uint4 *>(dout + at), dy);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) ss += x[j] * x[j];
        const float r = rsqrtf(lanes_sum<L>(ss) * (1.f / D) + eps);
        float un = 0.f, c[E];
#pragma unroll
        for (int j = 0; j < E; ++j) {
            // s = 1 / (1 + t) and 1 - s = t s with t = e^-z; below -80 e^80 keeps t finite.
            const float t = __expf(g[j] < -80.f ? 80.f : -g[j]);
            const float s = __fdividef(1.f, 1.f + t);
            c[j] = t * s;
            x[j] *= r;
            dy[j] *= s;
            if (live) dw[j] += dy[j] * x[j];
            dy[j] *= wv[j];
            un += dy[j] * x[j];
        }
        un = lanes_sum<L>(un) * (1.f / D);
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            c[j] *= dy[j] * x[j];
            x[j] = r * (dy[j] - x[j] * un);
        }
        *reinterpret_cast<uint4 *>(d_o + at) = pack16<T>(x);
        *reinterpret_cast<uint4 *>(dz + at) = pack16<T>(c);
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < E; ++j) sums[sub][E * li + j] = dw[j];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 32 * kGateWarps) {
        float t = 0.f;
#pragma unroll
        for (int s = 0; s < kRows; ++s) t += sums[s][c];
        part[(size_t)blockIdx.x * D + c] = t;
    }
}

template <int D, typename T>
cudaError_t launch_gate_bwd(const GateBwdArgs &a, cudaStream_t stream) {
    constexpr int kRows = kGateWarps * 32 / (D * (int)sizeof(T) / 16);
    const long long want = (a.rows + kRows - 1) / kRows;
    const unsigned blocks = (unsigned)(want < kGateParts ? want : kGateParts);
    gate_bwd_kernel<D, T><<<blocks, 32 * kGateWarps, 0, stream>>>(
        static_cast<const T *>(a.dout), static_cast<const T *>(a.o), static_cast<const T *>(a.z), a.w, a.eps,
        static_cast<T *>(a.d_o), static_cast<T *>(a.dz), a.dweight ? a.part : nullptr, a.rows);
    const cudaError_t err = cudaGetLastError();
    return err != cudaSuccess || !a.dweight ? err : launch_sum_parts(a.part, (int)blocks, D, a.dweight, stream);
}

// One CTA for 32 columns: 32 rows of threads take every 32nd part.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *__restrict__ part, int parts, int D, float *dweight) {
    __shared__ float sums[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    if (c < D)
        for (int p = threadIdx.y; p < parts; p += 32) t += part[(size_t)p * D + c];
    sums[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    t = lanes_sum<32>(sums[threadIdx.x][threadIdx.y]);
    const int to = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && to < D) dweight[to] = t;
}

}  // namespace

cudaError_t launch_sum_parts(const float *part, int parts, int D, float *dweight, cudaStream_t stream) {
    sum_parts_kernel<<<(D + 31) / 32, dim3(32, 32), 0, stream>>>(part, parts, D, dweight);
    return cudaGetLastError();
}

cudaError_t launch_rmsnorm_bwd(const NormBwdArgs &a, cudaStream_t stream) {
    if (a.rows == 0)
        return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.D * sizeof(float), stream) : cudaSuccess;
    if (a.dtype == KDA_DTYPE_F32) return launch_bwd_t<float, float>(a, stream);
    return a.h_dtype == KDA_DTYPE_F32 ? launch_bwd_t<__nv_bfloat16, float>(a, stream)
                                      : launch_bwd_t<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

cudaError_t launch_output_gate_rmsnorm_bwd(const GateBwdArgs &a, cudaStream_t stream) {
    if (a.rows == 0)
        return a.dweight ? cudaMemsetAsync(a.dweight, 0, (size_t)a.dv * sizeof(float), stream) : cudaSuccess;
    if (a.dtype == KDA_DTYPE_BF16)
        return a.dv == 128 ? launch_gate_bwd<128, __nv_bfloat16>(a, stream) : launch_gate_bwd<64, __nv_bfloat16>(a, stream);
    return a.dv == 128 ? launch_gate_bwd<128, float>(a, stream) : launch_gate_bwd<64, float>(a, stream);
}

}  // namespace kda
