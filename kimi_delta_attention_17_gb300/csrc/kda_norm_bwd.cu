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

// The launch that follows with cudaLaunchAttributeProgrammaticStreamSerialization may start once every CTA
// has said this (or ended); it waits for this kernel's writes by itself.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;"); }

constexpr int kSms = 152;
// What one CTA has done after so many rounds it does alone: without parts of the weight's gradient, their memory and
// the second launch, an eager call of the norm's takes 15.5-16 us for 19-19.5, of the gate's 16.5-17 for 21-21.5, at
// any number of rounds. In a captured graph, where only the GPU's time counts, 2 rounds are no slower, 4 take 3.5-3.9
// us for 2.7-3.2, 6 take 4.5-4.9 for 2.8-3.2 (rows of 64 to 2048), 8.8 for 4.9 (of 8192) and 9.0 for 3.0 (the gate's
// of 128, bf16), 12 take 7.4-15.8 for 2.7-5.0: up to 6 a graph loses at most what an eager call gains.
constexpr int kOneCta = 6;

RowThreads bwd_threads(int D) { return D <= 512 ? RowThreads{256, D <= 256 ? 1 : 2} : row_threads(D, true); }

// CTAs that an SM runs at once, by the registers that the kernels below take: what is launched, so that no rows
// wait for a second round.
int ctas_per_sm(int D) {
    const RowThreads s = bwd_threads(D);
    if (D <= 512) return 2;
    return s.groups == 1 ? 1024 / s.threads : s.groups == 2 && s.threads <= 256 ? 512 / s.threads : 1;
}

// Threads of a row: kTpr lanes of a CTA of 256 threads (8, 16 or 32), or the whole CTA (0).
template <int kTpr>
struct BwdShape {
    static constexpr int lanes = kTpr ? kTpr : 32;
    static constexpr int threads = 256;  // of a CTA, kTpr > 0
    static constexpr int rows = kTpr ? threads / kTpr : 1;  // at a time
};

// A CTA takes rows in turn: kPasses of them for each of its teams of threads. With 16-bit rows the next ones'
// loads are on their way while it works on one (32768 x 2048, bf16: 104 us without, 92 with; with an fp32 h
// enough is in flight: 166 us, and 179 with it).
template <typename X, typename Hh, int kTpr, int kGroups, int kPasses, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas)
rmsnorm_bwd_kernel(const X *dy, const Hh *__restrict__ h, const float *__restrict__ rstd,
                   const float *__restrict__ w, const Hh *dh, X *dx, Hh *dres,  // may be in place
                   float *__restrict__ part, long long rows, int D) {
    using S = BwdShape<kTpr>;
    extern __shared__ __align__(16) float rows_dw[];  // [S::rows][D], where a CTA has several rows
    __shared__ __align__(16) float sums[2][32];
    const int threads = kTpr ? S::threads : blockDim.x;
    const int tpr = kTpr ? kTpr : threads, lane = kTpr ? threadIdx.x % kTpr : threadIdx.x, sub = kTpr ? threadIdx.x / tpr : 0;
    const int warp = threadIdx.x >> 5, warps = threads >> 5;
    const int groups = D / 8;
    // Up to 16 values a thread the weights, u and n stay in registers. Wider rows form them again after the sum:
    // from the row as it was loaded where that fits (24 values a thread, or 32 with an h of 16 bits), or from the
    // L2 cache.
    constexpr bool kKeep = kGroups <= 2, kRaw = !kKeep && (sizeof(Hh) == 2 || kGroups == 3) && kThreads <= 512;
    constexpr bool kNext = kKeep && sizeof(Hh) == 2;
    float wv[kKeep ? kGroups : 1][8], dw[kGroups][8];
    auto weights = [&](int i, float *v) {
        const int c = lane + i * tpr;
        if (w && c < groups) {
            unpack8(load8(w + 8 * c), v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 1.f;
        }
    };
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        if constexpr (kKeep) weights(i, wv[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    if (!kTpr && warp == 0) sums[0][threadIdx.x] = sums[1][threadIdx.x] = 0.f;
    if (!kTpr) __syncthreads();
    Raw8<X> ry[kPasses][kGroups];
    Raw8<Hh> rh[kPasses][kGroups], rd[kPasses][kGroups];
    float r_next[kPasses];
    auto load = [&](long long row0) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const long long row = row0 + p * S::rows;
            if (row >= rows) break;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int c = lane + i * tpr;
                if (c >= groups) break;
                const size_t at = (size_t)row * D + 8 * c;
                ry[p][i] = load8(dy + at);
                rh[p][i] = load8(h + at);
                if (dh) rd[p][i] = load8(dh + at);
            }
            r_next[p] = rstd[row];
        }
    };
    const long long step = (long long)gridDim.x * (S::rows * kPasses);
    const long long start = (long long)blockIdx.x * (S::rows * kPasses);
    if (kNext) load(start + sub);
    int flip = 0;
    const float inv_d = 1.f / (float)D;
    for (long long first = start; first < rows; first += step) {
        if (!kNext) load(first + sub);
        float r[kPasses], un[kPasses], u[kPasses][kKeep ? kGroups : 1][8], n[kPasses][kKeep ? kGroups : 1][8];
        Raw8<Hh> cd[kPasses][kGroups];
        auto inside = [&](int p, int i) { return first + sub + p * S::rows < rows && lane + i * tpr < groups; };
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            r[p] = r_next[p];
            un[p] = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int k = kKeep ? i : 0;
                unpack8(ry[p][i], u[p][k]);
                unpack8(rh[p][i], n[p][k]);
                cd[p][i] = rd[p][i];
                if constexpr (!kKeep) weights(i, wv[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!inside(p, i)) u[p][k][j] = n[p][k][j] = 0.f;
                    else n[p][k][j] *= r[p];
                    dw[i][j] += u[p][k][j] * n[p][k][j];
                    u[p][k][j] *= wv[k][j];
                    un[p] += u[p][k][j] * n[p][k][j];
                }
            }
        }
        if (kNext) load(first + sub + step);
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            un[p] = lanes_sum<S::lanes>(un[p]);
            if constexpr (kTpr == 0) {
                if ((threadIdx.x & 31) == 0) sums[flip][warp] = un[p];
                __syncthreads();  // the other half of `sums` is read no more: one barrier a row
                un[p] = 0.f;
                for (int i = 0; i < warps; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sums[flip][i]);
                    un[p] += (v.x + v.y) + (v.z + v.w);
                }
                flip ^= 1;
            }
            un[p] *= inv_d;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                if (!inside(p, i)) continue;
                const size_t at = (size_t)(first + sub + p * S::rows) * D + 8 * (lane + i * tpr);
                const int k = kKeep ? i : 0;
                if constexpr (!kKeep) {
                    if constexpr (kRaw) {
                        unpack8(ry[p][i], u[p][0]);
                        unpack8(rh[p][i], n[p][0]);
                    } else {
                        unpack8(load8(dy + at), u[p][0]);
                        unpack8(load8(h + at), n[p][0]);
                        if (dh) cd[p][i] = load8(dh + at);
                    }
                    weights(i, wv[0]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        n[p][0][j] *= r[p];
                        u[p][0][j] *= wv[0][j];
                    }
                }
                float d[8];
                if (dh) {
                    unpack8(cd[p][i], d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] += r[p] * (u[p][k][j] - n[p][k][j] * un[p]);
                store8(dx + at, d);
                if (dres) store8(dres + at, d);
            }
        }
    }
    dependents_may_start();
    if (!part) return;
    if constexpr (S::rows > 1) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * tpr;
            if (c < groups) store8(rows_dw + (size_t)sub * D + 8 * c, dw[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += S::threads) {
            float t = 0.f;
            for (int s = 0; s < S::rows; ++s) t += rows_dw[(size_t)s * D + c];
            part[(size_t)blockIdx.x * D + c] = t;
        }
    } else {
        // Parts are 16-byte aligned; the weight's gradient itself, which one CTA writes, may begin at any float.
        const bool wide = (reinterpret_cast<uintptr_t>(part) & 15u) == 0;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = lane + i * tpr;
            if (c >= groups) continue;
            float *to = part + (size_t)blockIdx.x * D + 8 * c;
            if (wide) {
                store8(to, dw[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) to[j] = dw[i][j];
            }
        }
    }
}

template <typename X, typename Hh, int kTpr, int kGroups, int kPasses, int kThreads, int kCtas>
cudaError_t launch_bwd_k(const NormBwdArgs &a, int threads, cudaStream_t stream) {
    using S = BwdShape<kTpr>;
    const unsigned blocks = (unsigned)norm_bwd_parts(a.rows, a.D);
    const size_t smem = a.dweight && S::rows > 1 ? (size_t)S::rows * a.D * sizeof(float) : 0;
    rmsnorm_bwd_kernel<X, Hh, kTpr, kGroups, kPasses, kThreads, kCtas><<<blocks, threads, smem, stream>>>(
        static_cast<const X *>(a.dy), static_cast<const Hh *>(a.h), a.rstd, a.w, static_cast<const Hh *>(a.dh),
        static_cast<X *>(a.dx), static_cast<Hh *>(a.dres), blocks == 1 ? a.dweight : a.dweight ? a.part : nullptr, a.rows,
        a.D);
    const cudaError_t err = cudaGetLastError();
    return err != cudaSuccess || !a.dweight || blocks == 1 ? err : launch_sum_parts(a.part, (int)blocks, a.D, a.dweight, stream);
}

template <typename X, typename Hh>
cudaError_t launch_bwd_t(const NormBwdArgs &a, cudaStream_t stream) {
    const RowThreads s = bwd_threads(a.D);
    if (a.D <= 64) return launch_bwd_k<X, Hh, 8, 1, 2, 256, 2>(a, s.threads, stream);
    if (a.D <= 128) return launch_bwd_k<X, Hh, 16, 1, 2, 256, 2>(a, s.threads, stream);
    if (a.D <= 256) return launch_bwd_k<X, Hh, 32, 1, 2, 256, 2>(a, s.threads, stream);
    if (a.D <= 512) return launch_bwd_k<X, Hh, 32, 2, 1, 256, 2>(a, s.threads, stream);
    if (s.groups == 1) return launch_bwd_k<X, Hh, 0, 1, 1, 512, 2>(a, s.threads, stream);
    if (s.groups == 2 && s.threads <= 256) return launch_bwd_k<X, Hh, 0, 2, 1, 256, 2>(a, s.threads, stream);
    if (s.groups == 2) return launch_bwd_k<X, Hh, 0, 2, 1, 512, 1>(a, s.threads, stream);
    if (s.groups == 3) return launch_bwd_k<X, Hh, 0, 3, 1, 512, 1>(a, s.threads, stream);
    if (s.threads <= 512) return launch_bwd_k<X, Hh, 0, 4, 1, 512, 1>(a, s.threads, stream);
    return launch_bwd_k<X, Hh, 0, 4, 1, 1024, 1>(a, s.threads, stream);
}

// ---- the output gate

template <int D, typename T, int kGateWarps>
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
            // s = 1 / (1 + t) and 1 - s = t s with t = e^-z; below -80 e^80 keeps t finite. The fast exponential
            // and quotient, as in the forward call, are off by up to (10 + 2.4 |z|) 2^-24 of s; with expf and a
            // rounded quotient 16384 x 32 x 128 fp32 takes 220 us for 212, and for logits of order one the error's
            // mean square root is 2-3 % less.
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
    dependents_may_start();
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

// Rows that a CTA of so many warps takes at once.
template <int D, typename T>
constexpr int gate_rows(int warps) {
    return warps * 32 / (D * (int)sizeof(T) / 16);
}

template <int D, typename T, int kGateWarps>
cudaError_t launch_gate_bwd_k(const GateBwdArgs &a, unsigned blocks, float *part, cudaStream_t stream) {
    gate_bwd_kernel<D, T, kGateWarps><<<blocks, 32 * kGateWarps, 0, stream>>>(
        static_cast<const T *>(a.dout), static_cast<const T *>(a.o), static_cast<const T *>(a.z), a.w, a.eps,
        static_cast<T *>(a.d_o), static_cast<T *>(a.dz), part, a.rows);
    return cudaGetLastError();
}

template <int D, typename T>
cudaError_t launch_gate_bwd(const GateBwdArgs &a, cudaStream_t stream) {
    if (gate_bwd_parts(a.rows, D, a.dtype) == 1) return launch_gate_bwd_k<D, T, 32>(a, 1, a.dweight, stream);
    constexpr int kRows = gate_rows<D, T>(8);
    const long long want = (a.rows + kRows - 1) / kRows;
    const unsigned blocks = (unsigned)(want < kGateParts ? want : kGateParts);
    const cudaError_t err = launch_gate_bwd_k<D, T, 8>(a, blocks, a.dweight ? a.part : nullptr, stream);
    return err != cudaSuccess || !a.dweight ? err : launch_sum_parts(a.part, (int)blocks, D, a.dweight, stream);
}

// One CTA for 8 columns, its rows of threads sharing out the parts: 128 rows for many parts, 32 for few (1216 parts
// of 128 columns took 8.6 us with 32 columns and 32 rows of threads a CTA: four CTAs, 38 loads in turn).
constexpr int kSumCols = 8;
__global__ void __launch_bounds__(kSumCols * 128)
sum_parts_kernel(const float *__restrict__ part, int parts, int D, float *__restrict__ dweight) {
    __shared__ float sums[kSumCols][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, x = lane % kSumCols;
    const int c = blockIdx.x * kSumCols + x;  // D is a multiple of 8
    float t = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
    for (int p = threadIdx.x / kSumCols; p < parts; p += blockDim.x / kSumCols) t += part[(size_t)p * D + c];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    if (lane < kSumCols) sums[x][warp] = t;
    __syncthreads();
    if (warp >= kSumCols) return;
    t = lanes_sum<32>(lane < blockDim.x / 32 ? sums[warp][lane] : 0.f);
    if (lane == 0) dweight[blockIdx.x * kSumCols + warp] = t;
}

}  // namespace

cudaError_t launch_sum_parts(const float *part, int parts, int D, float *dweight, cudaStream_t stream) {
    // Launched as the kernel before it ends: what it needs of a launch's time is over when the parts are there.
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / kSumCols);
    cfg.blockDim = dim3(kSumCols * (parts > 256 ? 128 : 32));
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_parts_kernel, part, parts, D, dweight);
}

int norm_bwd_parts(long long rows, int D) {
    const RowThreads s = bwd_threads(D);
    const int per = D <= 64 ? 64 : D <= 128 ? 32 : D <= 256 ? 16 : D <= 512 ? 8 : 1, most = kSms * ctas_per_sm(D);
    const long long want = (rows + per - 1) / per;
    return want <= kOneCta ? 1 : want < most ? (int)want : most;
}

int gate_bwd_parts(long long rows, int dv, kda_dtype dtype) {
    const int per = 32 * 32 / (dv * (dtype == KDA_DTYPE_BF16 ? 2 : 4) / 16);
    return rows <= kOneCta * per ? 1 : rows < kGateParts ? (int)rows : kGateParts;
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
