// Gradient of the gated linear recurrence.
//
// With u_t = a_t e_t, the gradient that reaches h_{t-1}, the backward
// recurrence e_t = dout_t + u_{t+1} is again a chain of affine maps,
// u -> a_t u + a_t dout_t, taken from the last token to the first. It is cut
// and composed as the forward scan's is (kda_scan.cu): thread, warp, CTA, and
// a cluster of CTAs over consecutive tiles, which here goes through the
// sequence from its end. dg needs h_{t-1} as well; it is formed again within
// the tile by the forward composition, from the fp32 state that the forward
// call saved at the tile's first token (a tile is KDA_SCAN_CARRY_TOKENS
// tokens), so neither h nor a second pass over the sequence is read, and h is
// not taken from its rounded outputs. Bound by HBM: x, g and dout in, dx and
// dg out, once each.
#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename XT, typename GT>
struct BwdShape {
    using XP = typename Piece<XT>::type;
    using GP = typename Piece<GT>::type;
    static constexpr size_t slots = (size_t)kScanStages * kScanTpt * kScanThreads;
    static constexpr size_t smem = slots * (2 * sizeof(XP) + sizeof(GP));
    static constexpr int per_sm = smem <= 50 * 1024 ? 4 : smem <= 66 * 1024 ? 3 : 2;  // CTAs
};

template <typename XT, typename GT, int kGate, int kWrite>
__global__ void __launch_bounds__(kScanThreads, BwdShape<XT, GT>::per_sm)
scan_bwd(const XT *__restrict__ dout, const float *dfinal, const XT *__restrict__ x,
         const GT *__restrict__ g, const float *__restrict__ carries, const int32_t *__restrict__ cu,
         XT *__restrict__ dx, GT *__restrict__ dg, float *dinit, int T_fixed, long long tokens, int D,
         int blocks, int ranks, float lower) {
    using S = BwdShape<XT, GT>;
    using XP = typename S::XP;
    using GP = typename S::GP;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    GP *gs = reinterpret_cast<GP *>(smem_raw);
    XP *xs = reinterpret_cast<XP *>(smem_raw + S::slots * sizeof(GP));
    XP *ds = xs + S::slots;
    __shared__ __align__(16) float warp_map[2][kScanWarps][3][kScanCh];    // A, U (backward), H (forward)
    __shared__ __align__(16) float cta_map[2][kScanMaxRanks][2][kScanCh];  // A, U

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? (int)cluster_rank() : 0;
    const unsigned unit = blockIdx.x / (unsigned)ranks;
    const int n = (int)(unit / (unsigned)blocks);
    const int col = kScanVec * (lane & (kScanLanes - 1));
    const int ch = (int)(unit % (unsigned)blocks) * kScanCh + col;
    const bool has_ch = ch < D;
    const int group = tid / kScanLanes;

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    const int len = (int)(end - begin);
    const int super = kScanTile * ranks;
    const int steps = (int)(((long long)len + super - 1) / super);

    float u[kScanVec] = {0.f, 0.f, 0.f, 0.f};  // the gradient entering the cluster's tiles from behind
    if (dfinal && has_ch) unpack4(*reinterpret_cast<const float4 *>(dfinal + (size_t)n * D + ch), u);

    auto tokens_left = [&](int i) {
        const long long t = ((long long)i * ranks + rank) * kScanTile + group * kScanTpt;
        return has_ch ? (int)min(max(len - t, 0LL), (long long)kScanTpt) : 0;
    };
    auto first = [&](int i) {
        return (size_t)(begin + ((long long)i * ranks + rank) * kScanTile + group * kScanTpt) * D + ch;
    };
    auto prefetch = [&](int i) {
        if (i >= 0) {
            const int left = tokens_left(i);
            const int s0 = (i & 1) * kScanTpt * kScanThreads + tid;
            const size_t from = first(i);
            const float id = identity_gate<kGate>(), z[4] = {id, id, id, id}, zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < kScanTpt; ++j) {
                const int s = s0 + j * kScanThreads;
                if (j < left) {
                    async_piece<sizeof(GP)>(&gs[s], g + from + (size_t)j * D);
                    async_piece<sizeof(XP)>(&ds[s], dout + from + (size_t)j * D);
                    async_piece<sizeof(XP)>(&xs[s], x + from + (size_t)j * D);
                } else {
                    gs[s] = pack4<GT>(z);
                    ds[s] = xs[s] = pack4<XT>(zero);
                }
            }
        }
        async_commit();
    };

    prefetch(steps - 1);
    for (int i = steps - 1; i >= 0; --i) {
        const int p = i & 1, left = tokens_left(i);
        const int s0 = p * kScanTpt * kScanThreads + tid;
        const long long tile = (long long)i * ranks + rank;
        float h[kScanVec] = {0.f, 0.f, 0.f, 0.f};  // the state entering this CTA's tile
        if (has_ch && tile * kScanTile < len)
            unpack4(*reinterpret_cast<const float4 *>(carries + (size_t)carry_row(begin, n, tile) * D + ch), h);
        prefetch(i - 1);
        async_wait<1>();
        float a[kScanTpt][kScanVec], b[kScanTpt][kScanVec];
        float A[kScanVec], B[kScanVec];
        float H[kScanVec] = {0.f, 0.f, 0.f, 0.f}, U[kScanVec] = {0.f, 0.f, 0.f, 0.f};
        Decay<kGate> decay[kScanVec];
#pragma unroll
        for (int j = 0; j < kScanTpt; ++j) {
            float xv[kScanVec], zv[kScanVec];
            unpack4(xs[s0 + j * kScanThreads], xv);
            unpack4(gs[s0 + j * kScanThreads], zv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                const Gated q = gate_value<kGate, kWrite, false>(zv[c], lower);
                a[j][c] = q.a;
                b[j][c] = q.w * xv[c];
                H[c] = fmaf(q.a, H[c], b[j][c]);
                decay[c].then(q);
            }
        }
#pragma unroll
        for (int j = kScanTpt - 1; j >= 0; --j) {
            float dv[kScanVec];
            unpack4(ds[s0 + j * kScanThreads], dv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) U[c] = a[j][c] * (dv[c] + U[c]);
        }
        // In the warp: predecessors alone (PA, PH) for the states, successors
        // alone (QA, QU) for the gradients.
        float PA[kScanVec], PH[kScanVec], QA[kScanVec], QU[kScanVec];
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            A[c] = B[c] = decay[c].value();
#pragma unroll
            for (int off = kScanLanes; off < 32; off <<= 1) {
                const float A2 = __shfl_up_sync(0xffffffffu, A[c], off);
                const float H2 = __shfl_up_sync(0xffffffffu, H[c], off);
                const float B2 = __shfl_down_sync(0xffffffffu, B[c], off);
                const float U2 = __shfl_down_sync(0xffffffffu, U[c], off);
                if (lane >= off) {
                    H[c] = fmaf(A[c], H2, H[c]);
                    A[c] *= A2;
                }
                if (lane < 32 - off) {
                    U[c] = fmaf(B[c], U2, U[c]);
                    B[c] *= B2;
                }
            }
            PA[c] = __shfl_up_sync(0xffffffffu, A[c], kScanLanes);
            PH[c] = __shfl_up_sync(0xffffffffu, H[c], kScanLanes);
            QA[c] = __shfl_down_sync(0xffffffffu, B[c], kScanLanes);
            QU[c] = __shfl_down_sync(0xffffffffu, U[c], kScanLanes);
            if (lane < kScanLanes) {
                PA[c] = 1.f;
                PH[c] = 0.f;
            }
            if (lane >= 32 - kScanLanes) {
                QA[c] = 1.f;
                QU[c] = 0.f;
            }
        }
        if (lane >= 32 - kScanLanes) {
            *reinterpret_cast<float4 *>(&warp_map[p][warp][0][col]) = pack4<float>(A);
            *reinterpret_cast<float4 *>(&warp_map[p][warp][2][col]) = pack4<float>(H);
        }
        if (lane < kScanLanes) *reinterpret_cast<float4 *>(&warp_map[p][warp][1][col]) = pack4<float>(U);
        __syncthreads();
        float e[kScanVec];  // the gradient entering this warp's tokens, then this thread's, from behind
        auto apply = [&](float *state, const float *by, const float *plus) {
            float A2[kScanVec], H2[kScanVec];
            unpack4(*reinterpret_cast<const float4 *>(by + col), A2);
            unpack4(*reinterpret_cast<const float4 *>(plus + col), H2);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) state[c] = fmaf(A2[c], state[c], H2[c]);
        };
        if (ranks > 1) {
            if (warp == 0) {
                float TA = 1.f, TU = 0.f;
#pragma unroll
                for (int v = kScanWarps - 1; v >= 0; --v) {
                    const float A2 = warp_map[p][v][0][lane];
                    TU = fmaf(A2, TU, warp_map[p][v][1][lane]);
                    TA *= A2;
                }
                for (int r = 0; r < ranks; ++r) {
                    store_peer(&cta_map[p][rank][0][lane], r, TA);
                    store_peer(&cta_map[p][rank][1][lane], r, TU);
                }
            }
            cluster_sync();
            for (int r = ranks - 1; r > rank; --r) apply(u, cta_map[p][r][0], cta_map[p][r][1]);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) e[c] = u[c];
            for (int r = rank; r >= 0; --r) apply(u, cta_map[p][r][0], cta_map[p][r][1]);
            for (int v = kScanWarps - 1; v > warp; --v) apply(e, warp_map[p][v][0], warp_map[p][v][1]);
        } else {
            for (int v = kScanWarps - 1; v > warp; --v) apply(u, warp_map[p][v][0], warp_map[p][v][1]);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) e[c] = u[c];
            for (int v = warp; v >= 0; --v) apply(u, warp_map[p][v][0], warp_map[p][v][1]);
        }
        for (int v = 0; v < warp; ++v) apply(h, warp_map[p][v][0], warp_map[p][v][2]);
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            e[c] = fmaf(QA[c], e[c], QU[c]);
            h[c] = fmaf(PA[c], h[c], PH[c]);
        }
#pragma unroll
        for (int j = 0; j < kScanTpt; ++j)
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                const float before = h[c];
                h[c] = fmaf(a[j][c], h[c], b[j][c]);
                b[j][c] = a[j][c] * before;  // a_t h_{t-1}
            }
        const size_t at = first(i);
#pragma unroll
        for (int j = kScanTpt - 1; j >= 0; --j) {
            if (j >= left) continue;  // past the end: the identity map, e passes through
            const int s = s0 + j * kScanThreads;
            float xv[kScanVec], zv[kScanVec], dv[kScanVec], ox[kScanVec], og[kScanVec];
            unpack4(xs[s], xv);
            unpack4(gs[s], zv);
            unpack4(ds[s], dv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                // The gate's slopes are formed again: fewer registers than kept.
                const Gated q = gate_value<kGate, kWrite, true>(zv[c], lower);
                const float et = dv[c] + e[c];
                ox[c] = q.w * et;
                float inner = b[j][c] * q.slope;
                if (kWrite != KDA_WRITE_PLAIN) inner = fmaf(q.wslope, xv[c], inner);
                og[c] = et * inner;
                e[c] = a[j][c] * et;
            }
            *reinterpret_cast<XP *>(dx + at + (size_t)j * D) = pack4<XT>(ox);
            *reinterpret_cast<GP *>(dg + at + (size_t)j * D) = pack4<GT>(og);
        }
    }
    async_wait<0>();
    if (dinit && has_ch && rank == 0 && group == 0)
        *reinterpret_cast<float4 *>(dinit + (size_t)n * D + ch) = pack4<float>(u);
}

template <typename XT, typename GT, int kGate, int kWrite>
cudaError_t launch_bwd(const ScanArgs &s, cudaStream_t stream) {
    using S = BwdShape<XT, GT>;
    auto kernel = scan_bwd<XT, GT, kGate, kWrite>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem);
    if (err != cudaSuccess) return err;
    const int blocks = (s.D + kScanCh - 1) / kScanCh;
    const long long units = (long long)s.num_seqs * blocks;
    const int ranks = scan_ranks(units, s.cu ? s.tokens : s.T_fixed, 152 * S::per_sm);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * ranks));
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = S::smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const XT *>(s.dout), s.dfinal,
                              static_cast<const XT *>(s.x), static_cast<const GT *>(s.g), (const float *)s.carries,
                              s.cu, static_cast<XT *>(s.dx), static_cast<GT *>(s.dg), s.dinit, s.T_fixed,
                              s.tokens, s.D, blocks, ranks, s.gate.lower);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanArgs &s, cudaStream_t stream) {
    return KDA_SCAN_DISPATCH(launch_bwd, s, stream);
}

}  // namespace kda
