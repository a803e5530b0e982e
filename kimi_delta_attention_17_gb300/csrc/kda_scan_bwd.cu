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

constexpr int kLanes = 8;                    // threads across the channels
constexpr int kBlockCh = kLanes * kScanVec;  // channels per CTA
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kGroups = kScanThreads / kLanes;
constexpr int kTpt = 4;  // tokens per thread
constexpr int kTile = kGroups * kTpt;
constexpr int kMaxCluster = 8;
constexpr int kStages = 2;
static_assert(kTile == KDA_SCAN_CARRY_TOKENS, "a tile begins at a saved state");

template <typename XT, typename GT>
struct BwdShape {
    using XP = typename Piece<XT>::type;
    using GP = typename Piece<GT>::type;
    static constexpr size_t slots = (size_t)kStages * kTpt * kScanThreads;
    static constexpr size_t smem = slots * (2 * sizeof(XP) + sizeof(GP));
};

template <typename XT, typename GT, int kGate, int kWrite>
__global__ void __launch_bounds__(kScanThreads, 2)
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
    __shared__ __align__(16) float warp_map[2][kScanWarps][3][kBlockCh];  // A, H (forward), U (backward)
    __shared__ __align__(16) float cta_map[2][kMaxCluster][2][kBlockCh];  // A, U

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? (int)cluster_rank() : 0;
    const long long unit = blockIdx.x / (unsigned)ranks;
    const int n = (int)(unit / blocks);
    const int col = kScanVec * (lane & 7);
    const int ch = (int)(unit % blocks) * kBlockCh + col;
    const bool has_ch = ch < D;
    const int group = tid / kLanes;

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    const long long len = end - begin;
    const long long super = (long long)kTile * ranks;
    const long long steps = (len + super - 1) / super;

    float u[kScanVec] = {0.f, 0.f, 0.f, 0.f};  // the gradient entering the cluster's tiles from behind
    if (dfinal && has_ch) unpack4(*reinterpret_cast<const float4 *>(dfinal + (size_t)n * D + ch), u);

    auto tile_of = [&](long long i) { return i * ranks + rank; };
    auto prefetch = [&](long long i) {
        const int st = (int)(i & 1);
        const long long t = tile_of(i) * kTile + group * kTpt;
        if (has_ch && i >= 0) {
            const size_t at = (size_t)(begin + t) * D + ch;
#pragma unroll
            for (int j = 0; j < kTpt; ++j)
                if (t + j < len) {
                    const int s = (st * kTpt + j) * kScanThreads + tid;
                    async_piece<sizeof(GP)>(&gs[s], g + at + (size_t)j * D);
                    async_piece<sizeof(XP)>(&ds[s], dout + at + (size_t)j * D);
                    async_piece<sizeof(XP)>(&xs[s], x + at + (size_t)j * D);
                }
        }
        async_commit();
    };

    prefetch(steps - 1);
    for (long long i = steps - 1; i >= 0; --i) {
        const int st = (int)(i & 1), p = st;
        const long long t = tile_of(i) * kTile + group * kTpt;
        float h[kScanVec] = {0.f, 0.f, 0.f, 0.f};  // the state entering this CTA's tile
        if (has_ch && tile_of(i) * kTile < len)
            unpack4(*reinterpret_cast<const float4 *>(carries + (size_t)carry_row(begin, n, tile_of(i)) * D + ch), h);
        prefetch(i - 1);
        async_wait<1>();
        Gated q[kTpt][kScanVec];
        float A[kScanVec], B[kScanVec];
        float H[kScanVec] = {0.f, 0.f, 0.f, 0.f}, U[kScanVec] = {0.f, 0.f, 0.f, 0.f};
        Decay decay[kScanVec];
#pragma unroll
        for (int j = 0; j < kTpt; ++j) {
            const int s = (st * kTpt + j) * kScanThreads + tid;
            const bool valid = has_ch && t + j < len;
            float xv[kScanVec], zv[kScanVec];
            unpack4(xs[s], xv);
            unpack4(gs[s], zv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                q[j][c] = gate_value<kGate, kWrite, true>(zv[c], lower);
                q[j][c].a = valid ? q[j][c].a : 1.f;
                H[c] = fmaf(q[j][c].a, H[c], valid ? q[j][c].w * xv[c] : 0.f);
                decay[c].then(q[j][c].a, valid ? q[j][c].c : 0.f);
            }
        }
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) A[c] = decay[c].value();
#pragma unroll
        for (int j = kTpt - 1; j >= 0; --j) {
            const bool valid = has_ch && t + j < len;
            float dv[kScanVec];
            unpack4(ds[(st * kTpt + j) * kScanThreads + tid], dv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) U[c] = q[j][c].a * ((valid ? dv[c] : 0.f) + U[c]);
        }
        // In the warp: predecessors alone (PA, PH) for the states, successors
        // alone (QA, QU) for the gradients.
        float PA[kScanVec], PH[kScanVec], QA[kScanVec], QU[kScanVec];
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            B[c] = A[c];
#pragma unroll
            for (int off = kLanes; off < 32; off <<= 1) {
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
            PA[c] = __shfl_up_sync(0xffffffffu, A[c], kLanes);
            PH[c] = __shfl_up_sync(0xffffffffu, H[c], kLanes);
            QA[c] = __shfl_down_sync(0xffffffffu, B[c], kLanes);
            QU[c] = __shfl_down_sync(0xffffffffu, U[c], kLanes);
            if (lane < kLanes) {
                PA[c] = 1.f;
                PH[c] = 0.f;
            }
            if (lane >= 32 - kLanes) {
                QA[c] = 1.f;
                QU[c] = 0.f;
            }
        }
        if (lane >= 32 - kLanes) {
            *reinterpret_cast<float4 *>(&warp_map[p][warp][0][col]) = pack4<float>(A);
            *reinterpret_cast<float4 *>(&warp_map[p][warp][1][col]) = pack4<float>(H);
        }
        if (lane < kLanes) *reinterpret_cast<float4 *>(&warp_map[p][warp][2][col]) = pack4<float>(U);
        __syncthreads();
        float WA[kScanVec], WU[kScanVec], TA[kScanVec], TU[kScanVec];
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            WA[c] = TA[c] = 1.f;
            WU[c] = TU[c] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < kScanWarps; ++v) {
            if (v >= warp) break;
            float A2[kScanVec], H2[kScanVec];
            unpack4(*reinterpret_cast<const float4 *>(&warp_map[p][v][0][col]), A2);
            unpack4(*reinterpret_cast<const float4 *>(&warp_map[p][v][1][col]), H2);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) h[c] = fmaf(A2[c], h[c], H2[c]);
        }
#pragma unroll
        for (int v = kScanWarps - 1; v >= 0; --v) {
            float A2[kScanVec], U2[kScanVec];
            unpack4(*reinterpret_cast<const float4 *>(&warp_map[p][v][0][col]), A2);
            unpack4(*reinterpret_cast<const float4 *>(&warp_map[p][v][2][col]), U2);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                if (v == warp) {
                    WA[c] = TA[c];
                    WU[c] = TU[c];
                }
                TU[c] = fmaf(A2[c], TU[c], U2[c]);
                TA[c] *= A2[c];
            }
        }
        float e[kScanVec];  // the gradient entering this thread's last token from behind
        if (ranks == 1) {
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                e[c] = u[c];
                u[c] = fmaf(TA[c], u[c], TU[c]);
            }
        } else {
            if (warp == 0)
                for (int r = lane / kLanes; r < ranks; r += 32 / kLanes) {
                    store_peer4((uint32_t)__cvta_generic_to_shared(&cta_map[p][rank][0][col]), r, TA);
                    store_peer4((uint32_t)__cvta_generic_to_shared(&cta_map[p][rank][1][col]), r, TU);
                }
            cluster_sync();
            for (int r = ranks - 1; r >= 0; --r) {
                float A2[kScanVec], U2[kScanVec];
                unpack4(*reinterpret_cast<const float4 *>(&cta_map[p][r][0][col]), A2);
                unpack4(*reinterpret_cast<const float4 *>(&cta_map[p][r][1][col]), U2);
#pragma unroll
                for (int c = 0; c < kScanVec; ++c) {
                    if (r == rank) e[c] = u[c];
                    u[c] = fmaf(A2[c], u[c], U2[c]);
                }
            }
        }
        float before[kTpt][kScanVec];  // h_{t-1}
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            e[c] = fmaf(WA[c], e[c], WU[c]);
            e[c] = fmaf(QA[c], e[c], QU[c]);
            h[c] = fmaf(PA[c], h[c], PH[c]);
        }
#pragma unroll
        for (int j = 0; j < kTpt; ++j) {
            float xv[kScanVec];
            unpack4(xs[(st * kTpt + j) * kScanThreads + tid], xv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                before[j][c] = h[c];
                h[c] = fmaf(q[j][c].a, h[c], q[j][c].w * xv[c]);
            }
        }
#pragma unroll
        for (int j = kTpt - 1; j >= 0; --j) {
            const int s = (st * kTpt + j) * kScanThreads + tid;
            const bool valid = has_ch && t + j < len;
            if (!valid) continue;  // the identity map: e passes through
            float xv[kScanVec], dv[kScanVec], ox[kScanVec], og[kScanVec];
            unpack4(xs[s], xv);
            unpack4(ds[s], dv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                const Gated &r = q[j][c];
                const float et = dv[c] + e[c];
                ox[c] = r.w * et;
                float inner = r.a * before[j][c] * r.slope;
                if (kWrite != KDA_WRITE_PLAIN) inner = fmaf(r.wslope, xv[c], inner);
                og[c] = et * inner;
                e[c] = r.a * et;
            }
            const size_t at = (size_t)(begin + t + j) * D + ch;
            *reinterpret_cast<XP *>(dx + at) = pack4<XT>(ox);
            *reinterpret_cast<GP *>(dg + at) = pack4<GT>(og);
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
    const int blocks = (s.D + kBlockCh - 1) / kBlockCh;
    const long long units = (long long)s.num_seqs * blocks;
    const int ranks = scan_ranks(units, s.cu ? s.tokens : s.T_fixed, kTile);
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
