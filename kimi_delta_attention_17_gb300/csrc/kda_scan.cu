// Gated linear recurrence over whole sequences, h_t = a_t h_{t-1} + w_t x_t per
// channel, and its single-token step.
//
// A step is the affine map h -> A h + H with (A, H) = (a_t, w_t x_t); maps
// compose associatively, (A, H) then (A', H') being (A' A, A' H + H'), so time
// is cut into pieces whose maps are formed side by side and then composed in
// order. One thread holds kTpt consecutive tokens of four channels, a CTA 32
// such pieces of 32 channels (8 lanes across, 4 pieces per warp, 8 warps), and
// a cluster of CTAs consecutive tiles of the same channels. The thread maps
// are composed by shuffles in the warp, through shared memory in the CTA and
// through distributed shared memory in the cluster; every thread then knows
// the state that enters its piece and walks it once more, from the a and w x
// still in its registers. Each input is read once and each output written
// once; the cluster goes on to its next tiles with the state it has reached.
// The composition order is fixed, so the results do not depend on the run, and
// clusters never wait for one another.
//
// Bound by HBM. Each thread's inputs arrive by asynchronous copies into slots
// of its own (no barrier), one tile ahead.
#include "kda_scan.cuh"

namespace kda {
namespace {

constexpr int kLanes = 8;                          // threads across the channels
constexpr int kBlockCh = kLanes * kScanVec;        // channels per CTA
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kGroups = kScanThreads / kLanes;     // pieces of consecutive tokens per tile
constexpr int kMaxCluster = 8;

template <typename XT, typename GT>
struct FwdShape {
    static constexpr int kTpt = sizeof(XT) == 4 ? 4 : 8;  // tokens per thread
    static constexpr int kTile = kGroups * kTpt;
    using XP = typename Piece<XT>::type;
    using GP = typename Piece<GT>::type;
    static constexpr int kStages = 2;
    static constexpr size_t smem = (size_t)kStages * kTpt * kScanThreads * (sizeof(XP) + sizeof(GP));
};

template <typename XT, typename GT, int kGate, int kWrite>
__global__ void __launch_bounds__(kScanThreads, 2)
scan_fwd(const XT *__restrict__ x, const GT *__restrict__ g, const float *init,
         const int32_t *__restrict__ cu, XT *__restrict__ out, float *final_state,
         float *__restrict__ carries, int T_fixed, long long tokens, int D, int blocks, int ranks,
         float lower) {
    using S = FwdShape<XT, GT>;
    using XP = typename S::XP;
    using GP = typename S::GP;
    constexpr int kTpt = S::kTpt;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    XP *xs = reinterpret_cast<XP *>(smem_raw);
    GP *gs = reinterpret_cast<GP *>(smem_raw + (size_t)S::kStages * kTpt * kScanThreads * sizeof(XP));
    __shared__ __align__(16) float warp_map[2][kScanWarps][2][kBlockCh];
    __shared__ __align__(16) float cta_map[2][kMaxCluster][2][kBlockCh];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? (int)cluster_rank() : 0;
    const long long unit = blockIdx.x / (unsigned)ranks;  // (sequence, channel block)
    const int n = (int)(unit / blocks);
    const int col = kScanVec * (lane & 7);
    const int ch = (int)(unit % blocks) * kBlockCh + col;
    const bool has_ch = ch < D;
    const int group = tid / kLanes;

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    const long long len = end - begin;
    const long long super = (long long)S::kTile * ranks;  // tokens per cluster step
    const long long steps = (len + super - 1) / super;

    float carry[kScanVec] = {0.f, 0.f, 0.f, 0.f};
    if (init && has_ch) unpack4(*reinterpret_cast<const float4 *>(init + (size_t)n * D + ch), carry);

    auto first_token = [&](long long i) { return (i * ranks + rank) * S::kTile + group * kTpt; };
    auto prefetch = [&](long long i) {
        const int st = (int)(i & 1);
        const long long t = first_token(i);
        if (has_ch && i < steps) {
            const size_t at = (size_t)(begin + t) * D + ch;
#pragma unroll
            for (int j = 0; j < kTpt; ++j)
                if (t + j < len) {
                    async_piece<sizeof(XP)>(&xs[(st * kTpt + j) * kScanThreads + tid], x + at + (size_t)j * D);
                    async_piece<sizeof(GP)>(&gs[(st * kTpt + j) * kScanThreads + tid], g + at + (size_t)j * D);
                }
        }
        async_commit();
    };

    prefetch(0);
    for (long long i = 0; i < steps; ++i) {
        prefetch(i + 1);
        async_wait<1>();
        const int st = (int)(i & 1);
        const long long t = first_token(i);
        float a[kTpt][kScanVec], b[kTpt][kScanVec];
        float A[kScanVec], H[kScanVec] = {0.f, 0.f, 0.f, 0.f};
        Decay decay[kScanVec];
#pragma unroll
        for (int j = 0; j < kTpt; ++j) {
            const bool valid = has_ch && t + j < len;
            float xv[kScanVec], zv[kScanVec];
            unpack4(xs[(st * kTpt + j) * kScanThreads + tid], xv);
            unpack4(gs[(st * kTpt + j) * kScanThreads + tid], zv);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                const Gated q = gate_value<kGate, kWrite, false>(zv[c], lower);
                a[j][c] = valid ? q.a : 1.f;  // past the end: the identity map
                b[j][c] = valid ? q.w * xv[c] : 0.f;
                H[c] = fmaf(a[j][c], H[c], b[j][c]);
                decay[c].then(a[j][c], valid ? q.c : 0.f);
            }
        }
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) A[c] = decay[c].value();
        // Inclusive composition over the warp's four pieces, then each piece's
        // predecessors alone (PA, PH).
        float PA[kScanVec], PH[kScanVec];
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
#pragma unroll
            for (int off = kLanes; off < 32; off <<= 1) {
                const float A2 = __shfl_up_sync(0xffffffffu, A[c], off);
                const float H2 = __shfl_up_sync(0xffffffffu, H[c], off);
                if (lane >= off) {
                    H[c] = fmaf(A[c], H2, H[c]);
                    A[c] *= A2;
                }
            }
            PA[c] = __shfl_up_sync(0xffffffffu, A[c], kLanes);
            PH[c] = __shfl_up_sync(0xffffffffu, H[c], kLanes);
            if (lane < kLanes) {
                PA[c] = 1.f;
                PH[c] = 0.f;
            }
        }
        const int p = (int)(i & 1);
        if (lane >= 32 - kLanes) {
            *reinterpret_cast<float4 *>(&warp_map[p][warp][0][col]) = pack4<float>(A);
            *reinterpret_cast<float4 *>(&warp_map[p][warp][1][col]) = pack4<float>(H);
        }
        __syncthreads();
        // This warp's predecessors in the CTA (WA, WH), and the CTA's own map.
        float WA[kScanVec], WH[kScanVec], TA[kScanVec], TH[kScanVec];
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            WA[c] = TA[c] = 1.f;
            WH[c] = TH[c] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < kScanWarps; ++v) {
            float A2[kScanVec], H2[kScanVec];
            unpack4(*reinterpret_cast<const float4 *>(&warp_map[p][v][0][col]), A2);
            unpack4(*reinterpret_cast<const float4 *>(&warp_map[p][v][1][col]), H2);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                if (v == warp) {
                    WA[c] = TA[c];
                    WH[c] = TH[c];
                }
                TH[c] = fmaf(A2[c], TH[c], H2[c]);
                TA[c] *= A2[c];
            }
        }
        float h[kScanVec];
        if (ranks == 1) {
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) {
                h[c] = carry[c];
                carry[c] = fmaf(TA[c], carry[c], TH[c]);
            }
        } else {
            // Every CTA sends its map to every CTA of the cluster. The two
            // buffers alternate: a CTA writes into one again only after a
            // barrier that all arrive at having read it.
            if (warp == 0)
                for (int r = lane / kLanes; r < ranks; r += 32 / kLanes) {
                    store_peer4((uint32_t)__cvta_generic_to_shared(&cta_map[p][rank][0][col]), r, TA);
                    store_peer4((uint32_t)__cvta_generic_to_shared(&cta_map[p][rank][1][col]), r, TH);
                }
            cluster_sync();
            for (int r = 0; r < ranks; ++r) {
                float A2[kScanVec], H2[kScanVec];
                unpack4(*reinterpret_cast<const float4 *>(&cta_map[p][r][0][col]), A2);
                unpack4(*reinterpret_cast<const float4 *>(&cta_map[p][r][1][col]), H2);
#pragma unroll
                for (int c = 0; c < kScanVec; ++c) {
                    if (r == rank) h[c] = carry[c];
                    carry[c] = fmaf(A2[c], carry[c], H2[c]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            h[c] = fmaf(WA[c], h[c], WH[c]);
            h[c] = fmaf(PA[c], h[c], PH[c]);
        }
        if (carries && has_ch && t < len && t % KDA_SCAN_CARRY_TOKENS == 0)
            *reinterpret_cast<float4 *>(carries + (size_t)carry_row(begin, n, t / KDA_SCAN_CARRY_TOKENS) * D + ch) =
                pack4<float>(h);
        XT *o = out + (size_t)(begin + t) * D + ch;
#pragma unroll
        for (int j = 0; j < kTpt; ++j) {
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) h[c] = fmaf(a[j][c], h[c], b[j][c]);
            if (has_ch && t + j < len) *reinterpret_cast<XP *>(o + (size_t)j * D) = pack4<XT>(h);
        }
    }
    async_wait<0>();
    if (final_state && has_ch && rank == 0 && group == 0)
        *reinterpret_cast<float4 *>(final_state + (size_t)n * D + ch) = pack4<float>(carry);
}

template <typename XT, typename GT, int kGate, int kWrite>
cudaError_t launch_fwd(const ScanArgs &s, cudaStream_t stream) {
    using S = FwdShape<XT, GT>;
    auto kernel = scan_fwd<XT, GT, kGate, kWrite>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem);
    if (err != cudaSuccess) return err;
    const int blocks = (s.D + kBlockCh - 1) / kBlockCh;
    const long long units = (long long)s.num_seqs * blocks;
    const int ranks = scan_ranks(units, s.cu ? s.tokens : s.T_fixed, S::kTile);
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
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const XT *>(s.x), static_cast<const GT *>(s.g), s.init,
                              s.cu, static_cast<XT *>(s.out), s.final_state, s.carries, s.T_fixed, s.tokens,
                              s.D, blocks, ranks, s.gate.lower);
}

// One step: a thread per four channels of a row.
constexpr int kStepThreads = 128;
template <typename XT, typename GT, int kGate, int kWrite>
__global__ void __launch_bounds__(kStepThreads)
scan_step(const XT *__restrict__ x, const GT *__restrict__ g, float *__restrict__ state,
          const int32_t *__restrict__ slots, XT *__restrict__ out, long long pieces, int per_row, int num_slots,
          float lower) {
    const long long i = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    if (i >= pieces) return;
    const int n = (int)(i / per_row), c4 = (int)(i % per_row);
    const long long slot = slots ? slots[n] : n;
    const size_t at = (size_t)i * kScanVec;
    float h[kScanVec] = {0.f, 0.f, 0.f, 0.f};
    if (slot >= 0 && slot < num_slots) {
        float xv[kScanVec], zv[kScanVec];
        float4 *sp = reinterpret_cast<float4 *>(state) + (size_t)slot * per_row + c4;
        unpack4(*sp, h);
        unpack4(*reinterpret_cast<const typename Piece<XT>::type *>(x + at), xv);
        unpack4(*reinterpret_cast<const typename Piece<GT>::type *>(g + at), zv);
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            const Gated q = gate_value<kGate, kWrite, false>(zv[c], lower);
            h[c] = fmaf(q.a, h[c], q.w * xv[c]);
        }
        *sp = pack4<float>(h);
    }
    *reinterpret_cast<typename Piece<XT>::type *>(out + at) = pack4<XT>(h);
}

template <typename XT, typename GT, int kGate, int kWrite>
cudaError_t launch_step(const ScanStepArgs &s, cudaStream_t stream) {
    const int per_row = s.D / kScanVec;
    const long long pieces = (long long)s.N * per_row;
    const long long grid = (pieces + kStepThreads - 1) / kStepThreads;
    scan_step<XT, GT, kGate, kWrite><<<(unsigned)grid, kStepThreads, 0, stream>>>(
        static_cast<const XT *>(s.x), static_cast<const GT *>(s.g), s.state, s.slots, static_cast<XT *>(s.out),
        pieces, per_row, s.num_slots, s.gate.lower);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &s, cudaStream_t stream) {
    return KDA_SCAN_DISPATCH(launch_fwd, s, stream);
}

cudaError_t launch_scan_step(const ScanStepArgs &s, cudaStream_t stream) {
    if (s.N == 0) return cudaSuccess;
    return KDA_SCAN_DISPATCH(launch_step, s, stream);
}

}  // namespace kda
