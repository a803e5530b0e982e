// Gated linear recurrence over whole sequences, h_t = a_t h_{t-1} + w_t x_t per
// channel, and its single-token step.
//
// A step is the affine map h -> A h + H with (A, H) = (a_t, w_t x_t); maps
// compose associatively, (A, H) then (A', H') being (A' A, A' H + H'), so time
// is cut into pieces whose maps are formed side by side and then composed in
// order. One thread holds 8 consecutive tokens of four channels, a CTA 16 such
// pieces of 32 channels (8 lanes across, 4 pieces per warp, 4 warps), and a
// cluster of CTAs consecutive tiles of the same channels. The thread maps
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

template <typename XT, typename GT>
struct FwdShape {
    using XP = typename Piece<XT>::type;
    using GP = typename Piece<GT>::type;
    static constexpr size_t slots = (size_t)kScanStages * kScanTpt * kScanThreads;
    static constexpr size_t smem = slots * (sizeof(XP) + sizeof(GP));
    static constexpr int per_sm = smem <= 50 * 1024 ? 4 : 3;  // CTAs
};

template <typename XT, typename GT, int kGate, int kWrite>
__global__ void __launch_bounds__(kScanThreads, FwdShape<XT, GT>::per_sm)
scan_fwd(const XT *__restrict__ x, const GT *__restrict__ g, const float *init,
         const int32_t *__restrict__ cu, XT *__restrict__ out, float *final_state,
         float *__restrict__ carries, int T_fixed, long long tokens, int D, int blocks, int ranks,
         float lower) {
    using S = FwdShape<XT, GT>;
    using XP = typename S::XP;
    using GP = typename S::GP;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    GP *gs = reinterpret_cast<GP *>(smem_raw);
    XP *xs = reinterpret_cast<XP *>(smem_raw + S::slots * sizeof(GP));
    __shared__ __align__(16) float warp_map[2][kScanWarps][2][kScanCh];    // (A, H) of each warp
    __shared__ __align__(16) float cta_map[2][kScanMaxRanks][2][kScanCh];  // and of each CTA

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? (int)cluster_rank() : 0;
    const unsigned unit = blockIdx.x / (unsigned)ranks;  // (sequence, channel block)
    const int n = (int)(unit / (unsigned)blocks);
    const int col = kScanVec * (lane & (kScanLanes - 1));
    const int ch = (int)(unit % (unsigned)blocks) * kScanCh + col;
    const bool has_ch = ch < D;
    const int group = tid / kScanLanes;

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    const int len = (int)(end - begin);
    const int super = kScanTile * ranks;  // tokens per cluster step
    const int steps = (int)(((long long)len + super - 1) / super);

    float carry[kScanVec] = {0.f, 0.f, 0.f, 0.f};
    if (init && has_ch) unpack4(*reinterpret_cast<const float4 *>(init + (size_t)n * D + ch), carry);

    // Tokens of this thread in step i that lie before the sequence's end.
    auto tokens_left = [&](int i) {
        const long long t = ((long long)i * ranks + rank) * kScanTile + group * kScanTpt;
        return has_ch ? (int)min(max(len - t, 0LL), (long long)kScanTpt) : 0;
    };
    size_t at = (size_t)(begin + (long long)rank * kScanTile + group * kScanTpt) * D + ch;  // first element of a step
    const size_t stride = (size_t)super * D;
    auto prefetch = [&](int i, size_t from) {
        const int left = i < steps ? tokens_left(i) : 0;
        const int s0 = (i & 1) * kScanTpt * kScanThreads + tid;
        if (left == kScanTpt) {
#pragma unroll
            for (int j = 0; j < kScanTpt; ++j) {
                async_piece<sizeof(GP)>(&gs[s0 + j * kScanThreads], g + from + (size_t)j * D);
                async_piece<sizeof(XP)>(&xs[s0 + j * kScanThreads], x + from + (size_t)j * D);
            }
        } else if (i < steps) {
            const float id = identity_gate<kGate>(), z[4] = {id, id, id, id}, zero[4] = {0.f, 0.f, 0.f, 0.f};
            for (int j = 0; j < kScanTpt; ++j) {
                if (j < left) {
                    async_piece<sizeof(GP)>(&gs[s0 + j * kScanThreads], g + from + (size_t)j * D);
                    async_piece<sizeof(XP)>(&xs[s0 + j * kScanThreads], x + from + (size_t)j * D);
                } else {
                    gs[s0 + j * kScanThreads] = pack4<GT>(z);
                    xs[s0 + j * kScanThreads] = pack4<XT>(zero);
                }
            }
        }
        async_commit();
    };

    prefetch(0, at);
    for (int i = 0; i < steps; ++i, at += stride) {
        prefetch(i + 1, at + stride);
        async_wait<1>();
        const int p = i & 1, left = tokens_left(i);
        const int s0 = p * kScanTpt * kScanThreads + tid;
        float a[kScanTpt][kScanVec], b[kScanTpt][kScanVec];
        float A[kScanVec], H[kScanVec] = {0.f, 0.f, 0.f, 0.f};
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
        // Inclusive composition over the warp's four pieces, then each piece's
        // predecessors alone (PA, PH).
        float PA[kScanVec], PH[kScanVec];
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) {
            A[c] = decay[c].value();
#pragma unroll
            for (int off = kScanLanes; off < 32; off <<= 1) {
                const float A2 = __shfl_up_sync(0xffffffffu, A[c], off);
                const float H2 = __shfl_up_sync(0xffffffffu, H[c], off);
                if (lane >= off) {
                    H[c] = fmaf(A[c], H2, H[c]);
                    A[c] *= A2;
                }
            }
            PA[c] = __shfl_up_sync(0xffffffffu, A[c], kScanLanes);
            PH[c] = __shfl_up_sync(0xffffffffu, H[c], kScanLanes);
            if (lane < kScanLanes) {
                PA[c] = 1.f;
                PH[c] = 0.f;
            }
        }
        // The maps' buffers alternate between steps: one is written again only
        // after a barrier that every reader of it has arrived at.
        if (lane >= 32 - kScanLanes) {
            *reinterpret_cast<float4 *>(&warp_map[p][warp][0][col]) = pack4<float>(A);
            *reinterpret_cast<float4 *>(&warp_map[p][warp][1][col]) = pack4<float>(H);
        }
        __syncthreads();
        float h[kScanVec];
        auto apply = [&](float *state, const float (*map)[kScanCh]) {
            float A2[kScanVec], H2[kScanVec];
            unpack4(*reinterpret_cast<const float4 *>(&map[0][col]), A2);
            unpack4(*reinterpret_cast<const float4 *>(&map[1][col]), H2);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) state[c] = fmaf(A2[c], state[c], H2[c]);
        };
        if (ranks > 1) {
            if (warp == 0) {  // one lane per channel: the CTA's map, sent to every CTA of the cluster
                float TA = 1.f, TH = 0.f;
#pragma unroll
                for (int v = 0; v < kScanWarps; ++v) {
                    const float A2 = warp_map[p][v][0][lane];
                    TH = fmaf(A2, TH, warp_map[p][v][1][lane]);
                    TA *= A2;
                }
                for (int r = 0; r < ranks; ++r) {
                    store_peer(&cta_map[p][rank][0][lane], r, TA);
                    store_peer(&cta_map[p][rank][1][lane], r, TH);
                }
            }
            cluster_sync();
            for (int r = 0; r < rank; ++r) apply(carry, cta_map[p][r]);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) h[c] = carry[c];
            for (int r = rank; r < ranks; ++r) apply(carry, cta_map[p][r]);
            for (int v = 0; v < warp; ++v) apply(h, warp_map[p][v]);
        } else {
            for (int v = 0; v < warp; ++v) apply(carry, warp_map[p][v]);
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) h[c] = carry[c];
            for (int v = warp; v < kScanWarps; ++v) apply(carry, warp_map[p][v]);
        }
#pragma unroll
        for (int c = 0; c < kScanVec; ++c) h[c] = fmaf(PA[c], h[c], PH[c]);
        if (carries && group == 0 && left > 0)
            *reinterpret_cast<float4 *>(carries + (size_t)carry_row(begin, n, (long long)i * ranks + rank) * D + ch) =
                pack4<float>(h);
        XT *o = out + at;
#pragma unroll
        for (int j = 0; j < kScanTpt; ++j) {
#pragma unroll
            for (int c = 0; c < kScanVec; ++c) h[c] = fmaf(a[j][c], h[c], b[j][c]);
            if (j < left) *reinterpret_cast<XP *>(o + (size_t)j * D) = pack4<XT>(h);
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
