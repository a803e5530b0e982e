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

#ifndef FWD_STAGES
#define FWD_STAGES 2
#endif
struct FwdShared {
    float map[kScanGroups][2][kScanCh];       // (A, H) of each piece; then H gives way to the state entering it
    float2 warp_map[2][kScanWarps][kScanCh];  // (A, H) of each warp's tokens
    ClusterMaps peers;
};
template <typename XT, typename GT>
struct FwdShape {
    using XP = typename Piece<XT>::type;
    using GP = typename Piece<GT>::type;
    static constexpr int stages = FWD_STAGES;
    static constexpr size_t slots = (size_t)stages * kScanTpt * kScanThreads;
    static constexpr size_t smem = slots * (sizeof(XP) + sizeof(GP));
    static constexpr int fit = (int)(kSmSmem / (smem + sizeof(FwdShared) + kCtaReserved));
    static constexpr int per_sm = kScanTpt == 4 ? (fit < 3 ? fit : 3) : (fit < 4 ? fit : 4);  // CTAs
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
    __shared__ __align__(16) FwdShared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? (int)cluster_rank() : 0;
    const unsigned unit = blockIdx.x / (unsigned)ranks;  // (sequence, channel block)
    const int n = (int)(unit / (unsigned)blocks);
    const int ch0 = (int)(unit % (unsigned)blocks) * kScanCh;
    const int col = kScanVec * (lane & (kScanLanes - 1));
    const int ch = ch0 + col;
    const bool has_ch = ch < D;
    const int group = tid / kScanLanes;
    // In every warp, lane = channel: the state at the cluster's next tiles. Read
    // before the cluster's first barrier: final_state may be the same memory.
    float carry = init && ch0 + lane < D ? init[(size_t)n * D + ch0 + lane] : 0.f;
    if (ranks > 1) cluster_maps_init(sh.peers);

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    const int len = (int)(end - begin);
    const int super = kScanTile * ranks;  // tokens per cluster step
    const int steps = (int)(((long long)len + super - 1) / super);

    // Of this step: tokens from this thread's first one to the sequence's end
    // (none left where negative), and the first one's element.
    int left = has_ch ? len - (rank * kScanTile + group * kScanTpt) : -1;
    const int less = has_ch ? super : 0;
    size_t at = (size_t)(begin + (long long)rank * kScanTile + group * kScanTpt) * D + ch;
    const size_t stride = (size_t)super * D;
    auto prefetch = [&](int i, int left, size_t from) {
        const int s0 = i % S::stages * kScanTpt * kScanThreads + tid;
        const GT *gp = g + from;
        const XT *xp = x + from;
        if (left >= kScanTpt) {
#pragma unroll
            for (int j = 0; j < kScanTpt; ++j) {
                async_piece<sizeof(GP)>(&gs[s0 + j * kScanThreads], gp + (size_t)j * D);
                async_piece<sizeof(XP)>(&xs[s0 + j * kScanThreads], xp + (size_t)j * D);
            }
        } else if (i < steps) {
            const F2 id = f2(identity_gate<kGate>()), z[2] = {id, id}, zero[2] = {{0}, {0}};
            for (int j = 0; j < kScanTpt; ++j) {
                if (j < left) {
                    async_piece<sizeof(GP)>(&gs[s0 + j * kScanThreads], gp + (size_t)j * D);
                    async_piece<sizeof(XP)>(&xs[s0 + j * kScanThreads], xp + (size_t)j * D);
                } else {
                    gs[s0 + j * kScanThreads] = pack4<GT>(z);
                    xs[s0 + j * kScanThreads] = pack4<XT>(zero);
                }
            }
        }
        async_commit();
    };

#pragma unroll
    for (int i = 0; i < S::stages; ++i) prefetch(i, left - i * less, at + i * stride);
    for (int i = 0; i < steps; ++i, at += stride, left -= less) {
        async_wait<S::stages - 1>();
        const int s0 = i % S::stages * kScanTpt * kScanThreads + tid;
        F2 a[kScanTpt][kScanPairs], b[kScanTpt][kScanPairs];
        {
            F2 A[kScanPairs], H[kScanPairs] = {{0}, {0}};
            Decay<kGate> decay[kScanPairs];
#pragma unroll
            for (int j = 0; j < kScanTpt; ++j) {
                F2 xv[kScanPairs], zv[kScanPairs];
                unpack4(xs[s0 + j * kScanThreads], xv);
                unpack4(gs[s0 + j * kScanThreads], zv);
#pragma unroll
                for (int c = 0; c < kScanPairs; ++c) {
                    const Gated q = gate_value<kGate, kWrite>(zv[c], lower);
                    a[j][c] = q.a;
                    b[j][c] = written<kWrite>(q.a, q.c, xv[c]);
                    H[c] = fma2(q.a, H[c], b[j][c]);
                    decay[c].then(q);
                }
            }
#pragma unroll
            for (int c = 0; c < kScanPairs; ++c) A[c] = decay[c].value();
            *reinterpret_cast<float4 *>(&sh.map[group][0][col]) = pack4<float>(A);
            *reinterpret_cast<float4 *>(&sh.map[group][1][col]) = pack4<float>(H);
        }
        prefetch(i + S::stages, left - S::stages * less, at + S::stages * stride);  // into the slots just read
        // Lane = channel: the warp's pieces are composed in order.
        __syncwarp();
        float A[kWarpGroups], H[kWarpGroups];
        {
            float PA = 1.f, PH = 0.f;
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                A[v] = sh.map[warp * kWarpGroups + v][0][lane];
                H[v] = sh.map[warp * kWarpGroups + v][1][lane];
            }
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                PH = fmaf(A[v], PH, H[v]);
                PA *= A[v];
            }
            sh.warp_map[i & 1][warp][lane] = make_float2(PA, PH);
        }
        __syncthreads();  // warp_map's halves alternate: the only barrier of a step
        {
            float2 m[kScanWarps];
#pragma unroll
            for (int v = 0; v < kScanWarps; ++v) m[v] = sh.warp_map[i & 1][v][lane];
            float first = carry;  // the state entering the CTA's tile
            if (ranks > 1) {
                if (warp == 0) {
                    float TA = 1.f, TH = 0.f;
#pragma unroll
                    for (int v = 0; v < kScanWarps; ++v) {
                        TH = fmaf(m[v].x, TH, m[v].y);
                        TA *= m[v].x;
                    }
                    cluster_maps_send(sh.peers, i, rank, ranks, TA, TH);
                }
                if (!cluster_maps_wait(sh.peers, i)) carry = __uint_as_float(0x7fc00000u);
                for (int r = 0; r < ranks; ++r) {
                    if (r == rank) first = carry;
                    const float2 t = sh.peers.map[i & 1][r][lane];
                    carry = fmaf(t.x, carry, t.y);
                }
            }
            // The tile begins at a token whose entering state the backward pass needs.
            const long long tile = (long long)i * ranks + rank;
            if (carries && warp == 0 && tile * kScanTile < len && ch0 + lane < D)
                carries[(size_t)carry_row(begin, n, tile) * D + ch0 + lane] = first;
            float mine = 0.f;  // the state entering the warp's tokens
#pragma unroll
            for (int v = 0; v < kScanWarps; ++v) {
                if (v == warp) mine = first;
                first = fmaf(m[v].x, first, m[v].y);
            }
            if (ranks == 1) carry = first;
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                sh.map[warp * kWarpGroups + v][1][lane] = mine;
                mine = fmaf(A[v], mine, H[v]);
            }
        }
        __syncwarp();
        F2 h[kScanPairs];
        unpack4(*reinterpret_cast<const float4 *>(&sh.map[group][1][col]), h);
        XT *o = out + at;
#pragma unroll
        for (int j = 0; j < kScanTpt; ++j) {
#pragma unroll
            for (int c = 0; c < kScanPairs; ++c) h[c] = fma2(a[j][c], h[c], b[j][c]);
            if (j < left) *reinterpret_cast<XP *>(o + (size_t)j * D) = pack4<XT>(h);
        }
    }
    async_wait<0>();
    if (final_state && warp == 0 && rank == 0 && ch0 + lane < D) final_state[(size_t)n * D + ch0 + lane] = carry;
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
    F2 h[kScanPairs] = {{0}, {0}};
    if (slot >= 0 && slot < num_slots) {
        F2 xv[kScanPairs], zv[kScanPairs];
        float4 *sp = reinterpret_cast<float4 *>(state) + (size_t)slot * per_row + c4;
        unpack4(*sp, h);
        unpack4(*reinterpret_cast<const typename Piece<XT>::type *>(x + at), xv);
        unpack4(*reinterpret_cast<const typename Piece<GT>::type *>(g + at), zv);
#pragma unroll
        for (int c = 0; c < kScanPairs; ++c) {
            const Gated q = gate_value<kGate, kWrite>(zv[c], lower);
            h[c] = fma2(q.a, h[c], written<kWrite>(q.a, q.c, xv[c]));
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
