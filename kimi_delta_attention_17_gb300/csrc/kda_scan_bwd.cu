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

#ifndef BWD_STAGES
#define BWD_STAGES 2
#endif
struct BwdShared {
    float map[kScanGroups][3][kScanCh];          // A, H, U of each piece; then the state and the gradient entering it
    float warp_map[2][3][kScanWarps][kScanCh];   // A, H, U of each warp's tokens
    ClusterMaps peers;
};
template <typename XT, typename GT>
struct BwdShape {
    using XP = typename Piece<XT>::type;
    using GP = typename Piece<GT>::type;
    static constexpr int stages = BWD_STAGES;
    static constexpr size_t slots = (size_t)stages * kScanTpt * kScanThreads;
    static constexpr size_t smem = slots * (2 * sizeof(XP) + sizeof(GP));
    static constexpr int fit = (int)(kSmSmem / (smem + sizeof(BwdShared) + kCtaReserved));
    static constexpr int per_sm = kScanTpt == 4 ? (fit < 3 ? fit : 3) : (fit < 4 ? fit : 4);  // CTAs
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
    __shared__ __align__(16) BwdShared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = ranks > 1 ? (int)cluster_rank() : 0;
    const unsigned unit = blockIdx.x / (unsigned)ranks;
    const int n = (int)(unit / (unsigned)blocks);
    const int ch0 = (int)(unit % (unsigned)blocks) * kScanCh;
    const int col = kScanVec * (lane & (kScanLanes - 1));
    const int ch = ch0 + col;
    const bool has_ch = ch < D, lane_ch = ch0 + lane < D;
    const int group = tid / kScanLanes;
    // In every warp, lane = channel: the gradient entering the cluster's tiles
    // from behind. Read before the cluster's first barrier: dinit may be the
    // same memory.
    float u = dfinal && lane_ch ? dfinal[(size_t)n * D + ch0 + lane] : 0.f;
    if (ranks > 1) cluster_maps_init(sh.peers);

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    const int len = (int)(end - begin);
    const int super = kScanTile * ranks;
    const int steps = (int)(((long long)len + super - 1) / super);

    // Of a step: tokens from this thread's first one to the sequence's end (none
    // left where negative), and the first one's element.
    const long long t0 = ((long long)(steps - 1) * ranks + rank) * kScanTile + group * kScanTpt;
    int left = has_ch ? (int)(len - t0) : -1;
    const int more = has_ch ? super : 0;
    size_t at = (size_t)(begin + t0) * D + ch;
    const size_t stride = (size_t)super * D;
    auto prefetch = [&](int i, int left, size_t from) {
        const int s0 = (i + S::stages) % S::stages * kScanTpt * kScanThreads + tid;
        const GT *gp = g + from;
        const XT *xp = x + from, *dp = dout + from;
        if (i >= 0 && left >= kScanTpt) {
#pragma unroll
            for (int j = 0; j < kScanTpt; ++j) {
                const int s = s0 + j * kScanThreads;
                async_piece<sizeof(GP)>(&gs[s], gp + (size_t)j * D);
                async_piece<sizeof(XP)>(&ds[s], dp + (size_t)j * D);
                async_piece<sizeof(XP)>(&xs[s], xp + (size_t)j * D);
            }
        } else if (i >= 0) {
            const F2 id = f2(identity_gate<kGate>()), z[2] = {id, id}, zero[2] = {{0}, {0}};
            for (int j = 0; j < kScanTpt; ++j) {
                const int s = s0 + j * kScanThreads;
                if (j < left) {
                    async_piece<sizeof(GP)>(&gs[s], gp + (size_t)j * D);
                    async_piece<sizeof(XP)>(&ds[s], dp + (size_t)j * D);
                    async_piece<sizeof(XP)>(&xs[s], xp + (size_t)j * D);
                } else {
                    gs[s] = pack4<GT>(z);
                    ds[s] = xs[s] = pack4<XT>(zero);
                }
            }
        }
        async_commit();
    };

#pragma unroll
    for (int i = 1; i < S::stages; ++i) prefetch(steps - i, left + (i - 1) * more, at - (i - 1) * stride);
    for (int i = steps - 1; i >= 0; --i, at -= stride, left += more) {
        const int s0 = i % S::stages * kScanTpt * kScanThreads + tid, p = i & 1;
        const long long tile = (long long)i * ranks + rank;
        float h0 = 0.f;  // lane = channel: the state entering this CTA's tile
        if (lane_ch && tile * kScanTile < len) h0 = carries[(size_t)carry_row(begin, n, tile) * D + ch0 + lane];
        prefetch(i - (S::stages - 1), left + (S::stages - 1) * more, at - (S::stages - 1) * stride);
        async_wait<S::stages - 1>();
        // c = 1 - a is kept where the slopes need it.
        constexpr bool kKeepC = kGate == KDA_GATE_LOGSIGMOID || kWrite != KDA_WRITE_PLAIN;
        F2 a[kScanTpt][kScanPairs], b[kScanTpt][kScanPairs], c1[kKeepC ? kScanTpt : 1][kScanPairs];
        {
            F2 A[kScanPairs], H[kScanPairs] = {{0}, {0}}, U[kScanPairs] = {{0}, {0}};
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
                    if (kKeepC) c1[kKeepC ? j : 0][c] = q.c;
                    b[j][c] = written<kWrite>(q.a, q.c, xv[c]);
                    H[c] = fma2(q.a, H[c], b[j][c]);
                    decay[c].then(q);
                }
            }
#pragma unroll
            for (int j = kScanTpt - 1; j >= 0; --j) {
                F2 dv[kScanPairs];
                unpack4(ds[s0 + j * kScanThreads], dv);
#pragma unroll
                for (int c = 0; c < kScanPairs; ++c) U[c] = mul2(a[j][c], add2(dv[c], U[c]));
            }
#pragma unroll
            for (int c = 0; c < kScanPairs; ++c) A[c] = decay[c].value();
            *reinterpret_cast<float4 *>(&sh.map[group][0][col]) = pack4<float>(A);
            *reinterpret_cast<float4 *>(&sh.map[group][1][col]) = pack4<float>(H);
            *reinterpret_cast<float4 *>(&sh.map[group][2][col]) = pack4<float>(U);
        }
        __syncwarp();
        float A[kWarpGroups], H[kWarpGroups], U[kWarpGroups];
        {
            float PA = 1.f, PH = 0.f, QU = 0.f;
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                A[v] = sh.map[warp * kWarpGroups + v][0][lane];
                H[v] = sh.map[warp * kWarpGroups + v][1][lane];
                U[v] = sh.map[warp * kWarpGroups + v][2][lane];
            }
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                PH = fmaf(A[v], PH, H[v]);
                PA *= A[v];
                QU = fmaf(A[kWarpGroups - 1 - v], QU, U[kWarpGroups - 1 - v]);
            }
            sh.warp_map[p][0][warp][lane] = PA;
            sh.warp_map[p][1][warp][lane] = PH;
            sh.warp_map[p][2][warp][lane] = QU;
        }
        __syncthreads();  // warp_map's halves alternate: the only barrier of a step
        {
            float WA[kScanWarps], WU[kScanWarps];
#pragma unroll
            for (int v = 0; v < kScanWarps; ++v) {
                WA[v] = sh.warp_map[p][0][v][lane];
                WU[v] = sh.warp_map[p][2][v][lane];
            }
            if (ranks > 1 && warp == 0) {
                float TA = 1.f, TU = 0.f;
#pragma unroll
                for (int v = kScanWarps - 1; v >= 0; --v) {
                    TU = fmaf(WA[v], TU, WU[v]);
                    TA *= WA[v];
                }
                cluster_maps_send(sh.peers, steps - 1 - i, rank, ranks, TA, TU);
            }
            float mine = 0.f;  // the state entering the warp's tokens
#pragma unroll
            for (int v = 0; v < kScanWarps; ++v) {
                if (v == warp) mine = h0;
                h0 = fmaf(WA[v], h0, sh.warp_map[p][1][v][lane]);
            }
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                sh.map[warp * kWarpGroups + v][1][lane] = mine;
                mine = fmaf(A[v], mine, H[v]);
            }
            float last = u;  // the gradient entering the CTA's tile from behind
            if (ranks > 1) {
                const int step = steps - 1 - i;
                if (!cluster_maps_wait(sh.peers, step)) u = __uint_as_float(0x7fc00000u);
                for (int r = ranks - 1; r >= 0; --r) {
                    if (r == rank) last = u;
                    const float2 t = sh.peers.map[step & 1][r][lane];
                    u = fmaf(t.x, u, t.y);
                }
            }
#pragma unroll
            for (int v = kScanWarps - 1; v >= 0; --v) {
                if (v == warp) mine = last;
                last = fmaf(WA[v], last, WU[v]);
            }
            if (ranks == 1) u = last;
#pragma unroll
            for (int v = kWarpGroups - 1; v >= 0; --v) {
                sh.map[warp * kWarpGroups + v][2][lane] = mine;
                mine = fmaf(A[v], mine, U[v]);
            }
        }
        __syncwarp();
        F2 h[kScanPairs], e[kScanPairs];
        unpack4(*reinterpret_cast<const float4 *>(&sh.map[group][1][col]), h);
        unpack4(*reinterpret_cast<const float4 *>(&sh.map[group][2][col]), e);
#pragma unroll
        for (int j = 0; j < kScanTpt; ++j)
#pragma unroll
            for (int c = 0; c < kScanPairs; ++c) {
                const F2 before = h[c];
                h[c] = fma2(a[j][c], h[c], b[j][c]);
                b[j][c] = before;  // h_{t-1}
            }
        // dg = e a (dlog a/dg) (h_{t-1} - y), where a (-y) is x dw/dlog a: y = 0, x, or
        // a x / w.
        XT *dxp = dx + at;
        GT *dgp = dg + at;
#pragma unroll
        for (int j = kScanTpt - 1; j >= 0; --j) {
            if (j >= left) continue;  // past the end: the identity map, e passes through
            const int s = s0 + j * kScanThreads;
            F2 xv[kScanPairs], zv[kScanPairs], dv[kScanPairs], ox[kScanPairs], og[kScanPairs];
            if (kWrite != KDA_WRITE_PLAIN) unpack4(xs[s], xv);
            if (kGate == KDA_GATE_BOUNDED) unpack4(gs[s], zv);
            unpack4(ds[s], dv);
#pragma unroll
            for (int c = 0; c < kScanPairs; ++c) {
                const F2 aj = a[j][c], cj = c1[kKeepC ? j : 0][c];
                const F2 et = add2(dv[c], e[c]);
                F2 d = b[j][c];
                ox[c] = et;
                if (kWrite == KDA_WRITE_COMPLEMENT) {
                    ox[c] = mul2(cj, et);
                    d = fma2(xv[c], f2(-1.f), d);
                }
                if (kWrite == KDA_WRITE_NORM) {
                    const F2 w2 = fma2(cj, aj, cj);
                    const F2 r = each(w2, [](float v) { return v >= 1.17549435e-38f ? rsqrt_approx(v) : 0.f; });
                    ox[c] = mul2(mul2(w2, r), et);
                    d = fma2(mul2(mul2(aj, r), f2(-1.f)), xv[c], d);
                }
                e[c] = mul2(aj, et);
                og[c] = mul2(e[c], d);
                if (kGate == KDA_GATE_LOGSIGMOID) og[c] = mul2(og[c], cj);
                if (kGate == KDA_GATE_BOUNDED) {
                    F2 s1, sc;
                    sigmoid_pair(zv[c], s1, sc);
                    og[c] = mul2(og[c], mul2(mul2(f2(lower), s1), sc));
                }
            }
            *reinterpret_cast<XP *>(dxp + (size_t)j * D) = pack4<XT>(ox);
            *reinterpret_cast<GP *>(dgp + (size_t)j * D) = pack4<GT>(og);
        }
    }
    async_wait<0>();
    if (dinit && warp == 0 && rank == 0 && lane_ch) dinit[(size_t)n * D + ch0 + lane] = u;
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
