// Gradient of the gated linear recurrence.
//
// With u_t = a_t e_t, the gradient that reaches h_{t-1}, the backward
// recurrence e_t = dout_t + u_{t+1} is again a chain of affine maps,
// u -> a_t u + a_t dout_t, taken from the last token to the first. It is cut
// and composed as the forward scan's is (kda_scan.cu): thread, warp, CTA, and
// a cluster of CTAs over consecutive tiles, which here goes through the
// sequence from its end. dg needs h_{t-1} as well; it is formed again within
// the tile by the forward composition, from the fp32 state that the forward
// call saved at the tile's first token, so neither h nor a second pass over the
// sequence is read, and h is not taken from its rounded outputs. x, g and dout
// come in and dx and dg go out once each.
//
// The gates' slopes are formed after the exchange, from a and 1 - a kept in
// registers. Bound by HBM with fp32 gates (131072 x 2048, bf16 x: 576 us, 6.5
// TB/s); with bf16 gates by latency at 16 % of the warps resident (513 us, 5.2
// TB/s; 8 x 4096 x 2048 with the norm write 133 us, 5.0 TB/s).
#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename XT, typename GT>
struct BwdShape {
    using Tiling = ScanTiling<XT, GT>;
    static constexpr int threads = kScanThreads, tpt = Tiling::tpt, vec = Tiling::vec, pairs = vec / 2;
    static constexpr int warps = threads / 32, tile = Tiling::tile, ch = Tiling::ch;
    static_assert(tile % KDA_SCAN_CARRY_TOKENS == 0, "a tile begins at a saved state");
    using L = typename Lane<ch>::type;
    using XS = Slots<XT, vec, tpt, threads>;
    using GS = Slots<GT, vec, tpt, threads>;
    struct Shared {
        // A and H of each group's tokens, then U in A's place; then the gradient and the
        // state entering them. (A third row costs clusters of 12 the third CTA per
        // SM: 131072 x 2048, bf16 gates, 572 us for 517.)
        float map[Tiling::groups][2][ch];
        L warp_map[2][warps][3][32];  // A, H, U of each warp's tokens
    };
    static constexpr int stages = 2;
    static constexpr size_t smem = stages * (2 * XS::bytes_per_stage + GS::bytes_per_stage);
    // CTAs per SM that the registers are shared out for: with fp32 gates fewer than
    // the shared memory would hold (16 rows of 2048 x 2048: 208 us with 3, 160 with
    // 2; bf16 gates 141 and 135, but 130 with 3 in clusters; all fp32 215 and 218).
    static constexpr int per_sm = sizeof(XT) < sizeof(GT) ? 2 : 3;
};

// kNarrow: a sequence for each warp (ScanOrder).
template <typename XT, typename GT, int kGate, int kWrite, bool kNarrow>
__global__ void __launch_bounds__(BwdShape<XT, GT>::threads, BwdShape<XT, GT>::per_sm)
scan_bwd(const XT *__restrict__ dout, const float *dfinal, const XT *__restrict__ x,
         const GT *__restrict__ g, const float *__restrict__ carries, const int32_t *__restrict__ cu,
         XT *__restrict__ dx, GT *__restrict__ dg, float *dinit, int T_fixed, long long tokens, int D,
         int blocks, int ranks, int num_seqs, int order, bool zero_outside, float lower) {
    using S = BwdShape<XT, GT>;
    using L = typename S::L;
    using XS = typename S::XS;
    using GS = typename S::GS;
    constexpr int V = S::vec, kTpt = S::tpt, kPairs = S::pairs, kTile = S::tile, kWarps = S::warps, kLaneCh = S::ch / 32;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    void *gs = smem_raw;
    void *xs = smem_raw + S::stages * GS::bytes_per_stage;
    void *ds = smem_raw + S::stages * (GS::bytes_per_stage + XS::bytes_per_stage);
    __shared__ __align__(16) typename S::Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), group = tid / kScanLanes;
    const int rank = !kNarrow && ranks > 1 ? (int)tc::cluster_rank() : 0;
    const ClusterMaps<S::ch> peers = {reinterpret_cast<uint64_t *>(smem_raw + S::smem), rank, ranks};
    const unsigned unit = blockIdx.x / (unsigned)ranks;
    int n = (int)(unit / (unsigned)blocks);
    if (!kNarrow && order == kOrderLongest) n = kth_longest(cu, num_seqs, n, tokens, reinterpret_cast<int *>(&sh));
    if (kNarrow) n = uniform(n * kWarps + warp);
    const int ch0 = (int)(unit % (unsigned)blocks) * S::ch;
    const int col = V * (tid & (kScanLanes - 1));
    const bool has_ch = ch0 + col < D && n < num_seqs, lane_ch = ch0 + lane * kLaneCh < D && n < num_seqs;

    // In every warp, by lane: the gradient entering the cluster's tiles from
    // behind. Read before the cluster's first barrier: dinit may be the same
    // memory.
    L u;
    lane_set(u, 0.f);
    const size_t state_at = (size_t)n * D + ch0 + lane * kLaneCh;
    if (dfinal && lane_ch) u = *reinterpret_cast<const L *>(dfinal + state_at);
    bool lost = false;  // a wait for the cluster gave up
    if (!kNarrow && ranks > 1) cluster_maps_init(peers);

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    begin = uniform(begin);
    const int len = uniform((int)(end - begin));
    const int super = kTile * ranks;
    const int steps = (int)(((long long)len + super - 1) / super);

    // Of a step: tokens from this thread's first one to the sequence's end (none
    // left where negative), and the first one's element.
    const long long t0 = ((long long)(steps - 1) * ranks + rank) * kTile + (kNarrow ? lane / kScanLanes : group) * kTpt;
    int left = has_ch ? (int)(len - t0) : -1;
    const int more = has_ch ? super : 0;
    size_t at = (size_t)(begin + t0) * D + ch0 + col;
    const size_t stride = (size_t)super * D;
    auto prefetch = [&](int i, int left, size_t from) {
        const int st = i & 1;
        if (i >= 0 && left >= kTpt) {
#pragma unroll
            for (int j = 0; j < kTpt; ++j) {
                GS::copy(gs, st, j, g + from + (size_t)j * D);
                XS::copy(ds, st, j, dout + from + (size_t)j * D);
                XS::copy(xs, st, j, x + from + (size_t)j * D);
            }
        } else if (i >= 0) {
            for (int j = 0; j < kTpt; ++j) {
                if (j < left) {
                    GS::copy(gs, st, j, g + from + (size_t)j * D);
                    XS::copy(ds, st, j, dout + from + (size_t)j * D);
                    XS::copy(xs, st, j, x + from + (size_t)j * D);
                } else {
                    GS::fill(gs, st, j, identity_gate<kGate>());
                    XS::fill(ds, st, j, 0.f);
                    XS::fill(xs, st, j, 0.f);
                }
            }
        }
        async_commit();
    };

    prefetch(steps - 1, left, at);
    if (!kNarrow && zero_outside && has_ch)
        rows_outside(cu, num_seqs, tokens, (long long)(unit / (unsigned)blocks) * ranks + rank, (long long)num_seqs * ranks,
                     [&](size_t row) {
                         store_pairs<V>(dx + row * D + ch0 + col, Pairs<V>{});
                         store_pairs<V>(dg + row * D + ch0 + col, Pairs<V>{});
                     });
    for (int i = steps - 1; i >= 0; --i, at -= stride, left += more) {
        const int st = i & 1, p = i & 1;
        const long long tile = ((long long)i * ranks + rank) * kTile;  // the CTA's first token
        L h0;  // by lane: the state entering it
        lane_set(h0, 0.f);
        if (lane_ch && tile < len)
            h0 = *reinterpret_cast<const L *>(carries + (size_t)carry_row(begin, n, tile / KDA_SCAN_CARRY_TOKENS) * D + ch0 +
                                              lane * kLaneCh);
        prefetch(i - 1, left + more, at - stride);
        async_wait<1>();
        // c = 1 - a is kept where the slopes need it.
        constexpr bool kKeepC = kGate == KDA_GATE_LOGSIGMOID || kWrite != KDA_WRITE_PLAIN;
        F2 a[kTpt][kPairs], b[kTpt][kPairs], c1[kKeepC ? kTpt : 1][kPairs];
        {
            Pairs<V> A, H = {};
            Decay<kGate> decay[kPairs];
#pragma unroll
            for (int j = 0; j < kTpt; ++j) {
                const Pairs<V> xv = XS::get(xs, st, j), zv = GS::get(gs, st, j);
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const Gated q = gate_value<kGate, kWrite>(zv[c], lower);
                    a[j][c] = q.a;
                    if (kKeepC) c1[kKeepC ? j : 0][c] = q.c;
                    b[j][c] = written<kWrite>(q.a, q.c, xv[c]);
                    H[c] = fma2(q.a, H[c], b[j][c]);
                    decay[c].then(q);
                }
            }
#pragma unroll
            for (int c = 0; c < kPairs; ++c) A[c] = decay[c].value();
            store_pairs<V>(&sh.map[group][0][col], A);
            store_pairs<V>(&sh.map[group][1][col], H);
        }
        __syncwarp();
        auto entry = [&](int v, int k) -> L & {
            return *reinterpret_cast<L *>(&sh.map[warp * kWarpGroups + v][k][lane * kLaneCh]);
        };
        L A[kWarpGroups], H[kWarpGroups], U[kWarpGroups];
#pragma unroll
        for (int v = 0; v < kWarpGroups; ++v) {
            A[v] = entry(v, 0);
            H[v] = entry(v, 1);
        }
        {
            Pairs<V> back = {};
#pragma unroll
            for (int j = kTpt - 1; j >= 0; --j) {
                const Pairs<V> dv = XS::get(ds, st, j);
#pragma unroll
                for (int c = 0; c < kPairs; ++c) back[c] = mul2(a[j][c], add2(dv[c], back[c]));
            }
            __syncwarp();  // every lane has its A
            store_pairs<V>(&sh.map[group][0][col], back);
        }
        __syncwarp();
        {
            L PA, PH, QU;
            lane_set(PA, 1.f);
            lane_set(PH, 0.f);
            lane_set(QU, 0.f);
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) U[v] = entry(v, 0);
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                PH = lane_fma(A[v], PH, H[v]);
                PA = lane_mul(PA, A[v]);
                QU = lane_fma(A[kWarpGroups - 1 - v], QU, U[kWarpGroups - 1 - v]);
            }
            sh.warp_map[p][warp][0][lane] = PA;
            sh.warp_map[p][warp][1][lane] = PH;
            sh.warp_map[p][warp][2][lane] = QU;
        }
        __syncthreads();  // warp_map's halves alternate: the only barrier of a step
        {
            if (ranks > 1 && warp == 0 && !lost) {
                L TA, TU;
                lane_set(TA, 1.f);
                lane_set(TU, 0.f);
#pragma unroll
                for (int v = kWarps - 1; v >= 0; --v) {
                    const L WA = sh.warp_map[p][v][0][lane];
                    TU = lane_fma(WA, TU, sh.warp_map[p][v][2][lane]);
                    TA = lane_mul(TA, WA);
                }
                cluster_maps_send(peers, steps - 1 - i, TA, TU);
            }
            for (int v = 0; v < (kNarrow ? 0 : warp); ++v) h0 = lane_fma(sh.warp_map[p][v][0][lane], h0, sh.warp_map[p][v][1][lane]);
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                entry(v, 1) = h0;
                h0 = lane_fma(A[v], h0, H[v]);
            }
            L last = u;  // the gradient entering the CTA's tile from behind
            if (kNarrow) {
                u = lane_fma(sh.warp_map[p][warp][0][lane], u, sh.warp_map[p][warp][2][lane]);
            } else if (ranks > 1) {
                const int step = steps - 1 - i;
                cluster_maps_wait(peers, step, lost);
                if (lost) lane_set(u, __uint_as_float(0x7fc00000u));
                for (int r = ranks - 1; r >= 0; --r) {
                    if (r == rank) last = u;
                    const auto m = peers.map(step, r);
                    u = lane_fma(m.a, u, m.b);
                }
            }
            L mine = last;
            if (!kNarrow) {
#pragma unroll
                for (int v = kWarps - 1; v >= 0; --v) {
                    if (v == warp) mine = last;
                    if (ranks == 1 || v > 0) last = lane_fma(sh.warp_map[p][v][0][lane], last, sh.warp_map[p][v][2][lane]);
                }
                if (ranks == 1) u = last;
            }
#pragma unroll
            for (int v = kWarpGroups - 1; v >= 0; --v) {
                entry(v, 0) = mine;
                mine = lane_fma(A[v], mine, U[v]);
            }
        }
        __syncwarp();
        Pairs<V> h = load_pairs<V>(&sh.map[group][1][col]), e = load_pairs<V>(&sh.map[group][0][col]);
#pragma unroll
        for (int j = 0; j < kTpt; ++j)
#pragma unroll
            for (int c = 0; c < kPairs; ++c) {
                const F2 before = h[c];
                h[c] = fma2(a[j][c], h[c], b[j][c]);
                b[j][c] = before;  // h_{t-1}
            }
        // dg = e a (dlog a/dg) (h_{t-1} - y), where a (-y) is x dw/dlog a: y = 0, x, or
        // a x / w.
        XT *dxp = dx + at;
        GT *dgp = dg + at;
#pragma unroll
        for (int j = kTpt - 1; j >= 0; --j) {
            if (j >= left) continue;  // past the end: the identity map, e passes through
            Pairs<V> xv, zv, ox, og;
            if (kWrite != KDA_WRITE_PLAIN) xv = XS::get(xs, st, j);
            if (kGate == KDA_GATE_BOUNDED) zv = GS::get(gs, st, j);
            const Pairs<V> dv = XS::get(ds, st, j);
#pragma unroll
            for (int c = 0; c < kPairs; ++c) {
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
            store_pairs<V>(dxp + (size_t)j * D, ox);
            store_pairs<V>(dgp + (size_t)j * D, og);
        }
    }
    async_wait<0>();
    if (dinit && (kNarrow || warp == 0) && rank == 0 && lane_ch) *reinterpret_cast<L *>(dinit + state_at) = u;
    if (!kNarrow) cluster_maps_leave(lost);
}

template <typename XT, typename GT, int kGate, int kWrite>
cudaError_t launch_bwd(const ScanArgs &s, cudaStream_t stream) {
    return launch_scan<BwdShape<XT, GT>, scan_bwd<XT, GT, kGate, kWrite, false>, scan_bwd<XT, GT, kGate, kWrite, true>>(
        s, stream, static_cast<const XT *>(s.dout), s.dfinal, static_cast<const XT *>(s.x),
        static_cast<const GT *>(s.g), (const float *)s.carries, s.cu, static_cast<XT *>(s.dx), static_cast<GT *>(s.dg),
        s.dinit, s.T_fixed, s.tokens, s.D);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanArgs &s, cudaStream_t stream) {
    return KDA_SCAN_DISPATCH(launch_bwd, s, stream);
}

}  // namespace kda
