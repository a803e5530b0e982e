// Gated linear recurrence over whole sequences, h_t = a_t h_{t-1} + w_t x_t per
// channel, and its single-token step.
//
// A step is the affine map h -> A h + H with (A, H) = (a_t, w_t x_t); maps
// compose associatively, (A, H) then (A', H') being (A' A, A' H + H'), so time
// is cut into pieces whose maps are formed side by side and then composed in
// order. A thread holds 4 or 8 consecutive tokens of 4 or 8 channels, a CTA 16
// such groups of tokens in 128 bytes of channels, and a cluster of up to 16
// CTAs consecutive tiles of the same channels. The groups' maps are composed
// through shared memory with a lane for each channel or two: within a warp
// without a barrier, over the CTA's four warps after the one barrier of a step,
// and over the cluster by asynchronous stores to one another. Each thread then
// has the state that enters its tokens and walks them once more, from the a and
// w x still in its registers. Each input is read once and each output written
// once; the cluster goes on to its next tiles with the state it has reached.
// The composition order is fixed, so the results do not depend on the run, and
// clusters never wait for one another.
//
// Inputs arrive by asynchronous copies into slots of the thread's own (no
// barrier), up to two tiles ahead. Bound by HBM where the gates are fp32
// (131072 x 2048, bf16 x: 349 us, 6.2 TB/s); with bf16 gates the 6 bytes of a
// value leave 20 instructions or so for it, and latency shows: 272 us, 5.9 TB/s
// there, 78 us and 5.1 TB/s on 8 x 4096 x 2048 with the norm write. ncu, 32768
// tokens: issue slots 39 % busy with bf16 gates and 37 % with fp32 ones, 11 and
// 16 % of the warps resident (registers: a and w x of 64 and 32 values a
// thread); the largest stalls are fixed latency and the copies' arrival.
#include "kda_scan.cuh"

namespace kda {
namespace {

template <typename XT, typename GT, int kTokens = kScanTpt<XT, GT>>
struct FwdShape {
    using Tiling = ScanTiling<XT, GT, kTokens>;
    static constexpr int threads = kScanThreads, tpt = Tiling::tpt, vec = Tiling::vec, pairs = vec / 2;
    static constexpr int warps = threads / 32, tile = Tiling::tile, ch = Tiling::ch;
    using L = typename Lane<ch>::type;
    using XS = Slots<XT, vec, tpt, threads>;
    using GS = Slots<GT, vec, tpt, threads>;
    struct Shared {
        // (A, H) of each group's tokens; then H gives way to the state entering them.
        float map[Tiling::groups][2][ch];
        L warp_map[2][warps][2][32];  // (A, H) of each warp's tokens
    };
    static constexpr int stages = 2;
    static constexpr size_t smem = stages * (XS::bytes_per_stage + GS::bytes_per_stage);
    // CTAs per SM that the registers are shared out for. Fewer than the shared
    // memory would hold is faster where a thread has 32 values (fp32 gates, 16
    // rows of 2048 x 2048: 106 us with 4, 93 with 3; bf16 gates 72 with 4, 82 with
    // 3; all fp32, 20011 packed tokens: 62 with 5, 60 with 4).
    static constexpr int per_sm = vec * tpt > 32 ? 2 : sizeof(XT) < sizeof(GT) ? 3 : 4;
};

// kNarrow: a sequence for each warp (ScanOrder).
template <typename XT, typename GT, int kGate, int kWrite, int kTokens, bool kNarrow>
__global__ void __launch_bounds__(kScanThreads, FwdShape<XT, GT, kTokens>::per_sm)
scan_fwd(const XT *__restrict__ x, const GT *__restrict__ g, const float *init,
         const int32_t *__restrict__ cu, XT *__restrict__ out, float *final_state,
         float *__restrict__ carries, int T_fixed, long long tokens, int D, int blocks, int ranks,
         int num_seqs, int order, bool zero_outside, float lower) {
    using S = FwdShape<XT, GT, kTokens>;
    using L = typename S::L;
    using XS = typename S::XS;
    using GS = typename S::GS;
    constexpr int V = S::vec, kTpt = S::tpt, kPairs = S::pairs, kTile = S::tile, kWarps = S::warps, kLaneCh = S::ch / 32;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    void *gs = smem_raw;
    void *xs = smem_raw + S::stages * GS::bytes_per_stage;
    __shared__ __align__(16) typename S::Shared sh;

    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5), group = tid / kScanLanes;
    const int rank = !kNarrow && ranks > 1 ? (int)tc::cluster_rank() : 0;
    const ClusterMaps<S::ch> peers = {reinterpret_cast<uint64_t *>(smem_raw + S::smem), rank, ranks};
    const unsigned unit = blockIdx.x / (unsigned)ranks;  // (sequence, channel block)
    int n = (int)(unit / (unsigned)blocks);
    if (!kNarrow && order == kOrderLongest) n = kth_longest(cu, num_seqs, n, tokens, reinterpret_cast<int *>(&sh));
    if (kNarrow) n = uniform(n * kWarps + warp);
    const int ch0 = (int)(unit % (unsigned)blocks) * S::ch;
    const int col = V * (tid & (kScanLanes - 1));  // this thread's channels, and a lane's where warps compose
    const bool has_ch = ch0 + col < D && n < num_seqs, lane_ch = ch0 + lane * kLaneCh < D && n < num_seqs;

    // In every warp, by lane: the state at the cluster's next tiles. Read before
    // the cluster's first barrier: final_state may be the same memory.
    L carry;
    lane_set(carry, 0.f);
    const size_t state_at = (size_t)n * D + ch0 + lane * kLaneCh;
    if (init && lane_ch) carry = *reinterpret_cast<const L *>(init + state_at);
    bool lost = false;  // a wait for the cluster gave up
    if (!kNarrow && ranks > 1) cluster_maps_init(peers);

    long long begin, end;
    scan_bounds(cu, n, T_fixed, tokens, begin, end);
    begin = uniform(begin);
    const int len = uniform((int)(end - begin));
    const int super = kTile * ranks;  // tokens per cluster step
    const int steps = (int)(((long long)len + super - 1) / super);

    // Of this step: tokens from this thread's first one to the sequence's end
    // (none left where negative), and the first one's element.
    const int first_token = rank * kTile + (kNarrow ? lane / kScanLanes : group) * kTpt;
    int left = has_ch ? len - first_token : -1;
    const int less = has_ch ? super : 0;
    size_t at = (size_t)(begin + first_token) * D + ch0 + col;
    const size_t stride = (size_t)super * D;
    auto prefetch = [&](int i, int left, size_t from) {
        const int st = i % S::stages;
        if (left >= kTpt) {
#pragma unroll
            for (int j = 0; j < kTpt; ++j) {
                GS::copy(gs, st, j, g + from + (size_t)j * D);
                XS::copy(xs, st, j, x + from + (size_t)j * D);
            }
        } else if (i < steps) {
            for (int j = 0; j < kTpt; ++j) {
                if (j < left) {
                    GS::copy(gs, st, j, g + from + (size_t)j * D);
                    XS::copy(xs, st, j, x + from + (size_t)j * D);
                } else {
                    GS::fill(gs, st, j, identity_gate<kGate>());
                    XS::fill(xs, st, j, 0.f);
                }
            }
        }
        async_commit();
    };

#pragma unroll
    for (int i = 0; i < S::stages; ++i) prefetch(i, left - i * less, at + i * stride);
    if (!kNarrow && zero_outside && has_ch)
        rows_outside(cu, num_seqs, tokens, (long long)(unit / (unsigned)blocks) * ranks + rank, (long long)num_seqs * ranks,
                     [&](size_t row) { store_pairs<V>(out + row * D + ch0 + col, Pairs<V>{}); });
    for (int i = 0; i < steps; ++i, at += stride, left -= less) {
        async_wait<S::stages - 1>();
        const int st = i % S::stages;
        F2 a[kTpt][kPairs], b[kTpt][kPairs];
        {
            Pairs<V> H = {};
            Decay<kGate> decay[kPairs];
#pragma unroll
            for (int j = 0; j < kTpt; ++j) {
                const Pairs<V> xv = XS::get(xs, st, j), zv = GS::get(gs, st, j);
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const Gated q = gate_value<kGate, kWrite>(zv[c], lower);
                    a[j][c] = q.a;
                    b[j][c] = written<kWrite>(q.a, q.c, xv[c]);
                    H[c] = fma2(q.a, H[c], b[j][c]);
                    decay[c].then(q);
                }
            }
            Pairs<V> A;
#pragma unroll
            for (int c = 0; c < kPairs; ++c) A[c] = decay[c].value();
            store_pairs<V>(&sh.map[group][0][col], A);
            store_pairs<V>(&sh.map[group][1][col], H);
        }
        prefetch(i + S::stages, left - S::stages * less, at + S::stages * stride);  // into the slots just read
        __syncwarp();
        // By lane: the warp's groups are composed in order.
        L A[kWarpGroups], H[kWarpGroups];
        {
            L PA, PH;
            lane_set(PA, 1.f);
            lane_set(PH, 0.f);
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                A[v] = *reinterpret_cast<const L *>(&sh.map[warp * kWarpGroups + v][0][lane * kLaneCh]);
                H[v] = *reinterpret_cast<const L *>(&sh.map[warp * kWarpGroups + v][1][lane * kLaneCh]);
            }
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                PH = lane_fma(A[v], PH, H[v]);
                PA = lane_mul(PA, A[v]);
            }
            sh.warp_map[i & 1][warp][0][lane] = PA;
            sh.warp_map[i & 1][warp][1][lane] = PH;
        }
        __syncthreads();  // warp_map's halves alternate: the only barrier of a step
        {
            L first = carry;  // the state entering the CTA's tile
            if (kNarrow) {
                carry = lane_fma(sh.warp_map[i & 1][warp][0][lane], carry, sh.warp_map[i & 1][warp][1][lane]);
            } else if (ranks > 1) {
                if (warp == 0 && !lost) {
                    L TA, TH;
                    lane_set(TA, 1.f);
                    lane_set(TH, 0.f);
#pragma unroll
                    for (int v = 0; v < kWarps; ++v) {
                        const L WA = sh.warp_map[i & 1][v][0][lane];
                        TH = lane_fma(WA, TH, sh.warp_map[i & 1][v][1][lane]);
                        TA = lane_mul(TA, WA);
                    }
                    cluster_maps_send(peers, i, TA, TH);
                }
                cluster_maps_wait(peers, i, lost);
                if (lost) lane_set(carry, __uint_as_float(0x7fc00000u));
                for (int r = 0; r < ranks; ++r) {
                    if (r == rank) first = carry;
                    const auto m = peers.map(i, r);
                    carry = lane_fma(m.a, carry, m.b);
                }
            }
            L mine = first;  // the state entering the warp's tokens
            if (!kNarrow) {
#pragma unroll
                for (int v = 0; v < kWarps; ++v) {
                    if (v == warp) mine = first;
                    if (ranks == 1 || v + 1 < kWarps)
                        first = lane_fma(sh.warp_map[i & 1][v][0][lane], first, sh.warp_map[i & 1][v][1][lane]);
                }
                if (ranks == 1) carry = first;
            }
            // The states that the backward pass starts its tiles from.
            const long long t = ((long long)i * ranks + rank) * kTile + (kNarrow ? 0 : warp * kWarpGroups * kTpt);
            if (carries && t % KDA_SCAN_CARRY_TOKENS == 0 && t < len && lane_ch)
                *reinterpret_cast<L *>(carries + (size_t)carry_row(begin, n, t / KDA_SCAN_CARRY_TOKENS) * D + ch0 +
                                       lane * kLaneCh) = mine;
#pragma unroll
            for (int v = 0; v < kWarpGroups; ++v) {
                *reinterpret_cast<L *>(&sh.map[warp * kWarpGroups + v][1][lane * kLaneCh]) = mine;
                mine = lane_fma(A[v], mine, H[v]);
            }
        }
        __syncwarp();
        Pairs<V> h = load_pairs<V>(&sh.map[group][1][col]);
        XT *o = out + at;
#pragma unroll
        for (int j = 0; j < kTpt; ++j) {
#pragma unroll
            for (int c = 0; c < kPairs; ++c) h[c] = fma2(a[j][c], h[c], b[j][c]);
            if (j < left) store_pairs<V>(o + (size_t)j * D, h);
        }
    }
    async_wait<0>();
    if (final_state && (kNarrow || warp == 0) && rank == 0 && lane_ch) *reinterpret_cast<L *>(final_state + state_at) = carry;
    if (!kNarrow) cluster_maps_leave(lost);
}

template <auto kValue> struct Kernel {
    static constexpr auto value = kValue;
};

// Few long chains of bf16: what a step's composition and exchange cost shows,
// and twice the tokens a thread halve it (one sequence of 16384 tokens, 1024
// channels: 42 us with 4 tokens, 32 with 8; two of 8192, 2048 channels, 64
// pairs: 46 and 45). With more pairs, or packed sequences, the CTAs that fit
// beside one another hide it, and twice as many do with 4 (192 pairs: 106 us
// and 117; 4 packed sequences of 2048 channels: 48 and 56).
inline bool few_long_chains(const ScanArgs &s, int ch) {
    const long long units = (long long)s.num_seqs * ((s.D + ch - 1) / ch);
    return units <= 64 && (!s.cu || s.num_seqs == 1) && s.tokens / s.num_seqs >= 1024;
}

template <typename XT, typename GT, int kGate, int kWrite>
cudaError_t launch_fwd(const ScanArgs &s, cudaStream_t stream) {
    constexpr int kTokens = kScanTpt<XT, GT>;
    auto launch = [&](auto shape, auto wide, auto narrow) {
        return launch_scan<decltype(shape), wide.value, narrow.value>(
            s, stream, static_cast<const XT *>(s.x), static_cast<const GT *>(s.g), s.init, s.cu,
            static_cast<XT *>(s.out), s.final_state, s.carries, s.T_fixed, s.tokens, s.D);
    };
    using Narrow = Kernel<scan_fwd<XT, GT, kGate, kWrite, kTokens, true>>;
    if constexpr (sizeof(XT) + sizeof(GT) == 4) {
        if (few_long_chains(s, FwdShape<XT, GT>::ch))
            return launch(FwdShape<XT, GT, 2 * kTokens>(), Kernel<scan_fwd<XT, GT, kGate, kWrite, 2 * kTokens, false>>(),
                          Narrow());
    }
    return launch(FwdShape<XT, GT>(), Kernel<scan_fwd<XT, GT, kGate, kWrite, kTokens, false>>(), Narrow());
}

// One step: a thread per 16-byte piece of g, all of its loads in flight together
// (over slots from when the slot's number is there). Bound by HBM (2048 rows of
// 4096 channels out of a pool of twice as many: 22.6 us, 5.9 TB/s) or by the
// launch.
constexpr int kStepThreads = 128;
template <typename XT, typename GT, int kGate, int kWrite>
__global__ void __launch_bounds__(kStepThreads)
scan_step(const XT *__restrict__ x, const GT *__restrict__ g, float *__restrict__ state,
          const int32_t *__restrict__ slots, XT *__restrict__ out, long long pieces, int per_row, int num_slots,
          float lower) {
    constexpr int V = kVec<GT>;
    const long long i = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    if (i >= pieces) return;
    const int n = (int)(i / per_row), ch = (int)(i % per_row) * V;
    const long long slot = slots ? slots[n] : n;
    const size_t at = (size_t)i * V;
    Pairs<V> h = {};
    if (slot >= 0 && slot < num_slots) {
        float *sp = state + (size_t)slot * per_row * V + ch;
        h = load_pairs<V>(sp);
        const Pairs<V> xv = load_pairs<V>(x + at), zv = load_pairs<V>(g + at);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
            const Gated q = step_value<kGate, kWrite>(zv[c], lower);
            h[c] = fma2(q.a, h[c], written<kWrite>(q.a, q.c, xv[c]));
        }
        store_pairs<V>(sp, h);
    }
    store_pairs<V>(out + at, h);
}

template <typename XT, typename GT, int kGate, int kWrite>
cudaError_t launch_step(const ScanStepArgs &s, cudaStream_t stream) {
    const int per_row = s.D / kVec<GT>;
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
