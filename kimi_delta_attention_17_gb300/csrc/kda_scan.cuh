// Shared by the gated linear recurrence's kernels (h_t = a_t h_{t-1} + w_t x_t):
// the gate functions, 16-byte pieces, and the exchange of affine maps.
#pragma once

#include <atomic>

#include "kda_internal.cuh"
#include "kda_tc.cuh"

namespace kda {

// Validated kda_scan_options.
struct ScanGate {
    int gate;     // kda_gate
    int write;    // kda_write
    float lower;  // KDA_GATE_BOUNDED: lower bound of log a
};

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float x, float y) {  // NaN stays NaN
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
constexpr float kLog2E = 1.44269504088896341f;

// Two fp32 values that one instruction takes together (FFMA2 and its kin): few
// warps are resident, so a step's time goes with the instructions of its chain.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ void split(F2 x, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
template <typename F>
__device__ __forceinline__ F2 each(F2 x, F f) {
    float lo, hi;
    split(x, lo, hi);
    return f2(f(lo), f(hi));
}

// a = e^x and c = 1 - a for a log-decay x <= 0. Near 0 both come from the
// Taylor series of e^x - 1 (to x^7 / 7!, off by less than |x|^7 / 8! < 2e-8
// relative for |x| < 0.35): 1 - e^x from a rounded e^x would lose the digits
// of a small 1 - a.
__device__ __forceinline__ void decay_pair(F2 x, F2 &a, F2 &c) {
    F2 p = fma2(f2(1.f / 5040.f), x, f2(1.f / 720.f));
    p = fma2(p, x, f2(1.f / 120.f));
    p = fma2(p, x, f2(1.f / 24.f));
    p = fma2(p, x, f2(1.f / 6.f));
    p = fma2(p, x, f2(0.5f));
    p = fma2(p, x, f2(1.f));
    const F2 m = mul2(p, x);  // e^x - 1
    const F2 e = each(mul2(x, f2(kLog2E)), ex2_approx);
    const F2 e1 = add2(e, f2(-1.f)), m1 = add2(m, f2(1.f));
    float x0, x1, m0[2], e0[2], e10[2], m10[2];
    split(x, x0, x1);
    split(m, m0[0], m0[1]);
    split(e, e0[0], e0[1]);
    split(e1, e10[0], e10[1]);
    split(m1, m10[0], m10[1]);
    const bool s0 = fabsf(x0) < 0.35f, s1 = fabsf(x1) < 0.35f;
    a = f2(s0 ? m10[0] : e0[0], s1 ? m10[1] : e0[1]);
    c = f2(-(s0 ? m0[0] : e10[0]), -(s1 ? m0[1] : e10[1]));
}

// sigmoid(z) and 1 - sigmoid(z) = t sigmoid(z) with t = e^-z, both accurate to
// a few units in their own last place. Below -80 sigmoid(z) is taken as
// e^-80 = 2e-35, so that t stays finite.
__device__ __forceinline__ void sigmoid_pair(F2 z, F2 &s, F2 &c) {
    const F2 t = each(mul2(each(z, [](float v) { return max_nan(v, -80.f); }), f2(-kLog2E)), ex2_approx);
    s = each(add2(t, f2(1.f)), rcp_approx);
    c = mul2(t, s);
}

// What two gate values give: a, c = 1 - a (formed where the write or the gate
// has it), and log a or 1 - a (`rest`) for Decay.
struct Gated {
    F2 a, c, rest;
};
template <int kGate, int kWrite>
__device__ __forceinline__ Gated gate_value(F2 z, float lower) {
    Gated r;
    if (kGate == KDA_GATE_LOGSIGMOID) {
        sigmoid_pair(z, r.a, r.c);
        r.rest = r.c;
        return r;
    }
    r.rest = z;
    if (kGate == KDA_GATE_BOUNDED) {
        F2 s, sc;
        sigmoid_pair(z, s, sc);
        r.rest = mul2(f2(lower), s);
    }
    if (kWrite == KDA_WRITE_PLAIN) {
        r.a = each(mul2(r.rest, f2(kLog2E)), ex2_approx);
        r.c = f2(0.f);  // not used
    } else {
        decay_pair(r.rest, r.a, r.c);
    }
    return r;
}
// a, where 1 - a is below 1/2 taken from there: rounded once, to the nearest.
__device__ __forceinline__ F2 from_complement(F2 a, F2 c) {
    float a0, a1, c0, c1;
    split(a, a0, a1);
    split(c, c0, c1);
    return f2(c0 < 0.5f ? 1.f - c0 : a0, c1 < 0.5f ? 1.f - c1 : a1);
}
// The same for a state that meets the gates one by one, thousands of times in a
// serving loop: a from 1 - a. The approximate ex2 and reciprocal lean to one side,
// which is nothing over the few tokens between two compositions of a scan, but
// over 6000 steps at a ~ 0.9999 it put the last state off by 325 x 2^-24 (log-decays,
// plain write) and 961 x 2^-24 (logistic, complement write); so by 24 and 43.
template <int kGate, int kWrite>
__device__ __forceinline__ Gated step_value(F2 z, float lower) {
    Gated r = gate_value<kGate, kWrite == KDA_WRITE_PLAIN ? KDA_WRITE_COMPLEMENT : kWrite>(z, lower);
    if (kGate == KDA_GATE_LOGSIGMOID) r.a = from_complement(r.a, r.c);
    return r;
}
// w x: the input as it enters the state; 1 - a^2 is taken from its factors.
template <int kWrite>
__device__ __forceinline__ F2 written(F2 a, F2 c, F2 x) {
    if (kWrite == KDA_WRITE_PLAIN) return x;
    if (kWrite == KDA_WRITE_COMPLEMENT) return mul2(c, x);
    return mul2(each(fma2(c, a, c), sqrt_approx), x);
}

// The gate value of the identity map (a = 1), which stands past a sequence's end.
template <int kGate>
__device__ __forceinline__ float identity_gate() {
    return kGate == KDA_GATE_LOG ? 0.f
                                 : __uint_as_float(kGate == KDA_GATE_LOGSIGMOID ? 0x7f800000u : 0xff800000u);
}

// The decay A over a thread's tokens. Products of rounded decays will not do
// for slow channels: of two factors 1 - p and 1 - q with p q < 2^-25 the
// rounded product loses p q every time, always to the same side, which over
// the thousands of tokens that such a channel remembers comes to hundreds of
// roundings (measured at a ~ 0.9999 over 6000 tokens: 430 x 2^-24). A
// log-decay is summed instead; under the logistic gate, which gives 1 - a,
// 1 - A is carried beside the product and used while A > 1/2.
template <int kGate>
struct Decay {
    F2 sum = {0};
    __device__ __forceinline__ void then(const Gated &q) { sum = add2(sum, q.rest); }
    __device__ __forceinline__ F2 value() const {
        F2 a, c;
        decay_pair(sum, a, c);
        return a;
    }
};
template <>
struct Decay<KDA_GATE_LOGSIGMOID> {
    F2 A = f2(1.f), C = {0};
    __device__ __forceinline__ void then(const Gated &q) {
        C = fma2(q.rest, A, C);
        A = mul2(A, q.a);
    }
    __device__ __forceinline__ F2 value() const { return from_complement(A, C); }
};

// A thread holds the channels of one 16-byte piece of g: eight of bf16, four of
// fp32. Rows of 64 bytes cost bandwidth (copies alone, measured: 3.4 TB/s in
// 8-byte pieces of 64-byte rows, 6.5 TB/s in 16-byte pieces of 128-byte rows),
// so it is the wider operand that gets the 128 bytes.
template <typename GT>
constexpr int kVec = 16 / (int)sizeof(GT);

template <int kBytes> struct PieceOf { using type = uint4; };
template <> struct PieceOf<8> { using type = uint2; };
template <typename T, int V>
using Piece = typename PieceOf<V *(int)sizeof(T)>::type;  // V values of T: 8 or 16 bytes

// V values of one token, as pairs.
template <int V>
struct Pairs {
    F2 v[V / 2];
    __device__ __forceinline__ F2 &operator[](int i) { return v[i]; }
    __device__ __forceinline__ const F2 &operator[](int i) const { return v[i]; }
};
__device__ __forceinline__ F2 unpack2(uint32_t u) {
    return f2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(F2 x) {
    float lo, hi;
    split(x, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T, int V> struct Convert;
template <> struct Convert<float, 4> {
    static __device__ __forceinline__ void unpack(const uint4 &r, F2 *x) {
        x[0] = f2(__uint_as_float(r.x), __uint_as_float(r.y));
        x[1] = f2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    static __device__ __forceinline__ uint4 pack(const F2 *x) {
        float v[4];
        split(x[0], v[0], v[1]);
        split(x[1], v[2], v[3]);
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <> struct Convert<__nv_bfloat16, 4> {
    static __device__ __forceinline__ void unpack(const uint2 &r, F2 *x) {
        x[0] = unpack2(r.x);
        x[1] = unpack2(r.y);
    }
    static __device__ __forceinline__ uint2 pack(const F2 *x) { return make_uint2(pack2(x[0]), pack2(x[1])); }
};
template <> struct Convert<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void unpack(const uint4 &r, F2 *x) {
        x[0] = unpack2(r.x);
        x[1] = unpack2(r.y);
        x[2] = unpack2(r.z);
        x[3] = unpack2(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const F2 *x) {
        return make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
    }
};
template <int V>
__device__ __forceinline__ Pairs<V> load_pairs(const __nv_bfloat16 *from) {
    Pairs<V> x;
    Convert<__nv_bfloat16, V>::unpack(*reinterpret_cast<const Piece<__nv_bfloat16, V> *>(from), x.v);
    return x;
}
template <int V>
__device__ __forceinline__ void store_pairs(__nv_bfloat16 *to, const Pairs<V> &x) {
    *reinterpret_cast<Piece<__nv_bfloat16, V> *>(to) = Convert<__nv_bfloat16, V>::pack(x.v);
}
template <int V>
__device__ __forceinline__ Pairs<V> load_pairs(const float *from) {
    Pairs<V> x;
#pragma unroll
    for (int q = 0; q < V / 4; ++q) Convert<float, 4>::unpack(reinterpret_cast<const uint4 *>(from)[q], &x.v[2 * q]);
    return x;
}
template <int V>
__device__ __forceinline__ void store_pairs(float *to, const Pairs<V> &x) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) reinterpret_cast<uint4 *>(to)[q] = Convert<float, 4>::pack(&x.v[2 * q]);
}

// The tiling that the forward and the backward scan share: 8 threads span the
// pieces of a row's block of channels, a warp four groups of consecutive
// tokens, a CTA 16. 32 values a thread, 16 where all of them are fp32 and arrive
// in twice the bytes (measured, 131072 tokens of 2048 channels, forward: bf16
// 336 us with 32, 518 with 16 in twice the threads, and as these are few long
// chains 272 with the 64 that they have now, see few_long_chains; bf16 with fp32
// gates 346 and 381; the 20011 packed fp32 tokens 62 us with 16, 63 with 32).
constexpr int kScanThreads = 128;
constexpr int kScanLanes = 8;                 // threads across the channels
constexpr int kWarpGroups = 32 / kScanLanes;  // groups per warp
template <typename XT, typename GT>
constexpr int kScanTpt = sizeof(XT) < sizeof(GT) ? 8 : 4;  // tokens per thread
template <typename XT, typename GT, int kTpt = kScanTpt<XT, GT>>
struct ScanTiling {
    static constexpr int vec = kVec<GT>, tpt = kTpt;  // channels and tokens per thread
    static constexpr int groups = kScanThreads / kScanLanes, tile = groups * tpt;
    static constexpr int ch = kScanLanes * vec;                       // channels per CTA
};
constexpr int kScanMaxRanks = 16;

// The slots of shared memory that a thread's tokens arrive in, [stage][token of
// the thread][thread]: each thread copies what it reads itself.
template <typename T, int V, int kTpt, int kThreads>
struct Slots {
    using P = Piece<T, V>;
    static constexpr size_t bytes_per_stage = (size_t)kTpt * kThreads * sizeof(P);
    static __device__ __forceinline__ P *at(void *base, int stage, int j) {
        return static_cast<P *>(base) + (stage * kTpt + j) * kThreads + threadIdx.x;
    }
    static __device__ __forceinline__ void copy(void *base, int stage, int j, const T *from) {
        const uint32_t d = (uint32_t)__cvta_generic_to_shared(at(base, stage, j));
        if (sizeof(P) == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(from) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(from) : "memory");
    }
    static __device__ __forceinline__ void fill(void *base, int stage, int j, float value) {
        const F2 v[4] = {f2(value), f2(value), f2(value), f2(value)};
        *at(base, stage, j) = Convert<T, V>::pack(v);
    }
    static __device__ __forceinline__ Pairs<V> get(void *base, int stage, int j) {
        Pairs<V> x;
        Convert<T, V>::unpack(*at(base, stage, j), x.v);
        return x;
    }
};

// Where whole warps compose maps, a lane holds a block's channels / 32: one fp32
// value, or a pair.
template <int kCh> struct Lane { using type = F2; };
template <> struct Lane<32> { using type = float; };
__device__ __forceinline__ float lane_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ F2 lane_fma(F2 a, F2 b, F2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float lane_mul(float a, float b) { return a * b; }
__device__ __forceinline__ F2 lane_mul(F2 a, F2 b) { return mul2(a, b); }
__device__ __forceinline__ void lane_set(float &x, float v) { x = v; }
__device__ __forceinline__ void lane_set(F2 &x, float v) { x = f2(v); }

__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// The exchange of tile maps between the CTAs of a cluster. Each step every CTA
// sends its map (two values per channel) to every CTA, itself included, by
// asynchronous stores that the receiver's mbarrier counts: no fence, which
// would wait for the outputs on their way to memory. Buffers alternate between
// steps: a CTA sends step i + 2 only after it has everyone's maps of step
// i + 1, which each sends after a CTA barrier that follows its reads of step i.
template <int kCh>
struct ClusterMaps {
    using L = typename Lane<kCh>::type;
    struct __align__(2 * sizeof(L)) Map {
        L a, b;
    };
    // In shared memory: two mbarriers, then [2][ranks][32] maps.
    static constexpr size_t bytes(int ranks) { return ranks > 1 ? 16 + 2 * ranks * 32 * sizeof(Map) : 0; }
    uint64_t *bar;
    int rank, ranks;
    __device__ __forceinline__ Map &map(int step, int r) const {
        return reinterpret_cast<Map *>(bar + 2)[((step & 1) * ranks + r) * 32 + (threadIdx.x & 31)];
    }
};
// All threads of the cluster, once.
template <int kCh>
__device__ __forceinline__ void cluster_maps_init(const ClusterMaps<kCh> &m) {
    if (threadIdx.x == 0) {
        tc::mbar_init(&m.bar[0], 1);
        tc::mbar_init(&m.bar[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::cluster_sync();
}
__device__ __forceinline__ void send_async(uint32_t to, uint32_t bar, float a, float b) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(a),
                 "f"(b), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send_async(uint32_t to, uint32_t bar, F2 a, F2 b) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(to),
                 "l"(a.v), "l"(b.v), "r"(bar)
                 : "memory");
}
// One warp: sends (a, b) as step `step`'s map of this CTA.
template <int kCh>
__device__ __forceinline__ void cluster_maps_send(const ClusterMaps<kCh> &m, int step, typename Lane<kCh>::type a,
                                                  typename Lane<kCh>::type b) {
    uint64_t *bar = &m.bar[step & 1];
    const auto *mine = &m.map(step, m.rank);
    if ((threadIdx.x & 31) == 0) tc::mbar_expect_tx(bar, m.ranks * 32 * (int)sizeof(*mine));
    for (int r = 0; r < m.ranks; ++r) send_async(tc::cluster_addr(mine, r), tc::cluster_addr(bar, r), a, b);
}
// Waits for the maps of step `step`. The wait always ends: the CTAs of a cluster
// run together and send as many maps. Should it not within its bound, `lost`
// (one value for the warp) is set: the warp waits for no more maps and its
// results become NaN. A CTA whose warp 0 has lost sends nothing more either, as a
// map would go to a buffer that others may still read and arm a barrier whose
// phase is not over; the others' waits for it then give up in turn.
template <int kCh>
__device__ __forceinline__ void cluster_maps_wait(const ClusterMaps<kCh> &m, int step, bool &lost) {
    if (!lost)
        lost = __any_sync(0xffffffffu,
                          !tc::mbar_wait_cluster(&m.bar[step & 1], (uint32_t)(step >> 1) & 1u, 1u << 20));
}
// The last thing that a warp does: one that has lost stays until every other
// thread of the cluster is here or gone, for maps may still be on their way into
// this CTA's shared memory. (One that has not has received all there are.) The
// wait ends, as every wait of the others has a bound.
__device__ __forceinline__ void cluster_maps_leave(bool lost) {
    if (lost) asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// A value that is the same in every lane, so that the compiler knows: it then
// keeps the loops and branches that depend on it in uniform registers (an
// unmarked sequence number cost both scans 10 %).
template <typename T>
__device__ __forceinline__ T uniform(T x) {
    return __shfl_sync(0xffffffffu, x, 0);
}

// Tokens [begin, end) of sequence n among `tokens`: offsets are clamped, so
// that no content of cu_seqlens leads out of the arrays.
__device__ __forceinline__ void scan_bounds(const int32_t *cu, int n, int T_fixed, long long tokens,
                                            long long &begin, long long &end) {
    if (!cu) {
        begin = (long long)n * T_fixed;
        end = begin + T_fixed;
        return;
    }
    begin = min(max((long long)cu[n], 0LL), tokens);
    end = min(max((long long)cu[n + 1], begin), tokens);
}

// Packed sequences are taken longest first (ties by index): the sequence whose
// place in that order is k. All threads; up to kOrderedMost sequences.
constexpr int kOrderedMost = 128;
static_assert(kOrderedMost <= kScanThreads, "a thread ranks one sequence");
__device__ __forceinline__ int kth_longest(const int32_t *cu, int num_seqs, int k, long long tokens, int *lens) {
    const int tid = threadIdx.x;
    if (tid < num_seqs) {
        long long begin, end;
        scan_bounds(cu, tid, 0, tokens, begin, end);
        lens[tid] = (int)(end - begin);
    }
    __syncthreads();
    if (tid < num_seqs) {
        const int mine = lens[tid];
        int before = 0;
        for (int m = 0; m < num_seqs; ++m) before += lens[m] > mine || (lens[m] == mine && m < tid);
        if (before == k) lens[kOrderedMost] = tid;
    }
    __syncthreads();
    const int n = uniform(lens[kOrderedMost]);
    __syncthreads();
    return n;
}

// zero(row) for the rows that no packed sequence covers, those before the first
// offset and from the last one on, shared out over the CTAs of a channel block
// (this one is number `place` of `places`) and a CTA's groups.
template <typename F>
__device__ __forceinline__ void rows_outside(const int32_t *cu, int num_seqs, long long tokens, long long place,
                                             long long places, F zero) {
    constexpr int kGroups = kScanThreads / kScanLanes;
    const long long first = min(max((long long)cu[0], 0LL), tokens);
    const long long last = min(max((long long)cu[num_seqs], first), tokens);
    const long long rows = first + tokens - last;
    for (long long k = place * kGroups + threadIdx.x / kScanLanes; k < rows; k += places * kGroups)
        zero((size_t)(k < first ? k : k - first + last));
}

// Row of `carries` that holds the state entering token
// KDA_SCAN_CARRY_TOKENS * i of the sequence.
__device__ __forceinline__ long long carry_row(long long begin, int n, long long i) {
    return begin / KDA_SCAN_CARRY_TOKENS + n + i;
}

// A forward or backward call, checked.
struct ScanArgs {
    const void *x, *g, *dout;
    const float *init, *dfinal;
    const int32_t *cu;
    void *out, *dx, *dg;
    float *final_state, *dinit, *carries;
    bool zero_outside;  // kda_scan_options, with cu only
    int T_fixed;  // tokens per sequence without cu
    long long tokens;
    int D, num_seqs;
    kda_dtype dtype, g_dtype;
    ScanGate gate;
};
cudaError_t launch_scan_fwd(const ScanArgs &s, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanArgs &s, cudaStream_t stream);

struct ScanStepArgs {
    const void *x, *g;
    float *state;
    const int32_t *slots;
    void *out;
    int N, num_slots, D;
    kda_dtype dtype, g_dtype;
    ScanGate gate;
};
cudaError_t launch_scan_step(const ScanStepArgs &s, cudaStream_t stream);

// Which sequence a CTA works on: the one that the block index gives, or the one
// that has this place among them by length. Where every sequence fits one
// warp's share of a tile (16 tokens, 32 of bf16 with fp32 gates), a kernel of
// its own gives each warp one (512 sequences of 16 tokens, 4096 channels, bf16,
// forward: 140 us with a CTA each, 49 so).
enum ScanOrder { kOrderPlain, kOrderLongest };

// Dynamic shared memory of a scan's CTA: what it needs, and at least as much as
// keeps one CTA more than S::per_sm off an SM.
template <typename S>
constexpr size_t scan_smem(int ranks) {
    constexpr size_t sm = 228 * 1024, reserved = 1024;  // of an SM; of each CTA beside its own
    constexpr size_t least = sm / (S::per_sm + 1) - sizeof(typename S::Shared) - reserved + 16;
    const size_t need = S::smem + ClusterMaps<S::ch>::bytes(ranks);
    return need > least ? need : least;
}

// How many clusters of each size of one kernel run at the same time on a device,
// looked up on first use.
struct ScanFits {
    static constexpr int kDevices = 64;
    std::atomic<int> clusters[kDevices][kScanMaxRanks + 1];  // the number and 1; 0: not looked up
};

// Launches a scan over the (sequence, channel block) pairs. CTAs per cluster:
// as many as still let all clusters run at the same time, up to the tiles that
// the longest sequence can have (bf16 backward of 32 pairs of 16384 tokens:
// 420 us with 1, 123 with 4, 88 with 8, 81 with 12, the most that fit). Where
// not even two do, up to 4 as long as that makes no more than five rounds of
// CTAs: several rounds of short ones leave the SMs less unevenly loaded than
// one of long ones (512 pairs of 4096 tokens: 230 us with 2, 193 with 4). For
// packed sequences, whose lengths the host does not know, up to 8 within three
// and a half rounds, the longest sequences first (24 of 65536 tokens in all,
// 2048 channels, backward: 314 us with 1, 246 with 2, 269 with 4; forward 202
// with 1, 145 with 2, 149 with 3, 171 with 6).
template <typename S, auto kWide, auto kNarrow, typename... A>
cudaError_t launch_scan(const ScanArgs &s, cudaStream_t stream, A... args) {
    static ScanFits fits;  // one for each kernel
    const auto kernel = kWide;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= ScanFits::kDevices) return cudaErrorInvalidDevice;
    const int blocks = (s.D + S::ch - 1) / S::ch;
    if (!s.cu && s.num_seqs > 1 && s.T_fixed <= S::tile / S::warps) {
        const long long grid = (long long)((s.num_seqs + S::warps - 1) / S::warps) * blocks;
        err = cudaFuncSetAttribute(kNarrow, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)scan_smem<S>(1));
        if (err != cudaSuccess) return err;
        kNarrow<<<(unsigned)grid, S::threads, scan_smem<S>(1), stream>>>(args..., blocks, 1, s.num_seqs, kOrderPlain, false,
                                                                 s.gate.lower);
        return cudaGetLastError();
    }
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)scan_smem<S>(kScanMaxRanks));
    if (err == cudaSuccess) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err != cudaSuccess) return err;
    const int order = s.cu && s.num_seqs > 1 && s.num_seqs <= kOrderedMost ? kOrderLongest : kOrderPlain;
    const long long units = (long long)s.num_seqs * blocks;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(S::threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto shape = [&](int ranks) {
        attr[0].val.clusterDim.x = ranks;
        cfg.gridDim = dim3((unsigned)(units * ranks));
        cfg.dynamicSmemBytes = scan_smem<S>(ranks);
    };
    auto fit = [&](int ranks) {  // clusters of this size at the same time
        int n = fits.clusters[dev][ranks].load(std::memory_order_relaxed) - 1;
        if (n >= 0) return n;
        shape(ranks);
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) err = e;
        else fits.clusters[dev][ranks].store(n + 1, std::memory_order_relaxed);
        return n;
    };
    const long long mean = s.tokens / s.num_seqs;
    int ranks = kScanMaxRanks;
    if (s.cu && s.num_seqs > 1) {
        ranks = 8;
        while (ranks > 1 && (2 * ranks * units > 7LL * fit(1) || ranks * S::tile > 2 * mean)) --ranks;
    } else {
        while (ranks > 1 && ((long long)(ranks - 1) * S::tile >= mean || fit(ranks) < units)) --ranks;
        if (ranks == 1 && units > fit(2)) {
            ranks = 4;
            while (ranks > 1 && (ranks * units > 5LL * fit(1) || ranks * S::tile > mean)) ranks /= 2;
        }
    }
    if (err != cudaSuccess) return err;
    shape(ranks);
    return cudaLaunchKernelEx(&cfg, kernel, args..., blocks, ranks, s.num_seqs, order, s.zero_outside, s.gate.lower);
}

// fn<storage type, gate type, gate, write>(args, stream) for a checked call.
#define KDA_SCAN_WRITES(fn, XT, GT, G, s, stream)                                       \
    ((s).gate.write == KDA_WRITE_PLAIN        ? fn<XT, GT, G, KDA_WRITE_PLAIN>(s, stream)      \
     : (s).gate.write == KDA_WRITE_COMPLEMENT ? fn<XT, GT, G, KDA_WRITE_COMPLEMENT>(s, stream) \
                                              : fn<XT, GT, G, KDA_WRITE_NORM>(s, stream))
#define KDA_SCAN_GATES(fn, XT, GT, s, stream)                                                        \
    ((s).gate.gate == KDA_GATE_LOG          ? KDA_SCAN_WRITES(fn, XT, GT, KDA_GATE_LOG, s, stream)        \
     : (s).gate.gate == KDA_GATE_LOGSIGMOID ? KDA_SCAN_WRITES(fn, XT, GT, KDA_GATE_LOGSIGMOID, s, stream) \
                                            : KDA_SCAN_WRITES(fn, XT, GT, KDA_GATE_BOUNDED, s, stream))
#define KDA_SCAN_DISPATCH(fn, s, stream)                                                              \
    ((s).dtype == KDA_DTYPE_F32     ? KDA_SCAN_GATES(fn, float, float, s, stream)                      \
     : (s).g_dtype == KDA_DTYPE_F32 ? KDA_SCAN_GATES(fn, __nv_bfloat16, float, s, stream)              \
                                    : KDA_SCAN_GATES(fn, __nv_bfloat16, __nv_bfloat16, s, stream))

}  // namespace kda
