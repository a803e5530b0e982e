// Shared by the gated linear recurrence's kernels (h_t = a_t h_{t-1} + w_t x_t):
// the gate functions, four-channel pieces, and the composition of affine maps.
#pragma once

#include <stdlib.h>
#include "kda_internal.cuh"

namespace kda {

constexpr int kScanVec = 4;  // channels per thread: 8 bytes of bf16, 16 of fp32

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
constexpr float kLog2E = 1.44269504088896341f;

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

// Two fp32 values that one instruction takes together (FFMA2 and its kin): the
// scans are short of issue slots before they are short of anything else.
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
    __device__ __forceinline__ F2 value() const {
        float a0, a1, c0, c1;
        split(A, a0, a1);
        split(C, c0, c1);
        return f2(c0 < 0.5f ? 1.f - c0 : a0, c1 < 0.5f ? 1.f - c1 : a1);
    }
};

// Four values as they lie in memory.
template <typename T> struct Piece;
template <> struct Piece<float> { using type = float4; };
template <> struct Piece<__nv_bfloat16> { using type = uint2; };

__device__ __forceinline__ void unpack4(const float4 &r, F2 *x) {
    x[0] = f2(r.x, r.y);
    x[1] = f2(r.z, r.w);
}
__device__ __forceinline__ void unpack4(const uint2 &r, F2 *x) {
    x[0] = f2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u));
    x[1] = f2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}
template <typename T> __device__ __forceinline__ typename Piece<T>::type pack4(const F2 *x);
template <> __device__ __forceinline__ float4 pack4<float>(const F2 *x) {
    float4 r;
    split(x[0], r.x, r.y);
    split(x[1], r.z, r.w);
    return r;
}
template <> __device__ __forceinline__ uint2 pack4<__nv_bfloat16>(const F2 *x) {
    const float4 r = pack4<float>(x);
    const __nv_bfloat162 lo = __floats2bfloat162_rn(r.x, r.y), hi = __floats2bfloat162_rn(r.z, r.w);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

// The tiling that the forward and the backward scan share.
constexpr int kScanPairs = kScanVec / 2;
constexpr int kScanLanes = 8;                         // threads across the channels
constexpr int kScanCh = kScanLanes * kScanVec;        // channels per CTA
#ifndef SCAN_THREADS
#define SCAN_THREADS 128
#endif
constexpr int kScanThreads = SCAN_THREADS;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanGroups = kScanThreads / kScanLanes;  // pieces of consecutive tokens per tile
constexpr int kWarpGroups = 32 / kScanLanes;            // and per warp
constexpr int kScanTpt = 128 / kScanGroups;                           // tokens per thread
constexpr int kScanTile = kScanGroups * kScanTpt;
constexpr size_t kSmSmem = 228 * 1024, kCtaReserved = 1024;  // shared memory of an SM, and what each CTA takes beside its own
constexpr int kScanMaxRanks = 8;
static_assert(kScanTile == KDA_SCAN_CARRY_TOKENS, "a tile begins at a saved state");
static_assert(kScanCh == 32, "one lane per channel composes a tile's maps");

// Copies one piece to shared memory without passing through registers.
template <int kBytes>
__device__ __forceinline__ void async_piece(void *smem, const void *gmem) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(smem);
    if (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(gmem) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(gmem) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The exchange of tile maps between the CTAs of a cluster. Each step every CTA
// sends its map (two floats per channel) to every CTA, itself included, by
// asynchronous stores that the receiver's mbarrier counts: no fence, which
// would wait for the outputs on their way to memory. Buffers alternate between
// steps: a CTA sends step i + 2 only after it has everyone's maps of step
// i + 1, which each sends after a CTA barrier that follows its reads of step i.
struct ClusterMaps {
    float2 map[2][kScanMaxRanks][kScanCh];
    unsigned long long bar[2];
};
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// All threads of the cluster, once.
__device__ __forceinline__ void cluster_maps_init(ClusterMaps &m) {
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&m.bar[b])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cluster_sync();
}
// One warp, lane = channel: sends (a, b) as step `step`'s map of this CTA.
__device__ __forceinline__ void cluster_maps_send(ClusterMaps &m, int step, int rank, int ranks, float a, float b) {
    const int lane = threadIdx.x & 31, p = step & 1;
    const uint32_t bar = smem_addr(&m.bar[p]), mine = smem_addr(&m.map[p][rank][lane]);
    if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                     "r"(ranks * kScanCh * (int)sizeof(float2))
                     : "memory");
    for (int r = 0; r < ranks; ++r) {
        uint32_t to, to_bar;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(mine), "r"(r));
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to_bar) : "r"(bar), "r"(r));
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                     "f"(a), "f"(b), "r"(to_bar)
                     : "memory");
    }
}
// Waits for the maps of step `step`. The wait always ends (the CTAs of a cluster
// run together and send as many maps); should it not within its bound, false
// is returned and the caller's results become NaN.
__device__ __forceinline__ bool cluster_maps_wait(ClusterMaps &m, int step) {
    const uint32_t bar = smem_addr(&m.bar[step & 1]);
    for (int polls = 0; polls < (1 << 22); ++polls) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"((uint32_t)(step >> 1) & 1u)
            : "memory");
        if (__all_sync(0xffffffffu, done)) return true;
    }
    return false;
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

// CTAs per cluster, i.e. tiles of one (sequence, channel block) in flight at
// once: as many as still run all at the same time (`slots` CTAs fit the GPU),
// up to the tiles that the longest sequence can have.
inline int scan_ranks(long long units, long long longest, long long slots) {
    if (const char *e = getenv("KDA_RANKS")) return atoi(e);
    int ranks = 1;
    while (ranks < kScanMaxRanks && 2 * ranks * units <= slots && (long long)ranks * kScanTile < longest) ranks *= 2;
    return ranks;
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
