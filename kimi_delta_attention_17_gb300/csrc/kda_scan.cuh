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
__device__ __forceinline__ float max_nan(float x, float y) {  // NaN stays NaN
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// a = e^x and c = 1 - a for a log-decay x <= 0. Near 0 both come from the
// Taylor series of e^x - 1 (to x^7 / 7!, off by less than |x|^7 / 8! < 2e-8
// relative for |x| < 0.35): 1 - e^x from a rounded e^x would lose the digits
// of a small 1 - a.
__device__ __forceinline__ void decay_pair(float x, float &a, float &c) {
    float p = 1.f / 5040.f;
    p = fmaf(p, x, 1.f / 720.f);
    p = fmaf(p, x, 1.f / 120.f);
    p = fmaf(p, x, 1.f / 24.f);
    p = fmaf(p, x, 1.f / 6.f);
    p = fmaf(p, x, 0.5f);
    p = fmaf(p, x, 1.f);
    const float m = p * x;  // e^x - 1
    const float e = ex2_approx(x * kLog2E);
    const bool small = fabsf(x) < 0.35f;
    a = small ? 1.f + m : e;
    c = small ? -m : 1.f - e;
}

// sigmoid(z) and 1 - sigmoid(z) = t sigmoid(z) with t = e^-z, both accurate to
// a few units in their own last place. Below -80 sigmoid(z) is taken as
// e^-80 = 2e-35, so that t stays finite.
__device__ __forceinline__ void sigmoid_pair(float z, float &s, float &c) {
    const float t = ex2_approx(max_nan(z, -80.f) * -kLog2E);
    s = rcp_approx(1.f + t);
    c = t * s;
}

// What one gate value gives: a, the input weight w, 1 - a or log a (`rest`,
// for Decay), and, for the backward pass, slope = dlog a/dg and wslope = dw/dg.
struct Gated {
    float a, w, rest, slope, wslope;
};

template <int kGate, int kWrite, bool kGrad>
__device__ __forceinline__ Gated gate_value(float z, float lower) {
    Gated r;
    float c;  // 1 - a
    r.slope = 1.f;
    if (kGate == KDA_GATE_LOGSIGMOID) {
        sigmoid_pair(z, r.a, c);
        r.slope = r.rest = c;
    } else {
        r.rest = z;
        if (kGate == KDA_GATE_BOUNDED) {
            float s, sc;
            sigmoid_pair(z, s, sc);
            r.rest = lower * s;
            r.slope = r.rest * sc;
        }
        if (kWrite == KDA_WRITE_PLAIN)
            r.a = ex2_approx(r.rest * kLog2E);
        else
            decay_pair(r.rest, r.a, c);
    }
    r.wslope = 0.f;
    if (kWrite == KDA_WRITE_PLAIN) {
        r.w = 1.f;
    } else if (kWrite == KDA_WRITE_COMPLEMENT) {
        r.w = c;
        if (kGrad) r.wslope = -r.a * r.slope;  // dw/dlog a = -a
    } else {
        r.w = sqrt_approx(fmaf(c, r.a, c));  // 1 - a^2 from its factors
        // dw/dlog a = -a^2 / w. Under the logistic gate dlog a/dg = 1 - a
        // cancels the division: w^2 = (1 - a)(1 + a).
        if (kGrad)
            r.wslope = kGate == KDA_GATE_LOGSIGMOID
                           ? -r.a * r.a * r.w * rcp_approx(1.f + r.a)
                           : (r.w > 0.f ? -r.a * r.a * r.slope * rcp_approx(r.w) : 0.f);
    }
    return r;
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
    float sum = 0.f;
    __device__ __forceinline__ void then(const Gated &q) { sum += q.rest; }
    __device__ __forceinline__ float value() const {
        float a, c;
        decay_pair(sum, a, c);
        return a;
    }
};
template <>
struct Decay<KDA_GATE_LOGSIGMOID> {
    float A = 1.f, C = 0.f;
    __device__ __forceinline__ void then(const Gated &q) {
        A *= q.a;
        C = fmaf(-C, q.rest, C + q.rest);
    }
    __device__ __forceinline__ float value() const { return C < 0.5f ? 1.f - C : A; }
};

// Four values as they lie in memory.
template <typename T> struct Piece;
template <> struct Piece<float> { using type = float4; };
template <> struct Piece<__nv_bfloat16> { using type = uint2; };

__device__ __forceinline__ void unpack4(const float4 &r, float *x) {
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
}
__device__ __forceinline__ void unpack4(const uint2 &r, float *x) {
    x[0] = __uint_as_float(r.x << 16);
    x[1] = __uint_as_float(r.x & 0xFFFF0000u);
    x[2] = __uint_as_float(r.y << 16);
    x[3] = __uint_as_float(r.y & 0xFFFF0000u);
}
template <typename T> __device__ __forceinline__ typename Piece<T>::type pack4(const float *x);
template <> __device__ __forceinline__ float4 pack4<float>(const float *x) {
    return make_float4(x[0], x[1], x[2], x[3]);
}
template <> __device__ __forceinline__ uint2 pack4<__nv_bfloat16>(const float *x) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

// The tiling that the forward and the backward scan share.
constexpr int kScanLanes = 8;                         // threads across the channels
constexpr int kScanCh = kScanLanes * kScanVec;        // channels per CTA
constexpr int kScanThreads = 128;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanTpt = 8;                           // tokens per thread
constexpr int kScanTile = kScanThreads / kScanLanes * kScanTpt;
constexpr int kScanStages = 2;
constexpr int kScanMaxRanks = 8;
static_assert(kScanTile == KDA_SCAN_CARRY_TOKENS, "a tile begins at a saved state");
static_assert(kScanCh == 32, "a warp composes the CTA's maps with one lane per channel");

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
// A barrier over every thread of the cluster; what a thread wrote before it,
// into any CTA's shared memory, is seen after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_peer(float *mine, uint32_t rank, float v) {
    uint32_t peer;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(peer)
                 : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer), "f"(v) : "memory");
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
