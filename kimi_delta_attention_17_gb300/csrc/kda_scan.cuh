// Shared by the gated linear recurrence's kernels (h_t = a_t h_{t-1} + w_t x_t):
// the gate functions, four-channel pieces, and the composition of affine maps.
#pragma once

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

// a = e^x and c = 1 - a for a log-decay x <= 0. Near 0 both come from the
// Taylor series of e^x - 1 (to x^7 / 7!, off by less than |x|^7 / 8! < 2e-8
// relative for |x| < 0.35): 1 - e^x from a rounded e^x would lose the digits
// of a small 1 - a, and a biased rounding of an a near 1 adds up over the
// 1 / (1 - a) tokens that a slow channel remembers.
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

// sigmoid(z) and 1 - sigmoid(z), each to a few units in its own last place
// (the smaller of the two is t / (1 + t) with t = e^-|z| <= 1; the larger its
// difference from 1).
__device__ __forceinline__ void sigmoid_pair(float z, float &s, float &c) {
    const float t = ex2_approx(-fabsf(z) * kLog2E);
    const float m = t * rcp_approx(1.f + t);
    const float l = 1.f - m;
    s = z >= 0.f ? l : m;
    c = z >= 0.f ? m : l;
}

// What one gate value gives: a, c = 1 - a, the input weight w, and, for the
// backward pass, slope = dlog a/dg and wslope = dw/dg.
struct Gated {
    float a, c, w, slope, wslope;
};

// The decay over a thread's tokens: a product A of decays, and with it C = 1 - A
// from the tokens' 1 - a. Slow channels need C: of two factors 1 - p and 1 - q
// with p q < 2^-25 the rounded product loses p q every time, always to the same
// side, which over the thousands of tokens that such a channel remembers comes
// to hundreds of roundings (measured at a ~ 0.9999 over 6000 tokens: 430 x 2^-24
// off by products alone).
struct Decay {
    float A = 1.f, C = 0.f;
    __device__ __forceinline__ void then(float a, float c) {
        A *= a;
        C = fmaf(-C, c, C + c);
    }
    __device__ __forceinline__ float value() const { return C < 0.5f ? 1.f - C : A; }
};

template <int kGate, int kWrite, bool kGrad>
__device__ __forceinline__ Gated gate_value(float z, float lower) {
    Gated r;
    float c;
    r.slope = 1.f;
    if (kGate == KDA_GATE_LOGSIGMOID) {
        sigmoid_pair(z, r.a, c);
        r.slope = c;
    } else if (kGate == KDA_GATE_BOUNDED) {
        float s, sc;
        sigmoid_pair(z, s, sc);
        const float la = lower * s;
        decay_pair(la, r.a, c);
        r.slope = la * sc;
    } else {
        decay_pair(z, r.a, c);
    }
    r.c = c;
    r.wslope = 0.f;
    if (kWrite == KDA_WRITE_PLAIN) {
        r.w = 1.f;
    } else if (kWrite == KDA_WRITE_COMPLEMENT) {
        r.w = c;
        if (kGrad) r.wslope = -r.a * r.slope;  // dw/dlog a = -a
    } else {
        r.w = sqrtf(c * (1.f + r.a));  // 1 - a^2 from its factors
        // dw/dlog a = -a^2 / w. Under the logistic gate dlog a/dg = 1 - a
        // cancels the division: w^2 = (1 - a)(1 + a).
        if (kGrad)
            r.wslope = kGate == KDA_GATE_LOGSIGMOID
                           ? -r.a * r.a * r.w * rcp_approx(1.f + r.a)
                           : (r.w > 0.f ? -r.a * r.a * r.slope * rcp_approx(r.w) : 0.f);
    }
    return r;
}

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
__device__ __forceinline__ void store_peer4(uint32_t addr, uint32_t rank, const float *v) {
    uint32_t peer;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(peer), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3])
                 : "memory");
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
// once: more while the units alone leave SMs without work, up to the tiles
// that the longest sequence can have.
inline int scan_ranks(long long units, long long longest, int tile) {
    int ranks = 1;
    while (ranks < 8 && units * ranks < 2 * 152 && (long long)ranks * tile < longest) ranks *= 2;
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
