// The recurrent delta rule over several tokens a row (drafts to verify, accepted tokens to commit, a
// short continuation), one pass over the state whatever their number:
//     S~ = Diag(a_t) S,  e = beta_t (v_t - S~^T k_t),  S = S~ + k_t e^T,  o_t = S^T (s q_t).
// As in the single-token step the output is read from the old state, o = S^T (a o s q) + (s q.k) e.
//
// The columns of S never meet, so a warp owns 32 of them and keeps its d x 32 slab in registers over all
// tokens: 8 lanes across (four columns each) by 4 lanes down (every fourth row each). The sums over the
// key channels are a thread's own rows and two shuffles; no barrier stands between tokens. What the
// slabs of a head share (a, k, a o k, a o s q per channel, q.k, the norms) is prepared for kTokens tokens
// at a time by all of the head's threads, one channel each, into shared memory.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kTokens = 4;  // tokens prepared together

template <int D, typename InT>
__global__ void __launch_bounds__(D)
decode_tokens_kernel(const InT *__restrict__ q, const InT *__restrict__ k, const InT *__restrict__ v,
                     const float *__restrict__ g, const float *__restrict__ beta, float scale, float *__restrict__ state,
                     const int32_t *__restrict__ slots, int num_slots, const int32_t *__restrict__ counts, int K, int H,
                     InT *__restrict__ out, int write_state, Prologue pro) {
    constexpr int R = D / 4, kWarps = D / 32;
    __shared__ float4 coef[kTokens][D];        // a k, a s q, a, k
    __shared__ float vals[kTokens][D];
    __shared__ float sums[kTokens][kWarps][3];  // s q.k, |k|^2, |q|^2 of each warp's channels
    __shared__ float betas[kTokens];
    const int n = blockIdx.x / H, head = blockIdx.x % H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = slots ? slots[n] : n;
    int count = counts ? min(max(counts[n], 0), K) : K;
    if (slot < 0 || slot >= num_slots) count = 0;
    const size_t row0 = (size_t)n * K * H + head;  // token t's row: row0 + t H
    if (out)
        for (int t = count; t < K; ++t) out[(row0 + (size_t)t * H) * D + tid] = from_f32<InT>(0.f);
    if (count == 0) return;

    const int cq = lane & 7, rg = lane >> 3, col = warp * 32 + 4 * cq;
    float *S = state + ((size_t)slot * H + head) * D * D + col;
    float4 s[R];
#pragma unroll
    for (int m = 0; m < R; ++m) s[m] = *reinterpret_cast<const float4 *>(S + (size_t)(rg + 4 * m) * D);

    for (int t0 = 0; t0 < count; t0 += kTokens) {
        const int some = min(kTokens, count - t0);
        if (t0) __syncthreads();
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if (i >= some) break;
            const size_t row = row0 + (size_t)(t0 + i) * H, at = row * D + tid;
            const float a = pro.decay == KDA_DECAY_CHANNEL  ? decay_factor(g[at], pro)
                            : pro.decay == KDA_DECAY_SCALAR ? decay_factor(g[row], pro)
                                                            : 1.f;
            const float kk = to_f32(k[at]), q0 = to_f32(q[at]), qq = scale * q0;
            coef[i][tid] = make_float4(a * kk, a * qq, a, kk);
            vals[i][tid] = to_f32(v[at]);
            if (tid == 0) betas[i] = beta[row];
            float x[3] = {qq * kk, kk * kk, q0 * q0};
#pragma unroll
            for (int j = 0; j < 3; ++j) {
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) x[j] += __shfl_xor_sync(0xffffffffu, x[j], m);
                if (lane == 0) sums[i][warp][j] = x[j];
            }
        }
        __syncthreads();
        for (int i = 0; i < some; ++i) {
            float qk = 0.f, kss = 0.f, qss = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                qk += sums[i][w][0];
                kss += sums[i][w][1];
                qss += sums[i][w][2];
            }
            float vh[4] = {0.f, 0.f, 0.f, 0.f}, po[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const float4 c = coef[i][rg + 4 * m];
                vh[0] += c.x * s[m].x; vh[1] += c.x * s[m].y; vh[2] += c.x * s[m].z; vh[3] += c.x * s[m].w;
                po[0] += c.y * s[m].x; po[1] += c.y * s[m].y; po[2] += c.y * s[m].z; po[3] += c.y * s[m].w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int m = 8; m < 32; m <<= 1) {
                    vh[j] += __shfl_xor_sync(0xffffffffu, vh[j], m);
                    po[j] += __shfl_xor_sync(0xffffffffu, po[j], m);
                }
            }
            // The reads are linear in k and q: they are normalised afterwards.
            const float rk = pro.l2norm ? rsqrtf(kss + kL2Eps) : 1.f, rq = pro.l2norm ? rsqrtf(qss + kL2Eps) : 1.f;
            qk *= rk * rq;
            const float4 vv = *reinterpret_cast<const float4 *>(&vals[i][col]);
            const float b = betas[i];
            const float e[4] = {b * (vv.x - vh[0] * rk), b * (vv.y - vh[1] * rk), b * (vv.z - vh[2] * rk),
                                b * (vv.w - vh[3] * rk)};
            if (out && rg == 0) {
                InT *to = out + (row0 + (size_t)(t0 + i) * H) * D + col;
#pragma unroll
                for (int j = 0; j < 4; ++j) to[j] = from_f32<InT>(po[j] * rq + qk * e[j]);
            }
            const float ke[4] = {rk * e[0], rk * e[1], rk * e[2], rk * e[3]};
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const float4 c = coef[i][rg + 4 * m];
                s[m].x = c.z * s[m].x + c.w * ke[0];
                s[m].y = c.z * s[m].y + c.w * ke[1];
                s[m].z = c.z * s[m].z + c.w * ke[2];
                s[m].w = c.z * s[m].w + c.w * ke[3];
            }
        }
    }
    if (write_state) {
#pragma unroll
        for (int m = 0; m < R; ++m) *reinterpret_cast<float4 *>(S + (size_t)(rg + 4 * m) * D) = s[m];
    }
}

template <int D, typename InT>
cudaError_t launch_tokens_t(const TokensArgs &a, cudaStream_t stream) {
    decode_tokens_kernel<D, InT><<<(unsigned)((long long)a.N * a.H), D, 0, stream>>>(
        static_cast<const InT *>(a.q), static_cast<const InT *>(a.k), static_cast<const InT *>(a.v), a.g, a.beta, a.scale,
        a.state, a.slots, a.num_slots, a.counts, a.K, a.H, static_cast<InT *>(a.out), a.write_state, a.pro);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tokens(const TokensArgs &a, cudaStream_t stream) {
    if (a.N == 0 || a.K == 0) return cudaSuccess;
    if (a.dtype == KDA_DTYPE_BF16)
        return a.d == 128 ? launch_tokens_t<128, __nv_bfloat16>(a, stream) : launch_tokens_t<64, __nv_bfloat16>(a, stream);
    return a.d == 128 ? launch_tokens_t<128, float>(a, stream) : launch_tokens_t<64, float>(a, stream);
}

}  // namespace kda
