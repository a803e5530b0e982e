// The recurrent delta rule over several tokens a row (drafts to verify, accepted tokens to commit, a
// short continuation), one pass over the state whatever their number:
//     S~ = Diag(a_t) S,  e_t = beta_t (v_t - S~^T k_t),  S = S~ + k_t e_t^T,  o_t = S^T (s q_t).
//
// Tokens are taken in blocks of kBlock. With G_t the product of the decays up to t in the block and
// G_{j:t} that of tokens j + 1 .. t (products of factors <= 1: no quotient is formed, however steep they are),
//     P_t = S0^T (G_t o k_t),   R_t = S0^T (G_t o s q_t),
//     A_tj = sum_c k_t k_j G_{j:t},   H_tj = sum_c s q_t k_j G_{j:t},
//     e_t = beta_t (v_t - P_t - sum_{j<t} A_tj e_j),   o_t = R_t + sum_{j<=t} H_tj e_j,
//     S  <- G_C o S0 + sum_j (G_{j:C} o k_j) e_j^T,
// so the state is read once and updated once a block, both as matrix products over all its tokens.
//
// A warp owns 32 columns of the state and keeps them in registers over all blocks. The products run on
// mma.sync m16n8k8 with the state transposed (m: its columns, so that A's fragment of the read and C's of the
// update are the same registers: the order of the rows within eight is free in a sum). Operands are split
// into two tf32 parts, x = hi + lo, and three products hi hi + hi lo + lo hi taken: off by some 2^-22 of the
// magnitudes, as fp32 sums are. (The state's rows go through 16 columns x 8 rows a time, and there are at most
// 16 vectors to multiply: far too small for tcgen05, whose operands would have to pass through shared memory.)
// One token at a time in fp32, two rows an instruction, took 33 us a token on 256 x 32 heads of 128: as many
// cycles for the factors' way out of shared memory as for the arithmetic.
//
// The tokens' inputs come by asynchronous copies beside the state, which is on its way while they are
// prepared; the next block's come behind the block before it.
#include "kda_rows.cuh"

namespace kda {
namespace {

constexpr int kBlock = 8;  // tokens a block: an MMA's n

__device__ __forceinline__ void copy16(void *smem, const void *gmem) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(gmem) : "memory");
}

// The nearest value of 11 bits. (NaN may come out as a zero: what is left of it, x - hi, is NaN still.)
__device__ __forceinline__ float tf32_hi(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }

// c += a b: a 16 x 8 (row m = lane / 4 and m + 8; column k = lane % 4 and k + 4), b 8 x 8 (row k, column
// n = lane / 4), c 16 x 8 (row m; columns 2 (lane % 4) and the next).
__device__ __forceinline__ void mma_tf32(float *c, const float *a, float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// kN consecutive values in shared memory as fp32.
template <int kN>
__device__ __forceinline__ void some_of(const float *p, float *x) {
    if constexpr (kN == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x; x[1] = v.y;
    }
}
template <int kN>
__device__ __forceinline__ void some_of(const __nv_bfloat16 *p, float *x) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t *>(p + i);
        x[i] = __uint_as_float(v << 16);
        x[i + 1] = __uint_as_float(v & 0xffff0000u);
    }
}

constexpr int kCols = 16;  // state columns a warp: an MMA's m

template <int D, typename InT>
struct TokenSmem {
    static constexpr int kRead = 2 * D + 16, kWrite = 2 * D + 8, kTrans = 20;  // strides without bank conflicts
    float read[2][kBlock][kRead];  // G k and G s q: for rows r, r + 1 (r even) hi, hi', lo, lo'
    float write[kBlock][kWrite];   // G_{j:C} k: hi, lo of each row
    float trans[D / kCols][2 * kBlock][kTrans];  // a warp's values, columns across
    float total[D];                // G_C
    float a[kBlock][D];            // g, then a
    InT q[kBlock][D], k[kBlock][D], v[kBlock][D];
    float A[kBlock][kBlock], Hm[kBlock][kBlock];
    float beta[kBlock], rk[kBlock], rq[kBlock];
};

template <int D, typename InT>
__global__ void __launch_bounds__(2 * D, D == 128 ? 2 : 4)
decode_tokens_kernel(const InT *__restrict__ q, const InT *__restrict__ k, const InT *__restrict__ v,
                     const float *__restrict__ g, const float *__restrict__ beta, float scale, float *__restrict__ state,
                     const int32_t *__restrict__ slots, int num_slots, const int32_t *__restrict__ counts, int K, int H,
                     InT *__restrict__ out, int write_state, Prologue pro) {
    constexpr int KT = D / 8;   // row tiles
    constexpr int T = 2 * D;    // threads: D / kCols warps
    extern __shared__ __align__(16) unsigned char raw[];
    auto &sm = *reinterpret_cast<TokenSmem<D, InT> *>(raw);
    const int n = blockIdx.x / H, head = blockIdx.x % H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = slots ? slots[n] : n;
    int count = counts ? min(max(counts[n], 0), K) : K;
    const size_t row0 = (size_t)n * K * H + head;  // token t's row: row0 + t H

    // Inputs of tokens [t0, t0 + some) on their way into shared memory. A warp fetches the v of its own columns.
    constexpr int E = 16 / (int)sizeof(InT), kIn = D / E, kV = kCols / E, kG = D / 4;  // 16-byte pieces of a row
    auto fetch = [&](int t0, int some) {
        for (int p = tid; p < some * kIn; p += T) {
            const int i = p / kIn, c = p % kIn * E;
            const size_t at = (row0 + (size_t)(t0 + i) * H) * D + c;
            copy16(&sm.q[i][c], q + at);
            copy16(&sm.k[i][c], k + at);
        }
        if (pro.decay == KDA_DECAY_CHANNEL)
            for (int p = tid; p < some * kG; p += T) {
                const int i = p / kG, c = p % kG * 4;
                copy16(&sm.a[i][c], g + (row0 + (size_t)(t0 + i) * H) * D + c);
            }
    };
    auto fetch_v = [&](int t0, int some) {
        for (int p = lane; p < some * kV; p += 32) {
            const int i = p / kV, c = warp * kCols + p % kV * E;
            copy16(&sm.v[i][c], v + (row0 + (size_t)(t0 + i) * H) * D + c);
        }
    };
    // The first block's, before the slot and the count are here.
    fetch(0, min(kBlock, K));
    fetch_v(0, min(kBlock, K));
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (slot < 0 || slot >= num_slots) count = 0;
    if (out)
        for (int p = count * D + tid; p < K * D; p += T) out[(row0 + (size_t)(p / D) * H) * D + p % D] = from_f32<InT>(0.f);
    if (count == 0) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        return;
    }

    // Rows 8 i + 2 x and the next, columns 2 y and 2 y + 1 of the warp's.
    const int x = lane & 3, y = lane >> 2;
    float *S = state + ((size_t)slot * H + head) * D * D + (size_t)(2 * x) * D + warp * kCols + 2 * y;
    float s[KT][2][2];
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 w = *reinterpret_cast<const float2 *>(S + (size_t)(8 * i + r) * D);
            s[i][r][0] = w.x;
            s[i][r][1] = w.y;
        }

    for (int t0 = 0; t0 < count; t0 += kBlock) {
        const int some = min(kBlock, count - t0);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // the inputs are here, and no warp reads the block before them
        if (pro.decay == KDA_DECAY_CHANNEL) {
            for (int p = tid; p < some * (D / 4); p += T) {
                float4 *at = reinterpret_cast<float4 *>(&sm.a[p / (D / 4)][p % (D / 4) * 4]);
                const float4 z = *at;
                *at = make_float4(decay_factor(z.x, pro), decay_factor(z.y, pro), decay_factor(z.z, pro), decay_factor(z.w, pro));
            }
        } else {
            for (int p = tid; p < some * D; p += T)
                sm.a[p / D][p % D] = pro.decay == KDA_DECAY_NONE ? 1.f : decay_factor(g[row0 + (size_t)(t0 + p / D) * H], pro);
        }
        if (tid < some) sm.beta[tid] = beta[row0 + (size_t)(t0 + tid) * H];
        __syncthreads();
        // Of the warps, D / 64 each form the vectors of the reads by k, by q and of the update, two channels a
        // lane; then each takes tokens j: A_tj, H_tj for t >= j (A_jj is |k_j|^2), and |q_j|^2. The last warps,
        // whose j have the fewest t, have the vectors.
        constexpr int kW = T / 32, kPer = D / 64;
        if (const int role = (kW - 1 - warp) / kPer; role < 2) {
            const int c = ((kW - 1 - warp) % kPer * 32 + lane) * 2;
            const float f = role ? scale : 1.f;
            const InT(*from)[D] = role ? sm.q : sm.k;
            float G[2] = {1.f, 1.f};
#pragma unroll
            for (int i = 0; i < kBlock; ++i) {
                if (i >= some) break;  // what the places behind hold stays in their columns of the product
                float a[2], z[2];
                some_of<2>(&sm.a[i][c], a);
                some_of<2>(&from[i][c], z);
                G[0] *= a[0];
                G[1] *= a[1];
                const float w0 = G[0] * (f * z[0]), w1 = G[1] * (f * z[1]), h0 = tf32_hi(w0), h1 = tf32_hi(w1);
                *reinterpret_cast<float4 *>(&sm.read[role][i][2 * c]) = make_float4(h0, h1, w0 - h0, w1 - h1);
            }
        } else if (role == 2) {
            const int c = ((kW - 1 - warp) % kPer * 32 + lane) * 2;
            float G[2] = {1.f, 1.f};
#pragma unroll
            for (int i = kBlock - 1; i >= 0; --i) {
                float a[2] = {1.f, 1.f}, z[2] = {0.f, 0.f};
                if (i < some) {
                    some_of<2>(&sm.a[i][c], a);
                    some_of<2>(&sm.k[i][c], z);
                }
                const float w0 = G[0] * z[0], w1 = G[1] * z[1], h0 = tf32_hi(w0), h1 = tf32_hi(w1);
                *reinterpret_cast<float4 *>(&sm.write[i][2 * c]) = make_float4(h0, w0 - h0, h1, w1 - h1);
                G[0] *= a[0];
                G[1] *= a[1];
            }
            *reinterpret_cast<float2 *>(&sm.total[c]) = make_float2(G[0], G[1]);
        }
        for (int j = warp; j < some; j += kW) {
            constexpr int kC = D / 32;  // channels a lane
            const int c = kC * lane;
            float acc[2 * kBlock], w[kC], qss = 0.f;
            some_of<kC>(&sm.k[j][c], w);
#pragma unroll
            for (int t = 0; t < kBlock; ++t) {
                acc[t] = acc[kBlock + t] = 0.f;
                if (t < j || t >= some) continue;
                float kt[kC], qt[kC];
                some_of<kC>(&sm.k[t][c], kt);
                some_of<kC>(&sm.q[t][c], qt);
                if (t > j) {
                    float a[kC];
                    some_of<kC>(&sm.a[t][c], a);
#pragma unroll
                    for (int m = 0; m < kC; ++m) w[m] *= a[m];
                } else {
#pragma unroll
                    for (int m = 0; m < kC; ++m) qss += qt[m] * qt[m];
                }
#pragma unroll
                for (int m = 0; m < kC; ++m) {
                    acc[t] += kt[m] * w[m];
                    acc[kBlock + t] += qt[m] * w[m];
                }
            }
            // Sixteen sums over the warp: every step halves the values a lane holds.
#pragma unroll
            for (int m = 16, left = kBlock; left > 0; m >>= 1, left >>= 1) {
                const bool up = lane & m;
#pragma unroll
                for (int i = 0; i < left; ++i) {
                    const float keep = up ? acc[i + left] : acc[i], send = up ? acc[i] : acc[i + left];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
            }
            const float sum = acc[0] + __shfl_xor_sync(0xffffffffu, acc[0], 1);
            const int t = lane >> 1 & 7;
            if ((lane & 1) == 0 && t >= j) (lane < 16 ? sm.A : sm.Hm)[t][j] = lane < 16 ? sum : scale * sum;
            if (pro.l2norm) {
                qss = lanes_sum<32>(qss);
                const float kss = __shfl_sync(0xffffffffu, sum, 2 * j);
                if (lane == 0) {
                    sm.rk[j] = rsqrtf(kss + kL2Eps);
                    sm.rq[j] = rsqrtf(qss + kL2Eps);
                }
            } else if (lane == 0) {
                sm.rk[j] = sm.rq[j] = 1.f;
            }
        }
        __syncthreads();
        const int next = min(kBlock, count - t0 - kBlock);
        if (next > 0) fetch(t0 + kBlock, next);

        // P and R, 16 columns by 8 tokens each: in one product where there are at most four tokens (the eight
        // vectors of its n are then k's and q's), else in two. Two accumulators each shorten the chains.
        float acc[2][2][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i >> 3][i >> 2 & 1][i & 3] = 0.f;
        const bool both = some <= kBlock / 2;
        const float *from = both ? sm.read[y >> 2][y & 3] : sm.read[0][y];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const float4 b0 = *reinterpret_cast<const float4 *>(from + 16 * i + 4 * x);
            float hi[4], lo[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float w = s[i][c >> 1][c & 1];
                hi[c] = tf32_hi(w);
                lo[c] = w - hi[c];
            }
            mma_tf32(acc[0][0], hi, b0.x, b0.y);
            mma_tf32(acc[0][1], lo, b0.x, b0.y);
            mma_tf32(acc[0][1], hi, b0.z, b0.w);
            if (!both) {
                const float4 b1 = *reinterpret_cast<const float4 *>(&sm.read[1][y][16 * i + 4 * x]);
                mma_tf32(acc[1][0], hi, b1.x, b1.y);
                mma_tf32(acc[1][1], lo, b1.x, b1.y);
                mma_tf32(acc[1][1], hi, b1.z, b1.w);
            }
        }
        // A lane takes one column over all tokens: both halves of the warp solve for e, each forms the outputs of
        // every other token.
        float(*tr)[TokenSmem<D, InT>::kTrans] = sm.trans[warp];
        const int own = lane & 15, odd = lane >> 4;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int to = both ? 2 * x + (x & 2) * (kBlock / 4) : b * kBlock + 2 * x;  // R's rows begin at kBlock
            if (b && both) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][0][i] += acc[b][1][i];
            *reinterpret_cast<float2 *>(&tr[to][2 * y]) = make_float2(acc[b][0][0], acc[b][0][2]);
            *reinterpret_cast<float2 *>(&tr[to + 1][2 * y]) = make_float2(acc[b][0][1], acc[b][0][3]);
        }
        __syncwarp();
        float ke[kBlock];
#pragma unroll
        for (int t = 0; t < kBlock; ++t) {
            ke[t] = 0.f;
            if (t < some) {
                float u = tr[t][own];
#pragma unroll
                for (int j = 0; j < t; ++j) u += sm.A[t][j] * ke[j];
                // The reads are linear in k and q, which are normalised here.
                ke[t] = sm.rk[t] * (sm.beta[t] * (to_f32(sm.v[t][warp * kCols + own]) - sm.rk[t] * u));
            }
        }
        if (out) {
#pragma unroll
            for (int i = 0; i < kBlock / 2; ++i) {
                const int t = 2 * i + odd;
                if (t >= some) continue;
                float o = tr[kBlock + t][own];
#pragma unroll
                for (int j = 0; j < 2 * i + 1; ++j) o += sm.Hm[t][j] * ke[j];
                if (odd) o += sm.Hm[t][t] * ke[2 * i + 1];
                out[(row0 + (size_t)(t0 + t) * H) * D + warp * kCols + own] = from_f32<InT>(sm.rq[t] * o);
            }
        }
        if (next <= 0 && !write_state) return;
        __syncwarp();
        if (odd == 0) {
#pragma unroll
            for (int t = 0; t < kBlock; ++t) tr[t][own] = ke[t];
        }
        __syncwarp();
        if (next > 0) fetch_v(t0 + kBlock, next);
        asm volatile("cp.async.commit_group;" ::: "memory");
        // S <- G_C S + k e^T, the same registers as accumulators.
        float hi[4], lo[4];
        {
            float e[2][2];
            some_of<2>(&tr[x][2 * y], e[0]);
            some_of<2>(&tr[x + 4][2 * y], e[1]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float w = e[c >> 1][c & 1];
                hi[c] = tf32_hi(w);
                lo[c] = w - hi[c];
            }
        }
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const float2 tot = *reinterpret_cast<const float2 *>(&sm.total[8 * i + 2 * x]);
            const float2 w0 = *reinterpret_cast<const float2 *>(&sm.write[x][2 * (8 * i + y)]);
            const float2 w1 = *reinterpret_cast<const float2 *>(&sm.write[x + 4][2 * (8 * i + y)]);
            float c[4] = {tot.x * s[i][0][0], tot.y * s[i][1][0], tot.x * s[i][0][1], tot.y * s[i][1][1]};
            mma_tf32(c, lo, w0.x, w1.x);
            mma_tf32(c, hi, w0.y, w1.y);
            mma_tf32(c, hi, w0.x, w1.x);
            s[i][0][0] = c[0];
            s[i][1][0] = c[1];
            s[i][0][1] = c[2];
            s[i][1][1] = c[3];
        }
    }
#pragma unroll
    for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
            *reinterpret_cast<float2 *>(S + (size_t)(8 * i + r) * D) = make_float2(s[i][r][0], s[i][r][1]);
}

template <int D, typename InT>
cudaError_t launch_tokens_t(const TokensArgs &a, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(TokenSmem<D, InT>);
    const cudaError_t err =
        cudaFuncSetAttribute(decode_tokens_kernel<D, InT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    decode_tokens_kernel<D, InT><<<(unsigned)((long long)a.N * a.H), 2 * D, smem, stream>>>(
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
