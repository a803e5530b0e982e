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
// Two warps own 32 columns of the state, each half of the rows, and keep them in registers over all blocks (32
// columns, so that a row's pieces fill the lines of global and shared memory that they are in; half of the rows,
// so that eight warps a head have registers enough); they add up their halves of P and R. The products run on
// mma.sync m16n8k8 with the state transposed (m: its columns, so that A's fragment of the read and C's of the
// update are the same registers: the order of the rows within eight is free in a sum). Operands are split
// into two tf32 parts, x = hi + lo, and three products hi hi + hi lo + lo hi taken: off by some 2^-22 of the
// magnitudes, as fp32 sums are. (The state's rows go through 16 columns x 8 rows a time, and there are at most
// 16 vectors to multiply: far too small for tcgen05, whose operands would have to pass through shared memory.)
// One token at a time in fp32, two rows an instruction, took 33 us a token on 256 x 32 heads of 128.
//
// CTAs stay and take (row, head) pairs in turn. Teams of three warps prepare what the columns of a head share, a
// block or two ahead of the warps that work, and one warp moves the states, by TMA between global memory and two
// buffers in shared memory, so that a head's state comes and goes while another is worked on. (Loaded into
// registers, four rows of 64 bytes an instruction, the states kept the load unit busy for 2500 of 8500 cycles a
// head, and everything behind them in its queue waited; row by row, 128 bulk copies of 512 bytes took 8000
// cycles to issue.)
//
// 256 rows, 32 heads of 128: up to 8 tokens each committed 185-187 us (5.4 TB/s), 8 each 216, 4 each 186, one 181 (the
// single step takes 182), 16 each 389; 8 verified 162, 4 verified 113, one 103, 16 verified 328. HBM bounds the calls
// of few tokens that write states (1.07 GB: 158 us); with more, a head's chain of phases does (cycles with 8 tokens:
// copy waited for and state into registers 1400, read 2600, solve 800, outputs 700, update 1700, state out 500), and
// with 8 the teams that prepare come close to it; 40 % of the issue slots are busy. With fp32 inputs, which leave
// shared memory for one team, it bounds the call: 8 committed 291, verified 219. 32 heads of 64: 8 committed 100,
// verified 83, one committed 66; a head's phases are no shorter there, for a quarter of the state.
#include <cuda.h>  // CUtensorMap (the encoder is fetched at run time; no libcuda link)

#include "kda_rows.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kSms = 152;
constexpr int kBlock = 8;  // tokens a block: an MMA's n

// 3-D tiled TMA store of one box of `map`, of this thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const void *map, int x, int y, int z, const void *smem) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(smem))
                 : "memory");
}

// The nearest value of 11 bits. (NaN may come out as a zero: what is left of it, x - hi, is NaN still. From
// 2^128 (1 - 2^-12) on it is infinite, and what is left is no number: the call's documented range ends there.
// Limited to the largest finite value, one instruction more for each of a state's values, 256 rows of 8 tokens, 32
// heads of 128, took 229 us for 216 committed and 184 for 163 verified; of 64 channels 111 for 100.)
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

constexpr int kCols = 32;  // state columns of a pair of warps: two of an MMA's m

constexpr int kTeam = 96;     // threads that prepare a block; the teams take the blocks in turn
constexpr int kWindow = 128;  // pairs that a CTA looks at together

// A block of a head's tokens, as a team passes it on.
struct TokenTask {
    long long row, place;  // the block's first token among the rows; the state's place in units of D x D (-1: the end)
    long long before, older;  // the places of the head before this one, and of the one before that (-1: none)
    int count, t0;         // the head's tokens, the block's first
    int head;              // the CTA's heads before this one
};

template <int D, typename InT>
struct TokenSmem {
    // Two teams, but where fp32 inputs of 128 channels leave shared memory for one. (256 rows of 8 tokens, 32 heads
    // of 64, committed: 121 us with one, 100 with two.)
    static constexpr int kTeams = D == 64 || sizeof(InT) == 2 ? 2 : 1;
    // Strides without bank conflicts.
    static constexpr int kRead = 2 * D + 16, kWrite = 2 * D + 8, kTrans = kCols + 4;
    static constexpr int kRing = kTeams + 2;  // blocks between a value's fetch and its last use
    // Boxes of 32 columns by D rows, a row's 16-byte pieces swapped by the row's low three bits (piece ^ row % 8).
    alignas(1024) float state[2][D / kCols][D][kCols];
    struct alignas(16) Block {
        float read[2][kBlock][kRead];  // G k and G s q: for rows r, r + 1 (r even) hi, hi', lo, lo'
        float write[kBlock][kWrite];   // G_{j:C} k: hi, lo of each row
        float total[D];                // G_C
        float A[kBlock][kBlock], Hm[kBlock][kBlock];
        float rk[kBlock], rq[kBlock];
        TokenTask task;
    } block[2];
    alignas(16) float trans[D / 16][2 * kBlock][kTrans];  // a warp's values, columns across
    struct alignas(16) Inputs {
        float a[kBlock][D];  // g, then a
        InT q[kBlock][D], k[kBlock][D];
    } in[kTeams];
    alignas(16) InT v[kRing][kBlock][D];
    float beta[kRing][kBlock];
    long long row[kWindow], place[kWindow];  // the CTA's next pairs
    int count[kWindow];
    TokenTask ring[4];    // a step's task, for the warp that moves the states
    uint64_t arrived[2];  // mbarriers: a state is in its buffer
};

enum { kBarFull = 1, kBarEmpty = 9, kBarTeam = 11, kBarWindow = 13, kBarBegin = 14 };  // named barriers

// The working threads, the teams, a warp that moves the states, and what makes it whole fours of warps.
template <int D, typename InT>
constexpr int token_threads = (2 * D + TokenSmem<D, InT>::kTeams * kTeam + 32 + 127) / 128 * 128;

// Step i is in block i % 2. Its full barriers, one for each pair of warps (which need not keep step with one
// another), are passed by the team when the block is ready and by the pair before it reads it; until the empty
// barrier they also serve the two warps to wait for one another. Its empty barrier is passed by all working
// threads when they have read it (and have written the state behind a head's last block back into its buffer),
// by the team of step i + 2 before it fills it again, and by the warp that moves the states. The last step is the
// end, which the working threads answer too; its team passes the empty barriers that are left. Head h has state
// buffer h % 2: the empty barrier two steps before its first one says that the head that had the buffer before
// is done with.
//
// The teams look for heads in windows of kWindow pairs, which both fill: at a window's end a team waits in the
// window barrier until the other one is there too. With two teams, one that has passed step t on looks as far as
// step t + 4, so where it waits the other one comes by when it has passed step t + 1 on at the latest. For that
// block (t + 1) % 2 has to be empty: step t - 1, which the other one passed on itself, has to be worked off, and the
// mover, which the waiting team met in step t - 2's empty barrier, has to be there. None of it waits for the team
// that waits. The begin barrier, in which the mover waits for the ring's first two tasks, is passed by both teams
// when they have looked at steps 0 and 1. (Behind the look at steps 2 and 3, the first of which only team 0 takes
// and the second only team 1, three blocks before a window's end made team 1 wait in one barrier and team 0 in the
// other, for ever.)
template <int D, typename InT>
__global__ void __launch_bounds__(token_threads<D, InT>, D == 128 ? 1 : 2)
decode_tokens_kernel(const InT *__restrict__ q, const InT *__restrict__ k, const InT *__restrict__ v,
                     const float *__restrict__ g, const float *__restrict__ beta, float scale,
                     const __grid_constant__ CUtensorMap states,
                     const int32_t *__restrict__ slots, int num_slots, const int32_t *__restrict__ counts, int K, int H,
                     int items, InT *__restrict__ out, int write_state, Prologue pro) {
    constexpr int KT = D / 16;     // row tiles of a warp
    constexpr int kWork = 2 * D;   // threads that work: D / kCols pairs of warps
    constexpr int kTeams = TokenSmem<D, InT>::kTeams, kPrep = kTeams * kTeam;
    constexpr int kPairs = D / kCols, kFull = 64 + kTeam, kEmpty = kWork + kTeam + 32;
    extern __shared__ __align__(1024) unsigned char raw[];
    auto &sm = *reinterpret_cast<TokenSmem<D, InT> *>(raw + (-tc::smem_u32(raw) & 1023u));
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tc::mbar_init(&sm.arrived[0], 1);
        tc::mbar_init(&sm.arrived[1], 1);
        tc::mbar_fence_init();
    }
    __syncthreads();

    if (threadIdx.x >= kWork + kPrep + 32) return;
    if (threadIdx.x >= kWork + kPrep) {
        // The warp that moves the states: a head's one goes and the next but one comes as soon as it is done with.
        const auto store = [&](int head, long long place) {
            if (place < 0 || !write_state) return;
            if (lane < D / kCols) tma_store_3d(&states, lane * kCols, 0, (int)place, sm.state[head & 1][lane]);
            asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        };
        tc::bar_sync(kBarBegin, kPrep + 32);
        for (int step = 0;; ++step) {
            if (step >= 2) tc::bar_sync(kBarEmpty + (step & 1), kEmpty);
            const TokenTask &task = sm.ring[step & 3];
            if (task.place < 0) {
                if (step >= 1) tc::bar_sync(kBarEmpty + ((step - 1) & 1), kEmpty);
                tc::bar_sync(kBarEmpty + (step & 1), kEmpty);
                store(task.head - 2, task.older);
                store(task.head - 1, task.before);
                asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                return;
            }
            if (task.t0 == 0) {
                store(task.head - 2, task.older);
                if (lane == 0) tc::mbar_expect_tx(&sm.arrived[task.head & 1], D * D * 4);
                __syncwarp();
                if (lane < D / kCols)
                    tc::tma_load_3d(sm.state[task.head & 1][lane], &states, lane * kCols, 0, (int)task.place,
                                    &sm.arrived[task.head & 1]);
            }
        }
    }
    if (threadIdx.x >= kWork) {
        const int team = (threadIdx.x - kWork) / kTeam, tid = (threadIdx.x - kWork) % kTeam, warp = tid >> 5;
        const auto pass_full = [](int step) {
            __threadfence_block();
#pragma unroll
            for (int p = 0; p < kPairs; ++p) tc::bar_arrive(kBarFull + 2 * p + (step & 1), kFull);
        };
        auto team_wait = [&] { tc::bar_sync(kBarTeam + team, kTeam); };
        unsigned cursor = 0;  // the CTA's pairs that have been looked at
        // The next pair with tokens; what task holds is the head before. Both teams see the same pairs, by the
        // window that both have waited for.
        auto next_head = [&](TokenTask &task) {
            task.older = task.before;
            task.before = task.place;
            task.place = -1;
            ++task.head;
            for (;; ++cursor) {
                const long long item = blockIdx.x + (long long)cursor * gridDim.x;
                if (item >= items) return;
                const int at = cursor % kWindow;
                if (at == 0) {
                    tc::bar_sync(kBarWindow, kPrep);
                    for (int mine = threadIdx.x - kWork; mine < kWindow; mine += kPrep) {
                        const long long look = item + (long long)mine * gridDim.x;
                        int count = 0;
                        if (look < items) {
                            const int n = (int)look / H, head = (int)look % H, slot = slots ? slots[n] : n;
                            count = counts ? min(max(counts[n], 0), K) : K;
                            if (slot < 0 || slot >= num_slots) count = 0;
                            sm.row[mine] = (long long)n * K * H + head;
                            sm.place[mine] = (long long)slot * H + head;
                        }
                        sm.count[mine] = look < items ? count : K;
                    }
                    tc::bar_sync(kBarWindow, kPrep);
                    // The outputs behind the counts.
                    if (out) {
                        for (int w = (threadIdx.x - kWork) >> 5; w < kWindow; w += kPrep / 32)
                            for (int p = sm.count[w] * D + lane; p < K * D; p += 32)
                                out[(sm.row[w] + (long long)(p / D) * H) * D + p % D] = from_f32<InT>(0.f);
                    }
                }
                if (sm.count[at] > 0) {
                    task.row = sm.row[at];
                    task.place = sm.place[at];
                    task.count = sm.count[at];
                    task.t0 = 0;
                    ++cursor;
                    return;
                }
            }
        };
        auto advance = [&](const TokenTask &task) {
            TokenTask to = task;
            if (task.place < 0) return to;
            to.t0 += kBlock;
            to.row += (long long)kBlock * H;
            if (to.t0 >= to.count) next_head(to);
            return to;
        };
        // The inputs of a step's block on their way into shared memory.
        auto fetch = [&](const TokenTask &task, int step) {
            if (task.place >= 0) {
                constexpr int E = 16 / (int)sizeof(InT), kIn = D / E, kG = D / 4;  // 16-byte pieces of a row
                const int some = min(kBlock, task.count - task.t0);
                auto &in = sm.in[team];
                for (int p = tid; p < some * kIn; p += kTeam) {
                    const int i = p / kIn, c = p % kIn * E;
                    const long long at = (task.row + (long long)i * H) * D + c;
                    tc::cp_async16(&in.q[i][c], q + at, 16);
                    tc::cp_async16(&in.k[i][c], k + at, 16);
                    tc::cp_async16(&sm.v[step % TokenSmem<D, InT>::kRing][i][c], v + at, 16);
                }
                if (pro.decay == KDA_DECAY_CHANNEL)
                    for (int p = tid; p < some * kG; p += kTeam) {
                        const int i = p / kG, c = p % kG * 4;
                        tc::cp_async16(&in.a[i][c], g + (task.row + (long long)i * H) * D + c, 16);
                    }
                if (tid < some) {
                    const uint32_t to = (uint32_t)__cvta_generic_to_shared(&sm.beta[step % TokenSmem<D, InT>::kRing][tid]);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(beta + task.row + (long long)tid * H)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        TokenTask task = {0, -1, -1, -1, 0, 0, -1}, next, second;  // of this step and the two behind it
        next_head(task);
        bool first_end = true;  // the step before this one was a block
        if (tid == 0 && team == 0) sm.ring[0] = task;
        next = advance(task);
        if (tid == 0 && team == 0) sm.ring[1] = next;
        tc::bar_sync(kBarBegin, kPrep + 32);  // before either team looks further than the other (above)
        if (team == 1) {
            first_end = task.place >= 0;
            task = next;
            next = advance(task);
        }
        second = advance(next);
        fetch(task, team);
        for (int step = team;; step += kTeams) {
            auto &bl = sm.block[step & 1];
            auto &in = sm.in[team];
            const auto empty_wait = [step] {
                if (step >= 2) tc::bar_sync(kBarEmpty + (step & 1), kEmpty);
            };
            if (task.place < 0) {
                empty_wait();
                if (first_end) {
                    if (tid == 0) bl.task = task;
                    pass_full(step);
                    if (kTeams == 1 && step >= 1) tc::bar_sync(kBarEmpty + ((step - 1) & 1), kEmpty);
                    tc::bar_sync(kBarEmpty + (step & 1), kEmpty);
                }
                tc::cp_async_wait_all();
                return;
            }
            tc::cp_async_wait_all();
            team_wait();  // this block's inputs are here
            const int some = min(kBlock, task.count - task.t0);
            if (pro.decay == KDA_DECAY_CHANNEL) {
                for (int p = tid; p < some * (D / 4); p += kTeam) {
                    float4 *at = reinterpret_cast<float4 *>(&in.a[p / (D / 4)][p % (D / 4) * 4]);
                    const float4 z = *at;
                    *at = make_float4(decay_factor(z.x, pro), decay_factor(z.y, pro), decay_factor(z.z, pro), decay_factor(z.w, pro));
                }
            } else {
                for (int p = tid; p < some * D; p += kTeam)
                    in.a[p / D][p % D] =
                        pro.decay == KDA_DECAY_NONE ? 1.f : decay_factor(g[task.row + (long long)(p / D) * H], pro);
            }
            // Up to here the block that is filled may still be read: of 10000 cycles with 8 tokens half are over by then.
            empty_wait();
            team_wait();
            if (tid == 0) {
                bl.task = task;
                sm.ring[(step + 2) & 3] = second;
            }
            // For a block of at most kN tokens, without branches between them; places behind the last token hold what
            // they hold, and their results are not used.
            const auto prepare = [&](auto n) {
                constexpr int kN = decltype(n)::value;
                // The vectors of the reads by k and by q and of the update, two channels a lane.
                constexpr int kUnits = D / 64;  // warps' worth of channels
                for (int unit = kTeam / 32 - 1 - warp; unit < 3 * kUnits; unit += kTeam / 32) {
                    const int role = unit / kUnits, c = (unit % kUnits * 32 + lane) * 2;
                    const InT(*from)[D] = role == 1 ? in.q : in.k;
                    float a[kN][2], z[kN][2], G[2] = {1.f, 1.f};
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        some_of<2>(&in.a[i][c], a[i]);
                        some_of<2>(&from[i][c], z[i]);
                    }
                    if (role < 2) {
                        const float f = role ? scale : 1.f;
#pragma unroll
                        for (int i = 0; i < kN; ++i) {
                            G[0] *= a[i][0];
                            G[1] *= a[i][1];
                            const float w0 = G[0] * (f * z[i][0]), w1 = G[1] * (f * z[i][1]), h0 = tf32_hi(w0), h1 = tf32_hi(w1);
                            *reinterpret_cast<float4 *>(&bl.read[role][i][2 * c]) = make_float4(h0, h1, w0 - h0, w1 - h1);
                        }
                    } else {  // the update's product sums over all of its places: zeros behind the last token
#pragma unroll
                        for (int i = kBlock - 1; i >= 0; --i) {
                            float w0 = 0.f, w1 = 0.f;
                            if (i < kN && i < some) {
                                w0 = G[0] * z[i][0];
                                w1 = G[1] * z[i][1];
                                G[0] *= a[i][0];
                                G[1] *= a[i][1];
                            }
                            const float h0 = tf32_hi(w0), h1 = tf32_hi(w1);
                            *reinterpret_cast<float4 *>(&bl.write[i][2 * c]) = make_float4(h0, w0 - h0, h1, w1 - h1);
                        }
                        *reinterpret_cast<float2 *>(&bl.total[c]) = make_float2(G[0], G[1]);
                    }
                }
                // A_tj, H_tj for t >= j (A_jj is |k_j|^2), and |q_j|^2: a warp takes every third token j, all of them at
                // once where its registers hold their sums (64 channels, two CTAs an SM: one after another).
                constexpr int kC = D / 32, kMost = (kN + kTeam / 32 - 1) / (kTeam / 32), kJ = D == 128 ? kMost : 1;
                const int c = kC * lane;
#pragma unroll 1
                for (int j0 = warp; j0 < kN; j0 += kJ * (kTeam / 32)) {
                    float acc[kJ][2 * kN], w[kJ][kC], qss[kJ];
#pragma unroll
                    for (int i = 0; i < kJ; ++i) {
                        qss[i] = 0.f;
                        some_of<kC>(&in.k[min(j0 + i * (kTeam / 32), kN - 1)][c], w[i]);
                    }
#pragma unroll
                    for (int t = 0; t < kN; ++t) {
                        float a[kC], kt[kC], qt[kC];
                        some_of<kC>(&in.a[t][c], a);
                        some_of<kC>(&in.k[t][c], kt);
                        some_of<kC>(&in.q[t][c], qt);
#pragma unroll
                        for (int i = 0; i < kJ; ++i) {
                            const int j = j0 + i * (kTeam / 32);
                            acc[i][t] = acc[i][kN + t] = 0.f;
#pragma unroll
                            for (int m = 0; m < kC; ++m) {
                                if (t > j) w[i][m] *= a[m];
                                if (t == j) qss[i] += qt[m] * qt[m];
                                acc[i][t] += kt[m] * w[i][m];
                                acc[i][kN + t] += qt[m] * w[i][m];
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kJ; ++i) {
                        // 2 kN sums over the warp: every step halves the values a lane holds.
#pragma unroll
                        for (int m = 16, left = kN; m > 0; m >>= 1, left >>= 1) {
                            const bool up = lane & m;
                            if (left == 0) acc[i][0] += __shfl_xor_sync(0xffffffffu, acc[i][0], m);
#pragma unroll
                            for (int x = 0; x < left; ++x) {
                                const float keep = up ? acc[i][x + left] : acc[i][x], send = up ? acc[i][x] : acc[i][x + left];
                                acc[i][x] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                            }
                        }
                        // The sum for token t (of H in the upper half of the warp) is in 16 / kN lanes.
                        const int j = j0 + i * (kTeam / 32), t = lane % 16 / (16 / kN);
                        if (j < kN && lane % (16 / kN) == 0)
                            (lane < 16 ? bl.A : bl.Hm)[t][j] = lane < 16 ? acc[i][0] : scale * acc[i][0];
                        float rk = 1.f, rq = 1.f;
                        if (pro.l2norm) {
                            rk = rsqrtf(__shfl_sync(0xffffffffu, acc[i][0], min(j, kN - 1) * (16 / kN)) + kL2Eps);
                            rq = rsqrtf(lanes_sum<32>(qss[i]) + kL2Eps);
                        }
                        if (j < kN && lane == 0) {
                            bl.rk[j] = rk;
                            bl.rq[j] = rq;
                        }
                    }
                }
            };
            if (some <= kBlock / 2)
                prepare(std::integral_constant<int, kBlock / 2>{});
            else
                prepare(std::integral_constant<int, kBlock>{});
            pass_full(step);
            team_wait();  // the inputs are read no more
            first_end = kTeams == 1 || next.place >= 0;
            if (kTeams == 2) {
                task = second;
                next = advance(task);
            } else {
                task = next;
                next = second;
            }
            second = advance(next);
            fetch(task, step + kTeams);
        }
    }
    // The pair's columns from `first`, the warp's rows from `top`: rows 8 i + 2 x and the next, columns 4 y to 4 y + 3.
    const int warp = threadIdx.x >> 5, half = warp & 1, x = lane & 3, y = lane >> 2;
    const int first = (warp >> 1) * kCols, top = half * (D / 2), col = first + lane;
    float s[KT][2][4];
    for (int step = 0;; ++step) {
        const int bar = kBarFull + (warp & ~1) + (step & 1);
        tc::bar_sync(bar, kFull);
        const auto pair_wait = [bar] { tc::bar_sync(bar, 64); };
        const auto &bl = sm.block[step & 1];
        const int count = bl.task.count, t0 = bl.task.t0, head = bl.task.head;
        if (bl.task.place < 0) {
            tc::bar_arrive(kBarEmpty + (step & 1), kEmpty);
            return;
        }
        const int some = min(kBlock, count - t0);
        const bool last = t0 + kBlock >= count;
        // Rows 2 x and 2 x + 1 of every eight, the lane's piece where the copy put it.
        float *S[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) S[r] = &sm.state[head & 1][warp >> 1][top + 2 * x + r][(y ^ (2 * x + r)) * 4];
        if (t0 == 0) {
            // A copy that does not come (after a second or more) leaves NaN.
            const bool here = tc::mbar_wait(&sm.arrived[head & 1], head >> 1 & 1);
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) some_of<4>(S[r] + 8 * i * kCols, s[i][r]);
            if (!here) {
#pragma unroll
                for (int i = 0; i < KT * 8; ++i) s[i / 8][i / 4 % 2][i % 4] = __uint_as_float(0x7fffffffu);
            }
        }

        float(*tr)[TokenSmem<D, InT>::kTrans] = sm.trans[warp], (*other)[TokenSmem<D, InT>::kTrans] = sm.trans[warp ^ 1];
        float ke[kBlock];
        // Of a block of at most kN tokens. (Without branches between them, so that what a token waits for is under way
        // before: places behind the last token are computed and not used.)
        const auto tokens = [&](auto n) {
            constexpr int kN = decltype(n)::value;
            constexpr bool kBoth = kN <= kBlock / 2;
            // The warp's part of P and R, 32 columns by kN tokens each: in one product where the eight vectors of its n
            // are k's and q's, else in two. The small products have sums of their own: an MMA's sum is cut off, not
            // rounded, so the fewer at full size the better.
            float acc[kBoth ? 1 : 2][2][4], small[kBoth ? 1 : 2][2][4];
#pragma unroll
            for (int i = 0; i < (kBoth ? 8 : 16); ++i) acc[i >> 3][i >> 2 & 1][i & 3] = small[i >> 3][i >> 2 & 1][i & 3] = 0.f;
            const float *from = (kBoth ? bl.read[y >> 2][y & 3] : bl.read[0][y]) + 2 * top + 4 * x;
            const float *from_q = bl.read[1][y] + 2 * top + 4 * x;
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                float hi[2][4], lo[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float w = s[i][c >> 1][2 * m + (c & 1)];
                        hi[m][c] = tf32_hi(w);
                        lo[m][c] = w - hi[m][c];
                    }
                const float4 b0 = *reinterpret_cast<const float4 *>(from + 16 * i);
                float4 b1 = b0;
                if (!kBoth) b1 = *reinterpret_cast<const float4 *>(from_q + 16 * i);
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int b = 0; b < (kBoth ? 1 : 2); ++b)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const float4 v4 = b ? b1 : b0;
                            mma_tf32(part ? small[b][m] : acc[b][m], part == 1 ? lo[m] : hi[m], part == 2 ? v4.z : v4.x,
                                     part == 2 ? v4.w : v4.y);
                        }
            }
            // A lane takes one column over all tokens, the sum of both warps' parts: both solve for e, each forms the
            // outputs of every other token.
#pragma unroll
            for (int b = 0; b < (kBoth ? 1 : 2); ++b) {
                const int to = kBoth ? 2 * x + (x & 2) * (kBlock / 4) : b * kBlock + 2 * x;  // R's rows begin at kBlock
                auto &d = acc[b];
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i >> 2][i & 3] += small[b][i >> 2][i & 3];
                *reinterpret_cast<float4 *>(&tr[to][4 * y]) = make_float4(d[0][0], d[0][2], d[1][0], d[1][2]);
                *reinterpret_cast<float4 *>(&tr[to + 1][4 * y]) = make_float4(d[0][1], d[0][3], d[1][1], d[1][3]);
            }
            float vt[kN], rk[kN], bt[kN], o[kN / 2];
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                vt[t] = to_f32(sm.v[step % TokenSmem<D, InT>::kRing][t][col]);
                rk[t] = bl.rk[t];
                bt[t] = sm.beta[step % TokenSmem<D, InT>::kRing][t];
            }
            pair_wait();
            float u[kN];
#pragma unroll
            for (int t = 0; t < kN; ++t) u[t] = tr[t][lane] + other[t][lane];
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) o[i] = tr[kBlock + 2 * i + half][lane] + other[kBlock + 2 * i + half][lane];
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                float A[kBlock];
                some_of<4>(bl.A[t], A);
                if (t > 4) some_of<4>(bl.A[t] + 4, A + 4);
#pragma unroll
                for (int j = 0; j < t; ++j) u[t] += A[j] * ke[j];
                // The reads are linear in k and q, which are normalised here.
                ke[t] = t < some ? rk[t] * (bt[t] * (vt[t] - rk[t] * u[t])) : 0.f;
            }
#pragma unroll
            for (int t = kN; t < kBlock; ++t) ke[t] = 0.f;
            if (out) {
                InT *to = out + bl.task.row * D + col;
#pragma unroll
                for (int i = 0; i < kN / 2; ++i) {
                    const int t = 2 * i + half;
                    float Hm[kBlock];
                    some_of<4>(bl.Hm[t], Hm);
                    if (i >= 2) some_of<4>(bl.Hm[t] + 4, Hm + 4);
#pragma unroll
                    for (int j = 0; j < 2 * i + 1; ++j) o[i] += Hm[j] * ke[j];
                    if (half) o[i] += Hm[2 * i + 1] * ke[2 * i + 1];
                    if (t < some) to[(size_t)t * H * D] = from_f32<InT>(bl.rq[t] * o[i]);
                }
            }
        };
        if (some <= kBlock / 2)
            tokens(std::integral_constant<int, kBlock / 2>{});
        else
            tokens(std::integral_constant<int, kBlock>{});
        if (!last || write_state) {
            pair_wait();  // the other warp has read
#pragma unroll
            for (int t = 0; t < kBlock; ++t) tr[t][lane] = ke[t];
            __syncwarp();
            // S <- G_C S + k e^T: the products' sums by themselves, and one rounded fp32 step to the state (added to it
            // by the MMAs, whose sums are cut off, a slowly decaying state would lose 1e-7 of itself every block).
            float hi[2][4], lo[2][4];
            {
                float e[2][4];
                some_of<4>(&tr[x][4 * y], e[0]);
                some_of<4>(&tr[x + 4][4 * y], e[1]);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float w = e[c >> 1][2 * m + (c & 1)];
                        hi[m][c] = tf32_hi(w);
                        lo[m][c] = w - hi[m][c];
                    }
            }
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                const int at = top + 8 * i;
                const float2 tot = *reinterpret_cast<const float2 *>(&bl.total[at + 2 * x]);
                const float2 w0 = *reinterpret_cast<const float2 *>(&bl.write[x][2 * (at + y)]);
                const float2 w1 = *reinterpret_cast<const float2 *>(&bl.write[x + 4][2 * (at + y)]);
                float c[2][4] = {};
#pragma unroll
                for (int m = 0; m < 2; ++m) mma_tf32(c[m], lo[m], w0.x, w1.x);
#pragma unroll
                for (int m = 0; m < 2; ++m) mma_tf32(c[m], hi[m], w0.y, w1.y);
#pragma unroll
                for (int m = 0; m < 2; ++m) mma_tf32(c[m], hi[m], w0.x, w1.x);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float &w = s[i][j & 1][2 * m + (j >> 1)];
                        w = fmaf(j & 1 ? tot.y : tot.x, w, c[m][j]);
                    }
            }
            if (last) {
#pragma unroll
                for (int i = 0; i < KT; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        *reinterpret_cast<float4 *>(S[r] + 8 * i * kCols) =
                            make_float4(s[i][r][0], s[i][r][1], s[i][r][2], s[i][r][3]);
                tc::fence_async_smem();
            }
        }
        tc::bar_arrive(kBarEmpty + (step & 1), kEmpty);
    }
}

// cuTensorMapEncodeTiled, fetched from the driver at run time.
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encoder() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t err =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        return err == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
    }();
    return fn;
}

// The states [places][D][D] seen as 3-D (column, row, place) with boxes of 32 columns x D rows x 1 place.
cudaError_t states_map(CUtensorMap *m, float *state, int D, long long places) {
    const EncodeTiledFn enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)D, (cuuint64_t)places};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 4, (cuuint64_t)D * D * 4};
    const cuuint32_t box[3] = {(cuuint32_t)kCols, (cuuint32_t)D, 1u};
    const cuuint32_t unit[3] = {1u, 1u, 1u};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, state, dims, strides, box, unit,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, typename InT>
cudaError_t launch_tokens_t(const TokensArgs &a, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(TokenSmem<D, InT>) + 1024;  // and what aligns it
    static_assert(smem <= 227 << 10 && (D == 128 || 2 * (smem + 1024) <= 228 << 10), "");
    CUtensorMap states;
    cudaError_t err = states_map(&states, a.state, D, (long long)a.num_slots * a.H);
    if (err != cudaSuccess) return err;
    err = cudaFuncSetAttribute(decode_tokens_kernel<D, InT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    const long long items = (long long)a.N * a.H, most = kSms * (D == 128 ? 1 : 2);
    decode_tokens_kernel<D, InT>
        <<<(unsigned)(items < most ? items : most), token_threads<D, InT>, smem, stream>>>(
            static_cast<const InT *>(a.q), static_cast<const InT *>(a.k), static_cast<const InT *>(a.v), a.g, a.beta, a.scale,
            states, a.slots, a.num_slots, a.counts, a.K, a.H, (int)items, static_cast<InT *>(a.out), a.write_state, a.pro);
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
