// Maintenance of a pool of recurrent states, [layers][slots][slot_bytes]:
// copies between slots as one parallel assignment, and compaction.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kPoolThreads = 256;

__device__ __forceinline__ void async16(void *smem, const void *gmem) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(gmem) : "memory");
}

// ---- pool[dst[i]] = source[src[i]]
//
// In one pool a slot may be both read and written, so every source must be
// read before any slot is written. Bytes at different offsets of a slot never
// meet: a CTA takes one column of bytes (of one layer) of ALL the entries,
// gathers it into shared memory, and writes it out after a barrier. That
// makes any mapping (forks, swaps, cycles) exact with one read and one write
// per byte, no scratch memory and one launch. The columns are double-buffered.
//
// Each CTA first reduces the entries to the ones that hold: in range, the last
// of those that name one destination (a hash table in shared memory), and not
// a slot onto itself. Bound by HBM on large slots (256 beams of 1 MiB, 75 % of
// which move: 62-64 us, 5.6-5.8 TB/s; columns of 256 bytes there, and 512 change
// little: 63) and by some 5 us of lists and first loads on small ones.
constexpr size_t copy_list_bytes(int n) { return ((size_t)n * 8 + 127) / 128 * 128; }
constexpr int kFewEntries = 1024;  // launch_state_copy
constexpr int copy_hash_size(int n) {
    int h = 64;
    while (h < 2 * n) h *= 2;
    return h;
}

// `kItems` 16-byte pieces a thread in each column buffer. Sizes in pieces.
template <int kItems>
__global__ void __launch_bounds__(kPoolThreads)
state_copy_kernel(const uint4 *source, int source_slots, uint4 *pool, int num_slots,
                  const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n, int hash_size,
                  int layers, uint32_t slot, int list_bytes) {
    constexpr int kBuffer = kItems * kPoolThreads;
    extern __shared__ __align__(128) unsigned char smem[];
    int2 *list = reinterpret_cast<int2 *>(smem);  // (source or -1, destination): copies from the front,
                                                  // zeroed slots from the back
    unsigned char *buf = smem + list_bytes;
    __shared__ int found[2];
    const int tid = threadIdx.x;
    {
        int *key = reinterpret_cast<int *>(buf), *last = key + hash_size;
        const unsigned mask = (unsigned)hash_size - 1;
        if (tid < 2) found[tid] = 0;
        for (int h = tid; h < hash_size; h += kPoolThreads) key[h] = last[h] = -1;
        __syncthreads();
        for (int i = tid; i < n; i += kPoolThreads) {
            const int d = dst[i];
            if (d < 0 || d >= num_slots || src[i] >= source_slots) continue;
            unsigned h = (unsigned)d * 2654435761u & mask;
            for (;;) {  // ends: the table has at least twice as many places as entries
                const int k = atomicCAS(&key[h], -1, d);
                if (k == -1 || k == d) break;
                h = (h + 1) & mask;
            }
            atomicMax(&last[h], i);
        }
        __syncthreads();
        for (int i = tid; i < n; i += kPoolThreads) {
            const int d = dst[i], s = src[i];
            if (d < 0 || d >= num_slots || s >= source_slots) continue;
            unsigned h = (unsigned)d * 2654435761u & mask;
            while (key[h] != d) h = (h + 1) & mask;
            if (last[h] != i) continue;
            if (s < 0)
                list[n - 1 - atomicAdd(&found[1], 1)] = make_int2(-1, d);
            else if (s != d || source != pool)
                list[atomicAdd(&found[0], 1)] = make_int2(s, d);
        }
        __syncthreads();
    }
    const int copies = found[0], zeros = found[1];
    if (copies + zeros == 0) return;
    // Width of a column: as wide as a buffer allows, but narrow enough that
    // there are two columns for every CTA.
    int shift = 10;  // pieces per column and entry, as a power of two
    while (shift > 0 && ((long long)copies << shift) > kBuffer) --shift;
    while (shift > 3 && layers * (((long long)slot + (1 << shift) - 1) >> shift) < 2LL * gridDim.x) --shift;
    const uint32_t columns = (slot + (1u << shift) - 1) >> shift;
    const long long units = (long long)columns * layers;
    const uint32_t mask = (1u << shift) - 1;

    // Which pieces a thread takes is the same in every column; what is left of
    // an item there is two 32-bit products, a copy in and a copy out.
    uint4 *buf4 = reinterpret_cast<uint4 *>(buf) + tid;
    int2 entry[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int p = tid + k * kPoolThreads;
        entry[k] = p < copies << shift ? list[p >> shift] : make_int2(-1, -1);
    }
    const uint32_t in = (uint32_t)tid & mask;  // kPoolThreads is a multiple of a column's pieces, or
                                               // a column's pieces of kPoolThreads
    auto inside = [&](int k) { return shift > 8 ? ((uint32_t)(tid + k * kPoolThreads) & mask) : in; };
    auto gather = [&](long long unit, int b) {
        const uint32_t off = (uint32_t)(unit % columns) << shift;
        const uint4 *from = source + (size_t)(unit / columns) * source_slots * slot + off;
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            if (entry[k].x >= 0 && off + inside(k) < slot)
                async16(buf4 + (size_t)(b * kItems + k) * kPoolThreads, from + (size_t)(uint32_t)entry[k].x * slot + inside(k));
    };
    long long unit = blockIdx.x;
    if (unit < units) gather(unit, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int b = 0; unit < units; unit += gridDim.x, b ^= 1) {
        if (unit + gridDim.x < units) gather(unit + gridDim.x, b ^ 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // every source of this column has been read
        const uint32_t off = (uint32_t)(unit % columns) << shift;
        uint4 *to = pool + (size_t)(unit / columns) * num_slots * slot + off;
#pragma unroll
        for (int k = 0; k < kItems; ++k)  // the pieces this thread gathered
            if (entry[k].x >= 0 && off + inside(k) < slot)
                to[(size_t)(uint32_t)entry[k].y * slot + inside(k)] = buf4[(size_t)(b * kItems + k) * kPoolThreads];
        for (int p = tid; p < zeros << shift; p += kPoolThreads)
            if (off + ((uint32_t)p & mask) < slot)
                to[(size_t)(uint32_t)list[n - 1 - (p >> shift)].y * slot + ((uint32_t)p & mask)] = make_uint4(0, 0, 0, 0);
    }
}

// ---- compaction

// Larger pools. One CTA: counts the live slots, then lists in order the live slots at or
// above the count and the holes below it (as many of one as of the other).
// Workspace: moves, then mover[num_slots], hole[num_slots].
constexpr int kPlanThreads = 1024;
constexpr size_t kPlanHeader = 256;

__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(const uint8_t *__restrict__ live, int num_slots, int32_t *__restrict__ new_slot,
                    int32_t *__restrict__ count, int *__restrict__ moves, int *__restrict__ mover,
                    int *__restrict__ hole) {
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int total;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int mine = 0;
    for (int s = tid; s < num_slots; s += kPlanThreads) mine += live[s] != 0;
    if (tid == 0) total = 0;
    __syncthreads();
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) atomicAdd(&total, mine);
    __syncthreads();
    const int n = total;
    int base = 0;  // live slots before this round's
    for (int s0 = 0; s0 < num_slots; s0 += kPlanThreads) {
        const int s = s0 + tid;
        const bool alive = s < num_slots && live[s] != 0;
        const unsigned votes = __ballot_sync(0xffffffffu, alive);
        if (lane == 0) warp_sum[warp] = __popc(votes);
        __syncthreads();
        int before = base, round = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) before += warp_sum[w];
            round += warp_sum[w];
        }
        before += __popc(votes & ((1u << lane) - 1));  // live slots below s
        if (s < num_slots) {
            new_slot[s] = alive ? s : -1;
            if (!alive && s < n) hole[s - before] = s;  // dead slots below s
            if (alive && s >= n) mover[before] = s;  // the first at n - holes, see below
        }
        base += round;
        __syncthreads();
    }
    // mover is indexed by the live slots before it: its first index is the
    // number of live slots below n, n minus the number of holes.
    __shared__ int holes;
    if (tid == 0) holes = 0;
    __syncthreads();
    int dead = 0;
    for (int s = tid; s < n; s += kPlanThreads) dead += live[s] == 0;
    dead = __reduce_add_sync(0xffffffffu, dead);
    if (lane == 0) atomicAdd(&holes, dead);
    __syncthreads();
    const int m = holes;
    for (int k = tid; k < m; k += kPlanThreads) new_slot[mover[n - m + k]] = hole[k];
    if (tid == 0) {
        *count = n;
        *moves = m;
    }
}

// Copies slot mover[k] to hole[k] for k < m: sources and destinations are
// disjoint, so any order does. A unit is 16 KiB of one slot; four CTAs per SM
// take units in turn, with loads and stores marked as used once (96 moves of
// 2 x 1 MiB with the lists made: 72.1 us without the marks, 69.4 with, 68.7 with
// four CTAs for six, 5.9 TB/s; torch's copy of as many bytes in a row 63).
constexpr int kMoveUnroll = 4, kMoveCtas = 4;
constexpr long long kMoveBytes = 16LL * kPoolThreads * kMoveUnroll;

template <typename I>
__device__ __forceinline__ void move_slots(char *pool, int num_slots, int m, const I *mover, const I *hole, int layers,
                                           long long slot_bytes) {
    const long long pieces = (slot_bytes + kMoveBytes - 1) / kMoveBytes;
    const long long units = pieces * m * layers;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const long long piece = u % pieces, k = u / pieces % m, layer = u / pieces / m;
        char *base = pool + layer * num_slots * slot_bytes;
        const char *from = base + (long long)mover[k] * slot_bytes;
        char *to = base + (long long)hole[k] * slot_bytes;
        const long long at = piece * kMoveBytes + threadIdx.x * 16;
        uint4 v[kMoveUnroll];
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            const long long o = at + (long long)j * 16 * kPoolThreads;
            if (o < slot_bytes) v[j] = __ldcs(reinterpret_cast<const uint4 *>(from + o));
        }
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            const long long o = at + (long long)j * 16 * kPoolThreads;
            if (o < slot_bytes) __stcs(reinterpret_cast<uint4 *>(to + o), v[j]);
        }
    }
}

// The moves that compact_plan_kernel listed.
__global__ void __launch_bounds__(kPoolThreads)
compact_move_kernel(char *pool, int num_slots, const int32_t *__restrict__ count,
                    const int *__restrict__ moves, const int *__restrict__ mover,
                    const int *__restrict__ hole, int layers, long long slot_bytes) {
    move_slots(pool, num_slots, *moves, mover + (*count - *moves), hole, layers, slot_bytes);
}

// Pools of up to kFusedSlots slots: one launch, in which every CTA makes the
// lists for itself in shared memory (a plan by one CTA and a second launch cost
// 10 us more at 512 slots).
constexpr int kFusedSlots = 4096, kFusedPer = kFusedSlots / kPoolThreads;

__global__ void __launch_bounds__(kPoolThreads)
compact_kernel(char *pool, int num_slots, const uint8_t *__restrict__ live, int32_t *__restrict__ new_slot,
               int32_t *__restrict__ count, int layers, long long slot_bytes) {
    __shared__ __align__(16) uint8_t flags[kFusedSlots];
    __shared__ uint16_t mover[kFusedSlots / 2], hole[kFusedSlots / 2];
    __shared__ int warp_sum[kPoolThreads / 32], below;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int s = tid; s < kFusedSlots; s += kPoolThreads) flags[s] = s < num_slots && live[s] != 0;
    if (tid == 0) below = 0;
    __syncthreads();
    // Each thread counts a run of slots; `before` becomes the live slots below it.
    uint32_t mine = 0;  // bit i: slot first + i lives
    const int first = tid * kFusedPer;
#pragma unroll
    for (int i = 0; i < kFusedPer; ++i) mine |= (uint32_t)flags[first + i] << i;
    int before = __popc(mine);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += up;
    }
    if (lane == 31) warp_sum[warp] = before;
    __syncthreads();
    int n = 0;
#pragma unroll
    for (int w = 0; w < kPoolThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        n += warp_sum[w];
    }
    before -= __popc(mine);
    // Live slots below n: n minus the holes there.
    const int inside = min(max(n - first, 0), kFusedPer);
    const uint32_t low = mine & ((1u << inside) - 1);
    const int some = __reduce_add_sync(0xffffffffu, __popc(low));
    if (lane == 0) atomicAdd(&below, some);
    __syncthreads();
    const int kept = below, m = n - kept;
    for (int i = 0; i < kFusedPer; ++i) {
        const int s = first + i;
        if (s >= num_slots) break;
        const bool alive = mine >> i & 1;
        if (!alive && s < n) hole[s - before] = (uint16_t)s;
        if (alive && s >= n) mover[before - kept] = (uint16_t)s;
        if (blockIdx.x == 0 && !(alive && s >= n)) new_slot[s] = alive ? s : -1;
        before += alive;
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int k = tid; k < m; k += kPoolThreads) new_slot[mover[k]] = hole[k];
        if (tid == 0) *count = n;
    }
    move_slots(pool, num_slots, m, mover, hole, layers, slot_bytes);
}

cudaError_t sm_count(int *n) {
    int dev = 0;
    const cudaError_t err = cudaGetDevice(&dev);
    return err != cudaSuccess ? err : cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

cudaError_t launch_state_copy(const void *source, int source_slots, void *pool, int num_slots,
                              const int32_t *src, const int32_t *dst, int n, int layers,
                              size_t slot_bytes, cudaStream_t stream) {
    if (n == 0) return cudaSuccess;
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    // Two CTAs per SM; beyond kFewEntries entries a column of one piece each, and
    // the list, need an SM's whole shared memory for one. The limit on a kernel's
    // shared memory is the kernel's, not the launch's, so every call sets the same:
    // what its most entries need. A smaller one could come between another host
    // thread's limit and its launch, which would then be refused.
    const size_t lists = copy_list_bytes(n);
    auto launch = [&](auto kernel, int items, int per_sm, int most) {
        const size_t buffers = 2 * (size_t)items * kPoolThreads * 16;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(copy_list_bytes(most) + buffers));
        if (e != cudaSuccess) return e;
        kernel<<<sms * per_sm, kPoolThreads, lists + buffers, stream>>>(
            static_cast<const uint4 *>(source ? source : pool), source ? source_slots : num_slots,
            static_cast<uint4 *>(pool), num_slots, src, dst, n, copy_hash_size(n), layers, (uint32_t)(slot_bytes / 16),
            (int)lists);
        return cudaGetLastError();
    };
    return n > kFewEntries ? launch(state_copy_kernel<22>, 22, 1, KDA_STATE_COPY_MAX)
                           : launch(state_copy_kernel<12>, 12, 2, kFewEntries);
}

size_t compact_workspace(int num_slots) {
    return num_slots <= kFusedSlots ? 0 : kPlanHeader + 2 * align_up((size_t)num_slots * 4, 256);
}

cudaError_t launch_state_compact(void *pool, int num_slots, const uint8_t *live, int32_t *new_slot,
                                 int32_t *count, int layers, size_t slot_bytes, void *workspace,
                                 cudaStream_t stream) {
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    if (num_slots <= kFusedSlots) {
        compact_kernel<<<sms * kMoveCtas, kPoolThreads, 0, stream>>>(static_cast<char *>(pool), num_slots, live, new_slot,
                                                             count, layers, (long long)slot_bytes);
        return cudaGetLastError();
    }
    char *ws = static_cast<char *>(workspace);
    int *moves = reinterpret_cast<int *>(ws);
    int *mover = reinterpret_cast<int *>(ws + kPlanHeader);
    int *hole = reinterpret_cast<int *>(ws + kPlanHeader + align_up((size_t)num_slots * 4, 256));
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(live, num_slots, new_slot, count, moves, mover, hole);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    compact_move_kernel<<<sms * kMoveCtas, kPoolThreads, 0, stream>>>(static_cast<char *>(pool), num_slots, count, moves,
                                                              mover, hole, layers, (long long)slot_bytes);
    return cudaGetLastError();
}

}  // namespace kda
