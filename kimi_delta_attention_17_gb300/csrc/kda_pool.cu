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
// a slot onto itself.
constexpr size_t copy_list_bytes(int n) { return ((size_t)n * 8 + 127) / 128 * 128; }
constexpr int copy_hash_size(int n) {
    int h = 64;
    while (h < 2 * n) h *= 2;
    return h;
}

__global__ void __launch_bounds__(kPoolThreads)
state_copy_kernel(const char *source, long long source_slots, char *pool, long long num_slots,
                  const int32_t *__restrict__ src, const int32_t *__restrict__ dst, int n, int hash_size,
                  int layers, long long slot_bytes, int buffer_bytes, int list_bytes) {
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
    int shift = 10;  // 16-byte pieces per column and entry, as a power of two
    while (shift > 0 && ((long long)copies << (shift + 4)) > buffer_bytes) --shift;
    while (shift > 3 && layers * ((slot_bytes + (16LL << shift) - 1) >> (shift + 4)) < 2LL * gridDim.x) --shift;
    const long long columns = (slot_bytes + (16LL << shift) - 1) >> (shift + 4);
    const long long units = columns * layers;
    const int pieces = copies << shift, mask = (1 << shift) - 1;

    auto gather = [&](long long unit, int b) {
        const long long layer = unit / columns, off = (unit % columns) << (shift + 4);
        const char *from = source + layer * source_slots * slot_bytes + off;
        for (int p = tid; p < pieces; p += kPoolThreads) {
            const long long in = (long long)(p & mask) * 16;
            if (off + in < slot_bytes)
                async16(buf + (size_t)b * buffer_bytes + (size_t)p * 16,
                        from + (long long)list[p >> shift].x * slot_bytes + in);
        }
    };
    long long unit = blockIdx.x;
    if (unit < units) gather(unit, 0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    for (int b = 0; unit < units; unit += gridDim.x, b ^= 1) {
        if (unit + gridDim.x < units) gather(unit + gridDim.x, b ^ 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // every source of this column has been read
        const long long layer = unit / columns, off = (unit % columns) << (shift + 4);
        char *to = pool + layer * num_slots * slot_bytes + off;
        for (int p = tid; p < pieces; p += kPoolThreads) {  // the pieces this thread gathered
            const long long in = (long long)(p & mask) * 16;
            if (off + in < slot_bytes)
                *reinterpret_cast<uint4 *>(to + (long long)list[p >> shift].y * slot_bytes + in) =
                    *reinterpret_cast<const uint4 *>(buf + (size_t)b * buffer_bytes + (size_t)p * 16);
        }
        for (int p = tid; p < zeros << shift; p += kPoolThreads) {
            const long long in = (long long)(p & mask) * 16;
            if (off + in < slot_bytes)
                *reinterpret_cast<uint4 *>(to + (long long)list[n - 1 - (p >> shift)].y * slot_bytes + in) =
                    make_uint4(0, 0, 0, 0);
        }
    }
}

// ---- compaction

// One CTA: counts the live slots, then lists in order the live slots at or
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

// Copies mover[n - m + k] to hole[k]: sources and destinations are disjoint, so
// any order does. A unit is 16 KiB of one slot.
constexpr int kMoveUnroll = 4;
constexpr long long kMoveBytes = 16LL * kPoolThreads * kMoveUnroll;

__global__ void __launch_bounds__(kPoolThreads)
compact_move_kernel(char *pool, int num_slots, const int32_t *__restrict__ count,
                    const int *__restrict__ moves, const int *__restrict__ mover,
                    const int *__restrict__ hole, int layers, long long slot_bytes) {
    const int m = *moves, first = *count - m;
    const long long pieces = (slot_bytes + kMoveBytes - 1) / kMoveBytes;
    const long long units = pieces * m * layers;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const long long piece = u % pieces, k = u / pieces % m, layer = u / pieces / m;
        char *base = pool + layer * num_slots * slot_bytes;
        const char *from = base + (long long)mover[first + k] * slot_bytes;
        char *to = base + (long long)hole[k] * slot_bytes;
        const long long at = piece * kMoveBytes + threadIdx.x * 16;
        uint4 v[kMoveUnroll];
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            const long long o = at + (long long)j * 16 * kPoolThreads;
            if (o < slot_bytes) v[j] = *reinterpret_cast<const uint4 *>(from + o);
        }
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            const long long o = at + (long long)j * 16 * kPoolThreads;
            if (o < slot_bytes) *reinterpret_cast<uint4 *>(to + o) = v[j];
        }
    }
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
    // Two CTAs per SM; up to 4096 entries of 16 bytes need an SM's whole
    // shared memory for one.
    const bool wide = n > 1024;
    const size_t lists = copy_list_bytes(n);
    const int buffer = wide ? 90 * 1024 : 48 * 1024;
    const size_t smem = lists + 2 * (size_t)buffer;
    err = cudaFuncSetAttribute(state_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    state_copy_kernel<<<sms * (wide ? 1 : 2), kPoolThreads, smem, stream>>>(
        static_cast<const char *>(source ? source : pool), source ? source_slots : num_slots,
        static_cast<char *>(pool), num_slots, src, dst, n, copy_hash_size(n), layers, (long long)slot_bytes,
        buffer, (int)lists);
    return cudaGetLastError();
}

size_t compact_workspace(int num_slots) { return kPlanHeader + 2 * align_up((size_t)num_slots * 4, 256); }

cudaError_t launch_state_compact(void *pool, int num_slots, const uint8_t *live, int32_t *new_slot,
                                 int32_t *count, int layers, size_t slot_bytes, void *workspace,
                                 cudaStream_t stream) {
    int sms = 0;
    cudaError_t err = sm_count(&sms);
    if (err != cudaSuccess) return err;
    char *ws = static_cast<char *>(workspace);
    int *moves = reinterpret_cast<int *>(ws);
    int *mover = reinterpret_cast<int *>(ws + kPlanHeader);
    int *hole = reinterpret_cast<int *>(ws + kPlanHeader + align_up((size_t)num_slots * 4, 256));
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(live, num_slots, new_slot, count, moves, mover, hole);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    compact_move_kernel<<<sms * 6, kPoolThreads, 0, stream>>>(static_cast<char *>(pool), num_slots, count, moves,
                                                              mover, hole, layers, (long long)slot_bytes);
    return cudaGetLastError();
}

}  // namespace kda
