// lp_pages.cu -- sm_103a kernels of lp_kv_reserve: the pages, rows, positions
// and slots of a round from the groups' lengths.
//
// Three exclusive sums over the groups, in order: rows (group_indptr), pages
// lacking (whose sum says what each group takes from the head of the queue, and
// whether the queue still covers it), and pages given back by idle groups.  The
// groups that get pages are those up to the first that the queue does not cover,
// so the sums need no second look.
//
// One block sums (1,024 groups at a time, carrying on), and leaves four words per
// group to the second part, which writes what is long: table entries, the tail
// of the queue, positions and slots.  A short call's block goes on to the second
// part itself; otherwise a second kernel does, on every multiprocessor.  A row's
// page is read from the table or, where it is new, from the queue, so no part
// waits for the table's writes.  New pages and pages given back never share an
// entry of the ring: entries from the tail on are free of both.
//
// Bound: latency.
#include <cuda_runtime.h>
#include <stdint.h>

#include "lp_attn.h"

namespace lp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSumThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kFillRows = 4 * kFillThreads;  // rows of a block of the second kernel

struct Sums {
    long long rows, lack, back;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) { return {a.rows + b.rows, a.lack + b.lack, a.back + b.back}; }

// Sum of the block's values before this thread's; `total`: of all.
__device__ __forceinline__ Sums block_before(const Sums& mine, Sums& total) {
    __shared__ Sums warps[kSumThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums y = {__shfl_up_sync(kFull, x.rows, o), __shfl_up_sync(kFull, x.lack, o), __shfl_up_sync(kFull, x.back, o)};
        if (lane >= o) x = x + y;
    }
    __syncthreads();  // the values of the round before are read
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    Sums before = {0, 0, 0};
    total = before;
    for (int w = 0; w < kSumThreads / 32; ++w) {
        if (w == warp) before = total;
        total = total + warps[w];
    }
    return {before.rows + x.rows - mine.rows, before.lack + x.lack - mine.lack, before.back + x.back - mine.back};
}

__device__ void reserve_groups(const ReserveParams& p) {
    const int tid = threadIdx.x;
    const long long head = p.queue[0], tail = p.queue[1];
    const bool sound = head >= 0 && tail >= head && tail - head <= p.ring;
    const long long free = sound ? tail - head : 0, room = sound ? p.ring - (tail - head) : 0;
    __shared__ unsigned long long taken, returned;
    if (tid == 0) {
        taken = returned = 0;
        if (p.G == 0) p.indptr[0] = 0;
    }
    __syncthreads();
    unsigned int status = sound ? 0u : kStatusBadPage;
    Sums base = {0, 0, 0};
    for (int g0 = 0; g0 < p.G; g0 += kSumThreads) {
        const int g = g0 + tid;
        const bool exists = g < p.G;
        const int len = exists ? p.lens[g] : 0, count = exists ? p.counts[g] : 0, held = exists ? p.held[g] : 0;
        const int n = count > 0 ? count : 0;
        const long long pages = ((long long)(len > 0 ? len : 0) + n + (1 << p.page_shift) - 1) >> p.page_shift;
        const bool holds = held >= 0 && held <= p.max_pages;
        const bool idle = len < 0;
        bool bad = exists && (count < 0 || !holds || (!idle && pages > p.max_pages));
        Sums mine = {n, !exists || idle || bad || pages <= held ? 0 : pages - held, exists && idle && holds ? held : 0};
        Sums total;
        const Sums at = base + block_before(mine, total);
        base = base + total;
        if (!exists) continue;
        const long long start = at.rows < p.rows ? at.rows : p.rows;
        // past the capacity: then every later group is too
        const bool past = at.rows + n > p.rows;
        bad = bad || past;
        const bool covered = mine.lack == 0 || at.lack + mine.lack <= free;
        const bool gives = mine.back > 0 && at.back + mine.back <= room;
        const bool serves = !idle && !bad && covered;
        if (bad) status |= kStatusAttnBadGroup;
        else if (!idle && !covered) status |= kStatusNoPages;
        if (mine.back > 0 && !gives) status |= kStatusBadPage;
        p.indptr[g] = (int)start;
        if (g == p.G - 1) p.indptr[p.G] = (int)(past ? p.rows : at.rows + n);
        p.round_lens[g] = idle ? len : (serves ? len : -1);
        p.held_out[g] = gives ? 0 : held + (serves ? (int)mine.lack : 0);
        Reserved r;
        r.first = (int)(idle ? at.back : at.lack);
        r.held = held;
        r.change = serves ? (int)mine.lack : (gives ? -1 - held : 0);
        r.lens = serves ? len : -1;
        p.groups[g] = r;
        if (serves && mine.lack > 0) atomicMax(&taken, (unsigned long long)(at.lack + mine.lack));
        if (gives) atomicMax(&returned, (unsigned long long)(at.back + mine.back));
    }
    if (status != 0) atomicOr(p.status, status);
    __syncthreads();
    if (tid == 0) {
        p.ends[0] = head, p.ends[1] = tail;
        p.queue_out[0] = head + (long long)taken;
        p.queue_out[1] = tail + (long long)returned;
    }
}

// Entry `at` past an end of the queue.
__device__ __forceinline__ int ring_at(const ReserveParams& p, long long end, long long at) { return (int)((end + at) % p.ring); }

// Tables and queue of groups first, first + step, ..: a warp each.
__device__ __forceinline__ void move_pages(const ReserveParams& p, long long head, long long tail, int first, int step) {
    const int lane = threadIdx.x & 31;
    for (int g = first; g < p.G; g += step) {
        const Reserved r = p.groups[g];
        int* table = p.tables + (long long)g * p.max_pages;
        for (int i = lane; i < r.change; i += 32) table[r.held + i] = p.free_pages[ring_at(p, head, (long long)r.first + i)];
        for (int i = lane; i < -1 - r.change; i += 32) p.free_pages[ring_at(p, tail, (long long)r.first + i)] = table[i];
    }
}

// Positions and slots of rows first, first + step, .. below `end`.
__device__ __forceinline__ void place_rows(const ReserveParams& p, long long head, long long first, long long end, int step) {
    for (long long i = first; i < end; i += step) {
        const int row = (int)i;
        long long position = -1, slot = -1;
        if (row < p.indptr[p.G]) {
            int g = 0, over = p.G;  // the last group that starts at or before the row
            while (over - g > 1) {
                const int mid = (g + over) >> 1;
                (p.indptr[mid] <= row ? g : over) = mid;
            }
            const Reserved r = p.groups[g];
            if (r.lens >= 0) {
                const int token = r.lens + row - p.indptr[g], at = token >> p.page_shift;
                position = (p.starts != nullptr ? (long long)p.starts[g] : 0) + token;
                if (position < 0 || position > 0x7FFFFFFF) {
                    position = -1;
                    atomicOr(p.status, kStatusBadPosition);
                }
                if (p.slots != nullptr) {
                    const int page = at < r.held ? p.tables[(long long)g * p.max_pages + at]
                                                 : p.free_pages[ring_at(p, head, (long long)r.first + at - r.held)];
                    if (page >= 0 && page < p.num_pages) slot = ((long long)page << p.page_shift) + (token & ((1 << p.page_shift) - 1));
                    else atomicOr(p.status, kStatusBadPage);
                }
            }
        }
        p.positions[row] = (int)position;
        if (p.slots != nullptr) p.slots[row] = slot;
    }
}

// kAlone: the one block does both parts.
template <bool kAlone>
__global__ void __launch_bounds__(kSumThreads) lp_reserve_kernel(const ReserveParams p) {
    // resident before the kernel ahead has ended: nothing is read before this wait
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    reserve_groups(p);
    if constexpr (kAlone) {
        __syncthreads();
        const long long head = p.ends[0], tail = p.ends[1];
        move_pages(p, head, tail, threadIdx.x >> 5, kSumThreads / 32);
        place_rows(p, head, threadIdx.x, p.rows, kSumThreads);
    }
}

__global__ void __launch_bounds__(kFillThreads) lp_reserve_fill_kernel(const ReserveParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long head = p.ends[0], tail = p.ends[1];
    move_pages(p, head, tail, (int)((blockIdx.x * kFillThreads + threadIdx.x) >> 5), (int)(gridDim.x * (kFillThreads / 32)));
    for (long long r0 = (long long)blockIdx.x * kFillRows; r0 < p.rows; r0 += (long long)gridDim.x * kFillRows) {
        const long long end = r0 + kFillRows < p.rows ? r0 + kFillRows : p.rows;
        place_rows(p, head, r0 + threadIdx.x, end, kFillThreads);
    }
}

// Rows and groups of a call that one block does alone.
constexpr int kAloneRows = 4096, kAloneGroups = 1024;

}  // namespace

cudaError_t launch_reserve(const ReserveParams& p, int grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(1);
    lc.blockDim = dim3(kSumThreads);
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    if (p.rows <= kAloneRows && p.G <= kAloneGroups) return cudaLaunchKernelEx(&lc, lp_reserve_kernel<true>, p);
    const cudaError_t e = cudaLaunchKernelEx(&lc, lp_reserve_kernel<false>, p);
    if (e != cudaSuccess) return e;
    const long long by_rows = ((long long)p.rows + kFillRows - 1) / kFillRows, by_groups = ((long long)p.G * 32 + kFillThreads - 1) / kFillThreads;
    const long long blocks = by_rows > by_groups ? by_rows : by_groups, most = (long long)grid * 8;
    lc.gridDim = dim3((unsigned)(blocks < most ? (blocks > 0 ? blocks : 1) : most));
    lc.blockDim = dim3(kFillThreads);
    return cudaLaunchKernelEx(&lc, lp_reserve_fill_kernel, p);
}

}  // namespace lp
