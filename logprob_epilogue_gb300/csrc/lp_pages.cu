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
// Bound: latency.  128 groups of 4 rows: 6.2 us in one block (launch 2.5, the loads and
// sums 2, then two dependent reads per row).  4,099 groups of one row: 14.5 us, 11 of them
// the one block's five times 1,024 groups (2 us each; eight consecutive groups
// per thread took longer, 20: a block's writes then go out 32 bytes apart).  37 prompts,
// 638,367 rows: 11.2 us, the rows' 7.7 MB beside four dependent reads.  A group's pages
// are one warp's, 32 at a time, each time a read and then a write: beside 127 groups of 4
// rows one that gives 512 pages back takes 7.9 us, 2,048 15, 8,192 45, one that takes
// 8,192 new ones 48; 128 that give 8,192 each 170, all in one block.
#include <cuda_runtime.h>
#include <stdint.h>

#include "lp_attn.h"

namespace lp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSumThreads = 1024;
constexpr int kFillThreads = 256;

struct Sums {
    long long rows, lack, back;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) { return {a.rows + b.rows, a.lack + b.lack, a.back + b.back}; }

// Of one group: rows (at most one more than a call may have), pages.  32 groups' sums are below 2^32.
struct Mine {
    unsigned rows, lack, back;
};

// Sum of the block's values before this thread's; `total`: of all.
__device__ __forceinline__ Sums block_before(const Mine& mine, Sums& total) {
    static_assert(kSumThreads == 1024, "a warp's lane for each warp");
    __shared__ Sums before[33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Mine x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Mine y = {__shfl_up_sync(kFull, x.rows, o), __shfl_up_sync(kFull, x.lack, o), __shfl_up_sync(kFull, x.back, o)};
        if (lane >= o) x = {x.rows + y.rows, x.lack + y.lack, x.back + y.back};
    }
    __syncthreads();  // the sums of the round before are read
    if (lane == 31) before[warp + 1] = {x.rows, x.lack, x.back};
    __syncthreads();
    if (warp == 0) {
        Sums up = before[lane + 1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums y = {__shfl_up_sync(kFull, up.rows, o), __shfl_up_sync(kFull, up.lack, o), __shfl_up_sync(kFull, up.back, o)};
            if (lane >= o) up = up + y;
        }
        before[lane + 1] = up;
        if (lane == 0) before[0] = {0, 0, 0};
    }
    __syncthreads();
    total = before[32];
    const Sums of = before[warp];
    return {of.rows + (x.rows - mine.rows), of.lack + (x.lack - mine.lack), of.back + (x.back - mine.back)};
}

// kSumThreads groups at a time, a thread each; the next ones' values are on their way
// while these are summed.
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
    long long takes = 0, returns = 0;
    Sums base = {0, 0, 0};
    int next_len = 0, next_count = 0, next_held = 0;
    auto load = [&](int g) {
        if (g < p.G) next_len = p.lens[g], next_count = p.counts[g], next_held = p.held[g];
    };
    load(tid);
    for (int g0 = 0; g0 < p.G; g0 += kSumThreads) {
        const int g = g0 + tid, len = next_len, count = next_count, held = next_held;
        const bool exists = g < p.G;
        load(g + kSumThreads);
        const int n = exists && count > 0 ? count : 0;
        const long long pages = ((long long)(len > 0 ? len : 0) + n + (1 << p.page_shift) - 1) >> p.page_shift;
        const bool holds = held >= 0 && held <= p.max_pages;
        const bool idle = len < 0;
        bool bad = exists && (count < 0 || !holds || (!idle && pages > p.max_pages));
        const Mine mine = {(unsigned)(n <= p.rows ? n : p.rows + 1), (unsigned)(!exists || idle || bad || pages <= held ? 0 : pages - held),
                           (unsigned)(exists && idle && holds ? held : 0)};
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
        if (serves && mine.lack > 0) takes = at.lack + mine.lack;  // later groups' are no less
        if (gives) returns = at.back + mine.back;
    }
    if (status != 0) atomicOr(p.status, status);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) takes = max(takes, __shfl_xor_sync(kFull, takes, o)), returns = max(returns, __shfl_xor_sync(kFull, returns, o));
    if ((tid & 31) == 0 && takes > 0) atomicMax(&taken, (unsigned long long)takes);
    if ((tid & 31) == 0 && returns > 0) atomicMax(&returned, (unsigned long long)returns);
    __syncthreads();
    if (tid == 0) {
        p.ends[0] = sound ? head % p.ring : 0, p.ends[1] = sound ? tail % p.ring : 0;
        p.queue_out[0] = head + (long long)taken;
        p.queue_out[1] = tail + (long long)returned;
    }
}

// Entry `at` (below the ring's size) past an end of the queue, which is given by its entry.
__device__ __forceinline__ int ring_at(const ReserveParams& p, long long end, long long at) {
    return (int)(end + at < p.ring ? end + at : end + at - p.ring);
}

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

// The group of each lane's row, of rows that ascend: the last that starts at or
// before it.  The warp looks for the first row's, 32 groups at a time spread over what is
// left of them, and then over the 32 after it for all its rows; for the first row
// that starts later yet it looks again.
__device__ __forceinline__ int group_of(const ReserveParams& p, int row) {
    const int lane = threadIdx.x & 31;
    int base = 0, group = 0;
    unsigned open = kFull;  // lanes without a group yet
    while (open != 0) {
        const int target = __shfl_sync(kFull, row, __ffs(open) - 1);
        for (int over = p.G; over - base > 1;) {  // its group: one of base .. over - 1
            const int step = (over - base + 31) / 32, mine = base + lane * step;
            const unsigned upto = __ballot_sync(kFull, lane == 0 || (mine < over && p.indptr[mine] <= target));
            base += (31 - __clz((int)upto)) * step;
            over = base + step < over ? base + step : over;
        }
        const int next = base + 1 + lane, start = next < p.G ? p.indptr[next] : 0x7FFFFFFF;
        int before = 0;  // starts at or before this lane's row
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (__shfl_sync(kFull, start, before + o - 1) <= row) before += o;
        const bool all = __shfl_sync(kFull, start, 31) <= row;
        if ((open >> lane & 1u) != 0 && !all) group = base + before;
        open &= __ballot_sync(kFull, all);
    }
    return group;
}

// Positions and slots of rows first, first + step, .. below `end` (a warp's side by side).
__device__ __forceinline__ void place_rows(const ReserveParams& p, long long head, long long first, long long end, int step) {
    const int total = p.indptr[p.G];
    for (long long i = first - (threadIdx.x & 31); i < end; i += step) {
        const int row0 = (int)i, row = row0 + (threadIdx.x & 31);
        long long position = -1, slot = -1;
        const int g = row0 < total ? group_of(p, row < total ? row : total - 1) : 0;
        if (row >= end) continue;
        if (row < total) {
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

// The first row_blocks blocks place the rows, the others move the pages.
__global__ void __launch_bounds__(kFillThreads) lp_reserve_fill_kernel(const ReserveParams p, int row_blocks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long head = p.ends[0], tail = p.ends[1];
    if ((int)blockIdx.x < row_blocks) {
        place_rows(p, head, (long long)blockIdx.x * kFillThreads + threadIdx.x, p.rows, row_blocks * kFillThreads);
    } else {
        const int block = (int)blockIdx.x - row_blocks, blocks = (int)gridDim.x - row_blocks;
        move_pages(p, head, tail, (int)((block * kFillThreads + threadIdx.x) >> 5), blocks * (kFillThreads / 32));
    }
}

// Rows and groups of a call that one block does alone.  A second launch costs a caller on the host 1.8 us, and in a graph it
// gives a call's rows all multiprocessors.  Alone against with a second kernel, us in a graph: 128 groups of 4 rows 5.5 and
// 5.9, 128 of 8 5.7 and 5.8, 128 of 16 7.0 and 6.1, 128 of 32 9.6 and 6.1; 256 of 1 5.8 and 6.0, 256 of 8 7.6 and 5.9, 512 of 1
// 7.1 and 6.3, 1,024 of 1 11.1 and 6.8; one of 2,048 5.6 and 5.4.  From Python 7.7 to 8.0 and 9.4 to 9.7, but alone 9.7 for
// 128 of 32 and 11.2 for 1,024 of 1.  So up to where what a graph loses is what the host gains.
constexpr int kAloneRows = 2048, kAloneGroups = 256;

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
    const long long most = (long long)grid * 8;
    auto blocks = [&](long long threads) {
        const long long n = (threads + kFillThreads - 1) / kFillThreads;
        return (int)(n < most ? n : most);
    };
    const int row_blocks = blocks(p.rows), page_blocks = blocks((long long)p.G * 32);
    if (row_blocks + page_blocks == 0) return cudaSuccess;
    lc.gridDim = dim3((unsigned)(row_blocks + page_blocks));
    lc.blockDim = dim3(kFillThreads);
    return cudaLaunchKernelEx(&lc, lp_reserve_fill_kernel, p, row_blocks);
}

}  // namespace lp
