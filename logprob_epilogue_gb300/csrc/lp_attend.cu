// lp_attend.cu -- sm_103a kernels of lp_attend: attention of verify rows over
// a paged cache with shared prefixes.
//
// For a row's query head q over its visible tokens t:
//   s_t = scale q.k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t exp s_t.
// A sum over tokens splits into parts: over a set A of tokens keep
// m_A = max s, l_A = sum exp(s - m_A), o_A = sum exp(s - m_A) v; two parts join
// as m = max(m_A, m_B), l = l_A exp(m_A - m) + l_B exp(m_B - m), o alike.
//
// Split of the work.  What every row of a segment sees (a prefix's tokens by
// the rows of all its groups, a group's committed tokens by its own rows) goes
// to lp_attend_kernel on the tensor cores and needs no mask but the length;
// the round's own tokens (at most 32, masked row by row) are added by
// lp_attend_join_kernel, which also joins the parts.  So a NaN or infinity in a
// token that a row does not see never meets that row: nothing is multiplied
// by a zero probability.  (Slots past a length are zeroed in shared memory.)
//
// The query rows of a segment and key-value head (a row's `share` heads side
// by side) form units of up to two tiles of 128; a unit's tokens form tiles of
// 128.  The prefixes' token tiles, unit after unit, are cut into one equal run
// per block, wherever that falls, and after them the groups': one request at a
// long context and hundreds of short ones fill the machine alike, the blocks
// are all at the arithmetic or all at the memory at a time, and none waits on
// another.  Before that, a prefix with more units than blocks deals them out
// whole, one to every block at a time: the blocks of a head then go through
// its tokens side by side, and a tile that one of them fetched is still in L2
// for the others (2,048 rows behind 32,768 tokens: 762 us against 870).  A unit
// of two query tiles reads each K and V tile once for both; a unit of one tile
// gives its even token tiles to one warpgroup and its odd ones to the other,
// each with its own maximum, sum and accumulator.
//
// Block (one per SM, 12 warps): warp 0 splits the work and fetches pages by TMA
// into a ring of K and V tiles (160 KiB); warps 1 and 2 issue the products, each
// of one tensor tile; warp 3 loads the queries of one-tile units; warps 4-7 and
// 8-11 are two softmax warpgroups, one row per thread.
//   S_i = Q_i K^T    128 x 128, shared x shared -> tensor memory
//   softmax: S_i to registers, P_i (the plan's type) back over S_i
//   O_i += P_i V     tensor memory x shared -> tensor memory, the first 64
//                    tokens' part while the softmax of the others runs
// While one warpgroup works on its S the tensor core runs the other's
// products.  Each row keeps a running maximum and sum (the online softmax of
// Milakov and Gimelshein, 2018); after a published refinement of it the maximum
// moves only when it grows by more than 2^8 (then O and the sum are rescaled),
// so most tiles touch O not at all.
// P is rounded to the plan's type (the products take nothing wider); S, the
// maxima, the sums, O and the parts are 32 bits.
//
// What bounds it, by size (BF16, heads of 128, 32 over 8, in a CUDA graph):
// - bandwidth, where few rows share a token: 128 groups of 4 rows at contexts up
//   to 8,192 take 344 us, 6.5 TB/s of keys and values;
// - the tensor core, where many rows share a prefix: of 2,048 rows behind 32,768
//   tokens the prefix's part takes 595 us, 1.85 PFLOP/s (2,700 cycles a pair of
//   token tiles, the products alone 2,048).  The whole call takes 750 us: then
//   come the groups' own tokens (0.5 GB) in 110, and the parts' join in 40;
// - latency, in short calls: one row at 4,095 tokens takes 15.0 us: the launch and
//   the split 2.5, the first scores 2.5, two token tiles 4, the join 5.5.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "lp_attn.h"
#include "lp_tc.h"

namespace lp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
// Tokens of a tile whose probabilities are announced before the others', so that
// their part of P V runs under the rest of the softmax (2,048 rows behind 32,768
// tokens: 762 us; 32 tokens 785, 96 790, all at once 809).
constexpr int kEarly = 64;
constexpr float kRescale = 8.0f;  // growth of the maximum (log2) that moves it
// What a run is measured in, by the times of each: a token tile of a one-tile
// unit is 2, of a two-tile unit 3, and every unit 4 more (its queries, first
// loads and results).  No run is shorter than a tile, nor one of prefixes than
// four (every run of a unit leaves a part for the join to read).
constexpr int kTileCost = 2, kPairCost = 3, kUnitCost = 4;
constexpr int kLeastPrefix = 4 * kPairCost, kLeastGroup = kPairCost;
// Registers: the softmax warpgroups hold 128 scores per thread.  The split's
// sum is what the block is launched with, 384 x 168.
constexpr int kRegsLaunch = 168, kRegsSoftmax = 200, kRegsOther = 104;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "register split");

// Tensor memory columns: two score tiles, two accumulators.
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256, kColStep = 128;

template <int D>
struct Cfg {
    static constexpr int kTileBytes = kKTile * D * 2;     // one K, V or Q tile
    static constexpr int kSlots = 5 * 128 / D;            // ring of K and V tiles: 160 KiB
    static constexpr int kCtl = (2 + kSlots) * kTileBytes;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The call's vectors are read with ordinary loads: the kernels are resident
// before the kernel that writes them has ended, and a read-only load might be
// moved ahead of the wait for that.

// One verify group: its rows and committed tokens.  n = 0: idle or malformed.
struct Group {
    int r0, n, len;
    bool bad;
};

__device__ __forceinline__ Group load_group(const AttendParams& p, int g) {
    Group x;
    const int r0 = p.indptr[g], r1 = p.indptr[g + 1];
    x.r0 = r0;
    x.len = p.lens[g];
    const long long n = (long long)r1 - r0;
    x.bad = r0 < 0 || r1 > p.rows || n < 0 || n > p.max_group_rows ||
            (x.len >= 0 && (long long)x.len + n > ((long long)p.max_pages << p.page_shift));
    x.n = x.bad || x.len < 0 ? 0 : (int)n;
    return x;
}

// Prefix i: its groups, their rows, its tokens.  n = 0: none, or malformed.
struct Prefix {
    int g0, g1, r0, n, len;
    bool bad;
};

__device__ __forceinline__ Prefix load_prefix(const AttendParams& p, int i) {
    Prefix x;
    x.g0 = p.prefix_indptr[i];
    x.g1 = p.prefix_indptr[i + 1];
    x.len = p.prefix_lens[i];
    x.bad = x.g0 < 0 || x.g1 < x.g0 || x.g1 > p.G || x.len < 0 ||
            (long long)x.len > ((long long)p.max_prefix_pages << p.page_shift);
    x.r0 = x.n = 0;
    if (!x.bad) {
        const int r0 = p.indptr[x.g0], r1 = p.indptr[x.g1];
        x.bad = r0 < 0 || r1 < r0 || r1 > p.rows;
        if (!x.bad) x.r0 = r0, x.n = r1 - r0;
    }
    return x;
}

// Segment s: prefixes 0..P-1, then the groups' committed tokens.
struct Seg {
    int r0, n, len;
    int tiles, units;  // token tiles; units per key-value head; tiles = 0: no work
    int dealt;         // of all heads' units, those that go round the blocks whole
    bool bad;
    __device__ __forceinline__ int left(const AttendParams& p) const { return tiles > 0 ? units * p.kv_heads - dealt : 0; }
    int cost;          // of a token tile
    __device__ __forceinline__ long long span() const { return (long long)tiles * cost + kUnitCost; }  // of a unit in a run
    __device__ __forceinline__ unsigned long long work(const AttendParams& p) const { return (unsigned long long)(span() * left(p)); }
};

__device__ __forceinline__ Seg load_seg(const AttendParams& p, int s) {
    Seg x;
    if (s < p.P) {
        const Prefix f = load_prefix(p, s);
        x.r0 = f.r0, x.n = f.n, x.len = f.len, x.bad = f.bad;
    } else {
        const Group f = load_group(p, s - p.P);
        x.r0 = f.r0, x.n = f.n, x.len = f.len, x.bad = f.bad;
    }
    x.units = (x.n + 2 * p.rows_per_tile - 1) / (2 * p.rows_per_tile);
    x.tiles = x.n > 0 ? (x.len + kKTile - 1) / kKTile : 0;
    x.cost = x.n > p.rows_per_tile ? kPairCost : kTileCost;
    x.dealt = s < p.P && x.tiles > 0 ? x.units * p.kv_heads / p.grid * p.grid : 0;
    return x;
}

// The units' cost, `total` in all, cut into one run per block: blocks
// 0..more-1 take per + 1, the others per.
struct Runs {
    unsigned long long total, per;
    int blocks, more;
    __device__ __forceinline__ unsigned long long start(int c) const { return per * c + (c < more ? c : more); }
    __device__ __forceinline__ int block_of(unsigned long long t) const {
        const unsigned long long big = (per + 1) * more;
        return t < big ? (int)quotient(t, per + 1) : more + (int)quotient(t - big, per);
    }
    static __device__ __forceinline__ unsigned long long quotient(unsigned long long a, unsigned long long b) {
        return ((a | b) >> 32) == 0 ? (unsigned)a / (unsigned)b : a / b;  // the 64-bit division is slow
    }
};

__device__ __forceinline__ Runs make_runs(unsigned long long total, int grid, int kind) {
    Runs r;
    r.total = total;
    // a run as long as a tile holds the start of one, wherever it lies among a unit's tiles
    const unsigned long long most = Runs::quotient(total, kind == 0 ? kLeastPrefix : kLeastGroup);
    r.blocks = most < (unsigned long long)grid ? (int)most : grid;
    if (r.blocks == 0 && total > 0) r.blocks = 1;
    r.per = r.blocks > 0 ? Runs::quotient(total, r.blocks) : 0;
    r.more = (int)(total - r.per * r.blocks);
    return r;
}

// Index of row 0 of a piece's part (tile or warpgroup `set`); -1: past the
// scratch (only overlapping prefixes can ask for that).
__device__ __forceinline__ long long part_row(const AttendParams& p, bool prefix, long long slot, int set) {
    if (prefix) return slot < p.sc.prefix_slots ? (slot * 2 + set) * kQTile : -1;
    if (slot >= p.sc.group_slots) return -1;
    return p.sc.prefix_slots * 2 * kQTile + (slot * 2 + set) * p.sc.group_rows;
}

// Where a unit that is not dealt out is entered for the join; -1 as above.
__device__ __forceinline__ long long unit_index(const AttendParams& p, bool prefix, int unit) {
    if (prefix) return unit < p.sc.prefix_slots ? unit : -1;
    return unit < p.sc.group_slots ? p.sc.prefix_slots + unit : -1;
}

// A part's results lie chunk by chunk, four lanes of the head of every row
// side by side (a warp's stores are whole lines): index of a float4, `base`
// the part's first row and `cap` the rows it has room for.
template <int D>
__device__ __forceinline__ long long part_chunk(long long base, int cap, int row, int chunk) {
    return base * (D / 4) + (long long)chunk * cap + row;
}

// A block's share of one unit.
struct Piece {
    int row, rows;      // first row and rows of the unit; rows = 0: the run is done
    int kvh, tiles;
    int left;           // tokens from its first tile to the segment's end
    int part_stride;    // rows between the parts of its two tiles (or warpgroups)
    long long part;     // row 0 of its first part; -1: past the scratch (only overlapping prefixes can ask for that)
};

// Where a block's run begins: its first segment, the tiles and units before it.
struct Start {
    unsigned long long off;
    int seg, units;
    Seg s;
};

// Walks a block's pieces: its share of the units that go round whole, then its
// run of the other prefix units' tiles, then of the groups'.
struct Walk {
    Runs runs[2], run;                 // of prefixes, of groups; the current
    unsigned long long begin[2], finish[2];  // this block's
    const Start* start;
    int kind;
    int deal, deal_end, round, dealt;  // segments with units that go round; rounds dealt; units of earlier segments
    unsigned long long pos, end, off;  // off: tiles before the segment
    int seg, units, cta;               // units: the segment's first slot less cta
    Seg s;
    __device__ __forceinline__ void enter(int k) {
        kind = k;
        run = runs[k];
        pos = begin[k], end = finish[k];
        off = start[k].off, seg = start[k].seg, units = start[k].units, s = start[k].s;
    }
    const int* table;                  // pages of the piece, and its first token
    long long token;
    __device__ __forceinline__ void fill(const AttendParams& p, Piece& x, int sg, const Seg& y, int unit, int t0, int tiles, long long slot) {
        const bool prefix = sg < p.P;
        x.tiles = tiles;
        x.kvh = unit / y.units;
        const int first = (unit - x.kvh * y.units) * 2 * p.rows_per_tile;
        x.row = y.r0 + first;
        x.rows = y.n - first < 2 * p.rows_per_tile ? y.n - first : 2 * p.rows_per_tile;
        x.left = y.len - t0 * kKTile;
        table = prefix ? p.prefix_tables + (long long)sg * p.max_prefix_pages : p.tables + (long long)(sg - p.P) * p.max_pages;
        token = (long long)t0 * kKTile;
        x.part = part_row(p, prefix, slot, 0);
        x.part_stride = prefix ? kQTile : p.sc.group_rows;
    }
    __device__ __forceinline__ bool next(const AttendParams& p, Piece& x) {
        while (deal < deal_end) {
            const Seg y = load_seg(p, deal);
            const int unit = round * p.grid + cta;
            if (unit < y.dealt) {
                ++round;
                fill(p, x, deal, y, unit, 0, y.tiles, dealt + unit);
                return true;
            }
            dealt += y.dealt;
            ++deal;
            round = 0;
        }
        while (pos < end || kind == 0) {
            if (pos >= end) {
                enter(1);
                continue;
            }
            const unsigned long long work = s.work(p);
            if (pos >= off + work) {
                off += work;
                units += s.left(p);
                s = load_seg(p, ++seg);
                continue;
            }
            // the unit's cost lies before its tiles, and a tile belongs to the run that its start lies in
            const unsigned long long rel = pos - off, rest = end - pos, span = s.span();
            const int unit = (int)Runs::quotient(rel, span);
            const long long u0 = (long long)(rel - unit * span), u1 = rest < span - u0 ? u0 + (long long)rest : (long long)span;
            pos += u1 - u0;
            const int t0 = u0 > kUnitCost ? (int)((u0 - kUnitCost + s.cost - 1) / s.cost) : 0;
            const int t1 = u1 > kUnitCost ? (int)((u1 - kUnitCost + s.cost - 1) / s.cost) : 0;
            if (t1 <= t0) continue;
            fill(p, x, seg, s, s.dealt + unit, t0, t1 - t0, (long long)units + unit + cta);
            if (t0 == 0 && (threadIdx.x & 31) == 0) {
                // for the join: the unit's first slot and how many blocks have a piece of it
                const unsigned long long last = off + unit * span + kUnitCost + (unsigned long long)(s.tiles - 1) * s.cost;
                const long long at = unit_index(p, kind == 0, units + unit);
                if (at >= 0) p.sc.units[at] = make_int2(units + unit + cta, t1 == s.tiles ? 1 : run.block_of(last) - cta + 1);
            }
            return true;
        }
        x.rows = 0;
        return false;
    }
};

constexpr int kPieces = 8;        // pieces the fetching warp may be ahead
constexpr int kPieceReaders = 11; // warps that read each: two of the products, one that loads queries, eight of softmax

struct Ctl {
    uint64_t full[10], empty[10], piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    uint64_t q_full[2], q_free[2], s_full[2], p_early[2], p_ready[2], pv_done[2], o_free[2], q_grant, clean, drain;
    unsigned long long sum[kWarps][3];
    int sum_dealt[kWarps], deal_first, deal_last;
    Start start[2];
    uint32_t tmem, issued, batches[2];  // ring fills under way or done; see take_turn
    int abort;
};

// The call's tiles and units: every thread sums its share of the segments,
// the block scans the sums, and the thread that holds the block's first tile
// names its segment.  Block 0 leaves the offsets for the join.  False: the
// block has no work.
__device__ __forceinline__ bool plan_run(const AttendParams& p, Ctl* ctl, Runs (&runs)[2]) {
    const int S = p.P + p.G, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per < S ? tid * per : S, s1 = s0 + per < S ? s0 + per : S;
    // of prefixes and of groups; units: slots of units that do not go round, of prefixes in the high half
    unsigned long long cost0 = 0, cost1 = 0, units = 0;
    int dealt = 0, first = S, last = -1;
    for (int s = s0; s < s1; ++s) {
        const Seg x = load_seg(p, s);
        (s < p.P ? cost0 : cost1) += x.work(p);
        units += (unsigned long long)x.left(p) << (s < p.P ? 32 : 0);
        dealt += x.dealt;
        if (x.dealt > 0) {
            if (last < 0) first = s;
            last = s;
        }
        if (x.bad && blockIdx.x == 0) atomicOr(p.status, s < p.P ? kStatusBadPrefix : kStatusAttnBadGroup);
    }
    unsigned long long i0 = cost0, i1 = cost1, iu = units;
    int id = dealt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long a = __shfl_up_sync(kFull, i0, o), b = __shfl_up_sync(kFull, i1, o), c = __shfl_up_sync(kFull, iu, o);
        const int d = __shfl_up_sync(kFull, id, o);
        if (lane >= o) i0 += a, i1 += b, iu += c, id += d;
    }
    if (lane == 31) ctl->sum[warp][0] = i0, ctl->sum[warp][1] = i1, ctl->sum[warp][2] = iu, ctl->sum_dealt[warp] = id;
    if (tid == 0) ctl->deal_first = S, ctl->deal_last = -1;
    __syncthreads();
    if (last >= 0) atomicMin(&ctl->deal_first, first), atomicMax(&ctl->deal_last, last);
    unsigned long long b0 = 0, b1 = 0, bu = 0, total0 = 0, total1 = 0;
    int bd = 0, all_dealt = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) b0 = total0, b1 = total1, bd = all_dealt;
        if (w < warp) bu += ctl->sum[w][2];
        total0 += ctl->sum[w][0];
        total1 += ctl->sum[w][1];
        all_dealt += ctl->sum_dealt[w];
    }
    unsigned long long at0 = b0 + i0 - cost0, at1 = b1 + i1 - cost1, u = bu + iu - units;
    int d = bd + id - dealt;
    runs[0] = make_runs(total0, gridDim.x, 0);
    runs[1] = make_runs(total1, gridDim.x, 1);
    const int cta = blockIdx.x;
    const unsigned long long lo0 = cta < runs[0].blocks ? runs[0].start(cta) : ~0ull, lo1 = cta < runs[1].blocks ? runs[1].start(cta) : ~0ull;
    if (cta == 0 || (lo0 >= at0 && lo0 < at0 + cost0) || (lo1 >= at1 && lo1 < at1 + cost1)) {
        for (int s = s0; s < s1; ++s) {
            const Seg x = load_seg(p, s);
            const int kind = s < p.P ? 0 : 1;
            const unsigned long long work = x.work(p), off = kind == 0 ? at0 : at1, lo = kind == 0 ? lo0 : lo1;
            const int before = (int)(kind == 0 ? (u >> 32) + all_dealt : u & 0xFFFFFFFFull);  // slots: the dealt units', then the others'
            if (cta == 0) p.sc.seg_units[s] = make_int2(before, d);
            if (lo >= off && lo < off + work) ctl->start[kind].off = off, ctl->start[kind].seg = s, ctl->start[kind].units = before, ctl->start[kind].s = x;
            (kind == 0 ? at0 : at1) += work;
            u += (unsigned long long)x.left(p) << (kind == 0 ? 32 : 0);
            d += x.dealt;
        }
    }
    return all_dealt > 0 || cta < runs[0].blocks || cta < runs[1].blocks;
}

__device__ __forceinline__ unsigned long long pack2(uint32_t a, uint32_t b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One row's running softmax: the maximum, what is subtracted in base 2, the sum.
struct Row {
    float m, base, l;
};

// The maximum after scores up to `top`; f: what sums so far are worth under it.
// The first tile sets it; later it moves only where it grew by 2^kRescale
// (`used`: the row exists), so that most tiles leave the accumulator alone.
template <bool kBf16>
__device__ __forceinline__ bool raise(Row& row, float top, bool first, bool used, float c, float& f) {
    // F16 keeps probabilities down to 2^-24: lifting them by 2^6 (at most 2^14 then) keeps those above 2^-30
    constexpr float kBias = kBf16 ? 0.0f : 6.0f;
    f = 1.0f;
    if (first) {
        row.m = top;
        row.base = top == kNegInf ? 0.0f : top * c - kBias;
        row.l = 0.0f;
        return false;
    }
    const bool grow = used && (row.m == kNegInf ? top > row.m : top * c > row.m * c + kRescale);
    if (grow) {
        const float next = top * c - kBias;
        if (row.m != kNegInf) f = ex2(row.base - next);
        row.m = top;
        row.base = next;
        row.l *= f;
    }
    return __any_sync(kFull, grow);
}

// O *= f: the scores came after the products before them, so the accumulator
// is this warp's to change.
template <int D>
__device__ __forceinline__ void rescale(uint32_t o_col, float f) {
#pragma unroll 1
    for (int b = 0; b < D / 32; ++b) {
        uint32_t o[32];
        tc::tmem_ld32(o_col + b * 32, o);
        tc::wait_ld();
        tc::tie(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tc::tmem_st32(o_col + b * 32, o);
    }
}

__device__ __forceinline__ float max32(const uint32_t (&r)[32], float top) {
    float a = top, b = kNegInf;
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        a = max3(a, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
        b = max3(b, __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
    }
    return fmaxf(a, b);
}

// The scores of tokens from `valid` on to -infinity, in tensor memory: short
// code, since a call comes here once per unit (see the loop below).
__device__ __forceinline__ void mask_scores(uint32_t s_col, int valid) {
#pragma unroll 1
    for (int b = valid & ~15; b < kKTile; b += 16) {
        uint32_t r[16];
        tc::tmem_ld16(s_col + b, r);
        tc::wait_ld();
        tc::tie(r);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (b + e >= valid) r[e] = __float_as_uint(kNegInf);
        tc::tmem_st16(s_col + b, r);
    }
    tc::wait_st();
}

// Softmax of one score tile by one warp, a row per thread; `valid` of the 128
// tokens exist.  Writes the row's probabilities over the scores.
template <bool kBf16, int D>
__device__ __forceinline__ void softmax_tile(uint32_t s_col, uint32_t o_col, int valid, bool first, bool used, float c, Row& row, uint64_t* early) {
    if (valid < kKTile) mask_scores(s_col, valid);
    uint32_t r[4][32];
#pragma unroll
    for (int b = 0; b < 4; ++b) tc::tmem_ld32(s_col + b * 32, r[b]);
    tc::wait_ld();
#pragma unroll
    for (int b = 0; b < 4; ++b) tc::tie(r[b]);
    float top = kNegInf, f;
#pragma unroll
    for (int b = 0; b < 4; ++b) top = max32(r[b], top);
    if (raise<kBf16>(row, top, first, used, c, f)) rescale<D>(o_col, f);
    const unsigned long long c2 = pack2(__float_as_uint(c), __float_as_uint(c));
    const unsigned long long nb2 = pack2(__float_as_uint(-row.base), __float_as_uint(-row.base));
    unsigned long long sum[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < 4; ++b) {  // 32 scores to 16 words of probabilities
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float x, y;
            unpack2(fma2(pack2(r[b][2 * e], r[b][2 * e + 1]), c2, nb2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[e & 1] = add2(sum[e & 1], pack2(__float_as_uint(x), __float_as_uint(y)));
            w[e] = Half<kBf16>::pack(x, y);
        }
        tc::tmem_st16(s_col + b * 16, w);
        if (b == kEarly / 32 - 1) {  // the products of the tile's first tokens may begin
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) tc::mbar_arrive(early);
        }
    }
    float x, y;
    unpack2(add2(sum[0], sum[1]), x, y);
    row.l += x + y;
    tc::wait_st();
}

// Where the second warpgroup's copy of a one-tile unit's rows begins in the
// query tile: half of a tile that is at most half full is free, and there the
// rows are in tensor memory lanes of other warps, on other schedulers, than the
// first warpgroup's (four groups past 100,000 tokens: 48.7 us against 52.9, trees
// of drafts 43.6 against 44.6).
__device__ __forceinline__ int second_at(int rows) { return rows <= kQTile / 2 ? kQTile / 2 : 0; }

// The rows' heads into a query tile (128-byte swizzle) by `n` threads, visible
// to the tensor core; `again` > 0: a second time from that tile row on.  Tile
// rows without a query hold anything and reach nothing.
template <typename T, int D>
__device__ __forceinline__ void load_queries(const AttendParams& p, int row0, int rows, int kvh, uint32_t dst, int again, int t, int n) {
    constexpr int kChunks = D / 8;
    const T* src = reinterpret_cast<const T*>(p.q) + (long long)row0 * p.q_stride + (long long)kvh * p.share * D;
    for (int i = t; i < rows * p.share * kChunks; i += n) {
        const int row = i / kChunks, ch = i % kChunks;
        const int per = (row * p.share_inv) >> 16, head = row - per * p.share;
        const uint32_t at = dst + (ch >> 3) * (kQTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
        const T* from = src + per * p.q_stride + head * D + ch * 8;
        tc::copy16(at, from);
        if (again > 0) tc::copy16(at + again * 128, from);
    }
    tc::copies_done();
    tc::fence_async_shared();
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    lp_attend_kernel(const AttendParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using H = Half<kBf16>;
    using T = typename H::T;
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::kCtl);
    unsigned char* ring = smem + 2 * C::kTileBytes;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, as the compiler sees
    const unsigned long long limit = p.timeout_ns;
    // the barriers, while the kernel ahead still runs
    if (warp == kWarps - 1) {
        if (lane < C::kSlots) tc::mbar_init(&ctl->full[lane], 1), tc::mbar_init(&ctl->empty[lane], 2);
        if (lane < kPieces) tc::mbar_init(&ctl->piece_full[lane], 1), tc::mbar_init(&ctl->piece_empty[lane], kPieceReaders);
        if (lane < 2) {
            tc::mbar_init(&ctl->q_full[lane], 4);
            tc::mbar_init(&ctl->q_free[lane], 2);
            tc::mbar_init(&ctl->s_full[lane], 1);
            tc::mbar_init(&ctl->p_early[lane], 4);
            tc::mbar_init(&ctl->p_ready[lane], 4);
            tc::mbar_init(&ctl->pv_done[lane], 1);
            tc::mbar_init(&ctl->o_free[lane], 4);
            ctl->batches[lane] = 0;
        }
        if (lane == 0) {
            tc::mbar_init(&ctl->clean, 1);
            tc::mbar_init(&ctl->q_grant, 1);
            tc::mbar_init(&ctl->drain, 2);
            ctl->abort = 0;
            ctl->issued = 0;
        }
        tc::fence_async_shared();
    }
    if (tid == 0) tc::prefetch_map(&k_map), tc::prefetch_map(&v_map);
    // so far nothing of what earlier kernels write; the join may start once that is there, and waits for this grid's end by itself
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 2) tc::tmem_alloc(&ctl->tmem, kTmemCols);  // not held while waiting: the kernel ahead may need it to end
    Runs runs[2];  // of prefixes, of groups
    const bool any = plan_run(p, ctl, runs);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ctl->tmem;
    if (!any) {
        if (tid == 0) p.sc.gave_up[blockIdx.x] = 0;
        if (warp == 2) tc::tmem_dealloc(tmem, kTmemCols);
        return;
    }
    volatile int* abort = &ctl->abort;
    // test hook: nothing arrives on `drain` before the end, so this wait runs out
    if (p.force_timeout) tc::warp_wait(&ctl->drain, 0, limit, abort);

    Piece x;
    bool ok = !p.force_timeout;
    uint32_t n_piece = 0;
    // the next piece, from the fetching warp; false at the end of the run
    auto next_piece = [&]() {
        const uint32_t i = n_piece % kPieces;
        ok = tc::warp_wait(&ctl->piece_full[i], n_piece / kPieces & 1u, limit, abort);
        if (!ok) return false;
        x = ctl->piece[i];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->piece_empty[i]);
        ++n_piece;
        return x.rows > 0;
    };

    uint32_t it = 0;  // ring position: a tile's K, then its V

    // Each role sets its registers inside its own branch: code that both counts reach is held to the smaller.
    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax
        const int wg = (warp - 4) >> 2, quarter = warp & 3;  // tensor tile; lanes 32 * quarter of tensor memory
        const uint32_t lanes = (uint32_t)quarter << 21;
        const uint32_t s_col = tmem + lanes + kColS + wg * kColStep, o_col = tmem + lanes + kColO + wg * kColStep;
        const float c = p.scale * kLog2e;
        uint32_t s_phase = 0, pv_phase = 0, q_pos = 0, grant = 0, tile = 0;  // tile: tiles of the run before the piece
        int turn = 0;
        while (ok && next_piece()) {
            const bool two = x.rows > p.rows_per_tile;
            const int n = x.tiles, rt = p.rows_per_tile;
            const int valid_rows = (two ? (wg == 0 ? rt : x.rows - rt) : x.rows) * p.share;
            const int row0 = quarter * 32 - (wg == 1 && !two ? second_at(valid_rows) : 0), row = row0 + lane;  // of the query tile
            const bool live = row0 >= 0 && row0 < valid_rows, used = live && row < valid_rows;  // any row of this warp; this row
            const int first = two ? 0 : wg ^ turn, stride = two ? 1 : 2;
            if (!two) turn ^= n & 1;
            if (two) {
                ok = tc::warp_wait(&ctl->q_grant, grant, limit, abort);  // both buffers are free
                if (!ok) break;
                grant ^= 1u;
                const uint32_t b = (q_pos + wg) & 1u;
                load_queries<T, D>(p, x.row + wg * rt, wg == 0 ? rt : x.rows - rt, x.kvh, tc::smem_addr(smem + b * C::kTileBytes), 0, tid & 127, 128);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->q_full[b], 1);
            }
            q_pos += two ? 2 : 1;
            Row st = {kNegInf, 0.0f, 0.0f};
            for (int i = first; i < n; i += stride) {
                ok = tc::warp_wait(&ctl->s_full[wg], s_phase, limit, abort);
                if (!ok) break;
                s_phase ^= 1u;
                if (two && wg == 0 && quarter == 0 && lane == 0) {  // thread 0's products have read K of this tile and V of the one before
                    tc::mbar_arrive(&ctl->empty[(tile + i) * 2 % C::kSlots]);
                    if (i > 0) tc::mbar_arrive(&ctl->empty[((tile + i) * 2 - 1) % C::kSlots]);
                }
                if (live) {
                    tc::fence_after();
                    softmax_tile<kBf16, D>(s_col, o_col, x.left - i * kKTile, i == first, used, c, st, &ctl->p_early[wg]);
                    tc::fence_before();
                    __syncwarp();
                } else if (lane == 0) {
                    tc::mbar_arrive(&ctl->p_early[wg]);
                }
                if (lane == 0) tc::mbar_arrive(&ctl->p_ready[wg]);
            }
            tile += n;
            if (!ok) break;
            const long long part = x.part + wg * x.part_stride;
            const bool store = used && x.part >= 0;
            if (first >= n) {  // no tile of this piece was this warpgroup's
                if (store) p.sc.part_ml[part + row] = make_float2(kNegInf, 0.0f);
                continue;
            }
            ok = tc::warp_wait(&ctl->pv_done[wg], pv_phase, limit, abort);
            if (!ok) break;
            pv_phase ^= 1u;
            if (two && wg == 0 && quarter == 0 && lane == 0) tc::mbar_arrive(&ctl->empty[(tile * 2 - 1) % C::kSlots]);
            if (live) {
                tc::fence_after();
                if (store) p.sc.part_ml[part + row] = make_float2(st.m == kNegInf ? kNegInf : st.base, st.l);
                float4* dst = reinterpret_cast<float4*>(p.sc.part_o) + part_chunk<D>(part, x.part_stride, row, 0);
#pragma unroll 1
                for (int b = 0; b < D / 32; ++b) {
                    uint32_t o[32];
                    tc::tmem_ld32(o_col + b * 32, o);
                    tc::wait_ld();
                    tc::tie(o);
                    if (store) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[(b * 8 + e) * x.part_stride] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                           __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    }
                }
                tc::fence_before();
                __syncwarp();
            }
            if (lane == 0) tc::mbar_arrive(&ctl->o_free[wg]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 0) {
            // ---- pages into the ring
            constexpr int kHalves = D / 64;
            const int step = p.page_shift < 7 ? 1 << p.page_shift : kKTile;  // tokens per box
            const int tok = lane / kHalves * step, half = lane % kHalves;
            Walk walk;
            walk.cta = blockIdx.x;
            walk.deal = ctl->deal_first;
            walk.deal_end = ctl->deal_last + 1;
            walk.round = walk.dealt = 0;
            walk.start = ctl->start;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                walk.runs[k] = runs[k];
                const bool any = (int)blockIdx.x < runs[k].blocks;
                walk.begin[k] = any ? runs[k].start(blockIdx.x) : 0;
                walk.finish[k] = any ? runs[k].start(blockIdx.x + 1) : 0;
            }
            walk.enter(0);
            auto fetch = [&](const CUtensorMap* map, int n, int fy, int fh, int fp) {
                const uint32_t slot = it % C::kSlots;
                if (!tc::warp_wait(&ctl->empty[slot], (it / C::kSlots & 1u) ^ 1u, limit, abort)) return false;
                if (lane == 0) {
                    tc::mbar_expect(&ctl->full[slot], (uint32_t)n * step * 128u);
                    tc::store_release(&ctl->issued, it + 1);
                }
                __syncwarp();
                if (lane < n)
                    tc::tma_load_4d(ring + slot * C::kTileBytes + half * (kKTile * 128) + tok * 128, map, &ctl->full[slot], half * 64, fy, fh, fp);
                ++it;
                return true;
            };
            auto page_of = [&](int i) {
                const long long at = walk.token + i * kKTile + tok;
                return i < x.tiles && i * kKTile + tok < x.left ? walk.table[at >> p.page_shift] : -1;
            };
            for (bool more = ok; ok && more;) {
                more = walk.next(p, x);
                const uint32_t pi = n_piece % kPieces;
                ok = tc::warp_wait(&ctl->piece_empty[pi], (n_piece / kPieces & 1u) ^ 1u, limit, abort);
                if (!ok) break;
                if (lane == 0) {
                    ctl->piece[pi] = x;
                    tc::mbar_arrive(&ctl->piece_full[pi]);
                }
                ++n_piece;
                if (!more) break;
                // the pages of the next tile are read before this tile's waits
                int next_page = page_of(0);
                for (int i = 0; ok && i < x.tiles; ++i) {
                    const int left = x.left - i * kKTile, valid = left < kKTile ? left : kKTile;
                    const int boxes = (valid + step - 1) / step * kHalves, kvh = x.kvh;
                    const int y = (int)((walk.token + i * kKTile + tok) & ((1 << p.page_shift) - 1));
                    int page = next_page;
                    next_page = page_of(i + 1);
                    if (lane < boxes && (page < 0 || page >= p.num_pages)) {
                        page = (int)p.num_pages;  // outside the map: zeros
                        atomicOr(p.status, kStatusBadPage);
                    }
                    ok = fetch(&k_map, boxes, y, kvh, page) && fetch(&v_map, boxes, y, kvh, page);
                }
            }
            // no copy outlives the block, whatever its readers did
            int none = 0;
            for (uint32_t i = it > C::kSlots ? it - C::kSlots : 0; i < it; ++i)
                tc::mbar_wait(&ctl->full[i % C::kSlots], i / C::kSlots & 1u, limit, &none);
        } else if (warp <= 2) {
            // ---- the products of tensor tile s; the other tile's run while this warp waits and commits.  The whole warp
            // walks through, and one lane is elected for each instruction: descriptors stay in uniform registers, and 16
            // products are issued in 650 cycles (in a branch of one lane: 1,240 beside two busy softmax warps).
            constexpr uint32_t kIdescS = tc::make_idesc(kBf16, false, kQTile, kKTile), kIdescO = tc::make_idesc(kBf16, true, kQTile, D);
            constexpr uint32_t kTileStep = C::kTileBytes >> 4;
            const uint32_t one = tc::elect_one();
            const int s = warp - 1;
            const uint64_t q_desc = tc::make_desc(tc::smem_addr(smem), 16, 1024);
            const uint64_t k_desc = tc::make_desc(tc::smem_addr(ring), 16, 1024), v_desc = tc::make_desc(tc::smem_addr(ring), kKTile * 128, 1024);
            const uint32_t tm = __shfl_sync(kFull, tmem, 0), s_t = tm + kColS + s * kColStep, o_t = tm + kColO + s * kColStep;
            uint64_t *s_full = &ctl->s_full[s], *p_early = &ctl->p_early[s], *p_ready = &ctl->p_ready[s], *pv_done = &ctl->pv_done[s], *o_free = &ctl->o_free[s];
            uint32_t q_pos = 0, pos = 0, slot = 0, phase = 0, early_phase = 0, p_phase = 0, o_phase = 1, clean_phase = 0;  // pos, slot, phase: the next ring position
            uint32_t batch = 0;
            int turn = 0;  // whose the next tile of a one-tile unit is
            auto wait = [&](uint64_t* bar, uint32_t parity) { return tc::warp_wait(bar, parity, limit, abort); };
            auto advance = [&]() {
                ++pos;
                if (++slot == C::kSlots) slot = 0, phase ^= 1u;
            };
            // A position's fill.  In units of one tile this warp passes over the other's tiles, so it may look at a slot before
            // the fill ahead of its own has ended, and the parity of that older phase would let it through: it first waits
            // until its own fill is under way (which the older one's release comes before).
            auto wait_fill = [&](uint32_t at, uint32_t fill_slot, uint32_t fill_phase, bool two) {
                return (two || __all_sync(kFull, tc::wait_count(&ctl->issued, at, limit, abort))) && wait(&ctl->full[fill_slot], fill_phase);
            };
            // A slot comes free after two arrivals.  In units of two tiles warp 2, the last to use it, makes one as soon as its
            // products are in, and warpgroup 0 the other when it sees the scores that followed warp 1's; in units of one
            // tile the only user makes both.
            auto release = [&](uint64_t* bar, bool two) {
                if (!two || s == 1) tc::commit(bar, one);
                if (!two) tc::commit(bar, one);
            };
            // In units of two tiles the warps take turns with the tensor core: P V and the next Q K^T of one tile, then of the
            // other.  Left alone the two fall into step: both warpgroups in softmax, then both tiles' products, each idle
            // during the other.
            auto take_turn = [&]() { return (bool)__all_sync(kFull, tc::wait_count(&ctl->batches[s ^ 1], batch - (s ^ 1), limit, abort)); };
            auto pass_turn = [&]() {
                ++batch;
                if (one) tc::store_release(&ctl->batches[s], batch);
            };
            auto scores = [&](uint64_t a, uint32_t k_slot) {  // S = Q K^T
                const uint64_t b = k_desc + k_slot * kTileStep;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t o = (uint64_t)(((k / 4) * (kKTile * 128) + (k % 4) * 32) >> 4);
                    tc::mma_ss(s_t, a + o, b + o, kIdescS, k > 0, one);
                }
            };
            // what O += P V needs besides P: V's fill, with the slots past the length zeroed (they hold anything, and 0 * v
            // has to stay 0), and before a piece's first product the accumulator read
            auto ready = [&](uint32_t v_pos, uint32_t v_slot, uint32_t v_phase, int have, bool first, bool two) {
                if (!wait_fill(v_pos, v_slot, v_phase, two)) return false;
                if ((have & 15) != 0 && have < kKTile) {  // the rows that the last 16 of V take in
                    if (!two || s == 0) {
                        unsigned char* v = ring + v_slot * C::kTileBytes;
                        for (int r = have + (lane >> 3); r < ((have + 15) & ~15); r += 4)
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                *reinterpret_cast<uint4*>(v + h * (kKTile * 128) + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                        tc::fence_async_shared();
                        __syncwarp();
                        if (two && one) tc::mbar_arrive(&ctl->clean);
                    } else {
                        if (!wait(&ctl->clean, clean_phase)) return false;
                        clean_phase ^= 1u;
                    }
                }
                if (first) {
                    if (!wait(o_free, o_phase)) return false;
                    o_phase ^= 1u;
                }
                return true;
            };
            auto values = [&](uint32_t v_slot, int have, bool first, auto early) {  // O += P V, of the tile's first tokens or of the rest
                constexpr bool kFirst = decltype(early)::value;
                constexpr int kFrom = kFirst ? 0 : kEarly / 16, kTo = kFirst ? kEarly / 16 : kKTile / 16;
                const uint64_t b = v_desc + v_slot * kTileStep;
                if (have > kTo * 16 - 16) {
#pragma unroll
                    for (int k = kFrom; k < kTo; ++k) tc::mma_ts(o_t, s_t + k * 8, b + (uint64_t)(k * 2048 >> 4), kIdescO, k > 0 || !first, one);
                } else {
#pragma unroll 1
                    for (int k = kFrom; k < (have + 15) >> 4; ++k) tc::mma_ts(o_t, s_t + k * 8, b + (uint64_t)(k * 2048 >> 4), kIdescO, k > 0 || !first, one);
                }
            };
            while (ok && next_piece()) {
                const int tiles = __shfl_sync(kFull, x.tiles, 0);
                const bool two = __shfl_sync(kFull, x.rows, 0) > p.rows_per_tile;
                // Both warps see every fill of every query buffer and both free it, used or not: neither gets a phase ahead.
                const uint32_t q = q_pos + (two ? s : 0);
                ok = wait(&ctl->q_full[q_pos & 1u], q_pos >> 1 & 1u) && (!two || wait(&ctl->q_full[(q_pos + 1) & 1u], (q_pos + 1) >> 1 & 1u));
                const uint64_t a = q_desc + (q & 1u) * kTileStep;
                int left = __shfl_sync(kFull, x.left, 0);
                if (two) {
                    uint32_t k_slot = slot;
                    ok = ok && wait_fill(pos, slot, phase, true) && take_turn();
                    if (ok) {
                        tc::fence_after();
                        scores(a, k_slot);
                        pass_turn();
                        tc::commit(s_full, one);
                        release(&ctl->empty[k_slot], true);
                    }
                    for (int i = 0; ok && i < tiles; ++i, left -= kKTile) {
                        advance();
                        const uint32_t v_pos = pos, v_slot = slot, v_phase = phase;
                        advance();
                        const bool last = i + 1 == tiles;
                        k_slot = slot;
                        ok = ready(v_pos, v_slot, v_phase, left, i == 0, true) && (last || wait_fill(pos, slot, phase, true)) &&
                             wait(p_early, early_phase) && take_turn();
                        early_phase ^= 1u;
                        if (!ok) break;
                        tc::fence_after();
                        values(v_slot, left, i == 0, std::true_type());
                        ok = wait(p_ready, p_phase);
                        p_phase ^= 1u;
                        if (!ok) break;
                        tc::fence_after();
                        values(v_slot, left, i == 0, std::false_type());
                        // P V and the next Q K^T without a pause
                        if (!last) scores(a, k_slot);
                        pass_turn();
                        tc::commit(last ? pv_done : s_full, one);
                        release(&ctl->empty[v_slot], true);
                        if (!last) release(&ctl->empty[k_slot], true);
                    }
                } else {
                    // every other tile is this warp's
                    const uint32_t base = pos;
                    const int mine = turn == s ? 0 : 1;
                    auto score = [&](int t) {
                        const uint32_t at = base + 2 * t, k_slot = at % C::kSlots;
                        if (!wait_fill(at, k_slot, at / C::kSlots & 1u, false)) return false;
                        tc::fence_after();
                        scores(a, k_slot);
                        tc::commit(s_full, one);
                        release(&ctl->empty[k_slot], false);
                        return true;
                    };
                    if (mine < tiles) ok = ok && score(mine);
                    for (int t = mine; ok && t < tiles; t += 2) {
                        const uint32_t v_pos = base + 2 * t + 1, v_slot = v_pos % C::kSlots;
                        const int have = left - t * kKTile;
                        ok = ready(v_pos, v_slot, v_pos / C::kSlots & 1u, have, t == mine, false) && wait(p_early, early_phase);
                        early_phase ^= 1u;
                        if (!ok) break;
                        tc::fence_after();
                        values(v_slot, have, t == mine, std::true_type());
                        ok = wait(p_ready, p_phase);
                        p_phase ^= 1u;
                        if (!ok) break;
                        tc::fence_after();
                        values(v_slot, have, t == mine, std::false_type());
                        const bool last = t + 2 >= tiles;
                        if (last) tc::commit(pv_done, one);
                        release(&ctl->empty[v_slot], false);
                        if (!last) ok = score(t + 2);
                    }
                    pos = base + 2 * tiles;
                    slot = pos % C::kSlots, phase = pos / C::kSlots & 1u;
                }
                if (!two) turn ^= tiles & 1;
                if (ok) {
                    tc::commit(&ctl->q_free[q & 1u], one);
                    if (two && one) tc::mbar_arrive(&ctl->q_free[(q + 1) & 1u]);
                }
                q_pos += two ? 2 : 1;
            }
            int none = 0;  // no product outlives the block
            tc::commit(&ctl->drain, one);
            tc::mbar_wait(&ctl->drain, 0, limit, &none);
            __syncwarp();
        } else {
            // ---- the queries of one-tile units, ahead of the products
            uint32_t q_pos = 0;
            while (ok && next_piece()) {
                // this warp sees every buffer come free, in order; the softmax warpgroups load the tiles of two-tile units themselves
                const bool two = x.rows > p.rows_per_tile;
                for (int j = 0; ok && j <= (two ? 1 : 0); ++j)
                    ok = tc::warp_wait(&ctl->q_free[(q_pos + j) & 1u], ((q_pos + j) >> 1 & 1u) ^ 1u, limit, abort);
                if (!ok) break;
                if (two) {
                    if (lane == 0) tc::mbar_arrive(&ctl->q_grant);
                    q_pos += 2;
                    continue;
                }
                const uint32_t b = q_pos & 1u;
                load_queries<T, D>(p, x.row, x.rows, x.kvh, tc::smem_addr(smem + b * C::kTileBytes), second_at(x.rows * p.share), lane, 32);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->q_full[b], 4);
                ++q_pos;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        p.sc.gave_up[blockIdx.x] = *abort;
        if (*abort != 0) atomicOr(p.status, kStatusAttnTimeout);
    }
    if (warp == 2) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- the join
//
// A warp has four query heads of a row, eight threads each: a thread holds
// D / 8 lanes of its head, as D / 64 runs of eight.  What it reads (keys and
// values of the round's own tokens, then parts) comes by asynchronous copies
// into shared memory, several at a time, and is taken up by short loops: a
// call's join runs once through its code, and unrolled loads and sums are bound
// by the fetch of their instructions (188 rows of 40 heads: 74.5 us against 67
// for the whole call).  Neighbouring threads have neighbouring heads, which lie
// side by side in a part: a copy writes shared memory by runs that are
// contiguous on both sides, and with a head's threads side by side took 31
// writes per instruction (one row at 4,095 tokens: 19.2 us against 15.6).
template <int D>
struct Acc {
    static constexpr int kE = D / 8;
    float o[kE], m, l;  // in base 2
    __device__ __forceinline__ void add(float s, float w, const float (&v)[kE]) {  // a part: maximum s, sum w, result v
        const float top = fmaxf(m, s), base = top == kNegInf ? 0.0f : top;
        const float f = ex2(m - base), g = ex2(s - base);
        l = l * f + w * g;
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = o[e] * f + g * v[e];
        m = top;
    }
};

template <bool kBf16>
__device__ __forceinline__ void widen8(const uint4& w, float* x) {
    using H = Half<kBf16>;
    const float2 a = H::unpack(w.x), b = H::unpack(w.y), c = H::unpack(w.z), d = H::unpack(w.w);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y, x[4] = c.x, x[5] = c.y, x[6] = d.x, x[7] = d.y;
}

// The parts of a row's head from one segment: what the call's arguments say,
// and after the main kernel what its tables say.
struct Parts {
    int seg, unit, dealt;     // seg: -1 for none; of all heads' units
    int row, cap, set, sets;  // row of the unit; the parts of a piece that are its: sets of them from `set` on
    int count;
    long long slot;
    __device__ __forceinline__ void find(const AttendParams& p, int segment, int of, int head) {  // of: the row
        seg = -1;
        if (segment < 0) return;
        const Seg s = load_seg(p, segment);
        if (s.tiles == 0) return;
        seg = segment;
        const int rt = p.rows_per_tile, rel = of - s.r0, u = rel / (2 * rt), in = rel - u * 2 * rt, kvh = head / p.share;
        const bool two = s.n - u * 2 * rt > rt;
        unit = kvh * s.units + u;
        dealt = s.dealt;
        set = two && in >= rt ? 1 : 0;
        sets = two ? 1 : 2;  // a unit of one tile: a part of each warpgroup
        row = (in - set * rt) * p.share + head - kvh * p.share;
        cap = segment < p.P ? kQTile : p.sc.group_rows;
    }
    __device__ __forceinline__ int2 first_slots(const AttendParams& p) const { return seg >= 0 ? p.sc.seg_units[seg] : make_int2(0, 0); }
    __device__ __forceinline__ void locate(const AttendParams& p, int2 base) {
        slot = (long long)base.y + unit;
        int pieces = seg >= 0 ? 1 : 0;
        if (pieces != 0 && unit >= dealt) {
            const long long at = unit_index(p, seg < p.P, base.x + unit - dealt);
            const int2 e = at >= 0 ? p.sc.units[at] : make_int2(0, 0);
            slot = e.x;
            pieces = entry_pieces(e.x, e.y, seg < p.P ? p.sc.prefix_slots : p.sc.group_slots, p.grid);
        }
        count = pieces * sets;
    }
    __device__ __forceinline__ long long part(const AttendParams& p, int k) const {
        return part_row(p, seg < p.P, slot + (sets == 1 ? k : k >> 1), sets == 1 ? set : k & 1);
    }
};

// Tokens or parts on their way to a thread at a time.
__host__ __device__ constexpr int join_round(int sub) { return sub > 2 ? 6 : 3; }
__host__ __device__ constexpr int join_blocks(int sub) { return sub > 2 ? 2 : 4; }  // per SM
template <int D>
constexpr int join_bytes(int sub) { return join_round(sub) * kJoinThreads * (D / 32 * 16 + 8); }

// kSub warps per row and four heads: the round's own tokens that the row sees,
// then the parts of the row's prefix and of its group's committed tokens.
//
// What comes before the wait reads only what kernels ahead of the main one
// wrote (queries, lengths, tables, masks, the caches), and may: this kernel
// starts once every block of the main kernel has let it, which each does after
// its own wait for those kernels' end.  Parts and tables of the scratch are the
// main kernel's own and are read after the wait for it.
//
// With heads of 128 the forms of one and two warps per row spill 28 bytes a
// thread (F16: 36) at the 64 registers that four blocks per SM leave.
template <bool kBf16, int D, int kSub>
__global__ void __launch_bounds__(kJoinThreads, join_blocks(kSub)) lp_attend_join_kernel(const AttendParams p) {
    using H = Half<kBf16>;
    using T = typename H::T;
    constexpr int kE = D / 8, kRuns = D / 64, kRound = join_round(kSub);
    // what is on its way to a warp, 16 bytes of every thread side by side
    extern __shared__ __align__(16) unsigned char smem[];
    uint4* stage = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    float2* stage_ml = reinterpret_cast<float2*>(smem + kRound * 2 * kRuns * kJoinThreads * 16) + threadIdx.x;
    auto place = [](int h, int c) { return h * 8 + (c ^ 2 * h); };
    auto staged = [&](int b, int c) -> uint4& { return stage[(b * 2 * kRuns + c) * kJoinThreads]; };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kSub, l = lane >> 2;
    const int row = blockIdx.x, head = (blockIdx.y * (kJoinWarps / kSub) + warp / kSub) * 4 + (lane & 3);
    __shared__ int served_by;  // the prefix of the row
    if (threadIdx.x == 0) served_by = p.P;
    const int g = block_group_of(p.indptr, p.G, row);  // (a barrier)
    const bool mine = g >= 0;
    const bool exists = mine && head < p.q_heads;
    Group grp = {0, 0, 0, false};
    if (mine) grp = load_group(p, g);
    Acc<D> a;
#pragma unroll
    for (int e = 0; e < kE; ++e) a.o[e] = 0.0f;
    a.m = kNegInf, a.l = 0.0f;
    if (grp.n > 0) {
        float q[kE];
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
            widen8<kBf16>(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.q) + row * p.q_stride +
                                                          (long long)(exists ? head : 0) * D + r * 64 + l * 8), q + r * 8);
        const float c = p.scale * kLog2e;
        const int j = row - grp.r0;
        const unsigned mask = p.row_masks != nullptr ? p.row_masks[row] : (2u << j) - 1u;
        int page = 0;  // lane i: of token i
        if (lane < grp.n) page = p.tables[(long long)g * p.max_pages + ((grp.len + lane) >> p.page_shift)];
        const unsigned here = __ballot_sync(kFull, page >= 0 && page < p.num_pages);
        unsigned todo = mask & (grp.n < 32 ? (1u << grp.n) - 1u : kFull);
        if (lane == 0 && (todo & ~here) != 0u) atomicOr(p.status, kStatusBadPage);
        if (kSub > 1) todo &= kFull / ((1u << kSub) - 1u) << sub;  // every kSub-th is this warp's
        const int n = __popc(todo);
        // Keys and values lie side by side along a head, so here neighbouring threads copy along a head (to the places of the
        // threads that read them, turned so that a read meets every bank once).
        const int copy_head = head - (lane & 3) + (lane >> 3), copy_kvh = copy_head < p.q_heads ? copy_head / p.share : 0;
        const int copy_to = place(lane >> 3, lane & 7) - lane, read_at = place(lane & 3, l) - lane;
#pragma unroll 1
        for (int j = 0, slot = 0; j < n + kRound - 1; ++j) {
            __syncwarp();
            if (j < n) {
                const int i = __ffs(todo) - 1, t = grp.len + i;
                todo &= todo - 1u;
                const long long pg = __shfl_sync(kFull, page, i);
                const long long at = ((((pg * p.kv_heads + copy_kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1))) * D) + (lane & 7) * 8;
#pragma unroll
                for (int r = 0; r < kRuns; ++r) {
                    if (here >> i & 1u) {
                        tc::copy16(tc::smem_addr(&staged(slot, r) + copy_to), reinterpret_cast<const T*>(p.k_cache) + at + r * 64);
                        tc::copy16(tc::smem_addr(&staged(slot, kRuns + r) + copy_to), reinterpret_cast<const T*>(p.v_cache) + at + r * 64);
                    } else {
                        (&staged(slot, r))[copy_to] = (&staged(slot, kRuns + r))[copy_to] = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            tc::copies_commit();
            slot = slot == kRound - 1 ? 0 : slot + 1;
            if (j < kRound - 1) continue;
            tc::copies_wait<kRound - 1>();  // slot: of the oldest
            __syncwarp();
            float k[kE], v[kE];
#pragma unroll
            for (int r = 0; r < kRuns; ++r) widen8<kBf16>((&staged(slot, r))[read_at], k + r * 8), widen8<kBf16>((&staged(slot, kRuns + r))[read_at], v + r * 8);
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
            for (int o = 16; o > 2; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            a.add(s * c, 1.0f, v);
        }
    }
    // Of the first prefix that serves the row, of its group's committed tokens.  A prefix has parts for the rows from its first
    // group's to its last's: a group whose rows lie elsewhere (group_indptr then does not ascend) is not served.
    Parts shared, own;
    if (p.P > 0 && grp.n > 0) {  // the same for the block, whose threads look through the prefixes side by side
        for (int i = threadIdx.x; i < p.P; i += kJoinThreads) {
            if (p.prefix_indptr[i] > g || p.prefix_indptr[i + 1] <= g) continue;
            const Prefix x = load_prefix(p, i);
            if (!x.bad && grp.r0 >= x.r0 && grp.r0 + grp.n <= x.r0 + x.n) {
                atomicMin(&served_by, i);
                break;
            }
        }
        __syncthreads();
    }
    shared.find(p, grp.n > 0 && served_by < p.P ? served_by : -1, row, exists ? head : 0);
    own.find(p, grp.n > 0 ? p.P + g : -1, row, exists ? head : 0);
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // A block's waits ran out: it left its entries and parts as they were, and no row has a result.  With few blocks the
    // answer is put together at the end, when the loads have long come in (one row: 15.3 us; here: 15.6); with many it costs
    // nothing here.
    int gave_up = 0;
    for (int b = threadIdx.x; b < p.grid; b += kJoinThreads) gave_up |= p.sc.gave_up[b];
    const int2 shared_at = shared.first_slots(p), own_at = own.first_slots(p);
    if constexpr (kSub == 1) gave_up = __syncthreads_or(gave_up);
    shared.locate(p, shared_at);
    own.locate(p, own_at);
    const int count = shared.count + own.count, n = count > sub ? (count - sub + kSub - 1) / kSub : 0;
#pragma unroll 1
    for (int j = 0, slot = 0; j < n + kRound - 1; ++j) {
        if (j < n) {
            const int k = sub + j * kSub;
            const bool is_own = k >= shared.count;
            const int row_at = is_own ? own.row : shared.row, cap = is_own ? own.cap : shared.cap;
            const long long base = is_own ? own.part(p, k - shared.count) : shared.part(p, k);
            if (base < 0) {
                stage_ml[slot * kJoinThreads] = make_float2(kNegInf, 0.0f);
            } else {
                tc::copy8(tc::smem_addr(&stage_ml[slot * kJoinThreads]), p.sc.part_ml + base + row_at);
                const float4* src = reinterpret_cast<const float4*>(p.sc.part_o) + part_chunk<D>(base, cap, row_at, 2 * l);
#pragma unroll
                for (int r = 0; r < kRuns * 2; ++r) tc::copy16(tc::smem_addr(&staged(slot, r)), src + (r / 2 * 16 + (r & 1)) * cap);
            }
        }
        tc::copies_commit();
        slot = slot == kRound - 1 ? 0 : slot + 1;
        if (j < kRound - 1) continue;
        tc::copies_wait<kRound - 1>();
        const float2 ml = stage_ml[slot * kJoinThreads];
        if (ml.x == kNegInf && ml.y == 0.0f) continue;  // nothing was written
        float v[kE];
#pragma unroll
        for (int r = 0; r < kRuns * 2; ++r) {
            const uint4 w = staged(slot, r);
            v[4 * r] = __uint_as_float(w.x), v[4 * r + 1] = __uint_as_float(w.y), v[4 * r + 2] = __uint_as_float(w.z), v[4 * r + 3] = __uint_as_float(w.w);
        }
        a.add(ml.x, ml.y, v);
    }
    if constexpr (kSub > 1) {  // the warps' sums, in the order of the warps
        float* part = reinterpret_cast<float*>(smem);  // [e][thread]; then the maxima and sums
        float2* part_ml = reinterpret_cast<float2*>(part + kE * kJoinThreads);
        gave_up = __syncthreads_or(gave_up);
#pragma unroll
        for (int e = 0; e < kE; ++e) part[e * kJoinThreads + threadIdx.x] = a.o[e];
        part_ml[threadIdx.x] = make_float2(a.m, a.l);
        __syncthreads();
        if (sub != 0) return;
#pragma unroll 1
        for (int w = 1; w < kSub; ++w) {
            const float2 ml = part_ml[threadIdx.x + w * 32];
            float v[kE];
#pragma unroll
            for (int e = 0; e < kE; ++e) v[e] = part[e * kJoinThreads + threadIdx.x + w * 32];
            if (ml.x != kNegInf || ml.y != 0.0f) a.add(ml.x, ml.y, v);
        }
    }
    if (!exists) return;
    if (gave_up != 0) {
#pragma unroll
        for (int e = 0; e < kE; ++e) a.o[e] = 0.0f;
        a.m = kNegInf, a.l = 0.0f;
    }
    const float inv = a.l > 0.0f ? 1.0f / a.l : (a.l == 0.0f ? 0.0f : a.l);
    T* dst = reinterpret_cast<T*>(p.out) + row * p.out_stride + (long long)head * D + l * 8;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
        uint4 w;
        w.x = H::pack(a.o[r * 8] * inv, a.o[r * 8 + 1] * inv);
        w.y = H::pack(a.o[r * 8 + 2] * inv, a.o[r * 8 + 3] * inv);
        w.z = H::pack(a.o[r * 8 + 4] * inv, a.o[r * 8 + 5] * inv);
        w.w = H::pack(a.o[r * 8 + 6] * inv, a.o[r * 8 + 7] * inv);
        *reinterpret_cast<uint4*>(dst + r * 64) = w;
    }
    if (p.lse_out != nullptr && l == 0) p.lse_out[(long long)row * p.q_heads + head] = a.l == 0.0f ? kNegInf : a.m * kLn2 + logf(a.l);
}

template <int D>
constexpr int smem_bytes() { return Cfg<D>::kCtl + (int)sizeof(Ctl); }

template <bool kBf16, int D>
cudaError_t prepare() {
    static_assert(smem_bytes<D>() <= 232448, "shared memory");
    const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(lp_attend_kernel<kBf16, D>, most, smem_bytes<D>());
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 8>, most, join_bytes<D>(8));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 4>, most, join_bytes<D>(4));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 2>, most, join_bytes<D>(2));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 1>, most, join_bytes<D>(1));
    return e;
}

template <bool kBf16, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
    // Both kernels are launched while the one before still runs, and wait for its end before they read what it writes.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.grid);
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = smem_bytes<D>();
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, lp_attend_kernel<kBf16, D>, p, k_map, v_map);
    if (e != cudaSuccess) return e;
    // the most warps per row with which all blocks are resident at once: one row takes 15.5 us (one warp: 24.7), trees of
    // drafts 43.6 (one: 46.3, eight: 60), 2,048 rows behind a prefix 765 (eight: 1,015)
    const int chunks = (p.q_heads + 3) / 4;
    int sub = 8;
    auto per_row = [&]() { return (chunks * sub + kJoinWarps - 1) / kJoinWarps; };  // blocks
    while (sub > 1 && per_row() * (long long)p.rows > join_blocks(sub) * p.grid) sub /= 2;
    lc.gridDim = dim3((unsigned)p.rows, (unsigned)per_row());
    lc.blockDim = dim3(kJoinThreads);
    lc.dynamicSmemBytes = join_bytes<D>(sub);
    if (sub == 8) return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 8>, p);
    if (sub == 4) return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 4>, p);
    if (sub == 2) return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 2>, p);
    return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 1>, p);
}

}  // namespace

cudaError_t prepare_attend(int dtype, int head_dim) {
    if (dtype == 1) return head_dim == 128 ? prepare<true, 128>() : prepare<true, 64>();
    return head_dim == 128 ? prepare<false, 128>() : prepare<false, 64>();
}

cudaError_t launch_attend(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, int dtype, int head_dim,
                          cudaStream_t stream) {
    if (dtype == 1) return head_dim == 128 ? launch<true, 128>(p, k_map, v_map, stream) : launch<true, 64>(p, k_map, v_map, stream);
    return head_dim == 128 ? launch<false, 128>(p, k_map, v_map, stream) : launch<false, 64>(p, k_map, v_map, stream);
}

}  // namespace lp
