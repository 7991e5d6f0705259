// lp_split.h -- how an attention call's work is cut: its segments, their units,
// and the run of token tiles that each block takes.
//
// A segment is a prefix or a group's committed tokens.  Its query rows, with the
// heads that share a key-value head, form units; a unit's tokens form tiles of
// 128.  A rule says how many rows a unit has, what a tile of it costs, and how
// many parts a piece of it leaves for the join.
#pragma once

#include "lp_attn.h"

namespace lp {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kThreads = 384;  // of a block that sum up its plan (it may have more)
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// m 2^e, 1 <= m < 2, with e kept to FP32's normal numbers: finite and above 0, so that as a factor it leaves a masked
// score at -infinity and one of 0 at 0.
__device__ __forceinline__ float scaled(float m, int e) {
    e = e < -126 ? -126 : (e > 127 ? 127 : e);
    return m * __uint_as_float((uint32_t)(e + 127) << 23);
}

// The exponent of a positive normal number.
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// Units of up to two tiles of 128 query rows: a piece leaves a part for each
// tile, or for each warpgroup where the unit is one tile.  What a run is
// measured in, by the times of each: a token tile of a one-tile unit is 2, of a
// two-tile unit 3, and every unit 4 more (its queries, first loads and results).
struct Pairs {
    static constexpr bool kPairs = true;
    static constexpr int kSets = 2, kTileCost = 2, kPairCost = 3, kUnitCost = 4;
    static constexpr int kMostCost = kPairCost;  // of a tile
    static constexpr int kPrefixRows = kQTile;   // of a part of a prefix
    static __device__ __forceinline__ int unit_rows(const AttendParams& p) { return 2 * p.rows_per_tile; }
    static __device__ __forceinline__ int cost(const AttendParams& p, int n) { return n > p.rows_per_tile ? kPairCost : kTileCost; }
    static __device__ __forceinline__ const AttendScratch& scratch(const AttendParams& p) { return p.sc; }
    static __device__ __forceinline__ bool takes(const AttendParams&, bool) { return true; }
};

// The same for a cache in 4 bits, of the segments that they are chosen for.
struct Pairs4 : Pairs {
    static __device__ __forceinline__ bool takes(const AttendParams& p, bool prefix) { return (p.wide & (prefix ? kWidePrefixes : kWideGroups)) != 0; }
};

// Units of at most kUnitRows query rows, one or two fragments of 16, for calls with
// as few heads for a key-value head: a piece leaves one part.  A token tile of one
// fragment costs 2, of two 4, or 3 where both share a worker's codes (D = 64), and
// every unit 5 more.
struct Fragments {
    static constexpr bool kPairs = false;
    static constexpr int kSets = 1, kUnitCost = 5, kTileCost = 2, kMostCost = 4, kPrefixRows = kUnitRows;
    static __device__ __forceinline__ int unit_rows(const AttendParams& p) { return p.rows_per_unit; }
    static __device__ __forceinline__ int cost(const AttendParams& p, int n) {
        return (n < p.rows_per_unit ? n : p.rows_per_unit) * p.share > 16 ? p.two_cost : kTileCost;
    }
    static __device__ __forceinline__ const AttendScratch& scratch(const AttendParams& p) { return p.fragments; }
    static __device__ __forceinline__ bool takes(const AttendParams& p, bool prefix) { return !Pairs4::takes(p, prefix); }
};

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
template <class Rule>
struct Seg {
    int r0, n, len;
    int tiles, units;  // token tiles; units per key-value head; tiles = 0: no work
    int dealt;         // of all heads' units, those that go round the blocks whole
    bool bad;
    __device__ __forceinline__ int left(const AttendParams& p) const { return tiles > 0 ? units * p.kv_heads - dealt : 0; }
    int cost;          // of a token tile
    __device__ __forceinline__ long long span() const { return (long long)tiles * cost + Rule::kUnitCost; }  // of a unit in a run
    __device__ __forceinline__ unsigned long long work(const AttendParams& p) const { return (unsigned long long)(span() * left(p)); }
};

template <class Rule>
__device__ __forceinline__ Seg<Rule> load_seg(const AttendParams& p, int s) {
    Seg<Rule> x;
    if (s < p.P) {
        const Prefix f = load_prefix(p, s);
        x.r0 = f.r0, x.n = f.n, x.len = f.len, x.bad = f.bad;
    } else {
        const Group f = load_group(p, s - p.P);
        x.r0 = f.r0, x.n = f.n, x.len = f.len, x.bad = f.bad;
    }
    x.units = (x.n + Rule::unit_rows(p) - 1) / Rule::unit_rows(p);
    x.tiles = x.n > 0 && Rule::takes(p, s < p.P) ? (x.len + kKTile - 1) / kKTile : 0;
    x.cost = Rule::cost(p, x.n);
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

// `cost`: the most that a tile costs.  No run is shorter than that (it then holds
// the start of a tile, wherever it lies among a unit's), nor one of prefixes than
// four times that (every run of a unit leaves a part for the join to read).
__device__ __forceinline__ Runs make_runs(unsigned long long total, int grid, int kind, int cost) {
    Runs r;
    r.total = total;
    const unsigned long long most = Runs::quotient(total, kind == 0 ? 4 * cost : cost);
    r.blocks = most < (unsigned long long)grid ? (int)most : grid;
    if (r.blocks == 0 && total > 0) r.blocks = 1;
    r.per = r.blocks > 0 ? Runs::quotient(total, r.blocks) : 0;
    r.more = (int)(total - r.per * r.blocks);
    return r;
}

// Index of row 0 of a piece's part (tile or warpgroup `set`); -1: past the
// scratch (only overlapping prefixes can ask for that).
template <class Rule>
__device__ __forceinline__ long long part_row(const AttendParams& p, bool prefix, long long slot, int set) {
    const AttendScratch& sc = Rule::scratch(p);
    if (prefix) return slot < sc.prefix_slots ? (slot * Rule::kSets + set) * Rule::kPrefixRows : -1;
    if (slot >= sc.group_slots) return -1;
    return sc.prefix_slots * Rule::kSets * Rule::kPrefixRows + (slot * Rule::kSets + set) * sc.group_rows;
}

// Where a unit that is not dealt out is entered for the join; -1 as above.
__device__ __forceinline__ long long unit_index(const AttendScratch& sc, bool prefix, int unit) {
    if (prefix) return unit < sc.prefix_slots ? unit : -1;
    return unit < sc.group_slots ? sc.prefix_slots + unit : -1;
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
template <class Rule>
struct Start {
    unsigned long long off;
    int seg, units;
    Seg<Rule> s;
};

// Walks a block's pieces: its share of the units that go round whole, then its
// run of the other prefix units' tiles, then of the groups'.
template <class Rule>
struct Walk {
    Runs runs[2], run;                 // of prefixes, of groups; the current
    unsigned long long begin[2], finish[2];  // this block's
    const Start<Rule>* start;
    int kind;
    int deal, deal_end, round, dealt;  // segments with units that go round; rounds dealt; units of earlier segments
    unsigned long long pos, end, off;  // off: tiles before the segment
    int seg, units, cta;               // units: the segment's first slot less cta
    Seg<Rule> s;
    __device__ __forceinline__ void enter(int k) {
        kind = k;
        run = runs[k];
        pos = begin[k], end = finish[k];
        off = start[k].off, seg = start[k].seg, units = start[k].units, s = start[k].s;
    }
    const int* table;                  // pages of the piece, and its first token
    long long token;
    __device__ __forceinline__ void fill(const AttendParams& p, Piece& x, int sg, const Seg<Rule>& y, int unit, int t0, int tiles, long long slot) {
        const bool prefix = sg < p.P;
        x.tiles = tiles;
        x.kvh = unit / y.units;
        const int first = (unit - x.kvh * y.units) * Rule::unit_rows(p);
        x.row = y.r0 + first;
        x.rows = y.n - first < Rule::unit_rows(p) ? y.n - first : Rule::unit_rows(p);
        x.left = y.len - t0 * kKTile;
        table = prefix ? p.prefix_tables + (long long)sg * p.max_prefix_pages : p.tables + (long long)(sg - p.P) * p.max_pages;
        token = (long long)t0 * kKTile;
        x.part = part_row<Rule>(p, prefix, slot, 0);
        x.part_stride = prefix ? Rule::kPrefixRows : Rule::scratch(p).group_rows;
    }
    __device__ __forceinline__ bool next(const AttendParams& p, Piece& x) {
        while (deal < deal_end) {
            const Seg<Rule> y = load_seg<Rule>(p, deal);
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
                s = load_seg<Rule>(p, ++seg);
                continue;
            }
            // the unit's cost lies before its tiles, and a tile belongs to the run that its start lies in
            const unsigned long long rel = pos - off, rest = end - pos, span = s.span();
            const int unit = (int)Runs::quotient(rel, span);
            const long long u0 = (long long)(rel - unit * span), u1 = rest < span - u0 ? u0 + (long long)rest : (long long)span;
            pos += u1 - u0;
            const int t0 = u0 > Rule::kUnitCost ? (int)((u0 - Rule::kUnitCost + s.cost - 1) / s.cost) : 0;
            const int t1 = u1 > Rule::kUnitCost ? (int)((u1 - Rule::kUnitCost + s.cost - 1) / s.cost) : 0;
            if (t1 <= t0) continue;
            fill(p, x, seg, s, s.dealt + unit, t0, t1 - t0, (long long)units + unit + cta);
            if (t0 == 0 && (threadIdx.x & 31) == 0) {
                // for the join: the unit's first slot and how many blocks have a piece of it
                const unsigned long long last = off + unit * span + Rule::kUnitCost + (unsigned long long)(s.tiles - 1) * s.cost;
                const long long at = unit_index(Rule::scratch(p), kind == 0, units + unit);
                if (at >= 0) Rule::scratch(p).units[at] = make_int2(units + unit + cta, t1 == s.tiles ? 1 : run.block_of(last) - cta + 1);
            }
            return true;
        }
        x.rows = 0;
        return false;
    }
};

// A block's shared part of the plan.
template <class Rule>
struct PlanCtl {
    unsigned long long sum[kWarps][3];
    int sum_dealt[kWarps], deal_first, deal_last;
    Start<Rule> start[2];
};

// The call's tiles and units: every thread sums its share of the segments,
// the block scans the sums, and the thread that holds the block's first tile
// names its segment.  Block 0 leaves the offsets for the join.  False: the
// block has no work.
template <class Rule>
__device__ __forceinline__ bool plan_run(const AttendParams& p, PlanCtl<Rule>* ctl, Runs (&runs)[2]) {
    const int S = p.P + p.G, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per < S ? tid * per : S, s1 = s0 + per < S ? s0 + per : S;
    // of prefixes and of groups; units: slots of units that do not go round, of prefixes in the high half
    unsigned long long cost0 = 0, cost1 = 0, units = 0;
    int dealt = 0, first = S, last = -1;
    for (int s = s0; s < s1; ++s) {
        const Seg<Rule> x = load_seg<Rule>(p, s);
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
    if (lane == 31 && warp < kWarps) ctl->sum[warp][0] = i0, ctl->sum[warp][1] = i1, ctl->sum[warp][2] = iu, ctl->sum_dealt[warp] = id;
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
    runs[0] = make_runs(total0, gridDim.x, 0, Rule::kMostCost);
    runs[1] = make_runs(total1, gridDim.x, 1, Rule::kMostCost);
    const int cta = blockIdx.x;
    const unsigned long long lo0 = cta < runs[0].blocks ? runs[0].start(cta) : ~0ull, lo1 = cta < runs[1].blocks ? runs[1].start(cta) : ~0ull;
    if (cta == 0 || (lo0 >= at0 && lo0 < at0 + cost0) || (lo1 >= at1 && lo1 < at1 + cost1)) {
        for (int s = s0; s < s1; ++s) {
            const Seg<Rule> x = load_seg<Rule>(p, s);
            const int kind = s < p.P ? 0 : 1;
            const unsigned long long work = x.work(p), off = kind == 0 ? at0 : at1, lo = kind == 0 ? lo0 : lo1;
            const int before = (int)(kind == 0 ? (u >> 32) + all_dealt : u & 0xFFFFFFFFull);  // slots: the dealt units', then the others'
            if (cta == 0) Rule::scratch(p).seg_units[s] = make_int2(before, d);
            if (lo >= off && lo < off + work) ctl->start[kind].off = off, ctl->start[kind].seg = s, ctl->start[kind].units = before, ctl->start[kind].s = x;
            (kind == 0 ? at0 : at1) += work;
            u += (unsigned long long)x.left(p) << (kind == 0 ? 32 : 0);
            d += x.dealt;
        }
    }
    return all_dealt > 0 || cta < runs[0].blocks || cta < runs[1].blocks;
}

}  // namespace lp
