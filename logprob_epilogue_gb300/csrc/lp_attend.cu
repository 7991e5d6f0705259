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
// 128.  All token tiles of the call, unit after unit, are cut into one equal
// run per block, wherever that falls: one request at a long context and
// hundreds of short ones fill the machine alike, and no block waits on
// another.  A unit of two query tiles reads each K and V tile once for both; a
// unit of one tile gives its even token tiles to one warpgroup and its odd ones
// to the other, each with its own maximum, sum and accumulator.
//
// Block: warp 0 fetches pages by TMA into a ring, warp 1 issues the MMAs,
// warps 4-7 and 8-11 are two softmax warpgroups, one row per thread.
//   S_i = Q_i K^T    128 x 128, shared x shared -> tensor memory
//   softmax: S_i to registers, P_i (the plan's type) back over S_i
//   O_i += P_i V     tensor memory x shared -> tensor memory
// While one warpgroup works on its S the tensor core runs the other's
// products.  The running maximum moves only when it grows by more than 2^8
// (then O and the sum are rescaled), so most tiles touch O not at all.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
constexpr float kRescale = 8.0f;  // growth of the maximum (log2) that moves it

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

// One verify group: its rows and committed tokens.  n = 0: idle or malformed.
struct Group {
    int r0, n, len;
    bool bad;
};

__device__ __forceinline__ Group load_group(const AttendParams& p, int g) {
    Group x;
    const int r0 = __ldg(&p.indptr[g]), r1 = __ldg(&p.indptr[g + 1]);
    x.r0 = r0;
    x.len = __ldg(&p.lens[g]);
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
    x.g0 = __ldg(&p.prefix_indptr[i]);
    x.g1 = __ldg(&p.prefix_indptr[i + 1]);
    x.len = __ldg(&p.prefix_lens[i]);
    x.bad = x.g0 < 0 || x.g1 < x.g0 || x.g1 > p.G || x.len < 0 ||
            (long long)x.len > ((long long)p.max_prefix_pages << p.page_shift);
    x.r0 = x.n = 0;
    if (!x.bad) {
        const int r0 = __ldg(&p.indptr[x.g0]), r1 = __ldg(&p.indptr[x.g1]);
        x.bad = r0 < 0 || r1 < r0 || r1 > p.rows;
        if (!x.bad) x.r0 = r0, x.n = r1 - r0;
    }
    return x;
}

// Segment s: prefixes 0..P-1, then the groups' committed tokens.
struct Seg {
    int r0, n, len;
    int tiles, units;  // token tiles, units per key-value head; tiles = 0: no work
    bool bad;
    __device__ __forceinline__ unsigned long long work(const AttendParams& p) const {
        return (unsigned long long)tiles * units * p.kv_heads;
    }
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
    return x;
}

// First tile of block c's run of `total` tiles over n blocks.
__device__ __forceinline__ unsigned long long run_start(unsigned long long total, int c, int n) {
    return total * (unsigned)c / (unsigned)n;
}

// A block's share of one unit.
struct Piece {
    bool prefix;
    int row, rows;       // first row and rows of the unit
    int kvh, t0, t1, len;
    const int* table;
    long long slot;      // of its part, within prefixes or groups
};

// Walks the pieces of a run of tiles; every role of a block walks its own.
struct Walk {
    unsigned long long pos, end, off;  // off: tiles before the segment
    int seg, units, cta;               // units: before the segment, of its kind
    Seg s;
    __device__ __forceinline__ bool next(const AttendParams& p, Piece& x) {
        while (pos < end) {
            const unsigned long long work = s.work(p);
            if (pos >= off + work) {
                off += work;
                units += s.tiles > 0 ? s.units * p.kv_heads : 0;
                if (++seg == p.P) units = 0;
                if (seg >= p.P + p.G) return false;
                s = load_seg(p, seg);
                continue;
            }
            const unsigned long long rel = pos - off;
            const int unit = (int)(rel / (unsigned)s.tiles);
            x.t0 = (int)(rel % (unsigned)s.tiles);
            const unsigned long long left = end - pos;
            x.t1 = left < (unsigned long long)(s.tiles - x.t0) ? x.t0 + (int)left : s.tiles;
            x.kvh = unit / s.units;
            const int first = (unit % s.units) * 2 * p.rows_per_tile;
            x.row = s.r0 + first;
            x.rows = s.n - first < 2 * p.rows_per_tile ? s.n - first : 2 * p.rows_per_tile;
            x.len = s.len;
            x.prefix = seg < p.P;
            x.table = x.prefix ? p.prefix_tables + (long long)seg * p.max_prefix_pages
                               : p.tables + (long long)(seg - p.P) * p.max_pages;
            x.slot = (long long)units + unit + cta;
            pos += x.t1 - x.t0;
            return true;
        }
        return false;
    }
};

// Index of row 0 of a piece's part (tile or warpgroup `set`); -1: past the
// scratch (only tables of overlapping prefixes can ask for it).
__device__ __forceinline__ long long part_row(const AttendParams& p, bool prefix, long long slot, int set) {
    if (prefix) return slot < p.sc.prefix_slots ? (slot * 2 + set) * kQTile : -1;
    if (slot >= p.sc.group_slots) return -1;
    return p.sc.prefix_slots * 2 * kQTile + (slot * 2 + set) * p.sc.group_rows;
}

struct Ctl {
    uint64_t full[10], empty[10];
    uint64_t q_ready, q_free, s_full[2], p_ready[2], pv_done[2], o_free[2], drain;
    unsigned long long sum[kWarps][2];
    unsigned long long start_off;
    int start_seg, start_units;
    uint32_t tmem;
    int abort;
};

// The call's tiles and units: every thread sums its share of the segments,
// the block scans the sums, and the thread that holds the block's first tile
// names its segment.  Block 0 leaves the offsets for the join.  Returns the
// total.
__device__ __forceinline__ unsigned long long plan_run(const AttendParams& p, Ctl* ctl, int& blocks) {
    const int S = p.P + p.G, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (S + kThreads - 1) / kThreads;
    const int s0 = tid * per < S ? tid * per : S, s1 = s0 + per < S ? s0 + per : S;
    unsigned long long tiles = 0, units = 0;  // units: of prefixes in the high half, of groups in the low
    for (int s = s0; s < s1; ++s) {
        const Seg x = load_seg(p, s);
        tiles += x.work(p);
        if (x.tiles > 0) units += (unsigned long long)(x.units * p.kv_heads) << (s < p.P ? 32 : 0);
        if (x.bad && blockIdx.x == 0) atomicOr(p.status, s < p.P ? kStatusBadPrefix : kStatusAttnBadGroup);
    }
    unsigned long long it = tiles, iu = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long a = __shfl_up_sync(kFull, it, o), b = __shfl_up_sync(kFull, iu, o);
        if (lane >= o) it += a, iu += b;
    }
    if (lane == 31) ctl->sum[warp][0] = it, ctl->sum[warp][1] = iu;
    __syncthreads();
    unsigned long long bt = 0, bu = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) bt = total;
        if (w < warp) bu += ctl->sum[w][1];
        total += ctl->sum[w][0];
    }
    unsigned long long off = bt + it - tiles, u = bu + iu - units;
    blocks = total < (unsigned long long)gridDim.x ? (int)total : (int)gridDim.x;
    const bool mine = (int)blockIdx.x < blocks;
    const unsigned long long lo = mine ? run_start(total, blockIdx.x, blocks) : ~0ull;
    if (blockIdx.x == 0 || (lo >= off && lo < off + tiles)) {
        for (int s = s0; s < s1; ++s) {
            const Seg x = load_seg(p, s);
            const unsigned long long work = x.work(p);
            const int before = (int)(s < p.P ? u >> 32 : u & 0xFFFFFFFFull);
            if (blockIdx.x == 0) p.sc.seg_tiles[s] = off, p.sc.seg_units[s] = before;
            if (lo >= off && lo < off + work) ctl->start_seg = s, ctl->start_units = before, ctl->start_off = off;
            off += work;
            if (x.tiles > 0) u += (unsigned long long)(x.units * p.kv_heads) << (s < p.P ? 32 : 0);
        }
    }
    if (blockIdx.x == 0 && tid == 0) p.sc.seg_tiles[S] = total;
    return total;
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
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");  // the join waits for this grid's end by itself
    const unsigned long long limit = p.timeout_ns;
    int blocks;
    const unsigned long long total = plan_run(p, ctl, blocks);
    if ((int)blockIdx.x >= blocks) return;

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) tc::mbar_init(&ctl->full[i], 1), tc::mbar_init(&ctl->empty[i], 1);
        tc::mbar_init(&ctl->q_ready, 8);
        tc::mbar_init(&ctl->q_free, 1);
        tc::mbar_init(&ctl->drain, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ctl->s_full[i], 1);
            tc::mbar_init(&ctl->p_ready[i], 4);
            tc::mbar_init(&ctl->pv_done[i], 1);
            tc::mbar_init(&ctl->o_free[i], 4);
        }
        ctl->abort = 0;
        tc::fence_async_shared();
    }
    if (warp == 2) tc::tmem_alloc(&ctl->tmem, kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ctl->tmem;
    volatile int* abort = &ctl->abort;
    // test hook: nothing arrives on `drain` before the end, so this wait runs out
    if (p.force_timeout) tc::warp_wait(&ctl->drain, 0, limit, abort);

    Walk walk;
    walk.cta = blockIdx.x;
    walk.pos = run_start(total, blockIdx.x, blocks);
    walk.end = run_start(total, blockIdx.x + 1, blocks);
    walk.off = ctl->start_off;
    walk.seg = ctl->start_seg;
    walk.units = ctl->start_units;
    walk.s = load_seg(p, walk.seg);
    Piece x;
    bool ok = !p.force_timeout;
    uint32_t it = 0;  // ring position: K and V tiles fetched (warp 0) or taken (warp 1)

    if (warp == 0) {
        // ---- pages into the ring
        constexpr int kHalves = D / 64;
        const int step = p.page_shift < 7 ? 1 << p.page_shift : kKTile;  // tokens per box
        while (ok && walk.next(p, x)) {
            for (int t = x.t0; ok && t < x.t1; ++t) {
                const int left = x.len - t * kKTile, valid = left < kKTile ? left : kKTile;
                const int boxes = (valid + step - 1) / step * kHalves;
                const int tok = lane / kHalves * step, half = lane % kHalves;
                long long page = 0;
                int y = 0;
                if (lane < boxes) {
                    const long long at = (long long)t * kKTile + tok;
                    y = (int)(at & ((1 << p.page_shift) - 1));
                    page = __ldg(&x.table[at >> p.page_shift]);
                    if (page < 0 || page >= p.num_pages) {
                        page = p.num_pages;  // outside the map: zeros
                        atomicOr(p.status, kStatusBadPage);
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const uint32_t slot = it % C::kSlots;
                    ok = tc::warp_wait(&ctl->empty[slot], (it / C::kSlots & 1u) ^ 1u, limit, abort);
                    if (!ok) break;
                    if (lane == 0) tc::mbar_expect(&ctl->full[slot], (uint32_t)boxes * step * 128u);
                    __syncwarp();
                    if (lane < boxes)
                        tc::tma_load_4d(ring + slot * C::kTileBytes + half * (kKTile * 128) + tok * 128, kv == 0 ? &k_map : &v_map,
                                        &ctl->full[slot], half * 64, y, x.kvh, (int)page);
                }
            }
        }
        // no copy outlives the block, whatever its readers did
        int none = 0;
        for (uint32_t i = it > C::kSlots ? it - C::kSlots : 0; i < it; ++i)
            tc::mbar_wait(&ctl->full[i % C::kSlots], i / C::kSlots & 1u, limit, &none);
    } else if (warp == 1) {
        // ---- the products
        constexpr uint32_t kIdescS = tc::make_idesc(kBf16, false, kQTile, kKTile), kIdescO = tc::make_idesc(kBf16, true, kQTile, D);
        const uint32_t q_addr = tc::smem_addr(smem), ring_addr = tc::smem_addr(ring);
        uint32_t pieces = 0, p_phase[2] = {0, 0}, o_phase[2] = {1, 1};
        auto wait_full = [&](uint32_t i) {
            return tc::warp_wait(&ctl->full[i % C::kSlots], i / C::kSlots & 1u, limit, abort);
        };
        auto scores = [&](int s, int q, uint32_t i) {  // S_s = Q_q K^T
            if (lane == 0) {
                const uint64_t a = tc::make_desc(q_addr + q * C::kTileBytes, 16, 1024);
                const uint64_t b = tc::make_desc(ring_addr + i % C::kSlots * C::kTileBytes, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t o = (uint64_t)(((k / 4) * (kKTile * 128) + (k % 4) * 32) >> 4);
                    tc::mma_ss(tmem + kColS + s * kColStep, a + o, b + o, kIdescS, k > 0);
                }
                tc::commit(&ctl->s_full[s]);
            }
        };
        // O_s += P_s V; the first product of a piece waits for the accumulator to be read
        auto values = [&](int s, uint32_t i, bool first, int valid) {
            if (!tc::warp_wait(&ctl->p_ready[s], p_phase[s], limit, abort)) return false;
            p_phase[s] ^= 1u;
            if (first) {
                if (!tc::warp_wait(&ctl->o_free[s], o_phase[s], limit, abort)) return false;
                o_phase[s] ^= 1u;
            }
            if (valid > 0 && valid < kKTile) {
                // slots past the length hold anything: zero them, so that 0 * v stays 0
                unsigned char* v = ring + i % C::kSlots * C::kTileBytes;
                const int chunks = (kKTile - valid) * 8;
                for (int c = lane; c < chunks * (D / 64); c += 32) {
                    const int half = c / chunks, r = c % chunks;
                    *reinterpret_cast<uint4*>(v + half * (kKTile * 128) + (valid * 8 + r) * 16) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_async_shared();
                __syncwarp();
            }
            tc::fence_after();
            if (lane == 0) {
                const uint64_t b = tc::make_desc(ring_addr + i % C::kSlots * C::kTileBytes, kKTile * 128, 1024);
#pragma unroll
                for (int k = 0; k < kKTile / 16; ++k)
                    tc::mma_ts(tmem + kColO + s * kColStep, tmem + kColS + s * kColStep + k * 8, b + (uint64_t)(k * 2048 >> 4), kIdescO,
                               !(first && k == 0));
                tc::commit(&ctl->pv_done[s]);
            }
            return true;
        };
        auto release = [&](uint32_t i) {
            if (lane == 0) tc::commit(&ctl->empty[i % C::kSlots]);
        };
        while (ok && walk.next(p, x)) {
            const int n = x.t1 - x.t0;
            const bool two = x.rows > p.rows_per_tile;
            auto valid = [&](int i) { return x.len - (x.t0 + i) * kKTile; };  // V tokens of tile i, if fewer than a tile
            ok = tc::warp_wait(&ctl->q_ready, pieces++ & 1u, limit, abort);
            tc::fence_after();
            if (two) {
                for (int i = 0; ok && i <= n; ++i) {
                    const uint32_t k = it + 2 * i, v = it + 2 * i - 1;  // K of tile i, V of tile i - 1
                    if (i < n) ok = wait_full(k);
                    if (ok && i > 0) ok = wait_full(v);
                    for (int s = 0; ok && s < 2; ++s) {
                        if (i > 0) ok = values(s, v, i == 1, s == 0 ? valid(i - 1) : 0);
                        if (ok && i < n) scores(s, s, k);
                    }
                    if (ok && i > 0) release(v);
                    if (ok && i < n) release(k);
                    if (ok && i == n - 1 && lane == 0) tc::commit(&ctl->q_free);
                }
            } else {
                for (int i = 0; ok && i < n + 2; ++i) {
                    const int s = i & 1;
                    if (i >= 2) {
                        const uint32_t v = it + 2 * (i - 2) + 1;
                        if (i - 2 < n) {
                            ok = wait_full(v) && values(s, v, i - 2 < 2, valid(i - 2));
                            if (ok) release(v);
                        }
                    }
                    if (ok && i < n) {
                        const uint32_t k = it + 2 * i;
                        ok = wait_full(k);
                        if (ok) {
                            tc::fence_after();
                            scores(s, 0, k);
                            release(k);
                        }
                    }
                    if (ok && i == n - 1 && lane == 0) tc::commit(&ctl->q_free);
                }
            }
            it += 2 * n;
        }
        if (lane == 0) {  // nor does a product
            int none = 0;
            tc::commit(&ctl->drain);
            tc::mbar_wait(&ctl->drain, 0, limit, &none);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---- softmax
        const int wg = (warp - 4) >> 2;             // warpgroup: query tile, or parity of token tiles
        const int row = (warp & 3) * 32 + lane;     // tile row of this thread
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_col = tmem + lanes + kColS + wg * kColStep, o_col = tmem + lanes + kColO + wg * kColStep;
        const float c = p.scale * kLog2e;
        // F16 keeps probabilities down to 2^-24: lifting them by 2^6 (at most 2^14 then) keeps those above 2^-30
        constexpr float kBias = kBf16 ? 0.0f : 6.0f;
        uint32_t pieces = 0, s_phase = 0, pv = 0;
        while (ok && walk.next(p, x)) {
            const bool two = x.rows > p.rows_per_tile;
            const int n = x.t1 - x.t0, rt = p.rows_per_tile;
            const int rows = two ? (wg == 0 ? rt : x.rows - rt) : x.rows;
            const int valid_rows = rows * p.share;
            // the query tile: both warpgroups fill half of it when there is one
            if (pieces > 0) ok = tc::warp_wait(&ctl->q_free, (pieces - 1) & 1u, limit, abort);
            if (!ok) break;
            ++pieces;
            {
                const int per = row < valid_rows ? row / p.share : 0, head = x.kvh * p.share + (row < valid_rows ? row % p.share : 0);
                const T* src = reinterpret_cast<const T*>(p.q) + (long long)(x.row + (two ? wg * rt : 0) + per) * p.q_stride + (long long)head * D;
                unsigned char* dst = smem + (two ? wg * C::kTileBytes : 0) + row * 128;
                constexpr int kChunks = D / 8;
                const int c0 = two ? 0 : wg * (kChunks / 2), cn = two ? kChunks : kChunks / 2;
#pragma unroll 8
                for (int i = 0; i < cn; ++i) {
                    const int ch = c0 + i;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (row < valid_rows) w = __ldg(reinterpret_cast<const uint4*>(src + ch * 8));
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * (kKTile * 128) + (((ch & 7) ^ (row & 7)) << 4)) = w;
                }
            }
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->q_ready);

            const bool live = (warp & 3) * 32 < valid_rows;  // any row of this warp
            float m = kNegInf, base = 0.0f, l = 0.0f;        // maximum; what is subtracted in base 2; sum
            const int first = two ? 0 : wg, stride = two ? 1 : 2;
            for (int i = first; i < n; i += stride) {
                ok = tc::warp_wait(&ctl->s_full[wg], s_phase, limit, abort);
                if (!ok) break;
                s_phase ^= 1u;
                tc::fence_after();
                if (live) {
                    uint32_t r[4][32];
#pragma unroll
                    for (int b = 0; b < 4; ++b) tc::tmem_ld32(s_col + b * 32, r[b]);
                    tc::wait_ld();
#pragma unroll
                    for (int b = 0; b < 4; ++b) tc::tie(r[b]);
                    const int valid = x.len - (x.t0 + i) * kKTile;
                    if (valid < kKTile) {
#pragma unroll
                        for (int b = 0; b < 4; ++b)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (b * 32 + e >= valid) r[b][e] = __float_as_uint(kNegInf);
                    }
                    float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(r[b][e]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (i == first) {
                        m = top;
                        base = m == kNegInf ? 0.0f : m * c - kBias;
                    } else {
                        const bool grow = m == kNegInf ? top > m : top * c > m * c + kRescale;
                        if (__any_sync(kFull, grow)) {
                            float f = 1.0f;
                            if (grow) {
                                const float next = top * c - kBias;
                                if (m != kNegInf) f = ex2(base - next);
                                m = top;
                                base = next;
                                l *= f;
                            }
                            // the accumulator is this warp's to change once the products so far are in
                            ok = tc::warp_wait(&ctl->pv_done[wg], (pv - 1) & 1u, limit, abort);
                            if (!ok) break;
                            tc::fence_after();
#pragma unroll
                            for (int b = 0; b < D / 32; ++b) {
                                uint32_t o[32];
                                tc::tmem_ld32(o_col + b * 32, o);
                                tc::wait_ld();
                                tc::tie(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::tmem_st32(o_col + b * 32, o);
                            }
                            tc::wait_st();
                        }
                    }
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int b = 0; b < 4; b += 2) {
                        uint32_t w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float a0 = ex2(fmaf(__uint_as_float(r[b + e / 16][2 * (e % 16)]), c, -base));
                            const float a1 = ex2(fmaf(__uint_as_float(r[b + e / 16][2 * (e % 16) + 1]), c, -base));
                            sum[(2 * e) & 3] += a0;
                            sum[(2 * e + 1) & 3] += a1;
                            w[e] = H::pack(a0, a1);
                        }
                        tc::tmem_st32(s_col + b * 16, w);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc::wait_st();
                }
                ++pv;
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->p_ready[wg]);
            }
            if (!ok) break;
            if (first < n) {
                ok = tc::warp_wait(&ctl->pv_done[wg], (pv - 1) & 1u, limit, abort);
                if (!ok) break;
                tc::fence_after();
                if (live) {
                    const long long at = part_row(p, x.prefix, x.slot, wg) + row;
                    const bool store = row < valid_rows && at >= row;
                    if (store) p.sc.part_ml[at] = make_float2(m == kNegInf ? kNegInf : base, l);
                    float4* dst = reinterpret_cast<float4*>(p.sc.part_o + (store ? at : 0) * D);
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) {
                        uint32_t o[32];
                        tc::tmem_ld32(o_col + b * 32, o);
                        tc::wait_ld();
                        tc::tie(o);
                        if (store) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[b * 8 + e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                             __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->o_free[wg]);
            }
        }
    }
    __syncthreads();
    if (tid == 0 && *abort != 0) atomicOr(p.status, kStatusAttnTimeout);
    if (warp == 2) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool kBf16, int D>
__device__ __forceinline__ void load_lane(const void* base, long long elem, float (&x)[D / 32]) {
    using H = Half<kBf16>;
    const typename H::T* s = reinterpret_cast<const typename H::T*>(base) + elem;
    if constexpr (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(s);
        const float2 a = H::unpack(w.x), b = H::unpack(w.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    } else {
        const float2 a = H::unpack(*reinterpret_cast<const uint32_t*>(s));
        x[0] = a.x, x[1] = a.y;
    }
}

// Running softmax of one query head, D / 32 lanes of the head per thread, in base 2.
template <int D>
struct Acc {
    float o[D / 32], m, l;
    __device__ __forceinline__ void add(float s, float w, const float (&v)[D / 32]) {  // a part: maximum s, sum w, result v
        const float top = fmaxf(m, s), base = top == kNegInf ? 0.0f : top;
        const float f = ex2(m - base), g = ex2(s - base);
        l = l * f + w * g;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = o[e] * f + g * v[e];
        m = top;
    }
};

// Joins the parts of one segment for tile-row `row` of the unit that holds row
// `rel` of the segment.
template <int D>
__device__ __forceinline__ void join_parts(const AttendParams& p, Acc<D>& a, int seg, int rel, int head, int lane,
                                           unsigned long long total, int blocks) {
    const Seg s = load_seg(p, seg);
    if (s.tiles == 0) return;
    const bool prefix = seg < p.P;
    const int rt = p.rows_per_tile, u = rel / (2 * rt), left = s.n - u * 2 * rt;
    const bool two = left > rt;
    const int in = rel - u * 2 * rt, kvh = head / p.share;
    const int row = (two ? in % rt : in) * p.share + head % p.share;
    const unsigned long long begin = p.sc.seg_tiles[seg] + (unsigned long long)(kvh * s.units + u) * s.tiles, end = begin + s.tiles;
    const long long slot = (long long)p.sc.seg_units[seg] + kvh * s.units + u;
    // the blocks whose runs hold the unit's first and last tile
    const int c0 = (int)(((begin + 1) * (unsigned)blocks - 1) / total), c1 = (int)((end * (unsigned)blocks - 1) / total);
    const int sets = two ? 1 : 2;
    for (int k = 0; k < (c1 - c0 + 1) * sets; ++k) {
        const int c = c0 + k / sets, set = two ? in / rt : k % sets;
        if (!two && set == 1) {  // the second warpgroup had a tile only in a run of two or more
            const unsigned long long lo = run_start(total, c, blocks), hi = run_start(total, c + 1, blocks);
            if ((hi < end ? hi : end) - (lo > begin ? lo : begin) < 2) continue;
        }
        const long long at = part_row(p, prefix, slot + c, set);
        if (at < 0) continue;
        const float2 ml = p.sc.part_ml[at + row];
        float v[D / 32];
        const float* src = p.sc.part_o + (at + row) * D + lane * (D / 32);
        if constexpr (D == 128) {
            const float4 w = *reinterpret_cast<const float4*>(src);
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        } else {
            const float2 w = *reinterpret_cast<const float2*>(src);
            v[0] = w.x, v[1] = w.y;
        }
        a.add(ml.x, ml.y, v);
    }
}

// One warp per (row, query head): the parts of the row's prefix and of its
// group's committed tokens, then the round's own tokens that the row sees.
template <bool kBf16, int D>
__global__ void __launch_bounds__(kJoinThreads) lp_attend_join_kernel(const AttendParams p) {
    using H = Half<kBf16>;
    using T = typename H::T;
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, head = blockIdx.y * (kJoinThreads / 32) + warp;
    const int g = block_find_group(p.indptr, p.G, row);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (g < 0 || g >= p.G || head >= p.q_heads) return;
    if (row < __ldg(&p.indptr[g]) || row >= __ldg(&p.indptr[g + 1])) return;  // two entries claim the row
    const Group grp = load_group(p, g);
    Acc<D> a;
#pragma unroll
    for (int e = 0; e < kE; ++e) a.o[e] = 0.0f;
    a.m = kNegInf, a.l = 0.0f;
    if (grp.n > 0) {
        const unsigned long long total = p.sc.seg_tiles[p.P + p.G];
        const int blocks = total < (unsigned long long)p.grid ? (int)total : p.grid;
        for (int i = 0; i < p.P; ++i) {
            const Prefix x = load_prefix(p, i);
            if (x.bad || g < x.g0 || g >= x.g1) continue;
            join_parts<D>(p, a, i, row - x.r0, head, lane, total, blocks);
            break;
        }
        join_parts<D>(p, a, p.P + g, row - grp.r0, head, lane, total, blocks);
        float q[kE];
        load_lane<kBf16, D>(p.q, row * p.q_stride + (long long)head * D + lane * kE, q);
        const float c = p.scale * kLog2e;
        const int* table = p.tables + (long long)g * p.max_pages;
        const int j = row - grp.r0, kvh = head / p.share;
        const unsigned mask = p.row_masks != nullptr ? __ldg(&p.row_masks[row]) : (2u << j) - 1u;
        for (int i = 0; i < grp.n; ++i) {
            if (!(mask >> i & 1u)) continue;
            const int t = grp.len + i;
            const int page = __ldg(&table[t >> p.page_shift]);
            float k[kE] = {}, v[kE] = {};
            if (page >= 0 && page < p.num_pages) {
                const long long at =
                    (((((long long)page * p.kv_heads + kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1))) * D) + lane * kE;
                load_lane<kBf16, D>(p.k_cache, at, k);
                load_lane<kBf16, D>(p.v_cache, at, v);
            } else if (lane == 0) {
                atomicOr(p.status, kStatusBadPage);
            }
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < kE; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            a.add(s * c, 1.0f, v);
        }
    }
    const float inv = a.l > 0.0f ? 1.0f / a.l : (a.l == 0.0f ? 0.0f : a.l);
    T* dst = reinterpret_cast<T*>(p.out) + row * p.out_stride + (long long)head * D + lane * kE;
    if constexpr (D == 128) {
        uint2 w;
        w.x = H::pack(a.o[0] * inv, a.o[1] * inv);
        w.y = H::pack(a.o[2] * inv, a.o[3] * inv);
        *reinterpret_cast<uint2*>(dst) = w;
    } else {
        *reinterpret_cast<uint32_t*>(dst) = H::pack(a.o[0] * inv, a.o[1] * inv);
    }
    if (p.lse_out != nullptr && lane == 0)
        p.lse_out[(long long)row * p.q_heads + head] = a.l == 0.0f ? kNegInf : a.m * kLn2 + logf(a.l);
}

template <int D>
constexpr int smem_bytes() { return Cfg<D>::kCtl + (int)sizeof(Ctl); }

template <bool kBf16, int D>
cudaError_t prepare() {
    static_assert(smem_bytes<D>() <= 232448, "shared memory");
    return cudaFuncSetAttribute(lp_attend_kernel<kBf16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>());
}

template <bool kBf16, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
    lp_attend_kernel<kBf16, D><<<p.grid, kThreads, smem_bytes<D>(), stream>>>(p, k_map, v_map);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.rows, (unsigned)((p.q_heads + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    lc.blockDim = dim3(kJoinThreads);
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D>, p);
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
