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
//
// Over a cache in 4 bits (lp_attend4 where many rows share a token) four more warps
// expand codes into the ring of K and V tiles, 128 KiB then, and the products are F16.
// They bound it: a quarter of a K or V tile takes a warp 1,540 cycles (560 to
// convert and store it, 560 to fetch the next one's codes, the rest in waits), so the
// prefix's part of 2,048 rows takes 800 us, 1.37 PFLOP/s.  Codes by bulk copies of warp 0 took
// 174 us where these take 206 (19 groups of 12 rows and 16,384 tokens, pages of 256
// tokens; 364 with pages of 16), bulk copies of each warp's own 220, loads into
// registers one tile ahead 261; eight such warps leave the softmax too few registers.
// A thread spills 40 bytes (F16: 28).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "lp_join.h"
#include "lp_split.h"
#include "lp_tc.h"

namespace lp {
namespace {

// Tokens of a tile whose probabilities are announced before the others', so that
// their part of P V runs under the rest of the softmax (2,048 rows behind 32,768
// tokens: 762 us; 32 tokens 785, 96 790, all at once 809).
constexpr int kEarly = 64;
constexpr float kRescale = 8.0f;  // growth of the maximum (log2) that moves it
// Of a block.  Registers: the softmax warpgroups hold 128 scores per thread.  The
// split's sum is what the block is launched with (384 x 168, 512 x 128).
template <bool kFour>
struct Block {
    static constexpr int kThreads = kFour ? 512 : 384, kWarps = kThreads / 32;
    static constexpr int kRegsLaunch = kFour ? 128 : 168, kRegsSoftmax = kFour ? 184 : 200, kRegsOther = kFour ? 72 : 104;
    static constexpr int kPieceReaders = kFour ? 15 : 11;  // two warps of the products, one that loads queries, eight of softmax, four that expand
    static_assert(2 * kRegsSoftmax + (kFour ? 2 : 1) * kRegsOther <= kThreads / 128 * kRegsLaunch, "register split");
};

// Tensor memory columns: two score tiles, two accumulators.
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256, kColStep = 128;

template <int D, bool kFour>
struct Cfg {
    static constexpr int kTileBytes = kKTile * D * 2;                // one K, V or Q tile
    static constexpr int kSlots = (kFour ? 4 : 5) * 128 / D;         // ring of K and V tiles: 160 KiB (4 bits: 128)
    static constexpr int kEntries = 3;                               // 4 bits: a warp's ring of K and V codes and scales,
    static constexpr int kEntry = 32 * (D / 2 + D / kBlock4);        // 32 tokens each
    static constexpr int kCodes = (2 + kSlots) * kTileBytes;
    static constexpr int kCtl = kCodes + (kFour ? 4 * kEntries * kEntry : 0);
};

constexpr int kPieces = 8;        // pieces the fetching warp may be ahead

// Where the tokens of a piece lie.
struct Pages {
    const int* table;
    long long token;  // the first
};

template <bool kFour>
using RuleOf = std::conditional_t<kFour, Pairs4, Pairs>;

template <bool kFour>
struct Ctl : PlanCtl<RuleOf<kFour>> {
    uint64_t full[10], empty[10], piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    uint64_t q_full[2], q_free[2], s_full[2], p_early[2], p_ready[2], pv_done[2], o_free[2], q_grant, clean, drain;
    uint32_t tmem, issued, batches[2];  // ring fills under way or done; see take_turn
    int abort;
    // 4 bits: of the pieces; what a tile's row of queries was divided by, of the last four pieces
    Pages pages[kFour ? kPieces : 1];
    float unit[kFour ? 4 : 1][2][kFour ? kQTile : 1];
};

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
// One row's running softmax: the maximum, what is subtracted in base 2, the sum.
struct Row {
    float m, base, l;
    float taken;  // F16 over a cache in 4 bits: the sum of the probabilities as the products take them; by it, not by l, the
                  // results are divided, and what the rounding does to a row of few tokens cancels
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
        row.l = row.taken = 0.0f;
        return false;
    }
    const bool grow = used && (row.m == kNegInf ? top > row.m : top * c > row.m * c + kRescale);
    if (grow) {
        const float next = top * c - kBias;
        if (row.m != kNegInf) f = ex2(row.base - next);
        row.m = top;
        row.base = next;
        row.l *= f;
        row.taken *= f;
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
template <bool kBf16, int D, bool kTaken>
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
    unsigned long long sum[2] = {0, 0}, taken[2] = {0, 0};
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
            if constexpr (kTaken) {
                const float2 f = Half<kBf16>::unpack(w[e]);
                taken[e & 1] = add2(taken[e & 1], pack2(__float_as_uint(f.x), __float_as_uint(f.y)));
            }
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
    if constexpr (kTaken) {
        unpack2(add2(taken[0], taken[1]), x, y);
        row.taken += x + y;
    }
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

// The same from BF16 to F16, each row by a power of two of its own; D / 8 threads have a
// row, `n` a multiple of 32.  unit[row]: what undoes it.  All of it is under way at once,
// then each thread changes what it fetched.
template <int D>
__device__ __forceinline__ void lift_queries(const AttendParams& p, int row0, int rows, int kvh, uint32_t dst, int again, float* unit, int t, int n) {
    constexpr int kChunks = D / 8;
    const int ch = t % kChunks, total = rows * p.share, step = n / kChunks;
    const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(p.q) + (long long)row0 * p.q_stride + (long long)kvh * p.share * D + ch * 8;
    auto place = [&](int row) { return dst + (ch >> 3) * (kQTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4); };
    for (int row = t / kChunks; row < total; row += step) {
        const int per = (row * p.share_inv) >> 16, head = row - per * p.share;
        tc::copy16(place(row), src + per * p.q_stride + head * D);
    }
    tc::copies_done();
#pragma unroll 4
    for (int base = 0; base < total; base += step) {
        const int row = base + t / kChunks;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (row < total) w = tc::load16(place(row));
        // the largest magnitude: that of BF16 is its order as an integer without the sign
        const uint32_t m = 0x7FFF7FFFu;
        uint32_t top = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
#pragma unroll
        for (int o = kChunks / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, o));
        if (row >= total) continue;
        const float2 lift = lift_of(__uint_as_float(top >> 16 > (top & 0xFFFFu) ? top & 0xFFFF0000u : top << 16));
        if (ch == 0) unit[row] = lift.y;
        float x[8];
        widen8<true>(w, x);
        const uint4 y = make_uint4(Half<false>::pack(x[0] * lift.x, x[1] * lift.x), Half<false>::pack(x[2] * lift.x, x[3] * lift.x),
                                   Half<false>::pack(x[4] * lift.x, x[5] * lift.x), Half<false>::pack(x[6] * lift.x, x[7] * lift.x));
        tc::store16(place(row), y);
        if (again > 0) tc::store16(place(row) + again * 128, y);
    }
    tc::fence_async_shared();
}

// A cache in 4 bits into the ring of K and V tiles, by four warps: 32 tokens of
// each tile are a warp's, from their pages (a token's per lane) by way of a ring of
// its own to F16 in the places where the tensor core reads them.
template <int D>
__device__ __forceinline__ void expand(const AttendParams& p, unsigned char* smem, Ctl<true>* ctl, int quarter, bool ok, unsigned long long limit) {
    using C = Cfg<D, true>;
    constexpr int kParts = D / 32, kAtOnce = 32 / kParts;  // 16-byte parts of a token's codes; tokens of an instruction
    volatile int* abort = &ctl->abort;
    const int lane = threadIdx.x & 31, mask = (1 << p.page_shift) - 1;
    unsigned char* entries = smem + C::kCodes + quarter * (C::kEntries * C::kEntry);
    // a token's parts are turned, so that the lanes that read a part of eight tokens meet every bank once
    auto place = [](int token, int part) { return token * (D / 2) + (part ^ (D == 128 ? token >> 1 & 3 : token >> 2 & 1)) * 16; };

    // what is fetched: the piece, its tile, the slot of this lane's token; whether the keys of the tile are under way
    Piece x = {};
    Pages from = {nullptr, 0};
    uint32_t n_piece = 0, fetched = 0, done = 0;
    int tile = 0, next_page = -1;
    long long slot = -1;
    bool more = true, keys = false;
    auto page_of = [&](int i) {
        const int t = i * kKTile + quarter * 32 + lane;
        return i < x.tiles && t < x.left ? from.table[(from.token + t) >> p.page_shift] : -1;
    };
    auto fetch = [&]() {  // the next entry; false at the end of the run
        if (!keys) {
            while (tile >= x.tiles) {
                const uint32_t i = n_piece % kPieces;
                ok = tc::warp_wait(&ctl->piece_full[i], n_piece / kPieces & 1u, limit, abort);
                if (!ok) return false;
                x = ctl->piece[i];
                from = ctl->pages[i];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->piece_empty[i]);
                ++n_piece;
                if (x.rows == 0) return false;
                tile = 0;
                next_page = page_of(0);
            }
            const int page = next_page, t = tile * kKTile + quarter * 32 + lane;
            next_page = page_of(++tile);  // before the waits of this one
            const bool exists = t < x.left, good = page >= 0 && page < p.num_pages;
            if (exists && !good) atomicOr(p.status, kStatusBadPage);  // such a page reads as zeros
            slot = exists && good ? (((long long)page * p.kv_heads + x.kvh) << p.page_shift) + ((from.token + t) & mask) : -1;
        }
        keys = !keys;
        const unsigned char* codes = static_cast<const unsigned char*>(keys ? p.k_cache : p.v_cache);
        const uint32_t to = tc::smem_addr(entries + fetched % C::kEntries * C::kEntry);
#pragma unroll
        for (int j = 0; j < 32 / kAtOnce; ++j) {
            const int token = j * kAtOnce + lane / kParts, part = lane % kParts;
            const long long at = __shfl_sync(kFull, slot, token);
            tc::copy16_or_zeros(to + place(token, part), codes + (at < 0 ? 0 : at) * (D / 2) + part * 16, at >= 0);
        }
        tc::copy_or_zeros<D / kBlock4>(to + 16 * D + lane * (D / kBlock4), (keys ? p.k_scales : p.v_scales) + (slot < 0 ? 0 : slot) * (D / kBlock4), slot >= 0);
        ++fetched;
        return true;
    };
    while (ok) {
        while (more && fetched - done < C::kEntries) {
            more = fetch();
            tc::copies_commit();
        }
        if (!ok || done == fetched) break;
        const uint32_t ahead = fetched - done - 1 + (more ? 0 : 1);  // groups after the oldest (the last one is empty)
        if (ahead >= 2) tc::copies_wait<2>();
        else if (ahead == 1) tc::copies_wait<1>();
        else tc::copies_wait<0>();
        __syncwarp();
        const uint32_t at = done % C::kSlots;
        ok = tc::warp_wait(&ctl->empty[at], (done / C::kSlots & 1u) ^ 1u, limit, abort);
        if (!ok) break;
        if (quarter == 0 && lane == 0) tc::store_release(&ctl->issued, done + 1);
        const unsigned char* entry = entries + done % C::kEntries * C::kEntry;
        uint32_t e[D / 16];
        {
            uint32_t s[D / 64];
            if constexpr (D == 128) {
                const uint2 w = *reinterpret_cast<const uint2*>(entry + 16 * D + lane * 8);
                s[0] = w.x, s[D / 64 - 1] = w.y;
            } else {
                s[0] = *reinterpret_cast<const uint32_t*>(entry + 16 * D + lane * 4);
            }
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                uint32_t a, b;
                asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(a), "=r"(b) : "r"(s[i]));
                e[4 * i] = __byte_perm(a, 0, 0x1010), e[4 * i + 1] = __byte_perm(a, 0, 0x3232);
                e[4 * i + 2] = __byte_perm(b, 0, 0x1010), e[4 * i + 3] = __byte_perm(b, 0, 0x3232);
            }
        }
        const int row = quarter * 32 + lane;
        const uint32_t to = tc::smem_addr(smem + 2 * C::kTileBytes + at * C::kTileBytes) + row * 128;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(entry + place(lane, i));
            const uint32_t codes[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ch = i * 4 + k;
                uint32_t h[4];
                widen_codes(codes[k], h);
                tc::store16(to + (ch >> 3) * (kKTile * 128) + (((ch & 7) ^ (row & 7)) << 4),
                            make_uint4(mul2(h[0], e[ch / 2]), mul2(h[1], e[ch / 2]), mul2(h[2], e[ch / 2]), mul2(h[3], e[ch / 2])));
            }
        }
        tc::fence_async_shared();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->full[at]);
        ++done;
    }
    tc::copies_done();  // no copy outlives the block, whatever its readers did
}

// kFour: the caches are in 4 bits, and the products F16 whatever the plan's type.
template <bool kBf16, int D, bool kFour>
__device__ __forceinline__ void attend(const AttendParams& p, const CUtensorMap* k_map, const CUtensorMap* v_map) {
    using T = typename Half<kBf16>::T;
    using C = Cfg<D, kFour>;
    using B = Block<kFour>;
    constexpr bool kWide = kBf16 && !kFour;   // type of the products
    constexpr bool kTaken = kFour && !kBf16;  // results divided by Row::taken: BF16 results are rounded by more than that gives
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl<kFour>* ctl = reinterpret_cast<Ctl<kFour>*>(smem + C::kCtl);
    unsigned char* ring = smem + 2 * C::kTileBytes;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, as the compiler sees
    const unsigned long long limit = p.timeout_ns;
    // the barriers, while the kernel ahead still runs
    if (warp == B::kWarps - 1) {
        if (lane < C::kSlots) tc::mbar_init(&ctl->full[lane], kFour ? 4 : 1), tc::mbar_init(&ctl->empty[lane], 2);
        if (lane < kPieces) tc::mbar_init(&ctl->piece_full[lane], 1), tc::mbar_init(&ctl->piece_empty[lane], B::kPieceReaders);
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
    if (!kFour && tid == 0) tc::prefetch_map(k_map), tc::prefetch_map(v_map);
    // so far nothing of what earlier kernels write; the join may start once that is there, and waits for this grid's end by itself
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 2) tc::tmem_alloc(&ctl->tmem, kTmemCols);  // not held while waiting: the kernel ahead may need it to end
    Runs runs[2];  // of prefixes, of groups
    const bool any = plan_run<RuleOf<kFour>>(p, ctl, runs);
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
    if (warp >= 4 && warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(B::kRegsSoftmax));
        // ---- softmax
        const int wg = (warp - 4) >> 2, quarter = warp & 3;  // tensor tile; lanes 32 * quarter of tensor memory
        const uint32_t lanes = (uint32_t)quarter << 21;
        const uint32_t s_col = tmem + lanes + kColS + wg * kColStep, o_col = tmem + lanes + kColO + wg * kColStep;
        float c = kFour ? scaled(p.score, p.score_exp) : p.scale * kLog2e;
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
                const int first_row = x.row + wg * rt, rows = wg == 0 ? rt : x.rows - rt;
                const uint32_t to = tc::smem_addr(smem + b * C::kTileBytes);
                if constexpr (kFour && kBf16)
                    lift_queries<D>(p, first_row, rows, x.kvh, to, 0, ctl->unit[(n_piece - 1) & 3u][wg], tid & 127, 128);
                else
                    load_queries<T, D>(p, first_row, rows, x.kvh, to, 0, tid & 127, 128);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->q_full[b], 1);
            }
            q_pos += two ? 2 : 1;
            Row st = {kNegInf, 0.0f, 0.0f, 0.0f};
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
                    if constexpr (kFour && kBf16) {
                        if (i == first && used) c = scaled(p.score, p.score_exp + exponent_of(ctl->unit[(n_piece - 1) & 3u][two ? wg : 0][row]));
                    }
                    softmax_tile<kWide, D, kTaken>(s_col, o_col, x.left - i * kKTile, i == first, used, c, st, &ctl->p_early[wg]);
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
                        if constexpr (kTaken) {
                            const float by = st.taken == 0.0f ? 1.0f : st.l / st.taken;
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                        }
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
    } else if (kFour && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(B::kRegsOther));
        if constexpr (kFour) expand<D>(p, smem, ctl, warp - 12, ok, limit);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(B::kRegsOther));
        if (warp == 0) {
            // ---- pages into the ring
            constexpr int kHalves = D / 64;
            const int step = p.page_shift < 7 ? 1 << p.page_shift : kKTile;  // tokens per box
            const int tok = lane / kHalves * step, half = lane % kHalves;
            Walk<RuleOf<kFour>> walk;
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
                    if constexpr (kFour) ctl->pages[pi] = Pages{walk.table, walk.token};
                    tc::mbar_arrive(&ctl->piece_full[pi]);
                }
                ++n_piece;
                if (!more) break;
                if (kFour) continue;  // the expanding warps fetch
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
                    ok = fetch(k_map, boxes, y, kvh, page) && fetch(v_map, boxes, y, kvh, page);
                }
            }
            // no copy outlives the block, whatever its readers did
            int none = 0;
            for (uint32_t i = it > C::kSlots ? it - C::kSlots : 0; !kFour && i < it; ++i)
                tc::mbar_wait(&ctl->full[i % C::kSlots], i / C::kSlots & 1u, limit, &none);
        } else if (warp <= 2) {
            // ---- the products of tensor tile s; the other tile's run while this warp waits and commits.  The whole warp
            // walks through, and one lane is elected for each instruction: descriptors stay in uniform registers, and 16
            // products are issued in 650 cycles (in a branch of one lane: 1,240 beside two busy softmax warps).
            constexpr uint32_t kIdescS = tc::make_idesc(kWide, false, kQTile, kKTile), kIdescO = tc::make_idesc(kWide, true, kQTile, D);
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
                if (!kFour && (have & 15) != 0 && have < kKTile) {  // the rows that the last 16 of V take in
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
                if constexpr (kFour && kBf16)
                    lift_queries<D>(p, x.row, x.rows, x.kvh, tc::smem_addr(smem + b * C::kTileBytes), second_at(x.rows * p.share),
                                    ctl->unit[(n_piece - 1) & 3u][0], lane, 32);
                else
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

template <bool kBf16, int D>
__global__ void __launch_bounds__(Block<false>::kThreads, 1)
    lp_attend_kernel(const AttendParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    attend<kBf16, D, false>(p, &k_map, &v_map);
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(Block<true>::kThreads, 1) lp_attend4_pairs_kernel(const AttendParams p) {
    attend<kBf16, D, true>(p, nullptr, nullptr);
}

template <int D, bool kFour>
constexpr int smem_bytes() { return Cfg<D, kFour>::kCtl + (int)sizeof(Ctl<kFour>); }

template <bool kBf16, int D>
cudaError_t prepare() {
    static_assert(smem_bytes<D, false>() <= 232448, "shared memory");
    const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(lp_attend_kernel<kBf16, D>, most, smem_bytes<D, false>());
    return e == cudaSuccess ? prepare_join<kBf16, D, false>() : e;
}

template <bool kBf16, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
    // Both kernels are launched while the one before still runs, and wait for its end before they read what it writes.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.grid);
    lc.blockDim = dim3(Block<false>::kThreads);
    lc.dynamicSmemBytes = smem_bytes<D, false>();
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, lp_attend_kernel<kBf16, D>, p, k_map, v_map);
    if (e != cudaSuccess) return e;
    return launch_join<kBf16, D, false>(p, lc);
}

template <bool kBf16, int D>
cudaError_t prepare_pairs4() {
    static_assert(smem_bytes<D, true>() <= 232448, "shared memory");
    return cudaFuncSetAttribute(lp_attend4_pairs_kernel<kBf16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D, true>());
}

template <bool kBf16, int D>
cudaError_t launch_pairs4(const AttendParams& p, cudaLaunchConfig_t lc) {
    lc.blockDim = dim3(Block<true>::kThreads);
    lc.dynamicSmemBytes = smem_bytes<D, true>();
    return cudaLaunchKernelEx(&lc, lp_attend4_pairs_kernel<kBf16, D>, p);
}

}  // namespace

cudaError_t prepare_attend4_pairs(int dtype, int head_dim) {
    if (dtype == 1) return head_dim == 128 ? prepare_pairs4<true, 128>() : prepare_pairs4<true, 64>();
    return head_dim == 128 ? prepare_pairs4<false, 128>() : prepare_pairs4<false, 64>();
}

cudaError_t launch_attend4_pairs(const AttendParams& p, int dtype, int head_dim, const cudaLaunchConfig_t& lc) {
    if (dtype == 1) return head_dim == 128 ? launch_pairs4<true, 128>(p, lc) : launch_pairs4<true, 64>(p, lc);
    return head_dim == 128 ? launch_pairs4<false, 128>(p, lc) : launch_pairs4<false, 64>(p, lc);
}

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
