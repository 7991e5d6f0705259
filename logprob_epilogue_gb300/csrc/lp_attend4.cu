// lp_attend4.cu -- sm_103a kernel of lp_attend4 for few rows: attention of verify
// rows over a paged cache held in 4 bits.
//
// The sums, their parts and the split of the work are those of lp_attend (see
// lp_split.h and lp_join.h): prefixes and committed tokens here, the round's own
// tokens in the join.  A token and head is D / 2 bytes of codes and D / 16 of
// scales, 0.28 of the bytes of 16 bits, so what has to keep up is the way from
// codes to products.  With few rows the tokens are the long side, and the products
// are turned over: with K [tokens, D], V [tokens, D] and the unit's queries Q
// [rows, D] of at most 32 rows,
//   S^T = K Q^T     tokens x rows     K from tensor memory, Q from shared memory
//   O^T += V^T P^T  D x rows          V and P from shared memory
// A tile of 128 tokens is the 128 rows of the first and the sum of the second, and
// the tensor core's time goes by the few columns.
//
// Block (one per SM, 16 warps): warp 0 splits the work, warp 1 issues the products,
// warps 2 and 3 bring the units' queries; warps 4-11 fetch 32 tokens at a time by
// TMA into a ring of their own (18 KiB each in flight at most, no other warp waits on
// it) and expand them, a token per thread: keys into tensor memory, values into
// shared memory, F16; warps 12-15 are the softmax, a token per thread.  A column's
// maximum is one for all 128 threads: it holds until a score is 2^8 above it, which a
// vote finds, and only then are the tokens' maxima compared.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lp_join.h"
#include "lp_split.h"
#include "lp_tc.h"

namespace lp {
namespace {

constexpr float kRescale = 8.0f;  // growth of the maximum (log2) that moves it
// Probabilities are lifted by 2^6 (at most 2^14 then): F16 keeps those above 2^-30 of the largest.
constexpr float kBias = 6.0f;
constexpr int kBlockThreads = 512, kBlockWarps = kBlockThreads / 32;
constexpr int kQueryWarps = 2, kFirstExpand = 4, kExpandWarps = 8, kFirstSoftmax = 12;
constexpr int kChunk = 32;  // tokens of a warp's fetch
// Registers: the split's sum is what the block is launched with, 512 x 128.
constexpr int kRegsLaunch = 128, kRegsExpand = 136, kRegsSoftmax = 160, kRegsOther = 80;
static_assert(2 * kRegsExpand + kRegsSoftmax + kRegsOther <= 4 * kRegsLaunch, "register split");
// Tensor memory columns: two tiles of keys, two of scores, the result.
constexpr uint32_t kTmemCols = 256, kColK = 0, kColS = 128, kColO = 192;

template <int D>
struct Cfg4 {
    static constexpr int kValues = kKTile * D * 2;              // a tile of values, F16
    static constexpr int kProbs = kKTile * 128;                 // a tile of probabilities: 32 columns of 64
    static constexpr int kQuery = kUnitRows * D * 2;            // a unit's queries
    static constexpr int kCodes = kChunk * D / 2, kScales = kChunk * D / kBlock4;
    static constexpr int kBytes = 2 * (kCodes + kScales);       // K and V of a chunk: codes, then scales
    static constexpr int kRing = 3 * 128 / D;                   // a warp's chunks
    static constexpr int kAtProbs = 2 * kValues, kAtQueries = kAtProbs + 2 * kProbs, kAtRing = kAtQueries + 2 * kQuery;
    static constexpr int kCtl = kAtRing + kExpandWarps * kRing * kBytes;
};

constexpr int kPieces = 8, kAhead = 4;  // pieces the planning warp may be ahead, and a warp's fetches
constexpr int kPieceReaders = 1 + kQueryWarps + kExpandWarps + 4;

// Where the tokens of a piece lie.
struct Pages {
    const int* table;
    long long token;  // the first
};

template <int D>
struct Ctl4 : PlanCtl<Columns> {
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    Pages pages[kPieces];
    uint64_t chunk_full[kExpandWarps][Cfg4<D>::kRing];  // of the warps' rings
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t q_full[2], q_free[2], o_free, drain;
    alignas(16) float unit[2][kUnitRows];               // what a row of queries was divided by
    // the columns of a unit: scores into base 2, the maximum, what is added in base 2, what results are worth under a new one
    alignas(16) float c[kUnitRows], m[kUnitRows], minus[kUnitRows], f[kUnitRows];
    float warp_max[4][kUnitRows], warp_sum[4][kUnitRows];
    uint32_t tmem;
    int none;                                           // a column has no maximum yet
    int abort;
};

// The queries of a unit by two warps, rows past its last zeros, in the places where
// the tensor core reads them (128-byte swizzle).  BF16 becomes F16 by a power of two
// for each row; D / 8 threads have a row.
template <bool kBf16, int D>
__device__ __forceinline__ void lay_queries(const AttendParams& p, const Piece& x, uint32_t to, float* unit, int t) {
    using T = typename Half<kBf16>::T;
    constexpr int kChunks = D / 8, kAtOnce = kQueryWarps * 32 / kChunks, kTurns = kUnitRows / kAtOnce;
    const int ch = t % kChunks, rows = x.rows * p.share;
    uint4 w[kTurns];
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int row = k * kAtOnce + t / kChunks, per = (row * p.share_inv) >> 16, head = row - per * p.share;
        w[k] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows)
            w[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.q) + (long long)(x.row + per) * p.q_stride +
                                                   (long long)(x.kvh * p.share + head) * D + ch * 8);
    }
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int row = k * kAtOnce + t / kChunks;
        if constexpr (kBf16) {
            float q[8];
            widen8<true>(w[k], q);
            float top = fabsf(q[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, fabsf(q[e]));
#pragma unroll
            for (int o = kChunks / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            const float2 lift = lift_of(top);
            if (ch == 0) unit[row] = lift.y;
            w[k] = make_uint4(Half<false>::pack(q[0] * lift.x, q[1] * lift.x), Half<false>::pack(q[2] * lift.x, q[3] * lift.x),
                              Half<false>::pack(q[4] * lift.x, q[5] * lift.x), Half<false>::pack(q[6] * lift.x, q[7] * lift.x));
        } else if (ch == 0) {
            unit[row] = 1.0f;
        }
        tc::store16(to + (ch >> 3) * (kUnitRows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), w[k]);
    }
    tc::fence_async_shared();
}

// A warp's chunks of the run, fetched into its ring ahead of their turn: every
// eighth of a piece.  A chunk lies on one page, or on two or four: a lane has the
// copies of each.  The codes are turned within a token (64- or 32-byte swizzle), so
// that the lanes that read a part of eight tokens meet every bank once.
template <int D>
struct Fetch {
    using C = Cfg4<D>;
    const int* table;
    long long token;
    int kvh, tokens, next;           // of the piece: its tokens, the chunk that comes next
    int page;                        // of this lane's part of it, -1 for none
    uint32_t n_piece, fetched;
    bool ended;
    __device__ __forceinline__ int page_of(const AttendParams& p, int chunk, int part) const {
        const int t = chunk * kChunk + part;
        return part < kChunk && t < tokens ? table[(token + t) >> p.page_shift] : -1;
    }
    // The next chunk, of at most kAhead pieces past the `taken` that the warp has come to (the planning warp waits for it).
    // False when a wait ran out.
    __device__ __forceinline__ bool chunk(const AttendParams& p, const CUtensorMap* k_map, const CUtensorMap* v_map, Ctl4<D>* ctl, unsigned char* ring,
                                          int worker, uint32_t taken, unsigned long long limit) {
        const int lane = threadIdx.x & 31;
        const int shift = p.page_shift < 5 ? p.page_shift : 5, part = lane << shift;  // tokens of a copy; this lane's first
        while (!ended && next * kChunk >= tokens) {
            if (n_piece >= taken + kAhead) return true;
            const uint32_t i = n_piece % kPieces;
            if (!tc::warp_wait(&ctl->piece_full[i], n_piece / kPieces & 1u, limit, &ctl->abort)) return false;
            ++n_piece;
            const Piece& x = ctl->piece[i];
            if (x.rows == 0) {
                ended = true;
                break;
            }
            table = ctl->pages[i].table, token = ctl->pages[i].token, kvh = x.kvh;
            tokens = x.left < x.tiles * kKTile ? x.left : x.tiles * kKTile;
            next = worker;
            page = page_of(p, next, part);
        }
        if (ended) return true;
        const int t = next * kChunk + part, mine = page;
        next += kExpandWarps;
        page = page_of(p, next, part);  // before it is needed
        const bool exists = part < kChunk && t < tokens, good = mine >= 0 && mine < p.num_pages;
        const uint32_t at = fetched % C::kRing;
        unsigned char* to = ring + at * C::kBytes;
        uint64_t* bar = &ctl->chunk_full[worker][at];
        const unsigned copies = __ballot_sync(kFull, exists), sound = __ballot_sync(kFull, exists && good);
        if (exists && !good) {  // a page that does not exist reads as zeros
            atomicOr(p.status, kStatusBadPage);
            for (int i = 0; i < D / kBlock4 << shift; i += 4) {
                *reinterpret_cast<uint32_t*>(to + 2 * C::kCodes + part * (D / kBlock4) + i) = 0u;
                *reinterpret_cast<uint32_t*>(to + 2 * C::kCodes + C::kScales + part * (D / kBlock4) + i) = 0u;
            }
            tc::fence_async_shared();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_expect(bar, (uint32_t)(__popc(copies) * D + __popc(sound) * (D / 8)) << shift);
        __syncwarp();
        if (exists) {
            const int y = (int)((token + t) & ((1 << p.page_shift) - 1));
            unsigned char* codes = to + part * (D / 2);
            const int where = good ? mine : (int)p.num_pages;  // outside the map: zeros
            tc::tma_load_4d(codes, k_map, bar, 0, y, kvh, where);
            tc::tma_load_4d(codes + C::kCodes, v_map, bar, 0, y, kvh, where);
            if (good) {
                const long long slot = (((long long)mine * p.kv_heads + kvh) << p.page_shift) + y;
                const uint32_t scales = tc::smem_addr(to) + 2 * C::kCodes + part * (D / kBlock4);
                tc::bulk_load(scales, p.k_scales + slot * (D / kBlock4), D / kBlock4 << shift, bar);
                tc::bulk_load(scales + C::kScales, p.v_scales + slot * (D / kBlock4), D / kBlock4 << shift, bar);
            }
        }
        ++fetched;
        return true;
    }
    // As many as have room, `done` of them used.  False when a wait ran out.
    __device__ __forceinline__ bool fill(const AttendParams& p, const CUtensorMap* k_map, const CUtensorMap* v_map, Ctl4<D>* ctl, unsigned char* ring,
                                         int worker, uint32_t done, uint32_t taken, unsigned long long limit) {
        while (fetched - done < C::kRing) {
            const uint32_t before = fetched;
            if (!chunk(p, k_map, v_map, ctl, ring, worker, taken, limit)) return false;
            if (fetched == before) break;
        }
        return true;
    }
};

// The scales of a thread's token, each as a pair of F16; zeros where `zero`.
template <int D>
__device__ __forceinline__ void token_scales(const unsigned char* scales, bool zero, uint32_t (&e)[D / 16]) {
    const int lane = threadIdx.x & 31;
    uint32_t s[D / 64];
    if constexpr (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(scales + lane * 8);
        s[0] = w.x, s[D / 64 - 1] = w.y;
    } else {
        s[0] = *reinterpret_cast<const uint32_t*>(scales + lane * 4);
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        if (zero) s[i] = 0u;
        const uint32_t a = widen_scales(s[i]), b = widen_scales(s[i] >> 16);
        e[4 * i] = __byte_perm(a, 0, 0x1010), e[4 * i + 1] = __byte_perm(a, 0, 0x3232);
        e[4 * i + 2] = __byte_perm(b, 0, 0x1010), e[4 * i + 3] = __byte_perm(b, 0, 0x3232);
    }
}

// Sixteen bytes of a thread's token: 32 codes.
template <int D>
__device__ __forceinline__ uint4 token_codes(const unsigned char* codes, int part) {
    const int lane = threadIdx.x & 31;
    return *reinterpret_cast<const uint4*>(codes + lane * (D / 2) + (part ^ (D == 128 ? lane >> 1 & 3 : lane >> 2 & 1)) * 16);
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kBlockThreads, 1)
    lp_attend4_kernel(const AttendParams p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using C = Cfg4<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl4<D>* ctl = reinterpret_cast<Ctl4<D>*>(smem + C::kCtl);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, as the compiler sees
    const unsigned long long limit = p.timeout_ns;
    if (warp == kBlockWarps - 1) {  // while the kernel ahead still runs
        if (lane < kPieces) tc::mbar_init(&ctl->piece_full[lane], 1), tc::mbar_init(&ctl->piece_empty[lane], kPieceReaders);
        for (int i = lane; i < kExpandWarps * C::kRing; i += 32) tc::mbar_init(&ctl->chunk_full[0][i], 1);
        if (lane < 2) {
            tc::mbar_init(&ctl->k_full[lane], 4);
            tc::mbar_init(&ctl->k_empty[lane], 1);
            tc::mbar_init(&ctl->v_full[lane], 4);
            tc::mbar_init(&ctl->v_empty[lane], 1);
            tc::mbar_init(&ctl->s_full[lane], 1);
            tc::mbar_init(&ctl->s_empty[lane], 4);
            tc::mbar_init(&ctl->p_full[lane], 4);
            tc::mbar_init(&ctl->p_empty[lane], 1);
            tc::mbar_init(&ctl->q_full[lane], kQueryWarps);
            tc::mbar_init(&ctl->q_free[lane], 1 + 4);
        }
        if (lane == 0) {
            tc::mbar_init(&ctl->o_free, 4);
            tc::mbar_init(&ctl->drain, 1);
            ctl->abort = 0;
        }
        tc::fence_async_shared();
    }
    if (tid == 0) tc::prefetch_map(&k_map), tc::prefetch_map(&v_map);
    // so far nothing of what earlier kernels write; the join may start once that is there, and waits for this grid's end by itself
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 1) tc::tmem_alloc(&ctl->tmem, kTmemCols);  // not held while waiting: the kernel ahead may need it to end
    Runs runs[2];  // of prefixes, of groups
    const bool any = plan_run<Columns>(p, ctl, runs);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = ctl->tmem;
    if (!any) {
        if (tid == 0) p.columns.gave_up[blockIdx.x] = 0;
        if (warp == 1) tc::tmem_dealloc(tmem, kTmemCols);
        return;
    }
    volatile int* abort = &ctl->abort;
    // test hook: nothing arrives on `drain` before the end, so this wait runs out
    if (p.force_timeout) tc::warp_wait(&ctl->drain, 0, limit, abort);

    Piece x;
    bool ok = !p.force_timeout;
    uint32_t n_piece = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = tc::warp_wait(bar, parity, limit, abort); };
    auto arrive = [&](uint64_t* bar) {  // of the warp, after what all its lanes did
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };
    // the next piece, from the planning warp; false at the end of the run
    auto next_piece = [&]() {
        const uint32_t i = n_piece % kPieces;
        if (!wait(&ctl->piece_full[i], n_piece / kPieces & 1u)) return false;
        x = ctl->piece[i];
        arrive(&ctl->piece_empty[i]);
        ++n_piece;
        return x.rows > 0;
    };

    if (warp >= kFirstSoftmax) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---- softmax.  The four warps meet at barriers of their own, which have no limit: they part only after a vote, so
        // that none is left waiting.
        const int t = tid - kFirstSoftmax * 32, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)quarter << 21;
        auto meet = [&]() { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        auto vote = [&](bool mine) {
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, 1, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                : "=r"(r)
                : "r"((uint32_t)mine)
                : "memory");
            return r != 0u;
        };
        uint32_t use[2] = {0, 0};
        for (bool going = true; going;) {
            const bool more = next_piece();
            if (vote(!ok) || !more) break;
            const uint32_t n = n_piece - 1;
            const int rows = x.rows * p.share, blocks = (rows + 15) >> 4;
            ok = wait(&ctl->q_full[n & 1u], n >> 1 & 1u);
            if (t < kUnitRows) {
                // finite and above 0, so that a masked score stays -infinity and one of 0 stays 0
                ctl->c[t] = fminf(fmaxf(p.scale * kLog2e * p.k_factor * ctl->unit[n & 1u][t], 0x1p-126f), 0x1p127f);
                ctl->m[t] = kNegInf, ctl->minus[t] = 0.0f;
            }
            arrive(&ctl->q_free[n & 1u]);
            float l[kUnitRows];
#pragma unroll
            for (int e = 0; e < kUnitRows; ++e) l[e] = 0.0f;
            bool raise = true;  // the first tile sets the maxima
            meet();
            for (int i = 0; i < x.tiles; ++i) {
                const int b = i & 1;
                const uint32_t u = b == 0 ? use[0]++ : use[1]++;
                if (ok) wait(&ctl->s_full[b], u & 1u);
                tc::fence_after();
                uint32_t s[2][16];
                tc::tmem_ld16(tmem + lanes + kColS + b * kUnitRows, s[0]);
                if (blocks > 1) tc::tmem_ld16(tmem + lanes + kColS + b * kUnitRows + 16, s[1]);
                tc::wait_ld();
                tc::tie(s[0]);
                tc::tie(s[1]);
                tc::fence_before();
                arrive(&ctl->s_empty[b]);
                const int have = x.left - i * kKTile;
                if (t >= have) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[0][e] = s[1][e] = __float_as_uint(kNegInf);
                }
                float y[2][16];
                auto base2 = [&](int k) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(&ctl->c[k * 16 + e]), d = *reinterpret_cast<const float4*>(&ctl->minus[k * 16 + e]);
                        y[k][e] = fmaf(__uint_as_float(s[k][e]), c.x, d.x), y[k][e + 1] = fmaf(__uint_as_float(s[k][e + 1]), c.y, d.y);
                        y[k][e + 2] = fmaf(__uint_as_float(s[k][e + 2]), c.z, d.z), y[k][e + 3] = fmaf(__uint_as_float(s[k][e + 3]), c.w, d.w);
                    }
                };
                auto most = [&](int k, float top) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) top = fmaxf(top, y[k][e]);
                    return top;
                };
                base2(0);
                float top = most(0, kNegInf);
                if (blocks > 1) base2(1), top = most(1, top);
                if (vote(raise || top > kBias + kRescale || !ok)) {
                    if (vote(!ok)) {
                        going = false;
                        break;
                    }
                    // the tile's maximum of each column: of the warp's tokens (by the order of integers), then of the four warps'
                    int mine = 0;
                    auto order = [](int v) { return v ^ (v >> 31 & 0x7FFFFFFF); };
#pragma unroll
                    for (int e = 0; e < kUnitRows; ++e) {
                        if (e >= 16 && blocks == 1) continue;
                        const int r = __reduce_max_sync(kFull, order((int)s[e / 16][e % 16]));
                        if (lane == e) mine = r;
                    }
                    ctl->warp_max[quarter][lane] = __int_as_float(order(mine));
                    meet();
                    if (t < kUnitRows) {
                        const float high = fmaxf(fmaxf(ctl->warp_max[0][t], ctl->warp_max[1][t]), fmaxf(ctl->warp_max[2][t], ctl->warp_max[3][t]));
                        const float c = ctl->c[t], m = ctl->m[t];
                        float f = 1.0f;
                        if (t < blocks * 16 && (m == kNegInf ? high > kNegInf : high * c > m * c + kRescale)) {
                            const float minus = kBias - high * c;
                            if (m != kNegInf) f = ex2(minus - ctl->minus[t]);
                            ctl->m[t] = high, ctl->minus[t] = minus;
                        }
                        ctl->f[t] = f;
                        const bool none = __any_sync(kFull, t < blocks * 16 && ctl->m[t] == kNegInf);
                        if (t == 0) ctl->none = none;
                    }
                    meet();
                    raise = ctl->none != 0;
                    if (i > 0) {  // the result so far
                        const int before = b ^ 1;
                        wait(&ctl->p_empty[before], ((before == 0 ? use[0] : use[1]) - 1) & 1u);
                        tc::fence_after();
#pragma unroll 1
                        for (int k = 0; k < blocks; ++k) {
                            uint32_t o[16];
                            tc::tmem_ld16(tmem + lanes + kColO + k * 16, o);
                            tc::wait_ld();
                            tc::tie(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ctl->f[k * 16 + e]);
                            tc::tmem_st16(tmem + lanes + kColO + k * 16, o);
                        }
                        tc::wait_st();
                        tc::fence_before();
                    }
#pragma unroll
                    for (int e = 0; e < kUnitRows; ++e) l[e] *= ctl->f[e];
                    base2(0);
                    if (blocks > 1) base2(1);
                }
                uint4 w[4];
                auto weigh = [&](int k) {
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = ex2(y[k][2 * e]), d = ex2(y[k][2 * e + 1]);
                        l[k * 16 + 2 * e] += a, l[k * 16 + 2 * e + 1] += d;
                        h[e] = Half<false>::pack(a, d);
                    }
                    w[2 * k] = make_uint4(h[0], h[1], h[2], h[3]), w[2 * k + 1] = make_uint4(h[4], h[5], h[6], h[7]);
                };
                weigh(0);
                if (blocks > 1) weigh(1);
                if (ok) wait(&ctl->p_empty[b], (u & 1u) ^ 1u);
                const uint32_t to = tc::smem_addr(smem + C::kAtProbs + b * C::kProbs) + t * 128;
                tc::store16(to + ((t & 7) << 4), w[0]);
                tc::store16(to + ((1 ^ (t & 7)) << 4), w[1]);
                if (blocks > 1) tc::store16(to + ((2 ^ (t & 7)) << 4), w[2]), tc::store16(to + ((3 ^ (t & 7)) << 4), w[3]);
                tc::fence_async_shared();
                arrive(&ctl->p_full[b]);
            }
            if (!going) break;
            const int last = (x.tiles - 1) & 1;
            if (ok) wait(&ctl->p_empty[last], ((last == 0 ? use[0] : use[1]) - 1) & 1u);  // the products are in
            tc::fence_after();
            const int d = quarter * 32 + lane;  // lane of the head
#pragma unroll 1
            for (int k = 0; k < blocks; ++k) {
                uint32_t o[16];
                tc::tmem_ld16(tmem + lanes + kColO + k * 16, o);
                tc::wait_ld();
                tc::tie(o);
                if (d < D && x.part >= 0) {
                    float* dst = p.columns.part_o + part_chunk<D>(x.part, x.part_stride, k * 16, d >> 2) * 4 + (d & 3);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (k * 16 + e < rows) dst[e * 4] = __uint_as_float(o[e]);
                }
            }
            tc::fence_before();
            arrive(&ctl->o_free);
            // the columns' sums over the warp: half of the columns and half of the lanes at a time
            auto fold = [&](int k) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = l[k * 16 + e];
#pragma unroll
                for (int o = 16, half = 8; half > 0; o >>= 1, half >>= 1) {
#pragma unroll
                    for (int e = 0; e < half; ++e) {
                        const bool up = (lane & o) != 0;
                        const float give = up ? v[e] : v[e + half], keep = up ? v[e + half] : v[e];
                        v[e] = keep + __shfl_xor_sync(kFull, give, o);
                    }
                }
                v[0] += __shfl_xor_sync(kFull, v[0], 1);
                if ((lane & 1) == 0) ctl->warp_sum[quarter][k * 16 + (lane >> 1)] = v[0];
            };
            fold(0);
            if (blocks > 1) fold(1);
            meet();
            if (t < rows && x.part >= 0)
                p.columns.part_ml[x.part + t] = make_float2(ctl->m[t] == kNegInf ? kNegInf : -ctl->minus[t],
                                                            (ctl->warp_sum[0][t] + ctl->warp_sum[1][t]) + (ctl->warp_sum[2][t] + ctl->warp_sum[3][t]));
        }
    } else if (warp >= kFirstExpand) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
        // ---- codes to F16: 32 tokens of every other tile
        const int worker = warp - kFirstExpand, quarter = worker & 3, b = worker >> 2;
        const uint32_t keys = tmem + ((uint32_t)quarter << 21) + kColK + b * (D / 2);
        const int row = quarter * 32 + lane;
        const uint32_t values = tc::smem_addr(smem + b * C::kValues) + row * 128;
        unsigned char* ring = smem + C::kAtRing + worker * C::kRing * C::kBytes;
        Fetch<D> fetch = {};
        uint32_t done = 0, use = 0;
        // The fetches look at every piece before this loop takes it: its place may then be another's.
        while (ok && (ok = fetch.fill(p, &k_map, &v_map, ctl, ring, worker, done, n_piece + 1, limit)) && next_piece()) {
            const int tokens = x.left < x.tiles * kKTile ? x.left : x.tiles * kKTile;
            for (int i = b; i < x.tiles; i += 2, ++use) {
                const int have = tokens - i * kKTile - quarter * 32;  // of this warp's
                const unsigned char* chunk = ring + done % C::kRing * C::kBytes;
                if (have > 0) {
                    if (!(ok = fetch.fill(p, &k_map, &v_map, ctl, ring, worker, done, n_piece, limit))) break;
                    if (!wait(&ctl->chunk_full[worker][done % C::kRing], done / C::kRing & 1u)) break;
                }
                if (!wait(&ctl->k_empty[b], (use & 1u) ^ 1u)) break;
                if (have > 0) {
                    tc::fence_after();
                    uint32_t e[D / 16];
                    token_scales<D>(chunk + 2 * C::kCodes, false, e);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        uint32_t k[32];
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            const uint4 w = token_codes<D>(chunk, 2 * h + part);
                            const uint32_t codes[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t v[4];
                                widen_codes(codes[j], v);
#pragma unroll
                                for (int q = 0; q < 4; ++q) k[part * 16 + j * 4 + q] = mul2(v[q], e[h * 4 + part * 2 + (j >> 1)]);
                            }
                        }
                        tc::tmem_st32(keys + h * 32, k);
                    }
                    tc::wait_st();
                    tc::fence_before();
                }
                arrive(&ctl->k_full[b]);
                if (!wait(&ctl->v_empty[b], (use & 1u) ^ 1u)) break;
                if (have > 0) {
                    uint32_t e[D / 16];
                    token_scales<D>(chunk + 2 * C::kCodes + C::kScales, lane >= have, e);  // what lies past the tokens may be NaN, and 0 * v has to stay 0
#pragma unroll
                    for (int part = 0; part < D / 32; ++part) {
                        const uint4 w = token_codes<D>(chunk + C::kCodes, part);
                        const uint32_t codes[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int ch = part * 4 + j;
                            uint32_t v[4];
                            widen_codes(codes[j], v);
                            tc::store16(values + (ch >> 3) * (kKTile * 128) + (((ch & 7) ^ (row & 7)) << 4),
                                        make_uint4(mul2(v[0], e[ch / 2]), mul2(v[1], e[ch / 2]), mul2(v[2], e[ch / 2]), mul2(v[3], e[ch / 2])));
                        }
                    }
                    tc::fence_async_shared();
                    ++done;
                }
                arrive(&ctl->v_full[b]);
            }
        }
        int none = 0;  // no copy outlives the block, whatever its readers did
        for (uint32_t i = done; i < fetch.fetched; ++i) tc::mbar_wait(&ctl->chunk_full[worker][i % C::kRing], i / C::kRing & 1u, limit, &none);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 0) {
            // ---- the run's pieces
            Walk<Columns> walk;
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
            for (bool more = ok; more; ++n_piece) {
                more = walk.next(p, x);
                const uint32_t i = n_piece % kPieces;
                if (!wait(&ctl->piece_empty[i], (n_piece / kPieces & 1u) ^ 1u)) break;
                if (lane == 0) {
                    ctl->piece[i] = x;
                    ctl->pages[i] = Pages{walk.table, walk.token};
                    tc::mbar_arrive(&ctl->piece_full[i]);
                }
            }
        } else if (warp == 1) {
            // ---- products, the scores of a tile ahead of the results of the one before; by an elected lane
            const uint32_t one = tc::elect_one();
            const uint32_t tm = __shfl_sync(kFull, tmem, 0);
            const uint64_t q_desc = tc::make_desc(tc::smem_addr(smem + C::kAtQueries), 16, 1024);
            const uint64_t v_desc = tc::make_desc(tc::smem_addr(smem), kKTile * 128, 1024), p_desc = tc::make_desc(tc::smem_addr(smem + C::kAtProbs), 16, 1024);
            uint32_t use_k[2] = {0, 0}, use_v[2] = {0, 0};
            while (ok && next_piece()) {
                const uint32_t n = n_piece - 1;
                const int tiles = __shfl_sync(kFull, x.tiles, 0), tokens = __shfl_sync(kFull, x.left, 0);
                const int columns = __shfl_sync(kFull, ((x.rows * p.share + 15) >> 4) * 16, 0);
                const uint32_t idesc_s = tc::make_idesc(false, false, kKTile, columns), idesc_o = tc::make_idesc(false, true, kKTile, columns) | tc::kAMnMajor;
                const uint64_t q = q_desc + (n & 1u) * (C::kQuery >> 4);
                if (!wait(&ctl->q_full[n & 1u], n >> 1 & 1u)) break;
                auto scores = [&](int i) {
                    const int b = i & 1;
                    const uint32_t u = b == 0 ? use_k[0]++ : use_k[1]++;
                    if (!wait(&ctl->k_full[b], u & 1u) || !wait(&ctl->s_empty[b], (u & 1u) ^ 1u)) return false;
                    tc::fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc::mma_ts(tm + kColS + b * kUnitRows, tm + kColK + b * (D / 2) + k * 8, q + (uint64_t)(((k / 4) * (kUnitRows * 128) + (k % 4) * 32) >> 4), idesc_s, k > 0, one);
                    tc::commit(&ctl->s_full[b], one);
                    tc::commit(&ctl->k_empty[b], one);
                    return true;
                };
                if (!scores(0)) break;
                for (int i = 0; i < tiles; ++i) {
                    if (i + 1 < tiles && !scores(i + 1)) break;
                    if (i == (tiles > 1 ? tiles - 2 : 0)) tc::commit(&ctl->q_free[n & 1u], one);  // the last scores are on their way
                    const int b = i & 1, have = tokens - i * kKTile;
                    const uint32_t u = b == 0 ? use_v[0]++ : use_v[1]++;
                    if (!wait(&ctl->v_full[b], u & 1u) || !wait(&ctl->p_full[b], u & 1u) || (i == 0 && !wait(&ctl->o_free, (n & 1u) ^ 1u))) break;
                    tc::fence_after();
                    const uint64_t v = v_desc + (uint64_t)(b * C::kValues >> 4), pr = p_desc + (uint64_t)(b * C::kProbs >> 4);
                    const int steps = have >= kKTile ? kKTile / 16 : (have + 15) >> 4;
                    for (int k = 0; k < steps; ++k)
                        tc::mma_ss(tm + kColO, v + (uint64_t)(k * 2048 >> 4), pr + (uint64_t)(k * 2048 >> 4), idesc_o, i > 0 || k > 0, one);
                    tc::commit(&ctl->v_empty[b], one);
                    tc::commit(&ctl->p_empty[b], one);
                }
            }
            int none = 0;  // no product outlives the block
            tc::commit(&ctl->drain, one);
            tc::mbar_wait(&ctl->drain, 0, limit, &none);
            __syncwarp();
        } else {
            // ---- a unit's queries, ahead of the products
            while (ok && next_piece()) {
                const uint32_t n = n_piece - 1;
                if (!wait(&ctl->q_free[n & 1u], (n >> 1 & 1u) ^ 1u)) break;
                lay_queries<kBf16, D>(p, x, tc::smem_addr(smem + C::kAtQueries + (n & 1u) * C::kQuery), ctl->unit[n & 1u], (warp - 2) * 32 + lane);
                arrive(&ctl->q_full[n & 1u]);
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        p.columns.gave_up[blockIdx.x] = *abort;
        if (*abort != 0) atomicOr(p.status, kStatusAttnTimeout);
    }
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
constexpr int smem_bytes4() { return Cfg4<D>::kCtl + (int)sizeof(Ctl4<D>); }

template <bool kBf16, int D>
cudaError_t prepare4() {
    static_assert(smem_bytes4<D>() <= 232448, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(lp_attend4_kernel<kBf16, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes4<D>());
    return e == cudaSuccess ? prepare_join<kBf16, D, true>() : e;
}

template <bool kBf16, int D>
cudaError_t launch4(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
    // Each kernel is launched while the one before still runs, and waits for its end before it reads what that writes.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.grid);
    lc.blockDim = dim3(kBlockThreads);
    lc.dynamicSmemBytes = smem_bytes4<D>();
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    if (runs_columns(p)) e = cudaLaunchKernelEx(&lc, lp_attend4_kernel<kBf16, D>, p, k_map, v_map);
    if (e == cudaSuccess && runs_pairs(p)) e = launch_attend4_pairs(p, kBf16 ? 1 : 2, D, lc);
    return e == cudaSuccess ? launch_join<kBf16, D, true>(p, lc) : e;
}

}  // namespace

int pick_wide(const AttendParams& p) {
    if (p.rows_per_unit == 0) return kWidePrefixes | kWideGroups;
    const long long rows = (long long)p.rows * p.share;
    return (rows > (long long)kUnitRows * p.P ? kWidePrefixes : 0) | (rows > (long long)kUnitRows * p.G ? kWideGroups : 0);
}

cudaError_t prepare_attend4(int dtype, int head_dim) {
    const cudaError_t e = prepare_attend4_pairs(dtype, head_dim);
    if (e != cudaSuccess) return e;
    if (dtype == 1) return head_dim == 128 ? prepare4<true, 128>() : prepare4<true, 64>();
    return head_dim == 128 ? prepare4<false, 128>() : prepare4<false, 64>();
}

cudaError_t launch_attend4(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, int dtype, int head_dim,
                           cudaStream_t stream) {
    if (dtype == 1) return head_dim == 128 ? launch4<true, 128>(p, k_map, v_map, stream) : launch4<true, 64>(p, k_map, v_map, stream);
    return head_dim == 128 ? launch4<false, 128>(p, k_map, v_map, stream) : launch4<false, 64>(p, k_map, v_map, stream);
}

}  // namespace lp
