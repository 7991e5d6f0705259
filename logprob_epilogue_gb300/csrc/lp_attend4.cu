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
// the tensor core's time goes by the few columns.  A piece's even tiles and its odd
// ones are two streams of their own, each with its maxima, sums and result: two parts
// for the join.
//
// Block (one per SM, 20 warps): warp 0 splits the work, warps 1 and 2 issue the
// products of a stream each, warps 0 and 3 fetch a stream's tiles by TMA into a ring
// (54 KiB), warp 3 also brings the units' queries.  Of each stream, four warps expand its tiles, a token per thread
// (keys into tensor memory, values into shared memory, F16), and four are its softmax,
// a token per thread.  A column's maximum is one for all 128 threads: it holds until a
// score is 2^8 above it, which a vote finds, and only then are the tokens' maxima
// compared.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstddef>

#include "lp_join.h"
#include "lp_split.h"
#include "lp_tc.h"

namespace lp {
namespace {

constexpr float kRescale = 8.0f;  // growth of the maximum (log2) that moves it
// Probabilities are lifted by 2^6 (at most 2^14 then): F16 keeps those above 2^-30 of the largest.
constexpr float kBias = 6.0f;
constexpr int kBlockThreads = 640, kBlockWarps = kBlockThreads / 32;
constexpr int kFirstExpand = 4, kFirstSoftmax = 12;  // warps: four of stream 0, four of stream 1
// Registers: the split's sum is what the block is launched with, 640 x 96.
constexpr int kRegsLaunch = 96, kRegsExpand = 88, kRegsSoftmax = 120, kRegsOther = 64;
static_assert(2 * kRegsExpand + 2 * kRegsSoftmax + kRegsOther <= 5 * kRegsLaunch, "register split");
// Tensor memory columns, of each stream: a tile of keys, one of scores, the result.
constexpr uint32_t kTmemCols = 256, kColK = 0, kColS = 128, kColO = 192;

template <int D>
struct Cfg4 {
    static constexpr int kValues = kKTile * D * 2;              // a tile of values, F16
    static constexpr int kProbs = kKTile * 128;                 // a tile of probabilities: 32 columns of 64
    static constexpr int kQuery = kUnitRows * D * 2;            // a unit's queries
    static constexpr int kCodes = kKTile * D / 2, kScales = kKTile * D / kBlock4;
    static constexpr int kBytes = 2 * (kCodes + kScales);       // K and V of a tile: codes, then scales
    static constexpr int kRing = 3 * 128 / D;                   // a stream's tiles
    static constexpr int kAtProbs = 2 * kValues, kAtQueries = kAtProbs + 2 * kProbs, kAtRing = kAtQueries + 2 * kQuery;
    static constexpr int kCtl = kAtRing + 2 * kRing * kBytes;
};

constexpr int kPieces = 8;  // pieces the planning warp may be ahead
constexpr int kPieceReaders = kBlockWarps - 1;  // all but the planning one

// Where the tokens of a piece lie.
struct Pages {
    const int* table;
    long long token;  // the first
};

// The columns of a unit in a stream: the maximum, what is added in base 2, what results are worth under a new one.
struct alignas(16) Maxima {
    float m[kUnitRows], minus[kUnitRows], f[kUnitRows];
    float warp_max[4][kUnitRows], warp_sum[4][kUnitRows];
    int none;  // a column has no maximum yet
};

template <int D>
struct Ctl4 : PlanCtl<Columns> {
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    Pages pages[kPieces];
    uint64_t tile_full[2][Cfg4<D>::kRing], tile_empty[2][Cfg4<D>::kRing];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2], o_free[2];
    uint64_t q_full[2], q_free[2], drain;
    alignas(16) float unit[2][kUnitRows];  // what a row of queries was divided by
    alignas(16) float c[2][kUnitRows];     // of each stream: scores into base 2
    Maxima columns[2];
    uint32_t tmem;
    int abort;
};

// The queries of a unit by a warp, rows past its last up to sixteen zeros, in the
// places where the tensor core reads them (128-byte swizzle).  BF16 becomes F16 by a power of two for
// each row; D / 8 threads have a row.
template <bool kBf16, int D>
__device__ __forceinline__ void lay_queries(const AttendParams& p, const Piece& x, uint32_t to, float* unit) {
    using T = typename Half<kBf16>::T;
    constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks, kTurns = 8;
    const int lane = threadIdx.x & 31, ch = lane % kChunks, rows = x.rows * p.share;
    const T* src = reinterpret_cast<const T*>(p.q) + (long long)x.row * p.q_stride + (long long)x.kvh * p.share * D + ch * 8;
#pragma unroll 1
    for (int base = 0; base < ((rows + 15) & ~15); base += kTurns * kAtOnce) {
        uint4 w[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int row = base + k * kAtOnce + lane / kChunks, per = (row * p.share_inv) >> 16, head = row - per * p.share;
            w[k] = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows) w[k] = *reinterpret_cast<const uint4*>(src + per * p.q_stride + head * D);
        }
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int row = base + k * kAtOnce + lane / kChunks;
            if constexpr (kBf16) {
                // the largest magnitude: that of BF16 is its order as an integer without the sign
                const uint32_t m = 0x7FFF7FFFu;
                uint32_t top = __vmaxu2(__vmaxu2(w[k].x & m, w[k].y & m), __vmaxu2(w[k].z & m, w[k].w & m));
#pragma unroll
                for (int o = kChunks / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, o));
                const uint32_t most = top >> 16 > (top & 0xFFFFu) ? top & 0xFFFF0000u : top << 16;
                const float2 lift = lift_of(__uint_as_float(most));
                if (ch == 0) unit[row] = lift.y;
                uint32_t a[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 q = Half<true>::unpack(a[e]);
                    a[e] = Half<false>::pack(q.x * lift.x, q.y * lift.x);
                }
                w[k] = make_uint4(a[0], a[1], a[2], a[3]);
            } else if (ch == 0) {
                unit[row] = 1.0f;
            }
            tc::store16(to + (ch >> 3) * (kUnitRows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), w[k]);
        }
    }
    tc::fence_async_shared();
}

// A sixteenth of a tile's way to F16: 32 lanes of a thread's token.  The copies turn
// a token's parts of 16 bytes (64- or 32-byte swizzle), so that the threads that read a
// part of eight tokens meet every bank once.
template <int D>
__device__ __forceinline__ void expand_part(const unsigned char* codes, const unsigned char* scales, int token, int part, bool exists, uint32_t (&h)[16]) {
    const uint4 w = *reinterpret_cast<const uint4*>(codes + token * (D / 2) + (part ^ (D == 128 ? token >> 1 & 3 : token >> 2 & 1)) * 16);
    uint32_t two = *reinterpret_cast<const uint16_t*>(scales + token * (D / kBlock4) + part * 2);
    if (!exists) two = 0u;
    two = widen_scales(two);
    const uint32_t e[2] = {__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232)}, c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t v[4];
        widen_codes(c[j], v);
#pragma unroll
        for (int q = 0; q < 4; ++q) h[j * 4 + q] = mul2(v[q], e[j >> 1]);
    }
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
        if (lane < 2 * C::kRing) tc::mbar_init(&ctl->tile_full[0][lane], 1), tc::mbar_init(&ctl->tile_empty[0][lane], 4);
        if (lane < 2) {
            tc::mbar_init(&ctl->k_full[lane], 4);
            tc::mbar_init(&ctl->k_empty[lane], 1);
            tc::mbar_init(&ctl->v_full[lane], 4);
            tc::mbar_init(&ctl->v_empty[lane], 1);
            tc::mbar_init(&ctl->s_full[lane], 1);
            tc::mbar_init(&ctl->s_empty[lane], 4);
            tc::mbar_init(&ctl->p_full[lane], 4);
            tc::mbar_init(&ctl->p_empty[lane], 1);
            tc::mbar_init(&ctl->o_free[lane], 4);
            tc::mbar_init(&ctl->q_full[lane], 1);
            tc::mbar_init(&ctl->q_free[lane], 2 + 8);
        }
        if (lane == 0) {
            tc::mbar_init(&ctl->drain, 2);
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
    auto wait2 = [&](uint64_t* a, uint32_t parity_a, uint64_t* b, uint32_t parity_b) { return ok = tc::warp_wait2(a, parity_a, b, parity_b, limit, abort); };
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
        // ---- softmax.  A stream's four warps meet at a barrier of their own, which has no limit: they part only after a
        // vote, so that none is left waiting.
        const int stream = (warp - kFirstSoftmax) >> 2, t = (tid - kFirstSoftmax * 32) & 127, quarter = warp & 3, id = 1 + stream;
        const uint32_t lanes = (uint32_t)quarter << 21, scores = tmem + lanes + kColS + stream * kUnitRows, result = tmem + lanes + kColO + stream * kUnitRows;
        const uint32_t probs = tc::smem_addr(smem + C::kAtProbs + stream * C::kProbs) + t * 128;
        Maxima& col = ctl->columns[stream];
        const float* scale2 = ctl->c[stream];
        auto meet = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); };
        auto vote = [&](bool mine) {
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, %2, 128, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                : "=r"(r)
                : "r"((uint32_t)mine), "r"(id)
                : "memory");
            return r != 0u;
        };
        uint32_t use = 0;  // the stream's tiles
        for (bool going = true; going;) {
            const bool more = next_piece();
            if (vote(!ok) || !more) break;
            const uint32_t n = n_piece - 1;
            const int rows = x.rows * p.share, blocks = (rows + 15) >> 4;
            ok = wait(&ctl->q_full[n & 1u], n >> 1 & 1u);
            if (t < kUnitRows) {
                // finite and above 0, so that a masked score stays -infinity and one of 0 stays 0
                ctl->c[stream][t] = fminf(fmaxf(p.scale * kLog2e * p.k_factor * ctl->unit[n & 1u][t], 0x1p-126f), 0x1p127f);
                col.m[t] = kNegInf, col.minus[t] = 0.0f;
            }
            arrive(&ctl->q_free[n & 1u]);
            const long long part = x.part + stream * x.part_stride;
            if (stream >= x.tiles) {  // no tile of this piece is this stream's
                if (t < rows && x.part >= 0) p.columns.part_ml[part + t] = make_float2(kNegInf, 0.0f);
                continue;
            }
            float l[kUnitRows];
#pragma unroll
            for (int e = 0; e < kUnitRows; ++e) l[e] = 0.0f;
            bool raise = true;  // the first tile sets the maxima
            meet();
            for (int i = stream; i < x.tiles; i += 2, ++use) {
                if (ok) wait2(&ctl->s_full[stream], use & 1u, &ctl->p_empty[stream], (use & 1u) ^ 1u);  // and the products before are in
                tc::fence_after();
                const bool exists = t < x.left - i * kKTile;
                float y[2][16];
                auto base2 = [&](int k) {  // scores of 16 columns, in base 2 and less the maximum
                    uint32_t s[16];
                    tc::tmem_ld16(scores + k * 16, s);
                    tc::wait_ld();
                    tc::tie(s);
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(scale2 + k * 16 + e), d = *reinterpret_cast<const float4*>(&col.minus[k * 16 + e]);
                        y[k][e] = exists ? fmaf(__uint_as_float(s[e]), c.x, d.x) : kNegInf;
                        y[k][e + 1] = exists ? fmaf(__uint_as_float(s[e + 1]), c.y, d.y) : kNegInf;
                        y[k][e + 2] = exists ? fmaf(__uint_as_float(s[e + 2]), c.z, d.z) : kNegInf;
                        y[k][e + 3] = exists ? fmaf(__uint_as_float(s[e + 3]), c.w, d.w) : kNegInf;
                    }
                };
                auto most = [&](int k, float top) {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) top = max3(y[k][e], y[k][e + 1], top);
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
#pragma unroll 1
                    for (int k = 0; k < blocks; ++k) {
                        uint32_t s[16];
                        tc::tmem_ld16(scores + k * 16, s);
                        tc::wait_ld();
                        tc::tie(s);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int r = __reduce_max_sync(kFull, order(exists ? (int)s[e] : __float_as_int(kNegInf)));
                            if (lane == k * 16 + e) mine = r;
                        }
                    }
                    col.warp_max[quarter][lane] = __int_as_float(order(mine));
                    meet();
                    if (t < kUnitRows) {
                        const float high = fmaxf(fmaxf(col.warp_max[0][t], col.warp_max[1][t]), fmaxf(col.warp_max[2][t], col.warp_max[3][t]));
                        const float c = scale2[t], m = col.m[t];
                        float f = 1.0f, now = m;
                        if (t < blocks * 16 && (m == kNegInf ? high > kNegInf : high * c > m * c + kRescale)) {
                            const float minus = kBias - high * c;
                            if (m != kNegInf) f = ex2(minus - col.minus[t]);
                            col.m[t] = now = high, col.minus[t] = minus;
                        }
                        col.f[t] = f;
                        const bool none = __any_sync(kFull, t < blocks * 16 && now == kNegInf);
                        if (t == 0) col.none = none;
                    }
                    meet();
                    raise = col.none != 0;
                    if (i > stream) {  // the result so far
#pragma unroll 1
                        for (int k = 0; k < blocks; ++k) {
                            uint32_t o[16];
                            tc::tmem_ld16(result + k * 16, o);
                            tc::wait_ld();
                            tc::tie(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * col.f[k * 16 + e]);
                            tc::tmem_st16(result + k * 16, o);
                        }
                        tc::wait_st();
                    }
#pragma unroll
                    for (int e = 0; e < kUnitRows; ++e) l[e] *= col.f[e];
                    base2(0);
                    if (blocks > 1) base2(1);
                }
                tc::fence_before();
                arrive(&ctl->s_empty[stream]);
                auto weigh = [&](int k) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = ex2(y[k][j * 8 + 2 * e]), d = ex2(y[k][j * 8 + 2 * e + 1]);
                            l[k * 16 + j * 8 + 2 * e] += a, l[k * 16 + j * 8 + 2 * e + 1] += d;
                            h[e] = Half<false>::pack(a, d);
                        }
                        tc::store16(probs + (((2 * k + j) ^ (t & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                    }
                };
                weigh(0);
                if (blocks > 1) weigh(1);
                tc::fence_async_shared();
                arrive(&ctl->p_full[stream]);
            }
            if (!going) break;
            if (ok) wait(&ctl->p_empty[stream], (use & 1u) ^ 1u);  // the products are in
            tc::fence_after();
            const int d = quarter * 32 + lane;  // lane of the head
#pragma unroll 1
            for (int k = 0; k < blocks; ++k) {
                uint32_t o[16];
                tc::tmem_ld16(result + k * 16, o);
                tc::wait_ld();
                tc::tie(o);
                if (d < D && x.part >= 0) {
                    float* dst = p.columns.part_o + part_chunk<D>(part, x.part_stride, k * 16, d >> 2) * 4 + (d & 3);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (k * 16 + e < rows) dst[e * 4] = __uint_as_float(o[e]);
                }
            }
            tc::fence_before();
            arrive(&ctl->o_free[stream]);
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
                if ((lane & 1) == 0) col.warp_sum[quarter][k * 16 + (lane >> 1)] = v[0];
            };
            fold(0);
            if (blocks > 1) fold(1);
            meet();
            if (t < rows && x.part >= 0)
                p.columns.part_ml[part + t] = make_float2(col.m[t] == kNegInf ? kNegInf : -col.minus[t],
                                                          (col.warp_sum[0][t] + col.warp_sum[1][t]) + (col.warp_sum[2][t] + col.warp_sum[3][t]));
        }
    } else if (warp >= kFirstExpand) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExpand));
        // ---- codes to F16: 32 tokens of the stream's tiles.  A tile's keys go before the values of the one before, whose
        // place may still be in use.
        const int stream = (warp - kFirstExpand) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t keys = tmem + ((uint32_t)quarter << 21) + kColK + stream * (D / 2);
        const uint32_t values = tc::smem_addr(smem + stream * C::kValues) + row * 128;
        const unsigned char* ring = smem + C::kAtRing + stream * C::kRing * C::kBytes;
        uint32_t use_k = 0, slot = 0, phase = 0;  // the stream's tiles; of its ring
        uint32_t use_v = 0, v_slot = 0;
        int pending = 0;  // tokens of the tile whose values are left
        auto expand_keys = [&]() {
            const unsigned char* tile = ring + slot * C::kBytes;
            if (!wait2(&ctl->tile_full[stream][slot], phase, &ctl->k_empty[stream], (use_k & 1u) ^ 1u)) return false;
            tc::fence_after();
            // (short code in loops: with many warps at many places, unrolled loops wait for their instructions)
#pragma unroll 1
            for (int part = 0; part < D / 32; ++part) {
                uint32_t h[16];
                expand_part<D>(tile, tile + 2 * C::kCodes, row, part, true, h);
                tc::tmem_st16(keys + part * 16, h);
            }
            tc::wait_st();
            tc::fence_before();
            arrive(&ctl->k_full[stream]);
            ++use_k;
            if (++slot == C::kRing) slot = 0, phase ^= 1u;
            return true;
        };
        auto expand_values = [&]() {
            const unsigned char* tile = ring + v_slot * C::kBytes + C::kCodes;
            if (!wait(&ctl->v_empty[stream], (use_v & 1u) ^ 1u)) return false;
#pragma unroll 1
            for (int part = 0; part < D / 32; ++part) {
                uint32_t h[16];
                expand_part<D>(tile, tile + C::kCodes + C::kScales, row, part, row < pending, h);  // what lies past the tokens may be NaN, and 0 * v has to stay 0
                const uint32_t to = values + (part >> 1) * (kKTile * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j) tc::store16(to + ((((part & 1) * 4 + j) ^ (row & 7)) << 4), make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]));
            }
            tc::fence_async_shared();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->tile_empty[stream][v_slot]), tc::mbar_arrive(&ctl->v_full[stream]);
            ++use_v;
            if (++v_slot == C::kRing) v_slot = 0;
            pending = 0;
            return true;
        };
        // One place for each, so that neither's code comes twice: an iteration takes a tile's keys, or the next piece, and then
        // the values that are due.
        int i = 0;
        x.tiles = 0;
        for (bool more = ok; more || pending > 0;) {
            bool due = pending > 0;
            int have = 0;
            if (i < x.tiles) {
                have = x.left - i * kKTile;
                i += 2;
                if (!expand_keys()) break;
            } else if (more) {
                // The next piece, where it is known: the values left may be what the others wait for.
                const uint32_t at = n_piece % kPieces;
                if (due && !__all_sync(kFull, tc::mbar_try_wait(&ctl->piece_full[at], n_piece / kPieces & 1u))) {
                    // they first
                } else {
                    more = next_piece();
                    if (!ok) break;
                    if (!more) x.tiles = 0;
                    i = stream;
                    if (i < x.tiles) continue;
                }
            }
            if (due && !expand_values()) break;
            if (have > 0) pending = have;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 0 || warp == 3) {
            // ---- a stream's tiles into its ring: a tile lies on one page, or on several, and a lane has the copies of each.
            // Warp 0 plans the pieces, each after a ring's worth of the one before; warp 3 brings their queries.
            const int stream = warp == 0 ? 0 : 1;
            const int shift = p.page_shift < 7 ? p.page_shift : 7, step = 1 << shift, part = lane << shift;  // tokens of a copy; this lane's first
            uint32_t filled = 0, slot = 0, phase = 1;
            Pages from = {nullptr, 0};
            auto page_of = [&](int i) {
                const int t = i * kKTile + part;
                return i < x.tiles && part < kKTile && t < x.left ? from.table[(from.token + t) >> p.page_shift] : -1;
            };
            auto fetch = [&](int i, int page) {
                const int t = i * kKTile + part;
                const bool exists = part < kKTile && t < x.left, good = page >= 0 && page < p.num_pages;
                const unsigned copies = __ballot_sync(kFull, exists), sound = __ballot_sync(kFull, exists && good);
                unsigned char* to = smem + C::kAtRing + (stream * C::kRing + slot) * C::kBytes;
                uint64_t* bar = &ctl->tile_full[stream][slot];
                if (!wait(&ctl->tile_empty[stream][slot], phase)) return false;
                if (copies != sound) {
                    if (exists && !good) {  // a page that does not exist reads as zeros
                        atomicOr(p.status, kStatusBadPage);
                        for (int k = 0; k < step * (D / kBlock4); k += 4) {
                            *reinterpret_cast<uint32_t*>(to + 2 * C::kCodes + part * (D / kBlock4) + k) = 0u;
                            *reinterpret_cast<uint32_t*>(to + 2 * C::kCodes + C::kScales + part * (D / kBlock4) + k) = 0u;
                        }
                        tc::fence_async_shared();
                    }
                    __syncwarp();
                }
                if (lane == 0) tc::mbar_expect(bar, (uint32_t)(__popc(copies) * D + __popc(sound) * (D / 8)) << shift);
                __syncwarp();
                if (exists) {
                    const int y = (int)((from.token + t) & ((1 << p.page_shift) - 1));
                    unsigned char* codes = to + part * (D / 2);
                    const int where = good ? page : (int)p.num_pages;  // outside the map: zeros
                    tc::tma_load_4d(codes, &k_map, bar, 0, y, x.kvh, where);
                    tc::tma_load_4d(codes + C::kCodes, &v_map, bar, 0, y, x.kvh, where);
                    if (good) {
                        const long long at = (((long long)page * p.kv_heads + x.kvh) << p.page_shift) + y;
                        const uint32_t scales = tc::smem_addr(to) + 2 * C::kCodes + part * (D / kBlock4);
                        tc::bulk_load(scales, p.k_scales + at * (D / kBlock4), D / kBlock4 << shift, bar);
                        tc::bulk_load(scales + C::kScales, p.v_scales + at * (D / kBlock4), D / kBlock4 << shift, bar);
                    }
                }
                ++filled;
                if (++slot == C::kRing) slot = 0, phase ^= 1u;
                return true;
            };
            if (warp == 0) {
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
                Piece y;
                auto plan = [&]() {  // the next piece into y, and to the other warps; false at the end of the run
                    const bool more = walk.next(p, y);
                    const uint32_t i = n_piece % kPieces;
                    if (!wait(&ctl->piece_empty[i], (n_piece / kPieces & 1u) ^ 1u)) return false;
                    if (lane == 0) {
                        ctl->piece[i] = y;
                        ctl->pages[i] = Pages{walk.table, walk.token};
                        tc::mbar_arrive(&ctl->piece_full[i]);
                    }
                    ++n_piece;
                    return more;
                };
                for (bool more = ok && plan(); more && ok;) {
                    x = y, from.table = walk.table, from.token = walk.token;
                    int page = page_of(0);
                    for (int i = 0, planned = 0; i < x.tiles || planned == 0; i += 2) {
                        if (i < x.tiles) {
                            const int now = page;
                            page = page_of(i + 2);  // a tile's page is read before the waits of the one before
                            if (!fetch(i, now)) break;
                        }
                        if (planned == 0 && (i + 2 >= x.tiles || i + 2 >= 2 * C::kRing)) planned = 1, more = plan();
                        if (!ok) break;
                    }
                }
            } else {
                while (ok) {
                    const uint32_t i0 = n_piece % kPieces;
                    if (!wait(&ctl->piece_full[i0], n_piece / kPieces & 1u)) break;
                    from = ctl->pages[i0];
                    if (!next_piece()) break;
                    int page = page_of(1);
                    const uint32_t n = n_piece - 1;
                    if (!wait(&ctl->q_free[n & 1u], (n >> 1 & 1u) ^ 1u)) break;
                    lay_queries<kBf16, D>(p, x, tc::smem_addr(smem + C::kAtQueries + (n & 1u) * C::kQuery), ctl->unit[n & 1u]);
                    arrive(&ctl->q_full[n & 1u]);
                    for (int i = 1; i < x.tiles; i += 2) {
                        const int now = page;
                        page = page_of(i + 2);
                        if (!fetch(i, now)) break;
                    }
                }
            }
            int none = 0;  // no copy outlives the block, whatever its readers did
            for (uint32_t i = filled > C::kRing ? filled - C::kRing : 0; i < filled; ++i)
                tc::mbar_wait(&ctl->tile_full[stream][i % C::kRing], i / C::kRing & 1u, limit, &none);
        } else {
            // ---- a stream's products, by an elected lane: the next tile's scores are on their way before its results are asked for
            const uint32_t one = tc::elect_one();
            const int stream = warp - 1;
            const uint32_t tm = __shfl_sync(kFull, tmem, 0), keys = tm + kColK + stream * (D / 2), score = tm + kColS + stream * kUnitRows, result = tm + kColO + stream * kUnitRows;
            const uint64_t q_desc = tc::make_desc(tc::smem_addr(smem + C::kAtQueries), 16, 1024);
            const uint64_t v = tc::make_desc(tc::smem_addr(smem + stream * C::kValues), kKTile * 128, 1024);
            const uint64_t pr = tc::make_desc(tc::smem_addr(smem + C::kAtProbs + stream * C::kProbs), 16, 1024);
            uint32_t use_k = 0, use_v = 0, use_o = 0;
            while (ok && next_piece()) {
                const uint32_t n = n_piece - 1;
                const int tiles = __shfl_sync(kFull, x.tiles, 0), tokens = __shfl_sync(kFull, x.left, 0);
                const int columns = __shfl_sync(kFull, ((x.rows * p.share + 15) >> 4) * 16, 0);
                const uint32_t idesc_s = tc::make_idesc(false, false, kKTile, columns), idesc_o = tc::make_idesc(false, true, kKTile, columns) | tc::kAMnMajor;
                const uint64_t q = q_desc + (n & 1u) * (C::kQuery >> 4);
                if (!wait(&ctl->q_full[n & 1u], n >> 1 & 1u)) break;
                auto scores = [&]() {
                    if (!wait2(&ctl->k_full[stream], use_k & 1u, &ctl->s_empty[stream], (use_k & 1u) ^ 1u)) return false;
                    ++use_k;
                    tc::fence_after();
#pragma unroll 2
                    for (int k = 0; k < D / 16; ++k)
                        tc::mma_ts(score, keys + k * 8, q + (uint64_t)(((k / 4) * (kUnitRows * 128) + (k % 4) * 32) >> 4), idesc_s, k > 0, one);
                    tc::commit(&ctl->s_full[stream], one);
                    tc::commit(&ctl->k_empty[stream], one);
                    return true;
                };
                if (stream < tiles && !scores()) break;
                for (int i = stream; i < tiles; i += 2) {
                    if (i + 2 < tiles && !scores()) break;
                    const int have = tokens - i * kKTile;
                    if (!wait2(&ctl->v_full[stream], use_v & 1u, &ctl->p_full[stream], use_v & 1u)) break;
                    ++use_v;
                    if (i == stream && !wait(&ctl->o_free[stream], (use_o++ & 1u) ^ 1u)) break;
                    tc::fence_after();
                    const int steps = have < kKTile ? (have + 15) >> 4 : kKTile / 16;
#pragma unroll 2
                    for (int k = 0; k < steps; ++k)
                        tc::mma_ss(result, v + (uint64_t)(k * 2048 >> 4), pr + (uint64_t)(k * 2048 >> 4), idesc_o, k > 0 || i != stream, one);
                    tc::commit(&ctl->v_empty[stream], one);
                    tc::commit(&ctl->p_empty[stream], one);
                }
                if (ok) tc::commit(&ctl->q_free[n & 1u], one);
            }
            int none = 0;  // no product outlives the block
            tc::commit(&ctl->drain, one);
            tc::mbar_wait(&ctl->drain, 0, limit, &none);
            __syncwarp();
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

static_assert(sizeof(Maxima) % 16 == 0 && offsetof(Maxima, minus) % 16 == 0, "read four at a time");

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
