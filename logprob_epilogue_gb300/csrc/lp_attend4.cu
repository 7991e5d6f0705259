// lp_attend4.cu -- sm_103a kernel of lp_attend4 for few rows: attention of verify
// rows over a paged cache held in 4 bits.
//
// The sums, their parts and the split of the work are those of lp_attend (see
// lp_split.h and lp_join.h): prefixes and committed tokens here, the round's own
// tokens in the join.  A token and head is D / 2 bytes of codes and D / 16 of
// scales, 0.28 of the bytes of 16 bits, so what has to keep up is the way from
// codes to products: a code and its scale make an F16 without rounding (cvt, then a
// product), 64 of either for 16 tokens of D = 128 and a warp's 32 products of 16 x 8 x 16.
// A unit of at most 32 rows is one or two fragments of 16 rows of mma.sync: what
// tcgen05 takes has to lie in shared or tensor memory first, and with so few
// rows the codes' way there costs more than the products that it saves (measured
// with keys expanded into tensor memory and values into shared memory by eight
// warps: 238 us where this takes 191, and 20.6 us for one token where this takes 14.4).
//
// Block (one per SM, 12 warps): warp 0 splits the work, warps 0 and 3 bring every
// other tile of 128 tokens into a ring (144 KiB) by bulk copies, four per page;
// warps 1 and 2 bring the units' queries and add up the workers' results; warps 4 to
// 11 multiply, four to a tile, each a quarter of its tokens.  Every warp holds the
// maxima and sums of its own tokens.
//
// Roundings: codes times scales, and queries after their lift, are exact in F16; probabilities are rounded to it; scores, maxima,
// sums, results and parts are 32 bits.
//
// What bounds it, by size (BF16, heads of 128, 32 over 8, in a CUDA graph):
// - the workers' latencies, two warps per scheduler, each in turn waiting for its own
//   conversions and products (issue slots used to 49%, no pipe to more than 35%): 128
//   groups of 4 rows at contexts up to 8,192 take 191 us, 3.3 TB/s of codes and scales.
//   A tile of one fragment takes 1,480 cycles of a block, 1,200 where the tiles are
//   there already; at the rates of their pipes the conversions and their products with
//   the scales take 760, and beside them the products on the tensor core 510.  Twelve workers, with the queries in shared memory, take as long
//   (110 us for 19 groups of 16,384 tokens against 109), 32 tokens a step too (109).
// - fragments: 32 rows of a unit take 192 us for those 19 groups; with D = 64 both share
//   a worker's conversions, 98 against 70 (124 as two workers').
// - pages of few tokens: a bulk copy takes its warp about 100 cycles, so pages of
//   8 tokens take 197 us there, 16 137, 32 113, 64 and more 109 (copies of 16 bytes a
//   lane: 161, 159, 138, 138).
// - latency: one row at 4,095 tokens takes 14.4 us, the launch, the split and the first
//   pages 8, a tile or two 2, the join 4.5.
// A thread spills 12 bytes with D = 64 and 20 with D = 128.
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
constexpr int kFirstWorker = 4, kWorkers = 8, kHelpers = 2;  // warps: 0 and 3 fetch, 1 and 2 help, 4-11 work
constexpr int kStreams = kWorkers / 4;                        // a tile has four workers
constexpr int kStep = 16;                                     // tokens of a step
constexpr int kThreads4 = (kFirstWorker + kWorkers) * 32;
// Registers: the split's sum is what the block is launched with, 384 x 168.
constexpr int kRegsLaunch = 168, kRegsWorker = 208, kRegsOther = 88;
static_assert(kStreams * kRegsWorker + kRegsOther <= (kStreams + 1) * kRegsLaunch, "register split");

template <int D>
struct Cfg4 {
    static constexpr int kCodes = kKTile * D / 2, kScales = kKTile * D / kBlock4;
    static constexpr int kBytes = 2 * (kCodes + kScales);     // K and V of a tile: codes, then scales
    static constexpr int kRing = 8 * 128 / D;                 // tiles
    static constexpr int kQuery = kUnitRows * D * 2;          // a unit's queries, as the workers hold them
    static constexpr int kQueries = kRing * kBytes;           // two units'
    static constexpr int kMerge = kQueries + 2 * kQuery;      // the workers' results: 16 rows each
    static constexpr int kCtl = kMerge + kWorkers * 16 * D * 4;
    static constexpr int kFragments = 128 / D;  // of 16 rows, at most, that a worker holds: a unit's two, or one of them
    static_assert(kRing % kStreams == 0 && kRing % 2 == 0, "slots of a stream, of a fetching warp");
};

constexpr int kPieces = 8;                              // pieces the planning warp may be ahead
constexpr int kPieceReaders = kWorkers + kHelpers + 1;  // warps that read each

// Where the tokens of a piece lie.
struct Pages {
    const int* table;
    long long token;  // the first
};

template <int D>
struct Ctl4 : PlanCtl<Fragments> {
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    Pages pages[kPieces];
    uint64_t tile_full[Cfg4<D>::kRing], tile_empty[Cfg4<D>::kRing];
    uint64_t q_full[2], q_free[2], merge_full, merge_free, drain;
    float unit[2][kUnitRows];  // what a row of queries was divided by
    float2 ml[kWorkers][16];
    int abort;
};

// D += A B, 16 x 8 x 16, F16 with FP32 sums; mma0: D = A B.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

constexpr uint32_t kOnes = 0x3C003C00u;  // two of F16

// a where the mask is set, else b.
__device__ __forceinline__ uint32_t select(uint32_t a, uint32_t b, uint32_t mask) { return (a & mask) | (b & ~mask); }

// A worker's rows, kF fragments of 16: two of each per thread, lane / 4 and eight further.
template <int D, int kF>
struct Rows {
    uint32_t q[kF][2][D / 8];  // lanes lane % 4 * D / 4 .. of each, as pairs of F16
    float o[kF][D / 8][4];  // fragment j: lanes (D / 8) (2t) + j and (D / 8) (2t + 1) + j of the first row, then of the second
    float c[kF][2], base[kF][2], limit[kF][2], l[kF][2];  // limit: -infinity until a score is above that
    // the rows' sums of the probabilities as the products take them (a product with ones, so twice each): by these, not by l,
    // the results are divided, and what the rounding does to a row of few tokens cancels
    float taken[kF][4];
};

// The queries of a unit, by the helpers, to where a worker's thread has its part
// of a row in 16-byte words: [half of a fragment][word][thread].  BF16 becomes F16 by a
// power of two for each row; D / 8 threads have a row.
template <bool kBf16, int D>
__device__ __forceinline__ void lay_queries(const AttendParams& p, const Piece& x, unsigned char* to, float* unit, int helper) {
    using T = typename Half<kBf16>::T;
    constexpr int kChunks = D / 8, kWords = D / 32, kAtOnce = kHelpers * 32 / kChunks, kTurns = 16 / kAtOnce;
    const int t = helper * 32 + (threadIdx.x & 31), ch = t % kChunks, rows = x.rows * p.share;
    const T* src = reinterpret_cast<const T*>(p.q) + (long long)x.row * p.q_stride + (long long)x.kvh * p.share * D + ch * 8;
#pragma unroll 1
    for (int base = 0; base < rows; base += 16) {
        uint4 w[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int row = base + k * kAtOnce + t / kChunks, per = (row * p.share_inv) >> 16, head = row - per * p.share;
            w[k] = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows) w[k] = *reinterpret_cast<const uint4*>(src + per * p.q_stride + head * D);
        }
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int row = base + k * kAtOnce + t / kChunks;
            if constexpr (kBf16) {
                // the largest magnitude: that of BF16 is its order as an integer without the sign
                const uint32_t m = 0x7FFF7FFFu;
                uint32_t top = __vmaxu2(__vmaxu2(w[k].x & m, w[k].y & m), __vmaxu2(w[k].z & m, w[k].w & m));
#pragma unroll
                for (int o = kChunks / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, o));
                const float2 lift = lift_of(__uint_as_float(top >> 16 > (top & 0xFFFFu) ? top & 0xFFFF0000u : top << 16));
                if (ch == 0) unit[row] = lift.y;
                uint32_t a[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 q = Half<true>::unpack(a[e]);
                    a[e] = Half<false>::pack(q.x * lift.x, q.y * lift.x);
                }
                w[k] = make_uint4(a[0], a[1], a[2], a[3]);
            }
            reinterpret_cast<uint4*>(to)[((row >> 3) * kWords + ch % kWords) * 32 + (row & 7) * 4 + ch / kWords] = w[k];
        }
    }
}

// A worker's fragments of them, and its rows' softmax at the start.
template <bool kBf16, int D, int kF>
__device__ __forceinline__ void take_rows(const AttendParams& p, const unsigned char* from, const float* unit, Rows<D, kF>& r) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int f = 0; f < kF; ++f) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 w = reinterpret_cast<const uint4*>(from)[((f * 2 + h) * (D / 32) + i) * 32 + lane];
                r.q[f][h][i * 4] = w.x, r.q[f][h][i * 4 + 1] = w.y, r.q[f][h][i * 4 + 2] = w.z, r.q[f][h][i * 4 + 3] = w.w;
            }
            r.c[f][h] = scaled(p.score, p.score_exp + (kBf16 ? exponent_of(unit[f * 16 + h * 8 + (lane >> 2)]) : 0));
            r.limit[f][h] = kNegInf;
            r.base[f][h] = r.l[f][h] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) r.taken[f][e] = 0.0f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) r.o[f][j][0] = r.o[f][j][1] = r.o[f][j][2] = r.o[f][j][3] = 0.0f;
    }
}

// A step is sixteen tokens from `at` on of a tile, `have` of whose tokens exist.
//
// Column c of eight scores is token (c >> 1) + 4 (c & 1) of its eight, so that
// the values that a thread multiplies (columns 2t and 2t + 1) are tokens t and t
// + 4, and the four t of a load lie side by side.

// The products of one step's values and of the next one's scores: a product of
// either kind in turn, since a score's follow on one another.  kScores: s of the
// step at token `next` of `later`; kValues: the probabilities `a` times the values
// at token `at` of `tile`.
template <int D, int kF, bool kScores, bool kValues>
__device__ __forceinline__ void products(const unsigned char* later, int next, float (&s)[kF][2][4], const unsigned char* tile, int at, int have,
                                         const uint32_t (&a)[kF][4], Rows<D, kF>& r) {
    using C = Cfg4<D>;
    constexpr int kK = D / 32, kV = D / 64;  // words of a thread's part of a key, of a value
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    const unsigned char* ks = later + 2 * C::kCodes;
    const unsigned char* vs = tile + 2 * C::kCodes + C::kScales;
    uint32_t kw[2][kK], ke[2][kK / 2], vw[2][2][kV], ve[2];
    if constexpr (kScores) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int token = next + b * 8 + (g >> 1) + 4 * (g & 1);
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(later + token * (D / 2) + t * 16);
                kw[b][0] = x.x, kw[b][1] = x.y, kw[b][kK - 2] = x.z, kw[b][kK - 1] = x.w;
                const uint32_t two = widen_scales(*reinterpret_cast<const uint16_t*>(ks + token * (D / 16) + t * 2));
                ke[b][0] = __byte_perm(two, 0, 0x1010);
                ke[b][kK / 2 - 1] = __byte_perm(two, 0, 0x3232);
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(later + token * (D / 2) + t * 8);
                kw[b][0] = x.x, kw[b][1] = x.y;
                ke[b][0] = __byte_perm(widen_scales(ks[token * (D / 16) + t]), 0, 0x1010);
            }
        }
    }
    if constexpr (kValues) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t scale[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int token = at + b * 8 + t + 4 * u;
                scale[u] = vs[token * (D / 16) + (D == 128 ? g : g >> 1)];
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(tile + C::kCodes + token * (D / 2) + g * 8);
                    vw[b][u][0] = x.x, vw[b][u][kV - 1] = x.y;
                } else {
                    vw[b][u][0] = *reinterpret_cast<const uint32_t*>(tile + C::kCodes + token * (D / 2) + g * 4);
                }
            }
            ve[b] = scale[0] | scale[1] << 8;
        }
        if (at + 16 > have) {  // what lies past the tokens may be NaN, and 0 * v has to stay 0
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (at + b * 8 + t >= have) ve[b] = 0u;
                if (at + b * 8 + t + 4 >= have) ve[b] &= 0xFFu;
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) ve[b] = widen_scales(ve[b]);
    }
    if constexpr (kValues) {
#pragma unroll
        for (int f = 0; f < kF; ++f) mma(r.taken[f], a[f][0], a[f][1], a[f][2], a[f][3], kOnes, kOnes);
    }
#pragma unroll
    for (int i = 0; i < kK; ++i) {
        uint32_t kh[2][4], vh[2][4];
        if constexpr (kScores) widen_codes(kw[0][i], kh[0]), widen_codes(kw[1][i], kh[1]);
        if constexpr (kValues) {
            // two tokens' codes side by side
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t x = vw[b][0][i / 2], y = vw[b][1][i / 2];
                widen_codes(i & 1 ? select(x >> 4, y, 0x0F0F0F0Fu) : select(x, y << 4, 0x0F0F0F0Fu), vh[b]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (kScores) {
                const int b = j & 1, u = j >> 1, k = 2 * i + u;
                const uint32_t b0 = mul2(kh[b][2 * u], ke[b][i / 2]), b1 = mul2(kh[b][2 * u + 1], ke[b][i / 2]);
#pragma unroll
                for (int f = 0; f < kF; ++f) {
                    const uint32_t (&q)[2][D / 8] = r.q[f];
                    if (k == 0) mma0(s[f][b], q[0][0], q[1][0], q[0][1], q[1][1], b0, b1);
                    else mma(s[f][b], q[0][2 * k], q[1][2 * k], q[0][2 * k + 1], q[1][2 * k + 1], b0, b1);
                }
            }
            if constexpr (kValues) {
                const uint32_t b0 = mul2(vh[0][j], ve[0]), b1 = mul2(vh[1][j], ve[1]);
#pragma unroll
                for (int f = 0; f < kF; ++f) mma(r.o[f][i / 2 * 8 + 2 * j + (i & 1)], a[f][0], a[f][1], a[f][2], a[f][3], b0, b1);
            }
        }
    }
}

template <int kF>
__device__ __forceinline__ void mask_scores(int at, int have, float (&s)[kF][2][4]) {
    if (at + kStep <= have) return;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool none = at + b * 8 + (int)(threadIdx.x & 3) + 4 * (i & 1) >= have;
#pragma unroll
            for (int f = 0; f < kF; ++f)
                if (none) s[f][b][i] = kNegInf;
        }
}

// The rows' maxima: what they stand at holds until a score is 2^kRescale above it.
template <int D, int kF>
__device__ __forceinline__ void raise(const float (&s)[kF][2][4], Rows<D, kF>& r) {
    float top[kF][2];
    bool above = false;
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[f][h] = fmaxf(max3(s[f][0][2 * h], s[f][0][2 * h + 1], s[f][1][2 * h]), s[f][1][2 * h + 1]);
            above |= top[f][h] > r.limit[f][h];
        }
    if (__any_sync(kFull, above)) {
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            float by[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float t = top[f][h];
                t = fmaxf(t, __shfl_xor_sync(kFull, t, 1));
                t = fmaxf(t, __shfl_xor_sync(kFull, t, 2));
                by[h] = 1.0f;
                if (t > r.limit[f][h]) {
                    const float next = t * r.c[f][h] - kBias;
                    if (r.limit[f][h] != kNegInf) by[h] = ex2(r.base[f][h] - next);
                    r.base[f][h] = next;
                    r.limit[f][h] = t + kRescale / r.c[f][h];
                    r.l[f][h] *= by[h];
                    r.taken[f][2 * h] *= by[h];
                }
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) r.o[f][j][0] *= by[0], r.o[f][j][1] *= by[0], r.o[f][j][2] *= by[1], r.o[f][j][3] *= by[1];
        }
    }
}

// A step's probabilities.
template <int D, int kF>
__device__ __forceinline__ void probabilities(const float (&s)[kF][2][4], Rows<D, kF>& r, uint32_t (&a)[kF][4]) {
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float x = ex2(fmaf(s[f][b][2 * h], r.c[f][h], -r.base[f][h])), y = ex2(fmaf(s[f][b][2 * h + 1], r.c[f][h], -r.base[f][h]));
                r.l[f][h] += x + y;
                a[f][2 * b + h] = Half<false>::pack(x, y);
            }
}

// The workers' results of a fragment of a piece (split: of two, each every other
// worker's), by the helpers, half of its rows each:
// what each worker's rows count for, then four lanes of a row per thread at a time.
template <int D>
__device__ __forceinline__ void merge_rows(const AttendParams& p, const Piece& x, const Ctl4<D>* ctl, const float4* merge, int helper, int fragment, bool split) {
    static_assert(kHelpers == 2, "halves of a fragment");
    const int lane = threadIdx.x & 31, in = (lane >> 2) + 8 * helper, row = fragment * 16 + in, rows = x.rows * p.share;
    float f[kWorkers], top = kNegInf, l = 0.0f;
    unsigned saw = 0u;
#pragma unroll
    for (int w = 0; w < kWorkers; ++w) {
        const float2 ml = ctl->ml[w][in];
        f[w] = ml.x;
        if (!(ml.x == kNegInf && ml.y == 0.0f) && !(split && (w & 1) != fragment)) saw |= 1u << w, top = fmaxf(top, ml.x);
    }
    const float from = top == kNegInf ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kWorkers; ++w) {
        f[w] = ex2(f[w] - from);
        if (saw >> w & 1u) l = fmaf(ctl->ml[w][in].y, f[w], l);
    }
    if (row < rows && (lane & 3) == 0) p.fragments.part_ml[x.part + row] = make_float2(top, l);
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {
        const int chunk = helper * (D / 16) + i, e = i / (D / 32), j = i % (D / 32);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v[kWorkers];
#pragma unroll
        for (int w = 0; w < kWorkers; ++w) v[w] = merge[(w * (D / 8) + chunk) * 32 + lane];
#pragma unroll
        for (int w = 0; w < kWorkers; ++w)
            if (saw >> w & 1u)
                o.x = fmaf(v[w].x, f[w], o.x), o.y = fmaf(v[w].y, f[w], o.y), o.z = fmaf(v[w].z, f[w], o.z), o.w = fmaf(v[w].w, f[w], o.w);
        if (row < rows)
            reinterpret_cast<float4*>(p.fragments.part_o)[part_chunk<D>(x.part, x.part_stride, row, (D / 32) * (2 * (lane & 3) + e) + j)] = o;
    }
}

// The worker's way through the ring: its next tile's slot, that barrier's parity,
// how far the tile is from the piece's first, and the results that it has handed over.
struct Line {
    uint32_t slot, phase, ahead, merged;
};

// A worker's part of a piece: `chunk` tokens from `first` on of its tiles, for kF
// fragments from mt on.  False when a wait ran out.
template <bool kBf16, int D, int kF>
__device__ __forceinline__ bool work_piece(const AttendParams& p, const Piece& x, unsigned char* smem, Ctl4<D>* ctl, uint32_t n, int worker, int mt, int first,
                                           int chunk, Line& line, unsigned long long limit) {
    using C = Cfg4<D>;
    const int lane = threadIdx.x & 31;
    volatile int* abort = &ctl->abort;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return tc::warp_wait(bar, parity, limit, abort); };
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar);
    };
    Rows<D, kF> r;
    take_rows<kBf16, D, kF>(p, smem + C::kQueries + (n & 1u) * C::kQuery + mt * 16 * D * 2, ctl->unit[n & 1u] + mt * 16, r);
    arrive(&ctl->q_free[n & 1u]);
    int i = (int)line.ahead;
    auto take = [&]() -> const unsigned char* {
        return wait(&ctl->tile_full[line.slot], line.phase) ? smem + line.slot * C::kBytes : nullptr;
    };
    auto give = [&](uint32_t slot) { arrive(&ctl->tile_empty[slot]); };
    auto pass = [&]() {
        if ((line.slot += kStreams) >= C::kRing) line.slot -= C::kRing, line.phase ^= 1u;
    };
    // tiles of which none of these tokens exist (a piece's last, and then only it)
    const int last = x.left - (x.tiles - 1) * kKTile > first ? x.tiles : x.tiles - 1;
    if (i < last) {
        const unsigned char* tile = take();
        if (tile == nullptr) return false;
        float s[kF][2][4];
        uint32_t a[kF][4] = {};
        products<D, kF, true, false>(tile, first, s, tile, 0, kKTile, a, r);
        int at = first;
        // a step's values beside the next one's scores, so that the tensor core has work while the warp waits for either
        for (;;) {
            const int have = x.left - i * kKTile;
            mask_scores<kF>(at, have, s);
            raise<D, kF>(s, r);
            probabilities<D, kF>(s, r, a);
            const unsigned char* later = tile;
            const uint32_t now = line.slot;
            int next = at + kStep;
            if (next >= first + chunk || next >= have) {
                next = first;
                if (i + kStreams >= last) break;
                pass();
                later = take();
                if (later == nullptr) return false;
            }
            products<D, kF, true, true>(later, next, s, tile, at, have, a, r);
            if (later != tile) {
                give(now);
                i += kStreams;
                tile = later;
            }
            at = next;
        }
        products<D, kF, false, true>(tile, 0, s, tile, at, x.left - i * kKTile, a, r);
        give(line.slot);
        pass();
        i += kStreams;
    }
    for (; i < x.tiles; i += kStreams) {
        if (take() == nullptr) return false;
        give(line.slot);
        pass();
    }
    line.ahead = (uint32_t)(i - x.tiles);
    float4* merge = reinterpret_cast<float4*>(smem + C::kMerge) + worker * (D / 8) * 32 + lane;
#pragma unroll
    for (int f = 0; f < kF; ++f) {
        if (!wait(&ctl->merge_free, (line.merged & 1u) ^ 1u)) return false;  // the fragment before is added up
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            r.l[f][h] += __shfl_xor_sync(kFull, r.l[f][h], 1);
            r.l[f][h] += __shfl_xor_sync(kFull, r.l[f][h], 2);
            if ((lane & 3) == 0) ctl->ml[worker][(lane >> 2) + 8 * h] = make_float2(r.limit[f][h] == kNegInf ? kNegInf : r.base[f][h], r.l[f][h]);
            const float by = r.taken[f][2 * h] == 0.0f ? 1.0f : r.l[f][h] / r.taken[f][2 * h];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int j = 0; j < D / 32; ++j)
                    merge[((2 * h + e) * (D / 32) + j) * 32] = make_float4(r.o[f][4 * j][2 * h + e] * by, r.o[f][4 * j + 1][2 * h + e] * by,
                                                                           r.o[f][4 * j + 2][2 * h + e] * by, r.o[f][4 * j + 3][2 * h + e] * by);
        }
        arrive(&ctl->merge_full);
        ++line.merged;
    }
    return true;
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads4, 1) lp_attend4_kernel(const AttendParams p) {
    using C = Cfg4<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl4<D>* ctl = reinterpret_cast<Ctl4<D>*>(smem + C::kCtl);
    float4* merge = reinterpret_cast<float4*>(smem + C::kMerge);  // [worker][chunk][lane]
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, as the compiler sees
    const unsigned long long limit = p.timeout_ns;
    if (warp == kFirstWorker + kWorkers - 1) {  // while the kernel ahead still runs
        if (lane < kPieces) tc::mbar_init(&ctl->piece_full[lane], 1), tc::mbar_init(&ctl->piece_empty[lane], kPieceReaders);
        if (lane < C::kRing) tc::mbar_init(&ctl->tile_full[lane], 1), tc::mbar_init(&ctl->tile_empty[lane], 4);
        if (lane < 2) tc::mbar_init(&ctl->q_full[lane], kHelpers), tc::mbar_init(&ctl->q_free[lane], kWorkers);
        if (lane == 0) {
            tc::mbar_init(&ctl->merge_full, kWorkers);
            tc::mbar_init(&ctl->merge_free, kHelpers);
            tc::mbar_init(&ctl->drain, 1);
            ctl->abort = 0;
        }
        tc::fence_async_shared();
    }
    // so far nothing of what earlier kernels write; the join may start once that is there, and waits for this grid's end by itself
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    Runs runs[2];  // of prefixes, of groups
    const bool any = plan_run<Fragments>(p, ctl, runs);
    __syncthreads();
    if (!any) {
        if (tid == 0) p.fragments.gave_up[blockIdx.x] = 0;
        return;
    }
    volatile int* abort = &ctl->abort;
    // test hook: nothing arrives on `drain`, so this wait runs out
    if (p.force_timeout) tc::warp_wait(&ctl->drain, 0, limit, abort);

    Piece x;
    bool ok = !p.force_timeout;
    uint32_t n_piece = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = tc::warp_wait(bar, parity, limit, abort); };
    auto arrive = [&](uint64_t* bar, uint32_t count) {  // of the warp, after what all its lanes did
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar, count);
    };
    // the next piece, from the planning warp; false at the end of the run
    auto next_piece = [&]() {
        const uint32_t i = n_piece % kPieces;
        if (!wait(&ctl->piece_full[i], n_piece / kPieces & 1u)) return false;
        x = ctl->piece[i];
        arrive(&ctl->piece_empty[i], 1);
        ++n_piece;
        return x.rows > 0;
    };

    if (warp >= kFirstWorker) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWorker));
        // ---- products: every kStreams-th tile is a worker's, a quarter of its tokens.  Where it has registers for one fragment
        // and the unit has two, they are two workers', of twice the tokens.
        const int worker = warp - kFirstWorker, stream = worker >> 2, in = worker & 3;
        Line line{(uint32_t)stream, 0u, (uint32_t)stream, 0u};
        while (ok && next_piece()) {
            const uint32_t n = n_piece - 1;
            if (!wait(&ctl->q_full[n & 1u], n >> 1 & 1u)) break;
            const bool two = x.rows * p.share > 16;
            if (D == 64 && two) {
                ok = work_piece<kBf16, D, C::kFragments>(p, x, smem, ctl, n, worker, 0, in * (kKTile / 4), kKTile / 4, line, limit);
            } else {
                const int mt = two ? worker & 1 : 0, chunk = two ? kKTile / 2 : kKTile / 4;
                ok = work_piece<kBf16, D, 1>(p, x, smem, ctl, n, worker, mt, (two ? in >> 1 : in) * chunk, chunk, line, limit);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 0 || warp == 3) {
            // ---- every other tile into the ring: it lies on one page, or on several, and a lane has the copies of each.
            // Warp 0 plans the pieces, each after a ring's worth of the one before.
            const int shift = p.page_shift < 7 ? p.page_shift : 7, step = 1 << shift, part = lane << shift;  // tokens of a copy; this lane's first
            const uint32_t first = warp == 0 ? 0 : 1;
            uint32_t slot = first, phase = 1, ahead = first, filled = 0;  // this warp's next tile: its slot, how far it is from the piece's first
            Pages from = {nullptr, 0};
            auto page_of = [&](int i) {
                const int t = i * kKTile + part;
                return i < x.tiles && part < kKTile && t < x.left ? from.table[(from.token + t) >> p.page_shift] : -1;
            };
            auto fetch = [&](int i, int page) {
                const int t = i * kKTile + part;
                const bool exists = part < kKTile && t < x.left, good = page >= 0 && page < p.num_pages;
                const unsigned copies = __ballot_sync(kFull, exists), sound = __ballot_sync(kFull, exists && good);
                unsigned char* to = smem + slot * C::kBytes;
                uint64_t* bar = &ctl->tile_full[slot];
                if (!wait(&ctl->tile_empty[slot], phase)) return false;
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
                if (lane == 0) tc::mbar_expect(bar, (uint32_t)(__popc(sound) * (D + D / 8)) << shift);
                __syncwarp();
                // page by page: an instruction of one lane that is the same for all of them
                for (unsigned left = sound; left != 0; left &= left - 1) {
                    const int k = __ffs(left) - 1, first = k << shift;
                    const int of = __shfl_sync(kFull, page, k);
                    const long long at = (((long long)of * p.kv_heads + x.kvh) << p.page_shift) + ((from.token + i * kKTile + first) & ((1 << p.page_shift) - 1));
                    const uint32_t codes = tc::smem_addr(to) + first * (D / 2), scales = tc::smem_addr(to) + 2 * C::kCodes + first * (D / kBlock4);
                    if (tc::elect_one()) {
                        tc::bulk_load(codes, static_cast<const unsigned char*>(p.k_cache) + at * (D / 2), D / 2 << shift, bar);
                        tc::bulk_load(codes + C::kCodes, static_cast<const unsigned char*>(p.v_cache) + at * (D / 2), D / 2 << shift, bar);
                        tc::bulk_load(scales, p.k_scales + at * (D / kBlock4), D / kBlock4 << shift, bar);
                        tc::bulk_load(scales + C::kScales, p.v_scales + at * (D / kBlock4), D / kBlock4 << shift, bar);
                    }
                }
                if (filled < C::kRing / 2) ++filled;
                if ((slot += 2) >= C::kRing) slot -= C::kRing, phase ^= 1u;
                return true;
            };
            if (warp == 0) {
                Walk<Fragments> walk;
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
                    int i = (int)ahead, page = page_of(i);
                    for (bool planned = false; i < x.tiles || !planned;) {
                        if (i < x.tiles) {
                            const int now = page;
                            page = page_of(i + 2);  // a tile's page is read before the waits of the one before
                            if (!fetch(i, now)) break;
                        }
                        if (!planned && (i + 2 >= x.tiles || i + 2 >= C::kRing)) planned = true, more = plan();
                        if (!ok) break;
                        if (i < x.tiles) i += 2;
                    }
                    ahead = (uint32_t)(i - x.tiles);
                }
            } else {
                while (ok) {
                    const uint32_t i0 = n_piece % kPieces;
                    if (!wait(&ctl->piece_full[i0], n_piece / kPieces & 1u)) break;
                    from = ctl->pages[i0];
                    if (!next_piece()) break;
                    int i = (int)ahead, page = page_of(i);
                    for (; i < x.tiles; i += 2) {
                        const int now = page;
                        page = page_of(i + 2);
                        if (!fetch(i, now)) break;
                    }
                    ahead = (uint32_t)(i - x.tiles);
                }
            }
            int none = 0;  // no copy outlives the block, whatever its readers did
            for (; filled > 0; --filled) {
                if (slot < 2) slot += C::kRing, phase ^= 1u;
                slot -= 2;
                tc::mbar_wait(&ctl->tile_full[slot], phase ^ 1u, limit, &none);
            }
        } else {
            // ---- a unit's queries, a piece ahead of the workers; then their results of the piece before
            const int helper = warp - 1;
            Piece last = {};
            uint32_t merged = 0;
            for (;;) {
                const bool more = next_piece();
                if (!ok) break;
                const uint32_t n = n_piece - 1;
                if (more) {
                    if (!wait(&ctl->q_free[n & 1u], (n >> 1 & 1u) ^ 1u)) break;
                    lay_queries<kBf16, D>(p, x, smem + C::kQueries + (n & 1u) * C::kQuery, ctl->unit[n & 1u], helper);
                    arrive(&ctl->q_full[n & 1u], 1);
                }
                const int fragments = (last.rows * p.share + 15) >> 4;
                const bool split = fragments > C::kFragments;
                for (int f = 0; f < fragments; ++f) {
                    if ((f == 0 || !split) && !wait(&ctl->merge_full, merged & 1u)) break;
                    if (last.part >= 0) merge_rows<D>(p, last, ctl, merge, helper, f, split);
                    if (!split || f == fragments - 1) arrive(&ctl->merge_free, 1), ++merged;
                }
                if (!ok) break;
                if (!more) break;
                last = x;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        p.fragments.gave_up[blockIdx.x] = *abort;
        if (*abort != 0) atomicOr(p.status, kStatusAttnTimeout);
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
cudaError_t launch4(const AttendParams& p, cudaStream_t stream) {
    // Each kernel is launched while the one before still runs, and waits for its end before it reads what that writes.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)p.grid);
    lc.blockDim = dim3(kThreads4);
    lc.dynamicSmemBytes = smem_bytes4<D>();
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    if (runs_fragments(p)) e = cudaLaunchKernelEx(&lc, lp_attend4_kernel<kBf16, D>, p);
    if (e == cudaSuccess && runs_pairs(p)) e = launch_attend4_pairs(p, kBf16 ? 1 : 2, D, lc);
    return e == cudaSuccess ? launch_join<kBf16, D, true>(p, lc) : e;
}

}  // namespace

// Fragments take a token tile once for every 32 of a unit's rows, pairs once for every
// 256, and for longer.  Fragments against pairs with 8 key-value heads and four heads
// each, us: 19 groups of 16,384 tokens and 4 rows (16 of a unit) 109 and 191, 8 rows 192
// and 196, 12 rows 287 and 205, 16 rows 376 and 210; 608 groups of 512 tokens 201 and
// 314, 341 and 374, 564 and 470, 737 and 621; D = 64, 19 groups: 70 and 146, 98 and 149,
// 157 and 156, 187 and 159.  So by the rows that a prefix and a group have on average,
// padding and idle groups among them: what a call's sizes say before it runs.  Few large
// groups among many small ones so take fragments: one of 32 rows at 16,384 tokens beside
// 127 of one row at 1,024 takes 119 (142 by pairs), at 65,536 tokens 226 (169), eight of
// them at 16,384 beside 120 take 386 (208).
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

cudaError_t launch_attend4(const AttendParams& p, int dtype, int head_dim, cudaStream_t stream) {
    if (dtype == 1) return head_dim == 128 ? launch4<true, 128>(p, stream) : launch4<true, 64>(p, stream);
    return head_dim == 128 ? launch4<false, 128>(p, stream) : launch4<false, 64>(p, stream);
}

}  // namespace lp
