// lp_attend4.cu -- sm_103a kernel of lp_attend4: attention of verify rows over
// a paged cache held in 4 bits.
//
// The sums, their parts and the split of the work are those of lp_attend (see
// lp_split.h and lp_join.h): prefixes and committed tokens here, the round's
// own tokens in the join.  Here a token and head is D / 2 bytes of codes and
// D / 16 of scales, 0.28 of the bytes of 16 bits, and what has to keep up with
// them is the way from codes to products.
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
constexpr int kWorkers = 8;       // warps that multiply
constexpr int kFetchers = 4;      // warps that bring pages, a quarter of a tile's tokens each
constexpr int kStep = 16;         // tokens of a step
// Registers: the split's sum is what the block is launched with, 384 x 168.
constexpr int kRegsLaunch = 168, kRegsWorker = 200, kRegsOther = 104;
static_assert(2 * kRegsWorker + kRegsOther <= 3 * kRegsLaunch, "register split");

template <int D>
struct Cfg4 {
    static constexpr int kCodes = kKTile * D / 2, kScales = kKTile * D / kBlock4;
    static constexpr int kStage = 2 * (kCodes + kScales);  // K and V of a tile: codes, then scales
    static constexpr int kStages = 8 * 128 / D;            // 144 KiB
    static constexpr int kMerge = kStages * kStage;        // the workers' results: 16 rows each
    static constexpr int kCtl = kMerge + kWorkers * 16 * D * 4;
};

constexpr int kPieces = 8;                               // pieces the planning warp may be ahead
constexpr int kPieceReaders = kWorkers + kFetchers - 1;  // warps that read each

// Where the tokens of a piece lie.
struct Pages {
    const int* table;
    long long token;  // the first
};

struct Ctl4 : PlanCtl<Fragments> {
    uint64_t full[16], empty[16], piece_full[kPieces], piece_empty[kPieces];
    Piece piece[kPieces];
    Pages pages[kPieces];
    uint64_t merge_full, merge_done, drain;
    float2 ml[kWorkers][16];
    int abort;
};

// D += A B, 16 x 8 x 16, F16 with FP32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lop_select(uint32_t a, uint32_t b, uint32_t mask) { return (a & mask) | (b & ~mask); }

// A worker's rows: two per thread, lane / 4 and eight further.
template <int D>
struct Rows {
    uint32_t q[2][D / 8];        // lanes lane % 4 * D / 4 .. of each, as pairs of F16
    float o[D / 8][4];           // fragment j: lanes (D / 8) (2t) + j and (D / 8) (2t + 1) + j of the first row, then of the second
    float c[2], m[2], base[2], limit[2], l[2];
};

// The queries of fragment `mt` of a unit.
template <bool kBf16, int D>
__device__ __forceinline__ void load_rows(const AttendParams& p, const Piece& x, int mt, Rows<D>& r) {
    using T = typename Half<kBf16>::T;
    const int lane = threadIdx.x & 31, t = lane & 3;
    uint4 w[2][D / 32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = mt * 16 + (lane >> 2) + 8 * h;
        const int per = (row * p.share_inv) >> 16, head = row - per * p.share;
        const T* src = reinterpret_cast<const T*>(p.q) + (long long)(x.row + per) * p.q_stride + (long long)(x.kvh * p.share + head) * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            w[h][i] = row < x.rows * p.share ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float unit = 1.0f;
        if constexpr (kBf16) {
            // to F16 by a power of two that brings the row's largest lane to [2^14, 2^15)
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t a[4] = {w[h][i].x, w[h][i].y, w[h][i].z, w[h][i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = Half<true>::unpack(a[e]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
            const int field = (int)(__float_as_uint(top) >> 23);
            int up = 141 - field;
            up = up > 126 ? 126 : up;
            if (field == 255 || top == 0.0f) up = 0;
            const float lift = __uint_as_float((uint32_t)(up + 127) << 23);
            unit = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t a[4] = {w[h][i].x, w[h][i].y, w[h][i].z, w[h][i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = Half<true>::unpack(a[e]);
                    r.q[h][i * 4 + e] = Half<false>::pack(f.x * lift, f.y * lift);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) r.q[h][i * 4] = w[h][i].x, r.q[h][i * 4 + 1] = w[h][i].y, r.q[h][i * 4 + 2] = w[h][i].z, r.q[h][i * 4 + 3] = w[h][i].w;
        }
        // finite and above 0, so that a masked score stays -infinity and one of 0 stays 0
        r.c[h] = fminf(fmaxf(p.scale * kLog2e * p.k_factor * unit, 0x1p-126f), 0x1p127f);
        r.m[h] = r.limit[h] = kNegInf;
        r.base[h] = r.l[h] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < D / 8; ++j) r.o[j][0] = r.o[j][1] = r.o[j][2] = r.o[j][3] = 0.0f;
}

// A step is sixteen tokens from `at` on of a stage, `have` of whose tokens exist.
//
// Column c of eight scores is token (c >> 1) + 4 (c & 1) of its eight, so that
// the values that a thread multiplies (columns 2t and 2t + 1) are tokens t and t
// + 4, and the four t of a load lie side by side.

// The products of one step's values and of another's scores: a product of either
// kind in turn, since a score's follow on one another.  kScores: s of the step at
// token `next`; kValues: the probabilities `a` times the values at token `at`.
template <int D, bool kScores, bool kValues>
__device__ __forceinline__ void products(const unsigned char* stage, int next, float (&s)[2][4], int at, int have, const uint32_t (&a)[4], Rows<D>& r) {
    using C = Cfg4<D>;
    constexpr int kK = D / 32, kV = D / 64;  // words of a thread's part of a key, of a value
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    const unsigned char* ks = stage + 2 * C::kCodes;
    const unsigned char* vs = ks + C::kScales;
    uint32_t kw[2][kK], ke[2][kK / 2], vw[2][2][kV], ve[2];
    if constexpr (kScores) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int token = next + b * 8 + (g >> 1) + 4 * (g & 1);
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4*>(stage + token * (D / 2) + t * 16);
                kw[b][0] = x.x, kw[b][1] = x.y, kw[b][kK - 2] = x.z, kw[b][kK - 1] = x.w;
                const uint32_t two = widen_scales(*reinterpret_cast<const uint16_t*>(ks + token * (D / 16) + t * 2));
                ke[b][0] = __byte_perm(two, 0, 0x1010);
                ke[b][kK / 2 - 1] = __byte_perm(two, 0, 0x3232);
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(stage + token * (D / 2) + t * 8);
                kw[b][0] = x.x, kw[b][1] = x.y;
                ke[b][0] = __byte_perm(widen_scales(ks[token * (D / 16) + t]), 0, 0x1010);
            }
            s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.0f;
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
                if (token >= have) scale[u] = 0u;  // what lies there may be NaN, and 0 * v has to stay 0
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(stage + C::kCodes + token * (D / 2) + g * 8);
                    vw[b][u][0] = x.x, vw[b][u][kV - 1] = x.y;
                } else {
                    vw[b][u][0] = *reinterpret_cast<const uint32_t*>(stage + C::kCodes + token * (D / 2) + g * 4);
                }
            }
            ve[b] = widen_scales(scale[0] | scale[1] << 8);
        }
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
                widen_codes(i & 1 ? lop_select(x >> 4, y, 0x0F0F0F0Fu) : lop_select(x, y << 4, 0x0F0F0F0Fu), vh[b]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (kScores) {
                const int b = j & 1, u = j >> 1, k = 2 * i + u;
                mma(s[b], r.q[0][2 * k], r.q[1][2 * k], r.q[0][2 * k + 1], r.q[1][2 * k + 1], mul2(kh[b][2 * u], ke[b][i / 2]), mul2(kh[b][2 * u + 1], ke[b][i / 2]));
            }
            if constexpr (kValues)
                mma(r.o[i / 2 * 8 + 2 * j + (i & 1)], a[0], a[1], a[2], a[3], mul2(vh[0][j], ve[0]), mul2(vh[1][j], ve[1]));
        }
    }
}

__device__ __forceinline__ void mask_scores(int at, int have, float (&s)[2][4]) {
    if (at + kStep <= have) return;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + b * 8 + (int)(threadIdx.x & 3) + 4 * (i & 1) >= have) s[b][i] = kNegInf;
}

// The rows' maxima: what they stand at holds until a score is 2^kRescale above it.
template <int D>
__device__ __forceinline__ void raise(const float (&s)[2][4], Rows<D>& r) {
    float top[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) top[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
    if (__any_sync(kFull, top[0] > r.limit[0] || top[1] > r.limit[1])) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
            f[h] = 1.0f;
            if (top[h] > r.limit[h]) {
                const float next = top[h] * r.c[h] - kBias;
                if (r.m[h] != kNegInf) f[h] = ex2(r.base[h] - next);
                r.m[h] = top[h];
                r.base[h] = next;
                r.limit[h] = top[h] + kRescale / r.c[h];
                r.l[h] *= f[h];
            }
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) r.o[j][0] *= f[0], r.o[j][1] *= f[0], r.o[j][2] *= f[1], r.o[j][3] *= f[1];
    }
}

// A step's probabilities.
template <int D>
__device__ __forceinline__ void probabilities(const float (&s)[2][4], Rows<D>& r, uint32_t (&a)[4]) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float x = ex2(fmaf(s[b][2 * h], r.c[h], -r.base[h])), y = ex2(fmaf(s[b][2 * h + 1], r.c[h], -r.base[h]));
            r.l[h] += x + y;
            a[2 * b + h] = Half<false>::pack(x, y);
        }
}

// Steps from token `at` to `end` of a stage: a step's values beside the next one's scores, so that the tensor core has
// work while a warp waits for either.
template <int D>
__device__ __forceinline__ void steps(const unsigned char* stage, int at, int end, int have, Rows<D>& r) {
    float s[2][4];
    uint32_t a[4] = {0u, 0u, 0u, 0u};
    products<D, true, false>(stage, at, s, 0, 0, a, r);
#pragma unroll 1
    for (;; at += kStep) {
        mask_scores(at, have, s);
        raise<D>(s, r);
        probabilities<D>(s, r, a);
        if (at + kStep >= end) break;
        products<D, true, true>(stage, at + kStep, s, at, have, a, r);
    }
    products<D, false, true>(stage, 0, s, at, have, a, r);
}

// The workers' results of a piece, fragment by fragment of the rows: each thread
// adds up what the workers of a fragment have of four lanes of a row.
template <int D>
__device__ __forceinline__ void merge_piece(const AttendParams& p, const Piece& x, const Ctl4* ctl, const float4* merge, int worker, int fragments) {
    const int lane = threadIdx.x & 31, rows = x.rows * p.share;
    for (int i = worker; i < fragments * (D / 8) && x.part >= 0; i += kWorkers) {
        const int mt = i / (D / 8), chunk = i % (D / 8), h = chunk / (D / 16), e = chunk / (D / 32) & 1, j = chunk % (D / 32);
        const int in = (lane >> 2) + 8 * h, row = mt * 16 + in;
        if (row >= rows) continue;
        float top = kNegInf, l = 0.0f;
        for (int w = mt; w < kWorkers; w += fragments) top = fmaxf(top, ctl->ml[w][in].x);
        const float from = top == kNegInf ? 0.0f : top;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = mt; w < kWorkers; w += fragments) {
            const float2 ml = ctl->ml[w][in];
            if (ml.x == kNegInf && ml.y == 0.0f) continue;  // saw nothing
            const float f = ex2(ml.x - from);
            const float4 v = merge[(w * (D / 8) + chunk) * 32 + lane];
            l = fmaf(ml.y, f, l);
            o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        }
        if (chunk % (D / 16) == 0 && (lane & 3) == 0) p.fragments.part_ml[x.part + row] = make_float2(top, l);
        reinterpret_cast<float4*>(p.fragments.part_o)[part_chunk<D>(x.part, x.part_stride, row, (D / 32) * (2 * (lane & 3) + e) + j)] = o;
    }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1) lp_attend4_kernel(const AttendParams p) {
    using C = Cfg4<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl4* ctl = reinterpret_cast<Ctl4*>(smem + C::kCtl);
    float4* merge = reinterpret_cast<float4*>(smem + C::kMerge);  // [worker][chunk][lane]
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, as the compiler sees
    const unsigned long long limit = p.timeout_ns;
    if (warp == kWarps - 1) {  // while the kernel ahead still runs
        if (lane < C::kStages) tc::mbar_init(&ctl->full[lane], kFetchers * 32), tc::mbar_init(&ctl->empty[lane], kWorkers);
        if (lane < kPieces) tc::mbar_init(&ctl->piece_full[lane], 1), tc::mbar_init(&ctl->piece_empty[lane], kPieceReaders);
        if (lane == 0) {
            tc::mbar_init(&ctl->merge_full, kWorkers);
            tc::mbar_init(&ctl->merge_done, kWorkers);
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
    uint32_t n_piece = 0, it = 0;  // it: stages
    // the next piece, from the planning warp; false at the end of the run
    auto next_piece = [&](Pages* pages) {
        const uint32_t i = n_piece % kPieces;
        ok = tc::warp_wait(&ctl->piece_full[i], n_piece / kPieces & 1u, limit, abort);
        if (!ok) return false;
        x = ctl->piece[i];
        if (pages != nullptr) *pages = ctl->pages[i];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl->piece_empty[i]);
        ++n_piece;
        return x.rows > 0;
    };

    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWorker));
        // ---- products: fragment mt of the unit's rows, every slices-th chunk of the tokens
        const int worker = warp - 4;
        uint32_t merged = 0;
        while (ok && next_piece(nullptr)) {
            const int fragments = (x.rows * p.share + 15) >> 4, mt = worker % fragments, slice = worker / fragments;
            const int slices = (kWorkers - mt + fragments - 1) / fragments;
            Rows<D> r;
            load_rows<kBf16, D>(p, x, mt, r);
            // tokens that a worker takes in a row: long ones keep the products close, short ones give every worker some
            const int chunk = x.tiles * 2 >= slices ? 64 : (x.tiles * 4 >= slices ? 32 : 16);
            int s = slice * chunk;  // the next, in its tile
            for (int i = 0; ok && i < x.tiles; ++i, ++it) {
                const uint32_t at = it % C::kStages;
                ok = tc::warp_wait(&ctl->full[at], it / C::kStages & 1u, limit, abort);
                if (!ok) break;
                const int left = x.left - i * kKTile, have = left < kKTile ? left : kKTile;
                for (; s < have; s += slices * chunk) steps<D>(smem + at * C::kStage, s, s + chunk < have ? s + chunk : have, have, r);
                s -= kKTile;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl->empty[at]);
            }
            ok = ok && tc::warp_wait(&ctl->merge_done, (merged & 1u) ^ 1u, limit, abort);  // the piece before is read
            if (!ok) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                r.l[h] += __shfl_xor_sync(kFull, r.l[h], 1);
                r.l[h] += __shfl_xor_sync(kFull, r.l[h], 2);
                if ((lane & 3) == 0) ctl->ml[worker][(lane >> 2) + 8 * h] = make_float2(r.m[h] == kNegInf ? kNegInf : r.base[h], r.l[h]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j)
                        merge[(worker * (D / 8) + (2 * h + e) * (D / 32) + j) * 32 + lane] =
                            make_float4(r.o[4 * j][2 * h + e], r.o[4 * j + 1][2 * h + e], r.o[4 * j + 2][2 * h + e], r.o[4 * j + 3][2 * h + e]);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->merge_full);
            ok = tc::warp_wait(&ctl->merge_full, merged & 1u, limit, abort);
            if (!ok) break;
            ++merged;
            merge_piece<D>(p, x, ctl, merge, worker, fragments);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->merge_done);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        // ---- pages into the ring: 32 tokens of each tile, a token's page per lane.  Warp 0 plans, a piece ahead.
        Walk<Fragments> walk;
        Pages from = {nullptr, 0}, ahead = from;
        Piece y;
        auto plan_piece = [&]() {  // into y and `ahead`, and to the other warps
            const bool more = walk.next(p, y);
            ahead.table = walk.table, ahead.token = walk.token;
            const uint32_t i = n_piece % kPieces;
            ok = tc::warp_wait(&ctl->piece_empty[i], (n_piece / kPieces & 1u) ^ 1u, limit, abort);
            if (!ok) return false;
            if (lane == 0) {
                ctl->piece[i] = y;
                ctl->pages[i] = ahead;
                tc::mbar_arrive(&ctl->piece_full[i]);
            }
            ++n_piece;
            return more;
        };
        bool more = false;
        if (warp == 0) {
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
            more = ok && plan_piece();
        }
        const int mask = (1 << p.page_shift) - 1, quarter = warp * 32;
        while (ok) {
            if (warp == 0) {
                if (!more) break;
                x = y, from = ahead;
                more = plan_piece();
                if (!ok) break;
            } else if (!next_piece(&from)) {
                break;
            }
            auto page_of = [&](int i) {
                const int t = i * kKTile + quarter + lane;
                return i < x.tiles && t < x.left ? from.table[(from.token + t) >> p.page_shift] : -1;
            };
            int next_page = page_of(0);  // a tile's pages are read before the waits of the one before
            for (int i = 0; i < x.tiles; ++i, ++it) {
                const int page = next_page, t = i * kKTile + quarter + lane;
                next_page = page_of(i + 1);
                const uint32_t at = it % C::kStages;
                ok = tc::warp_wait(&ctl->empty[at], (it / C::kStages & 1u) ^ 1u, limit, abort);
                if (!ok) break;
                const bool exists = t < x.left, good = page >= 0 && page < p.num_pages;
                if (exists && !good) atomicOr(p.status, kStatusBadPage);  // such a page reads as zeros
                const long long slot = exists && good ? (((long long)page * p.kv_heads + x.kvh) << p.page_shift) + ((from.token + t) & mask) : -1;
                const uint32_t to = tc::smem_addr(smem + at * C::kStage);
                constexpr int kPer = D / 32, kAtOnce = 32 / kPer;  // 16-byte parts of a token's codes; tokens of an instruction
#pragma unroll
                for (int j = 0; j < 32 / kAtOnce; ++j) {
                    const int token = j * kAtOnce + lane / kPer;
                    const long long from_slot = __shfl_sync(kFull, slot, token);
                    const long long byte = (from_slot < 0 ? 0 : from_slot) * (D / 2) + lane % kPer * 16;
                    const uint32_t dst = to + (quarter + token) * (D / 2) + lane % kPer * 16;
                    tc::copy16_or_zeros(dst, static_cast<const unsigned char*>(p.k_cache) + byte, from_slot >= 0);
                    tc::copy16_or_zeros(dst + C::kCodes, static_cast<const unsigned char*>(p.v_cache) + byte, from_slot >= 0);
                }
                {
                    // scales: 16 bytes are those of 256 / D tokens (of one page), lanes 0-15 of keys, 16-31 of values
                    constexpr int kTokens = 256 / D, kLanes = 32 / kTokens;
                    const int l = lane & 15, token = l * kTokens & 31;
                    const long long from_slot = __shfl_sync(kFull, slot, token);
                    const unsigned char* src = (lane < 16 ? p.k_scales : p.v_scales) + (from_slot < 0 ? 0 : from_slot) * (D / kBlock4);
                    const uint32_t dst = to + 2 * C::kCodes + (lane < 16 ? 0 : C::kScales) + (quarter + token) * (D / kBlock4);
                    if (l < kLanes) tc::copy16_or_zeros(dst, src, from_slot >= 0);
                }
                tc::copies_arrive(&ctl->full[at]);
            }
        }
        tc::copies_done();  // no copy outlives the block, whatever its readers did
    }
    __syncthreads();
    if (tid == 0) {
        p.fragments.gave_up[blockIdx.x] = *abort;
        if (*abort != 0) atomicOr(p.status, kStatusAttnTimeout);
    }
}

template <int D>
constexpr int smem_bytes4() { return Cfg4<D>::kCtl + (int)sizeof(Ctl4); }

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
    lc.blockDim = dim3(kThreads);
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

int pick_wide(const AttendParams& p) {
    const bool groups = (long long)p.rows * p.share > 32LL * p.G;
    return (p.P > 0 ? kWidePrefixes : 0) | (groups ? kWideGroups : 0);
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
