// lp_join.h -- the join of an attention call: a row's attention to the round's
// own tokens, and the parts that the main kernel left of its prefix and of its
// group's committed tokens.
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
#pragma once

#include "lp_split.h"
#include "lp_tc.h"

namespace lp {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

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

// Eight lanes in 4 bits with their block's scale byte; exact.
__device__ __forceinline__ void widen_four(uint32_t codes, uint32_t scale, float* x) {
    uint32_t s;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(s) : "r"(scale));
    const float f = Half<false>::unpack(s).x;
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = Half<false>::unpack(h[i]);
        x[2 * i] = v.x * f, x[2 * i + 1] = v.y * f;
    }
}

// The parts of a row's head from one segment: what the call's arguments say,
// and after the main kernel what its tables say.
template <bool kFour>
struct Parts {
    int seg, unit, dealt;     // seg: -1 for none; of all heads' units
    int row, cap, set, sets;  // row of the unit; the parts of a piece that are its: sets of them from `set` on
    int count;
    long long slot;
    bool pairs;               // units of pairs of tiles
    template <class Rule>
    __device__ __forceinline__ void find_by(const AttendParams& p, int segment, int of, int head) {
        const Seg<Rule> s = load_seg<Rule>(p, segment);
        if (s.tiles == 0) return;
        seg = segment;
        const int rt = p.rows_per_tile, unit_rows = Rule::unit_rows(p), rel = of - s.r0, u = rel / unit_rows, in = rel - u * unit_rows, kvh = head / p.share;
        const bool two = Rule::kPairs && s.n - u * unit_rows > rt;
        unit = kvh * s.units + u;
        dealt = s.dealt;
        set = two && in >= rt ? 1 : 0;
        sets = two ? 1 : Rule::kSets;  // a unit of one tile: a part of each warpgroup
        row = (in - set * rt) * p.share + head - kvh * p.share;
        cap = segment < p.P ? Rule::kPrefixRows : Rule::scratch(p).group_rows;
    }
    __device__ __forceinline__ void find(const AttendParams& p, int segment, int of, int head) {  // of: the row
        seg = -1;
        pairs = true;
        if (segment < 0) return;
        if constexpr (kFour) {
            pairs = Pairs4::takes(p, segment < p.P);
            if (pairs) find_by<Pairs4>(p, segment, of, head);
            else find_by<Fragments>(p, segment, of, head);
        } else {
            find_by<Pairs>(p, segment, of, head);
        }
    }
    __device__ __forceinline__ const AttendScratch& scratch(const AttendParams& p) const { return kFour && !pairs ? p.fragments : p.sc; }
    __device__ __forceinline__ int2 first_slots(const AttendParams& p) const { return seg >= 0 ? scratch(p).seg_units[seg] : make_int2(0, 0); }
    __device__ __forceinline__ void locate(const AttendParams& p, int2 base) {
        const AttendScratch& sc = scratch(p);
        slot = (long long)base.y + unit;
        int pieces = seg >= 0 ? 1 : 0;
        if (pieces != 0 && unit >= dealt) {
            const long long at = unit_index(sc, seg < p.P, base.x + unit - dealt);
            const int2 e = at >= 0 ? sc.units[at] : make_int2(0, 0);
            slot = e.x;
            pieces = entry_pieces(e.x, e.y, seg < p.P ? sc.prefix_slots : sc.group_slots, p.grid);
        }
        count = pieces * sets;
    }
    __device__ __forceinline__ long long part(const AttendParams& p, int k) const {
        const long long at = slot + (sets == 1 ? k : k >> 1);
        const int s = sets == 1 ? set : k & 1;
        if (kFour && !pairs) return part_row<Fragments>(p, seg < p.P, at, s);
        return part_row<Pairs>(p, seg < p.P, at, s);
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
// With heads of 128 the forms of one and two warps per row spill at the 64
// registers that four blocks per SM leave: 28 bytes a thread (F16: 36), over a
// cache in 4 bits, two tokens of whose words wait in registers, 80 (148 reloaded).
template <bool kBf16, int D, int kSub, bool kFour>
__global__ void __launch_bounds__(kJoinThreads, join_blocks(kSub)) lp_attend_join_kernel(const AttendParams p) {
    using H = Half<kBf16>;
    using T = typename H::T;
    constexpr int kE = D / 8, kRuns = D / 64, kRound = join_round(kSub);
    // What is on its way to a warp, 16 bytes of every thread side by side: on lines of 128 bytes (one row at 4,095 tokens:
    // 15.3 us; wherever the words before it end, 17.1).
    extern __shared__ __align__(128) unsigned char join_smem[];
    uint4* stage = reinterpret_cast<uint4*>(join_smem) + threadIdx.x;
    float2* stage_ml = reinterpret_cast<float2*>(join_smem + kRound * 2 * kRuns * kJoinThreads * 16) + threadIdx.x;
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
        const int j = row - grp.r0;
        const unsigned mask = p.row_masks != nullptr ? p.row_masks[row] : (2u << j) - 1u;
        int page = 0;  // lane i: of token i
        if (lane < grp.n) page = p.tables[(long long)g * p.max_pages + ((grp.len + lane) >> p.page_shift)];
        const unsigned here = __ballot_sync(kFull, page >= 0 && page < p.num_pages);
        unsigned todo = mask & (grp.n < 32 ? (1u << grp.n) - 1u : kFull);
        if (lane == 0 && (todo & ~here) != 0u) atomicOr(p.status, kStatusBadPage);
        if (kSub > 1) todo &= kFull / ((1u << kSub) - 1u) << sub;  // every kSub-th is this warp's
        const int n = __popc(todo);
        if constexpr (kFour) {
            // A thread's lanes of a token are kRuns words of codes, each of one block, of K and of V: few enough to load two
            // tokens' at once into registers.
            const int kvh = exists ? head / p.share : 0;
            // in two factors: what the first one, kept to FP32's normal numbers, lacks (1, as a rule) is the second
            const float ck = scaled(p.score, p.score_exp), more = scaled(1.0f, p.score_exp - exponent_of(ck));
#pragma unroll 1
            for (int j = 0; j < n; j += 2) {
                uint32_t w[2][2][kRuns], e[2][2][kRuns];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int i = todo != 0u ? __ffs(todo) - 1 : 0, t = grp.len + i;
                    const bool read = todo != 0u && (here >> i & 1u) != 0u;
                    todo &= todo - 1u;
                    const long long pg = __shfl_sync(kFull, page, i);
                    const long long slot = ((pg * p.kv_heads + kvh) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
#pragma unroll
                    for (int r = 0; r < kRuns; ++r) {
                        w[u][0][r] = w[u][1][r] = e[u][0][r] = e[u][1][r] = 0u;
                        if (!read) continue;
                        w[u][0][r] = reinterpret_cast<const uint32_t*>(p.k_cache)[slot * (D / 8) + r * 8 + l];
                        w[u][1][r] = reinterpret_cast<const uint32_t*>(p.v_cache)[slot * (D / 8) + r * 8 + l];
                        e[u][0][r] = p.k_scales[slot * (D / kBlock4) + r * 4 + (l >> 1)];
                        e[u][1][r] = p.v_scales[slot * (D / kBlock4) + r * 4 + (l >> 1)];
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (j + u >= n) break;
                    float k[kE], v[kE];
#pragma unroll
                    for (int r = 0; r < kRuns; ++r) widen_four(w[u][0][r], e[u][0][r], k + r * 8), widen_four(w[u][1][r], e[u][1][r], v + r * 8);
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < kE; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
                    for (int o = 16; o > 2; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                    a.add(s * ck * more, 1.0f, v);
                }
            }
        } else {
            const float c = p.scale * kLog2e;
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
    }
    // Of the first prefix that serves the row, of its group's committed tokens.  A prefix has parts for the rows from its first
    // group's to its last's: a group whose rows lie elsewhere (group_indptr then does not ascend) is not served.
    Parts<kFour> shared, own;
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
    for (int b = threadIdx.x; b < p.grid; b += kJoinThreads) {
        if constexpr (kFour) {
            if (runs_pairs(p)) gave_up |= p.sc.gave_up[b];
            if (runs_fragments(p)) gave_up |= p.fragments.gave_up[b];
        } else {
            gave_up |= p.sc.gave_up[b];
        }
    }
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
            const AttendScratch& sc = is_own ? own.scratch(p) : shared.scratch(p);
            if (base < 0) {
                stage_ml[slot * kJoinThreads] = make_float2(kNegInf, 0.0f);
            } else {
                tc::copy8(tc::smem_addr(&stage_ml[slot * kJoinThreads]), sc.part_ml + base + row_at);
                const float4* src = reinterpret_cast<const float4*>(sc.part_o) + part_chunk<D>(base, cap, row_at, 2 * l);
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
        float* part = reinterpret_cast<float*>(join_smem);  // [e][thread]; then the maxima and sums
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
    // the factor last: a small one, divided by the sum, would lose bits below FP32's normal numbers
    auto lane_of = [&](int e) { return kFour ? a.o[e] * inv * p.v_factor : a.o[e] * inv; };
    T* dst = reinterpret_cast<T*>(p.out) + row * p.out_stride + (long long)head * D + l * 8;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
        uint4 w;
        w.x = H::pack(lane_of(r * 8), lane_of(r * 8 + 1));
        w.y = H::pack(lane_of(r * 8 + 2), lane_of(r * 8 + 3));
        w.z = H::pack(lane_of(r * 8 + 4), lane_of(r * 8 + 5));
        w.w = H::pack(lane_of(r * 8 + 6), lane_of(r * 8 + 7));
        *reinterpret_cast<uint4*>(dst + r * 64) = w;
    }
    if (p.lse_out != nullptr && l == 0) p.lse_out[(long long)row * p.q_heads + head] = a.l == 0.0f ? kNegInf : a.m * kLn2 + logf(a.l);
}

template <bool kBf16, int D, bool kFour>
cudaError_t prepare_join() {
    const cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 8, kFour>, most, join_bytes<D>(8));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 4, kFour>, most, join_bytes<D>(4));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 2, kFour>, most, join_bytes<D>(2));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(lp_attend_join_kernel<kBf16, D, 1, kFour>, most, join_bytes<D>(1));
    return e;
}

// `lc`: the main kernel's launch, whose stream and attributes the join's has too.
template <bool kBf16, int D, bool kFour>
cudaError_t launch_join(const AttendParams& p, cudaLaunchConfig_t lc) {
    // the most warps per row with which all blocks are resident at once: one row takes 15.5 us (one warp: 24.7), trees of
    // drafts 43.6 (one: 46.3, eight: 60), 2,048 rows behind a prefix 765 (eight: 1,015)
    const int chunks = (p.q_heads + 3) / 4;
    int sub = 8;
    auto per_row = [&]() { return (chunks * sub + kJoinWarps - 1) / kJoinWarps; };  // blocks
    while (sub > 1 && per_row() * (long long)p.rows > join_blocks(sub) * p.grid) sub /= 2;
    lc.gridDim = dim3((unsigned)p.rows, (unsigned)per_row());
    lc.blockDim = dim3(kJoinThreads);
    lc.dynamicSmemBytes = join_bytes<D>(sub);
    if (sub == 8) return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 8, kFour>, p);
    if (sub == 4) return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 4, kFour>, p);
    if (sub == 2) return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 2, kFour>, p);
    return cudaLaunchKernelEx(&lc, lp_attend_join_kernel<kBf16, D, 1, kFour>, p);
}

}  // namespace
}  // namespace lp
