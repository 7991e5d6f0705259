// lp_attend.cu -- sm_103a kernels of lp_attend: attention of verify rows over
// a paged cache with shared prefixes.
//
// For a row's query head q over its visible tokens t:
//   s_t = scale q.k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t exp s_t.
//
// One warp per (row, query head), D / 32 lanes of the head per thread: one
// pass over the tokens with the running maximum and sum of the softmax, FP32
// throughout.
#include <cuda_runtime.h>
#include <stdint.h>

#include "lp_attn.h"

namespace lp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kThreads = 256;

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

// Prefix p: its groups' rows and its tokens.  len = 0: none, or malformed.
struct Prefix {
    int g0, g1, len;
    bool bad;
};

__device__ __forceinline__ Prefix load_prefix(const AttendParams& p, int i) {
    Prefix x;
    x.g0 = __ldg(&p.prefix_indptr[i]);
    x.g1 = __ldg(&p.prefix_indptr[i + 1]);
    x.len = __ldg(&p.prefix_lens[i]);
    x.bad = x.g0 < 0 || x.g1 < x.g0 || x.g1 > p.G || x.len < 0 ||
            (long long)x.len > ((long long)p.max_prefix_pages << p.page_shift);
    if (x.bad) x.len = 0;
    return x;
}

template <bool kBf16, int D>
struct Acc {
    static constexpr int kE = D / 32;  // lanes of the head per thread
    float q[kE], o[kE], m, l;          // q scaled by scale * log2(e)
};

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

// Adds token t of the table to the running softmax.
template <bool kBf16, int D>
__device__ __forceinline__ void visit(const AttendParams& p, Acc<kBf16, D>& a, const int* table, int t, int kvh, int lane) {
    constexpr int kE = D / 32;
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
    for (int e = 0; e < kE; ++e) s = fmaf(a.q[e], k[e], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    const float m = fmaxf(a.m, s);
    const float base = m == kNegInf ? 0.0f : m;
    const float f = ex2(a.m - base), w = ex2(s - base);
    a.l = a.l * f + w;
#pragma unroll
    for (int e = 0; e < kE; ++e) a.o[e] = a.o[e] * f + w * v[e];
    a.m = m;
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads) lp_attend_kernel(AttendParams p) {
    using H = Half<kBf16>;
    using T = typename H::T;
    constexpr int kE = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, head = blockIdx.y * (kThreads / 32) + warp;
    if (blockIdx.x == 0 && blockIdx.y == 0) {  // the malformed groups and prefixes of the call
        for (int i = threadIdx.x; i < p.G; i += kThreads)
            if (load_group(p, i).bad) atomicOr(p.status, kStatusAttnBadGroup);
        for (int i = threadIdx.x; i < p.P; i += kThreads)
            if (load_prefix(p, i).bad) atomicOr(p.status, kStatusBadPrefix);
    }
    const int g = block_find_group(p.indptr, p.G, row);
    if (g < 0 || g >= p.G || head >= p.q_heads) return;
    if (row < __ldg(&p.indptr[g]) || row >= __ldg(&p.indptr[g + 1])) return;  // two entries claim the row
    const Group grp = load_group(p, g);
    const int kvh = head / p.share;
    Acc<kBf16, D> a;
    load_lane<kBf16, D>(p.q, row * p.q_stride + (long long)head * D + lane * kE, a.q);
#pragma unroll
    for (int e = 0; e < kE; ++e) a.q[e] *= p.scale * kLog2e, a.o[e] = 0.0f;
    a.m = kNegInf, a.l = 0.0f;
    if (grp.n > 0) {
        for (int i = 0; i < p.P; ++i) {
            const Prefix x = load_prefix(p, i);
            if (g < x.g0 || g >= x.g1) continue;
            const int* table = p.prefix_tables + (long long)i * p.max_prefix_pages;
            for (int t = 0; t < x.len; ++t) visit<kBf16, D>(p, a, table, t, kvh, lane);
            break;
        }
        const int* table = p.tables + (long long)g * p.max_pages;
        for (int t = 0; t < grp.len; ++t) visit<kBf16, D>(p, a, table, t, kvh, lane);
        const int j = row - grp.r0;
        const unsigned mask = p.row_masks != nullptr ? __ldg(&p.row_masks[row]) : (2u << j) - 1u;
        for (int i = 0; i < grp.n; ++i)
            if (mask >> i & 1u) visit<kBf16, D>(p, a, table, grp.len + i, kvh, lane);
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

template <bool kBf16, int D>
cudaError_t launch(const AttendParams& p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.rows, (unsigned)((p.q_heads + kThreads / 32 - 1) / (kThreads / 32)));
    lp_attend_kernel<kBf16, D><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, int dtype, int head_dim, cudaStream_t stream) {
    if (dtype == 1) return head_dim == 128 ? launch<true, 128>(p, stream) : launch<true, 64>(p, stream);
    return head_dim == 128 ? launch<false, 128>(p, stream) : launch<false, 64>(p, stream);
}

}  // namespace lp
