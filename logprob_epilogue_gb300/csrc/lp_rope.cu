// lp_rope.cu -- sm_103a kernel of lp_norm_rope and lp_kv_append: RMS norm and
// position rotation of query and key heads, keys and values into the paged
// cache.
//
// Per head x of D lanes: y = x * rsqrt(mean(x^2) + eps) * (offset + w), then
// each pair (a, b) of the first `rot` lanes becomes (a cos - b sin, b cos + a
// sin), in FP32, with the one rounding at the store.  With the weights folded
// into the rotation a lane is
//   y = rs * (x * (cos (offset + w)) + x' * (+-sin (offset + w'))),
// x' the pair's other lane: two products per lane, the factors the same for
// every head of a row.
//
// D / 8 threads hold a head, eight consecutive lanes (one 16-byte word) each.
// The mean square is a shuffle reduction among them; the other lane of a
// half-split pair (rot / 2 lanes away, a multiple of 8) sits at the same place
// of another thread's word, so it comes with four shuffles of the words as
// loaded.  A task is one row and up to four (eight) heads of one of q, k and v:
// their loads are in flight before anything is waited for, and the row's
// factors are formed once for them.  No shared memory.
//
// Bound: bytes in and out, and close behind them the instructions (about 75
// per word).  16,411 rows of 32 + 8 + 8 heads of 128 lanes, BF16, into a cache:
// 79 us, 6.0 TB/s; 8,191 rows of 24 + 4 heads of 64 lanes, F16: 13.0 us, 4.6
// TB/s; one row into a cache: 3.2 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "lp_attn.h"

namespace lp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRopeThreads = 128;

__host__ __device__ constexpr int chunks_of(int heads, int per) { return (heads + per - 1) / per; }

template <bool kBf16>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8]) {
    using H = Half<kBf16>;
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = H::unpack(a[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}

template <bool kBf16, int D, bool kAppend, int kHeads>  // heads per task
__global__ void __launch_bounds__(kRopeThreads, kHeads == 8 ? 6 : 8) lp_rope_kernel(RopeParams p) {
    using H = Half<kBf16>;
    using T = typename H::T;
    constexpr int kLanes = D / 8;                  // threads per head
    constexpr int kTasks = kRopeThreads / kLanes;  // tasks per block
    const int lane = threadIdx.x % kLanes, e0 = lane * 8;
    const int cq = chunks_of(p.q_heads, kHeads), ck = chunks_of(p.kv_heads, kHeads), per_row = cq + (kAppend ? 2 : 1) * ck;
    const unsigned first = blockIdx.x * kTasks, task = first + threadIdx.x / kLanes;
    const unsigned at = task / per_row;
    const bool live = at < (unsigned)p.rows;
    const int row = live ? (int)at : 0;
    const int c = (int)(task - at * per_row);
    const int kind = c < cq ? 0 : (c < cq + ck ? 1 : 2);  // q, k, v
    const int h0 = (kind == 0 ? c : (kind == 1 ? c - cq : c - cq - ck)) * kHeads;
    const int heads = (kind == 0 ? p.q_heads : p.kv_heads) - h0, n = !live ? 0 : (heads < kHeads ? heads : kHeads);
    const T* src = kind == 0   ? reinterpret_cast<const T*>(p.q) + row * p.q_stride
                   : kind == 1 ? reinterpret_cast<const T*>(p.k) + row * p.k_stride
                               : reinterpret_cast<const T*>(p.v) + row * p.v_stride;
    src += h0 * D + e0;

    // Resident before the kernel ahead has ended: nothing is read before this wait, and with ordinary loads, since read-only
    // ones might be moved ahead of it.
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // the heads' words, whatever the row's position
    uint4 w[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i < n) w[i] = __ldcs(reinterpret_cast<const uint4*>(src + i * D));
    }
    const int pos = live ? p.positions[row] : -1;
    const void* weight = kind == 0 ? p.q_weight : (kind == 1 ? p.k_weight : nullptr);
    int g = -1;
    bool ascends = true;
    if constexpr (kAppend) {
        g = block_find_group(p.indptr, p.G, (int)(first / per_row), ascends);
        if (!ascends && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusAttnBadGroup);
    }
    if (pos >= p.max_pos && lane == 0 && c == 0) atomicOr(p.status, kStatusBadPosition);
    const bool work = pos >= 0 && pos < p.max_pos;

    // the cache slot of the row's token: (page * kv_heads) * page_size + offset, head 0
    long long slot = -1;
    if constexpr (kAppend) {
        if (work && kind != 0) {
            if (ascends) {
                if (g < 0) g = 0;
                while (g < p.G && p.indptr[g + 1] <= row) ++g;
            } else {  // the one group that claims the row
                int claims = 0;
                for (int i = 0; i < p.G; ++i)
                    if (p.indptr[i] <= row && row < p.indptr[i + 1]) ++claims, g = i;
                if (claims != 1) g = p.G;
            }
            if (g < p.G) {
                const int r0 = p.indptr[g], r1 = p.indptr[g + 1], len = p.lens[g];
                if (row >= r0 && len >= 0) {
                    const long long t = (long long)len + row - r0;
                    const bool fits = r0 >= 0 && r1 <= p.rows &&
                                      (long long)len + (r1 - r0) <= ((long long)p.max_pages << p.page_shift);
                    if (!fits) {
                        if (lane == 0) atomicOr(p.status, kStatusAttnBadGroup);
                    } else {
                        const int page = p.tables[(long long)g * p.max_pages + (t >> p.page_shift)];
                        if (page < 0 || page >= p.num_pages) {
                            if (lane == 0) atomicOr(p.status, kStatusBadPage);
                        } else {
                            slot = (((long long)page * p.kv_heads) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
                        }
                    }
                }
            }
            slot += slot >= 0 ? (long long)h0 << p.page_shift : 0;
        }
    }
    const long long step = (long long)D << p.page_shift;  // elements from a head's slot to the next's

    // factors of a lane and of its pair's other one, the weights in them
    const int half = p.rot >> 1;
    const bool turn = kind != 2 && work && e0 < p.rot;
    float fa[8], fb[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) fa[e] = 1.0f, fb[e] = 0.0f;
    // a half-split pair's other thread (threads past rot: their own)
    const int mate = (p.interleaved || e0 >= p.rot) ? lane : (e0 < half ? lane + half / 8 : lane - half / 8);
    if (turn) {
        const float* t = p.cos_sin + (long long)pos * p.rot;
        if (p.interleaved) {
            const float4 cc = *reinterpret_cast<const float4*>(t + e0 / 2);
            const float4 ss = *reinterpret_cast<const float4*>(t + half + e0 / 2);
            const float a[4] = {cc.x, cc.y, cc.z, cc.w}, b[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) fa[e] = a[e / 2], fb[e] = (e & 1) ? b[e / 2] : -b[e / 2];
        } else {
            const int i0 = e0 < half ? e0 : e0 - half;
            const float sign = e0 < half ? -1.0f : 1.0f;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4 cc = reinterpret_cast<const float4*>(t + i0)[v];
                const float4 ss = reinterpret_cast<const float4*>(t + half + i0)[v];
                fa[4 * v] = cc.x, fa[4 * v + 1] = cc.y, fa[4 * v + 2] = cc.z, fa[4 * v + 3] = cc.w;
                fb[4 * v] = sign * ss.x, fb[4 * v + 1] = sign * ss.y, fb[4 * v + 2] = sign * ss.z, fb[4 * v + 3] = sign * ss.w;
            }
        }
    }
    if (weight != nullptr) {
        float u[8], v[8];
        widen8<kBf16>(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(weight) + e0), u);
        widen8<kBf16>(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(weight) + mate * 8), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            fa[e] *= p.weight_offset + u[e];
            fb[e] *= p.weight_offset + (p.interleaved ? u[e ^ 1] : v[e]);
        }
    }

    T* dst = nullptr;
    if (kind == 0) dst = reinterpret_cast<T*>(p.q_out) + row * p.q_out_stride + h0 * D + e0;
    else if (kind == 1 && p.k_out != nullptr) dst = reinterpret_cast<T*>(p.k_out) + row * p.k_out_stride + h0 * D + e0;
    T* cache = nullptr;
    if constexpr (kAppend) {
        if (slot >= 0) cache = reinterpret_cast<T*>(kind == 1 ? p.k_cache : p.v_cache) + slot * D + e0;
    }
    const bool norms = p.q_weight != nullptr || p.k_weight != nullptr, turns = p.rot > 0 && !p.interleaved;  // of the call
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        float x[8], o[8];
        widen8<kBf16>(w[i], x);
        float rs = 1.0f;
        if (norms) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int s = kLanes / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(kFull, ss, s, kLanes);
            if (weight != nullptr) rs = rsqrtf(ss * (1.0f / D) + p.eps);
        }
        if (turns) {
            uint4 m;
            m.x = __shfl_sync(kFull, w[i].x, mate, kLanes);
            m.y = __shfl_sync(kFull, w[i].y, mate, kLanes);
            m.z = __shfl_sync(kFull, w[i].z, mate, kLanes);
            m.w = __shfl_sync(kFull, w[i].w, mate, kLanes);
            widen8<kBf16>(m, o);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
        }
        if (!work || i >= n) continue;
        uint4 y = w[i];  // values go as they are
        if (kind != 2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = x[e] * fa[e];
                x[e] = (turn ? fmaf(o[e], fb[e], z) : z) * rs;
            }
            y.x = H::pack(x[0], x[1]);
            y.y = H::pack(x[2], x[3]);
            y.z = H::pack(x[4], x[5]);
            y.w = H::pack(x[6], x[7]);
        }
        if (dst != nullptr) __stcs(reinterpret_cast<uint4*>(dst + i * D), y);
        if (kAppend && cache != nullptr) *reinterpret_cast<uint4*>(cache + i * step) = y;
    }
}

template <bool kBf16, int D, int kHeads>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
    const bool append = p.k_cache != nullptr;
    const long long tasks = (long long)p.rows * (chunks_of(p.q_heads, kHeads) + (append ? 2 : 1) * chunks_of(p.kv_heads, kHeads));
    constexpr int kTasks = kRopeThreads / (D / 8);
    const unsigned grid = (unsigned)((tasks + kTasks - 1) / kTasks);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(grid);
    lc.blockDim = dim3(kRopeThreads);
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return append ? cudaLaunchKernelEx(&lc, lp_rope_kernel<kBf16, D, true, kHeads>, p)
                  : cudaLaunchKernelEx(&lc, lp_rope_kernel<kBf16, D, false, kHeads>, p);
}

// Eight heads per task spread a row's factors further, but leave a short call
// fewer threads and a long chain of its own: with 128 lanes, 16,411 rows of 48
// heads take 79 us against 82, 512 rows 5.0 us against 4.4; with 64 lanes 8,191
// rows of 28 heads take 14.8 us against 13.0.
constexpr long long kManyHeads = 1 << 18;

template <bool kBf16>
cudaError_t pick(const RopeParams& p, int head_dim, cudaStream_t stream) {
    if (head_dim == 64) return launch<kBf16, 64, 4>(p, stream);
    return (long long)p.rows * (p.q_heads + p.kv_heads) >= kManyHeads ? launch<kBf16, 128, 8>(p, stream) : launch<kBf16, 128, 4>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream) {
    return dtype == 1 ? pick<true>(p, head_dim, stream) : pick<false>(p, head_dim, stream);
}

}  // namespace lp
