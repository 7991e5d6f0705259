// lp_rope.cu -- sm_103a kernel of lp_norm_rope and lp_kv_append: RMS norm and
// position rotation of query and key heads, keys and values into the paged
// cache.
//
// Per head x of D lanes: y = x * rsqrt(mean(x^2) + eps) * (offset + w), then
// each pair (a, b) of the first `rot` lanes becomes (a cos - b sin, b cos + a
// sin), in FP32, with the one rounding at the store.
//
// D / 8 threads hold a head, eight consecutive lanes (one 16-byte word) each:
// the mean square is a shuffle reduction among them, the partner of a rotated
// lane (rot / 2 lanes away, a multiple of 8) sits at the same place of another
// thread's word, so the rotation is one more shuffle and no shared memory is
// needed.  A task is one row and four heads: four loads in flight per thread,
// and the row's cos and sin are loaded once for the four.  Bound: bytes in and
// out.
#include <cuda_runtime.h>
#include <stdint.h>

#include "lp_attn.h"

namespace lp {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRopeThreads = 256;
constexpr int kHeads = 4;  // heads per task

template <bool kBf16, int D, bool kAppend>
__global__ void __launch_bounds__(kRopeThreads) lp_rope_kernel(RopeParams p) {
    using H = Half<kBf16>;
    using T = typename H::T;
    constexpr int kLanes = D / 8;                     // threads per head
    constexpr int kTasks = kRopeThreads / kLanes;     // tasks per block
    const int lane = threadIdx.x % kLanes;
    const int heads = p.q_heads + (kAppend ? 2 : 1) * p.kv_heads;
    const int per_row = (heads + kHeads - 1) / kHeads;
    const long long first = (long long)blockIdx.x * kTasks;
    const long long task = first + threadIdx.x / kLanes;
    int g = -1;
    if constexpr (kAppend) g = block_find_group(p.indptr, p.G, (int)(first / per_row));
    const long long row64 = task / per_row;
    const bool live = row64 < p.rows;
    const int row = live ? (int)row64 : 0;
    const int h0 = (int)(task % per_row) * kHeads;
    const int pos = live ? __ldg(&p.positions[row]) : -1;
    if (pos >= p.max_pos && lane == 0 && h0 == 0) atomicOr(p.status, kStatusBadPosition);
    const bool work = live && pos >= 0 && pos < p.max_pos;
    const int e0 = lane * 8;

    // loads: four heads' words, then the row's cos and sin
    uint4 w[kHeads] = {};
    if (work) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i;
            if (h >= heads) continue;
            const T* src;
            if (h < p.q_heads) src = reinterpret_cast<const T*>(p.q) + row * p.q_stride + (long long)h * D;
            else if (!kAppend || h < p.q_heads + p.kv_heads)
                src = reinterpret_cast<const T*>(p.k) + row * p.k_stride + (long long)(h - p.q_heads) * D;
            else
                src = reinterpret_cast<const T*>(p.v) + row * p.v_stride + (long long)(h - p.q_heads - p.kv_heads) * D;
            w[i] = *reinterpret_cast<const uint4*>(src + e0);
        }
    }
    const int half = p.rot >> 1;
    float cs[8], sn[8];  // y_e = x_e * cs + partner * sn
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 1.0f, sn[e] = 0.0f;
    if (work && e0 < p.rot) {
        const float* t = p.cos_sin + (long long)pos * p.rot;
        if (p.interleaved) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(t + e0 / 2));
            const float4 s = __ldg(reinterpret_cast<const float4*>(t + half + e0 / 2));
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) cs[e] = cc[e / 2], sn[e] = (e & 1) ? ss[e / 2] : -ss[e / 2];
        } else {
            const int i0 = e0 < half ? e0 : e0 - half;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4 c = __ldg(reinterpret_cast<const float4*>(t + i0) + v);
                const float4 s = __ldg(reinterpret_cast<const float4*>(t + half + i0) + v);
                const float sign = e0 < half ? -1.0f : 1.0f;
                cs[4 * v] = c.x, cs[4 * v + 1] = c.y, cs[4 * v + 2] = c.z, cs[4 * v + 3] = c.w;
                sn[4 * v] = sign * s.x, sn[4 * v + 1] = sign * s.y, sn[4 * v + 2] = sign * s.z, sn[4 * v + 3] = sign * s.w;
            }
        }
    }
    // the partner's thread (half-split pairs): threads past rot keep their own
    const int mate = (p.interleaved || e0 >= p.rot) ? lane : (e0 < half ? lane + half / 8 : lane - half / 8);

    // the cache slot of the row's token
    long long slot = -1;  // (page * kv_heads) * page_size + offset, head 0
    if constexpr (kAppend) {
        if (work && h0 + kHeads > p.q_heads) {
            if (g < 0) g = 0;
            while (g < p.G && __ldg(&p.indptr[g + 1]) <= row) ++g;
            if (g < p.G) {
                const int r0 = __ldg(&p.indptr[g]), r1 = __ldg(&p.indptr[g + 1]), len = __ldg(&p.lens[g]);
                if (row >= r0 && len >= 0) {
                    const long long t = (long long)len + (row - r0);
                    const bool fits = r0 >= 0 && r1 <= p.rows &&
                                      (long long)len + (r1 - r0) <= ((long long)p.max_pages << p.page_shift);
                    if (!fits) {
                        if (lane == 0) atomicOr(p.status, kStatusAttnBadGroup);
                    } else {
                        const int page = __ldg(&p.tables[(long long)g * p.max_pages + (t >> p.page_shift)]);
                        if (page < 0 || page >= p.num_pages) {
                            if (lane == 0) atomicOr(p.status, kStatusBadPage);
                        } else {
                            slot = (((long long)page * p.kv_heads) << p.page_shift) + (t & ((1 << p.page_shift) - 1));
                        }
                    }
                }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        const bool is_q = h < p.q_heads, is_k = !is_q && h < p.q_heads + p.kv_heads;
        const bool turn = h < heads && (is_q || is_k);
        const void* weight = is_q ? p.q_weight : (is_k ? p.k_weight : nullptr);
        float x[8];
        {
            const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = H::unpack(a[j]);
                x[2 * j] = f.x;
                x[2 * j + 1] = f.y;
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o, kLanes);
        if (weight != nullptr && h < heads) {
            const float rs = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
            const uint4 ww = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(weight) + e0));
            const uint32_t a[4] = {ww.x, ww.y, ww.z, ww.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = H::unpack(a[j]);
                x[2 * j] *= rs * (p.weight_offset + f.x);
                x[2 * j + 1] *= rs * (p.weight_offset + f.y);
            }
        }
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float other = __shfl_sync(kFull, x[e], mate, kLanes);  // the thread's own lane when interleaved
            const float partner = p.interleaved ? x[e ^ 1] : other;
            y[e] = (turn && e0 < p.rot) ? x[e] * cs[e] + partner * sn[e] : x[e];
        }
        if (!work || h >= heads) continue;
        uint4 o;
        o.x = H::pack(y[0], y[1]);
        o.y = H::pack(y[2], y[3]);
        o.z = H::pack(y[4], y[5]);
        o.w = H::pack(y[6], y[7]);
        if (is_q) {
            *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.q_out) + row * p.q_out_stride + (long long)h * D + e0) = o;
        } else if (is_k) {
            const int kh = h - p.q_heads;
            if (p.k_out != nullptr)
                *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.k_out) + row * p.k_out_stride + (long long)kh * D + e0) = o;
            if constexpr (kAppend) {
                if (slot >= 0)
                    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.k_cache) + (slot + ((long long)kh << p.page_shift)) * D + e0) = o;
            }
        } else if constexpr (kAppend) {
            const int vh = h - p.q_heads - p.kv_heads;
            if (slot >= 0)  // unchanged bits
                *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.v_cache) + (slot + ((long long)vh << p.page_shift)) * D + e0) = w[i];
        }
    }
}

template <bool kBf16, int D>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
    const bool append = p.k_cache != nullptr;
    const int heads = p.q_heads + (append ? 2 : 1) * p.kv_heads;
    const long long tasks = (long long)p.rows * ((heads + kHeads - 1) / kHeads);
    constexpr int kTasks = kRopeThreads / (D / 8);
    const unsigned grid = (unsigned)((tasks + kTasks - 1) / kTasks);
    if (append) lp_rope_kernel<kBf16, D, true><<<grid, kRopeThreads, 0, stream>>>(p);
    else lp_rope_kernel<kBf16, D, false><<<grid, kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream) {
    if (dtype == 1) return head_dim == 128 ? launch<true, 128>(p, stream) : launch<true, 64>(p, stream);
    return head_dim == 128 ? launch<false, 128>(p, stream) : launch<false, 64>(p, stream);
}

}  // namespace lp
