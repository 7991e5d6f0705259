// lp_attn.h -- shared between the attention plan's host code and its kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lp {

constexpr int kAttnMaxGroupRows = 32;
constexpr unsigned kStatusAttnBadGroup = 0x8u, kStatusAttnTimeout = 0x10u, kStatusBadPosition = 0x40u,
                   kStatusBadPage = 0x80u, kStatusBadPrefix = 0x100u;

struct RopeParams {
    const void *q, *k, *v;                 // [rows, heads, D]; v: append only
    void *q_out, *k_out;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // elements
    const void *q_weight, *k_weight;       // [D] or null
    const float* cos_sin;                  // [max_pos, rot]
    const int* positions;
    unsigned int* status;
    float eps, weight_offset;
    int max_pos, rot, interleaved;
    int rows, q_heads, kv_heads;           // q_heads 0: no q; kv_heads 0: no k
    // append (k_cache != nullptr)
    const int *indptr, *lens, *tables;
    void *k_cache, *v_cache;
    int G, max_pages, page_shift;
    long long num_pages;
};

constexpr int kQTile = 128;    // query rows (row, head) of one tensor-core tile
constexpr int kKTile = 128;    // tokens of one tile

// Scratch of lp_attend.  A segment is a prefix or a group's committed tokens;
// a unit is at most two tiles of its query rows for one key-value head; a
// piece is the run of a unit's token tiles that one block takes.
struct AttendScratch {
    int2* seg_units;                // [P + G] units before the segment, of those that are cut into pieces and of those that
                                    // go round the blocks whole
    int2* units;                    // of prefixes, then of groups: a cut unit's first slot and its pieces
    int* gave_up;                   // [grid] the block's waits ran out in the last call
    float* part_o;                  // pieces of prefixes, then of groups: unnormalised results [2][rows][D]
    float2* part_ml;                // (maximum in base 2, sum) [2][rows]
    long long prefix_slots, group_slots;
    int group_rows;                 // rows per tile in a group slot (prefix slots: kQTile)
};

struct AttendParams {
    const void* q;
    long long q_stride, out_stride;
    const void *k_cache, *v_cache;
    const int *indptr, *lens, *tables;
    const unsigned int* row_masks;
    const int *prefix_indptr, *prefix_lens, *prefix_tables;
    void* out;
    float* lse_out;
    unsigned int* status;
    float scale;
    int rows, G, P;
    int q_heads, kv_heads, share;          // share = q_heads / kv_heads
    int max_group_rows, max_pages, max_prefix_pages, page_shift;
    long long num_pages;
    int rows_per_tile;                     // kQTile / share
    int share_inv;                         // row / share = row * share_inv >> 16 for rows of a tile
    int grid;                              // blocks of the attention kernel
    AttendScratch sc;
    unsigned long long timeout_ns;
    int force_timeout;
};

// The pieces of a cut unit as the join may take them from its entry (first
// slot, pieces): as many as there can be, in slots that exist.  Whatever an
// entry holds, the join's loop ends and stays inside the scratch.
#ifdef __CUDACC__
__host__ __device__
#endif
inline int entry_pieces(int first_slot, int pieces, long long slots, int grid) {
    const bool sound = pieces >= 1 && pieces <= grid && first_slot >= 0 && (long long)first_slot + pieces <= slots;
    return sound ? pieces : 0;
}

// Token columns of a box of the caches' tensor maps: a page, or a tile of it.
inline int cache_box_rows(int page_size) { return page_size < kKTile ? page_size : kKTile; }

cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t prepare_attend(int dtype, int head_dim);  // once per plan: kernel attributes
cudaError_t launch_attend(const AttendParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map, int dtype,
                          int head_dim, cudaStream_t stream);

#ifdef __CUDACC__
// Element type of an attention plan.
template <bool kBf16>
struct Half;
template <>
struct Half<true> {
    using T = __nv_bfloat16;
    using T2 = __nv_bfloat162;
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const T2 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Half<false> {
    using T = __half;
    using T2 = __half2;
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const T2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const T2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// The group that `row` belongs to; -1 where no group claims it, or several do
// (indptr then does not ascend).  All threads of the block take part and get
// the answer.
__device__ __forceinline__ int block_group_of(const int* indptr, int G, int row) {
    __shared__ int found;
    int n = 0;
    for (int b = 0; b < G; b += blockDim.x) {
        const int i = b + (int)threadIdx.x;
        const int lo = i < G ? indptr[i] : 0, hi = i < G ? indptr[i + 1] : 0;
        const bool claims = lo <= row && row < hi;
        if (claims) found = i;
        n += __syncthreads_count(claims);
    }
    return n == 1 ? found : -1;
}

// The number of entries of indptr[0..G] that are <= row, less one: the group
// of `row` when indptr ascends (the caller checks the answer); and whether it
// ascends.  All threads of the block take part and get the answers.
__device__ __forceinline__ int block_find_group(const int* indptr, int G, int row, bool& ascends) {
    int n = 0;
    bool falls = false;
    for (int b = 0; b <= G; b += blockDim.x) {
        const int i = b + (int)threadIdx.x;
        const int at = indptr[i <= G ? i : G], next = indptr[i < G ? i + 1 : G];
        falls |= next < at;
        n += __syncthreads_count(i <= G && at <= row);
    }
    ascends = __syncthreads_or(falls) == 0;
    return n - 1;
}
#endif

}  // namespace lp
