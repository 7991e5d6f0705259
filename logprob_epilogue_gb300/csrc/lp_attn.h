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
                   kStatusBadPage = 0x80u, kStatusBadPrefix = 0x100u, kStatusNoPages = 0x200u;
constexpr int kBlock4 = 16;  // lanes that share a scale in a cache of 4 bits

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
    // append in 4 bits (k_scales != nullptr); k_cache, v_cache: the codes
    unsigned char *k_scales, *v_scales;
    void *k_held, *v_held;                 // [rows, kv_heads, D] or null
    long long k_held_stride, v_held_stride;
    float k_factor, v_factor;              // powers of two
};

// A group as lp_kv_reserve's first part leaves it for the second.
struct Reserved {
    int first;   // entries of the ring before the group's new pages (of those that it gives back, when idle)
    int held;    // pages before the call
    int change;  // new pages; -1 - n: idle, gives n back
    int lens;    // of the round
};

struct ReserveParams {
    const int *lens, *counts, *starts, *held;
    const long long* queue;
    int *free_pages, *tables;
    int *indptr, *round_lens, *held_out;
    long long* queue_out;
    int* positions;
    long long* slots;
    unsigned int* status;
    int rows, G, ring, max_pages, page_shift;
    long long num_pages;
    Reserved* groups;      // [max_groups] scratch
    long long* ends;       // [2] scratch: head and tail of the queue before the call
};

constexpr int kQTile = 128;    // query rows (row, head) of one tensor-core tile
constexpr int kUnitRows = 32;  // of a unit of fragments
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
    int group_rows;                 // rows per tile in a group slot
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
    // a cache of 4 bits; k_cache, v_cache: the codes
    const unsigned char *k_scales, *v_scales;
    float score;           // scale log2(e) k_factor = score 2^score_exp, 1 <= score < 2
    int score_exp;
    float v_factor;
    int wide;              // segments whose units are pairs of tiles: kWidePrefixes, kWideGroups; the others' are fragments
    AttendScratch fragments;  // of those
    int two_cost;             // of those with two fragments: of a token tile, see Fragments
    int rows_per_unit;        // of those: kUnitRows / share (0: only pairs)
};

constexpr int kWidePrefixes = 1, kWideGroups = 2;

// Whether a call over 4 bits has segments of either kind.
#ifdef __CUDACC__
__host__ __device__
#endif
inline bool runs_pairs(const AttendParams& p) { return (p.wide & kWideGroups) != 0 || (p.P > 0 && (p.wide & kWidePrefixes) != 0); }
#ifdef __CUDACC__
__host__ __device__
#endif
inline bool runs_fragments(const AttendParams& p) { return (p.wide & kWideGroups) == 0 || (p.P > 0 && (p.wide & kWidePrefixes) == 0); }

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

cudaError_t launch_reserve(const ReserveParams& p, int grid, cudaStream_t stream);
cudaError_t launch_rope(const RopeParams& p, int dtype, int head_dim, cudaStream_t stream);
cudaError_t prepare_attend(int dtype, int head_dim);  // once per plan: kernel attributes
int pick_wide(const AttendParams& p);  // AttendParams::wide
cudaError_t prepare_attend4_pairs(int dtype, int head_dim);
cudaError_t launch_attend4_pairs(const AttendParams& p, int dtype, int head_dim, const cudaLaunchConfig_t& lc);
cudaError_t prepare_attend4(int dtype, int head_dim);
cudaError_t launch_attend4(const AttendParams& p, int dtype, int head_dim, cudaStream_t stream);
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

// Caches in 4 bits: the four bytes of a word, two codes each, to pairs of F16.
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two scale bytes to a pair of F16.
__device__ __forceinline__ uint32_t widen_scales(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 s, t;\n\tmov.b32 {s, t}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(two));
    return h;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The power of two that brings a row's largest lane, `top`, to [2^14, 2^15) and
// what undoes it (1 for rows of zeros, infinities or NaN).
__device__ __forceinline__ float2 lift_of(float top) {
    const int field = (int)(__float_as_uint(top) >> 23);
    int up = 141 - field;
    up = up > 126 ? 126 : up;
    if (field == 255 || top == 0.0f) up = 0;
    return make_float2(__uint_as_float((uint32_t)(up + 127) << 23), __uint_as_float((uint32_t)(127 - up) << 23));
}

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
