// lp_attn.cu -- host side of the attention plan: descriptor and argument
// checks, scratch, and the launches of lp_norm_rope, lp_kv_append and
// lp_attend.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <new>

#include "lp_attn.h"
#include "lp_epilogue.h"
#include "lp_host.h"

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct lp_attn_s {
    lp_attn_desc d;
    int page_shift;
    int grid;
    unsigned char* scratch;
    lp::AttendScratch sc;
    EncodeTiled encode;
};

namespace {

using lp::aligned;
using lp::cuda_fail;
using lp::DeviceGuard;

static_assert(lp::kAttnMaxGroupRows == LP_ATTN_MAX_GROUP_ROWS, "row mask bits");
static_assert(lp::kStatusAttnBadGroup == LP_STATUS_BAD_GROUP && lp::kStatusAttnTimeout == LP_STATUS_TIMEOUT &&
                  lp::kStatusBadPosition == LP_STATUS_BAD_POSITION && lp::kStatusBadPage == LP_STATUS_BAD_PAGE &&
                  lp::kStatusBadPrefix == LP_STATUS_BAD_PREFIX,
              "status bits");

int page_shift_of(int page_size) {
    for (int s = 3; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

int check_desc(const lp_attn_desc* d) {
    if (!d) return LP_EINVAL;
    if (d->dtype != LP_BF16 && d->dtype != LP_F16) return LP_EDTYPE;
    if (d->max_rows < 1 || d->max_groups < 1 || d->max_pages < 1 || d->num_pages < 1) return LP_ESHAPE;
    if (d->kv_heads < 1 || d->q_heads < d->kv_heads || d->q_heads % d->kv_heads != 0) return LP_ESHAPE;
    if (d->head_dim != 64 && d->head_dim != 128) return LP_ESHAPE;
    if (page_shift_of(d->page_size) < 0) return LP_ESHAPE;
    if (d->max_prefixes < 0 || d->max_prefix_pages < 0 || (d->max_prefixes > 0 && d->max_prefix_pages < 1)) return LP_ESHAPE;
    if (d->max_group_rows < 1 || d->max_group_rows > LP_ATTN_MAX_GROUP_ROWS) return LP_ECAPACITY;
    if (d->q_heads / d->kv_heads > 128 || d->q_heads > 4096) return LP_ECAPACITY;
    if (d->max_rows > (1 << 22) || d->max_groups > (1 << 22) || d->max_prefixes > (1 << 16)) return LP_ECAPACITY;
    if (d->num_pages > 0x7FFFFFFF) return LP_ECAPACITY;
    // token indexes are 32-bit (page ids and slots are combined in 64 bits)
    if (((int64_t)d->max_pages + 1) * d->page_size > 0x3FFFFFFF) return LP_ECAPACITY;
    if (((int64_t)d->max_prefix_pages + 1) * d->page_size > 0x3FFFFFFF) return LP_ECAPACITY;
    if ((d->flags & ~(uint32_t)LP_PLAN_DEBUG_FORCE_TIMEOUT) != 0 || d->timeout_ns < 0) return LP_EINVAL;
    return LP_OK;
}

struct Layout {
    size_t seg_units, units, gave_up, part_o, part_ml, total;  // the tables come first
    long long prefix_slots, group_slots;
    int group_rows;
};

// Pieces of a kind: every unit starts one and every block boundary one more.
Layout layout_of(const lp_attn_desc* d, int grid) {
    Layout L{};
    const int share = d->q_heads / d->kv_heads, per_tile = lp::kQTile / share;
    const long long group_units = (long long)d->max_groups * ((d->max_group_rows + 2 * per_tile - 1) / (2 * per_tile));
    const long long prefix_units = d->max_prefixes == 0 ? 0 : d->max_rows / (2 * per_tile) + d->max_prefixes;
    L.group_rows = (d->max_group_rows < per_tile ? d->max_group_rows : per_tile) * share;
    L.group_slots = group_units * d->kv_heads + grid;
    L.prefix_slots = d->max_prefixes == 0 ? 0 : prefix_units * d->kv_heads + grid;
    const size_t segs = (size_t)d->max_prefixes + (size_t)d->max_groups;
    const size_t part_rows = 2 * ((size_t)L.prefix_slots * lp::kQTile + (size_t)L.group_slots * (size_t)L.group_rows);
    size_t off = 0;
    L.seg_units = off;
    off = lp::align_up(off + segs * 8);
    L.units = off;
    off = lp::align_up(off + (size_t)(L.prefix_slots + L.group_slots) * 8);
    L.gave_up = off;
    off = lp::align_up(off + (size_t)grid * 4);
    L.part_ml = off;
    off = lp::align_up(off + part_rows * 8);
    L.part_o = off;
    off = lp::align_up(off + part_rows * (size_t)d->head_dim * 4);
    L.total = off;
    return L;
}

// The 4-D map of a cache: lanes, slots of a page, heads, pages; boxes of 64
// lanes (128 bytes, the swizzle's span) by a page's slots.
bool encode_cache(const lp_attn_s* plan, CUtensorMap* map, const void* cache) {
    const lp_attn_desc& d = plan->d;
    const cuuint64_t row = (cuuint64_t)d.head_dim * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size, (cuuint64_t)d.kv_heads, (cuuint64_t)d.num_pages};
    const cuuint64_t strides[3] = {row, row * d.page_size, row * d.page_size * d.kv_heads};
    const cuuint32_t box[4] = {64, (cuuint32_t)lp::cache_box_rows(d.page_size), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return plan->encode(map, d.dtype == LP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(cache), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A [rows, heads, D] tensor: present, 16-byte aligned, rows a multiple of 16
// bytes apart and not overlapping.
int check_rows(const lp_attn_s* plan, const void* t, int64_t stride, int heads) {
    if (!t) return LP_EINVAL;
    if (!aligned(t, 16) || stride % 8 != 0) return LP_EALIGN;
    if (stride < (int64_t)heads * plan->d.head_dim) return LP_ESHAPE;
    return LP_OK;
}

int check_rope(const lp_attn_s* plan, const lp_rope_io* io, bool append) {
    const lp_attn_desc& d = plan->d;
    if (io->rows < 0 || io->rows > d.max_rows) return LP_ESHAPE;
    if (io->rot_dim < 0 || io->rot_dim > d.head_dim || io->rot_dim % 16 != 0) return LP_ESHAPE;
    if (io->max_positions < 0) return LP_ESHAPE;
    if (!io->status || !(io->eps >= 0.0f) || !std::isfinite(io->eps) || !std::isfinite(io->weight_offset)) return LP_EINVAL;
    if (!aligned(io->status, 4)) return LP_EALIGN;
    if (io->rows == 0) return LP_OK;
    if (!io->positions || (!io->q && !io->k) || (append && !io->k)) return LP_EINVAL;
    if (io->rot_dim > 0 && !io->cos_sin) return LP_EINVAL;
    if (!aligned(io->positions, 4) || !aligned(io->cos_sin, 16)) return LP_EALIGN;
    if (!aligned(io->q_weight, 16) || !aligned(io->k_weight, 16)) return LP_EALIGN;
    int rc;
    if (io->q) {
        if ((rc = check_rows(plan, io->q, io->q_stride, d.q_heads)) != LP_OK) return rc;
        if ((rc = check_rows(plan, io->q_out, io->q_out_stride, d.q_heads)) != LP_OK) return rc;
    }
    if (io->k) {
        if ((rc = check_rows(plan, io->k, io->k_stride, d.kv_heads)) != LP_OK) return rc;
        if (io->k_out || !append)
            if ((rc = check_rows(plan, io->k_out, io->k_out_stride, d.kv_heads)) != LP_OK) return rc;
    }
    return LP_OK;
}

lp::RopeParams rope_params(const lp_attn_s* plan, const lp_rope_io& io) {
    lp::RopeParams p{};
    p.q = io.q;
    p.k = io.k;
    p.q_out = io.q_out;
    p.k_out = io.k_out;
    p.q_stride = io.q_stride;
    p.k_stride = io.k_stride;
    p.q_out_stride = io.q_out_stride;
    p.k_out_stride = io.k_out_stride;
    p.q_weight = io.q_weight;
    p.k_weight = io.k_weight;
    p.cos_sin = io.cos_sin;
    p.positions = io.positions;
    p.status = io.status;
    p.eps = io.eps;
    p.weight_offset = io.weight_offset;
    p.max_pos = io.max_positions;
    p.rot = io.rot_dim;
    p.interleaved = io.interleaved != 0;
    p.rows = io.rows;
    p.q_heads = io.q ? plan->d.q_heads : 0;
    p.kv_heads = io.k ? plan->d.kv_heads : 0;
    return p;
}

}  // namespace

extern "C" {

size_t lp_attn_scratch_bytes(const lp_attn_desc* desc) {
    if (check_desc(desc) != LP_OK) return 0;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, desc->device) != cudaSuccess || sms < 1) {
        (void)cudaGetLastError();
        sms = 152;  // no such device here: a GB300's
    }
    return layout_of(desc, sms).total;
}

int lp_attn_create(lp_attn_t* out, const lp_attn_desc* desc) {
    if (!out) return LP_EINVAL;
    *out = nullptr;
    const int rc = check_desc(desc);
    if (rc != LP_OK) return rc;
    DeviceGuard guard(desc->device);
    if (!guard.ok) return cuda_fail(cudaGetLastError());
    lp_attn_s* plan = new (std::nothrow) lp_attn_s();
    if (!plan) return LP_EINVAL;
    plan->d = *desc;
    plan->page_shift = page_shift_of(desc->page_size);
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    cudaError_t e = cudaDeviceGetAttribute(&plan->grid, cudaDevAttrMultiProcessorCount, desc->device);
    if (e == cudaSuccess) e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e == cudaSuccess && (found != cudaDriverEntryPointSuccess || !fn)) e = cudaErrorNotSupported;
    if (e == cudaSuccess) e = lp::prepare_attend(desc->dtype, desc->head_dim);
    Layout L{};
    if (e == cudaSuccess) {
        plan->encode = reinterpret_cast<EncodeTiled>(fn);
        L = layout_of(desc, plan->grid);
        e = cudaMalloc(&plan->scratch, L.total);
        // a table entry that no call has written names no part
        if (e == cudaSuccess) e = cudaMemset(plan->scratch, 0, L.part_ml);
        if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        cudaFree(plan->scratch);
        delete plan;
        return cuda_fail(e);
    }
    plan->sc.seg_units = reinterpret_cast<int2*>(plan->scratch + L.seg_units);
    plan->sc.units = reinterpret_cast<int2*>(plan->scratch + L.units);
    plan->sc.gave_up = reinterpret_cast<int*>(plan->scratch + L.gave_up);
    plan->sc.part_ml = reinterpret_cast<float2*>(plan->scratch + L.part_ml);
    plan->sc.part_o = reinterpret_cast<float*>(plan->scratch + L.part_o);
    plan->sc.prefix_slots = L.prefix_slots;
    plan->sc.group_slots = L.group_slots;
    plan->sc.group_rows = L.group_rows;
    *out = plan;
    return LP_OK;
}

int lp_attn_destroy(lp_attn_t plan) {
    if (!plan) return LP_EINVAL;
    DeviceGuard guard(plan->d.device);
    const cudaError_t e = cudaFree(plan->scratch);
    delete plan;
    return e == cudaSuccess ? LP_OK : cuda_fail(e);
}

int lp_norm_rope(lp_attn_t plan, const lp_rope_io* io, void* stream) {
    if (!plan || !io) return LP_EINVAL;
    const int rc = check_rope(plan, io, false);
    if (rc != LP_OK) return rc;
    if (io->rows == 0) return LP_OK;
    DeviceGuard guard(plan->d.device);
    if (!guard.ok) return cuda_fail(cudaGetLastError());
    const cudaError_t e = lp::launch_rope(rope_params(plan, *io), plan->d.dtype, plan->d.head_dim,
                                          static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LP_OK : cuda_fail(e);
}

int lp_kv_append(lp_attn_t plan, const lp_append_io* io, void* stream) {
    if (!plan || !io) return LP_EINVAL;
    const lp_attn_desc& d = plan->d;
    int rc = check_rope(plan, &io->rope, true);
    if (rc != LP_OK) return rc;
    if (io->groups < 0 || io->groups > d.max_groups) return LP_ESHAPE;
    if (io->rope.rows == 0) return LP_OK;
    if ((rc = check_rows(plan, io->v, io->v_stride, d.kv_heads)) != LP_OK) return rc;
    if (!io->k_cache || !io->v_cache || !io->group_indptr) return LP_EINVAL;
    if (io->groups > 0 && (!io->lens || !io->block_tables)) return LP_EINVAL;
    if (!aligned(io->k_cache, 16) || !aligned(io->v_cache, 16)) return LP_EALIGN;
    if (!aligned(io->group_indptr, 4) || !aligned(io->lens, 4) || !aligned(io->block_tables, 4)) return LP_EALIGN;
    DeviceGuard guard(d.device);
    if (!guard.ok) return cuda_fail(cudaGetLastError());
    lp::RopeParams p = rope_params(plan, io->rope);
    p.v = io->v;
    p.v_stride = io->v_stride;
    p.indptr = io->group_indptr;
    p.lens = io->lens;
    p.tables = io->block_tables;
    p.k_cache = io->k_cache;
    p.v_cache = io->v_cache;
    p.G = io->groups;
    p.max_pages = d.max_pages;
    p.page_shift = plan->page_shift;
    p.num_pages = d.num_pages;
    const cudaError_t e = lp::launch_rope(p, d.dtype, d.head_dim, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LP_OK : cuda_fail(e);
}

int lp_attend(lp_attn_t plan, const lp_attend_io* io, void* stream) {
    if (!plan || !io) return LP_EINVAL;
    const lp_attn_desc& d = plan->d;
    if (io->rows < 0 || io->rows > d.max_rows || io->groups < 0 || io->groups > d.max_groups) return LP_ESHAPE;
    if (io->prefixes < 0 || io->prefixes > d.max_prefixes) return LP_ESHAPE;
    if (!io->status || !(io->scale > 0.0f) || !std::isfinite(io->scale)) return LP_EINVAL;
    if (!aligned(io->status, 4)) return LP_EALIGN;
    if (io->rows == 0 || io->groups == 0) return LP_OK;
    int rc;
    if ((rc = check_rows(plan, io->q, io->q_stride, d.q_heads)) != LP_OK) return rc;
    if ((rc = check_rows(plan, io->out, io->out_stride, d.q_heads)) != LP_OK) return rc;
    if (!io->k_cache || !io->v_cache || !io->group_indptr || !io->lens || !io->block_tables) return LP_EINVAL;
    if (io->prefixes > 0 && (!io->prefix_indptr || !io->prefix_lens || !io->prefix_tables)) return LP_EINVAL;
    if (!aligned(io->k_cache, 16) || !aligned(io->v_cache, 16)) return LP_EALIGN;
    const void* w4[] = {io->group_indptr, io->lens, io->block_tables, io->row_masks, io->prefix_indptr,
                        io->prefix_lens, io->prefix_tables, io->lse_out};
    for (const void* q : w4)
        if (!aligned(q, 4)) return LP_EALIGN;
    DeviceGuard guard(d.device);
    if (!guard.ok) return cuda_fail(cudaGetLastError());
    lp::AttendParams p{};
    p.q = io->q;
    p.q_stride = io->q_stride;
    p.out_stride = io->out_stride;
    p.k_cache = io->k_cache;
    p.v_cache = io->v_cache;
    p.indptr = io->group_indptr;
    p.lens = io->lens;
    p.tables = io->block_tables;
    p.row_masks = io->row_masks;
    p.prefix_indptr = io->prefix_indptr;
    p.prefix_lens = io->prefix_lens;
    p.prefix_tables = io->prefix_tables;
    p.out = io->out;
    p.lse_out = io->lse_out;
    p.status = io->status;
    p.scale = io->scale;
    p.rows = io->rows;
    p.G = io->groups;
    p.P = io->prefixes;
    p.q_heads = d.q_heads;
    p.kv_heads = d.kv_heads;
    p.share = d.q_heads / d.kv_heads;
    p.max_group_rows = d.max_group_rows;
    p.max_pages = d.max_pages;
    p.max_prefix_pages = d.max_prefix_pages;
    p.page_shift = plan->page_shift;
    p.num_pages = d.num_pages;
    p.rows_per_tile = lp::kQTile / p.share;
    p.share_inv = (65536 + p.share - 1) / p.share;
    p.grid = plan->grid;
    p.sc = plan->sc;
    p.timeout_ns = (unsigned long long)(d.timeout_ns > 0 ? d.timeout_ns : lp::kDefaultTimeoutNs);
    p.force_timeout = (d.flags & LP_PLAN_DEBUG_FORCE_TIMEOUT) != 0;
    CUtensorMap k_map, v_map;
    if (!encode_cache(plan, &k_map, io->k_cache) || !encode_cache(plan, &v_map, io->v_cache))
        return cuda_fail(cudaErrorInvalidValue);
    const cudaError_t e = lp::launch_attend(p, k_map, v_map, d.dtype, d.head_dim, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LP_OK : cuda_fail(e);
}

}  // extern "C"
