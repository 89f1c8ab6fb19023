// dcp_paged_api.cu -- the extern "C" entry points of the paged cache (see include/dcp_paged.h for
// the contract of each call): argument validation before any CUDA call, then the launch.
#include "dcp_paged.h"

#include <math.h>

#include <utility>

#include "dcp_paged.cuh"
#include "dcp_testing.h"

namespace {

using dcp_host::fail;
using dcp_host::ok;

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxPositions = kLimit - 1024;  // positions and tile ends are ints in the kernels

int elem_size(int32_t dtype) { return dtype == DCP_FP32 ? 4 : dtype == DCP_BF16 || dtype == DCP_FP16 ? 2 : 0; }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

dcp::FastDiv fast_div(uint64_t d) {
    dcp::FastDiv f;
    const unsigned __int128 one = 1;
    f.magic = d <= 1 ? 0 : (uint64_t)(((one << 64) + d - 1) / d);
    f.d = (uint32_t)d;
    return f;
}

dcp::IntDiv int_div(uint32_t d) {
    dcp::IntDiv f;
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    f.mul = (uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d);
    f.shift = 31 + s;
    f.d = d;
    return f;
}

int64_t attention_workspace(int32_t group, int32_t head_dim, int32_t dtype) {
    switch (dtype) {
        case DCP_BF16: return dcp_host::attention_workspace_bf16(group, head_dim);
        case DCP_FP16: return dcp_host::attention_workspace_fp16(group, head_dim);
        default: return dcp_host::attention_workspace_fp32(group, head_dim);
    }
}

// Whether some of the n[0] x n[1] x n[2] rows of `width` elements with strides s share elements.  Layouts
// in which each dimension steps over all smaller ones, the usual kind, are seen at once; others are
// looked through, differences of two dimensions against steps of the longest one, as far as that is
// 2^18 differences (an overlap past those is not found).
bool rows_overlap(const int64_t (&n)[3], const int64_t (&s)[3], int64_t width) {
    int by_stride[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (s[by_stride[j]] > s[by_stride[j + 1]]) std::swap(by_stride[j], by_stride[j + 1]);
    __int128 span = width;
    bool apart = true;
    for (int i : by_stride) {
        if (n[i] <= 1) continue;
        if (s[i] < width) return true;
        apart = apart && s[i] >= span;
        span += (__int128)(n[i] - 1) * s[i];
    }
    if (apart || width <= 0) return false;
    const int c = n[0] >= n[1] && n[0] >= n[2] ? 0 : n[1] >= n[2] ? 1 : 2, a = (c + 1) % 3, b = (c + 2) % 3;
    const int64_t na = n[a] > 1 ? n[a] : 1, nb = n[b] > 1 ? n[b] : 1;
    int64_t left = int64_t(1) << 18;
    for (int64_t i = 0; i < na; ++i)
        for (int64_t j = 1 - nb; j < nb; ++j) {
            if (--left < 0) return false;
            const __int128 at = (__int128)i * s[a] + (__int128)j * s[b], near = at / s[c];
            for (__int128 k = near - 1; k <= near + 1; ++k) {
                const __int128 d = at - k * s[c];
                if ((i || j || k) && -n[c] < k && k < n[c] && -(__int128)width < d && d < width) return true;
            }
        }
    return false;
}

// `used`: the call reads the block table (it has requests), so its pointers must be there.
// `written`: the call writes the pools, whose rows must then be apart.
int32_t check_cache(const char *fn, const dcp_paged_kv *kv, bool used, bool written, dcp::PagedCache &c) {
    if (!kv) return fail(DCP_ERR_INVALID_ARG, "%s: the cache description is null", fn);
    const int es = elem_size(kv->dtype);
    if (es == 0) return fail(DCP_ERR_UNSUPPORTED_DTYPE, "%s: unsupported dtype %d", fn, (int)kv->dtype);
    if (kv->head_dim < 1 || kv->head_dim > DCP_MAX_PAGED_DIM)
        return fail(DCP_ERR_INVALID_ARG, "%s: head dim %d outside [1, %d]", fn, (int)kv->head_dim, DCP_MAX_PAGED_DIM);
    if ((kv->head_dim * es) % 16 != 0)
        return fail(DCP_ERR_MISALIGNED, "%s: a row of %d elements is not a multiple of 16 bytes", fn,
                    (int)kv->head_dim);
    if (kv->heads < 1 || kv->heads > DCP_MAX_PAGED_HEADS)
        return fail(DCP_ERR_INVALID_ARG, "%s: key head count %d outside [1, %d]", fn, (int)kv->heads, DCP_MAX_PAGED_HEADS);
    if (kv->page_size < 1) return fail(DCP_ERR_INVALID_ARG, "%s: page size %d < 1", fn, (int)kv->page_size);
    if (kv->num_pages < 0 || kv->max_pages < 0) return fail(DCP_ERR_INVALID_ARG, "%s: negative page count", fn);
    if (kv->max_pages >= kLimit || kv->max_pages * kv->page_size >= kMaxPositions)
        return fail(DCP_ERR_INVALID_ARG, "%s: a block table row names 2^31 - 1024 positions or more", fn);
    const int64_t st[7] = {kv->k_stride_page, kv->k_stride_slot, kv->k_stride_head, kv->v_stride_page,
                           kv->v_stride_slot, kv->v_stride_head, kv->table_stride};
    for (int i = 0; i < 7; ++i)
        if (st[i] < 0) return fail(DCP_ERR_INVALID_ARG, "%s: negative stride", fn);
    for (int i = 0; i < 6; ++i)
        if (st[i] % (16 / es)) return fail(DCP_ERR_MISALIGNED, "%s: cache strides must be multiples of 16 bytes", fn);
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16))
        return fail(DCP_ERR_MISALIGNED, "%s: k and v must be 16-byte aligned", fn);
    if (!aligned(kv->block_table, 4)) return fail(DCP_ERR_MISALIGNED, "%s: block_table must be 4-byte aligned", fn);
    if (used && kv->max_pages > 0 && !kv->block_table) return fail(DCP_ERR_INVALID_ARG, "%s: null block_table", fn);
    if (used && kv->num_pages > 0 && (!kv->k || !kv->v)) return fail(DCP_ERR_INVALID_ARG, "%s: null cache pointer", fn);
    for (int i = 0; written && i < 6; i += 3)
        if (rows_overlap({kv->num_pages, kv->page_size, kv->heads}, {st[i], st[i + 1], st[i + 2]}, kv->head_dim))
            return fail(DCP_ERR_INVALID_ARG, "%s: rows of the cache that is written overlap", fn);
    c.k = static_cast<uint32_t *>(kv->k);
    c.v = static_cast<uint32_t *>(kv->v);
    c.table = kv->block_table;
    c.k_page_w = st[0] * es / 4;
    c.k_slot_w = st[1] * es / 4;
    c.k_head_w = st[2] * es / 4;
    c.v_page_w = st[3] * es / 4;
    c.v_slot_w = st[4] * es / 4;
    c.v_head_w = st[5] * es / 4;
    c.table_stride = st[6];
    c.num_pages = kv->num_pages;
    c.capacity = (int32_t)(kv->max_pages * kv->page_size);
    c.heads = kv->heads;
    c.data_w = kv->head_dim * es / 4;
    c.page = int_div((uint32_t)kv->page_size);
    return DCP_OK;
}

int32_t check_shards(const char *fn, int32_t shard, int32_t num_shards, int32_t interleave, dcp::Shards &s) {
    if (num_shards < 1 || num_shards > DCP_MAX_SHARDS)
        return fail(DCP_ERR_INVALID_ARG, "%s: shard count %d outside [1, %d]", fn, (int)num_shards, DCP_MAX_SHARDS);
    if (shard < 0 || shard >= num_shards)
        return fail(DCP_ERR_INVALID_ARG, "%s: shard %d outside [0, %d)", fn, (int)shard, (int)num_shards);
    if (interleave < 1) return fail(DCP_ERR_INVALID_ARG, "%s: interleave %d < 1", fn, (int)interleave);
    const int64_t block = (int64_t)interleave * num_shards, first = (int64_t)interleave * shard;
    s.block = fast_div((uint64_t)(block < kLimit ? block : kLimit));
    s.run = fast_div((uint64_t)interleave);
    s.count = fast_div((uint64_t)num_shards);
    s.first = (uint32_t)(first < kLimit ? first : kLimit);
    s.shard = shard;
    s.one = num_shards == 1;
    return DCP_OK;
}

// The pools' strides in the largest unit (16 to 4096 bytes) that divides them; false where a row's
// offset does not fit 32 bits.  Strides of dimensions of one entry do not matter.
bool unit_strides(const dcp_paged_kv *kv, dcp::AttentionArgs &a) {
    const int es = elem_size(kv->dtype);
    const int64_t counts[3] = {kv->num_pages, kv->page_size, kv->heads};
    const int64_t strides[6] = {kv->k_stride_page, kv->k_stride_slot, kv->k_stride_head,
                                kv->v_stride_page, kv->v_stride_slot, kv->v_stride_head};
    uint32_t *to[6] = {&a.k_page_u, &a.k_slot_u, &a.k_head_u, &a.v_page_u, &a.v_slot_u, &a.v_head_u};
    a.unit = 4096;
    for (int i = 0; i < 6; ++i)
        while (counts[i % 3] > 1 && (strides[i] * es) % a.unit) a.unit >>= 1;
    for (int pool = 0; pool < 2; ++pool) {
        __int128 last = 0;
        for (int i = 3 * pool; i < 3 * pool + 3; ++i) {
            const __int128 u = counts[i % 3] > 1 ? (__int128)strides[i] * es / a.unit : 0;
            last += u * (counts[i % 3] > 1 ? counts[i % 3] - 1 : 0);
            *to[i] = (uint32_t)u;
        }
        if (last >> 32) return false;
    }
    return true;
}

// What both attention calls check and fill; result is `out` either way.
int32_t attention(const char *fn, const dcp_paged_kv *kv, const void *q, const int32_t *seq_lens, void *out,
                  float *lse, float *logits, int64_t B, int64_t H, int32_t world_size, int64_t q_stride_b,
                  int64_t q_stride_h, int64_t logits_stride_b, int64_t logits_stride_h, int64_t logits_cap,
                  float scale, int32_t shard, int32_t num_shards, int32_t interleave, int32_t is_lse_base_on_e,
                  void *workspace, int64_t workspace_bytes, void *cuda_stream,
                  uint64_t wait_limit_ns = dcp::kWaitLimitNs, uint32_t stall_bytes = 0) {
    dcp::AttentionArgs a{};
    int32_t st = check_cache(fn, kv, B != 0, false, a.kv);
    if (st == DCP_OK) st = check_shards(fn, shard, num_shards, interleave, a.sh);
    if (st != DCP_OK) return st;
    const int es = elem_size(kv->dtype);
    if (B < 0) return fail(DCP_ERR_INVALID_ARG, "%s: negative request count %lld", fn, (long long)B);
    if (H < 1) return fail(DCP_ERR_INVALID_ARG, "%s: head count %lld < 1", fn, (long long)H);
    if (H >= kLimit || B >= kLimit || B * H >= kLimit)
        return fail(DCP_ERR_INVALID_ARG, "%s: 2^31 query rows or more", fn);
    if (H % kv->heads)
        return fail(DCP_ERR_SHAPE, "%s: %lld query heads do not split over %d key heads", fn, (long long)H,
                    (int)kv->heads);
    if (world_size) {
        if (world_size < 1 || world_size > DCP_MAX_SHARDS)
            return fail(DCP_ERR_INVALID_ARG, "%s: world size %d outside [1, %d]", fn, (int)world_size,
                        DCP_MAX_SHARDS);
        if (H % world_size)
            return fail(DCP_ERR_SHAPE, "%s: H=%lld is not divisible by world_size=%d", fn, (long long)H,
                        (int)world_size);
    }
    if (q_stride_b < 0 || q_stride_h < 0 || logits_stride_b < 0 || logits_stride_h < 0)
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride", fn);
    if ((q_stride_b * es) % 16 || (q_stride_h * es) % 16)
        return fail(DCP_ERR_MISALIGNED, "%s: query strides must be multiples of 16 bytes", fn);
    if (!isfinite(scale)) return fail(DCP_ERR_INVALID_ARG, "%s: scale is not finite", fn);
    if (logits && (logits_cap < 0 || logits_cap >= kLimit))
        return fail(DCP_ERR_INVALID_ARG, "%s: logits_cap outside [0, 2^31)", fn);
    if (B == 0) return ok();
    if (!unit_strides(kv, a))
        return fail(DCP_ERR_INVALID_ARG, "%s: a pool spans more than 2^32 times %u bytes, the unit of its strides", fn,
                    a.unit);
    if (!q || !seq_lens || !out || (!world_size && !lse))
        return fail(DCP_ERR_INVALID_ARG, "%s: null buffer pointer", fn);
    if (!aligned(q, 16) || !aligned(out, 16))
        return fail(DCP_ERR_MISALIGNED, "%s: the query and the result must be 16-byte aligned", fn);
    if (!aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(logits, 4))
        return fail(DCP_ERR_MISALIGNED, "%s: seq_lens, lse and logits must be 4-byte aligned", fn);
    if (logits && rows_overlap({B, H, 1}, {logits_stride_b, logits_stride_h, 0}, logits_cap))
        return fail(DCP_ERR_INVALID_ARG, "%s: the rows of logits overlap", fn);
    const int64_t need = attention_workspace((int32_t)(H / kv->heads), kv->head_dim, kv->dtype);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(DCP_ERR_INVALID_ARG, "%s: the workspace holds %lld bytes, %lld are needed", fn,
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        if (!aligned(workspace, 16)) return fail(DCP_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    }
    a.q = static_cast<const uint32_t *>(q);
    a.seq_lens = seq_lens;
    a.out = static_cast<uint32_t *>(out);
    a.lse = lse;
    a.logits = logits;
    a.partial = static_cast<float *>(workspace);
    a.q_sb_w = q_stride_b * es / 4;
    a.q_sh_w = q_stride_h * es / 4;
    a.logits_sb = logits_stride_b;
    a.logits_sh = logits_stride_h;
    a.logits_cap = logits ? (int32_t)logits_cap : 0;
    a.B = (int32_t)B;
    a.H = (int32_t)H;
    a.group = (int32_t)(H / kv->heads);
    a.pack_hr = world_size ? (int32_t)(H / world_size) : 0;
    a.pack_div = fast_div(world_size ? (uint64_t)(H / world_size) : 1);
    a.scale = scale;
    a.base_e = is_lse_base_on_e != 0;
    a.stall_bytes = stall_bytes;
    a.wait_limit_ns = wait_limit_ns;
    const cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    switch (kv->dtype) {
        case DCP_BF16: return dcp_host::paged_attention_bf16(a, stream);
        case DCP_FP16: return dcp_host::paged_attention_fp16(a, stream);
        default: return dcp_host::paged_attention_fp32(a, stream);
    }
}

}  // namespace

extern "C" {

int64_t dcp_paged_attention_workspace(int64_t H, int32_t heads, int32_t head_dim, int32_t dtype) {
    if (heads < 1 || H < 1 || H >= kLimit || H % heads || head_dim < 1 || head_dim > DCP_MAX_PAGED_DIM ||
        elem_size(dtype) == 0)
        return -1;
    return attention_workspace((int32_t)(H / heads), head_dim, dtype);
}

int32_t dcp_paged_attention(const dcp_paged_kv *kv, const void *q, const int32_t *seq_lens, void *result, float *lse,
                            float *logits, int64_t B, int64_t H, int64_t q_stride_b, int64_t q_stride_h,
                            int64_t logits_stride_b, int64_t logits_stride_h, int64_t logits_cap, float scale,
                            int32_t shard, int32_t num_shards, int32_t interleave, int32_t is_lse_base_on_e,
                            void *workspace, int64_t workspace_bytes, void *cuda_stream) {
    return attention("dcp_paged_attention", kv, q, seq_lens, result, lse, logits, B, H, 0, q_stride_b, q_stride_h,
                     logits_stride_b, logits_stride_h, logits_cap, scale, shard, num_shards, interleave,
                     is_lse_base_on_e, workspace, workspace_bytes, cuda_stream);
}

int32_t dcp_paged_attention_pack(const dcp_paged_kv *kv, const void *q, const int32_t *seq_lens, void *send_buf,
                                 float *logits, int64_t B, int64_t H, int32_t world_size, int64_t q_stride_b,
                                 int64_t q_stride_h, int64_t logits_stride_b, int64_t logits_stride_h,
                                 int64_t logits_cap, float scale, int32_t shard, int32_t num_shards,
                                 int32_t interleave, int32_t is_lse_base_on_e, void *workspace,
                                 int64_t workspace_bytes, void *cuda_stream) {
    const char *fn = "dcp_paged_attention_pack";
    if (world_size < 1 || world_size > DCP_MAX_SHARDS)
        return fail(DCP_ERR_INVALID_ARG, "%s: world size %d outside [1, %d]", fn, (int)world_size, DCP_MAX_SHARDS);
    return attention(fn, kv, q, seq_lens, send_buf, nullptr, logits, B, H, world_size, q_stride_b, q_stride_h,
                     logits_stride_b, logits_stride_h, logits_cap, scale, shard, num_shards, interleave,
                     is_lse_base_on_e, workspace, workspace_bytes, cuda_stream);
}

int32_t dcp_testing_paged_attention_stalled(const dcp_paged_kv *kv, const void *q, const int32_t *seq_lens,
                                            void *result, float *lse, int64_t B, int64_t H, int64_t q_stride_b,
                                            int64_t q_stride_h, float scale, void *workspace, int64_t workspace_bytes,
                                            void *cuda_stream) {
    return attention("dcp_testing_paged_attention_stalled", kv, q, seq_lens, result, lse, nullptr, B, H, 0, q_stride_b,
                     q_stride_h, 0, 0, 0, scale, 0, 1, 1, 1, workspace, workspace_bytes, cuda_stream,
                     20000000ull, 16u);
}

int32_t dcp_testing_paged_attention_resident(int32_t group, int32_t head_dim, int32_t dtype, int32_t page_size,
                                             int32_t cluster, int32_t *out) {
    if (group < 1 || head_dim < 1 || head_dim > DCP_MAX_PAGED_DIM || page_size < 1 || elem_size(dtype) == 0 || !out)
        return fail(DCP_ERR_INVALID_ARG, "dcp_testing_paged_attention_resident: argument out of range");
    const int box = page_size % 16 == 0 ? 16 : page_size % 8 == 0 ? 8 : 0;
    switch (dtype) {
        case DCP_BF16: return dcp_host::attention_resident_bf16(group, head_dim, box, cluster != 0, out);
        case DCP_FP16: return dcp_host::attention_resident_fp16(group, head_dim, box, cluster != 0, out);
        default: return dcp_host::attention_resident_fp32(group, head_dim, box, cluster != 0, out);
    }
}

int32_t dcp_testing_rows_overlap(int64_t n0, int64_t n1, int64_t n2, int64_t s0, int64_t s1, int64_t s2,
                                 int64_t width) {
    return rows_overlap({n0, n1, n2}, {s0, s1, s2}, width);
}

int32_t dcp_kv_append(const dcp_paged_kv *kv, const void *k_new, const void *v_new, const int32_t *seq_lens,
                      const int32_t *query_start_loc, int64_t T, int32_t num_reqs, int64_t k_stride_t,
                      int64_t k_stride_h, int64_t v_stride_t, int64_t v_stride_h, int32_t shard, int32_t num_shards,
                      int32_t interleave, void *cuda_stream) {
    const char *fn = "dcp_kv_append";
    dcp::AppendArgs a{};
    int32_t st = check_cache(fn, kv, T != 0 && num_reqs != 0, true, a.kv);
    if (st == DCP_OK) st = check_shards(fn, shard, num_shards, interleave, a.sh);
    if (st != DCP_OK) return st;
    const int es = elem_size(kv->dtype);
    if (T < 0 || num_reqs < 0) return fail(DCP_ERR_INVALID_ARG, "%s: negative token or request count", fn);
    if (T >= kLimit || T * kv->heads >= kLimit) return fail(DCP_ERR_INVALID_ARG, "%s: 2^31 new rows or more", fn);
    const int64_t s[4] = {k_stride_t, k_stride_h, v_stride_t, v_stride_h};
    for (int i = 0; i < 4; ++i) {
        if (s[i] < 0) return fail(DCP_ERR_INVALID_ARG, "%s: negative stride", fn);
        if ((s[i] * es) % 16)
            return fail(DCP_ERR_MISALIGNED, "%s: strides of the new rows must be multiples of 16 bytes", fn);
    }
    if (T == 0 || num_reqs == 0) return ok();
    if (!k_new || !v_new || !seq_lens || !query_start_loc)
        return fail(DCP_ERR_INVALID_ARG, "%s: null buffer pointer", fn);
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(DCP_ERR_MISALIGNED, "%s: k_new and v_new must be 16-byte aligned", fn);
    if (!aligned(seq_lens, 4) || !aligned(query_start_loc, 4))
        return fail(DCP_ERR_MISALIGNED, "%s: seq_lens and query_start_loc must be 4-byte aligned", fn);
    a.k_new = static_cast<const uint32_t *>(k_new);
    a.v_new = static_cast<const uint32_t *>(v_new);
    a.seq_lens = seq_lens;
    a.qsl = query_start_loc;
    a.k_st_w = s[0] * es / 4;
    a.k_sh_w = s[1] * es / 4;
    a.v_st_w = s[2] * es / 4;
    a.v_sh_w = s[3] * es / 4;
    a.T = (int32_t)T;
    a.num_reqs = num_reqs;
    return dcp_host::kv_append(a, static_cast<cudaStream_t>(cuda_stream));
}

int32_t dcp_kv_weights(const float *logits, const float *global_lse, const int32_t *seq_lens, float *weights,
                       int64_t B, int64_t H, int64_t heads, int64_t cap, int64_t logits_stride_b,
                       int64_t logits_stride_h, int64_t lse_stride_b, int64_t lse_stride_h, int64_t weights_stride_b,
                       int64_t weights_stride_h, int32_t shard, int32_t num_shards, int32_t interleave,
                       int32_t is_lse_base_on_e, void *cuda_stream) {
    const char *fn = "dcp_kv_weights";
    dcp::WeightsArgs a{};
    const int32_t st = check_shards(fn, shard, num_shards, interleave, a.sh);
    if (st != DCP_OK) return st;
    if (B < 0 || H < 1 || heads < 1) return fail(DCP_ERR_INVALID_ARG, "%s: request or head count out of range", fn);
    if (H >= kLimit || B >= kLimit || B * H >= kLimit)
        return fail(DCP_ERR_INVALID_ARG, "%s: 2^31 query rows or more", fn);
    if (H % heads)
        return fail(DCP_ERR_SHAPE, "%s: %lld query heads do not split over %lld key heads", fn, (long long)H,
                    (long long)heads);
    if (cap < 0 || cap >= kLimit) return fail(DCP_ERR_INVALID_ARG, "%s: cap outside [0, 2^31)", fn);
    if (logits_stride_b < 0 || logits_stride_h < 0 || lse_stride_b < 0 || lse_stride_h < 0 || weights_stride_b < 0 ||
        weights_stride_h < 0)
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (B == 0 || cap == 0) return ok();
    if (!logits || !global_lse || !seq_lens || !weights) return fail(DCP_ERR_INVALID_ARG, "%s: null buffer pointer", fn);
    if (!aligned(logits, 4) || !aligned(global_lse, 4) || !aligned(seq_lens, 4) || !aligned(weights, 4))
        return fail(DCP_ERR_MISALIGNED, "%s: all arrays must be 4-byte aligned", fn);
    if (rows_overlap({B, heads, 1}, {weights_stride_b, weights_stride_h, 0}, cap))
        return fail(DCP_ERR_INVALID_ARG, "%s: the rows of weights overlap", fn);
    a.logits = logits;
    a.lse = global_lse;
    a.seq_lens = seq_lens;
    a.weights = weights;
    a.logits_sb = logits_stride_b;
    a.logits_sh = logits_stride_h;
    a.lse_sb = lse_stride_b;
    a.lse_sh = lse_stride_h;
    a.w_sb = weights_stride_b;
    a.w_sh = weights_stride_h;
    a.B = (int32_t)B;
    a.heads = (int32_t)heads;
    a.group = (int32_t)(H / heads);
    a.cap = (int32_t)cap;
    a.base_e = is_lse_base_on_e != 0;
    return dcp_host::kv_weights(a, static_cast<cudaStream_t>(cuda_stream));
}

int32_t dcp_kv_evict(const dcp_paged_kv *src, const dcp_paged_kv *dst, const int32_t *seq_lens, const float *weights,
                     float *new_weights, int32_t *kept, int32_t *new_lens, int64_t B, int64_t cap, int64_t new_cap,
                     int64_t weights_stride_b, int64_t weights_stride_h, int64_t new_weights_stride_b,
                     int64_t new_weights_stride_h, int64_t keep, int64_t recent, int32_t shard, int32_t num_shards,
                     int32_t interleave, void *cuda_stream) {
    const char *fn = "dcp_kv_evict";
    dcp::EvictArgs a{};
    int32_t st = check_cache(fn, src, B != 0, false, a.src);
    if (st == DCP_OK) st = check_cache(fn, dst, B != 0, true, a.dst);
    if (st == DCP_OK) st = check_shards(fn, shard, num_shards, interleave, a.sh);
    if (st != DCP_OK) return st;
    if (src->heads != dst->heads || src->head_dim != dst->head_dim || src->dtype != dst->dtype)
        return fail(DCP_ERR_INVALID_ARG, "%s: source and destination caches differ in heads, head dim or dtype", fn);
    if (B < 0 || B >= kLimit || B * src->heads >= kLimit)
        return fail(DCP_ERR_INVALID_ARG, "%s: request count out of range", fn);
    if (keep < 1 || keep >= kLimit) return fail(DCP_ERR_INVALID_ARG, "%s: keep outside [1, 2^31)", fn);
    if (recent < 0 || recent > keep) return fail(DCP_ERR_INVALID_ARG, "%s: recent outside [0, keep]", fn);
    if (cap < 0 || cap >= kLimit) return fail(DCP_ERR_INVALID_ARG, "%s: cap outside [0, 2^31)", fn);
    if (new_cap < keep || new_cap >= kLimit) return fail(DCP_ERR_INVALID_ARG, "%s: new_cap outside [keep, 2^31)", fn);
    if (a.dst.capacity < keep)
        return fail(DCP_ERR_INVALID_ARG, "%s: the new block table names %d positions, keep is %lld", fn,
                    (int)a.dst.capacity, (long long)keep);
    if (weights_stride_b < 0 || weights_stride_h < 0 || new_weights_stride_b < 0 || new_weights_stride_h < 0)
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (B == 0) return ok();
    if (!seq_lens || (cap > 0 && !weights) || !new_weights || !kept || !new_lens)
        return fail(DCP_ERR_INVALID_ARG, "%s: null buffer pointer", fn);
    if (!aligned(seq_lens, 4) || !aligned(weights, 4) || !aligned(new_weights, 4) || !aligned(kept, 4) ||
        !aligned(new_lens, 4))
        return fail(DCP_ERR_MISALIGNED, "%s: all arrays must be 4-byte aligned", fn);
    if (rows_overlap({B, dst->heads, 1}, {new_weights_stride_b, new_weights_stride_h, 0}, new_cap))
        return fail(DCP_ERR_INVALID_ARG, "%s: the rows of new_weights overlap", fn);
    a.seq_lens = seq_lens;
    a.weights = weights;
    a.new_weights = new_weights;
    a.kept = kept;
    a.new_lens = new_lens;
    a.w_sb = weights_stride_b;
    a.w_sh = weights_stride_h;
    a.nw_sb = new_weights_stride_b;
    a.nw_sh = new_weights_stride_h;
    a.B = (int32_t)B;
    a.cap = (int32_t)cap;
    a.new_cap = (int32_t)new_cap;
    a.keep = (int32_t)keep;
    a.recent = (int32_t)recent;
    return dcp_host::kv_evict(a, static_cast<cudaStream_t>(cuda_stream));
}

}  // extern "C"
