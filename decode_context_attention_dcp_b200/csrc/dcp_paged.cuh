// dcp_paged.cuh -- what the paged-cache kernels share: the cache as the device sees it, the
// positions a rank holds, and the host-side dispatchers.
//
// Rows are handled as 16-byte chunks and pointers advance in 32-bit words (dcp_kernels.cuh): a
// row of D elements is a whole number of chunks and every stride a multiple of 16 bytes
// (host-checked).  All offsets into a pool are 64-bit: a pool may hold more than 2^31 elements.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dcp_host.h"
#include "dcp_kernels.cuh"
#include "dcp_paged.h"

namespace dcp {

// n / d for 32-bit n and a divisor fixed at launch: magic = ceil(2^64 / d), 0 for d == 1.
struct FastDiv {
    uint64_t magic;
    uint32_t d;
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)div_magic(n, magic); }
};

// n / d for n < 2^31: with 2^(s-1) < d <= 2^s and mul = ceil(2^(31+s) / d), the product exceeds
// 2^(31+s) n / d by less than 2^(31+s) / d, so its quotient is exact; mul < 2^32.
struct IntDiv {
    uint32_t mul, shift, d;
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
};

struct PagedCache {
    uint32_t *k, *v;
    const int32_t *table;
    int64_t k_page_w, k_slot_w, k_head_w;  // strides in words
    int64_t v_page_w, v_slot_w, v_head_w;
    int64_t table_stride;
    int64_t num_pages;
    int32_t capacity;  // max_pages * page_size: positions a table row can name
    int32_t heads;
    int32_t data_w;  // words per row, a multiple of 4
    IntDiv page;     // page_size
};

// The part of each request's positions that this rank holds.
struct Shards {
    FastDiv block;         // min(interleave * num_shards, 2^31): a longer block is one no length fills
    FastDiv run;           // interleave
    FastDiv count;         // num_shards
    uint32_t first;        // min(shard * interleave, 2^31)
    int32_t shard;
    int32_t one;           // num_shards == 1: lengths are local already
};

// Local length of a request of `seq` positions, cut to `cap`.
__device__ __forceinline__ int32_t local_length(const Shards &s, int32_t seq, int32_t cap) {
    if (seq <= 0) return 0;
    if (!s.one) {
        const uint32_t full = s.block.div((uint32_t)seq);
        const uint32_t rest = (uint32_t)seq - full * s.block.d;
        const uint32_t part = rest > s.first ? rest - s.first : 0u;
        seq = (int32_t)(full * s.run.d + (part < s.run.d ? part : s.run.d));
    }
    return seq < cap ? seq : cap;
}

// Slot of local position p (0 <= p < capacity) of a table row: page number and slot in the
// page; false when the page is outside the pool.
__device__ __forceinline__ bool locate(const PagedCache &c, const int32_t *row, uint32_t p, int64_t &page,
                                       uint32_t &slot) {
    const uint32_t j = c.page.div(p);
    slot = p - j * c.page.d;
    page = row[j];
    return page >= 0 && page < c.num_pages;
}

constexpr float kLog2e = 1.44269504088896340736f;

// 2^x, results below 2^-126 as 0 (a weight that small adds nothing to an fp32 sum near 1).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// ---- arguments --------------------------------------------------------------------------------
struct AttentionArgs {
    PagedCache kv;
    // The same strides in units of `unit` bytes (a power of two that divides them all): a row's offset
    // in its pool then fits 32 bits (host-checked), and an address is one multiply-add.
    uint32_t unit;
    uint32_t k_page_u, k_slot_u, k_head_u;
    uint32_t v_page_u, v_slot_u, v_head_u;
    uint32_t stall_bytes;  // added to the bytes that a wait for tensor copies expects: 0, except in the timeout check
    Shards sh;
    const uint32_t *q;
    const int32_t *seq_lens;
    uint32_t *out;   // result rows, or packed rows when pack_hr != 0
    float *lse;      // plain result only
    float *logits;   // or null
    float *partial;  // workspace
    int64_t q_sb_w, q_sh_w;
    int64_t logits_sb, logits_sh;
    int32_t logits_cap;   // 0: no logits
    int32_t B, H, group;  // group = H / kv.heads
    int32_t row_blocks, head_blocks;  // passes per group (set at launch), and over all key heads
    int32_t pack_hr;      // heads per rank of the packed send buffer, 0 = plain result
    FastDiv pack_div;
    float scale;
    int32_t base_e;
    uint64_t wait_limit_ns;  // limit of a wait for tensor copies (kWaitLimitNs)
};

struct AppendArgs {
    PagedCache kv;
    Shards sh;
    const uint32_t *k_new, *v_new;
    const int32_t *seq_lens, *qsl;
    int64_t k_st_w, k_sh_w, v_st_w, v_sh_w;
    int32_t T, num_reqs;
};

struct WeightsArgs {
    Shards sh;
    const float *logits, *lse;
    const int32_t *seq_lens;
    float *weights;
    int64_t logits_sb, logits_sh, lse_sb, lse_sh, w_sb, w_sh;
    int32_t B, heads, group, cap, base_e;
};

struct EvictArgs {
    PagedCache src, dst;
    Shards sh;
    const int32_t *seq_lens;
    const float *weights;
    float *new_weights;
    int32_t *kept, *new_lens;
    int64_t w_sb, w_sh, nw_sb, nw_sh;
    int32_t B, cap, new_cap, keep, recent;
};

}  // namespace dcp

namespace dcp_host {

// Launches of one element type (attention) and of the type-free row movers.
int32_t paged_attention_bf16(const dcp::AttentionArgs &a, cudaStream_t stream);
int32_t paged_attention_fp16(const dcp::AttentionArgs &a, cudaStream_t stream);
int32_t paged_attention_fp32(const dcp::AttentionArgs &a, cudaStream_t stream);
// Bytes of workspace the launches above use on the current device.
int64_t attention_workspace_bf16(int32_t group, int32_t head_dim);
int64_t attention_workspace_fp16(int32_t group, int32_t head_dim);
int64_t attention_workspace_fp32(int32_t group, int32_t head_dim);
// Resident and assumed CTAs per SM (dcp_testing_paged_attention_resident).
int32_t attention_resident_bf16(int32_t group, int32_t head_dim, int box, bool cluster, int32_t *out);
int32_t attention_resident_fp16(int32_t group, int32_t head_dim, int box, bool cluster, int32_t *out);
int32_t attention_resident_fp32(int32_t group, int32_t head_dim, int box, bool cluster, int32_t *out);
int32_t kv_append(const dcp::AppendArgs &a, cudaStream_t stream);
int32_t kv_weights(const dcp::WeightsArgs &a, cudaStream_t stream);
int32_t kv_evict(const dcp::EvictArgs &a, cudaStream_t stream);

}  // namespace dcp_host
