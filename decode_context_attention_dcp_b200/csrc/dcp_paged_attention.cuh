// dcp_paged_attention.cuh -- attention of one new token per request over a paged cache.
//
// x_p = scale (q . k_p), m = max x, result = sum exp(x - m) v / sum exp(x - m), in one pass over
// K and V with the running maximum and sum of the softmax.
#pragma once

#include "dcp_paged.cuh"

namespace dcp {

// One warp per (request, query head): lane i owns words i, i + 32, ... of the row.
template <class T>
__global__ void __launch_bounds__(128) attention_rows_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int kW = 256 / T::kPerWord / 32;  // words per lane of the longest row
    constexpr int E = T::kPerWord;
    const int64_t unit = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (unit >= (int64_t)a.B * a.H) return;
    const int b = (int)(unit / a.H), h = (int)(unit - (int64_t)b * a.H), kvh = h / a.group;
    const int lane = threadIdx.x & 31;
    const int n = local_length(a.sh, a.seq_lens[b], a.kv.capacity);
    float q[kW * E], acc[kW * E];
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        const int w = lane + 32 * i;
#pragma unroll
        for (int e = 0; e < E; ++e) q[i * E + e] = acc[i * E + e] = 0.f;
        if (w < a.kv.data_w) T::decode(a.q[b * a.q_sb_w + h * a.q_sh_w + w], q + i * E);
    }
    float m = -INFINITY, sum = 0.f;
    const int32_t *row = a.kv.table + b * a.kv.table_stride;
    for (int p = 0; p < n; ++p) {
        int64_t page;
        uint32_t slot;
        const bool held = locate(a.kv, row, p, page, slot);
        float x = 0.f;
        if (held) {
            const uint32_t *k = a.kv.k + page * a.kv.k_page_w + slot * a.kv.k_slot_w + kvh * a.kv.k_head_w;
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                const int w = lane + 32 * i;
                if (w < a.kv.data_w) {
                    float f[E];
                    T::decode(k[w], f);
#pragma unroll
                    for (int e = 0; e < E; ++e) x = fmaf(q[i * E + e], f[e], x);
                }
            }
        }
        x = group_sum<32>(x) * a.scale;
        if (!held) x = -INFINITY;
        if (a.logits && lane == 0 && p < a.logits_cap) a.logits[b * a.logits_sb + h * a.logits_sh + p] = x;
        if (x == -INFINITY) continue;
        const float nm = fmaxf(m, x);
        const float c = m == -INFINITY ? 0.f : expf(m - nm), e1 = expf(x - nm);
        m = nm;
        sum = fmaf(sum, c, e1);
        const uint32_t *v = a.kv.v + page * a.kv.v_page_w + slot * a.kv.v_slot_w + kvh * a.kv.v_head_w;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int w = lane + 32 * i;
            if (w < a.kv.data_w) {
                float f[E];
                T::decode(v[w], f);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[i * E + e] = fmaf(e1, f[e], acc[i * E + e] * c);
            }
        }
    }
    float lse = -INFINITY;
    if (m != -INFINITY) lse = a.base_e ? logf(sum) + m : log2f(sum) + m * 1.44269504088896340736f;
    int64_t off = unit * a.kv.data_w;
    if (a.pack_hr) {
        const int r = a.pack_div.div(h);
        off = (((int64_t)r * a.B + b) * a.pack_hr + (h - r * a.pack_hr)) * (a.kv.data_w + 1);
        if (lane == 0) a.out[off + a.kv.data_w] = __float_as_uint(lse);
    } else if (lane == 0) {
        a.lse[unit] = lse;
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        const int w = lane + 32 * i;
        if (w < a.kv.data_w) {
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = m == -INFINITY ? 0.f : acc[i * E + e] / sum;
            a.out[off + w] = T::encode(f);
        }
    }
}

}  // namespace dcp

namespace dcp_host {

template <class T>
int32_t paged_attention(const dcp::AttentionArgs &a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.H;
    dcp::attention_rows_kernel<T><<<(unsigned)((units + 3) / 4), 128, 0, stream>>>(a);
    return launch_status("dcp_paged_attention");
}

}  // namespace dcp_host
