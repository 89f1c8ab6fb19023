// dcp_paged_cache.cu -- the row movers of the paged cache: append, accumulated weights, eviction.
#include "dcp_paged.cuh"

namespace dcp {

// ---- append -----------------------------------------------------------------------------------
// One warp per (token, key head): finds the token's request, its position and slot, and copies
// the key and value row.
__global__ void __launch_bounds__(256) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    const uint32_t unit = blockIdx.x * 8 + threadIdx.x / 32;
    if (unit >= (uint32_t)a.T * (uint32_t)a.kv.heads) return;
    const uint32_t t = unit / (uint32_t)a.kv.heads, h = unit - t * a.kv.heads, lane = threadIdx.x & 31;
    // the last request that starts at or before t
    int lo = 0, hi = a.num_reqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.qsl[mid] <= (int32_t)t) lo = mid + 1; else hi = mid;
    }
    const int r = lo - 1;
    if (r < 0) return;
    const int64_t left = (int64_t)a.qsl[r + 1] - t;
    if (left <= 0) return;
    const int64_t pos = (int64_t)a.seq_lens[r] - left;
    if (pos < 0) return;
    uint32_t p = (uint32_t)pos;
    if (!a.sh.one) {
        const uint32_t run = a.sh.run.div(p), round = a.sh.count.div(run);
        if ((int32_t)(run - round * a.sh.count.d) != a.sh.shard) return;
        p = round * a.sh.run.d + (p - run * a.sh.run.d);
    }
    if (p >= (uint32_t)a.kv.capacity) return;
    int64_t page;
    uint32_t slot;
    if (!locate(a.kv, a.kv.table + r * a.kv.table_stride, p, page, slot)) return;
    const uint32_t *ks = a.k_new + t * a.k_st_w + h * a.k_sh_w, *vs = a.v_new + t * a.v_st_w + h * a.v_sh_w;
    uint32_t *kd = a.kv.k + page * a.kv.k_page_w + slot * a.kv.k_slot_w + h * a.kv.k_head_w;
    uint32_t *vd = a.kv.v + page * a.kv.v_page_w + slot * a.kv.v_slot_w + h * a.kv.v_head_w;
    for (int c = lane * 4; c < a.kv.data_w; c += 128) {
        const Words<4> k = load_stream<4>(ks + c), v = load_stream<4>(vs + c);
        store_words<4>(kd + c, k);
        store_words<4>(vd + c, v);
    }
}

// ---- accumulated weights ----------------------------------------------------------------------
// One CTA per (request, key head), threads along the positions.
__global__ void __launch_bounds__(256) kv_weights_kernel(const __grid_constant__ WeightsArgs a) {
    const int j = blockIdx.x % a.heads, b = blockIdx.x / a.heads;
    const int n = local_length(a.sh, a.seq_lens[b], a.cap);
    for (int p = threadIdx.x; p < n; p += 256) {
        float w = 0.f;
        for (int g = 0; g < a.group; ++g) {
            const int h = j * a.group + g;
            const float l = a.lse[b * a.lse_sb + h * a.lse_sh];
            const float x = a.logits[b * a.logits_sb + h * a.logits_sh + p];
            if (isfinite(l)) w += a.base_e ? expf(x - l) : exp2f(x * 1.44269504088896340736f - l);
        }
        a.weights[b * a.w_sb + j * a.w_sh + p] += w;
    }
}

// ---- eviction ---------------------------------------------------------------------------------
// Weights as unsigned keys of the same order: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One CTA per (request, key head): the threshold key by four passes of 8 bits over the weights,
// then an ordered pass that writes the kept positions and their weights.
__global__ void __launch_bounds__(256) kv_select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_need, scan[9], s_ties[9];
    const int j = blockIdx.x % a.src.heads, b = blockIdx.x / a.src.heads, tid = threadIdx.x;
    const float *w = a.weights + b * a.w_sb + j * a.w_sh;
    float *nw = a.new_weights + b * a.nw_sb + j * a.nw_sh;
    int32_t *kept = a.kept + (int64_t)blockIdx.x * a.keep;
    const int cap = a.src.capacity < a.cap ? a.src.capacity : a.cap;
    const int n = local_length(a.sh, a.seq_lens[b], cap);
    const int m = n < a.keep ? n : a.keep;
    if (j == 0 && tid == 0) a.new_lens[b] = m;
    const int body = n > a.keep ? n - a.recent : 0;  // positions that compete
    uint32_t prefix = 0, need = (uint32_t)(a.keep - a.recent);
    if (body && need) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            hist[tid] = 0;
            __syncthreads();
            for (int p = tid; p < body; p += 256) {
                const uint32_t key = weight_key(w[p]);
                if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(key >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                int d = 255;
                while (d > 0 && hist[d] < need) need -= hist[d--];
                s_prefix = prefix | ((uint32_t)d << shift);
                s_need = need;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
    }
    // keys above `prefix` are kept, and the first `need` equal to it
    uint32_t out = 0, ties = 0;
    for (int p0 = 0; p0 < n; p0 += 256) {
        const int p = p0 + tid;
        const bool in = p < n;
        const float x = in ? w[p] : 0.f;
        const uint32_t key = weight_key(x);
        const bool tie = in && p < body && key == prefix;
        const unsigned tm = __ballot_sync(0xffffffffu, tie);
        if ((tid & 31) == 0) s_ties[tid / 32] = __popc(tm);
        __syncthreads();
        uint32_t before = ties + __popc(tm & ((1u << (tid & 31)) - 1u)), all = 0;
        for (int i = 0; i < 8; ++i) {
            if (i < tid / 32) before += s_ties[i];
            all += s_ties[i];
        }
        const bool keep = in && (p >= body || (a.keep > a.recent && (key > prefix || (tie && before < need))));
        const unsigned km = __ballot_sync(0xffffffffu, keep);
        if ((tid & 31) == 0) scan[tid / 32] = __popc(km);
        __syncthreads();
        uint32_t at = out + __popc(km & ((1u << (tid & 31)) - 1u)), total = 0;
        for (int i = 0; i < 8; ++i) {
            if (i < tid / 32) at += scan[i];
            total += scan[i];
        }
        if (keep) {
            kept[at] = p;
            nw[at] = x;
        }
        ties += all;
        out += total;
        __syncthreads();
    }
    for (int i = m + tid; i < a.keep; i += 256) kept[i] = -1;
    for (int i = m + tid; i < a.new_cap; i += 256) nw[i] = 0.f;
}

// One warp per kept row: its key and value row from the source page to the destination page.
__global__ void __launch_bounds__(256) kv_move_kernel(const __grid_constant__ EvictArgs a) {
    const int b = blockIdx.y / a.src.heads, h = blockIdx.y % a.src.heads, lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + threadIdx.x / 32;
    if (i >= a.keep) return;
    const int32_t p = a.kept[(int64_t)blockIdx.y * a.keep + i];
    if (p < 0) return;
    int64_t sp, dp;
    uint32_t ss, ds;
    if (!locate(a.src, a.src.table + b * a.src.table_stride, p, sp, ss)) return;
    if (!locate(a.dst, a.dst.table + b * a.dst.table_stride, i, dp, ds)) return;
    const uint32_t *ks = a.src.k + sp * a.src.k_page_w + ss * a.src.k_slot_w + h * a.src.k_head_w;
    const uint32_t *vs = a.src.v + sp * a.src.v_page_w + ss * a.src.v_slot_w + h * a.src.v_head_w;
    uint32_t *kd = a.dst.k + dp * a.dst.k_page_w + ds * a.dst.k_slot_w + h * a.dst.k_head_w;
    uint32_t *vd = a.dst.v + dp * a.dst.v_page_w + ds * a.dst.v_slot_w + h * a.dst.v_head_w;
    for (int c = lane * 4; c < a.src.data_w; c += 128) {
        const uint4 k = *reinterpret_cast<const uint4 *>(ks + c), v = *reinterpret_cast<const uint4 *>(vs + c);
        *reinterpret_cast<uint4 *>(kd + c) = k;
        *reinterpret_cast<uint4 *>(vd + c) = v;
    }
}

}  // namespace dcp

namespace dcp_host {

int32_t kv_append(const dcp::AppendArgs &a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.T * a.kv.heads;
    dcp::kv_append_kernel<<<(unsigned)((units + 7) / 8), 256, 0, stream>>>(a);
    return launch_status("dcp_kv_append");
}

int32_t kv_weights(const dcp::WeightsArgs &a, cudaStream_t stream) {
    dcp::kv_weights_kernel<<<(unsigned)(a.B * a.heads), 256, 0, stream>>>(a);
    return launch_status("dcp_kv_weights");
}

int32_t kv_evict(const dcp::EvictArgs &a, cudaStream_t stream) {
    const unsigned rows = (unsigned)a.B * (unsigned)a.src.heads;
    dcp::kv_select_kernel<<<rows, 256, 0, stream>>>(a);
    dcp::kv_move_kernel<<<dim3((unsigned)((a.keep + 7) / 8), rows), 256, 0, stream>>>(a);
    return launch_status("dcp_kv_evict");
}

}  // namespace dcp_host
