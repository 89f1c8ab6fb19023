// dcp_paged_cache.cu -- the row movers of the paged cache: append, accumulated weights, eviction.
//
// None of them computes much: append and the moves of an eviction are copies, the weights one
// exp per logit.  They are bound by HBM where they are long and by the chain of dependent reads
// (request, length, page, row) where they are short, so each kernel first finds the places of a
// block's rows with one thread per row and then copies with every thread, several 16-byte
// loads in flight each.
#include "dcp_paged.cuh"

#include <cooperative_groups.h>

namespace dcp {

namespace cg = cooperative_groups;

constexpr int kCopyThreads = 256;

// Words of a K and a V row, source and destination; k_from < 0: nothing to copy.
struct RowMove {
    int64_t k_from, v_from, k_to, v_to;
};

// 16 bytes that this kernel reads once.
__device__ __forceinline__ uint4 ld_once(const uint32_t *p) {
    const Words<4> r = load_stream<4>(p);
    return make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}

// Copies the rows listed in `moves` (in shared memory): 16-byte chunk c of row r by thread
// (r * chunks + c) mod kCopyThreads, U chunks of K and of V in flight per thread.
template <int U>
__device__ __forceinline__ void copy_rows(const RowMove *moves, int rows, FastDiv chunks, const uint32_t *k_src,
                                          const uint32_t *v_src, uint32_t *k_dst, uint32_t *v_dst) {
    const int items = rows * (int)chunks.d;
    for (int i0 = threadIdx.x; i0 < items; i0 += U * kCopyThreads) {
        uint4 k[U], v[U];
        int at[U];  // row and word; -1: nothing
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kCopyThreads;
            at[u] = -1;
            if (i < items) {
                const int r = (int)chunks.div((uint32_t)i), w = (i - r * (int)chunks.d) * 4;
                const int64_t k_from = moves[r].k_from, v_from = moves[r].v_from;
                if (k_from >= 0) {
                    k[u] = *reinterpret_cast<const uint4 *>(k_src + k_from + w);
                    v[u] = *reinterpret_cast<const uint4 *>(v_src + v_from + w);
                    at[u] = r << 16 | w;  // w < 256
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (at[u] >= 0) {
                const RowMove &mv = moves[at[u] >> 16];
                const int w = at[u] & 0xffff;
                *reinterpret_cast<uint4 *>(k_dst + mv.k_to + w) = k[u];
                *reinterpret_cast<uint4 *>(v_dst + mv.v_to + w) = v[u];
            }
    }
}

// ---- append -----------------------------------------------------------------------------------
constexpr int kAppendTokens = 32;  // tokens a block places at a time, at most

// The last request that starts at or before token t, or -1.  First the one that the token's share of
// all tokens points to (exact for plain decode), else a binary search.  Reads stay inside
// qsl[0 .. num_reqs].
__device__ __forceinline__ int request_of(const AppendArgs &a, int t) {
    int lo = 0, hi = a.num_reqs;  // the number of starts <= t lies in [lo, hi]
    const int g = (int)((int64_t)t * a.num_reqs / a.T);
    const int here = __ldg(a.qsl + g), next = __ldg(a.qsl + g + 1);
    if (here > t) {
        hi = g;
    } else {
        lo = g + 1;
        if (next > t) hi = lo;
    }
    while (lo < hi) {
        const int mid = lo + ((hi - lo) >> 1);
        if (__ldg(a.qsl + mid) <= t) lo = mid + 1; else hi = mid;
    }
    return lo - 1;
}

// 8192 rows of 8 heads x 256 bytes (67 MB moved): 15.0 us, 4.5 TB/s; 256 single tokens: 3.1 us, four
// dependent reads (start, length, page, row).
// A block takes `per` <= 32 tokens at a time: lane i of its first warp finds the place of token i,
// the tokens that this rank holds are put together, and the whole block copies their rows, all
// heads, U chunks of K and of V in flight per thread.
__global__ void __launch_bounds__(kCopyThreads) kv_append_kernel(const __grid_constant__ AppendArgs a, int per,
                                                                 FastDiv chunks, FastDiv heads) {
    constexpr int U = 4;
    __shared__ RowMove moves[kAppendTokens];
    __shared__ int s_tokens;
    const int64_t groups = (int64_t)(a.T - 1) / per + 1;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        if (threadIdx.x < 32) {
            const int64_t t = g * per + threadIdx.x;
            const int r = (int)threadIdx.x < per && t < a.T ? request_of(a, (int)t) : -1;
            RowMove mv{-1, 0, 0, 0};
            if (r >= 0) {
                const int64_t left = (int64_t)__ldg(a.qsl + r + 1) - t, pos = (int64_t)__ldg(a.seq_lens + r) - left;
                bool mine = left > 0 && pos >= 0;
                uint32_t p = (uint32_t)pos;
                if (mine && !a.sh.one) {
                    const uint32_t run = a.sh.run.div(p), round = a.sh.count.div(run);
                    mine = (int32_t)(run - round * a.sh.count.d) == a.sh.shard;
                    p = round * a.sh.run.d + (p - run * a.sh.run.d);
                }
                int64_t page = 0;
                uint32_t slot = 0;
                if (mine && p < (uint32_t)a.kv.capacity &&
                    locate(a.kv, a.kv.table + r * a.kv.table_stride, p, page, slot)) {
                    mv.k_from = t * a.k_st_w;
                    mv.v_from = t * a.v_st_w;
                    mv.k_to = page * a.kv.k_page_w + slot * a.kv.k_slot_w;
                    mv.v_to = page * a.kv.v_page_w + slot * a.kv.v_slot_w;
                }
            }
            const unsigned held = __ballot_sync(0xffffffffu, mv.k_from >= 0);
            if (mv.k_from >= 0) moves[__popc(held & ((1u << threadIdx.x) - 1u))] = mv;
            if (threadIdx.x == 0) s_tokens = __popc(held);
        }
        __syncthreads();
        // item i: chunk c of head h of held token x, chunk fastest
        const int64_t per_token = (int64_t)heads.d * chunks.d, items = s_tokens * per_token;
        for (int64_t i0 = threadIdx.x; i0 < items; i0 += U * kCopyThreads) {
            uint4 k[U], v[U];
            uint32_t *k_to[U], *v_to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * kCopyThreads;
                if (i < items) {
                    const uint32_t row = chunks.div((uint32_t)i), c = (uint32_t)i - row * chunks.d;
                    const uint32_t x = heads.div(row), h = row - x * heads.d;
                    const RowMove mv = moves[x];
                    k[u] = ld_once(a.k_new + mv.k_from + h * a.k_sh_w + c * 4);
                    v[u] = ld_once(a.v_new + mv.v_from + h * a.v_sh_w + c * 4);
                    k_to[u] = a.kv.k + mv.k_to + h * a.kv.k_head_w + c * 4;
                    v_to[u] = a.kv.v + mv.v_to + h * a.kv.v_head_w + c * 4;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * kCopyThreads < items) {
                    *reinterpret_cast<uint4 *>(k_to[u]) = k[u];
                    *reinterpret_cast<uint4 *>(v_to[u]) = v[u];
                }
        }
        __syncthreads();
    }
}

// ---- accumulated weights ----------------------------------------------------------------------
constexpr int kWeighThreads = 128;

// 64 requests of 2048 to 8192 positions, 8 heads per key head (108 MB): 20.1 us, 5.4 TB/s; 128
// threads per block (20.1 us) beat 256 (21.8) and 512 (23.0): less waste at the ragged ends.
// w[p] += sum_h exp(x[h][p] - l[h]): a block takes one row (request, key head) and every
// `splits`-th stretch of 512 of its positions; a thread owns 4 positions (adjacent ones and 16-byte
// accesses where VEC, i.e. all rows start on 16 bytes).
template <bool VEC, int U>
__global__ void __launch_bounds__(kWeighThreads) kv_weights_kernel(const __grid_constant__ WeightsArgs a, int splits) {
    const int row = blockIdx.x / splits, part = blockIdx.x - row * splits;
    const int b = row / a.heads, j = row - b * a.heads;
    const int n = local_length(a.sh, a.seq_lens[b], a.cap);
    const float *x0 = a.logits + b * a.logits_sb + (int64_t)j * a.group * a.logits_sh;
    const float *l0 = a.lse + b * a.lse_sb + (int64_t)j * a.group * a.lse_sh;
    float *w = a.weights + b * a.w_sb + j * a.w_sh;
    for (int64_t p0 = (int64_t)part * (4 * kWeighThreads); p0 < n; p0 += (int64_t)splits * (4 * kWeighThreads)) {
        const int64_t p = p0 + (VEC ? threadIdx.x * 4 : threadIdx.x);
        constexpr int STEP = VEC ? 1 : kWeighThreads;
        if (p >= n) continue;
        const bool whole = p + 3 * STEP < n;
        float old[4], add[4] = {0.f, 0.f, 0.f, 0.f};
        if (VEC && whole) {
            const float4 o = *reinterpret_cast<const float4 *>(w + p);
            old[0] = o.x, old[1] = o.y, old[2] = o.z, old[3] = o.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) old[e] = p + e * STEP < n ? w[p + e * STEP] : 0.f;
        }
        for (int g0 = 0; g0 < a.group; g0 += U) {  // U heads' logits in flight
            float l[U], v[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = min(g0 + u, a.group - 1);  // a head too many is read again and not added
                const float *x = x0 + g * a.logits_sh + p;
                l[u] = __ldg(l0 + g * a.lse_sh);
                if (VEC && whole) {
                    const float4 q = __ldcs(reinterpret_cast<const float4 *>(x));
                    v[u][0] = q.x, v[u][1] = q.y, v[u][2] = q.z, v[u][3] = q.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[u][e] = p + e * STEP < n ? __ldcs(x + e * STEP) : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (g0 + u < a.group && isfinite(l[u])) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        add[e] += exp2_fast(a.base_e ? (v[u][e] - l[u]) * kLog2e : fmaf(v[u][e], kLog2e, -l[u]));
                }
            }
        }
        if (VEC && whole) {
            *reinterpret_cast<float4 *>(w + p) =
                make_float4(old[0] + add[0], old[1] + add[1], old[2] + add[2], old[3] + add[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p + e * STEP < n) w[p + e * STEP] = old[e] + add[e];
        }
    }
}

// ---- eviction ---------------------------------------------------------------------------------
// Weights as unsigned keys of the same order: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The weight of a key; zeros and NaN, whose keys have several weights, are read again.
__device__ __forceinline__ float key_weight(uint32_t key, const float *w) {
    if (key == 0u || key == 0x80000000u) return __ldg(w);
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

constexpr int kBins = 2048;
constexpr int kKeys = 16;  // weights per thread

// Exclusive prefix and total of one value per thread over a block of W warps; `sums` is shared scratch.
template <int W>
__device__ __forceinline__ uint32_t block_prefix(uint32_t mine, uint32_t *sums, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    // every warp adds up the W sums
    const uint32_t own = lane < W ? sums[lane] : 0;
    uint32_t all = own;
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += x;
    }
    total = __shfl_sync(0xffffffffu, all, W - 1);
    return __shfl_sync(0xffffffffu, all - own, warp) + upto - mine;
}

constexpr int kMoveRows = 64;  // kept rows a block moves at a time

// The places of kept position p (-1: none) of request b and key head h, the i-th one kept.
__device__ __forceinline__ RowMove place(const EvictArgs &a, int b, int h, int32_t p, int i) {
    RowMove mv{-1, 0, 0, 0};
    int64_t sp, dp;
    uint32_t ss, ds;
    if (p >= 0 && locate(a.src, a.src.table + b * a.src.table_stride, (uint32_t)p, sp, ss) &&
        locate(a.dst, a.dst.table + b * a.dst.table_stride, (uint32_t)i, dp, ds)) {
        mv.k_from = sp * a.src.k_page_w + ss * a.src.k_slot_w + h * a.src.k_head_w;
        mv.v_from = sp * a.src.v_page_w + ss * a.src.v_slot_w + h * a.src.v_head_w;
        mv.k_to = dp * a.dst.k_page_w + ds * a.dst.k_slot_w + h * a.dst.k_head_w;
        mv.v_to = dp * a.dst.v_page_w + ds * a.dst.v_slot_w + h * a.dst.v_head_w;
    }
    return mv;
}

// How a selection kernel holds a row's weights (as keys):
//   kRegisters  one CTA, kKeys adjacent weights per thread in registers;
//   kShared     one CTA, in shared memory: longer rows without a second reading;
//   kCluster    a cluster of CTAs, in registers; what they cannot hold is read again per pass.
// Measured at 256 rows of 20000 to 32768 weights (27 MB read, as much written): kShared 40 us in two
// waves of 148 CTAs, kCluster (4 CTAs, a barrier and remote histograms per pass) 72 us.  Few rows do not
// turn that round: whole calls with 4096 kept (kCluster with 8 CTAs), 8 rows of 8192 15.9 / 32.6 us, of 32768 25.6 /
// 30.2; 32 rows 33.9 / 78.0 and 44.3 / 73.7; 256 rows of 32768 215 / 530.  So kCluster is left with the rows that
// shared memory cannot hold, by the arrays' width (the host does not see the lengths): 256 rows of
// 32768 in arrays of 131072 take 540 us.  At 24
// rows of up to 2000: 6.9 us with 256 threads, 9.3 us with 1024.  Bound by the chain load,
// three histograms and prefix sums, output (16 us per CTA), not by bytes.
enum KeyStore { kRegisters, kShared, kCluster };

// The kept positions of one (request, key head) row.
//   threshold: the key of the last kept position, by its 11, 11 and 10 highest bits in turn: a
//   shared-memory histogram per pass (summed over the cluster through distributed shared memory)
//   and a prefix sum from the highest bin down;
//   output: keys above it and the first ties are placed by a prefix sum in position order.
// Positions past the end enter as key 0: below or equal to every weight and after it, they are
// never among the kept.
//
// MOVE (short rows): `parts` CTAs per row, each of which selects all of the row for itself and then
// writes and moves its own kMoveRows of the kept ones: one launch, no CTA waits for another.
template <int THREADS, int STORE, bool MOVE>
__global__ void __launch_bounds__(THREADS) kv_select_kernel(const __grid_constant__ EvictArgs a, FastDiv row_chunks,
                                                            int parts) {
    static_assert(!MOVE || (STORE == kRegisters && THREADS == kCopyThreads), "MOVE: short rows, copy_rows' block");
    constexpr bool CLUSTER = STORE == kCluster, SHARED = STORE == kShared;
    constexpr int W = THREADS / 32, BPT = kBins / THREADS;  // bins per thread
    static_assert(BPT % 2 == 0 && (SHARED || THREADS * kKeys < 65536), "pairs of bins; 16-bit counts");
    extern __shared__ uint4 s_keys[];  // kShared: the row's keys, four to a chunk
    __shared__ __align__(16) uint32_t hist[3][kBins];
    __shared__ uint32_t sums[4][W];  // one per prefix sum in turn
    __shared__ uint32_t s_total[1];
    __shared__ uint32_t s_digit, s_need;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ RowMove moves[MOVE ? kMoveRows : 1];
    __shared__ int32_t s_kept[MOVE ? kMoveRows : 1];
    const int ctas = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
    const int tid = threadIdx.x;
    const int sharing = MOVE ? parts : ctas;  // CTAs of this row, and this one's number among them
    const int part = blockIdx.x % sharing, row = blockIdx.x / sharing, b = row / a.src.heads, j = row - b * a.src.heads;
    const float *w = a.weights + b * a.w_sb + j * a.w_sh;
    float *nw = a.new_weights + b * a.nw_sb + j * a.nw_sh;
    int32_t *kept = a.kept + (int64_t)row * a.keep;
    const int cap = a.src.capacity < a.cap ? a.src.capacity : a.cap;
    const int n = local_length(a.sh, a.seq_lens[b], cap);
    const int m = n < a.keep ? n : a.keep;
    if (j == 0 && part == 0 && tid == 0) a.new_lens[b] = m;
    const bool full = n <= a.keep;
    const uint32_t body = full ? 0 : (uint32_t)(n - a.recent);  // positions that compete
    const uint32_t want = full ? 0 : (uint32_t)(a.keep - a.recent);
    // registers: this thread's keys start at `mine`, and every `round` after it
    const uint32_t round = (uint32_t)ctas * THREADS * kKeys;  // below 2^17
    const uint32_t mine = ((uint32_t)rank * THREADS + tid) * kKeys;
    const uint32_t chunks = (body + 127) / 128 * 32;  // shared memory: whole warps of chunks

    auto load = [&](uint32_t p, uint32_t *key) {
        if (p + kKeys <= body && (reinterpret_cast<uintptr_t>(w + p) & 15) == 0) {
            float4 v[kKeys / 4];
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) v[i] = __ldg(reinterpret_cast<const float4 *>(w + p) + i);
#pragma unroll
            for (int i = 0; i < kKeys / 4; ++i) {
                key[4 * i] = weight_key(v[i].x), key[4 * i + 1] = weight_key(v[i].y);
                key[4 * i + 2] = weight_key(v[i].z), key[4 * i + 3] = weight_key(v[i].w);
            }
        } else {
            float v[kKeys];
#pragma unroll
            for (int i = 0; i < kKeys; ++i) v[i] = p + i < body ? __ldg(w + p + i) : 0.f;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) key[i] = p + i < body ? weight_key(v[i]) : 0u;
        }
    };
    uint32_t first[SHARED ? 1 : kKeys];
    if (want) {
        for (int i = tid; i < 3 * kBins / 4; i += THREADS) reinterpret_cast<uint4 *>(&hist[0][0])[i] = make_uint4(0, 0, 0, 0);
        if constexpr (SHARED) {
            const bool vec = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
            constexpr int U = 8;
            for (uint32_t c0 = tid; c0 < chunks; c0 += U * THREADS) {
                float v[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t p = 4 * (c0 + u * THREADS);
                    if (vec && p + 4 <= body) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(w + p));
                        v[u][0] = f.x, v[u][1] = f.y, v[u][2] = f.z, v[u][3] = f.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[u][e] = p + e < body ? __ldg(w + p + e) : 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint32_t c = c0 + u * THREADS;
                    uint32_t k[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) k[e] = 4 * c + e < body ? weight_key(v[u][e]) : 0u;
                    if (c < chunks) s_keys[c] = make_uint4(k[0], k[1], k[2], k[3]);
                }
            }
        } else {
            load(mine, first);
        }
    }
    // kept position p becomes entry `to`, which is one of this CTA's own
    const uint32_t own0 = MOVE ? (uint32_t)part * kMoveRows : 0;
    auto keep = [&](uint32_t to, uint32_t p, float weight) {
        kept[to] = (int32_t)p;
        nw[to] = weight;
        if (MOVE) s_kept[to - own0] = (int32_t)p;
    };
    auto owned = [&](uint32_t to) { return MOVE ? to - own0 < (uint32_t)kMoveRows : true; };
    // the outputs that do not depend on the selection: the last positions, and what is left over
    const int step = sharing * THREADS, id = part * THREADS + tid;
    if constexpr (MOVE) {
        const int64_t i = (int64_t)own0 + tid;
        if (tid < kMoveRows) {
            s_kept[tid] = -1;
            if (i >= want && i < m) keep((uint32_t)i, (uint32_t)(body + i - want), w[body + i - want]);
            if (i >= m && i < a.keep) kept[i] = -1;
        }
    } else {
        for (int64_t p = (int64_t)body + id; p < n; p += step) keep((uint32_t)(want + (p - body)), (uint32_t)p, w[p]);
        for (int64_t i = (int64_t)m + id; i < a.keep; i += step) kept[i] = -1;
    }
    {
        // to the next 16 bytes one by one, then 4 at a time
        const int64_t lead = m + ((4 - ((reinterpret_cast<uintptr_t>(nw + m) >> 2) & 3)) & 3);
        const int64_t at4 = lead < a.new_cap ? lead : a.new_cap, end4 = at4 + (a.new_cap - at4) / 4 * 4;
        for (int64_t i = (int64_t)m + id; i < at4; i += step) nw[i] = 0.f;
        for (int64_t i = at4 + 4 * (int64_t)id; i < end4; i += 4 * (int64_t)step)
            *reinterpret_cast<float4 *>(nw + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int64_t i = end4 + id; i < a.new_cap; i += step) nw[i] = 0.f;
    }
    if (!MOVE && !want) return;  // the same for the whole cluster
    __syncthreads();

    uint32_t prefix = 0, need = want;
    // MOVE: without a selection (want == 0) these passes see no key and are not used
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        if (MOVE && !want) break;
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        auto count = [&](uint32_t key) {
            if (pass == 0 || (key >> (shift + bits)) == prefix >> (shift + bits))
                atomicAdd(&hist[pass][(key >> shift) & ((1u << bits) - 1u)], 1u);
        };
        if constexpr (SHARED) {
#pragma unroll 4
            for (uint32_t c = tid; c < chunks; c += THREADS) {
                const uint4 k = s_keys[c];
                count(k.x), count(k.y), count(k.z), count(k.w);
            }
        } else {
            uint32_t key[kKeys];
            for (uint32_t p0 = mine; p0 < body; p0 += round) {
                if (p0 == mine) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) key[i] = first[i];
                } else {
                    load(p0, key);
                }
#pragma unroll
                for (int i = 0; i < kKeys; ++i) count(key[i]);
            }
        }
        if constexpr (CLUSTER)
            cluster.sync();
        else
            __syncthreads();
        // bins in descending order: thread t holds the BPT bins that end at kBins - 1 - BPT t
        uint32_t c[BPT];
#pragma unroll
        for (int i = 0; i < BPT; ++i) c[i] = 0;
        const int low = kBins - BPT * (tid + 1);
        for (int r = 0; r < ctas; ++r) {
            const uint32_t *other = CLUSTER ? cluster.map_shared_rank(&hist[pass][0], r) : &hist[pass][0];
#pragma unroll
            for (int i = 0; i < BPT; i += 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(other + low + i);
                c[i] += v.x, c[i + 1] += v.y;
            }
        }
        uint32_t sum = 0, total;
#pragma unroll
        for (int i = 0; i < BPT; ++i) sum += c[i];
        uint32_t above = block_prefix<W>(sum, sums[pass], total);
        if (tid == 0 && total < need) s_digit = 0, s_need = need;  // only if the weights changed meanwhile
        if (above < need && need <= above + sum) {
            int d = BPT - 1;
#pragma unroll
            for (int i = BPT - 1; i > 0; --i)
                if (d == i && need > above + c[i]) above += c[i], d = i - 1;
            s_digit = (uint32_t)(low + d);
            s_need = need - above;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        need = s_need;
    }
    // keys above `prefix` are kept, and the first `need` that equal it
    if constexpr (SHARED) {
        // each warp owns a stretch of positions, 128 adjacent ones per step (four per lane): a count, the
        // warps' prefix sums, then the places by ballots
        const int lane = tid & 31, warp = tid >> 5;
        const uint32_t units = chunks / 32, own = (units + W - 1) / W;
        const uint32_t begin = min(warp * own, units), end = min(begin + own, units);
        uint32_t gt = 0, eq = 0, total;
        for (uint32_t i = begin; i < end; ++i) {
            const uint4 k = s_keys[32 * i + lane];
            gt += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
            eq += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
        }
        // below 65536 keys: 16-bit halves do not overflow
        const uint32_t at = block_prefix<W>(gt | eq << 16, sums[3], total);
        const uint32_t start = __shfl_sync(0xffffffffu, at, 0);
        uint32_t above = start & 0xffffu, ties = start >> 16;  // before the step
        const uint32_t lower = (1u << lane) - 1u;
        for (uint32_t i = begin; i < end; ++i) {
            const uint4 k4 = s_keys[32 * i + lane];
            const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
            uint32_t my_above = above, my_ties = ties;
            unsigned any = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const unsigned some = __ballot_sync(0xffffffffu, key[e] > prefix);
                my_above += __popc(some & lower);
                above += __popc(some);
                any |= key[e] == prefix;
            }
            if (__any_sync(0xffffffffu, any)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned some = __ballot_sync(0xffffffffu, key[e] == prefix);
                    my_ties += __popc(some & lower);
                    ties += __popc(some);
                }
            }
            const uint32_t p = 4 * (32 * i + lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool is_gt = key[e] > prefix, is_eq = key[e] == prefix;
                if (is_gt || (is_eq && my_ties < need)) {
                    const uint32_t to = my_above + (my_ties < need ? my_ties : need);
                    if (to < want) keep(to, p + e, key_weight(key[e], w + p + e));  // < want: unless the weights changed
                }
                my_above += is_gt;
                my_ties += is_eq;
            }
        }
    } else {
        uint32_t above0 = 0, ties0 = 0;  // in earlier rounds
        for (uint32_t q = 0; q < (want ? body : 0); q += round) {
            const uint32_t p = q + mine;
            uint32_t gt = 0, eq = 0;  // bit i: key i
            {
                uint32_t key[kKeys];
                if (q == 0) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i) key[i] = first[i];
                } else {
                    load(p, key);
                }
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    gt |= key[i] > prefix ? 1u << i : 0u;
                    eq |= key[i] == prefix ? 1u << i : 0u;
                }
            }
            uint32_t total;
            if (q) __syncthreads();  // the scratch is read by the last round
            const uint32_t at = block_prefix<W>((uint32_t)__popc(gt) | (uint32_t)__popc(eq) << 16, sums[3], total);
            uint32_t above = above0 + (at & 0xffffu), ties = ties0 + (at >> 16);
            above0 += total & 0xffffu;
            ties0 += total >> 16;
            if constexpr (CLUSTER) {
                if (tid == 0) s_total[0] = total;
                cluster.sync();
                for (int r = 0; r < ctas; ++r) {
                    const uint32_t x = *cluster.map_shared_rank(&s_total[0], r);
                    if (r < rank) above += x & 0xffffu, ties += x >> 16;
                    if (r != rank) above0 += x & 0xffffu, ties0 += x >> 16;
                }
                cluster.sync();  // also: no CTA leaves while another reads its shared memory
            }
            for (uint32_t some = gt | eq; some; some &= some - 1) {
                const int i = __ffs(some) - 1;
                const bool is_eq = (eq >> i) & 1u;
                if (!is_eq || ties < need) {
                    const uint32_t to = above + (ties < need ? ties : need);
                    if (to < want && owned(to)) keep(to, p + i, __ldg(w + p + i));  // < want: unless the weights changed
                }
                if (is_eq) ++ties; else ++above;
            }
        }
    }
    if constexpr (MOVE) {
        __syncthreads();
        if (tid < kMoveRows) moves[tid] = place(a, b, j, s_kept[tid], (int)own0 + tid);
        __syncthreads();
        copy_rows<4>(moves, kMoveRows, row_chunks, a.src.k, a.src.v, a.dst.k, a.dst.v);
    }
}

// Kept rows to their new places: rows of 256 bytes from random slots (1.07 GB moved) in 176 us, 6.1 TB/s.
__global__ void __launch_bounds__(kCopyThreads) kv_move_kernel(const __grid_constant__ EvictArgs a, FastDiv chunks,
                                                               int64_t rows, int pieces) {
    __shared__ RowMove moves[kMoveRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t g = blockIdx.x; g < rows * pieces; g += gridDim.x) {
        const int64_t row = g / pieces;
        const int i0 = (int)(g - row * pieces) * kMoveRows;
        const int b = (int)(row / a.src.heads), h = (int)(row - (int64_t)b * a.src.heads);
        const int rn = min(kMoveRows, a.keep - i0);
        if (threadIdx.x < rn) moves[threadIdx.x] = place(a, b, h, a.kept[row * a.keep + i0 + threadIdx.x], i0 + threadIdx.x);
        __syncthreads();
        copy_rows<4>(moves, rn, chunks, a.src.k, a.src.v, a.dst.k, a.dst.v);
        __syncthreads();
    }
}

}  // namespace dcp

namespace dcp_host {

namespace {

dcp::FastDiv divisor(uint32_t d) {
    dcp::FastDiv f;
    const unsigned __int128 one = 1;
    f.magic = d <= 1 ? 0 : (uint64_t)(((one << 64) + d - 1) / d);
    f.d = d;
    return f;
}

template <class T>
T clamp(T v, T lo, T hi) {
    return v < lo ? lo : v > hi ? hi : v;
}

bool vector_rows(const void *p, int64_t s0, int64_t s1) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && s0 % 4 == 0 && s1 % 4 == 0;
}

}  // namespace

int32_t kv_append(const dcp::AppendArgs &a, cudaStream_t stream) {
    // as many tokens per block as leave every SM eight blocks
    const int64_t per = clamp<int64_t>(a.T / (8 * sm_count()), 1, dcp::kAppendTokens);
    const int64_t groups = ((int64_t)a.T - 1) / per + 1;
    const int64_t grid = groups < 16 * sm_count() ? groups : 16 * sm_count();
    dcp::kv_append_kernel<<<(unsigned)grid, dcp::kCopyThreads, 0, stream>>>(a, (int)per, divisor(a.kv.data_w / 4),
                                                                            divisor(a.kv.heads));
    return launch_status("dcp_kv_append");
}

int32_t kv_weights(const dcp::WeightsArgs &a, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.heads;
    // blocks per row: one per 512 positions, as long as that is not more than 16 waves
    const int64_t stretches = ((int64_t)a.cap - 1) / (4 * dcp::kWeighThreads) + 1;
    const int64_t splits = clamp<int64_t>(16 * 8 * sm_count() / rows, 1, stretches);
    const bool vec = vector_rows(a.logits, a.logits_sb, a.logits_sh) && vector_rows(a.weights, a.w_sb, a.w_sh);
    const int64_t grid = rows * splits;  // below 2^31: rows is, and splits is 1 where rows is large
    const bool few = a.group <= 4;
    auto kernel = vec ? few ? dcp::kv_weights_kernel<true, 4> : dcp::kv_weights_kernel<true, 8>
                      : few ? dcp::kv_weights_kernel<false, 4> : dcp::kv_weights_kernel<false, 8>;
    kernel<<<(unsigned)grid, dcp::kWeighThreads, 0, stream>>>(a, (int)splits);
    return launch_status("dcp_kv_weights");
}

template <int THREADS, int STORE, bool MOVE = false>
cudaError_t launch_select(const dcp::EvictArgs &a, int ctas, size_t smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)a.B * a.src.heads * ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)ctas;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = STORE == dcp::kCluster ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, dcp::kv_select_kernel<THREADS, STORE, MOVE>, a, divisor(a.src.data_w / 4), ctas);
}

constexpr int64_t kMaxShared = 49152;  // weights a CTA's shared memory holds (192 KB)

int32_t kv_evict(const dcp::EvictArgs &a, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.src.heads;
    const int64_t longest = a.cap < a.src.capacity ? a.cap : a.src.capacity;  // the longest row there can be
    const int64_t parts = (a.keep - 1) / dcp::kMoveRows + 1;
    cudaError_t e;
    if (longest <= 256 * dcp::kKeys && rows * parts <= 3 * sm_count()) {
        // all of it at once on the device: every CTA selects for itself (24 rows of up to 2000, 512 kept: 9.1 us,
        // selection and moves apart 10.6; 512 CTAs for 128 rows of 4000: 16.1 against 15.0)
        if (launch_select<256, dcp::kRegisters, true>(a, (int)parts, 0, stream) != cudaSuccess)
            return launch_status("dcp_kv_evict");
        return launch_status("dcp_kv_evict");
    }
    if (longest <= 256 * dcp::kKeys) {
        e = launch_select<256, dcp::kRegisters>(a, 1, 0, stream);
    } else if (longest <= kMaxShared) {
        static InstanceCache cache;
        if (!reserve_smem(dcp::kv_select_kernel<1024, dcp::kShared, false>, cache, kMaxShared * 4))
            return fail(DCP_ERR_CUDA, "dcp_kv_evict: cannot reserve shared memory");
        e = launch_select<1024, dcp::kShared>(a, 1, (size_t)((longest + 127) / 128 * 512), stream);
    } else {
        // as many CTAs (at most 8) as hold the row in registers, as far as the grid's size allows
        int ctas = rows * 8 < (int64_t(1) << 31) ? 8 : 1;
        e = launch_select<512, dcp::kCluster>(a, ctas, 0, stream);
    }
    if (e != cudaSuccess) return launch_status("dcp_kv_evict");
    const int pieces = (a.keep - 1) / dcp::kMoveRows + 1;
    const int64_t blocks = rows * pieces;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(blocks < 32 * sm_count() ? blocks : 32 * sm_count()));
    cfg.blockDim = dim3(dcp::kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dcp::kv_move_kernel, a, divisor(a.src.data_w / 4), rows, pieces) != cudaSuccess)
        return launch_status("dcp_kv_evict");
    return launch_status("dcp_kv_evict");
}

}  // namespace dcp_host
