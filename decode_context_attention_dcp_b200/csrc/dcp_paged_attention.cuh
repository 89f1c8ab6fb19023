// dcp_paged_attention.cuh -- attention of one new token per request over a paged cache.
//
// x_p = scale (q . k_p), m = max x, result = sum exp(x - m) v / sum exp(x - m), in one pass over
// K and V with the running maximum and sum of the softmax.
//
// What bounds it.  A position costs 2 D elements of K and V per key head and 4 G D flops for the G
// query heads that share it: G flops per byte (16-bit), far below the machine's balance for groups of up to
// 16 heads, so the kernel is a stream over the held pages and everything else is
// arranged to keep that stream full.  The products run on mma.sync (m16n8k16, fp32 sums) with
// positions (x = K q^T) and then columns (o^T = V^T p^T) as the 16 rows and query heads as the 8 columns, so
// that a group of up to 8 heads costs one product per 16 x 16 block of K or V.  Operands come
// straight from the streamed tile.  tcgen05 would want 128 rows per product and an operand round
// trip through tensor memory, for a pipe that is idle most of the time either way (14% busy with 8 heads, 27% with
// 16).  Wider groups are not covered by that: above 32 heads K and V are streamed once per block of heads
// (8 requests of 131072, one key head, D = 128, bf16, 82 us of bytes: 8 heads 94 us, 16 102, 32 112, 64 203, 128 385).
//
// Measured (device time; share of the 6548 GB/s copy rate of the bytes that have to move): 128 requests of 2048 to
// 8192 positions, 128 heads on 8, D = 128, bf16: 422 us, 96% (437 us, 92%, after seconds of it under the power
// cap); 64 of 0 to 8192, 64 heads on 8: 179 us, 93%; 3 of 100000 to 131072, 64 heads on 4, fp16: 128 us, 87%; one of
// 777, 32 heads on 8: 5.9 us.  SMs get bandwidth that differs by up to 15%, so the first CTAs of a
// wave end that much before the last; cutting the end of the work into smaller shares gained 2% on the
// second case and cost 11% on the third.
//
// Work split.  The tiles (TILE positions of one request, key head and block of query heads) of the
// whole batch are numbered in a row and divided evenly over the CTAs of one resident wave, whatever
// the lengths: a CTA's share may begin and end inside a request.  Each CTA finds its share from
// the lengths on the device.  A request that lies in one share is finished there; the others leave
// one fp32 partial (unnormalised row, maximum, sum) per share in the workspace, and
// attention_join_kernel merges them in share order (no atomics: the same bits every time).
//
// Short calls (few requests, tables of a few tiles) instead give each request, key head and block of
// heads a cluster of CTAs, which merge through distributed shared memory: one launch, no workspace.
//
// Inside a CTA each warp streams its own positions (warp w of NW takes every NW-th group of
// 16) through its own ring of shared-memory stages, and keeps its own softmax state; warps meet
// only where a request begins (the query) and ends (the merge).  A stage is filled by tensor
// copies (a box of 8 or 16 slots of one page, 128 bytes of each row) where the page size is a
// multiple of 8, else row by row with cp.async.
#pragma once

#include <cooperative_groups.h>

#include "dcp_paged.cuh"

namespace dcp {

// ---- instructions -----------------------------------------------------------------------------
__device__ __forceinline__ void ldmatrix4(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// The transpose of an 8 x 8 block of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void mma(Bf16, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma(Fp16, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma(Fp32, float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}

// 16 bytes global -> shared, or 16 zero bytes (nothing read).
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16u : 0u));
}

// A box of a 4-dimensional tensor map into shared memory, completing on `bar`.
__device__ __forceinline__ void tensor_copy(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
        : "memory");
}

// A float as two tf32 values: hi is x rounded to 10 fraction bits (half a step away from zero), lo
// the rest (at most 2^-11 |x|), of which the product keeps 10 fraction bits: hi + lo = x to
// 2^-21 |x|.
__device__ __forceinline__ void tf32_split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// ---- shapes -----------------------------------------------------------------------------------
// T element type, DP head dim as laid out in shared memory (D <= DP, the rest zero), NH blocks of 8
// query heads per pass over K and V, NW warps per CTA, ST stages per warp, CTAS resident CTAs per SM.
template <class T_, int DP_, int NH_, int NW_, int ST_, int CTAS_, int BOX_ = 0>
struct AttentionShape {
    using T = T_;
    // slots per tensor copy (16 or 8, which the page size is a multiple of), 0: cp.async
    static constexpr int BOX = BOX_;
    template <int BOX2>
    using With = AttentionShape<T_, DP_, NH_, NW_, ST_, CTAS_, BOX2>;
    static constexpr int DP = DP_, NH = NH_, NW = NW_, ST = ST_, CTAS = CTAS_;
    static constexpr bool kHalfType = T::kPerWord == 2;
    static constexpr int kBytes = 4 / T::kPerWord;     // element size
    static constexpr int WP = 16;                      // positions per warp and stage
    static constexpr int TILE = WP * NW;               // positions per CTA tile
    static constexpr int kHeads = 8 * NH;              // query heads per pass
    static constexpr int kChunks = DP * kBytes / 16;   // 16-byte chunks per row
    // K and V of a stage lie in panels of 16 rows x 128 bytes, chunk c of row r of a panel at c ^ (r mod 8)
    // (the tensor copies' 128-byte swizzle): the 8 rows of an ldmatrix, or of a fragment's float
    // reads, fall into different banks
    static constexpr int kPanels = DP * kBytes / 128;
    static constexpr int kPanel = WP * 128;
    static constexpr int kHalf = WP * DP * kBytes;     // bytes of a stage's K (and of its V)
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kThreads = NW * 32;
    // the query: a ring of buffers that cp.async fills ahead; fp32: one, as (hi, lo) pairs
    static constexpr int kQuery = kHeads * DP * kBytes;
    static constexpr int kQueries = kHalfType ? ST * kQuery : 2 * kQuery;
    static constexpr bool kQueryRegs = NH * DP * kBytes * kBytes <= 1024;  // at most 32 registers
    static constexpr size_t kSmem = (size_t)NW * ST * kStage + kQueries;
    // Static shared memory, in units of the dynamic part's alignment: the warps' scratch, held bits, barriers
    // (tensor copies), and the scan and place (even shares) or the heads' sums (clusters).  CTAS blocks fit an
    // SM's 228 KB, of which each block takes 1 KB for the system.
    static constexpr int kScratch = 8 * (WP > kHeads ? WP : kHeads);  // per warp
    static constexpr int kEnds = 8 * NW + 16 > 8 * kHeads ? 8 * NW + 16 : 8 * kHeads;
    static constexpr int kStatic = NW * kScratch + 4 * ST * NW + (BOX ? 8 * NW * ST : 0) + kEnds;
    static_assert((kSmem + (kStatic + 1023) / 1024 * 1024 + 1024) * CTAS <= 228 * 1024, "CTAS blocks per SM");
    static_assert(ST > 1 || !kHalfType, "16-bit types copy the query with the first tile, ahead of the loop");
    static_assert(kStage >= 16 * DP * 4, "a stage holds 16 fp32 rows (the merge)");
};

// How far a logit (base 2) may exceed the running maximum before the sums are rescaled.
constexpr float kSlack = 7.f;

// Weights are carried as 2^(x - m + shift): the two fp16 parts of a weight then keep their 11 + 11
// bits down to weights of 2^-22, where those below 2^-14 would otherwise be subnormal.  The
// largest, 2^(8 + kSlack), stays below the fp16 maximum.  The factor cancels in the division by the
// sum.
template <class T>
struct WeightShift {
    static constexpr float value = 0.f;
};
template <>
struct WeightShift<Fp16> {
    static constexpr float value = 8.f;
};

constexpr float kLn2 = 0.69314718055994530942f;

// ---- workspace --------------------------------------------------------------------------------
// Two partials per CTA (the request it entered in the middle, the one it left unfinished): ROWS query
// heads' rows of DP floats each, then (maximum, sum) per row, then one int4 per CTA: the number of
// parts of the request that starts in this CTA and is finished by later ones (0: none), its
// request, key head and head block.
struct Workspace {
    float *rows;
    float2 *stats;
    int4 *spill;
};

template <int ROWS, int DP>
__host__ __device__ __forceinline__ int64_t workspace_bytes(int64_t ctas) {
    return ctas * (2 * ROWS * (DP * 4 + 8) + 16);
}

template <int ROWS, int DP>
__device__ __forceinline__ Workspace workspace_at(float *base, int64_t ctas) {
    Workspace w;
    w.rows = base;
    w.stats = reinterpret_cast<float2 *>(base + 2 * ctas * ROWS * DP);
    w.spill = reinterpret_cast<int4 *>(w.stats + 2 * ctas * ROWS);
    return w;
}

// ---- a CTA's share ------------------------------------------------------------------------------
// `tiles` tiles over `ctas` CTAs: share c has tiles / ctas, the first tiles % ctas one more.
struct Shares {
    int64_t each, extra;
    __device__ __forceinline__ Shares(int64_t tiles, int64_t ctas) {
        if (tiles < (int64_t(1) << 32)) {  // the usual case without 64-bit division
            each = (uint32_t)tiles / (uint32_t)ctas;
            extra = tiles - each * ctas;
        } else {
            each = tiles / ctas;
            extra = tiles - each * ctas;
        }
    }
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * each + (c < extra ? c : extra); }
    // the share that holds tile x (each >= 1)
    __device__ __forceinline__ int64_t of(int64_t x) const {
        const int64_t big = extra * (each + 1);
        return x < big ? x / (each + 1) : extra + (x - big) / each;
    }
};

// Position in the sequence of tiles: tile t of nt of request b, key head kvh and head block rb; n
// is the request's local length.  The next request's length is read one request ahead.
struct TileIter {
    int b, kvh, rb, t, n, nt, next_seq;
};

__device__ __forceinline__ int tiles_of(int n, int tile) { return n > tile ? (n - 1) / tile + 1 : 1; }

template <int TILE>
__device__ __forceinline__ void iter_request(const AttentionArgs &a, TileIter &it) {
    it.n = local_length(a.sh, it.next_seq, a.kv.capacity);
    it.nt = tiles_of(it.n, TILE);
    it.next_seq = it.b + 1 < a.B ? a.seq_lens[it.b + 1] : 0;
}

template <int TILE>
__device__ __forceinline__ void iter_next(const AttentionArgs &a, TileIter &it) {
    if (++it.t < it.nt) return;
    it.t = 0;
    if (++it.rb < a.row_blocks) return;
    it.rb = 0;
    if (++it.kvh < a.kv.heads) return;
    it.kvh = 0;
    ++it.b;
    iter_request<TILE>(a, it);
}

// ---- results ------------------------------------------------------------------------------------
// Word offset of the result row of (b, h).
__device__ __forceinline__ int64_t result_row(const AttentionArgs &a, int b, int h) {
    if (!a.pack_hr) return ((int64_t)b * a.H + h) * a.kv.data_w;
    const int rank = (int)a.pack_div.div((uint32_t)h);
    return (((int64_t)rank * a.B + b) * a.pack_hr + (h - rank * a.pack_hr)) * (a.kv.data_w + 1);
}

// Four columns of the result row of (b, h), and with column 0 its LSE; sum == 0 is an empty row.
template <class T>
__device__ __forceinline__ void write_result(const AttentionArgs &a, int b, int h, int col, const float4 &o, float m,
                                             float sum) {
    const bool empty = sum == 0.f;
    const float r = empty ? 0.f : 1.f / sum;
    const float f[4] = {empty ? 0.f : o.x * r, empty ? 0.f : o.y * r, empty ? 0.f : o.z * r, empty ? 0.f : o.w * r};
    const int64_t off = result_row(a, b, h);
    const int w = col / T::kPerWord;
    if (w < a.kv.data_w) {  // a row is a whole number of 16-byte chunks: four columns are in or out together
        uint32_t *p = a.out + off + w;
        if constexpr (T::kPerWord == 2) {
            const uint32_t w0 = T::encode(f), w1 = T::encode(f + 2);
            if (a.pack_hr) {  // packed rows are 4-byte aligned
                p[0] = w0;
                p[1] = w1;
            } else {
                *reinterpret_cast<uint2 *>(p) = make_uint2(w0, w1);
            }
        } else {
            if (a.pack_hr) {
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = __float_as_uint(f[i]);
            } else {
                *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
    }
    if (col == 0) {
        // sum holds the factor 2^kShift
        const float l2 = empty ? -INFINITY : log2f(sum) + (m - WeightShift<T>::value);
        const float lse = a.base_e ? l2 * kLn2 : l2;
        if (a.pack_hr)
            a.out[off + a.kv.data_w] = __float_as_uint(lse);
        else
            a.lse[(int64_t)b * a.H + h] = lse;
    }
}

// Whether a row's sums call for mend_columns: some are not finite although its weights are (m and sum: their
// maximum and sum; a row without weights is written as an empty one).
__device__ __forceinline__ bool needs_mending(const float4 &o, float m, float sum) {
    const float zero = fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f)));
    return zero != 0.f && isfinite(m) && isfinite(sum) && sum > 0.f;
}

// What non-finite values make of four columns of the result row of (b, h), which write_result has
// written: the sum of their products with the weights 2^(x - m) as IEEE forms it (inf, -inf or NaN).  The
// stream's products cannot say: a weight enters them as two parts, of which the second may be 0 or
// negative (0 inf and inf - inf are NaN where the formula gives inf).  Columns whose values are all finite
// stay as they are.  One thread reads the values of its columns again, four positions at a time until all
// four columns are NaN, and a key row for each value that is not finite (its weight may be 0, which
// makes NaN of an infinity): a path that finite caches never take.  4 requests of 8192 positions, 32 heads
// on 8, D = 128, bf16, every value an infinity: 13 ms; every value NaN: 42 us (finite ones: 29 us).
template <class T>
__device__ __noinline__ void mend_columns(const AttentionArgs &a, int b, int h, int col, float m) {
    constexpr int PW = T::kPerWord, U = 4;
    if (col / PW >= a.kv.data_w) return;
    const int n = local_length(a.sh, a.seq_lens[b], a.kv.capacity), j = h / a.group;
    const int32_t *table = a.kv.table + b * a.kv.table_stride;
    const uint32_t *q = a.q + b * a.q_sb_w + h * a.q_sh_w;
    const uint32_t *values = a.kv.v + j * a.kv.v_head_w + col / PW, *keys = a.kv.k + j * a.kv.k_head_w;
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    for (int p0 = 0; p0 < n && !(isnan(r[0]) && isnan(r[1]) && isnan(r[2]) && isnan(r[3])); p0 += U) {
        float v[U][4];
        int64_t key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.f;
            key[u] = 0;
            int64_t page;
            uint32_t slot;
            if (p0 + u < n && locate(a.kv, table, (uint32_t)(p0 + u), page, slot)) {
                const uint32_t *at = values + page * a.kv.v_page_w + slot * a.kv.v_slot_w;
#pragma unroll
                for (int i = 0; i < 4 / PW; ++i) T::decode(__ldg(at + i), &v[u][PW * i]);
                key[u] = page * a.kv.k_page_w + slot * a.kv.k_slot_w;
            }
        }
        bool counts[U], some = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            counts[u] = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) counts[u] = counts[u] || !(isfinite(v[u][e]) || isnan(r[e]));
            some = some || counts[u];
        }
        if (!some) continue;
        float x[U] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int i = 0; i < a.kv.data_w; i += 4) {
            const uint4 qw = __ldg(reinterpret_cast<const uint4 *>(q + i));
            const uint32_t q4[4] = {qw.x, qw.y, qw.z, qw.w};
            uint4 kw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                kw[u] = counts[u] ? __ldg(reinterpret_cast<const uint4 *>(keys + key[u] + i)) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k4[4] = {kw[u].x, kw[u].y, kw[u].z, kw[u].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float qf[2], kf[2];
                    T::decode(q4[c], qf);
                    T::decode(k4[c], kf);
#pragma unroll
                    for (int e = 0; e < PW; ++e) x[u] = fmaf(qf[e], kf[e], x[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = exp2_fast(x[u] * (a.scale * kLog2e) - m);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!isfinite(v[u][e])) r[e] += w * v[u][e];  // never 0
        }
    }
    uint32_t *to = a.out + result_row(a, b, h) + col / PW;
#pragma unroll
    for (int i = 0; i < 4 / PW; ++i) {
        float f[2];
        T::decode(to[i], f);
#pragma unroll
        for (int e = 0; e < PW; ++e)
            if (r[PW * i + e] != 0.f) f[e] = r[PW * i + e];
        to[i] = T::encode(f);
    }
}

__device__ __forceinline__ float finite_or_zero_max(float m) { return m == -INFINITY ? 0.f : m; }

// mend_columns for the requests that a CTA's share of `count` tiles holds whole; it begins at tile
// where[2] of request where[0] and key head and head block where[1].
template <class T, int TILE, int HEADS>
__device__ __noinline__ void mend_share(const AttentionArgs &a, const int *where, int64_t count) {
    TileIter it;
    it.b = where[0];
    it.kvh = where[1] / a.row_blocks;
    it.rb = where[1] - it.kvh * a.row_blocks;
    it.t = where[2];
    it.next_seq = a.seq_lens[it.b];
    iter_request<TILE>(a, it);
    while (count > 0) {
        const int left = it.nt - it.t, head0 = it.rb * HEADS, chunks = a.kv.data_w * T::kPerWord / 4;
        const int rows = it.t == 0 && count >= left ? min(HEADS, a.group - head0) : 0;
        for (int x = threadIdx.x; x < rows * chunks; x += blockDim.x) {
            const int r = x / chunks, c = x - r * chunks, h = it.kvh * a.group + head0 + r;
            const int64_t row = result_row(a, it.b, h);
            float f[4];
#pragma unroll
            for (int i = 0; i < 4 / T::kPerWord; ++i) T::decode(a.out[row + c * 4 / T::kPerWord + i], f + T::kPerWord * i);
            const float lse = a.pack_hr ? __uint_as_float(a.out[row + a.kv.data_w]) : a.lse[(int64_t)it.b * a.H + h];
            // 2^(x - lse) are the weights divided by their sum
            if (needs_mending(make_float4(f[0], f[1], f[2], f[3]), lse, 1.f))
                mend_columns<T>(a, it.b, h, c * 4, a.base_e ? lse * kLog2e : lse);
        }
        count -= left;
        it.t = it.nt - 1;
        iter_next<TILE>(a, it);
    }
}

// ---- the stream ---------------------------------------------------------------------------------
// Tensor maps of the pools: [pages, slots, heads, D].
struct PoolMaps {
    CUtensorMap k, v;
};

template <class S, bool CLUSTER>
__global__ void __launch_bounds__(S::kThreads, S::CTAS)
    attention_stream_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ PoolMaps maps) {
    using T = typename S::T;
    constexpr int DP = S::DP, NH = S::NH, NW = S::NW, ST = S::ST, WP = S::WP, TILE = S::TILE;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[NW];
    __shared__ int s_where[3];
    __shared__ int s_mend;                         // a finished request needs mend_columns
    // Each warp's: at a merge the maximum and sum of its heads; with cp.async, between merges, the offsets of the
    // K and V rows that it is copying.
    __shared__ __align__(8) uint8_t s_scratch[NW][S::kScratch];
    auto s_stat = [&](int w) { return reinterpret_cast<float2 *>(s_scratch[w]); };
    auto s_row = [&](int w) { return reinterpret_cast<uint2 *>(s_scratch[w]); };
    __shared__ uint32_t s_held[ST][NW];            // bit r: position r of the warp's stage counts
    __shared__ uint64_t s_full[NW][ST];            // tensor copies: a stage's bytes have arrived
    __shared__ float2 s_part[S::kHeads];           // cluster: maximum and sum of this CTA's heads
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if constexpr (!CLUSTER) {
        // the join may be launched; a cluster's results are final, what follows it has to wait for its end
        asm volatile("griddepcontrol.launch_dependents;");
        if (tid == 0) s_mend = 0;
    }
    constexpr bool TENSOR = S::BOX > 0;
    if (TENSOR && lane == 0) {
        for (int st = 0; st < ST; ++st) mbar_init(&s_full[warp][st], 1);
        mbar_fence_init();
    }

    int64_t begin, count;
    Shares shares(0, 1);
    TileIter ld;
    if constexpr (CLUSTER) {
        // one request, key head and head block per cluster, its tiles in even parts
        const int seg = blockIdx.x / cluster.num_blocks(), hb = seg % a.head_blocks;
        ld.b = seg / a.head_blocks;
        ld.kvh = hb / a.row_blocks;
        ld.rb = hb - ld.kvh * a.row_blocks;
        ld.n = local_length(a.sh, a.seq_lens[ld.b], a.kv.capacity);
        ld.nt = tiles_of(ld.n, TILE);
        ld.next_seq = 0;
        shares = Shares(ld.nt, cluster.num_blocks());
        begin = shares.begin(cluster.block_rank());
        count = shares.begin(cluster.block_rank() + 1) - begin;
        ld.t = (int)begin;
        __syncwarp();  // the warp's barriers are initialised
    } else {
        // the share: all lengths summed in one block scan, then the request where it begins
        const int per = (a.B - 1) / S::kThreads + 1;
        const int b0 = (int)min((int64_t)tid * per, (int64_t)a.B), b1 = (int)min((int64_t)b0 + per, (int64_t)a.B);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += tiles_of(local_length(a.sh, a.seq_lens[b], a.kv.capacity), TILE);
        mine *= a.head_blocks;
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) upto += s_scan[w];
            total += s_scan[w];
        }
        const int64_t ctas = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
        if ((int64_t)blockIdx.x >= ctas) {
            if (tid == 0) workspace_at<S::kHeads, DP>(a.partial, gridDim.x).spill[blockIdx.x] = make_int4(0, 0, 0, 0);
            return;
        }
        shares = Shares(total, ctas);
        begin = shares.begin(blockIdx.x);
        count = shares.begin((int64_t)blockIdx.x + 1) - begin;
        if (begin >= upto - mine && begin < upto) {
            int64_t rest = begin - (upto - mine);
            int b = b0, nt = 1;
            for (; b < b1; ++b) {
                nt = tiles_of(local_length(a.sh, a.seq_lens[b], a.kv.capacity), TILE);
                if (rest < (int64_t)nt * a.head_blocks) break;
                rest -= (int64_t)nt * a.head_blocks;
            }
            const int hb = (int)(rest / nt);
            s_where[0] = b;
            s_where[1] = hb;
            s_where[2] = (int)(rest - (int64_t)hb * nt);
        }
        __syncthreads();
        ld.b = s_where[0];
        ld.kvh = s_where[1] / a.row_blocks;
        ld.rb = s_where[1] - ld.kvh * a.row_blocks;
        ld.t = s_where[2];
        ld.next_seq = a.seq_lens[ld.b];
        iter_request<TILE>(a, ld);
    }
    TileIter cp = ld;
    const int ld0_b = ld.b, ld0_kvh = ld.kvh, ld0_rb = ld.rb;  // cluster: its request, key head and head block

    const uint32_t stages = smem_addr(smem) + warp * (ST * S::kStage);
    const uint32_t queries = smem_addr(smem) + NW * ST * S::kStage;
    uint2 *const query_pairs = reinterpret_cast<uint2 *>(smem + NW * ST * S::kStage);  // fp32
    float *const cluster_rows = reinterpret_cast<float *>(smem + NW * ST * S::kStage);  // this CTA's rows at the merge
    static_assert(!CLUSTER || S::kQueries >= S::kHeads * DP * 4, "the query's buffers hold the rows");

    // What this lane copies of a tile: cp.async, row lane mod 16; tensor copies, box `lane` of kBoxes (K's
    // then V's, row groups of BOX slots, panels).  Its page is read one tile ahead.
    constexpr int kGroups = TENSOR ? WP / (TENSOR ? S::BOX : 1) : 1, kBoxes = 2 * kGroups * S::kPanels;
    static_assert(kBoxes <= 32, "one box per lane");
    const int box_panel = lane % S::kPanels, box_group = lane / S::kPanels % kGroups;
    const int my_first = TENSOR ? box_group * S::BOX : lane & (WP - 1);
    int entry = -1;
    uint32_t slot = 0;
    auto next_page = [&]() {
        const int p = ld.t * TILE + warp * WP + my_first;
        entry = -1;
        if (p < ld.n) {
            const uint32_t j = a.kv.page.div((uint32_t)p);
            slot = (uint32_t)p - j * a.kv.page.d;
            entry = __ldg(a.kv.table + ld.b * a.kv.table_stride + j);
        }
    };
    next_page();
    int ld_query = 0, ld_stage = 0;
    // Tensor copies: the lane, or kLate once a wait of it ran out.  It then neither copies, arms nor waits any
    // more (lane 0 must not arm a barrier again whose phase is not complete); the result is not valid.
    // Lanes need not agree: without the copies of some a phase stays incomplete, and the next wait
    // runs out for the others too.
    constexpr int kLate = 32;
    int copier = lane;

    // cp.async: one warp-wide copy covers kRowsPerCopy rows (or a 32-chunk part of one)
    constexpr int kRowsPerCopy = 32 / S::kChunks > 0 ? 32 / S::kChunks : 1;
    constexpr int kCopiesPerRow = S::kChunks > 32 ? S::kChunks / 32 : 1;
    const int my_row = S::kChunks > 32 ? 0 : lane / S::kChunks, my_chunk = S::kChunks > 32 ? lane : lane % S::kChunks;
    const uint32_t lane_to = (my_chunk >> 3) * S::kPanel + my_row * 128;
    const uint32_t lane_sw = (uint32_t)((my_chunk & 7) ^ my_row) << 4;
    const char *const k_base = reinterpret_cast<const char *>(a.kv.k) + my_chunk * 16;
    const char *const v_base = reinterpret_cast<const char *>(a.kv.v) + my_chunk * 16;

    // Starts the copies of the next tile (this warp's positions of it; the query with a new
    // request or head block) and moves on.
    auto copy_next = [&](bool first) {
        if (S::kHalfType && (first || ld.t == 0)) {
            const int head0 = ld.rb * S::kHeads;
            const uint32_t dst = queries + ld_query * S::kQuery;
            const uint32_t *src = a.q + ld.b * a.q_sb_w + (int64_t)(ld.kvh * a.group + head0) * a.q_sh_w;
            for (int i = tid; i < S::kHeads * S::kChunks; i += S::kThreads) {
                const int r = i / S::kChunks, c = i - r * S::kChunks;
                const bool in = head0 + r < a.group && c * 4 < a.kv.data_w;
                cp_async_or_zero(dst + (r * S::kChunks + (c ^ (r & 7))) * 16, in ? src + r * a.q_sh_w + c * 4 : a.q, in);
            }
            ld_query = ld_query + 1 == ST ? 0 : ld_query + 1;
        }
        const int p0 = ld.t * TILE + warp * WP;
        if (p0 < ld.n) {
            const bool held = entry >= 0 && entry < a.kv.num_pages;
            const uint32_t votes = __ballot_sync(0xffffffffu, held);
            if constexpr (TENSOR) {
                const int left = ld.n - p0;
                uint32_t bits = left < WP ? (1u << left) - 1u : (1u << WP) - 1u;
#pragma unroll
                for (int r = 0; r < kGroups; ++r)
                    if (!((votes >> (r * S::kPanels)) & 1u)) bits &= ~(((1u << S::BOX) - 1u) << (r * S::BOX));
                if (copier == 0) {
                    s_held[ld_stage][warp] = bits;
                    mbar_arrive_expect_tx(&s_full[warp][ld_stage], S::kStage + a.stall_bytes);
                }
                __syncwarp();
                // a page outside the pool, or past the length (-1), reads zeros
                if (copier < kBoxes) {
                    const bool is_v = lane >= kBoxes / 2;
                    tensor_copy(stages + ld_stage * S::kStage + (is_v ? S::kHalf : 0) + box_panel * S::kPanel +
                                    box_group * (S::BOX * 128),
                                is_v ? &maps.v : &maps.k, box_panel * (128 / S::kBytes), ld.kvh,
                                entry < 0 ? 0 : (int)slot, entry, &s_full[warp][ld_stage]);
                }
            } else {
                const uint32_t bits = votes & ((1u << WP) - 1u);
                __syncwarp();  // the last tile's offsets have been read
                if (lane < WP)
                    s_row(warp)[lane] = make_uint2(entry * a.k_page_u + slot * a.k_slot_u + ld.kvh * a.k_head_u,
                                                   entry * a.v_page_u + slot * a.v_slot_u + ld.kvh * a.v_head_u);
                if (lane == 0) s_held[ld_stage][warp] = bits;
                __syncwarp();
                const uint32_t dst = stages + ld_stage * S::kStage + lane_to;
                if (bits == (1u << WP) - 1u && S::DP * S::kBytes == 4 * a.kv.data_w) {
#pragma unroll
                    for (int i = 0; i < WP * S::kChunks / 32; ++i) {
                        const int row0 = i / kCopiesPerRow * kRowsPerCopy, c0 = i % kCopiesPerRow * 32;
                        const uint2 at = s_row(warp)[row0 + my_row];
                        // (row0 + my_row) mod 8 = (row0 mod 8) ^ my_row: my_row < kRowsPerCopy, which divides row0
                        const uint32_t to = dst + (lane_sw ^ ((row0 & 7) << 4));
                        const int more = row0 * 128 + c0 / 8 * S::kPanel;
                        cp_async_16(to + more, k_base + (uint64_t)at.x * a.unit + c0 * 16);
                        cp_async_16(to + more + S::kHalf, v_base + (uint64_t)at.y * a.unit + c0 * 16);
                    }
                } else {  // rows that are not held, or are shorter, are filled with zeros
#pragma unroll 1
                    for (int i = 0; i < WP * S::kChunks / 32; ++i) {
                        const int row0 = i / kCopiesPerRow * kRowsPerCopy, c0 = i % kCopiesPerRow * 32;
                        const uint2 at = s_row(warp)[row0 + my_row];
                        const uint32_t to = dst + (lane_sw ^ ((row0 & 7) << 4)) + row0 * 128 + c0 / 8 * S::kPanel;
                        const bool in = ((bits >> (row0 + my_row)) & 1u) && (my_chunk + c0) * 4 < a.kv.data_w;
                        cp_async_or_zero(to, in ? k_base + (uint64_t)at.x * a.unit + c0 * 16 : (const char *)a.kv.k, in);
                        cp_async_or_zero(to + S::kHalf,
                                         in ? v_base + (uint64_t)at.y * a.unit + c0 * 16 : (const char *)a.kv.v, in);
                    }
                }
            }
        }
        ld_stage = ld_stage + 1 == ST ? 0 : ld_stage + 1;
        iter_next<TILE>(a, ld);
        next_page();
    };

    for (int i = 0; i < ST - 1; ++i) {
        if (i < count) copy_next(i == 0);
        cp_async_commit();
    }

    // The state of this warp's positions: o[h][j] holds columns 16 j + g (+ 8) of heads 8 h + 2 t4 (+ 1);
    // m and sum (this lane's part) of those two heads.  A logit x (base 2) enters as
    // 2^(x + raise), raise = shift - m; with no logit yet raise is +inf, which sends the first tile
    // through the slow path below.
    const float scale2 = a.scale * kLog2e;
    const int g = lane >> 2, t4 = lane & 3;
    constexpr float kShift = WeightShift<T>::value;
    float o[NH][DP / 16][4], m[NH][2], raise[NH][2], sum[NH][2];
    uint32_t qf[S::kQueryRegs ? NH : 1][S::kQueryRegs ? DP * S::kBytes / 32 : 1][S::kHalfType ? 2 : 4];
    int cp_query = 0, cp_stage = 0, first_t = cp.t;
    uint32_t query = queries;
    // Places of this lane in a stage: ldmatrix rows of K (16-bit) or its floats of K (fp32), and of V.  Of
    // chunk c = 2 j + e the part that depends on j mod 4 is in these, the rest is panel j / 4.
    uint32_t phases = 0;   // bit st: parity of stage st's next arrival
    uint32_t k_at[4], v_at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (S::kHalfType) {
            const int rk = lane & 15, rv = (lane & 7) + ((lane >> 4) << 3);
            k_at[j] = rk * 128 + (((2 * j + (lane >> 4)) ^ (rk & 7)) << 4);
            v_at[j] = S::kHalf + rv * 128 + (((2 * j + ((lane >> 3) & 1)) ^ (rv & 7)) << 4);
        } else {
            k_at[j] = g * 128 + (((2 * j) ^ g) << 4) + t4 * 4;
            // position 2 t4 (the next one's chunks differ in bit 0), column 8 j + g
            v_at[j] = S::kHalf + 2 * t4 * 128 + (((2 * j + (g >> 2)) ^ (2 * t4)) << 4) + (g & 3) * 4;
        }
    }

    for (int64_t i = 0; i < count; ++i) {
        if (i + ST - 1 < count) copy_next(false);
        cp_async_commit();
        cp_async_wait<ST - 1>();
        if (i == 0 || cp.t == 0) {  // a new request or head block
            first_t = cp.t;
            if constexpr (S::kHalfType) {
                __syncthreads();  // every warp's part of the query has arrived
                query = queries + cp_query * S::kQuery;
                cp_query = cp_query + 1 == ST ? 0 : cp_query + 1;
                if constexpr (S::kQueryRegs) {
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ks += 2) {
                            uint32_t q[4];
                            ldmatrix4(q, query + ((h * 8 + (lane & 7)) * S::kChunks +
                                                  ((2 * ks + (lane >> 3)) ^ (lane & 7))) * 16);
                            qf[h][ks][0] = q[0], qf[h][ks][1] = q[1], qf[h][ks + 1][0] = q[2], qf[h][ks + 1][1] = q[3];
                        }
                }
            } else {
                // (hi, lo) pairs, split once: head r, element d at r * DP + (d ^ 4 (r mod 8))
                const int head0 = cp.rb * S::kHeads;
                const uint32_t *src = a.q + cp.b * a.q_sb_w + (int64_t)(cp.kvh * a.group + head0) * a.q_sh_w;
                constexpr int kEach = (S::kHeads * DP + S::kThreads - 1) / S::kThreads;
                float v[kEach];  // all in flight together
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int x = tid + e * S::kThreads, r = x / DP, d = x - r * DP;
                    const bool in = head0 + r < a.group && r < S::kHeads && d < a.kv.data_w;
                    v[e] = in ? __uint_as_float(__ldg(src + r * a.q_sh_w + d)) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const int x = tid + e * S::kThreads, r = x / DP, d = x - r * DP;
                    uint2 pair;
                    tf32_split(v[e], pair.x, pair.y);
                    if (r < S::kHeads) query_pairs[r * DP + (d ^ ((r & 7) << 2))] = pair;
                }
                __syncthreads();
                if constexpr (S::kQueryRegs) {
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int ks = 0; ks < DP / 8; ++ks) {
                            const uint2 *q = query_pairs + (h * 8 + g) * DP + t4;
                            const uint2 q0 = q[((2 * ks) ^ g) * 4], q1 = q[((2 * ks + 1) ^ g) * 4];
                            qf[h][ks][0] = q0.x, qf[h][ks][1] = q1.x, qf[h][ks][2] = q0.y, qf[h][ks][3] = q1.y;
                        }
                }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[h][e] = -INFINITY;
                    raise[h][e] = INFINITY;
                    sum[h][e] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < DP / 16; ++j) o[h][j][0] = o[h][j][1] = o[h][j][2] = o[h][j][3] = 0.f;
            }
        } else {
            __syncwarp();
        }
        const int p0 = cp.t * TILE + warp * WP;
        if (p0 < cp.n) {
            const uint32_t stage = stages + cp_stage * S::kStage;
            const uint32_t held = s_held[cp_stage][warp];
            if constexpr (TENSOR) {
                if (copier != kLate &&
                    !mbar_wait_bounded(&s_full[warp][cp_stage], (phases >> cp_stage) & 1u, a.wait_limit_ns)) {
                    copier = kLate;
                    if (lane == __ffs(__activemask()) - 1) atomicAdd(&g_wait_timeouts, 1ull);
                }
                phases ^= 1u << cp_stage;
                if (held != (1u << WP) - 1u) {
                    // slots past the length hold anything; a weight of 0 must find a finite value there
                    for (int x = lane; x < WP * S::kChunks; x += 32) {
                        const int r = x / S::kChunks, c = x - r * S::kChunks;
                        if (!((held >> r) & 1u))
                            *reinterpret_cast<uint4 *>(smem + (stage - smem_addr(smem)) + S::kHalf + (c >> 3) * S::kPanel +
                                                       r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async();  // before the stage's next tensor copy
                    __syncwarp();
                }
            }
            const bool held0 = (held >> g) & 1u, held1 = (held >> (g + 8)) & 1u;
            // ---- x = K q^T: x[h][0, 1] position g and heads 2 t4, 2 t4 + 1; x[h][2, 3] position g + 8
            float x[NH][4];
            if constexpr (S::kHalfType) {
                float x1[NH][4];  // odd steps, to halve the chain of dependent products
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[h][e] = x1[h][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ks += 2) {
                    uint32_t k0[4], k1[4];
                    ldmatrix4(k0, stage + k_at[ks & 3] + (ks >> 2) * S::kPanel);
                    ldmatrix4(k1, stage + k_at[(ks + 1) & 3] + (ks >> 2) * S::kPanel);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        uint32_t q[4];
                        if constexpr (S::kQueryRegs) {
                            q[0] = qf[h][ks][0], q[1] = qf[h][ks][1], q[2] = qf[h][ks + 1][0], q[3] = qf[h][ks + 1][1];
                        } else {
                            ldmatrix4(q, query + ((h * 8 + (lane & 7)) * S::kChunks +
                                                  ((2 * ks + (lane >> 3)) ^ (lane & 7))) * 16);
                        }
                        mma(T{}, x[h], k0, q[0], q[1]);
                        mma(T{}, x1[h], k1, q[2], q[3]);
                    }
                }
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[h][e] += x1[h][e];
            } else {
                // three tf32 products: hi hi + hi lo + lo hi (lo lo is below 2^-22 of the product)
                // hi hi in sums of 16 elements, added in fp32: the product units cut what they add to a sum
                float x1[NH][4], x2[NH][4], part[NH][4];
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[h][e] = x1[h][e] = x2[h][e] = 0.f;
                // all of it unrolled: 3% faster than a loop over panels at D = 64 with 64 heads on 4, no slower elsewhere
#pragma unroll
                for (int pn = 0; pn < S::kPanels; ++pn) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ks = 4 * pn + i;
                        if (i % 2 == 0) {
#pragma unroll
                            for (int h = 0; h < NH; ++h)
#pragma unroll
                                for (int e = 0; e < 4; ++e) part[h][e] = 0.f;
                        }
                        const uint32_t at = stage - smem_addr(smem) + k_at[i] + pn * S::kPanel, next = at ^ 16;
                        uint32_t kh[4], kl[4];
                        tf32_split(*reinterpret_cast<const float *>(smem + at), kh[0], kl[0]);
                        tf32_split(*reinterpret_cast<const float *>(smem + at + 8 * 128), kh[1], kl[1]);
                        tf32_split(*reinterpret_cast<const float *>(smem + next), kh[2], kl[2]);
                        tf32_split(*reinterpret_cast<const float *>(smem + next + 8 * 128), kh[3], kl[3]);
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            uint32_t q[4];
                            if constexpr (S::kQueryRegs) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) q[e] = qf[h][ks][e];
                            } else {
                                const uint2 *qp = query_pairs + (h * 8 + g) * DP + t4;
                                const uint2 q0 = qp[((2 * ks) ^ g) * 4], q1 = qp[((2 * ks + 1) ^ g) * 4];
                                q[0] = q0.x, q[1] = q1.x, q[2] = q0.y, q[3] = q1.y;
                            }
                            mma(T{}, part[h], kh, q[0], q[1]);
                            mma(T{}, x1[h], kh, q[2], q[3]);
                            mma(T{}, x2[h], kl, q[0], q[1]);
                        }
                        if (i % 2 == 1) {
#pragma unroll
                            for (int h = 0; h < NH; ++h)
#pragma unroll
                                for (int e = 0; e < 4; ++e) x[h][e] += part[h][e];
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[h][e] += x1[h][e] + x2[h][e];
            }
            // ---- logits: 8 lanes write 8 adjacent positions of a head
            if (a.logits_cap) {
                const int end = min(cp.n, a.logits_cap), p = p0 + g;
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int head = cp.rb * S::kHeads + h * 8 + 2 * t4 + e;
                        if (head >= a.group) continue;
                        float *to = a.logits + cp.b * a.logits_sb + (int64_t)(cp.kvh * a.group + head) * a.logits_sh + p;
                        if (p < end) to[0] = held0 ? x[h][e] * a.scale : -INFINITY;
                        if (p + 8 < end) to[8] = held1 ? x[h][2 + e] * a.scale : -INFINITY;
                    }
            }
            // ---- weights 2^(x scale2 + raise).  The maximum m moves only when a logit exceeds it by more
            // than kSlack: weights up to 2^kSlack are as exact, and neither the reduction over
            // the warp nor the rescale is needed in the usual tile.
            float w[NH][4];
            bool usual = true;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[h][e] = fmaf(x[h][e], scale2, raise[h][e & 1]);
                    if (held != (1u << WP) - 1u && !(e < 2 ? held0 : held1)) w[h][e] = -INFINITY;
                    usual = usual && w[h][e] <= kSlack + kShift;  // false for NaN
                }
            if (!__all_sync(0xffffffffu, usual)) {
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y0 = held0 ? x[h][e] * scale2 : -INFINITY, y1 = held1 ? x[h][2 + e] * scale2 : -INFINITY;
                        float top = fmaxf(y0, y1);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        if (top > m[h][e] + kSlack) {
                            const float keep = exp2_fast(m[h][e] - top);  // 0 when there was no logit
                            m[h][e] = top;
                            raise[h][e] = kShift - top;
                            sum[h][e] *= keep;
#pragma unroll
                            for (int j = 0; j < DP / 16; ++j) {
                                o[h][j][e] *= keep;
                                o[h][j][2 + e] *= keep;
                            }
                        }
                        // no finite logit yet: -inf gives 0, NaN gives NaN
                        const float add = m[h][e] == -INFINITY ? 0.f : raise[h][e];
                        w[h][e] = y0 + add;
                        w[h][2 + e] = y1 + add;
                    }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[h][e] = exp2_fast(w[h][e]);
                sum[h][0] += w[h][0] + w[h][2];
                sum[h][1] += w[h][1] + w[h][3];
            }
            // ---- o^T += V^T w^T, each weight as two parts of the element type
            if constexpr (S::kHalfType) {
                uint32_t hi[NH][2], lo[NH][2];  // positions 2 t4, 2 t4 + 1 (+ 8) of head g
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float back[2], rest[2];
                        const uint32_t top = T::encode(&w[h][2 * f]);
                        T::decode(top, back);
                        rest[0] = w[h][2 * f] - back[0];
                        rest[1] = w[h][2 * f + 1] - back[1];
                        hi[h][f] = transpose8x8(top);
                        lo[h][f] = transpose8x8(T::encode(rest));
                    }
#pragma unroll
                for (int j = 0; j < DP / 16; ++j) {
                    uint32_t v[4];
                    ldmatrix4_trans(v, stage + v_at[j & 3] + (j >> 2) * S::kPanel);
#pragma unroll
                    for (int h = 0; h < NH; ++h) mma(T{}, o[h][j], v, hi[h][0], hi[h][1]);
#pragma unroll
                    for (int h = 0; h < NH; ++h) mma(T{}, o[h][j], v, lo[h][0], lo[h][1]);
                }
            } else {
                // two steps of 8 positions, in the order 0 2 4 6 1 3 5 7; the weights of position 2 t4 (+ 1)
                // and head g come from the lane that holds them
                uint32_t wh[NH][2][2], wl[NH][2][2];
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int from = 8 * t4 + 4 * e + (g >> 1);
                            const float even = __shfl_sync(0xffffffffu, w[h][2 * f], from);
                            const float odd = __shfl_sync(0xffffffffu, w[h][2 * f + 1], from);
                            tf32_split(g & 1 ? odd : even, wh[h][f][e], wl[h][f][e]);
                        }
                // the tile's products in sums of their own, added to o in fp32: the product units cut what they
                // add to a long sum, which over thousands of positions would be seen (1.6e-6 of the result)
#pragma unroll
                for (int j = 0; j < DP / 16; ++j) {
                    float tile[NH][4];
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) tile[h][e] = 0.f;
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        // columns 16 j + g and, 2 chunks on, 16 j + 8 + g; position 2 t4 + 1 is a row on, its chunks
                        // differ in bit 0
                        const uint32_t base = stage - smem_addr(smem) + f * (8 * 128) + (j >> 1) * S::kPanel;
                        const uint32_t c0 = base + v_at[(2 * j) & 3], c1 = base + v_at[(2 * j + 1) & 3];
                        uint32_t vh[4], vl[4];
                        tf32_split(*reinterpret_cast<const float *>(smem + c0), vh[0], vl[0]);
                        tf32_split(*reinterpret_cast<const float *>(smem + c1), vh[1], vl[1]);
                        tf32_split(*reinterpret_cast<const float *>(smem + (c0 ^ 16) + 128), vh[2], vl[2]);
                        tf32_split(*reinterpret_cast<const float *>(smem + (c1 ^ 16) + 128), vh[3], vl[3]);
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            mma(T{}, tile[h], vl, wh[h][f][0], wh[h][f][1]);
                            mma(T{}, tile[h], vh, wl[h][f][0], wl[h][f][1]);
                            mma(T{}, tile[h], vh, wh[h][f][0], wh[h][f][1]);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[h][j][e] += tile[h][e];
                }
            }
        }
        __syncwarp();

        // ---- the end of a request, or of the share: merge the warps
        const bool last = cp.t + 1 == cp.nt;
        if (last || i + 1 == count) {
            const int head0 = cp.rb * S::kHeads;
            const bool whole = last && first_t == 0;
            const Workspace ws = workspace_at<S::kHeads, DP>(a.partial, gridDim.x);
            const int64_t part = 2 * (int64_t)blockIdx.x + (first_t == 0 ? 1 : 0);
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float s = sum[h][e];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    if (g == 0) s_stat(warp)[h * 8 + 2 * t4 + e] = make_float2(m[h][e], s);
                }
#pragma unroll
            for (int h0 = 0; h0 < NH; h0 += 2) {  // 16 fp32 rows fit this tile's stage, free until the next copy_next
                float *mine = reinterpret_cast<float *>(smem + (size_t)(warp * ST + cp_stage) * S::kStage);
#pragma unroll
                for (int h = h0; h < h0 + 2 && h < NH; ++h)
#pragma unroll
                    for (int j = 0; j < DP / 16; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // row r, column d at d ^ 8 (r / 2 mod 4): the lanes' rows fall into different banks
                            const int r = (h - h0) * 8 + 2 * t4 + (e & 1), d = 16 * j + 8 * (e >> 1) + g;
                            mine[r * DP + (d ^ (t4 << 3))] = o[h][j][e];
                        }
                __syncthreads();
                const int rows = min(16, min(S::kHeads, a.group - head0) - h0 * 8);
                for (int x = tid; x < rows * (DP / 4); x += S::kThreads) {
                    const int r = x / (DP / 4), c = x - r * (DP / 4);
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < NW; ++w) top = fmaxf(top, s_stat(w)[h0 * 8 + r].x);
                    const float base = finite_or_zero_max(top);
                    float total = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float2 st = s_stat(w)[h0 * 8 + r];
                        const float f = exp2_fast(st.x - base);
                        const float4 v = *reinterpret_cast<const float4 *>(
                            reinterpret_cast<const float *>(smem + (size_t)(w * ST + cp_stage) * S::kStage) + r * DP +
                            ((c * 4) ^ (((r >> 1) & 3) << 3)));
                        total = fmaf(st.y, f, total);
                        acc.x = fmaf(v.x, f, acc.x);
                        acc.y = fmaf(v.y, f, acc.y);
                        acc.z = fmaf(v.z, f, acc.z);
                        acc.w = fmaf(v.w, f, acc.w);
                    }
                    if constexpr (CLUSTER) {  // the query's buffers are free now
                        *reinterpret_cast<float4 *>(cluster_rows + (h0 * 8 + r) * DP + c * 4) = acc;
                        if (c == 0) s_part[h0 * 8 + r] = make_float2(top, total);
                    } else if (whole) {
                        write_result<T>(a, cp.b, cp.kvh * a.group + head0 + h0 * 8 + r, c * 4, acc, top, total);
                        if (needs_mending(acc, top, total)) s_mend = 1;
                    } else {
                        const int64_t at = part * S::kHeads + h0 * 8 + r;
                        *reinterpret_cast<float4 *>(ws.rows + at * DP + c * 4) = acc;
                        if (c == 0) ws.stats[at] = make_float2(top, total);
                    }
                }
                __syncthreads();
            }
            if (TENSOR) fence_proxy_async();  // the rows written above, before the stage's next tensor copy
            if (!CLUSTER && i + 1 == count && tid == 0) {
                int4 spill = make_int4(0, cp.b, cp.kvh, cp.rb);
                // parts: this share and those up to the one with the request's last tile
                if (first_t == 0 && !last)
                    spill.x = (int)(shares.of(begin + i + (cp.nt - 1 - cp.t)) - blockIdx.x) + 1;
                ws.spill[blockIdx.x] = spill;
            }
        }
        cp_stage = cp_stage + 1 == ST ? 0 : cp_stage + 1;
        iter_next<TILE>(a, cp);
    }
    if constexpr (CLUSTER) {
        if (count == 0)
            for (int r = tid; r < S::kHeads; r += S::kThreads) s_part[r] = make_float2(-INFINITY, 0.f);
        cluster.sync();
        constexpr int kMost = 8;
        const int ctas = (int)cluster.num_blocks(), head0 = ld0_rb * S::kHeads;
        const int rows = min(S::kHeads, a.group - head0);
        for (int x = (int)cluster.block_rank() * S::kThreads + tid; x < rows * (DP / 4); x += ctas * S::kThreads) {
            const int r = x / (DP / 4), c = x - r * (DP / 4);
            float2 st[kMost];
            float4 v[kMost];
#pragma unroll
            for (int k = 0; k < kMost; ++k) {
                const int from = min(k, ctas - 1);
                st[k] = *cluster.map_shared_rank(&s_part[r], from);
                v[k] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(cluster_rows + r * DP + c * 4, from));
            }
            float top = -INFINITY, total = 0.f;
#pragma unroll
            for (int k = 0; k < kMost; ++k) top = fmaxf(top, st[k].x);
            const float base = finite_or_zero_max(top);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kMost; ++k) {
                if (k >= ctas || (st[k].x == -INFINITY && st[k].y == 0.f)) continue;  // its rows may hold anything
                const float f = exp2_fast(st[k].x - base);
                total = fmaf(st[k].y, f, total);
                acc.x = fmaf(v[k].x, f, acc.x);
                acc.y = fmaf(v[k].y, f, acc.y);
                acc.z = fmaf(v[k].z, f, acc.z);
                acc.w = fmaf(v[k].w, f, acc.w);
            }
            const int h = ld0_kvh * a.group + head0 + r;
            write_result<T>(a, ld0_b, h, c * 4, acc, top, total);
            if (needs_mending(acc, top, total)) mend_columns<T>(a, ld0_b, h, c * 4, top);
        }
        cluster.sync();  // no CTA leaves while another reads its shared memory
    } else if (s_mend) {  // the same for all threads: read after the last merge's barrier
        mend_share<T, TILE, S::kHeads>(a, s_where, count);
    }
    if (TENSOR && copier == kLate) {  // copies may still be on their way into this CTA's shared memory: wait, bounded
        const uint64_t t0 = global_ns();
        for (uint32_t spin = 0; spin < (1u << 26) && global_ns() - t0 < a.wait_limit_ns; ++spin) {
        }
    }
}

// Loads that stay where they are written, so that all of a round's are in flight together.
__device__ __forceinline__ float4 load_float4(const float *p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ float2 load_float2(const float2 *p) {
    float2 v;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}

// Merges the parts of a request that several shares hold: block (c, y) heads R y .. R y + R - 1 of the
// request that starts in share c.  Warp w takes parts w, w + 4, ..., U of them in flight for all R
// heads at once, with a running maximum; the warps meet in shared memory.  R and U keep a round at
// 16 float4 per lane, which the registers hold (32 took 4 us a round instead of 0.9).
template <int DP>
constexpr int kJoinHeads = DP > 128 ? 2 : 4;

template <class T, int HEADS, int DP>
__global__ void __launch_bounds__(128) attention_join_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int R = kJoinHeads<DP>, LANES = DP / 4 < 32 ? DP / 4 : 32, CV = DP / 4 / LANES;  // CV float4 per lane
    constexpr int SUB = 32 / LANES;                    // parts side by side in a warp
    constexpr int U = 4;
    __shared__ float4 s_acc[4][R][DP / 4];
    __shared__ float2 s_st[4][R];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Workspace ws = workspace_at<HEADS, DP>(a.partial, gridDim.x);
    const int4 spill = ws.spill[blockIdx.x];
    const int parts = spill.x, r0 = blockIdx.y * R, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LANES, c = lane % LANES;
    const int rows = min(R, min(HEADS, a.group - spill.w * HEADS) - r0);
    if (parts == 0 || rows <= 0) return;
    float m[R], sum[R];
    float4 acc[R][CV];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int v = 0; v < CV; ++v) acc[r][v] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // all lanes of the warp make the same rounds
    for (int p0 = warp * SUB; p0 < parts; p0 += 4 * SUB * U) {
        float2 st[U][R];
        float4 o[U][R][CV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // part 0 is the share's unfinished request, the others the requests entered in the middle; a part or
            // head too many reads the last one and counts nothing
            const int p = p0 + sub + u * 4 * SUB, pc = min(p, parts - 1);
            const int64_t at = (int64_t)(2 * ((int64_t)blockIdx.x + pc) + (pc == 0 ? 1 : 0)) * HEADS + r0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t row = at + min(r, rows - 1);
                st[u][r] = load_float2(ws.stats + row);
#pragma unroll
                for (int v = 0; v < CV; ++v) o[u][r][v] = load_float4(ws.rows + row * DP + (c + v * LANES) * 4);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + sub + u * 4 * SUB >= parts) st[u][r] = make_float2(-INFINITY, 0.f);
                top = fmaxf(top, st[u][r].x);
            }
            const float base = finite_or_zero_max(top), f0 = exp2_fast(m[r] - base);
            m[r] = top;
            sum[r] *= f0;
#pragma unroll
            for (int v = 0; v < CV; ++v) {
                acc[r][v].x *= f0;
                acc[r][v].y *= f0;
                acc[r][v].z *= f0;
                acc[r][v].w *= f0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + sub + u * 4 * SUB >= parts) continue;  // what was read there may be anything
                const float f = exp2_fast(st[u][r].x - base);
                sum[r] = fmaf(st[u][r].y, f, sum[r]);
#pragma unroll
                for (int v = 0; v < CV; ++v) {
                    acc[r][v].x = fmaf(o[u][r][v].x, f, acc[r][v].x);
                    acc[r][v].y = fmaf(o[u][r][v].y, f, acc[r][v].y);
                    acc[r][v].z = fmaf(o[u][r][v].z, f, acc[r][v].z);
                    acc[r][v].w = fmaf(o[u][r][v].w, f, acc[r][v].w);
                }
            }
        }
    }
#pragma unroll
    for (int d = LANES; d < 32; d <<= 1)  // the warp's halves
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float om = __shfl_xor_sync(0xffffffffu, m[r], d), top = fmaxf(m[r], om);
            const float base = finite_or_zero_max(top), f0 = exp2_fast(m[r] - base), f1 = exp2_fast(om - base);
            m[r] = top;
            sum[r] = fmaf(__shfl_xor_sync(0xffffffffu, sum[r], d), f1, sum[r] * f0);
#pragma unroll
            for (int v = 0; v < CV; ++v) {
                acc[r][v].x = fmaf(__shfl_xor_sync(0xffffffffu, acc[r][v].x, d), f1, acc[r][v].x * f0);
                acc[r][v].y = fmaf(__shfl_xor_sync(0xffffffffu, acc[r][v].y, d), f1, acc[r][v].y * f0);
                acc[r][v].z = fmaf(__shfl_xor_sync(0xffffffffu, acc[r][v].z, d), f1, acc[r][v].z * f0);
                acc[r][v].w = fmaf(__shfl_xor_sync(0xffffffffu, acc[r][v].w, d), f1, acc[r][v].w * f0);
            }
        }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (lane == 0) s_st[warp][r] = make_float2(m[r], sum[r]);
        if (sub == 0)
#pragma unroll
            for (int v = 0; v < CV; ++v) s_acc[warp][r][c + v * LANES] = acc[r][v];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < rows * (DP / 4); x += 128) {
        const int r = x / (DP / 4), col = x - r * (DP / 4);
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, s_st[w][r].x);
        const float base = finite_or_zero_max(top);
        float total = 0.f;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float2 st = s_st[w][r];
            const float4 v = s_acc[w][r][col];
            const float f = exp2_fast(st.x - base);
            total = fmaf(st.y, f, total);
            t.x = fmaf(v.x, f, t.x);
            t.y = fmaf(v.y, f, t.y);
            t.z = fmaf(v.z, f, t.z);
            t.w = fmaf(v.w, f, t.w);
        }
        const int h = spill.z * a.group + spill.w * HEADS + r0 + r;
        write_result<T>(a, spill.y, h, col * 4, t, top, total);
        if (needs_mending(t, top, total)) mend_columns<T>(a, spill.y, h, col * 4, top);
    }
}

}  // namespace dcp

namespace dcp_host {

// CTAs per request, key head and head block of a short call, 0 where the tiles are shared evenly
// instead: as many as leave all of them resident, at most 8 and at most one per tile of the longest
// request that the table can hold, if each then has at most kClusterTiles tiles.  One request of 777, 32
// heads on 8: 6.9 us so, 8.0 with the tiles shared evenly; 24 of 181, 32 heads on 4: 8.7 and 9.8.  The
// host sees the table's width and not the lengths, so a wide table brings the second form to short requests.
constexpr int64_t kClusterTiles = 4;

inline int cluster_size(int64_t segments, int64_t tiles, int64_t most) {
    int c = 1;
    while (c < 8 && c < tiles && 2 * c * segments <= most) c *= 2;
    return segments * c <= most && tiles <= kClusterTiles * c ? c : 0;
}

template <class S>
int32_t launch_stream(dcp::AttentionArgs a, const dcp::PoolMaps &maps, cudaStream_t stream) {
    using T = typename S::T;
    const char *fn = "dcp_paged_attention";
    a.row_blocks = (a.group + S::kHeads - 1) / S::kHeads;
    a.head_blocks = a.kv.heads * a.row_blocks;
    const int64_t most = (int64_t)sm_count() * S::CTAS;
    if constexpr (S::NH <= 2) {
        const int64_t segments = (int64_t)a.B * a.head_blocks;
        const int ctas = cluster_size(segments, a.kv.capacity / S::TILE + 1, most);
        if (ctas) {
            static InstanceCache cache;
            if (!reserve_smem(dcp::attention_stream_kernel<S, true>, cache, S::kSmem))
                return fail(DCP_ERR_CUDA, "%s: cannot reserve shared memory", fn);
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3((unsigned)(segments * ctas));
            cfg.blockDim = dim3(S::kThreads);
            cfg.dynamicSmemBytes = S::kSmem;
            cfg.stream = stream;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)ctas;
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaLaunchKernelEx(&cfg, dcp::attention_stream_kernel<S, true>, a, maps) != cudaSuccess)
                return launch_status(fn);
            return launch_status(fn);
        }
    }
    static InstanceCache cache;
    if (!reserve_smem(dcp::attention_stream_kernel<S, false>, cache, S::kSmem))
        return fail(DCP_ERR_CUDA, "%s: cannot reserve shared memory", fn);
    const int64_t tiles = (int64_t)a.B * a.head_blocks * (a.kv.capacity / S::TILE + 1);
    const int grid = (int)(tiles < most ? tiles : most);
    dcp::attention_stream_kernel<S, false><<<grid, S::kThreads, S::kSmem, stream>>>(a, maps);
    int32_t st = launch_status(fn);
    if (st != DCP_OK) return st;
    // the join's launch overlaps the stream's end; its blocks wait for it before they read
    cudaLaunchConfig_t cfg{};
    const int heads = a.group < S::kHeads ? a.group : S::kHeads;
    cfg.gridDim = dim3(grid, (heads - 1) / dcp::kJoinHeads<S::DP> + 1);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dcp::attention_join_kernel<T, S::kHeads, S::DP>, a) != cudaSuccess)
        return launch_status(fn);
    return launch_status(fn);
}

// The tensor map of a pool, boxes of `box` slots x 128 bytes of one head's rows; false where the
// driver refuses it.
inline bool pool_map(CUtensorMap &map, const void *base, const dcp::PagedCache &c, int64_t page_w, int64_t slot_w,
                     int64_t head_w, int es, int box) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode || c.num_pages < 1) return false;
    const cuuint64_t dim[4] = {(cuuint64_t)c.data_w * 4 / es, (cuuint64_t)c.heads, (cuuint64_t)c.page.d,
                               (cuuint64_t)(c.num_pages < INT32_MAX ? c.num_pages : INT32_MAX)};
    // a dimension of one entry takes any stride
    const int64_t w[3] = {head_w, slot_w, page_w};
    cuuint64_t stride[3];
    for (int i = 0; i < 3; ++i) stride[i] = dim[i + 1] > 1 ? (cuuint64_t)w[i] * 4 : (cuuint64_t)c.data_w * 4;
    const cuuint32_t boxes[4] = {(cuuint32_t)(128 / es), 1, (cuuint32_t)box, 1}, one[4] = {1, 1, 1, 1};
    return encode(&map, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
                  const_cast<void *>(base), dim, stride, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B,
                  c.data_w >= 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class S>
int32_t launch_attention(const dcp::AttentionArgs &a, cudaStream_t stream) {
    dcp::PoolMaps maps;
    const int box = a.kv.page.d % 16 == 0 ? 16 : a.kv.page.d % 8 == 0 ? 8 : 0;
    if (box && pool_map(maps.k, a.kv.k, a.kv, a.kv.k_page_w, a.kv.k_slot_w, a.kv.k_head_w, S::kBytes, box) &&
        pool_map(maps.v, a.kv.v, a.kv, a.kv.v_page_w, a.kv.v_slot_w, a.kv.v_head_w, S::kBytes, box))
        return box == 16 ? launch_stream<typename S::template With<16>>(a, maps, stream)
                         : launch_stream<typename S::template With<8>>(a, maps, stream);
    return launch_stream<S>(a, maps, stream);
}

// The shape for a group of G query heads per key head and D elements, as measured.  fp32 above D = 64 has
// room for 12 (D = 256: 6) warps of one stage or half as many of two, and computes for so long that the
// number of warps counts: a stage is not refilled while its warp computes, but the other warps' copies
// run.  24 requests of 3000, 12 heads on 4, one stage against two: D = 128 59.7 / 65.6 us, D = 256 129 / 176;
// 64 heads on 4, D = 128: 80 / 92 (pages of 20 slots: 87).  For 16-bit types of D = 256 the exchange does not pay (54.5 / 55 us; 64 heads
// on 4: 89 / 59).
template <class T, class F>
auto with_shape(int32_t group, int32_t head_dim, F &&f) {
    using dcp::AttentionShape;
    if constexpr (T::kPerWord == 2) {
        if (head_dim <= 64)
            return group <= 8    ? f(AttentionShape<T, 64, 1, 4, 4, 3>{})
                   : group <= 16 ? f(AttentionShape<T, 64, 2, 4, 4, 3>{})
                                 : f(AttentionShape<T, 64, 4, 4, 4, 2>{});
        if (head_dim <= 128)
            return group <= 8    ? f(AttentionShape<T, 128, 1, 4, 2, 3>{})
                   : group <= 16 ? f(AttentionShape<T, 128, 2, 4, 2, 3>{})
                                 : f(AttentionShape<T, 128, 4, 4, 2, 2>{});
        return group <= 8 ? f(AttentionShape<T, 256, 1, 6, 2, 1>{}) : f(AttentionShape<T, 256, 2, 6, 2, 1>{});
    } else {
        if (head_dim <= 64)
            return group <= 8 ? f(AttentionShape<T, 64, 1, 4, 2, 3>{}) : f(AttentionShape<T, 64, 2, 4, 2, 3>{});
        if (head_dim <= 128)
            return group <= 8 ? f(AttentionShape<T, 128, 1, 4, 1, 3>{}) : f(AttentionShape<T, 128, 2, 6, 1, 2>{});
        return f(AttentionShape<T, 256, 1, 3, 1, 2>{});
    }
}

template <class T>
int32_t paged_attention(const dcp::AttentionArgs &a, cudaStream_t stream) {
    return with_shape<T>(a.group, (int32_t)(a.kv.data_w * T::kPerWord), [&](auto shape) {
        return launch_attention<decltype(shape)>(a, stream);
    });
}

// Internal linkage: each translation unit has its own counter and needs its own reader of it.
static cudaError_t attention_timeouts(unsigned long long &count, int32_t reset) {
    unsigned long long v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, dcp::g_wait_timeouts, sizeof(v));
    if (e == cudaSuccess && reset) {
        const unsigned long long zero = 0;
        e = cudaMemcpyToSymbol(dcp::g_wait_timeouts, &zero, sizeof(zero));
    }
    count += v;
    return e;
}

// Resident CTAs per SM of the kernel that a call of this shape launches, and how many its launch counts on;
// box as in launch_attention.
template <class T>
int32_t attention_resident(int32_t group, int32_t head_dim, int box, bool cluster, int32_t *out) {
    return with_shape<T>(group, head_dim, [&](auto shape) {
        using S = decltype(shape);
        auto ask = [&](auto kernel, size_t smem) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
                return fail(DCP_ERR_CUDA, "attention_resident: cannot reserve shared memory");
            out[0] = resident_ctas(kernel, S::kThreads, smem);
            out[1] = S::CTAS;
            return ok();
        };
        auto boxed = [&](auto s) {
            using B = decltype(s);
            if constexpr (S::NH <= 2)
                if (cluster) return ask(dcp::attention_stream_kernel<B, true>, B::kSmem);
            return ask(dcp::attention_stream_kernel<B, false>, B::kSmem);
        };
        return box == 16 ? boxed(typename S::template With<16>{})
               : box == 8 ? boxed(typename S::template With<8>{})
                          : boxed(S{});
    });
}

template <class T>
int64_t attention_workspace(int32_t group, int32_t head_dim) {
    return with_shape<T>(group, head_dim, [&](auto shape) {
        using S = decltype(shape);
        return dcp::workspace_bytes<S::kHeads, S::DP>((int64_t)sm_count() * S::CTAS);
    });
}

}  // namespace dcp_host
