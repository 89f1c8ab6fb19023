// dcp_paged_attention.cuh -- attention of one new token per request over a paged cache.
//
// x_p = scale (q . k_p), m = max x, result = sum exp(x - m) v / sum exp(x - m), in one pass over
// K and V with the running maximum and sum of the softmax.
//
// What bounds it.  A position costs 2 D elements of K and V per key head and 4 G D flops for the G
// query heads that share it: G flops per byte (16-bit), far below the machine's balance for any
// group of this size, so the kernel is a stream over the held pages and everything else is
// arranged to keep that stream full.  The products are small (G rows); they run on
// mma.sync (m16n8k16, fp32 sums), whose operands come straight from the streamed tile.  tcgen05
// would want 128 rows per product and an operand round trip through tensor memory, for a pipe
// that is idle most of the time either way.
//
// Work split.  The tiles (TILE positions of one request, key head and block of query rows) of the whole batch
// are numbered in a row and divided evenly over the CTAs of one resident wave, whatever the
// lengths: a CTA's share may begin and end inside a request.  Each CTA finds its share from the
// lengths on the device.  A request that lies in one share is finished there; the others leave
// one fp32 partial (unnormalised row, maximum, sum) per share in the workspace, and attention_join_kernel
// merges them in share order (no atomics: the same bits every time).
//
// Inside a CTA each warp streams its own positions (warp w of NW takes every NW-th group of
// WP) through its own ring of shared-memory stages with cp.async, and keeps its own softmax
// state; warps meet only where a request begins (the query) and ends (the merge).
#pragma once

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

// 2^x, results below 2^-126 as 0 (a weight that small adds nothing to an fp32 sum near 1).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}

// 16 bytes global -> shared, or 16 zero bytes (nothing read).
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16u : 0u));
}

// A float as two tf32 values: hi is x rounded to 10 fraction bits (half a step away from zero), lo
// the rest (at most 2^-11 |x|), of which the product keeps 10 fraction bits: hi + lo = x to
// 2^-21 |x|.
__device__ __forceinline__ void tf32_split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

// ---- shapes -----------------------------------------------------------------------------------
// T element type, DP head dim as laid out in shared memory (D <= DP, the rest zero), MT 16-row
// blocks of query heads per pass over K and V, NW warps per CTA, ST stages per warp, CTAS resident
// CTAs per SM.
template <class T_, int DP_, int MT_, int NW_, int ST_, int CTAS_>
struct AttentionShape {
    using T = T_;
    static constexpr int DP = DP_, MT = MT_, NW = NW_, ST = ST_, CTAS = CTAS_;
    static constexpr bool kHalfType = T::kPerWord == 2;
    static constexpr int kBytes = 4 / T::kPerWord;     // element size
    static constexpr int WP = kHalfType ? 16 : 8;      // positions per warp and stage: one k step of P V
    static constexpr int TILE = WP * NW;               // positions per CTA tile
    static constexpr int kRows = 16 * MT;              // query rows per pass
    static constexpr int kChunks = DP * kBytes / 16;   // 16-byte chunks per row
    static constexpr int kHalf = WP * DP * kBytes;     // bytes of a stage's K (and of its V)
    static constexpr int kStage = 2 * kHalf;           // = 64 DP: also 16 fp32 rows of DP
    static constexpr int kQuery = kRows * DP * kBytes;  // bytes of one query buffer
    static constexpr int kQueries = kHalfType ? ST * kQuery : 2 * kQuery;  // one per stage; fp32: one, as pairs
    static constexpr int kThreads = NW * 32;
    static constexpr bool kQueryRegs = kHalfType && MT * DP <= 128;
    static constexpr size_t kSmem = (size_t)NW * ST * kStage + kQueries;
    static_assert(kStage == 16 * DP * 4, "a stage holds one block of fp32 rows");
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

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// ---- workspace --------------------------------------------------------------------------------
// Two partials per CTA (the request it entered in the middle, the one it left unfinished): kRows
// rows of DP floats each, then (maximum, sum) per row, then one int4 per CTA: the number of
// parts of the request that starts in this CTA and is finished by later ones (0: none), its
// request, key head and row block.
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

// Position in the sequence of tiles: tile t of nt of request b, key head kvh and row block rb; n
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
// Four columns of the result row of (b, h), and with column 0 its LSE; sum == 0 is an empty row.
template <class T>
__device__ __forceinline__ void write_result(const AttentionArgs &a, int b, int h, int col, const float4 &o, float m,
                                             float sum) {
    const bool empty = sum == 0.f;
    const float r = empty ? 0.f : 1.f / sum;
    const float f[4] = {empty ? 0.f : o.x * r, empty ? 0.f : o.y * r, empty ? 0.f : o.z * r, empty ? 0.f : o.w * r};
    int64_t off = ((int64_t)b * a.H + h) * a.kv.data_w;
    if (a.pack_hr) {
        const int rank = (int)a.pack_div.div((uint32_t)h);
        off = (((int64_t)rank * a.B + b) * a.pack_hr + (h - rank * a.pack_hr)) * (a.kv.data_w + 1);
    }
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

__device__ __forceinline__ float finite_or_zero_max(float m) { return m == -INFINITY ? 0.f : m; }

// ---- the stream ---------------------------------------------------------------------------------
template <class S>
__global__ void __launch_bounds__(S::kThreads, S::CTAS) attention_stream_kernel(const __grid_constant__ AttentionArgs a) {
    using T = typename S::T;
    constexpr int DP = S::DP, MT = S::MT, NW = S::NW, ST = S::ST, WP = S::WP, TILE = S::TILE;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[NW], s_at[2];
    __shared__ int s_where[4];
    __shared__ float2 s_stat[NW][S::kRows];        // maximum and sum of each warp's rows at a merge
    __shared__ uint32_t s_held[ST][NW];            // bit r: position r of the warp's stage counts
    __shared__ longlong2 s_row[NW][WP];            // addresses of the K and V rows being copied
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;");

    // the share: all lengths summed in one block scan, then the request where it begins
    int64_t begin, count;
    Shares shares(0, 1);
    {
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
            if (tid == 0) workspace_at<S::kRows, DP>(a.partial, gridDim.x).spill[blockIdx.x] = make_int4(0, 0, 0, 0);
            return;
        }
        shares = Shares(total, ctas);
        begin = shares.begin(blockIdx.x);
        count = shares.begin((int64_t)blockIdx.x + 1) - begin;
        if (begin >= upto - mine && begin < upto) {
            int64_t rest = begin - (upto - mine);
            int b = b0, nt = 0;
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
    }
    TileIter ld;
    ld.b = s_where[0];
    ld.kvh = s_where[1] / a.row_blocks;
    ld.rb = s_where[1] - ld.kvh * a.row_blocks;
    ld.t = s_where[2];
    ld.next_seq = a.seq_lens[ld.b];
    iter_request<TILE>(a, ld);
    TileIter cp = ld;

    const uint32_t stages = smem_addr(smem) + warp * (ST * S::kStage);
    const uint32_t queries = smem_addr(smem) + NW * ST * S::kStage;
    uint2 *const query_pairs = reinterpret_cast<uint2 *>(smem + NW * ST * S::kStage);  // fp32

    // This lane's row of the tile that is copied next: its page is read one tile ahead.
    int entry = -1;
    uint32_t slot = 0;
    auto next_page = [&]() {
        const int p = ld.t * TILE + warp * WP + (lane & (WP - 1));
        entry = -1;
        if (p < ld.n) {
            const uint32_t j = a.kv.page.div((uint32_t)p);
            slot = (uint32_t)p - j * a.kv.page.d;
            entry = __ldg(a.kv.table + ld.b * a.kv.table_stride + j);
        }
    };
    next_page();
    int ld_query = 0, ld_stage = 0;

    // One warp-wide copy covers kRowsPerCopy rows (or a 32-chunk part of one).  Chunk c of row r lies
    // at chunk c ^ (r mod 8) of its row in shared memory, so that the 8 rows of an ldmatrix, or
    // of a fragment's float reads, fall into different banks.
    constexpr int kRowsPerCopy = 32 / S::kChunks > 0 ? 32 / S::kChunks : 1;  // rows per warp-wide copy
    constexpr int kCopiesPerRow = S::kChunks > 32 ? S::kChunks / 32 : 1;
    const int my_row = S::kChunks > 32 ? 0 : lane / S::kChunks, my_chunk = S::kChunks > 32 ? lane : lane % S::kChunks;
    const uint32_t lane_to = my_row * S::kChunks * 16, lane_sw = (uint32_t)(my_chunk ^ my_row) << 4;

    // Starts the copies of the next tile (this warp's positions of it; the query with a new
    // request or head block) and moves on.
    auto copy_next = [&](bool first) {
        if (S::kHalfType && (first || ld.t == 0)) {
            const int row0 = ld.rb * S::kRows;
            const uint32_t dst = queries + ld_query * S::kQuery;
            const uint32_t *src = a.q + ld.b * a.q_sb_w + (int64_t)(ld.kvh * a.group + row0) * a.q_sh_w;
            for (int i = tid; i < S::kRows * S::kChunks; i += S::kThreads) {
                const int r = i / S::kChunks, c = i - r * S::kChunks;
                const bool in = row0 + r < a.group && c * 4 < a.kv.data_w;
                cp_async_or_zero(dst + (r * S::kChunks + (c ^ (r & 7))) * 16, in ? src + r * a.q_sh_w + c * 4 : a.q, in);
            }
            ld_query = ld_query + 1 == ST ? 0 : ld_query + 1;
        }
        if (ld.t * TILE + warp * WP < ld.n) {
            const bool held = entry >= 0 && entry < a.kv.num_pages;
            __syncwarp();  // the last tile's addresses have been read
            if (lane < WP) {
                longlong2 at;  // byte addresses of the rows' first chunks
                at.x = reinterpret_cast<int64_t>(a.kv.k) +
                       4 * (entry * a.kv.k_page_w + slot * a.kv.k_slot_w + ld.kvh * a.kv.k_head_w);
                at.y = reinterpret_cast<int64_t>(a.kv.v) +
                       4 * (entry * a.kv.v_page_w + slot * a.kv.v_slot_w + ld.kvh * a.kv.v_head_w);
                s_row[warp][lane] = at;
            }
            const uint32_t bits = __ballot_sync(0xffffffffu, held) & ((1u << WP) - 1u);
            if (lane == 0) s_held[ld_stage][warp] = bits;
            __syncwarp();
            const uint32_t dst = stages + ld_stage * S::kStage + lane_to;
            const bool all = bits == (1u << WP) - 1u && S::DP * S::kBytes == 4 * a.kv.data_w;
#pragma unroll
            for (int i = 0; i < WP * S::kChunks / 32; ++i) {
                const int row0 = i / kCopiesPerRow * kRowsPerCopy, c0 = i % kCopiesPerRow * 32;
                const longlong2 at = s_row[warp][row0 + my_row];
                // row0 + my_row mod 8 = (row0 mod 8) ^ my_row: my_row < kRowsPerCopy, which divides row0
                const uint32_t to = dst + ((lane_sw ^ ((row0 & 7) << 4)) + (row0 * S::kChunks + c0) * 16);
                const char *k = reinterpret_cast<const char *>(at.x) + (my_chunk + c0) * 16;
                const char *v = reinterpret_cast<const char *>(at.y) + (my_chunk + c0) * 16;
                if (all) {
                    cp_async_16(to, k);
                    cp_async_16(to + S::kHalf, v);
                } else {
                    const bool in = ((bits >> (row0 + my_row)) & 1u) && (my_chunk + c0) * 4 < a.kv.data_w;
                    cp_async_or_zero(to, in ? (const void *)k : a.kv.k, in);
                    cp_async_or_zero(to + S::kHalf, in ? (const void *)v : a.kv.v, in);
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

    const float scale2 = a.scale * kLog2e;
    const int g = lane >> 2, t4 = lane & 3;
    const bool upper = a.group > 8;  // rows 8..15 of a block hold query heads
    float o[MT][DP / 8][4], m[MT][2], sum[MT][2];
    uint32_t qf[S::kQueryRegs ? MT : 1][S::kQueryRegs ? DP / 16 : 1][4];
    int cp_query = 0, cp_stage = 0, first_t = cp.t;
    uint32_t query = queries;
    // ldmatrix places of this lane: K rows for the first product, V rows (transposed) for the second.
    // Chunk 2 j + e of row r lies at ((2 j + e) ^ (r mod 8)): 16-byte steps that depend on j mod 4
    // through these, the rest is a constant 128 (j / 4).
    uint32_t k_at[4], v_at[4];
    {
        const int rk = (lane & 7) + ((lane >> 4) << 3), rv = lane & 15;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            k_at[j] = rk * (DP * 2) + (((2 * j + ((lane >> 3) & 1)) ^ (rk & 7)) << 4);
            v_at[j] = S::kHalf + rv * (DP * 2) + (((2 * j + (lane >> 4)) ^ (rv & 7)) << 4);
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
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ++ks) {
                            const int r = mt * 16 + (lane & 15), c = 2 * ks + (lane >> 4);
                            ldmatrix4(qf[mt][ks], query + (r * S::kChunks + (c ^ (r & 7))) * 16);
                        }
                }
            } else {
                // the query as (hi, lo) pairs, split once: row r, element d at r * DP + (d ^ 4 (r mod 8))
                const int row0 = cp.rb * S::kRows;
                const uint32_t *src = a.q + cp.b * a.q_sb_w + (int64_t)(cp.kvh * a.group + row0) * a.q_sh_w;
                for (int x = tid; x < S::kRows * DP; x += S::kThreads) {
                    const int r = x / DP, d = x - r * DP;
                    const bool in = row0 + r < a.group && d < a.kv.data_w;
                    uint2 pair;
                    tf32_split(in ? __uint_as_float(src[r * a.q_sh_w + d]) : 0.f, pair.x, pair.y);
                    query_pairs[r * DP + (d ^ ((r & 7) << 2))] = pair;
                }
                __syncthreads();
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                m[mt][0] = m[mt][1] = -INFINITY;
                sum[mt][0] = sum[mt][1] = 0.f;
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
            }
        } else {
            __syncwarp();
        }
        const int p0 = cp.t * TILE + warp * WP;
        if (p0 < cp.n) {
            constexpr int NT = WP / 8;  // 8-position blocks of the product
            const uint32_t stage = stages + cp_stage * S::kStage;
            const uint32_t held = s_held[cp_stage][warp];
            float x[MT][NT][4];
            // ---- x = q . k
            if constexpr (S::kHalfType) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[mt][0][e] = x[mt][NT - 1][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    uint32_t kb[4];
                    ldmatrix4(kb, stage + k_at[ks & 3] + (ks >> 2) * 128);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t qa[4];
                        if constexpr (S::kQueryRegs) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) qa[e] = qf[mt][ks][e];
                        } else {
                            const int qr = mt * 16 + (lane & 15), c = 2 * ks + (lane >> 4);
                            ldmatrix4(qa, query + (qr * S::kChunks + (c ^ (qr & 7))) * 16);
                        }
                        mma(T{}, x[mt][0], qa, kb[0], kb[1]);
                        mma(T{}, x[mt][NT - 1], qa, kb[2], kb[3]);
                    }
                }
            } else {
                // three tf32 products: hi hi + hi lo + lo hi (lo lo is below 2^-22 of the product)
                float x1[4] = {0.f, 0.f, 0.f, 0.f}, x2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) x[0][0][e] = 0.f;
                const float *kr = reinterpret_cast<const float *>(smem + (stage - smem_addr(smem))) + g * DP + t4;
                const uint2 *qr = query_pairs + g * DP + t4;
#pragma unroll
                for (int ks = 0; ks < DP / 8; ++ks) {
                    const int c0 = ((2 * ks) ^ g) * 4, c1 = ((2 * ks + 1) ^ g) * 4;
                    uint32_t kh[2], kl[2];
                    tf32_split(kr[c0], kh[0], kl[0]);
                    tf32_split(kr[c1], kh[1], kl[1]);
                    const uint2 q0 = qr[c0], q1 = upper ? qr[8 * DP + c0] : make_uint2(0u, 0u), q2 = qr[c1],
                                q3 = upper ? qr[8 * DP + c1] : make_uint2(0u, 0u);
                    const uint32_t qh[4] = {q0.x, q1.x, q2.x, q3.x}, ql[4] = {q0.y, q1.y, q2.y, q3.y};
                    mma(T{}, x[0][0], qh, kh[0], kh[1]);
                    mma(T{}, x1, qh, kl[0], kl[1]);
                    mma(T{}, x2, ql, kh[0], kh[1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[0][0][e] += x1[e] + x2[e];
            }
            // ---- logits
            if (a.logits_cap) {
                const int row0 = cp.rb * S::kRows, end = min(cp.n, a.logits_cap);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int r = row0 + mt * 16 + half * 8 + g;
                        if (r >= a.group) continue;
                        float *to = a.logits + cp.b * a.logits_sb + (int64_t)(cp.kvh * a.group + r) * a.logits_sh + p0;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int c = nt * 8 + 2 * t4;
                            const float v0 = (held >> c) & 1u ? x[mt][nt][2 * half] * a.scale : -INFINITY;
                            const float v1 = (held >> (c + 1)) & 1u ? x[mt][nt][2 * half + 1] * a.scale : -INFINITY;
                            if (a.logits_pairs && p0 + WP <= end) {
                                *reinterpret_cast<float2 *>(to + c) = make_float2(v0, v1);
                            } else {
                                if (p0 + c < end) to[c] = v0;
                                if (p0 + c + 1 < end) to[c + 1] = v1;
                            }
                        }
                    }
            }
            // ---- base-2 logits, masked
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[mt][nt][e] *= scale2;
            if (held != (1u << WP) - 1u) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!((held >> (nt * 8 + 2 * t4 + (e & 1))) & 1u)) x[mt][nt][e] = -INFINITY;
            }
            // ---- running maximum and weights.  The maximum m moves only when a logit exceeds it by more
            // than kSlack: weights up to 2^kSlack are as exact, and the rescale is nearly never needed.
            bool grew = false;
            float keep[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    keep[mt][half] = 1.f;
                    if (half == 1 && !upper) {  // no query heads there: zero weights
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) x[mt][nt][2] = x[mt][nt][3] = 0.f;
                        continue;
                    }
                    float top = fmaxf(x[mt][0][2 * half], x[mt][0][2 * half + 1]);
                    if (NT == 2) top = fmaxf(top, fmaxf(x[mt][NT - 1][2 * half], x[mt][NT - 1][2 * half + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const float old = m[mt][half];
                    if (top > old + kSlack) {
                        grew = true;
                        m[mt][half] = top;
                        keep[mt][half] = exp2_fast(old - top);
                    }
                    const float base = finite_or_zero_max(m[mt][half]) - WeightShift<T>::value;
                    float add = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &v = x[mt][nt][2 * half + e];
                            v = exp2_fast(v - base);
                            add += v;
                        }
                    sum[mt][half] = fmaf(sum[mt][half], keep[mt][half], add);
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < DP / 8; ++j) {
                        o[mt][j][0] *= keep[mt][0];
                        o[mt][j][1] *= keep[mt][0];
                        o[mt][j][2] *= keep[mt][1];
                        o[mt][j][3] *= keep[mt][1];
                    }
            }
            // ---- o += weights . v, each weight as two parts of the element type
            if constexpr (S::kHalfType) {
                uint32_t hi[MT][4], lo[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        const float *w = &x[mt][f >> 1][2 * (f & 1)];
                        float back[2], rest[2];
                        hi[mt][f] = T::encode(w);
                        T::decode(hi[mt][f], back);
                        rest[0] = w[0] - back[0];
                        rest[1] = w[1] - back[1];
                        lo[mt][f] = T::encode(rest);
                    }
#pragma unroll
                for (int j = 0; j < DP / 16; ++j) {
                    uint32_t vb[4];
                    ldmatrix4_trans(vb, stage + v_at[j & 3] + (j >> 2) * 128);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma(T{}, o[mt][2 * j], hi[mt], vb[0], vb[1]);
                        mma(T{}, o[mt][2 * j + 1], hi[mt], vb[2], vb[3]);
                        mma(T{}, o[mt][2 * j], lo[mt], vb[0], vb[1]);
                        mma(T{}, o[mt][2 * j + 1], lo[mt], vb[2], vb[3]);
                    }
                }
            } else {
                // the k index of the product runs over positions in the order 0 2 4 6 1 3 5 7, which
                // is how the weights lie in the registers of the first product
                uint32_t wh[4], wl[4];
                tf32_split(x[0][0][0], wh[0], wl[0]);
                tf32_split(x[0][0][2], wh[1], wl[1]);
                tf32_split(x[0][0][1], wh[2], wl[2]);
                tf32_split(x[0][0][3], wh[3], wl[3]);
                const float *v0 = reinterpret_cast<const float *>(smem + (stage + S::kHalf - smem_addr(smem))) +
                                  (2 * t4) * DP + (g & 3);
#pragma unroll
                for (int j = 0; j < DP / 8; ++j) {
                    const int c = 2 * j + (g >> 2);
                    uint32_t vh[2], vl[2];
                    tf32_split(v0[(c ^ (2 * t4)) * 4], vh[0], vl[0]);
                    tf32_split(v0[DP + (c ^ (2 * t4 + 1)) * 4], vh[1], vl[1]);
                    mma(T{}, o[0][j], wh, vh[0], vh[1]);
                    mma(T{}, o[0][j], wh, vl[0], vl[1]);
                    mma(T{}, o[0][j], wl, vh[0], vh[1]);
                }
            }
        }
        __syncwarp();

        // ---- the end of a request, or of the share: merge the warps
        const bool last = cp.t + 1 == cp.nt;
        if (last || i + 1 == count) {
            const int kvh = cp.kvh, row0 = cp.rb * S::kRows;
            const bool whole = last && first_t == 0;
            const Workspace ws = workspace_at<S::kRows, DP>(a.partial, gridDim.x);
            const int64_t slot = 2 * (int64_t)blockIdx.x + (first_t == 0 ? 1 : 0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float s = sum[mt][half];
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    if (t4 == 0) s_stat[warp][mt * 16 + half * 8 + g] = make_float2(m[mt][half], s);
                }
                // this tile's stage is free until the next copy_next: 16 fp32 rows
                uint8_t *mine = smem + (size_t)(warp * ST + cp_stage) * S::kStage;
#pragma unroll
                for (int j = 0; j < DP / 8; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int r = half * 8 + g, c = 2 * j + (t4 >> 1);
                        *reinterpret_cast<float2 *>(mine + r * (DP * 4) + ((c ^ (r & 7)) << 4) + (t4 & 1) * 8) =
                            make_float2(o[mt][j][2 * half], o[mt][j][2 * half + 1]);
                    }
                __syncthreads();
                const int rows = min(16, a.group - row0 - mt * 16);
                for (int x = tid; x < rows * (DP / 4); x += S::kThreads) {
                    const int r = x / (DP / 4), c = x - r * (DP / 4);
                    float2 st[NW];
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        st[w] = s_stat[w][mt * 16 + r];
                        top = fmaxf(top, st[w].x);
                    }
                    const float base = finite_or_zero_max(top);
                    float total = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float f = exp2_fast(st[w].x - base);
                        const float4 v = *reinterpret_cast<const float4 *>(
                            smem + (size_t)(w * ST + cp_stage) * S::kStage + r * (DP * 4) + ((c ^ (r & 7)) << 4));
                        total = fmaf(st[w].y, f, total);
                        acc.x = fmaf(v.x, f, acc.x);
                        acc.y = fmaf(v.y, f, acc.y);
                        acc.z = fmaf(v.z, f, acc.z);
                        acc.w = fmaf(v.w, f, acc.w);
                    }
                    if (whole) {
                        write_result<T>(a, cp.b, kvh * a.group + row0 + mt * 16 + r, c * 4, acc, top, total);
                    } else {
                        const int64_t at = slot * S::kRows + mt * 16 + r;
                        *reinterpret_cast<float4 *>(ws.rows + at * DP + c * 4) = acc;
                        if (c == 0) ws.stats[at] = make_float2(top, total);
                    }
                }
                __syncthreads();
            }
            if (i + 1 == count && tid == 0) {
                int4 spill = make_int4(0, cp.b, kvh, cp.rb);
                // parts: this share and those up to the one with the request's last tile
                if (first_t == 0 && !last)
                    spill.x = (int)(shares.of(begin + i + (cp.nt - 1 - cp.t)) - blockIdx.x) + 1;
                ws.spill[blockIdx.x] = spill;
            }
        }
        cp_stage = cp_stage + 1 == ST ? 0 : cp_stage + 1;
        iter_next<TILE>(a, cp);
    }
}

// Merges the parts of a request that several shares hold: block (c, r) row r of the request that
// starts in share c.  Its 128 threads cover DP / 4 column groups times 512 / DP parts at a time.
template <class T, int ROWS, int DP>
__global__ void __launch_bounds__(128) attention_join_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int CG = DP / 4, PG = 128 / CG;
    __shared__ float4 s_acc[PG][CG];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Workspace ws = workspace_at<ROWS, DP>(a.partial, gridDim.x);
    const int4 spill = ws.spill[blockIdx.x];
    const int parts = spill.x, r = blockIdx.y, lane = threadIdx.x & 31;
    if (parts == 0) return;
    const int kvh = spill.z, row = spill.w * ROWS + r;
    if (row >= a.group) return;
    // part 0 is the share's unfinished request, the others the requests entered in the middle
    auto slot = [&](int p) { return (int64_t)(2 * ((int64_t)blockIdx.x + p) + (p == 0 ? 1 : 0)) * ROWS + r; };
    float top = -INFINITY;
    for (int p = lane; p < parts; p += 32) top = fmaxf(top, ws.stats[slot(p)].x);
    top = group_max<32>(top);
    const float base = finite_or_zero_max(top);
    float total = 0.f;
    for (int p = lane; p < parts; p += 32) {
        const float2 st = ws.stats[slot(p)];
        total = fmaf(st.y, exp2_fast(st.x - base), total);
    }
    total = group_sum<32>(total);
    const int c = threadIdx.x % CG, pg = threadIdx.x / CG;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = pg; p < parts; p += PG) {
        const int64_t at = slot(p);
        const float f = exp2_fast(ws.stats[at].x - base);
        const float4 v = *reinterpret_cast<const float4 *>(ws.rows + at * DP + c * 4);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
    }
    s_acc[pg][c] = acc;
    __syncthreads();
    if (pg == 0) {
#pragma unroll
        for (int i = 1; i < PG; ++i) {
            const float4 v = s_acc[i][c];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        write_result<T>(a, spill.y, kvh * a.group + row, c * 4, acc, top, total);
    }
}

}  // namespace dcp

namespace dcp_host {

template <class S>
int32_t launch_attention(dcp::AttentionArgs a, cudaStream_t stream) {
    using T = typename S::T;
    static InstanceCache cache;
    const char *fn = "dcp_paged_attention";
    if (!reserve_smem(dcp::attention_stream_kernel<S>, cache, S::kSmem))
        return fail(DCP_ERR_CUDA, "%s: cannot reserve shared memory", fn);
    a.row_blocks = (a.group + S::kRows - 1) / S::kRows;
    a.head_blocks = a.kv.heads * a.row_blocks;
    const int64_t most = (int64_t)sm_count() * S::CTAS;
    const int64_t tiles = (int64_t)a.B * a.head_blocks * (a.kv.capacity / S::TILE + 1);
    const int grid = (int)(tiles < most ? tiles : most);
    dcp::attention_stream_kernel<S><<<grid, S::kThreads, S::kSmem, stream>>>(a);
    int32_t st = launch_status(fn);
    if (st != DCP_OK) return st;
    // the join's launch overlaps the stream's end; its blocks wait for it before they read
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid, a.group < S::kRows ? a.group : S::kRows);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dcp::attention_join_kernel<T, S::kRows, S::DP>, a) != cudaSuccess)
        return launch_status(fn);
    return launch_status(fn);
}

// The shape for a group of G query heads per key head and D elements: 64 DP bytes per warp and
// stage, stages to keep 90 to 200 KB of an SM's shared memory in flight.  Groups over 16 heads take
// two row blocks per pass where the registers hold them (the cache is then read half as often).
template <class T, class F>
auto with_shape(int32_t group, int32_t head_dim, F &&f) {
    if constexpr (T::kPerWord == 2) {
        if (head_dim <= 64)
            return group <= 16 ? f(dcp::AttentionShape<T, 64, 1, 4, 5, 2>{}) : f(dcp::AttentionShape<T, 64, 2, 4, 5, 2>{});
        if (head_dim <= 128)
            return group <= 16 ? f(dcp::AttentionShape<T, 128, 1, 4, 3, 2>{})
                               : f(dcp::AttentionShape<T, 128, 2, 8, 3, 1>{});
        return f(dcp::AttentionShape<T, 256, 1, 4, 3, 1>{});
    } else {
        if (head_dim <= 64) return f(dcp::AttentionShape<T, 64, 1, 4, 5, 2>{});
        if (head_dim <= 128) return f(dcp::AttentionShape<T, 128, 1, 8, 3, 1>{});
        return f(dcp::AttentionShape<T, 256, 1, 4, 2, 1>{});
    }
}

template <class T>
int32_t paged_attention(const dcp::AttentionArgs &a, cudaStream_t stream) {
    return with_shape<T>(a.group, (int32_t)(a.kv.data_w * T::kPerWord), [&](auto shape) {
        return launch_attention<decltype(shape)>(a, stream);
    });
}

template <class T>
int64_t attention_workspace(int32_t group, int32_t head_dim) {
    return with_shape<T>(group, head_dim, [&](auto shape) {
        using S = decltype(shape);
        return dcp::workspace_bytes<S::kRows, S::DP>((int64_t)sm_count() * S::CTAS);
    });
}

}  // namespace dcp_host
