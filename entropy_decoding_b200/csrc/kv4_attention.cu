// kv4_attention.cu -- attention over the paged 4-bit key/value cache, the
// cache decoded on chip.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "df11.h"
#include "kv4.cuh"
#include "serve.h"
#include "walk.cuh"

namespace df11 {
namespace {

struct AttnParams {
    const uint8_t *pages;
    uint64_t n_pages;
    uint32_t kv_heads, group, page_shift;
    Kv4Block block;
    float k_scale, v_scale;
    df11_kv4_attention_args a;
    int *err;
    uint64_t wait_ns;   // limit of each wait for a copy
    uint32_t ws_parts;  // workspace, in floats: counters before, partial results from here
};

__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float &lo, float &hi) {
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
}

// ------------------------------------------------------------------ few rows: keys shared out over the GPU

// S^T = K Q^T and O^T += V^T P^T with m16n8k16: keys (then head elements) are
// the 16 rows, the 8 columns are up to 8 (token, query head) rows that share a
// cache head, so a group of 8 wastes nothing and the accumulators of 64 keys
// and of O fit registers.  A thread's codes are consecutive bytes of one key
// (or of 4 keys' same 16 elements), so operands go from the cache's bytes to
// MMA fragments inside a thread: the order of elements within a product and of
// keys within a tile is free as long as both operands agree.  tcgen05 would
// want the decoded tile written to shared memory with 128 rows of which 8
// columns are used; here nothing decoded is ever stored.
constexpr int kSplitWarps = 10;
constexpr int kSplitThreads = 32 * kSplitWarps;
constexpr int kSplitCols = 8;    // rows of a unit
constexpr int kSplitKeys = 64;   // keys of a chunk: a warp's step, one stage of its ring
constexpr int kSplitStages = 2;
constexpr int kSplitMaxRows = 64;  // rows (tokens x heads of a group) of a request that go this way

template <int D>
struct SplitShared {
    static constexpr uint32_t kStage = kSplitKeys * D * 9 / 8;
    static constexpr int kPitch = D + 4;  // floats; spreads a thread's columns over the banks
    alignas(128) uint8_t ring[kSplitWarps][kSplitStages][kStage];
    alignas(16) float o[kSplitWarps][kSplitCols][kPitch];
    float m[kSplitWarps][kSplitCols], l[kSplitWarps][kSplitCols];
    alignas(8) uint64_t full[kSplitWarps][kSplitStages];
    int64_t sums[kSplitWarps];
    int64_t total, start_off;
    int32_t start_req, last;
};

// A partial result in the workspace: unnormalised O (8 x D), then m and l.
template <int D>
__host__ __device__ constexpr uint32_t split_partial_floats() {
    return kSplitCols * D + 2 * kSplitCols;
}

// The part of a request that this path handles: chunks [c_lo, c_lo + chunks)
// of its keys for each of `units` (cache head, tile of 8 rows) pairs.  A
// request that sees no key still has one chunk, which writes its zeros.
struct SplitReq {
    int32_t q0, n, rows, tiles, units, c_lo, chunks;
    int64_t kv, begin;  // keys; the first that any row sees
};

__device__ __forceinline__ bool rows_valid(const df11_kv4_attention_args &A, int q0, int q1) {
    return q0 >= 0 && q1 >= q0 && q1 <= A.n_tokens && q1 - q0 <= A.max_q_len;
}

__device__ __forceinline__ SplitReq split_req(const AttnParams &P, int r) {
    const df11_kv4_attention_args &A = P.a;
    SplitReq q{};
    q.q0 = __ldg(A.q_start + r);
    const int q1 = __ldg(A.q_start + r + 1);
    if (!rows_valid(A, q.q0, q1)) return q;
    q.n = q1 - q.q0;
    const int64_t rows = static_cast<int64_t>(q.n) * P.group;
    if (rows == 0 || rows > kSplitMaxRows) return q;
    q.rows = static_cast<int32_t>(rows);
    q.tiles = (q.rows + kSplitCols - 1) / kSplitCols;
    q.kv = max(__ldg(A.kv_lens + r), 0);
    const int64_t cap = static_cast<int64_t>(A.max_pages) << P.page_shift;
    const int64_t end = min(q.kv, cap);
    q.begin = A.window ? min(max(q.kv - q.n + 1 - A.window, static_cast<int64_t>(0)), end) : 0;
    q.c_lo = static_cast<int32_t>(q.begin / kSplitKeys);
    q.chunks = max(static_cast<int32_t>((end + kSplitKeys - 1) / kSplitKeys) - q.c_lo, 1);
    q.units = static_cast<int32_t>(P.kv_heads) * q.tiles;
    return q;
}

// A position in the launch's chunks, in the order request, unit, chunk.
struct SplitPos {
    SplitReq q;
    int r, head, tile, c;
    // The request at or after r that has chunks here.
    __device__ __forceinline__ void load(const AttnParams &P) {
        for (; r < P.a.n_reqs; ++r) {
            q = split_req(P, r);
            if (q.units) return;
        }
    }
    // `by` chunks on; the caller knows that they exist.
    __device__ __forceinline__ void advance(const AttnParams &P, int by) {
        c += by;
        while (c >= q.chunks && r < P.a.n_reqs) {
            c -= q.chunks;
            if (++tile < q.tiles) continue;
            tile = 0;
            if (++head < static_cast<int>(P.kv_heads)) continue;
            head = 0;
            ++r;
            load(P);
        }
    }
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a warp has of a unit: its queries as the B operand, and per column
// (the thread's are 2t and 2t + 1) the factor of the scores (log2 units), the
// keys seen, the running maximum and sum, and O.
template <int D>
struct SplitUnit {
    uint32_t qb[D / 16][2];
    float f[2], m[2], l[2];
    int64_t lo[2], hi[2], all_lo, all_hi, any_lo, any_hi;
    float o[D / 16][4];
};

// Loads the unit's queries: thread (g, t) takes elements [t D / 4, (t + 1) D /
// 4) of column g.  A column is scaled by a power of two that brings its
// largest element into [1, 2): FP16 holds it without loss but for elements
// below 2^-24 of that one.
template <int D>
__device__ __forceinline__ void split_load_unit(const AttnParams &P, const SplitPos &at, int lane, SplitUnit<D> &U) {
    const df11_kv4_attention_args &A = P.a;
    const int g = lane >> 2, t = lane & 3;
    const int tile = at.tile, row = tile * kSplitCols + g;
    float x[D / 4];
    if (row < at.q.rows) {
        const uint4 *p = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(A.q) +
            static_cast<int64_t>(at.q.q0 + row / static_cast<int>(P.group)) * static_cast<int64_t>(A.q_token_stride) +
            (at.head * static_cast<int>(P.group) + row % static_cast<int>(P.group)) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 v = __ldg(p + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.0f;
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // 2^e <= top < 2^(e + 1), e in -126 .. 127 (0 for zeros and infinities)
    const uint32_t field = __float_as_uint(top) >> 23;
    const int e = top == 0.0f || field == 255u ? 0 : max(static_cast<int>(field) - 127, -126);
    const float down = e == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
        U.qb[j][0] = pack_f16(x[4 * j] * down, x[4 * j + 1] * down);
        U.qb[j][1] = pack_f16(x[4 * j + 2] * down, x[4 * j + 3] * down);
    }
    U.all_lo = 0;
    U.all_hi = INT64_MAX;
    U.any_lo = INT64_MAX;
    U.any_hi = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = 2 * t + i, ec = __shfl_sync(0xFFFFFFFFu, e, 4 * col);
        U.f[i] = A.scale * P.k_scale * 1.44269504088896341f * __uint_as_float(static_cast<uint32_t>(ec + 127) << 23);
        U.m[i] = -INFINITY;
        U.l[i] = 0.0f;
        const int rc = tile * kSplitCols + col;
        U.lo[i] = 0;
        U.hi[i] = INT64_MAX;
        if (rc < at.q.rows) {
            const int64_t pos = at.q.kv - at.q.n + rc / static_cast<int>(P.group);
            U.hi[i] = max(A.causal ? pos + 1 : at.q.kv, static_cast<int64_t>(0));
            U.lo[i] = A.window ? max(pos + 1 - A.window, static_cast<int64_t>(0)) : 0;
        }
    }
    {
        // what every row of the tile sees, and what any does (rows ascend)
        const int r0 = tile * kSplitCols, r1 = min(r0 + kSplitCols, at.q.rows) - 1;
        const int64_t p0 = at.q.kv - at.q.n + r0 / static_cast<int>(P.group);
        const int64_t p1 = at.q.kv - at.q.n + r1 / static_cast<int>(P.group);
        const int64_t cap = static_cast<int64_t>(A.max_pages) << P.page_shift, end = min(at.q.kv, cap);
        U.all_hi = min(A.causal ? p0 + 1 : end, end);
        U.any_hi = min(A.causal ? p1 + 1 : end, end);
        U.all_lo = A.window ? p1 + 1 - A.window : 0;
        U.any_lo = A.window ? max(p0 + 1 - A.window, static_cast<int64_t>(0)) : 0;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) U.o[i][j] = 0.0f;
}

// Lane p < (pages of a chunk): the block-table entry of the chunk's page p, or
// kNoPage for one that holds no key a row sees.  Pages of 128 tokens are read
// by halves: page 0 of the chunk is the half.
constexpr int64_t kNoPage = INT64_MIN;

__device__ __forceinline__ int64_t split_page(const AttnParams &P, const SplitPos &at, int lane) {
    const int eps_shift = min(static_cast<int>(P.page_shift), 6);
    const int64_t key = static_cast<int64_t>(at.q.c_lo + at.c) * kSplitKeys + (static_cast<int64_t>(lane) << eps_shift);
    const int64_t pg = key >> P.page_shift;
    if ((lane << eps_shift) >= kSplitKeys || key >= at.q.kv || key + (1 << eps_shift) <= at.q.begin ||
        pg >= P.a.max_pages)
        return kNoPage;
    return __ldg(P.a.block_table + static_cast<int64_t>(at.r) * P.a.max_pages + pg);
}

// Copies a chunk's pages (of the unit's head) into a stage, each as its own
// block of min(page_size, 64) tokens.  Returns the mask of the pages that are
// there (bit p, all lanes); flags bad entries.
template <int D>
__device__ __forceinline__ uint32_t split_issue(const AttnParams &P, const SplitPos &at, int64_t id, int lane,
                                                uint8_t *stage, uint64_t *bar, uint32_t &err) {
    const bool have = id >= 0 && static_cast<uint64_t>(id) < P.n_pages;
    if (!have && id != kNoPage) err |= DF11_DEV_ERR_PAGES;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, have);
    const uint8_t *src =
        P.pages + (static_cast<uint64_t>(have ? id : 0) * P.kv_heads + static_cast<uint32_t>(at.head)) * P.block.bytes;
    if (P.page_shift <= 6) {
        const uint32_t bytes = P.block.bytes;
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(mask) * bytes);
        __syncwarp();
        if (have) bulk_load(stage + lane * bytes, src, bytes, bar);
    } else {
        // half of a 128-token page: its rows of the three row-ordered sections
        // are contiguous, the V scales are 64 bytes of each block's 128
        constexpr Kv4Block H = kv4_block(64, D);
        const uint32_t half = static_cast<uint32_t>((at.q.c_lo + at.c) & 1);
        if (lane == 0) mbar_arrive_expect_tx(bar, mask ? H.bytes : 0);
        const uint64_t base = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(src), 0);
        const uint8_t *s0 = reinterpret_cast<const uint8_t *>(base);
        __syncwarp();
        if (mask) {
            if (lane == 0) bulk_load(stage, s0 + half * H.k_scales, H.k_scales, bar);
            if (lane == 1)
                bulk_load(stage + H.k_scales, s0 + P.block.k_scales + half * (H.v_codes - H.k_scales),
                          H.v_codes - H.k_scales, bar);
            if (lane == 2)
                bulk_load(stage + H.v_codes, s0 + P.block.v_codes + half * (H.v_scales - H.v_codes),
                          H.v_scales - H.v_codes, bar);
            if (lane >= 3 && lane < 3 + D / 16)
                bulk_load(stage + H.v_scales + (lane - 3) * 64, s0 + P.block.v_scales + (lane - 3) * 128 + half * 64, 64,
                          bar);
        }
    }
    return mask;
}

// One chunk: scores of 64 keys, their softmax against the running maximum, and
// the products with V.
template <int D>
__device__ __forceinline__ void split_chunk(const AttnParams &P, const uint8_t *stage, int64_t key0, uint32_t pages,
                                            int lane, SplitUnit<D> &U) {
    constexpr int KW = D / 32;  // words of a thread's K codes of one key
    const int g = lane >> 2, t = lane & 3;
    const int eps_shift = min(static_cast<int>(P.page_shift), 6);
    const uint32_t eps = 1u << eps_shift;
    const Kv4Block B = kv4_block(eps, D);
    const bool whole = pages == (1u << (kSplitKeys >> eps_shift)) - 1u && key0 >= U.all_lo &&
                       key0 + kSplitKeys <= U.all_hi;
    // rows g and g + 8 of a tile of 16 keys are keys kg and kg + 2, so that
    // the 4 slots of the second product that a thread holds are 4 consecutive keys
    const uint32_t kg = 4u * (static_cast<uint32_t>(g) >> 1) + (g & 1u);
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t in = 16u * i;
        const uint8_t *blk = stage + (in >> eps_shift) * B.bytes;
        const uint32_t off = in & (eps - 1u);
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
        uint32_t w[2][KW], sc[2][KW / 2 ? KW / 2 : 1];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t k = off + kg + 2u * r;
            const uint8_t *c = blk + B.k_codes + k * (D / 2) + t * (D / 8);
            if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4 *>(c);
                w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
                const uint32_t two = e4m3x2_to_f16x2(
                    *reinterpret_cast<const uint16_t *>(blk + B.k_scales + k * (D / 16) + 2 * t));
                sc[r][0] = __byte_perm(two, 0, 0x1010);
                sc[r][1] = __byte_perm(two, 0, 0x3232);
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(c);
                w[r][0] = v.x, w[r][1] = v.y;
                sc[r][0] = e4m3x2_to_f16x2(blk[B.k_scales + k * (D / 16) + t] * 0x0101u);
            }
        }
#pragma unroll
        for (int j = 0; j < KW; ++j) {
            uint32_t a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                e2m1x8_to_f16(w[r][j], a[r]);
#pragma unroll
                for (int x = 0; x < 4; ++x) a[r][x] = f16x2_mul(a[r][x], sc[r][j / 2]);
            }
            mma16816(s[i], a[0][0], a[1][0], a[0][1], a[1][1], U.qb[2 * j][0], U.qb[2 * j][1]);
            mma16816(s[i], a[0][2], a[1][2], a[0][3], a[1][3], U.qb[2 * j + 1][0], U.qb[2 * j + 1][1]);
        }
    }
    // scores in log2 units; what a row does not see is -inf
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            s[i][x] *= U.f[x & 1];
            if (!whole) {
                const uint32_t in = 16u * i + kg + (x & 2u);
                const int64_t key = key0 + in;
                if (!(pages >> (in >> eps_shift) & 1u) || key < U.lo[x & 1] || key >= U.hi[x & 1] || key >= U.any_hi)
                    s[i][x] = -INFINITY;
            }
            top[x & 1] = fmaxf(top[x & 1], s[i][x]);
        }
    }
    bool moved = false;
    float shift[2], alpha[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], x));
        const float mn = fmaxf(U.m[c], top[c]);
        shift[c] = mn == -INFINITY ? 0.0f : mn;
        alpha[c] = ex2(U.m[c] - shift[c]);
        moved |= U.m[c] != mn;
        U.m[c] = mn;
        U.l[c] *= alpha[c];
    }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) U.o[i][x] *= alpha[x & 1];
    }
    uint32_t pb[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            s[i][x] = ex2(s[i][x] - shift[x & 1]);
            U.l[x & 1] += s[i][x];
        }
        // rounded to FP16 (2^-11 relative): a probability's error is far below that of the 4-bit values it weighs
        pb[i][0] = transpose8x8(pack_f16(s[i][0], s[i][1]));
        pb[i][1] = transpose8x8(pack_f16(s[i][2], s[i][3]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t in = 16u * i;
        const uint8_t *blk = stage + (in >> eps_shift) * B.bytes;
        const uint32_t off = in & (eps - 1u);
        const int b = D == 128 ? g : g >> 1;  // the scale block of the thread's elements [g D / 8, (g + 1) D / 8)
        const uint8_t *c = blk + B.v_codes + (((off >> 2) + t) * (D / 16) + b) * 32u;
        uint32_t vs = *reinterpret_cast<const uint32_t *>(blk + B.v_scales + (b << eps_shift) + off + 4 * t);
        if (!whole) {
            // a key that no row sees may hold anything, NaN scales too: 0 times NaN must not reach a sum
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t k = in + 4 * t + x;
                const int64_t key = key0 + k;
                if (!(pages >> (k >> eps_shift) & 1u) || key < U.any_lo || key >= U.any_hi) vs &= ~(0xFFu << (8 * x));
            }
        }
        const uint32_t sc[2] = {e4m3x2_to_f16x2(vs & 0xFFFFu), e4m3x2_to_f16x2(vs >> 16)};
        uint32_t w[4][D / 64];
        if constexpr (D == 128) {
            const uint4 v0 = *reinterpret_cast<const uint4 *>(c), v1 = *reinterpret_cast<const uint4 *>(c + 16);
            w[0][0] = v0.x, w[0][1] = v0.y, w[1][0] = v0.z, w[1][1] = v0.w;
            w[2][0] = v1.x, w[2][1] = v1.y, w[3][0] = v1.z, w[3][1] = v1.w;
        } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x][0] = *reinterpret_cast<const uint32_t *>(c + 8 * x + 4 * (g & 1));
        }
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            // two keys' codes of an element side by side in a byte: a pair of
            // FP16 along the keys, as the operand wants it, after one conversion
            uint32_t a[2][2][4];  // [keys 0, 1 | keys 2, 3][even | odd element]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = w[2 * h][j], y = w[2 * h + 1][j];
                e2m1x8_to_f16((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), a[h][0]);
                e2m1x8_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), a[h][1]);
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    a[h][0][z] = f16x2_mul(a[h][0][z], sc[h]);
                    a[h][1][z] = f16x2_mul(a[h][1][z], sc[h]);
                }
            }
#pragma unroll
            for (int z = 0; z < 4; ++z)
                mma16816(U.o[4 * j + z], a[0][0][z], a[0][1][z], a[1][0][z], a[1][1][z], pb[i][0], pb[i][1]);
        }
    }
}

// Four elements of a finished row.
template <int D>
__device__ __forceinline__ void split_store(const AttnParams &P, const SplitPos &at, int col, int d, float4 o, float m,
                                            float l) {
    const df11_kv4_attention_args &A = P.a;
    const int row = at.tile * kSplitCols + col, group = static_cast<int>(P.group);
    if (row >= at.q.rows) return;
    const int64_t token = at.q.q0 + row / group;
    const int hq = at.head * group + row % group;
    const float s = l > 0.0f ? P.v_scale / l : 0.0f;
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * s, o.y * s), b = __floats2bfloat162_rn(o.z * s, o.w * s);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t *>(&a);
    w.y = *reinterpret_cast<const uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(A.o) + token * static_cast<int64_t>(A.o_token_stride) + hq * D + d) =
        w;
    if (A.lse && d == 0)
        A.lse[token * A.n_q_heads + hq] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Persistent CTAs, each a contiguous, equal share of the launch's chunks
// (request, unit, chunk in order), so a long request spreads over the GPU and
// short ones share a CTA, whatever the mix.  A share's chunks go to the warps
// in turn; each warp keeps a ring of stages that its own bulk copies fill, two
// chunks ahead and across unit ends.  At the end of a unit (or of the share)
// the warps' results are joined in shared memory; a unit that spans CTAs goes
// through the workspace, and the CTA that arrives last joins its parts in
// order: no CTA waits for another, and the result does not depend on which
// one was last.
template <int D>
__global__ void __launch_bounds__(kSplitThreads, 1) attention_split_kernel(const AttnParams P) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    SplitShared<D> &S = *reinterpret_cast<SplitShared<D> *>(smem_raw);
    const df11_kv4_attention_args &A = P.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t err = 0;
    if (lane == 0)
        for (int i = 0; i < kSplitStages; ++i) mbar_init(&S.full[warp][i], 1);
    fence_mbar_init();

    // ---- the launch's chunks, and the request in which this CTA's share starts
    auto weight = [&](int r) -> int64_t {
        if (r >= A.n_reqs) return 0;
        const SplitReq q = split_req(P, r);
        return static_cast<int64_t>(q.units) * q.chunks;
    };
    const bool one = A.n_reqs <= kSplitThreads;
    int64_t mine = 0;
    for (int r = tid; r < A.n_reqs; r += kSplitThreads) mine += weight(r);
    if (blockIdx.x == 0)
        for (int r = tid; r < A.n_reqs; r += kSplitThreads) {
            if (!rows_valid(A, __ldg(A.q_start + r), __ldg(A.q_start + r + 1))) err |= DF11_DEV_ERR_AUX;
            if (static_cast<int64_t>(__ldg(A.kv_lens + r)) > static_cast<int64_t>(A.max_pages) << P.page_shift)
                err |= DF11_DEV_ERR_PAGES;
        }
    auto block_scan = [&](int64_t v, int64_t &all) -> int64_t {  // exclusive
        int64_t incl = v;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, x);
            if (lane >= x) incl += o;
        }
        __syncthreads();
        if (lane == 31) S.sums[warp] = incl;
        __syncthreads();
        int64_t before = 0;
        all = 0;
        for (int w = 0; w < kSplitWarps; ++w) {
            if (w < warp) before += S.sums[w];
            all += S.sums[w];
        }
        return before + incl - v;
    };
    int64_t total, at0 = block_scan(mine, total);
    // no share is empty: a unit's parts are then those of every CTA from its first to its last
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
    if (blockIdx.x >= ctas) {
        report(P.err, err);
        return;
    }
    const int64_t x0 = total * blockIdx.x / ctas, x1 = total * (blockIdx.x + 1) / ctas;
    if (one) {
        if (mine && at0 <= x0 && x0 < at0 + mine) {
            S.start_req = tid;
            S.start_off = x0 - at0;
        }
    } else {
        int64_t base = 0;
        for (int b = 0; b < A.n_reqs && base <= x0; b += kSplitThreads) {
            const int64_t v = weight(b + tid);
            int64_t all;
            const int64_t at = base + block_scan(v, all);
            if (v && at <= x0 && x0 < at + v) {
                S.start_req = b + tid;
                S.start_off = x0 - at;
            }
            base += all;
        }
    }
    __syncthreads();
    SplitPos seg;  // the unit being computed, at the share's first chunk of it
    seg.r = S.start_req;
    seg.q = split_req(P, seg.r);
    const int unit = static_cast<int>(S.start_off / seg.q.chunks);
    seg.head = unit / seg.q.tiles;
    seg.tile = unit % seg.q.tiles;
    seg.c = static_cast<int>(S.start_off % seg.q.chunks);
    // the copies run ahead of the computation on their own position
    SplitPos ahead = seg;
    int64_t ax = x0 + warp, cx = x0 + warp;  // this warp's next chunk to copy, to compute
    uint32_t have[kSplitStages];
    uint32_t issued = 0, used = 0;
    int64_t id = kNoPage;
    if (ax < x1) {
        ahead.advance(P, warp);
        id = split_page(P, ahead, lane);
    }
    auto issue = [&]() {
        const uint32_t st = issued % kSplitStages;
        const uint32_t got = split_issue<D>(P, ahead, id, lane, S.ring[warp][st], &S.full[warp][st], err);
#pragma unroll
        for (int i = 0; i < kSplitStages; ++i)
            if (st == static_cast<uint32_t>(i)) have[i] = got;
        ++issued;
        ax += kSplitWarps;
        if (ax < x1) {
            ahead.advance(P, kSplitWarps);
            id = split_page(P, ahead, lane);
        }
    };
    for (int i = 0; i < kSplitStages; ++i)
        if (ax < x1) issue();

    int64_t x = x0;
    bool dead = false;
    SplitUnit<D> U;
    while (x < x1) {
        const int n = static_cast<int>(min(static_cast<int64_t>(seg.q.chunks - seg.c), x1 - x));  // the share's chunks of this unit
        const bool whole_unit = n == seg.q.chunks;
        // the warp's own chunks of it
        const bool mine_any = cx < x + n;
        if (mine_any) {
            split_load_unit<D>(P, seg, lane, U);
            for (; cx < x + n; cx += kSplitWarps) {
                const uint32_t st = used % kSplitStages;
                uint32_t pages = have[0];
#pragma unroll
                for (int i = 1; i < kSplitStages; ++i)
                    if (st == static_cast<uint32_t>(i)) pages = have[i];
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&S.full[warp][st], used / kSplitStages & 1u, dead ? 0 : P.wait_ns))) {
                    err |= DF11_DEV_ERR_TIMEOUT;
                    dead = true;
                    pages = 0;
                }
                ++used;
                split_chunk<D>(P, S.ring[warp][st], (seg.q.c_lo + seg.c + (cx - x)) * static_cast<int64_t>(kSplitKeys), pages, lane, U);
                __syncwarp();
                if (ax < x1 && !dead) {
                    if (lane < 16) fence_proxy_async_smem();
                    __syncwarp();
                    issue();
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) U.l[c] += __shfl_xor_sync(0xFFFFFFFFu, U.l[c], y);
        }
        // ---- join: the warps' results in shared memory
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (g == 0) {
                S.m[warp][2 * t + c] = mine_any ? U.m[c] : -INFINITY;
                S.l[warp][2 * t + c] = mine_any ? U.l[c] : 0.0f;
            }
            if (mine_any) {
                float *o = &S.o[warp][2 * t + c][g * (D / 8)];
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
                    *reinterpret_cast<float4 *>(o + 2 * i) =
                        make_float4(U.o[i][c], U.o[i][2 + c], U.o[i + 1][c], U.o[i + 1][2 + c]);
            }
        }
        __syncthreads();
        // parts of a unit that spans CTAs: CTAs first_cta .. last_cta, each one part
        const int64_t u0 = x - seg.c, u1 = u0 + seg.q.chunks;
        auto owner = [&](int64_t y) { return static_cast<int>(((y + 1) * ctas + total - 1) / total - 1); };
        const int first_cta = whole_unit ? 0 : owner(u0), last_cta = whole_unit ? 0 : owner(u1 - 1);
        // a CTA has at most two parts: of the unit that its share starts inside (0), and of the one it ends inside (1)
        auto part = [&](int cta) {
            return static_cast<float *>(A.workspace) + P.ws_parts +
                   (2ull * cta + (cta == first_cta ? 1 : 0)) * split_partial_floats<D>();
        };
        for (int it = tid; it < kSplitCols * D / 4; it += kSplitThreads) {
            const int col = it / (D / 4), d = it % (D / 4) * 4;
            float m = -INFINITY, l = 0.0f;
            for (int w = 0; w < kSplitWarps; ++w) m = fmaxf(m, S.m[w][col]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < kSplitWarps; ++w) {
                if (S.m[w][col] == -INFINITY) continue;
                const float f = ex2(S.m[w][col] - m);
                const float4 v = *reinterpret_cast<const float4 *>(&S.o[w][col][d]);
                o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
                l += f * S.l[w][col];
            }
            if (whole_unit) {
                split_store<D>(P, seg, col, d, o, m, l);
            } else {
                float *p = part(blockIdx.x);
                __stcg(reinterpret_cast<float4 *>(p + col * D + d), o);
                if (d == 0) {
                    __stcg(p + kSplitCols * D + col, m);
                    __stcg(p + kSplitCols * D + kSplitCols + col, l);
                }
            }
        }
        if (!whole_unit) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                int *counter = static_cast<int *>(A.workspace) + first_cta;
                S.last = atomicAdd(counter, 1) == last_cta - first_cta;
                if (S.last) *counter = 0;
            }
            __syncthreads();
            if (S.last) {
                __threadfence();
                for (int it = tid; it < kSplitCols * D / 4; it += kSplitThreads) {
                    const int col = it / (D / 4), d = it % (D / 4) * 4;
                    float m = -INFINITY, l = 0.0f;
#pragma unroll 4
                    for (int c = first_cta; c <= last_cta; ++c)
                        m = fmaxf(m, __ldcg(part(c) + kSplitCols * D + col));
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int c = first_cta; c <= last_cta; ++c) {
                        const float *p = part(c);
                        const float mc = __ldcg(p + kSplitCols * D + col);
                        const float lc = __ldcg(p + kSplitCols * D + kSplitCols + col);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + col * D + d));
                        const float f = mc == -INFINITY ? 0.0f : ex2(mc - m);
                        o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
                        l += f * lc;
                    }
                    split_store<D>(P, seg, col, d, o, m, l);
                }
            }
        }
        x += n;
        if (x < x1) seg.advance(P, n);
        __syncthreads();
    }
    // after a timeout: the copies still out must land before the memory is given up
    for (; dead && used < issued; ++used) mbar_wait(&S.full[warp][used % kSplitStages], used / kSplitStages & 1u, P.wait_ns);
    report(P.err, __reduce_or_sync(0xFFFFFFFFu, err) * (lane == 0));
}

// A warp per row and query head, 4 warps of a CTA splitting the row's keys; a
// lane holds D / 32 elements.
template <int D>
__global__ void __launch_bounds__(128) attention_rows_kernel(const AttnParams P) {
    constexpr int E = D / 32;
    __shared__ float s_m[4], s_l[4], s_o[4][D];
    const df11_kv4_attention_args &A = P.a;
    const int t = blockIdx.x, hq = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t h = hq / P.group;
    uint32_t bad = 0;
    // the last request that starts at or before row t
    int lo = 0, hi = A.n_reqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (A.q_start[mid] <= t ? lo : hi) = mid;
    }
    const int q0 = A.q_start[lo], q1 = A.q_start[lo + 1];
    if (t < q0 || t >= q1) return;
    if (!rows_valid(A, q0, q1) || static_cast<int64_t>(q1 - q0) * P.group <= kSplitMaxRows) return;
    int64_t kv = max(A.kv_lens[lo], 0);
    const int64_t cap = static_cast<int64_t>(A.max_pages) << P.page_shift;
    const int64_t pos = kv - (q1 - q0) + (t - q0);
    int64_t j0 = 0, j1 = A.causal ? min(pos + 1, kv) : kv;
    if (A.window) j0 = max(j0, pos + 1 - A.window);
    j1 = min(j1, cap);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
    const __nv_bfloat16 *qp =
        static_cast<const __nv_bfloat16 *>(A.q) + t * static_cast<int64_t>(A.q_token_stride) + hq * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] = __bfloat162float(qp[i]) * A.scale * P.k_scale, o[i] = 0.0f;
    for (int64_t j = j0 + warp; j < j1; j += 4) {
        const int32_t id = A.block_table[static_cast<int64_t>(lo) * A.max_pages + (j >> P.page_shift)];
        if (id < 0 || static_cast<uint64_t>(id) >= P.n_pages) {
            bad |= DF11_DEV_ERR_PAGES;
            continue;
        }
        const uint8_t *blk = P.pages + (static_cast<uint64_t>(id) * P.kv_heads + h) * P.block.bytes;
        const uint32_t off = static_cast<uint32_t>(j) & ((1u << P.page_shift) - 1u), b = lane * E / 16;
        // the lane's E codes in the low bits of the aligned word that holds them
        const uint32_t byte = lane * (E / 2), sh = 8 * (byte & 3u);
        const uint32_t kw =
            *reinterpret_cast<const uint32_t *>(blk + P.block.k_codes + off * (D / 2) + (byte & ~3u)) >> sh;
        const uint32_t vw = *reinterpret_cast<const uint32_t *>(blk + P.block.v_codes +
                                                                (((off >> 2) * (D / 16) + b) * 4u + (off & 3u)) * 8u +
                                                                (byte & 4u)) >> sh;
        const uint32_t ks = e4m3x2_to_f16x2(blk[P.block.k_scales + off * (D / 16) + b] * 0x0101u);
        const uint32_t vs = e4m3x2_to_f16x2(blk[P.block.v_scales + (b << P.page_shift) + off] * 0x0101u);
        uint32_t kr[4], vr[4];
        e2m1x8_to_f16(kw, kr);
        e2m1x8_to_f16(vw, vr);
        float s = 0.0f, v[E];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            float a, c;
            f16x2_to_f32(f16x2_mul(kr[i], ks), a, c);
            s += q[2 * i] * a + q[2 * i + 1] * c;
            f16x2_to_f32(f16x2_mul(vr[i], vs), v[2 * i], v[2 * i + 1]);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
        const float mn = fmaxf(m, s), c = __expf(m - mn), p = __expf(s - mn);
        m = mn;
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * c + p * v[i];
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i];
    __syncthreads();
    if (bad && P.err) atomicOr(P.err, static_cast<int>(bad));
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_m[w]);
    for (int w = 0; w < 4; ++w) ll += s_l[w] > 0.0f ? s_l[w] * __expf(s_m[w] - mm) : 0.0f;
    for (int d = threadIdx.x; d < D; d += 128) {
        float y = 0.0f;
        for (int w = 0; w < 4; ++w) y += s_l[w] > 0.0f ? s_o[w][d] * __expf(s_m[w] - mm) : 0.0f;
        static_cast<__nv_bfloat16 *>(A.o)[t * static_cast<int64_t>(A.o_token_stride) + hq * D + d] =
            __float2bfloat16_rn(ll > 0.0f ? y / ll * P.v_scale : 0.0f);
    }
    if (A.lse && threadIdx.x == 0)
        A.lse[static_cast<int64_t>(t) * A.n_q_heads + hq] = ll > 0.0f ? mm + logf(ll) : -INFINITY;
}

// A multiprocessor each for the persistent CTAs; the workspace has room for kMaxCtas.
constexpr int kMaxCtas = 256;

AttnParams attn_params(const df11_kv4_cache &c, const df11_kv4_attention_args &a, int *err) {
    AttnParams P{};
    P.pages = static_cast<const uint8_t *>(c.pages);
    P.n_pages = c.n_pages;
    P.kv_heads = static_cast<uint32_t>(c.n_heads);
    P.group = static_cast<uint32_t>(a.n_q_heads / c.n_heads);
    while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
    P.block = kv4_block(c.page_size, c.head_dim);
    P.k_scale = c.k_scale;
    P.v_scale = c.v_scale;
    P.a = a;
    P.err = err;
    P.wait_ns = 2000000000ull;
    P.ws_parts = kMaxCtas;
    return P;
}

bool prepare(int *sms) {
    constexpr int kDevices = 64;
    static std::mutex mu;
    static int known[kDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    std::lock_guard<std::mutex> lk(mu);
    if (!known[dev]) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
        if (cudaFuncSetAttribute(reinterpret_cast<const void *>(&attention_split_kernel<64>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SplitShared<64>)) != cudaSuccess ||
            cudaFuncSetAttribute(reinterpret_cast<const void *>(&attention_split_kernel<128>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(SplitShared<128>)) != cudaSuccess)
            return false;
        known[dev] = v;
    }
    *sms = known[dev] < kMaxCtas ? known[dev] : kMaxCtas;
    return true;
}

}  // namespace

LaunchStatus kv4_attention_workspace(const df11_kv4_cache &c, const df11_kv4_attention_args &, uint64_t *bytes) {
    const uint64_t part = c.head_dim == 128 ? split_partial_floats<128>() : split_partial_floats<64>();
    *bytes = 4 * (kMaxCtas + 2 * kMaxCtas * part);
    return LaunchStatus::kOk;
}

LaunchStatus launch_kv4_attention(const df11_kv4_cache &c, const df11_kv4_attention_args &a, int *err,
                                  cudaStream_t s) {
    const AttnParams P = attn_params(c, a, err);
    int sms = 0;
    if (!prepare(&sms)) return LaunchStatus::kCuda;
    if (c.head_dim == 128) attention_split_kernel<128><<<sms, kSplitThreads, sizeof(SplitShared<128>), s>>>(P);
    else attention_split_kernel<64><<<sms, kSplitThreads, sizeof(SplitShared<64>), s>>>(P);
    if (static_cast<int64_t>(a.max_q_len) * P.group > kSplitMaxRows) {
        const dim3 grid(a.n_tokens, a.n_q_heads);
        if (c.head_dim == 128) attention_rows_kernel<128><<<grid, 128, 0, s>>>(P);
        else attention_rows_kernel<64><<<grid, 128, 0, s>>>(P);
    }
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

}  // namespace df11
