// kv4_attention.cu -- attention over the paged 4-bit key/value cache, the
// cache decoded on chip.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "df11.h"
#include "kv4.cuh"
#include "packed.cuh"
#include "serve.h"
#include "tcgen05.cuh"
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
    int32_t split_rows; // a request's rows that the few-row kernel takes at most
    int32_t parts;      // CTAs that share the keys of a pair of tiles (many rows)
    bool early;         // the many-row kernel may start before the few-row one has ended
    uint32_t ws_parts, ws_warps;  // workspace, in floats: counters, then the CTAs' partial results, then the warps'
};

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
// 64 requests of 256 to 16384 keys (8 cache heads of 128, groups of 4, 651 MB)
// take 148 us, 4.4 TB/s; two of 98301 to 131072 keys 64 us.  Bound by instructions
// at 3 warps a scheduler: 1170 for a chunk with its part of the unit, of which
// 256 are conversions, 256 products with the scales and 64 MMAs; copies alone
// took 118 us.
constexpr int kSplitWarps = 12;
constexpr int kSplitThreads = 32 * kSplitWarps;
constexpr int kSplitCols = 8;      // rows of a unit
constexpr int kSplitKeys = 64;     // keys of a chunk: a warp's step
constexpr int kSplitStages = 2;    // chunks that a warp has room for
// Rows (tokens x heads of a group) of a request that go this way at most: the
// time goes with them in steps of 8, since each 8 rows decode the keys again,
// the other kernel's hardly.  32 requests on 2000 keys of 8 heads of 128 take 77
// us with 32 rows each, 110 with 48 and 138 with 64, the other kernel 91; one
// request alone 15 to 17 us with 32 to 64 rows, the other kernel 23 (on 8000
// keys: 21 to 28, and 34).
constexpr int kSplitRows = 32, kSplitRowsFew = 64;
constexpr int kSplitFew = 16;  // requests times cache heads, at most, with the second bound
// What a unit costs a CTA beside its chunks (queries, joins), in chunks: shares
// are equal in this measure, in which a unit starts with so many empty places.
// With 4, 8 and 16, 64 requests of 256 to 16384 keys (8 cache heads of 128,
// groups of 4) take 147, 146 and 149 us, 2 of 98301 to 131072 keys 66, 65 and 64,
// one of 12000 17, 16 and 16, and 8 of 1000 16, 15 and 14.
constexpr int kSplitUnitCost = 16;
constexpr int32_t kMaxKeys = INT32_MAX - 255;

// A partial result in the workspace: unnormalised O (8 x D), then m and l.
template <int D>
__host__ __device__ constexpr uint32_t split_partial_floats() {
    return kSplitCols * D + 2 * kSplitCols;
}

// The many-row kernel may start while the few-row one, launched before it, still
// runs: neither reads what the other writes.  The few-row kernel lets it, and
// its first CTA waits for that one's end, so what follows in the stream follows
// both.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The part of a request that this path handles: chunks [c_lo, c_lo + chunks)
// of its keys for each of `units` (cache head, tile of 8 rows) pairs.  A
// request that sees no key still has one chunk, which writes its zeros.
struct SplitReq {
    int32_t q0, n, rows, tiles, units, c_lo, chunks;
    int32_t kv, begin, end;  // keys; the first that any row sees; the last + 1 that the table holds
};

__device__ __forceinline__ bool rows_valid(const df11_kv4_attention_args &A, int q0, int q1) {
    return q0 >= 0 && q1 >= q0 && q1 <= A.n_tokens && q1 - q0 <= A.max_q_len;
}

// Keys that a request's block-table row has room for.
__device__ __forceinline__ int32_t key_room(const AttnParams &P) {
    return static_cast<int32_t>(min(static_cast<int64_t>(P.a.max_pages) << P.page_shift, static_cast<int64_t>(kMaxKeys)));
}

// First key of the window of the row at position `pos`, which is negative for
// rows before the first key: the widest window's differences would pass 32 bits there.
__device__ __forceinline__ int32_t window_start(int32_t pos, int32_t window) { return pos >= window ? pos + 1 - window : 0; }

__device__ __forceinline__ SplitReq split_req(const AttnParams &P, int r) {
    const df11_kv4_attention_args &A = P.a;
    SplitReq q{};
    q.q0 = __ldg(A.q_start + r);
    const int q1 = __ldg(A.q_start + r + 1);
    if (!rows_valid(A, q.q0, q1)) return q;
    q.n = q1 - q.q0;
    const int64_t rows = static_cast<int64_t>(q.n) * P.group;
    if (rows == 0 || rows > P.split_rows) return q;
    q.rows = static_cast<int32_t>(rows);
    q.tiles = (q.rows + kSplitCols - 1) / kSplitCols;
    q.kv = min(max(__ldg(A.kv_lens + r), 0), kMaxKeys);
    q.end = min(q.kv, key_room(P));
    q.begin = A.window ? min(window_start(q.kv - q.n, A.window), q.end) : 0;
    q.c_lo = q.begin / kSplitKeys;
    q.chunks = max((q.end + kSplitKeys - 1) / kSplitKeys - q.c_lo, 1);
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
    __device__ __forceinline__ int key0() const { return (q.c_lo + c) * kSplitKeys; }
};

// Keys that every row of a unit sees [all_lo, all_hi), and that any does [any_lo, any_hi).
struct SplitSeen {
    int all_lo, all_hi, any_lo, any_hi;
};

__device__ __forceinline__ SplitSeen split_seen(const AttnParams &P, const SplitPos &at) {
    const int group = static_cast<int>(P.group), base = at.q.kv - at.q.n;
    const int p0 = base + at.tile * kSplitCols / group;  // rows ascend
    const int p1 = base + (min((at.tile + 1) * kSplitCols, at.q.rows) - 1) / group;
    SplitSeen s;
    s.all_hi = P.a.causal ? min(p0 + 1, at.q.end) : at.q.end;
    s.any_hi = P.a.causal ? min(p1 + 1, at.q.end) : at.q.end;
    s.all_lo = P.a.window ? window_start(p1, P.a.window) : 0;
    s.any_lo = P.a.window ? window_start(p0, P.a.window) : 0;
    return s;
}

template <int D>
struct SplitShared {
    static constexpr uint32_t kStage = kSplitKeys * D * 9 / 8;  // a chunk's K and V
    alignas(128) uint8_t ring[kSplitWarps][kSplitStages][kStage];
    alignas(8) uint64_t full[kSplitWarps][kSplitStages];
    SplitPos pos[kSplitWarps][kSplitStages];  // of the chunk in a stage
    SplitSeen seen[kSplitWarps];
    // A warp's results that others join: of the unit that its range starts
    // inside, if that ends in the range (0, in the workspace), and of the one
    // at its range's end (1, in shared memory); by the unit's first chunk, -1: none.
    int part_unit[kSplitWarps][2];
    SplitPos part_pos[kSplitWarps][2];
    int join_first[2], join_last[2], join[2];
    SplitPos join_pos[2];
    int joins[2];  // of those, the ones that this CTA's arrival completes
    int dead;  // a wait gave up: what the CTA has is not joined
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

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// log(sum exp) from a maximum in log2 units and the sum relative to it: -inf
// where no key was seen (l is 0), NaN where a score was.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a warp has of a unit: its queries as the B operand, and per column
// (the thread's are 2t and 2t + 1) the factor of the scores (log2 units), the
// token's position, the running maximum and sum, and O.
template <int D>
struct SplitUnit {
    uint32_t qb[D / 16][2];
    float f[2], m[2], l[2];
    int pos[2];  // key position of the column's token
    float o[D / 16][4];
};

// Loads the unit's queries: thread (g, t) takes elements [t D / 4, (t + 1) D /
// 4) of column g.  A column is scaled by a power of two that brings its
// largest element into [1, 2): FP16 holds it to 2^-25 of that one, which for
// BF16's 8 bits is without loss down to 2^-17 of it.
template <int D>
__device__ __forceinline__ void split_load_unit(const AttnParams &P, const SplitPos &at, int lane, SplitUnit<D> &U) {
    const df11_kv4_attention_args &A = P.a;
    const int g = lane >> 2, t = lane & 3, group = static_cast<int>(P.group);
    const int tile = at.tile, row = tile * kSplitCols + g;
    float x[D / 4];
    if (row < at.q.rows) {
        const uint4 *p = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(A.q) +
            static_cast<int64_t>(at.q.q0 + row / group) * static_cast<int64_t>(A.q_token_stride) +
            (at.head * group + row % group) * D + t * (D / 4));
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
    const int base = at.q.kv - at.q.n;  // the key position of the request's row 0
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = 2 * t + i, ec = __shfl_sync(0xFFFFFFFFu, e, 4 * col);
        U.f[i] = A.scale * P.k_scale * 1.44269504088896341f * __uint_as_float(static_cast<uint32_t>(ec + 127) << 23);
        U.m[i] = -INFINITY;
        U.l[i] = 0.0f;
        U.pos[i] = base + min(tile * kSplitCols + col, at.q.rows - 1) / group;
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

template <int ES>
__device__ __forceinline__ int64_t split_page(const AttnParams &P, const SplitPos &at, int lane) {
    const int key = at.key0() + (lane << ES), pg = key >> P.page_shift;
    if (lane >= (kSplitKeys >> ES) || key >= at.q.end || key + (1 << ES) <= at.q.begin) return kNoPage;
    return __ldg(P.a.block_table + static_cast<int64_t>(at.r) * P.a.max_pages + pg);
}

// Copies a chunk's pages, of the unit's head, into a stage, each as a block of 2^ES tokens.
template <int D, int ES>
__device__ __forceinline__ void split_issue(const AttnParams &P, const uint8_t *block, bool have, uint32_t mask, int half,
                                            int lane, uint8_t *dst, uint64_t *bar) {
    constexpr Kv4Block B = kv4_block(1u << ES, D);
    if (ES < 6 || P.page_shift == 6) {
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(mask) * B.bytes);
        __syncwarp();
        if (have) bulk_load(dst + lane * B.bytes, block, B.bytes, bar);
    } else {
        // half of a 128-token page: its rows of the row-ordered sections are
        // contiguous, the V scales are 64 bytes of each element block's 128
        if (lane == 0) mbar_arrive_expect_tx(bar, mask ? B.bytes : 0u);
        const uint8_t *s = reinterpret_cast<const uint8_t *>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(block), 0));
        constexpr uint32_t codes = B.k_scales, scales = B.v_codes - B.k_scales;
        if (mask) {
            if (lane == 0) bulk_load(dst, s + half * codes, codes, bar);
            if (lane == 1) bulk_load(dst + B.k_scales, s + P.block.k_scales + half * scales, scales, bar);
            if (lane == 2) bulk_load(dst + B.v_codes, s + P.block.v_codes + half * codes, codes, bar);
            if (lane >= 3 && lane < 3 + D / 16)
                bulk_load(dst + B.v_scales + (lane - 3) * 64, s + P.block.v_scales + (lane - 3) * 128 + half * 64, 64, bar);
        }
    }
}

// The scores of a chunk's 64 keys, in log2 units; what a row does not see is -inf.
template <int D, int ES>
__device__ __forceinline__ void split_scores(const AttnParams &P, const uint8_t *stage, int key0, uint32_t pages,
                                             bool whole, const SplitSeen &seen, int lane, const SplitUnit<D> &U,
                                             float (&s)[4][4]) {
    constexpr int KW = D / 32;  // words of a thread's K codes of one key
    constexpr Kv4Block B = kv4_block(1u << ES, D);
    const int g = lane >> 2, t = lane & 3;
    // rows g and g + 8 of a tile of 16 keys are keys kg and kg + 2, so that
    // the 4 slots of the second product that a thread holds are 4 consecutive keys
    const uint32_t kg = 4u * (static_cast<uint32_t>(g) >> 1) + (g & 1u);
    const uint8_t *codes = stage + kg * (D / 2) + t * (D / 8);
    const uint8_t *scales = stage + B.k_scales + kg * (D / 16) + (D == 128 ? 2 * t : t);
    // two tiles at a time, two accumulators each: four chains of MMAs that do
    // not wait for one another
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        float acc[2][2][4];
        uint32_t w[2][2][KW], sc[2][2][2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const uint32_t page = (16u * (i + z)) >> ES, off = (16u * (i + z)) & ((1u << ES) - 1u);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t *c = codes + page * B.bytes + (off + 2u * r) * (D / 2);
                const uint8_t *x = scales + page * B.bytes + (off + 2u * r) * (D / 16);
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(c);
                    w[z][r][0] = v.x, w[z][r][1] = v.y, w[z][r][2] = v.z, w[z][r][3] = v.w;
                    const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(x));
                    sc[z][r][0] = __byte_perm(two, 0, 0x1010);
                    sc[z][r][1] = __byte_perm(two, 0, 0x3232);
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(c);
                    w[z][r][0] = v.x, w[z][r][1] = v.y;
                    sc[z][r][0] = e4m3x2_to_f16x2(*x * 0x0101u);
                }
            }
#pragma unroll
            for (int y = 0; y < 8; ++y) acc[z][y / 4][y % 4] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < KW; ++j) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                uint32_t a[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    e2m1x8_to_f16(w[z][r][j], a[r]);
#pragma unroll
                    for (int x = 0; x < 4; ++x) a[r][x] = f16x2_mul(a[r][x], sc[z][r][j / 2]);
                }
                mma16816(acc[z][0], a[0][0], a[1][0], a[0][1], a[1][1], U.qb[2 * j][0], U.qb[2 * j][1]);
                mma16816(acc[z][1], a[0][2], a[1][2], a[0][3], a[1][3], U.qb[2 * j + 1][0], U.qb[2 * j + 1][1]);
            }
        }
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[i + z][x] = (acc[z][0][x] + acc[z][1][x]) * U.f[x & 1];
    }
    if (!whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t in = 16u * i + kg + (x & 2u);
                const int key = key0 + static_cast<int>(in);
                if (!(pages >> (in >> ES) & 1u) || key >= seen.any_hi || (P.a.causal && key > U.pos[x & 1]) ||
                    (P.a.window && U.pos[x & 1] - key >= P.a.window))
                    s[i][x] = -INFINITY;
            }
    }
}

// Softmax of the scores against the running maximum; the probabilities as the
// B operand of the second product.
template <int D>
__device__ __forceinline__ void split_softmax(float (&s)[4][4], SplitUnit<D> &U, uint32_t (&pb)[4][2]) {
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) top[x & 1] = fmaxf(top[x & 1], s[i][x]);
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
}

// O^T += V^T P^T over the chunk's keys.
template <int D, int ES>
__device__ __forceinline__ void split_values(const uint8_t *stage, int key0, uint32_t pages, bool whole,
                                             const SplitSeen &seen, int lane, SplitUnit<D> &U,
                                             const uint32_t (&pb)[4][2]) {
    constexpr Kv4Block B = kv4_block(1u << ES, D);
    const int g = lane >> 2, t = lane & 3;
    const int b = D == 128 ? g : g >> 1;  // the scale block of the thread's elements [g D / 8, (g + 1) D / 8)
    const uint8_t *codes = stage + B.v_codes + (t * (D / 16) + b) * 32;
    const uint8_t *scales = stage + B.v_scales + (b << ES) + 4 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t in = 16u * i, page = in >> ES, off = in & ((1u << ES) - 1u);
        const uint8_t *c = codes + page * B.bytes + (off >> 2) * (D / 16) * 32u;
        uint32_t vs = *reinterpret_cast<const uint32_t *>(scales + page * B.bytes + off);
        if (!whole) {
            // a key that no row sees may hold anything, NaN scales too: 0 times NaN must not reach a sum
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t k = in + 4 * t + x;
                const int key = key0 + static_cast<int>(k);
                if (!(pages >> (k >> ES) & 1u) || key < seen.any_lo || key >= seen.any_hi) vs &= ~(0xFFu << (8 * x));
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

// Elements [d, d + N) of a finished row.
template <int D, int N>
__device__ __forceinline__ void split_store(const AttnParams &P, const SplitPos &at, int col, int d, const float *o, float m,
                                            float l) {
    const df11_kv4_attention_args &A = P.a;
    const int row = at.tile * kSplitCols + col, group = static_cast<int>(P.group);
    if (row >= at.q.rows) return;
    const int64_t token = at.q.q0 + row / group;
    const int hq = at.head * group + row % group;
    const float s = l > 0.0f ? P.v_scale / l : l;  // 0 where no key was seen
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16x2_of(o[2 * i] * s, o[2 * i + 1] * s);
    uint16_t *p = static_cast<uint16_t *>(A.o) + token * static_cast<int64_t>(A.o_token_stride) + hq * D + d;
    if constexpr (N == 4) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; i += 4)
            *reinterpret_cast<uint4 *>(p + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
    if (A.lse && d == 0) A.lse[token * A.n_q_heads + hq] = lse_of(m, l);
}

// CTA b's share of the launch's places starts here: equal parts, the first total % ctas one longer.
struct SplitShares {
    int base, rem;
    __device__ __forceinline__ int start(int b) const { return b * base + min(b, rem); }
    // The CTA that has place y.
    __device__ __forceinline__ int owner(int y) const {
        const int longer = rem * (base + 1);
        return y < longer ? y / (base + 1) : rem + (y - longer) / base;
    }
};

// A place in the launch: its request and the unit there, the unit's chunks, the
// place's offset in it, and the chunks before the place.
struct SplitPlace {
    int at, r, unit, chunks, off, before;
};

// Finds N places, the last the greatest, with all lanes of a warp; a unit has
// COST empty places before those of its chunks.
template <int N, int COST>
__device__ __forceinline__ void split_find(const AttnParams &P, int lane, SplitPlace (&p)[N]) {
    int base = 0, units = 0;
    for (int b = 0; b < P.a.n_reqs && base <= p[N - 1].at; b += 32) {
        SplitReq q{};
        if (b + lane < P.a.n_reqs) q = split_req(P, b + lane);
        const int size = q.chunks + COST, w = q.units * size;
        int incl = w, uncl = q.units;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, incl, y), v = __shfl_up_sync(0xFFFFFFFFu, uncl, y);
            if (lane >= y) incl += o, uncl += v;
        }
        const int at = base + incl - w, before = units + uncl - q.units;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t holds = __ballot_sync(0xFFFFFFFFu, w && at <= p[i].at && p[i].at < at + w);
            if (!holds) continue;
            const int src = __ffs(holds) - 1, in = p[i].at - at, unit = size > 0 ? in / size : 0;
            p[i].r = b + src;
            p[i].unit = __shfl_sync(0xFFFFFFFFu, unit, src);
            p[i].off = __shfl_sync(0xFFFFFFFFu, in - unit * size, src);
            p[i].chunks = __shfl_sync(0xFFFFFFFFu, q.chunks, src);
            p[i].before = p[i].at - __shfl_sync(0xFFFFFFFFu, before + unit, src) * COST - min(p[i].off, COST);
        }
        base += __shfl_sync(0xFFFFFFFFu, incl, 31);
        units += __shfl_sync(0xFFFFFFFFu, uncl, 31);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (base <= p[i].at) {  // the end of the launch
            p[i].off = 0;
            p[i].before = base - units * COST;
        }
}

// A thread's part of a warp's result: columns 2t and 2t + 1, elements [g D / 8, (g + 1) D / 8).
template <int D>
__device__ __forceinline__ void split_put(float *at, int lane, const SplitUnit<D> &U) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float *o = at + (2 * t + c) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
            *reinterpret_cast<float4 *>(o + 2 * i) = make_float4(U.o[i][c], U.o[i][2 + c], U.o[i + 1][c], U.o[i + 1][2 + c]);
        if (g == 0) {
            at[kSplitCols * D + 2 * t + c] = U.m[c];
            at[kSplitCols * D + kSplitCols + 2 * t + c] = U.l[c];
        }
    }
}

// Column col, elements [d, d + 4) of partial results joined one after another.
template <int D>
struct SplitJoin {
    float m = -INFINITY, l = 0.0f, o[4] = {};
    template <int N>
    __device__ __forceinline__ void add(const float (&mb)[N], const float (&lb)[N], const float4 (&ob)[N]) {
        float top = m;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, mb[i]);
        const float sh = top == -INFINITY ? 0.0f : top, f = ex2(m - sh);
        m = top;
        l *= f, o[0] *= f, o[1] *= f, o[2] *= f, o[3] *= f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float h = ex2(mb[i] - sh);
            l += lb[i] * h;
            o[0] += ob[i].x * h, o[1] += ob[i].y * h, o[2] += ob[i].z * h, o[3] += ob[i].w * h;
        }
    }
};

// Whether units of at most `longest` chunks are not divided between CTAs, whose
// shares are of `share` places: units of a chunk a warp, and those that come to
// one or a few a CTA.  A join of CTAs takes 1 to 3 us, and the last CTA to finish
// has up to a unit more.  8 heads of 128, with the kernel built for whole and
// for divided units: one token on 500 keys 11.0 and 12.1 us, on 1000 12.5 and
// 12.5, on 2000 15.9 and 12.6; 8 tokens on 1000 keys each 13.4 and 15.3, on 3000
// 20.4 and 18.6; 32 on 2000 27.3 and 30.3; 100 on 1000 43.7 and 48.2, on 2000 66.8
// and 69.5, on 3000 92.4 and 90.4; 8 with 24 rows each on 8000 keys 74 and 57.  With
// the rule in it the kernel takes the better side's time, up to 0.9 us more (one
// token on 1000 keys: 13.3).
__device__ __forceinline__ bool split_whole(int longest, int share) {
    return longest <= kSplitWarps || (longest <= 4 * kSplitWarps && longest <= share + share / 4 && share <= 320);
}

// Persistent CTAs, each a contiguous, equal share of the launch's chunks
// (request, unit, chunk in order), so a long request spreads over the GPU and
// short ones share a CTA, whatever the mix; each warp a contiguous part of its
// CTA's share.  The warps run on their own, each with a ring of two chunks that
// its own copies fill, across unit ends.  (With a chunk to each warp in turn,
// every unit was joined from 12 results: 156 us instead of 148, and 100 requests
// of 500 keys 35 instead of 29.)  A unit that lies in a warp's range is
// finished there; of others the warp leaves its part, and the CTA joins the
// parts of each unit at the end.  A unit that spans CTAs goes through the
// workspace, and the CTA that arrives last joins its parts, in order: no warp or
// CTA waits for another, and the result does not depend on which one was last.
// Where units are short (split_whole), a unit goes whole to the CTA whose
// share holds its first chunk: fewer CTAs work, but none joins.
template <int D, int ES>
__global__ void __launch_bounds__(kSplitThreads, 1) attention_split_kernel(const AttnParams P) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    SplitShared<D> &S = *reinterpret_cast<SplitShared<D> *>(smem_raw);
    const df11_kv4_attention_args &A = P.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t err = 0;
    if (P.early) grid_release();
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kSplitStages; ++i) mbar_init(&S.full[warp][i], 1);
        fence_mbar_init();
        S.part_unit[warp][0] = S.part_unit[warp][1] = -1;
        if (warp < 2) S.join[warp] = 0;
        if (warp == 0) S.dead = 0;
    }

    // ---- the launch's places (the host has seen that they fit 31 bits);
    // every warp counts them by itself, so none waits
    int total = 0, longest = 0;
    for (int r = lane; r < A.n_reqs; r += 32) {
        const SplitReq q = split_req(P, r);
        total += q.units * (q.chunks + kSplitUnitCost);
        if (q.units) longest = max(longest, q.chunks);
        if (blockIdx.x == 0 && warp == 0) {
            if (!rows_valid(A, __ldg(A.q_start + r), __ldg(A.q_start + r + 1))) err |= DF11_DEV_ERR_AUX;
            if (__ldg(A.kv_lens + r) > key_room(P)) err |= DF11_DEV_ERR_PAGES;
        }
    }
    total = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(total)));
    const int ctas = min(static_cast<int>(gridDim.x), total);
    const bool aligned = split_whole(__reduce_max_sync(0xFFFFFFFFu, longest), total / max(ctas, 1));
    __syncthreads();
    if (static_cast<int>(blockIdx.x) >= ctas) {
        report(P.err, err);
        return;
    }
    // ---- the CTA's share: no share of places is empty, and a unit's chunks follow one
    // another, so its parts are those of every CTA from its first chunk's to its last's
    const SplitShares shares{total / ctas, total % ctas};
    SplitPlace ends[2];
    ends[0].at = shares.start(blockIdx.x);
    ends[1].at = shares.start(blockIdx.x + 1);
    split_find<2, kSplitUnitCost>(P, lane, ends);
    // first places of the units that the ends lie in
    const int unit0 = ends[0].at - ends[0].off, unit1 = ends[1].at - ends[1].off;
    if (aligned) {
        // both ends move to the next unit's start
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (ends[i].off) ends[i].before += ends[i].chunks - max(ends[i].off - kSplitUnitCost, 0);
    }
    // chunks [x0, x1) of the launch, and this warp's of them
    const int x0 = ends[0].before, x1 = ends[1].before, per = (x1 - x0) / kSplitWarps, more = (x1 - x0) % kSplitWarps;
    if (x0 >= x1) {
        report(P.err, err);
        return;
    }
    const int w0 = x0 + warp * per + min(warp, more), share = per + (warp < more);

    // ---- this warp's copies, up to two chunks ahead of its computation
    SplitPos ahead;  // of its next chunk to copy
    if (share) {
        // in the share's first request, if it has so many chunks, else looked for
        ahead.r = ends[0].r;
        ahead.q = split_req(P, ahead.r);
        const int skip = aligned && ends[0].off ? ahead.q.chunks : max(ends[0].off - kSplitUnitCost, 0);
        int at = ends[0].unit * ahead.q.chunks + skip + (w0 - x0);
        if (at >= ahead.q.units * ahead.q.chunks) {
            SplitPlace start[1];
            start[0].at = w0;
            split_find<1, 0>(P, lane, start);
            ahead.r = start[0].r;
            ahead.q = split_req(P, ahead.r);
            at = start[0].unit * ahead.q.chunks + start[0].off;
        }
        const int unit = at / ahead.q.chunks;
        ahead.head = unit / ahead.q.tiles;
        ahead.tile = unit % ahead.q.tiles;
        ahead.c = at - unit * ahead.q.chunks;
    }
    int copied = 0;
    uint32_t pages[kSplitStages] = {};
    int64_t id = kNoPage;
    if (share) id = split_page<ES>(P, ahead, lane);
    // copies the chunk at `ahead` into stage st and moves on to the one after
    auto issue = [&](int st) {
        if (lane == 0) S.pos[warp][st] = ahead;
        const bool have = id >= 0 && static_cast<uint64_t>(id) < P.n_pages;
        if (!have && id != kNoPage) err |= DF11_DEV_ERR_PAGES;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, have);
        const uint8_t *block = P.pages + (static_cast<uint64_t>(have ? id : 0) * P.kv_heads +
                                          static_cast<uint32_t>(ahead.head)) * P.block.bytes;
        split_issue<D, ES>(P, block, have, mask, (ahead.q.c_lo + ahead.c) & 1, lane, S.ring[warp][st], &S.full[warp][st]);
        if (st) pages[1] = mask;
        else pages[0] = mask;
        if (++copied < share) {
            ahead.advance(P, 1);
            id = split_page<ES>(P, ahead, lane);
        }
    };
#pragma unroll 1
    for (int i = 0; i < kSplitStages && i < share; ++i) issue(i);

    const int g = lane >> 2, t = lane & 3;
    SplitUnit<D> U;
    bool dead = false;  // a wait gave up: no more copies
    for (int cx = 0, st = 0, parity = 0, s0 = 0; cx < share; ++cx) {
        const SplitPos &at = S.pos[warp][st];
        __syncwarp();
        if (cx == 0 || at.c == 0) {
            s0 = cx;
            if (lane == 0) S.seen[warp] = split_seen(P, at);
            split_load_unit<D>(P, at, lane, U);
            __syncwarp();
        }
        const int key0 = at.key0();
        const SplitSeen &seen = S.seen[warp];
        const uint8_t *stage = S.ring[warp][st];
        uint32_t there = st ? pages[1] : pages[0];
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&S.full[warp][st], parity, P.wait_ns))) {
            err |= DF11_DEV_ERR_TIMEOUT;
            dead = true;
            there = 0;
            if (lane == 0) atomicExch(&S.dead, 1);
            mbar_wait(&S.full[warp][st], parity, P.wait_ns);  // the memory is not given up with a copy on its way
        }
        const bool whole = there == (1u << (kSplitKeys >> ES)) - 1u && key0 >= seen.all_lo && key0 + kSplitKeys <= seen.all_hi;
        float s[4][4];
        split_scores<D, ES>(P, stage, key0, there, whole, seen, lane, U, s);
        uint32_t pb[4][2];
        split_softmax<D>(s, U, pb);
        split_values<D, ES>(stage, key0, there, whole, seen, lane, U, pb);
        __syncwarp();
        const bool ends_unit = at.c + 1 == at.q.chunks;
        if (ends_unit || cx + 1 == share) {
            // ---- the end of the unit, or of the range in it
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) U.l[c] += __shfl_xor_sync(0xFFFFFFFFu, U.l[c], y);
            if (ends_unit && cx - s0 == at.c) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float o[D / 8];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) o[2 * i] = U.o[i][c], o[2 * i + 1] = U.o[i][2 + c];
                    split_store<D, D / 8>(P, at, 2 * t + c, g * (D / 8), o, U.m[c], U.l[c]);
                }
            } else {
                const int last = cx + 1 == share;
                if (lane == 0) {
                    S.part_unit[warp][last] = w0 + cx - at.c;
                    S.part_pos[warp][last] = at;
                }
                if (!last)
                    split_put<D>(static_cast<float *>(A.workspace) + P.ws_warps +
                                     static_cast<uint64_t>(blockIdx.x * kSplitWarps + warp) * split_partial_floats<D>(),
                                 lane, U);
            }
        }
        if (dead) {
            // the rest of the range is given up, but for the copy that may still be out
            if (copied > cx + 1) mbar_wait(&S.full[warp][st ^ 1], parity ^ st, P.wait_ns);
            break;
        }
        if (copied < share) {
            __syncwarp();  // every lane has read `at`, which the next chunk's position replaces
            fence_proxy_async_smem();
            issue(st);
        }
        st ^= 1;
        if (!st) parity ^= 1;
    }

    // ---- the units that warps have left parts of, a column to a warp at a time
    __syncthreads();
    if (S.dead) {
        report(P.err, __reduce_or_sync(0xFFFFFFFFu, err) * (lane == 0));
        return;
    }
    float *results = reinterpret_cast<float *>(&S.ring[0][0][0]);
    constexpr int kPart = split_partial_floats<D>();
    static_assert(kPart * 4 <= static_cast<int>(SplitShared<D>::kStage * kSplitStages), "results fit the rings");
    if (S.part_unit[warp][1] >= 0) split_put<D>(results + warp * kPart, lane, U);
    __syncthreads();
    const float *early = static_cast<const float *>(A.workspace) + P.ws_warps +
                         static_cast<uint64_t>(blockIdx.x) * kSplitWarps * kPart;
    // a CTA's parts: of the unit that its share starts inside (0), and of the one that goes on in the next CTA's (1)
    auto cta_part = [&](int cta, int first) {
        return static_cast<float *>(A.workspace) + P.ws_parts + (2ull * cta + (cta == first ? 1 : 0)) * kPart;
    };
    // the warps whose part at the range's end is the first of its unit, and
    // above them, if the first warp has one, its early part, which is alone
    uint32_t units;
    {
        const int u = lane < kSplitWarps ? S.part_unit[lane][1] : -1, before = __shfl_up_sync(0xFFFFFFFFu, u, 1);
        units = __ballot_sync(0xFFFFFFFFu, u >= 0 && (lane == 0 || before != u)) |
                (S.part_unit[0][0] >= 0 ? 1u << kSplitWarps : 0u);
    }
    int task = 0;
#pragma unroll 1
    for (; units; units &= units - 1) {
        const int cand = __ffs(units) - 1, which = cand < kSplitWarps, lead = which ? cand : 0;
        const int unit = S.part_unit[lead][which];
        const SplitPos &at = S.part_pos[lead][which];
        const bool in_share = unit >= x0 && unit + at.q.chunks <= x1;
        // of a unit that spans CTAs: the place of its first chunk, and the CTAs
        const int u0 = (unit < x0 ? unit0 : unit1) + kSplitUnitCost;
        const int first = in_share ? 0 : shares.owner(u0), last = in_share ? 0 : shares.owner(u0 + at.q.chunks - 1);
        if (!in_share && tid == 0) {
            const int kind = unit < x0 ? 0 : 1;
            S.join[kind] = 1;
            S.join_first[kind] = first;
            S.join_last[kind] = last;
            S.join_pos[kind] = at;
        }
        // its parts: `n` warps' at their ends, then perhaps an early one
        int n = 0;
        if (which)
            while (lead + n < kSplitWarps && S.part_unit[lead + n][1] == unit) ++n;
        const bool tail = lead + n < kSplitWarps && S.part_unit[lead + n][0] == unit;
        const float *ends_at = results + lead * kPart, *tail_at = early + (lead + n) * kPart;
        for (int col = 0; col < kSplitCols; ++col, ++task) {
            if (task % kSplitWarps != warp || lane >= D / 4) continue;
            const int d = 4 * lane;
            float m = tail ? tail_at[kSplitCols * D + col] : -INFINITY, l = 0.0f, o[4] = {};
#pragma unroll 4
            for (int i = 0; i < n; ++i) m = fmaxf(m, ends_at[i * kPart + kSplitCols * D + col]);
            const float sh = m == -INFINITY ? 0.0f : m;
            auto take = [&](const float *r) {
                const float h = ex2(r[kSplitCols * D + col] - sh);
                const float4 v = *reinterpret_cast<const float4 *>(r + col * D + d);
                l += h * r[kSplitCols * D + kSplitCols + col];
                o[0] += h * v.x, o[1] += h * v.y, o[2] += h * v.z, o[3] += h * v.w;
            };
#pragma unroll 4
            for (int i = 0; i < n; ++i) take(ends_at + i * kPart);
            if (tail) take(tail_at);
            if (in_share) {
                split_store<D, 4>(P, at, col, d, o, m, l);
            } else {
                float *p = cta_part(blockIdx.x, first);
                __stcg(reinterpret_cast<float4 *>(p + col * D + d), make_float4(o[0], o[1], o[2], o[3]));
                if (lane == 0) {
                    __stcg(p + kSplitCols * D + col, m);
                    __stcg(p + kSplitCols * D + kSplitCols + col, l);
                }
            }
        }
    }
    // ---- units that span CTAs: joined by the CTA whose part is the last
    __syncthreads();
    if (!S.join[0] && !S.join[1]) {
        report(P.err, __reduce_or_sync(0xFFFFFFFFu, err) * (lane == 0));
        return;
    }
    if (tid == 0) {
        __threadfence();  // the CTA's stores, seen at the barrier, before the arrivals
        // into words of their own: other threads may still be reading S.join above
        for (int kind = 0; kind < 2; ++kind) {
            S.joins[kind] = 0;
            if (!S.join[kind]) continue;
            int *counter = static_cast<int *>(A.workspace) + S.join_first[kind];
            S.joins[kind] = atomicAdd(counter, 1) == S.join_last[kind] - S.join_first[kind];
            if (S.joins[kind]) *counter = 0;
        }
        __threadfence();
    }
    __syncthreads();
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        if (!S.joins[kind]) continue;
        const int b0 = S.join_first[kind], b1 = S.join_last[kind];
        for (int it = tid; it < kSplitCols * D / 4; it += kSplitThreads) {
            const int col = it / (D / 4), d = it % (D / 4) * 4;
            SplitJoin<D> J;
#pragma unroll 1
            for (int b = b0; b <= b1; b += 8) {
                float mb[8], lb[8];
                float4 ob[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *p = cta_part(min(b + i, b1), b0);
                    mb[i] = b + i > b1 ? -INFINITY : __ldcg(p + kSplitCols * D + col);
                    lb[i] = __ldcg(p + kSplitCols * D + kSplitCols + col);
                    ob[i] = __ldcg(reinterpret_cast<const float4 *>(p + col * D + d));
                }
                J.add(mb, lb, ob);
            }
            split_store<D, 4>(P, S.join_pos[kind], col, d, J.o, J.m, J.l);
        }
    }
    report(P.err, __reduce_or_sync(0xFFFFFFFFu, err) * (lane == 0));
}

// ------------------------------------------------------------------ many rows: tcgen05

// A CTA takes 256 rows (token, query head of the group) of one request and
// cache head, as two tiles of 128 that share every decoded key and value:
//   * warps 0-3 and 4-7: softmax of a tile each, a thread per row: scores out
//     of TMEM, probabilities (FP16) back into the same columns;
//   * warps 8-11: the cache's codes to FP16 operand tiles of 128 keys in
//     shared memory, K as rows of keys and V as rows of elements (transposed
//     while it is decoded: two keys' codes become one byte, one conversion
//     gives the pair, and a thread's 8 keys make a 16-byte chunk);
//   * warp 12: the MMAs, S = Q K^T and O += P V with P taken from TMEM.  The
//     tiles alternate, so the tensor cores work on one while the other's
//     softmax runs.
// TMEM holds both tiles' S (128 columns, P over them) and O.  O is rescaled
// only when a row's maximum grew by more than 2^8: P then stays below 2^8 in
// FP16, and most steps leave O alone.  Waits are bounded; one that gives up
// sets a flag that ends the others.
// A prompt of 8192 tokens, 32 heads on 8 of 128: 547 us, 1.0 PFLOP/s of the 1.6
// that a plain product reaches.  A step of both tiles takes 4250 clocks: 2050 of
// MMA, 2050 of the exp2 unit, and a tile's S, softmax (2900) and P V wait for
// one another.  The decode is hidden (536 us without its conversions).
constexpr int kPrefillThreads = 512;
constexpr int kPrefillTile = 128;  // rows of a tile, keys of a step
// Registers of a thread of the 8 softmax, the 4 decode and the last 4 warps.  More
// than the block was launched with would be waited for without end.
constexpr int kSoftmaxRegs = 184, kDecodeRegs = 104, kMmaRegs = 40;
constexpr int kPrefillRegs = 32 * (8 * kSoftmaxRegs + 4 * kDecodeRegs + 4 * kMmaRegs);
constexpr int kPrefillParts = 8;   // CTAs of a cluster that share a pair's keys, at most
// Steps of a pair that one CTA takes alone: a join takes as long as 3 (D = 64)
// to 5 (D = 128) steps, most of it the transfer between the CTAs' shared memories.
constexpr int kPrefillAlone = 6;
constexpr int kPrefillSort = 64;   // requests that are put in order of their keys, at most
constexpr float kLazy = 8.0f;      // log2 units a row's maximum may grow before O is rescaled

template <int D>
struct PrefillShared {
    static constexpr uint32_t kOperand = kPrefillTile * D * 2;
    static constexpr uint32_t kQ = 0, kK = 2 * kOperand, kV = 4 * kOperand;  // offsets of q, k, v
    alignas(1024) uint8_t q[2][kOperand];
    uint8_t k[2][kOperand], v[2][kOperand];
    alignas(16) uint32_t ok[4][4];  // keys of a step that are there; the softmax may read a step's while the next two are decoded
    float row[2][kPrefillTile];  // factor of a row's scores
    union {
        float2 part[2 * kPrefillTile];  // (m, l) of a row, where CTAs share its keys
        int2 list[kPrefillThreads];     // (keys, pairs of tiles) of requests, before that
    };
    uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_done[2], end;
    int32_t sums[kPrefillThreads / 32];
    uint32_t some[kPrefillThreads / 32];
    uint32_t tmem, abort;
    int32_t req, pair;
};

// Byte offset of 16-byte chunk `chunk` of row `row` in an operand tile whose
// rows are 128 bytes in the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz_chunk(uint32_t row, uint32_t chunk) {
    return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// Shared-memory matrix descriptor of such a tile (K-major, 8-row groups 1024
// bytes apart): the low word from its address, to which multiples of 16 bytes
// may be added as units, and the whole from the low word.
__device__ __forceinline__ uint32_t swz128_desc_low(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }

__device__ __forceinline__ uint64_t swz128_desc(uint32_t low) {
    return static_cast<uint64_t>(low) | (static_cast<uint64_t>((1024u >> 4) | (1u << 14) | (2u << 29)) << 32);
}

// The CTAs of a cluster.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

__device__ __forceinline__ float2 cluster_ld2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// All of the CTA's warps, wherever each is.
__device__ __forceinline__ void prefill_sync() { asm volatile("barrier.sync 1, %0;" ::"n"(kPrefillThreads) : "memory"); }

template <class Shared>
__device__ __forceinline__ bool prefill_wait_slow(uint64_t *bar, uint32_t parity, Shared &S, uint64_t limit_ns) {
    // the clock is slow to read, and a wait that it delays holds up the others
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if (n % 256) continue;
        if (*reinterpret_cast<volatile uint32_t *>(&S.abort)) return false;
        const uint64_t t = global_ns();
        if (!t0) t0 = t;
        if (t - t0 > limit_ns) {
            atomicExch(&S.abort, 1u);
            return false;
        }
    }
}

template <class Shared>
__device__ __forceinline__ bool prefill_wait(uint64_t *bar, uint32_t parity, Shared &S, uint64_t limit_ns) {
    return mbar_try_wait(bar, parity) || prefill_wait_slow(bar, parity, S, limit_ns);
}

// What the CTA works on: rows [row0, rows) of a request, and per tile the key
// steps [a0, a1) that its rows see, counted from key first * 128.
struct PrefillWork {
    int32_t req, q0, n, rows, row0, first, steps, a0[2], a1[2];
    int64_t kv, begin, end;  // keys; the first and the last + 1 that any row can see
};

__device__ __forceinline__ int prefill_pairs(const AttnParams &P, int r) {
    if (r >= P.a.n_reqs) return 0;
    const int q0 = __ldg(P.a.q_start + r), q1 = __ldg(P.a.q_start + r + 1);
    if (!rows_valid(P.a, q0, q1)) return 0;
    const int64_t rows = static_cast<int64_t>(q1 - q0) * P.group;
    return rows > P.split_rows ? static_cast<int>((rows + 2 * kPrefillTile - 1) / (2 * kPrefillTile)) : 0;
}

// The most keys that rows of a tile see, nearly: what its time goes with.
__device__ __forceinline__ int prefill_keys(const AttnParams &P, int r) {
    const int kv = __ldg(P.a.kv_lens + r);
    return P.a.window ? min(kv, P.a.window) : kv;
}

// Keys [lo, hi) that row `row` of the request sees.
__device__ __forceinline__ void prefill_row(const AttnParams &P, const PrefillWork &W, int row, int64_t &lo, int64_t &hi) {
    const int64_t pos = W.kv - W.n + row / static_cast<int>(P.group);
    hi = max(P.a.causal ? min(pos + 1, W.end) : W.end, static_cast<int64_t>(0));
    lo = P.a.window ? min(max(pos + 1 - P.a.window, static_cast<int64_t>(0)), hi) : 0;
}

__device__ __forceinline__ PrefillWork prefill_work(const AttnParams &P, int req, int pair) {
    PrefillWork W;
    W.req = req;
    W.q0 = __ldg(P.a.q_start + req);
    W.n = __ldg(P.a.q_start + req + 1) - W.q0;
    W.rows = W.n * static_cast<int>(P.group);
    W.row0 = pair * 2 * kPrefillTile;
    W.kv = max(__ldg(P.a.kv_lens + req), 0);
    W.end = min(W.kv, static_cast<int64_t>(P.a.max_pages) << P.page_shift);
    int64_t b[2], e[2], first = INT64_MAX, last = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int r0 = W.row0 + x * kPrefillTile, r1 = min(r0 + kPrefillTile, W.rows) - 1;
        b[x] = e[x] = 0;
        if (r0 <= r1) {
            int64_t lo0, hi0, lo1, hi1;
            prefill_row(P, W, r0, lo0, hi0);
            prefill_row(P, W, r1, lo1, hi1);
            if (x == 0) W.begin = lo0;
            if (hi1 > 0) b[x] = lo0 / kPrefillTile, e[x] = (hi1 + kPrefillTile - 1) / kPrefillTile;
        }
        if (e[x] > b[x]) first = min(first, b[x]), last = max(last, e[x]);
    }
    if (last == 0) first = 0;
    W.first = static_cast<int32_t>(first);
    W.steps = static_cast<int32_t>(last - first);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        W.a0[x] = e[x] > b[x] ? static_cast<int32_t>(b[x] - first) : 0;
        W.a1[x] = e[x] > b[x] ? static_cast<int32_t>(e[x] - first) : 0;
    }
    return W;
}

// Part `part` of the pair's steps, of equal ones.
__device__ __forceinline__ void prefill_part(PrefillWork &W, int part, int parts) {
    const int per = (W.steps + parts - 1) / parts, s0 = min(part * per, W.steps), s1 = min(s0 + per, W.steps);
    W.first += s0;
    W.steps = s1 - s0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        W.a0[x] = max(W.a0[x] - s0, 0);
        W.a1[x] = min(W.a1[x] - s0, W.steps);
        if (W.a0[x] >= W.a1[x]) W.a0[x] = W.a1[x] = 0;
    }
}

// Joins the parts of rows [rank * 256 / PARTS, ...) of the pair, which the
// CTAs of the cluster hold in shared memory: O in FP32 at `o`, a row's 16-byte
// chunks xored with its number's last 3 bits, and (m, l) at `ml`.  16 chunks
// of a thread's rows are in flight together.
template <int D, int PARTS>
__device__ __forceinline__ void prefill_join(const AttnParams &P, const PrefillWork &W, int head, int warp, int lane,
                                             uint32_t o, uint32_t ml) {
    const df11_kv4_attention_args &A = P.a;
    constexpr int kLanes = D / 4, kAt = 32 / kLanes;  // lanes of a row; rows at a time
    constexpr int kRows = 2 * kPrefillTile / PARTS, kBatch = 16 / PARTS;
    const int group = static_cast<int>(P.group), c = lane % kLanes;
    const int first = static_cast<int>(cluster_rank()) * kRows + lane / kLanes;
    uint32_t from_o[PARTS], from_ml[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) from_o[p] = cluster_addr(o, p), from_ml[p] = cluster_addr(ml, p);
#pragma unroll 1
    for (int i = warp * kAt; i < kRows; i += 8 * kAt * kBatch) {
        float2 s[kBatch][PARTS];
        float4 v[kBatch][PARTS];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = first + min(i + 8 * kAt * b, kRows - kAt);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                s[b][p] = cluster_ld2(from_ml[p] + r * 8);
                v[b][p] = cluster_ld4(from_o[p] + (r * D + 4 * (c ^ (r & 7))) * 4);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int row = W.row0 + first + i + 8 * kAt * b;
            if (i + 8 * kAt * b >= kRows || row >= W.rows) continue;
            float top = -INFINITY;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) top = fmaxf(top, s[b][p].x);
            const float shift = top == -INFINITY ? 0.0f : top;
            float l = 0.0f, x[4] = {};
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                if (s[b][p].y == 0.0f) continue;  // no key of this part was seen, and its O may be anything
                const float h = ex2(s[b][p].x - shift);
                l += s[b][p].y * h;
                x[0] += v[b][p].x * h, x[1] += v[b][p].y * h, x[2] += v[b][p].z * h, x[3] += v[b][p].w * h;
            }
            const float inv = l > 0.0f ? P.v_scale / l : l;  // NaN stays NaN
            const int64_t token = W.q0 + row / group;
            const int hq = head * group + row % group;
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(A.o) + token * static_cast<int64_t>(A.o_token_stride) + hq * D +
                                       4 * c) = make_uint2(bf16x2_of(x[0] * inv, x[1] * inv), bf16x2_of(x[2] * inv, x[3] * inv));
            if (A.lse && c == 0) A.lse[token * A.n_q_heads + hq] = lse_of(top, l);
        }
    }
}

// The block-table entry of key `key`, or kNoPage where the page holds no key a row sees.
__device__ __forceinline__ int64_t prefill_page(const AttnParams &P, const PrefillWork &W, int64_t key) {
    if (key >= W.end || (((key >> P.page_shift) + 1) << P.page_shift) <= W.begin) return kNoPage;
    return __ldg(P.a.block_table + static_cast<int64_t>(W.req) * P.a.max_pages + (key >> P.page_shift));
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kPrefillThreads, 1) attention_prefill_kernel(const AttnParams P) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    PrefillShared<D> &S =
        *reinterpret_cast<PrefillShared<D> *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
    const df11_kv4_attention_args &A = P.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = static_cast<int>(P.group);

    // ---- this CTA's request and rows: pairs of tiles in the order of the most
    // keys that a row of the request sees, a request's last rows first (the
    // last to start should not be long: 6 prompt chunks of 21 to 765 tokens on
    // 209 to 7278 keys take 50 us so, and 62 in the order of the requests)
    const uint32_t place = SHARED ? blockIdx.x / P.parts : blockIdx.x;
    const int want = static_cast<int>(place / P.kv_heads), head = static_cast<int>(place % P.kv_heads);
    int64_t all = 0;  // 64 bits: row starts that are no ascending ones could count the same rows many times
    int many = 0;
    for (int b = 0; b < A.n_reqs; b += kPrefillThreads) {
        const int w = prefill_pairs(P, b + tid);
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, w > 0);
        const uint32_t sum = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(w));
        __syncthreads();
        if (lane == 0) {
            S.sums[warp] = static_cast<int32_t>(sum);
            S.some[warp] = mask;
        }
        S.list[tid] = make_int2(w ? prefill_keys(P, b + tid) : 0, w);
        __syncthreads();
        for (int i = 0; i < kPrefillThreads / 32; ++i) {
            all += S.sums[i];
            many += __popc(S.some[i]);
        }
    }
    if (want >= all) {
        if (blockIdx.x == 0) grid_wait();
        return;
    }
    if (A.n_reqs <= kPrefillThreads && many <= kPrefillSort) {
        const int2 mine = S.list[tid];
        int at = 0;
        if (mine.y)
            for (int i = 0; i < kPrefillThreads / 32; ++i)
                for (uint32_t m = S.some[i]; m; m &= m - 1) {
                    const int j = 32 * i + __ffs(m) - 1;
                    const int2 other = S.list[j];
                    if (other.x > mine.x || (other.x == mine.x && j > tid)) at += other.y;
                }
        if (mine.y && at <= want && want < at + mine.y) {
            S.req = tid;
            S.pair = mine.y - 1 - (want - at);
        }
    } else {
        // in the order of the requests, from the last
        int64_t base = 0;
        const int64_t from = all - 1 - want;
        for (int b = 0; b < A.n_reqs; b += kPrefillThreads) {
            const int w = prefill_pairs(P, b + tid);
            int incl = w;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, incl, x);
                if (lane >= x) incl += o;
            }
            __syncthreads();
            if (lane == 31) S.sums[warp] = incl;
            __syncthreads();
            int64_t before = base;
            for (int i = 0; i < kPrefillThreads / 32; ++i) {
                if (i < warp) before += S.sums[i];
                base += S.sums[i];
            }
            const int64_t at = before + incl - w;
            if (w && at <= from && from < at + w) {
                S.req = b + tid;
                S.pair = static_cast<int32_t>(from - at);
            }
        }
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.q_full[i], 128);
            mbar_init(&S.k_full[i], 128);
            mbar_init(&S.k_empty[i], 1);
            mbar_init(&S.v_full[i], 128);
            mbar_init(&S.v_empty[i], 1);
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i], 128);
            mbar_init(&S.o_done[i], 1);
        }
        mbar_init(&S.end, 1);
        S.abort = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(&S.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    PrefillWork W = prefill_work(P, S.req, S.pair);
    const bool shared = SHARED && W.steps > kPrefillAlone;
    const int part = SHARED ? static_cast<int>(blockIdx.x) % P.parts : 0;
    if constexpr (SHARED) prefill_part(W, part, shared ? P.parts : 1);
    uint32_t err = 0;

    if (warp < 8) {
        // =============================== softmax of tile x, a thread per row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int x = warp >> 2, r = tid & 127;
        const int row = W.row0 + x * kPrefillTile + r;
        const bool live = row < W.rows;
        const int64_t token = W.q0 + row / group;
        const int hq = head * group + row % group;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's TMEM lanes
        const uint32_t s_col = tmem + lanes + x * kPrefillTile, o_col = tmem + lanes + 2 * kPrefillTile + x * D;
        const int a0 = x ? W.a0[1] : W.a0[0], steps = (x ? W.a1[1] : W.a1[0]) - a0;
        float f = 0.0f;
        if (steps) {
            // The warp's 32 rows of queries, a row's 16-byte chunks on D / 8 lanes,
            // all loads in flight at once.  A row is scaled by a power of two
            // into FP16's range (and by the sign of the scores' factor, which
            // is then >= 0).
            constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // lanes of a row; rows at a time
            const int c = lane % kLanes, base = W.row0 + x * kPrefillTile + (warp & 3) * 32 + lane / kLanes;
            const float f0 = A.scale * P.k_scale * 1.44269504088896341f;
            uint4 v[32 / kAt];
#pragma unroll
            for (int i = 0; i < 32 / kAt; ++i) {
                const int rw = base + i * kAt;
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (rw < W.rows)
                    v[i] = __ldg(reinterpret_cast<const uint4 *>(
                        static_cast<const uint16_t *>(A.q) +
                        static_cast<int64_t>(W.q0 + rw / group) * static_cast<int64_t>(A.q_token_stride) +
                        (head * group + rw % group) * D + c * 8));
            }
#pragma unroll
            for (int i = 0; i < 32 / kAt; ++i) {
                uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    top = max3(top, fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u)));
#pragma unroll
                for (int y = 1; y < kLanes; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, y));
                const uint32_t field = __float_as_uint(top) >> 23;
                const int e = top == 0.0f || field == 255u ? 0 : max(static_cast<int>(field) - 127, -126);
                float down = e == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                float fr = fabsf(f0) * __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                if (f0 < 0.0f) down = -down;
                if (fr == 0.0f) fr = 1.0f, down = 0.0f;  // all scores 0, and still -inf where masked
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = pack_f16(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xFFFF0000u) * down);
                const int rt = (warp & 3) * 32 + i * kAt + lane / kLanes;
                *reinterpret_cast<uint4 *>(S.q[x] + (c / 8) * (kPrefillTile * 128) + swz_chunk(rt, c % 8)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
                if (c == 0) S.row[x][rt] = fr;
            }
            __syncwarp();
            f = S.row[x][r];
            fence_proxy_async_smem();
            mbar_arrive(&S.q_full[x]);
        }
        // keys [lo, hi) seen by this row, from the tile's first step on; rows past
        // the last (zeros) as that one: they must not make every step a masked one
        int lo = 0, hi = 0;
        {
            int64_t lo64, hi64;
            prefill_row(P, W, min(row, W.rows - 1), lo64, hi64);
            const int64_t from = static_cast<int64_t>(W.first + a0) * kPrefillTile;
            lo = static_cast<int>(max(lo64 - from, static_cast<int64_t>(0)));
            hi = static_cast<int>(max(hi64 - from, static_cast<int64_t>(0)));
        }
        float m = -INFINITY, l = 0.0f;
        bool run = true;
        for (int it = 0; it < steps; ++it) {
            const int j = a0 + it;
            run = __all_sync(0xFFFFFFFFu, prefill_wait(&S.s_full[x], it & 1u, S, P.wait_ns));
            if (!run) break;
            tc_fence_after();
            uint32_t s[kPrefillTile];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc_ld32(s_col + 32 * i, s + 32 * i);
            uint4 ok;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(ok.x), "=r"(ok.y), "=r"(ok.z), "=r"(ok.w)
                         : "r"(smem_addr(S.ok[j & 3]))
                         : "memory");
            tc_wait_ld();
            const int left = hi - it * kPrefillTile, right = lo - it * kPrefillTile;
            const bool full = left >= kPrefillTile && right <= 0 && (ok.x & ok.y & ok.z & ok.w) == 0xFFFFFFFFu;
            if (__any_sync(0xFFFFFFFFu, !full)) {
                const uint32_t words[4] = {ok.x, ok.y, ok.z, ok.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ai = min(max(right - 32 * i, 0), 32), bi = min(max(left - 32 * i, 0), 32);
                    const uint32_t below = bi == 32 ? 0xFFFFFFFFu : (1u << bi) - 1u;
                    const uint32_t seen = ai == 32 ? 0u : words[i] & below & (0xFFFFFFFFu << ai);
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (!(seen >> y & 1u)) s[32 * i + y] = 0xFF800000u;  // -inf
                }
            }
            float t0 = __uint_as_float(s[0]), t1 = __uint_as_float(s[1]), t2 = __uint_as_float(s[2]),
                  t3 = __uint_as_float(s[3]);
#pragma unroll
            for (int i = 4; i < kPrefillTile - 4; i += 8) {
                t0 = max3(t0, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                t1 = max3(t1, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
                t2 = max3(t2, __uint_as_float(s[i + 4]), __uint_as_float(s[i + 5]));
                t3 = max3(t3, __uint_as_float(s[i + 6]), __uint_as_float(s[i + 7]));
            }
            t0 = max3(t0, t1, t2);
            t3 = max3(t3, __uint_as_float(s[kPrefillTile - 4]), __uint_as_float(s[kPrefillTile - 3]));
            t0 = max3(t0, __uint_as_float(s[kPrefillTile - 2]), __uint_as_float(s[kPrefillTile - 1]));
            const float top = fmaxf(t0, t3);
            const float mt = top == -INFINITY ? -INFINITY : top * f;
            const bool grow = mt > m + kLazy || (m == -INFINITY && mt != -INFINITY);
            if (__any_sync(0xFFFFFFFFu, grow)) {
                const float mn = grow ? mt : m;
                const float alpha = grow ? ex2(m - mn) : 1.0f;
                m = mn;
                l *= alpha;
                if (it) {
                    run = __all_sync(0xFFFFFFFFu, prefill_wait(&S.o_done[x], (it - 1) & 1u, S, P.wait_ns));
                    if (!run) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < D; i += 16) {
                        uint32_t o[16];
                        tc_ld16(o_col + i, o);
                        tc_wait_ld();
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
                        tc_st16(o_col + i, o);
                    }
                }
            }
            const float shift = m == -INFINITY ? 0.0f : m;
            // two at a time: p = 2^(s f - shift), and their sums
            const uint64_t f2 = pair(f, f), shift2 = pair(-shift, -shift);
            uint64_t la = 0, lb = 0;
#pragma unroll
            for (int c = 0; c < kPrefillTile; c += 32) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t e = fma2(pair(__uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1])), f2, shift2);
                    const float p0 = ex2(low(e)), p1 = ex2(high(e));
                    (i & 1 ? lb : la) = add2(i & 1 ? lb : la, pair(p0, p1));
                    w[i] = pack_f16(p0, p1);
                }
                tc_st16(s_col + c / 2, w);
            }
            la = add2(la, lb);
            l += low(la) + high(la);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&S.p_full[x]);
        }
        if (run && steps) {
            run = __all_sync(0xFFFFFFFFu, prefill_wait(&S.o_done[x], (steps - 1) & 1u, S, P.wait_ns));
            tc_fence_after();
        }
        if (!run) err |= DF11_DEV_ERR_TIMEOUT;
        if (shared) {
            // the part's rows to shared memory, where no MMA reads any more
            prefill_sync();
            float *o = reinterpret_cast<float *>(S.q[0]);
            const int at = x * kPrefillTile + r;
            if (!run || !steps) m = -INFINITY, l = 0.0f;
            S.part[at] = make_float2(m, l);
            if (run && steps) {
#pragma unroll
                for (int i = 0; i < D; i += 16) {
                    uint32_t v[16];
                    tc_ld16(o_col + i, v);
                    tc_wait_ld();
#pragma unroll
                    for (int y = 0; y < 16; y += 4)
                        *reinterpret_cast<uint4 *>(o + at * D + 4 * (((i + y) / 4) ^ (at & 7))) =
                            make_uint4(v[y], v[y + 1], v[y + 2], v[y + 3]);
                }
            }
            cluster_sync();
            const uint32_t so = smem_addr(o), sp = smem_addr(S.part);
            if (P.parts == 8) prefill_join<D, 8>(P, W, head, warp, lane, so, sp);
            else if (P.parts == 4) prefill_join<D, 4>(P, W, head, warp, lane, so, sp);
            else prefill_join<D, 2>(P, W, head, warp, lane, so, sp);
            cluster_sync();
        } else if (part == 0) {
            // Rows out of TMEM into the tile's query operand, which no MMA reads any
            // more (a thread its own row), and from there to o, a row's chunks on
            // D / 8 lanes.  l == 0: the row saw no key, whatever the accumulator holds.
            const float inv = !run ? 0.0f : l > 0.0f ? P.v_scale / l : l;  // NaN stays NaN
            if (steps) {
#pragma unroll
                for (int i = 0; i < D; i += 16) {
                    uint32_t o[16];
                    tc_ld16(o_col + i, o);
                    tc_wait_ld();
#pragma unroll
                    for (int y = 0; y < 16; y += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            w[z] = l == 0.0f ? 0u
                                             : bf16x2_of(__uint_as_float(o[y + 2 * z]) * inv, __uint_as_float(o[y + 2 * z + 1]) * inv);
                        const int c = (i + y) / 8;
                        *reinterpret_cast<uint4 *>(S.q[x] + (c / 8) * (kPrefillTile * 128) + swz_chunk(r, c % 8)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
            }
            {
                constexpr int kLanes = D / 8, kAt = 32 / kLanes;
                const int c = lane % kLanes;
#pragma unroll 4
                for (int i = 0; i < 32 / kAt; ++i) {
                    const int rt = (warp & 3) * 32 + i * kAt + lane / kLanes, rw = W.row0 + x * kPrefillTile + rt;
                    if (rw >= W.rows) continue;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (steps)
                        v = *reinterpret_cast<const uint4 *>(S.q[x] + (c / 8) * (kPrefillTile * 128) + swz_chunk(rt, c % 8));
                    *reinterpret_cast<uint4 *>(
                        static_cast<uint16_t *>(A.o) +
                        static_cast<int64_t>(W.q0 + rw / group) * static_cast<int64_t>(A.o_token_stride) +
                        (head * group + rw % group) * D + c * 8) = v;
                }
            }
            if (live && A.lse) A.lse[token * A.n_q_heads + hq] = lse_of(m, l);
        }
        tc_fence_before();
    } else if (warp < 12) {
        // =============================== the cache to FP16 operand tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDecodeRegs));
        constexpr uint32_t NB = D / 16;
        const int u = tid - 256;  // K: the step's key; V: 8 keys and 16 elements
        const int unit = u >> 3;  // V: 16 chunks of 8 keys x NB blocks, lanes of 8 over the chunks of one 128-byte row
        const uint32_t vb = static_cast<uint32_t>(unit) % NB, vc = (static_cast<uint32_t>(unit) / NB) * 8u + (u & 7u);
        const bool v_mine = vc < 16u;
        const uint32_t mask = (1u << P.page_shift) - 1u;
        auto block = [&](int64_t id, bool &have) -> const uint8_t * {
            have = id >= 0 && static_cast<uint64_t>(id) < P.n_pages;
            return P.pages + (static_cast<uint64_t>(have ? id : 0) * P.kv_heads + static_cast<uint32_t>(head)) * P.block.bytes;
        };
        uint32_t kw[D / 8], vw[16];
        uint2 ks = make_uint2(0u, 0u), vs = make_uint2(0u, 0u);
        bool k_have = false;
        auto load_k = [&](int j, int64_t id) {
            const int64_t key = static_cast<int64_t>(W.first + j) * kPrefillTile + u;
            const uint8_t *b = block(id, k_have);
            if (!k_have && id != kNoPage) err |= DF11_DEV_ERR_PAGES;
#pragma unroll
            for (uint32_t i = 0; i < D / 8; ++i) kw[i] = 0u;
            ks = make_uint2(0u, 0u);
            if (!k_have) return;
            const uint32_t off = static_cast<uint32_t>(key) & mask;
            const uint4 *c = reinterpret_cast<const uint4 *>(b + P.block.k_codes + off * (D / 2));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = __ldg(c + i);
                kw[4 * i] = v.x, kw[4 * i + 1] = v.y, kw[4 * i + 2] = v.z, kw[4 * i + 3] = v.w;
            }
            if constexpr (D == 128) ks = __ldg(reinterpret_cast<const uint2 *>(b + P.block.k_scales + off * NB));
            else ks.x = __ldg(reinterpret_cast<const uint32_t *>(b + P.block.k_scales + off * NB));
        };
        auto load_v = [&](int j, int64_t id) {
            const int64_t key = static_cast<int64_t>(W.first + j) * kPrefillTile + 8 * vc;
            bool have;
            const uint8_t *b = block(id, have);
#pragma unroll
            for (int i = 0; i < 16; ++i) vw[i] = 0u;
            vs = make_uint2(0u, 0u);
            if (!v_mine || !have) return;
            const uint32_t off = static_cast<uint32_t>(key) & mask;
            const uint8_t *c = b + P.block.v_codes + ((off >> 2) * NB + vb) * 32u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(c + (i / 2) * (NB * 32u)) + i % 2);
                vw[4 * i] = v.x, vw[4 * i + 1] = v.y, vw[4 * i + 2] = v.z, vw[4 * i + 3] = v.w;
            }
            vs = __ldg(reinterpret_cast<const uint2 *>(b + P.block.v_scales + (vb << P.page_shift) + off));
            // keys past the end may hold anything, NaN scales too: they count as 0
            const int left = static_cast<int>(min(W.end - key, static_cast<int64_t>(8)));
            if (left < 4) vs.x &= (1u << (8 * left)) - 1u;
            if (left <= 4) vs.y = 0u;
            else if (left < 8) vs.y &= (1u << (8 * (left - 4))) - 1u;
        };
        auto k_page = [&](int j) { return prefill_page(P, W, static_cast<int64_t>(W.first + j) * kPrefillTile + u); };
        auto v_page = [&](int j) { return prefill_page(P, W, static_cast<int64_t>(W.first + j) * kPrefillTile + 8 * vc); };
        int64_t idk = kNoPage, idv = kNoPage;
        if (W.steps) {
            load_k(0, k_page(0));
            load_v(0, v_page(0));
            if (W.steps > 1) idk = k_page(1), idv = v_page(1);
        }
        for (int j = 0; j < W.steps; ++j) {
            const int st = j & 1;
            if (j >= 2 && !__all_sync(0xFFFFFFFFu, prefill_wait(&S.k_empty[st], ((j >> 1) - 1) & 1u, S, P.wait_ns))) {
                err |= DF11_DEV_ERR_TIMEOUT;
                break;
            }
            {
                const uint32_t ok = __ballot_sync(0xFFFFFFFFu, k_have);
                if (lane == 0) S.ok[j & 3][warp - 8] = ok;
                uint8_t *dst = S.k[st];
#pragma unroll
                for (uint32_t b = 0; b < NB; ++b) {
                    const uint32_t sw = b < 4 ? ks.x : ks.y;
                    const uint32_t two = e4m3x2_to_f16x2(__byte_perm(sw, 0, (b & 3u) * 0x11u));
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        uint32_t w[4];
                        e2m1x8_to_f16(kw[2 * b + h], w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = f16x2_mul(w[i], two);
                        const uint32_t c = 2 * b + h;
                        *reinterpret_cast<uint4 *>(dst + (c / 8) * (kPrefillTile * 128) + swz_chunk(u, c % 8)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&S.k_full[st]);
            if (j + 1 < W.steps) {
                load_k(j + 1, idk);
                if (j + 2 < W.steps) idk = k_page(j + 2);
            }
            if (j >= 2 && !__all_sync(0xFFFFFFFFu, prefill_wait(&S.v_empty[st], ((j >> 1) - 1) & 1u, S, P.wait_ns))) {
                err |= DF11_DEV_ERR_TIMEOUT;
                break;
            }
            if (v_mine) {
                uint8_t *dst = S.v[st] + (vc / 8) * (D * 128);
                const uint32_t sc[4] = {e4m3x2_to_f16x2(vs.x & 0xFFFFu), e4m3x2_to_f16x2(vs.x >> 16),
                                        e4m3x2_to_f16x2(vs.y & 0xFFFFu), e4m3x2_to_f16x2(vs.y >> 16)};
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    uint32_t ev[4][4], od[4][4];  // [pair of keys][element / 2]
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a = vw[4 * i + h], b = vw[4 * i + 2 + h];
                        e2m1x8_to_f16((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), ev[i]);
                        e2m1x8_to_f16(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), od[i]);
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            ev[i][z] = f16x2_mul(ev[i][z], sc[i]);
                            od[i][z] = f16x2_mul(od[i][z], sc[i]);
                        }
                    }
#pragma unroll
                    for (uint32_t z = 0; z < 4; ++z) {
                        const uint32_t d = 16 * vb + 8 * h + 2 * z;
                        *reinterpret_cast<uint4 *>(dst + swz_chunk(d, vc % 8)) =
                            make_uint4(ev[0][z], ev[1][z], ev[2][z], ev[3][z]);
                        *reinterpret_cast<uint4 *>(dst + swz_chunk(d + 1, vc % 8)) =
                            make_uint4(od[0][z], od[1][z], od[2][z], od[3][z]);
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&S.v_full[st]);
            if (j + 1 < W.steps) {
                load_v(j + 1, idv);
                if (j + 2 < W.steps) idv = v_page(j + 2);
            }
        }
    } else {
        // =============================== MMAs
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        // one elected lane walks: the instructions between a wait and the MMAs it
        // holds back are on the critical path, so descriptors are made once and
        // the steps go in pairs, whose stages are then constants
        if (warp == 12 && W.steps && elect_one()) {
            // FP32 accumulate, FP16 A and B, M = 128; N = keys of a step, then head elements
            constexpr uint32_t idesc_s = (1u << 4) | ((kPrefillTile >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t idesc_o = (1u << 4) | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24);
            using Sh = PrefillShared<D>;
            // low words of the descriptors: the shared block's address (in 16
            // bytes) and a constant; `here` keeps the sums from being made
            // ahead of the loop, in registers that this role does not have
            auto here = [](uint32_t v) {
                asm volatile("" : "+r"(v));
                return v;
            };
            const uint32_t base = swz128_desc_low(smem_addr(&S));
            const int a0[2] = {W.a0[0], W.a0[1]}, a1[2] = {W.a1[0], W.a1[1]}, steps = W.steps;
            bool run = true;
            uint32_t parity = 0;  // of both stages' phases in this pair of steps
            auto wait = [&](uint64_t *bar, uint32_t ph) { run = run && prefill_wait(bar, ph, S, P.wait_ns); };
            // x, st: constants where this is inlined
            auto scores = [&](int x, int st, int j) {
                if (j == a0[x]) wait(&S.q_full[x], 0);
                if (!run) return;
                tc_fence_after();
                const uint32_t b = here(base);
#pragma unroll
                for (uint32_t i = 0; i < D / 16; ++i) {
                    const uint32_t at = (i / 4) * (kPrefillTile * 128) + (i % 4) * 32;
                    tc_mma(tmem + x * kPrefillTile, swz128_desc(b + ((Sh::kQ + x * Sh::kOperand + at) >> 4)),
                           swz128_desc(b + ((Sh::kK + st * Sh::kOperand + at) >> 4)), idesc_s, i > 0);
                }
                tc_commit(&S.s_full[x]);
            };
            auto values = [&](int x, int st, uint32_t ph, int j) {
                wait(&S.v_full[st], ph);
                wait(&S.p_full[x], (j - a0[x]) & 1u);
                if (!run) return;
                tc_fence_after();
                const uint32_t more = j > a0[x], b = here(base);
#pragma unroll
                for (uint32_t i = 0; i < kPrefillTile / 16; ++i)
                    tc_mma_ts(tmem + 2 * kPrefillTile + x * D, tmem + x * kPrefillTile + i * 8,
                              swz128_desc(b + ((Sh::kV + st * Sh::kOperand + (i / 4) * (D * 128) + (i % 4) * 32) >> 4)),
                              idesc_o, i > 0 ? 1u : more);
                tc_commit(&S.o_done[x]);
            };
            auto active = [&](int x, int j) { return j >= a0[x] && j < a1[x]; };
            auto step = [&](int st, int j) {
                wait(&S.k_full[st], parity);
                if (run && active(0, j)) scores(0, st, j);
                if (run && j) {
                    if (active(1, j - 1)) values(1, st ^ 1, st ? parity : parity ^ 1u, j - 1);
                    if (run) tc_commit(&S.v_empty[st ^ 1]);
                }
                if (run && active(1, j)) scores(1, st, j);
                if (run) tc_commit(&S.k_empty[st]);
                if (run && active(0, j)) values(0, st, parity, j);
            };
            for (int j = 0; j < steps && run; j += 2, parity ^= 1u) {
                step(0, j);
                if (run && j + 1 < steps) step(1, j + 1);
            }
            if (run && active(1, steps - 1)) values(1, (steps - 1) & 1, ((steps - 1) >> 1) & 1u, steps - 1);
            // every MMA has completed before the CTA ends
            tc_commit(&S.end);
            if (!mbar_wait(&S.end, 0, P.wait_ns) || !run) err |= DF11_DEV_ERR_TIMEOUT;
        }
        __syncwarp();
    }
    if (shared && warp >= 8) {
        prefill_sync();
        cluster_sync();
        cluster_sync();
    }
    err = __reduce_or_sync(0xFFFFFFFFu, err);
    if (lane == 0) report(P.err, err);
    if (blockIdx.x == 0) grid_wait();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
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
    P.parts = 1;
    P.split_rows = static_cast<int64_t>(a.n_reqs) * c.n_heads <= kSplitFew ? kSplitRowsFew : kSplitRows;
    P.ws_parts = kMaxCtas;
    P.ws_warps = kMaxCtas + 2 * kMaxCtas * (c.head_dim == 128 ? split_partial_floats<128>() : split_partial_floats<64>());
    return P;
}

template <int D>
void launch_split(const AttnParams &P, int ctas, cudaStream_t s) {
    constexpr size_t smem = sizeof(SplitShared<D>);
    switch (P.page_shift) {
        case 4: attention_split_kernel<D, 4><<<ctas, kSplitThreads, smem, s>>>(P); break;
        case 5: attention_split_kernel<D, 5><<<ctas, kSplitThreads, smem, s>>>(P); break;
        default: attention_split_kernel<D, 6><<<ctas, kSplitThreads, smem, s>>>(P); break;
    }
}

template <int D>
constexpr size_t kPrefillSmem = sizeof(PrefillShared<D>) + 1024;  // and what aligns it
static_assert(3 * 2 * PrefillShared<64>::kOperand >= 2 * kPrefillTile * 64 * 4 && 3 * 2 * PrefillShared<128>::kOperand >= 2 * kPrefillTile * 128 * 4,
              "a part's rows fit the operands' place");

template <int D>
cudaError_t launch_prefill(const AttnParams &P, unsigned pairs, cudaStream_t s) {
    cudaLaunchAttribute attrs[2]{};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(pairs * P.kv_heads * P.parts);
    cfg.blockDim = dim3(kPrefillThreads);
    cfg.dynamicSmemBytes = kPrefillSmem<D>;
    cfg.stream = s;
    cfg.attrs = attrs;
    if (P.early) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (P.parts > 1) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs++].val.clusterDim = {static_cast<unsigned>(P.parts), 1, 1};
    }
    return cudaLaunchKernelEx(&cfg, P.parts > 1 ? attention_prefill_kernel<D, true> : attention_prefill_kernel<D, false>, P);
}

// Clusters of `parts` prefill CTAs that run at the same time.
int max_clusters(int parts) {
    cudaLaunchAttribute cluster{};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {static_cast<unsigned>(parts), 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(parts);
    cfg.blockDim = dim3(kPrefillThreads);
    cfg.dynamicSmemBytes = kPrefillSmem<128>;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, attention_prefill_kernel<128, true>, &cfg) == cudaSuccess) return n;
    cudaGetLastError();  // they then share no keys
    return 0;
}

struct Device {
    int sms = 0;
    int clusters[4] = {};  // of 1 << i prefill CTAs, at the same time
};

bool prepare(Device *d) {
    constexpr int kDevices = 64;
    static std::mutex mu;
    static Device known[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    std::lock_guard<std::mutex> lk(mu);
    if (!known[dev].sms) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
        auto allow = [](auto *kernel, size_t bytes) {
            return cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) == cudaSuccess;
        };
        if (!allow(&attention_split_kernel<64, 4>, sizeof(SplitShared<64>)) ||
            !allow(&attention_split_kernel<64, 5>, sizeof(SplitShared<64>)) ||
            !allow(&attention_split_kernel<64, 6>, sizeof(SplitShared<64>)) ||
            !allow(&attention_split_kernel<128, 4>, sizeof(SplitShared<128>)) ||
            !allow(&attention_split_kernel<128, 5>, sizeof(SplitShared<128>)) ||
            !allow(&attention_split_kernel<128, 6>, sizeof(SplitShared<128>)) ||
            !allow(&attention_prefill_kernel<64, false>, kPrefillSmem<64>) ||
            !allow(&attention_prefill_kernel<64, true>, kPrefillSmem<64>) ||
            !allow(&attention_prefill_kernel<128, false>, kPrefillSmem<128>) ||
            !allow(&attention_prefill_kernel<128, true>, kPrefillSmem<128>))
            return false;
        // a build with fewer registers a thread than the roles share out is not launched
        auto holds = [](auto *kernel) {
            cudaFuncAttributes f{};
            return cudaFuncGetAttributes(&f, reinterpret_cast<const void *>(kernel)) == cudaSuccess &&
                   f.numRegs * kPrefillThreads >= kPrefillRegs;
        };
        if (!holds(&attention_prefill_kernel<64, false>) || !holds(&attention_prefill_kernel<64, true>) ||
            !holds(&attention_prefill_kernel<128, false>) || !holds(&attention_prefill_kernel<128, true>))
            return false;
        for (int i = 1; 1 << i <= kPrefillParts; ++i) known[dev].clusters[i] = max_clusters(1 << i);
        known[dev].sms = std::min(v, kMaxCtas);
    }
    *d = known[dev];
    return true;
}

}  // namespace

LaunchStatus kv4_attention_workspace(const df11_kv4_cache &c, const df11_kv4_attention_args &, uint64_t *bytes) {
    const uint64_t part = c.head_dim == 128 ? split_partial_floats<128>() : split_partial_floats<64>();
    *bytes = 4 * (kMaxCtas + (2 + kSplitWarps) * kMaxCtas * part);
    return LaunchStatus::kOk;
}

LaunchStatus launch_kv4_attention(const df11_kv4_cache &c, const df11_kv4_attention_args &a, int *err,
                                  cudaStream_t s) {
    AttnParams P = attn_params(c, a, err);
    Device dev;
    // rows, and the split path's places, are counted in 31 bits
    if (static_cast<int64_t>(a.n_tokens) * a.n_q_heads > INT32_MAX) return LaunchStatus::kUnsupported;
    const int64_t tiles = (std::min<int64_t>(static_cast<int64_t>(a.max_q_len) * P.group, kSplitRowsFew) + kSplitCols - 1) / kSplitCols;
    const int64_t chunks =
        std::max<int64_t>(((static_cast<int64_t>(a.max_pages) << P.page_shift) + kSplitKeys - 1) / kSplitKeys, 1) + kSplitUnitCost;
    if (static_cast<double>(a.n_reqs) * P.kv_heads * tiles * chunks >= 2147483648.0) return LaunchStatus::kUnsupported;
    if (!prepare(&dev)) return LaunchStatus::kCuda;
    int64_t pairs = 0;
    if (static_cast<int64_t>(a.max_q_len) * P.group > P.split_rows) {
        // as many pairs of tiles as the rows can make, the last one of each
        // request that has more rows than the other path takes with one row, and
        // no request with more than max_q_len has
        const int64_t rows = static_cast<int64_t>(a.n_tokens) * P.group;
        const int64_t some = std::min<int64_t>(a.n_reqs, rows / (P.split_rows + 1));
        const int64_t most = (std::min<int64_t>(a.max_q_len, a.n_tokens) * P.group + 2 * kPrefillTile - 1) / (2 * kPrefillTile);
        pairs = std::min((rows + some * (2 * kPrefillTile - 1)) / (2 * kPrefillTile), some * most);
        // where clusters of CTAs, one for each pair and head, run all at the same
        // time, they share the keys: 85 tokens in groups of 3 against 8192 keys of
        // 8 heads take 135 us alone (D = 64; 139 for D = 128), 32 (39) with 8
        const int64_t steps = ((static_cast<int64_t>(a.max_pages) << P.page_shift) + kPrefillTile - 1) / kPrefillTile;
        for (int i = 1; pairs && 1 << i <= kPrefillParts && steps > kPrefillAlone; ++i)
            if (pairs * P.kv_heads <= dev.clusters[i]) P.parts = 1 << i;
        // a launch of up to two CTAs a multiprocessor starts while the first
        // kernel runs (9 ragged requests: 61 us, not 62); a larger one is
        // slower that way (a prompt of 8192 tokens: 557 us, not 547)
        P.early = pairs && pairs * P.kv_heads * P.parts <= 2 * dev.sms;
    }
    if (c.head_dim == 128) launch_split<128>(P, dev.sms, s);
    else launch_split<64>(P, dev.sms, s);
    if (pairs) {
        const cudaError_t e = c.head_dim == 128 ? launch_prefill<128>(P, static_cast<unsigned>(pairs), s)
                                                : launch_prefill<64>(P, static_cast<unsigned>(pairs), s);
        if (e != cudaSuccess) return LaunchStatus::kCuda;
    }
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

}  // namespace df11
