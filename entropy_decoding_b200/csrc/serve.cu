// serve.cu -- what a decode step does around the fused GEMMs of a block's
// attention, short of the cache itself: the step's pages, slots and positions
// from the requests' lengths, and the norm and rotation of queries and keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "df11.h"
#include "serve.h"

namespace df11 {
namespace {

__device__ __forceinline__ void flag(int *err, uint32_t bits) {
    if (err && bits) atomicOr(err, static_cast<int>(bits));
}

// ------------------------------------------------------------------ pages, slots, positions

// One launch, a thread per row (new token).  Every CTA scans the requests'
// row and page counts itself, up to the requests its rows belong to: the
// lengths are a few KB in L2, and a second launch or a wait between CTAs would
// cost more than reading them again.  Sums are 64-bit, so no length overflows
// them.  A row finds its request by bisection among the scanned starts; the
// row that starts a page is the one that writes the page into the block table,
// and every row computes its page's id from the free stack itself, so no
// thread reads what another writes.  Pages are those that the table has room
// for; where rows are cut off at max_tokens, the first CTA writes the pages
// that they would have started, so every page taken is in the table.  Bound by the launch and two rounds through
// L2: 3.1 us for 128 requests of a token each, 4.8 us for 509 with up to 2048
// new tokens each.
constexpr int kExtendThreads = 512;

__device__ __forceinline__ int64_t warp_incl(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

__global__ void __launch_bounds__(kExtendThreads) kv_extend_kernel(const df11_kv_extend_args A, int shift, int *err) {
    __shared__ int64_t s_row[kExtendThreads], s_page[kExtendThreads];
    __shared__ int32_t s_kv[kExtendThreads];
    __shared__ int64_t s_sum[2][kExtendThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first = blockIdx.x == 0;
    const int64_t t_end = (static_cast<int64_t>(blockIdx.x) + 1) * kExtendThreads, t = t_end - kExtendThreads + tid;
    const int32_t mask = A.page_size - 1;
    const int64_t n_free = max(*A.n_free, 0), room = A.max_pages;
    uint32_t bad = 0;
    int64_t rows = 0, pages = 0;  // of the requests before this tile
    for (int base = 0; base < A.n_reqs && (first || rows < t_end); base += kExtendThreads) {
        const int r = base + tid, cnt = min(kExtendThreads, A.n_reqs - base);
        int32_t kv = 0, nw = 0;
        if (r < A.n_reqs) {
            kv = A.kv_lens[r];
            nw = A.new_lens[r];
            if (kv < 0 || nw < 0) bad |= DF11_DEV_ERR_AUX;
            kv = max(kv, 0);
            nw = max(nw, 0);
        }
        const int64_t len = static_cast<int64_t>(kv) + nw;
        const int64_t np = min((len + mask) >> shift, room) - min((static_cast<int64_t>(kv) + mask) >> shift, room);
        int64_t ri = warp_incl(nw, lane), pi = warp_incl(np, lane);
        if (lane == 31) {
            s_sum[0][warp] = ri;
            s_sum[1][warp] = pi;
        }
        __syncthreads();
        int64_t all_rows = 0, all_pages = 0;
#pragma unroll
        for (int w = 0; w < kExtendThreads / 32; ++w) {
            if (w == warp) {
                ri += all_rows;
                pi += all_pages;
            }
            all_rows += s_sum[0][w];
            all_pages += s_sum[1][w];
        }
        const int64_t row0 = rows + ri - nw;
        s_row[tid] = row0;
        s_page[tid] = pages + pi - np;
        s_kv[tid] = kv;
        if (first && r < A.n_reqs) {
            A.kv_lens_out[r] = static_cast<int32_t>(min(len, static_cast<int64_t>(INT32_MAX)));
            A.q_start[r] = static_cast<int32_t>(min(row0, static_cast<int64_t>(A.max_tokens)));
            if (len > (static_cast<int64_t>(A.max_pages) << shift)) bad |= DF11_DEV_ERR_PAGES;
        }
        __syncthreads();
        if (t >= rows && t < rows + all_rows && t < A.max_tokens) {
            int i = 0;  // the last request that starts at or before t: the one with rows there
#pragma unroll
            for (int step = kExtendThreads / 2; step; step >>= 1)
                if (i + step < cnt && s_row[i + step] <= t) i += step;
            const int64_t pos = s_kv[i] + (t - s_row[i]);
            const int64_t pg = pos >> shift;
            int32_t id = -1;
            if (pg < A.max_pages) {
                int32_t *entry = A.block_table + static_cast<int64_t>(base + i) * A.max_pages + pg;
                const int64_t held = (static_cast<int64_t>(s_kv[i]) + mask) >> shift;
                if (pg < held) {
                    id = *entry;
                } else {
                    const int64_t taken = s_page[i] + pg - held;
                    if (taken < n_free) id = A.free_pages[n_free - 1 - taken];
                    if ((pos & mask) == 0) *entry = id;
                }
            }
            if (id < 0) bad |= DF11_DEV_ERR_PAGES;
            A.slots[t] = id < 0 ? -1 : (static_cast<int64_t>(id) << shift) + (pos & mask);
            A.positions[t] = static_cast<int32_t>(min(pos, static_cast<int64_t>(INT32_MAX)));
        }
        if (first && rows + all_rows > A.max_tokens) {
            for (int i = 0; i < cnt; ++i) {
                const int64_t held = (static_cast<int64_t>(s_kv[i]) + mask) >> shift;
                const int64_t end = min((s_kv[i] + static_cast<int64_t>(max(A.new_lens[base + i], 0)) + mask) >> shift, room);
                // page p starts at row s_row + (p << shift) - s_kv; the first such row that is cut off
                const int64_t cut = (A.max_tokens - s_row[i] + s_kv[i] + mask) >> shift;
                for (int64_t pg = max(held, cut) + tid; pg < end; pg += kExtendThreads) {
                    const int64_t taken = s_page[i] + pg - held;
                    A.block_table[static_cast<int64_t>(base + i) * A.max_pages + pg] =
                        taken < n_free ? A.free_pages[n_free - 1 - taken] : -1;
                }
            }
        }
        rows += all_rows;
        pages += all_pages;
        __syncthreads();
    }
    if (t >= rows && t < A.max_tokens) {  // padding
        A.slots[t] = -1;
        A.positions[t] = 0;
    }
    if (first && tid == 0) {
        A.q_start[A.n_reqs] = static_cast<int32_t>(min(rows, static_cast<int64_t>(A.max_tokens)));
        *A.n_free_out = static_cast<int32_t>(max(n_free - pages, static_cast<int64_t>(0)));
        if (rows > A.max_tokens) bad |= DF11_DEV_ERR_AUX;
        if (pages > n_free) bad |= DF11_DEV_ERR_PAGES;
    }
    flag(err, bad);
}

// ------------------------------------------------------------------ norm and rotation

// A CTA takes a token, head_dim / 8 lanes a head, 8 elements (4 pairs) each.
// The 64-bit angle and the sincos of a pair are paid once per token, while the
// heads' loads are on their way.  The pass reads each element once and writes
// it once; nothing else goes to memory.  8191 tokens of 32 + 8 heads of 128 in
// BF16 take 40 us, 4.1 TB/s, bound by instructions (69 % of the issue slots; 35
// us without norm and sine); 16 tokens 2.1 us.  A warp per token, which makes the
// factors once, took 39 to 45 us for 2 to 5 heads in flight, and 2.3 for 16.
constexpr int kRopeThreads = 128;
constexpr int kRopeBatch = 5;  // heads whose loads a thread has in flight
// CTAs (token, group of heads) up to which a token's heads are shared out: some 7
// for each of a B200's 148 multiprocessors, about what is resident at a time.
// Shared out and not, FP32 with norm: 32 + 8 heads of 128 (5 groups) 16 tokens 2.1
// and 3.5 us, 200 tokens 3.9 and 4.1, 250 4.1 and 4.1, 300 4.8 and 4.3; of 64 (3
// groups) 200 tokens 2.6 and 2.9, 300 3.5 and 3.1; 16 + 8 heads of 256 (6 groups)
// 150 tokens 3.8 and 4.6, 200 4.2 and 4.7, 300 5.3 and 4.9.
constexpr int kRopeGroupedCtas = 7 * 148;

// Four elements as they lie in memory, and as floats.
template <bool FP32>
struct Four;
template <>
struct Four<true> {
    float4 a;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    }
    __device__ __forceinline__ void get(float *v) const { v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w; }
};
template <>
struct Four<false> {
    uint2 a;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        a = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    }
    __device__ __forceinline__ void get(float *v) const {
        v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xFFFF0000u);
        v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xFFFF0000u);
    }
};

__device__ __forceinline__ void store4(void *p, int64_t i, const float *v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t *>(&a);
    o.y = *reinterpret_cast<const uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = o;
}

template <bool FP32, int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const df11_qk_norm_rope_args A) {
    constexpr int L = D / 8;                     // lanes of a head
    constexpr int kHeads = kRopeThreads / L;     // heads the CTA holds at a time
    const int64_t t = blockIdx.x;
    const int j = threadIdx.x % L, half = A.rot_dim / 2;
    // the thread's elements: 4 at oa, 4 at ob.  Halves layout: elements 4j ..
    // of both halves while those are rotated, else 8 consecutive ones
    // (rot_dim is a multiple of 8, so the two meet at element 8j = rot_dim)
    const bool rotated = 4 * j < half;
    const bool split = rotated && !INTER;
    const int oa = split ? 4 * j : 8 * j, ob = split ? 4 * j + half : 8 * j + 4;
    const uint32_t group = (L == 32 ? 0xFFFFFFFFu : (1u << (L % 32)) - 1u) << (threadIdx.x & 31 & ~(L - 1));
    const int heads = A.q.n_heads + A.k.n_heads;
    const int h0 = blockIdx.y * kHeads + threadIdx.x / L, dh = gridDim.y * kHeads;
    // a batch of heads at a time, its loads in flight together, the first
    // batch's while the angles are made
    Four<FP32> xa[kRopeBatch], xb[kRopeBatch];
    auto side = [&](int h, int64_t &hd) -> const df11_rope_side & {
        const bool is_k = h >= A.q.n_heads;
        hd = static_cast<int64_t>(is_k ? h - A.q.n_heads : h) * D;
        return is_k ? A.k : A.q;
    };
    auto fetch = [&](int hb) {
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            const int h = hb + b * dh;
            if (h >= heads) break;
            int64_t hd;
            const df11_rope_side &S = side(h, hd);
            const int64_t at = t * static_cast<int64_t>(S.token_stride) + hd;
            xa[b].load(S.x, at + oa);
            xb[b].load(S.x, at + ob);
        }
    };
    fetch(h0);
    // a thread per pair; the heads' threads read them from shared memory
    __shared__ __align__(16) float s_cos[D / 2], s_sin[D / 2];
    for (int p = threadIdx.x; p < half; p += kRopeThreads) {
        // in half turns, reduced to [-1, 1] in 64 bits: what 32 bits then
        // round is the remainder, however far the position
        double x = A.positions[t] * A.inv_freq[p] * 0.31830988618379067154;
        x -= 2.0 * rint(0.5 * x);
        sincospif(static_cast<float>(x), &s_sin[p], &s_cos[p]);
    }
    Four<false> wq[2] = {}, wk[2] = {};
    if (A.q.weight) wq[0].load(A.q.weight, oa), wq[1].load(A.q.weight, ob);
    if (A.k.weight) wk[0].load(A.k.weight, oa), wk[1].load(A.k.weight, ob);
    __syncthreads();
    float cs[4] = {}, sn[4] = {};
    if (rotated) {
        Four<true> c, s;
        c.load(s_cos, 4 * j);
        s.load(s_sin, 4 * j);
        c.get(cs);
        s.get(sn);
    }
    for (int hb = h0; hb < heads; hb += kRopeBatch * dh) {
        if (hb != h0) fetch(hb);
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
            const int h = hb + b * dh;
            if (h >= heads) break;
            const bool is_k = h >= A.q.n_heads;
            int64_t hd;
            const df11_rope_side &S = side(h, hd);
            float v[8];
            xa[b].get(v);
            xb[b].get(v + 4);
            if (S.weight) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss += v[i] * v[i];
#pragma unroll
                for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                const float inv = 1.0f / sqrtf(ss * (1.0f / D) + A.eps);
                float w[8];
                (is_k ? wk[0] : wq[0]).get(w);
                (is_k ? wk[1] : wq[1]).get(w + 4);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
            }
            if (rotated) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float &a = v[INTER ? 2 * i : i], &c = v[INTER ? 2 * i + 1 : i + 4];
                    const float ra = a * cs[i] - c * sn[i];
                    c = c * cs[i] + a * sn[i];
                    a = ra;
                }
            }
            const int64_t to = t * static_cast<int64_t>(S.out_token_stride) + hd;
            store4(S.out, to + oa, v);
            store4(S.out, to + ob, v + 4);
        }
    }
}

template <int D>
void launch_rope(const df11_qk_norm_rope_args &a, dim3 grid, cudaStream_t s) {
    if (a.dtype == DF11_FP32)
        a.interleaved ? qk_norm_rope_kernel<true, D, true><<<grid, kRopeThreads, 0, s>>>(a)
                      : qk_norm_rope_kernel<true, D, false><<<grid, kRopeThreads, 0, s>>>(a);
    else
        a.interleaved ? qk_norm_rope_kernel<false, D, true><<<grid, kRopeThreads, 0, s>>>(a)
                      : qk_norm_rope_kernel<false, D, false><<<grid, kRopeThreads, 0, s>>>(a);
}

}  // namespace

LaunchStatus launch_kv_extend(const df11_kv_extend_args &a, int *err, cudaStream_t s) {
    if (a.n_reqs > INT_MAX - kExtendThreads) return LaunchStatus::kUnsupported;  // a tile past them would pass 31 bits
    int shift = 0;
    while ((1 << shift) < a.page_size) ++shift;
    const unsigned grid = a.max_tokens > 0 ? (static_cast<unsigned>(a.max_tokens) + kExtendThreads - 1) / kExtendThreads : 1;
    kv_extend_kernel<<<grid, kExtendThreads, 0, s>>>(a, shift, err);
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

LaunchStatus launch_qk_norm_rope(const df11_qk_norm_rope_args &args, cudaStream_t s) {
    df11_qk_norm_rope_args a = args;
    for (df11_rope_side *side : {&a.q, &a.k})
        if (side->n_heads == 0) *side = {};  // nothing of an absent side is read, nor are its weights
    const int heads = a.q.n_heads + a.k.n_heads, per = kRopeThreads / (a.head_dim / 8);
    // few tokens: a CTA per token and group of heads, so that every element
    // has its own thread at once; many: one CTA per token, which makes the
    // angles once for all heads
    const int groups = (heads + per - 1) / per;
    const dim3 grid(a.n_tokens, static_cast<int64_t>(a.n_tokens) * groups <= kRopeGroupedCtas ? groups : 1);
    switch (a.head_dim) {
        case 64: launch_rope<64>(a, grid, s); break;
        case 128: launch_rope<128>(a, grid, s); break;
        case 256: launch_rope<256>(a, grid, s); break;
        default: return LaunchStatus::kUnsupported;
    }
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

}  // namespace df11
