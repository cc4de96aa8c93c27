// kv4_attention.cu -- attention over the paged 4-bit key/value cache, the
// cache decoded on chip.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "df11.h"
#include "kv4.cuh"
#include "serve.h"

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
};

__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float &lo, float &hi) {
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
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
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int r = threadIdx.x; r < A.n_reqs; r += 128)
            if (A.q_start[r] < 0 || A.q_start[r + 1] < A.q_start[r] || A.q_start[r + 1] > A.n_tokens ||
                A.q_start[r + 1] - A.q_start[r] > A.max_q_len)
                if (P.err) atomicOr(P.err, static_cast<int>(DF11_DEV_ERR_AUX));
    // the last request that starts at or before row t
    int lo = 0, hi = A.n_reqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (A.q_start[mid] <= t ? lo : hi) = mid;
    }
    const int q0 = A.q_start[lo], q1 = A.q_start[lo + 1];
    if (t < q0 || t >= q1) return;
    if (q0 < 0 || q1 > A.n_tokens || q1 - q0 > A.max_q_len) return;
    int64_t kv = max(A.kv_lens[lo], 0);
    const int64_t cap = static_cast<int64_t>(A.max_pages) << P.page_shift;
    const int64_t pos = kv - (q1 - q0) + (t - q0);
    int64_t j0 = 0, j1 = A.causal ? min(pos + 1, kv) : kv;
    if (A.window) j0 = max(j0, pos + 1 - A.window);
    if (kv > cap) bad |= DF11_DEV_ERR_PAGES;
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
    return P;
}

}  // namespace

LaunchStatus kv4_attention_workspace(const df11_kv4_cache &, const df11_kv4_attention_args &, uint64_t *bytes) {
    *bytes = 16;
    return LaunchStatus::kOk;
}

LaunchStatus launch_kv4_attention(const df11_kv4_cache &c, const df11_kv4_attention_args &a, int *err,
                                  cudaStream_t s) {
    const AttnParams P = attn_params(c, a, err);
    const dim3 grid(a.n_tokens, a.n_q_heads);
    if (c.head_dim == 128) attention_rows_kernel<128><<<grid, 128, 0, s>>>(P);
    else attention_rows_kernel<64><<<grid, 128, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

}  // namespace df11
