// kv4.cu -- writing and reading the paged 4-bit key/value cache (layout and
// number format in df11.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "df11.h"
#include "kv4.cuh"
#include "serve.h"

namespace df11 {
namespace {

constexpr int kKv4Threads = 256;

struct Kv4Params {
    uint8_t *pages;
    uint64_t n_slots;
    uint32_t n_heads, page_shift;
    Kv4Block block;
    float k_scale, v_scale;
    const int64_t *slots;
    int32_t n_tokens;
    int *err;
    const void *k, *v;  // append: the rows written
    uint64_t k_stride, v_stride;
    void *k_out, *v_out;  // gather
};

// A thread handles 16 elements of one head of one token, of K (blockIdx.y 0)
// or V (1): one scale, 8 code bytes.  `u` numbers them so that neighbouring
// threads touch neighbouring bytes of the cache: K by block within the token
// (a head's row is contiguous), V by token within 4 (their 8-byte pieces are).
template <int D>
__device__ __forceinline__ void unit(const Kv4Params &P, bool is_v, uint64_t u, uint32_t &t, uint32_t &h, uint32_t &b) {
    constexpr uint32_t NB = D / kKv4Group;
    if (is_v) {
        const uint32_t c = static_cast<uint32_t>(u & 3u);
        const uint64_t w = u >> 2;
        b = static_cast<uint32_t>(w % NB);
        const uint64_t x = w / NB;
        h = static_cast<uint32_t>(x % P.n_heads);
        t = static_cast<uint32_t>(x / P.n_heads) * 4u + c;
    } else {
        b = static_cast<uint32_t>(u % NB);
        const uint64_t x = u / NB;
        h = static_cast<uint32_t>(x % P.n_heads);
        t = static_cast<uint32_t>(x / P.n_heads);
    }
}

// Places of the codes and the scale of block b of head h in slot `slot`.
template <int D>
__device__ __forceinline__ void place(const Kv4Params &P, bool is_v, uint64_t slot, uint32_t h, uint32_t b,
                                      uint8_t **codes, uint8_t **scale) {
    constexpr uint32_t NB = D / kKv4Group;
    const uint32_t off = static_cast<uint32_t>(slot) & ((1u << P.page_shift) - 1u);
    uint8_t *blk = P.pages + ((slot >> P.page_shift) * P.n_heads + h) * P.block.bytes;
    if (is_v) {
        *codes = blk + P.block.v_codes + (((off >> 2) * NB + b) * 4u + (off & 3u)) * 8u;
        *scale = blk + P.block.v_scales + (b << P.page_shift) + off;
    } else {
        *codes = blk + P.block.k_codes + (off * NB + b) * 8u;
        *scale = blk + P.block.k_scales + off * NB + b;
    }
}

// Slot of token t: false for a negative one, and (flagged) past the cache.
__device__ __forceinline__ bool slot_of(const Kv4Params &P, uint32_t t, uint64_t &slot) {
    const int64_t s = P.slots[t];
    if (s < 0) return false;
    slot = static_cast<uint64_t>(s);
    if (slot < P.n_slots) return true;
    if (P.err) atomicOr(P.err, static_cast<int>(DF11_DEV_ERR_PAGES));
    return false;
}

// The scale and the codes follow the definition step by step with IEEE
// division: a block's scale has 4 significant bits and an element 8, so
// quotients fall exactly on the borders between levels often, and a
// reciprocal's last bit would move them.
template <bool FP32, int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Params P) {
    const bool is_v = blockIdx.y;
    uint32_t t, h, b;
    unit<D>(P, is_v, static_cast<uint64_t>(blockIdx.x) * kKv4Threads + threadIdx.x, t, h, b);
    uint64_t slot;
    if (t >= static_cast<uint32_t>(P.n_tokens) || !slot_of(P, t, slot)) return;
    const uint64_t at = t * (is_v ? P.v_stride : P.k_stride) + h * D + b * kKv4Group;
    const void *src = is_v ? P.v : P.k;
    float x[2][8];
    if constexpr (FP32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(src) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(p + i);
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i / 2][4 * (i % 2) + j] = __bfloat162float(__float2bfloat16_rn(f[j]));
        }
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = __ldg(p + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][2 * j] = __uint_as_float(w[j] << 16);
                x[i][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    }
    float top = 0.0f;  // fmaxf leaves NaN out
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i / 8][i % 8]));
    const float g = is_v ? P.v_scale : P.k_scale;
    const uint32_t sb = f32_to_e4m3(fminf(__fdiv_rn(__fdiv_rn(top, 6.0f), g), 448.0f));
    const uint32_t sh = e4m3x2_to_f16x2(sb);
    float s;
    asm("cvt.f32.f16 %0, %1;" : "=f"(s) : "h"(static_cast<uint16_t>(sh)));
    const float step = s * g;
    uint2 codes = make_uint2(0u, 0u);
    if (step > 0.0f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i / 8][i % 8] = __fdiv_rn(x[i / 8][i % 8], step);
        codes = make_uint2(f32x8_to_e2m1(x[0]), f32x8_to_e2m1(x[1]));
    }
    uint8_t *cp, *sp;
    place<D>(P, is_v, slot, h, b, &cp, &sp);
    *reinterpret_cast<uint2 *>(cp) = codes;
    *sp = static_cast<uint8_t>(sb);
}

// level * s is exact in FP16 (2 and 4 significant bits, at most 6 * 448); the
// product with the cache's scale is rounded to FP32 and then to the output.
template <bool FP32, int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_gather_kernel(const Kv4Params P) {
    const bool is_v = blockIdx.y;
    uint32_t t, h, b;
    unit<D>(P, is_v, static_cast<uint64_t>(blockIdx.x) * kKv4Threads + threadIdx.x, t, h, b);
    void *dst = is_v ? P.v_out : P.k_out;
    uint64_t slot;
    if (!dst || t >= static_cast<uint32_t>(P.n_tokens) || !slot_of(P, t, slot)) return;
    uint8_t *cp, *sp;
    place<D>(P, is_v, slot, h, b, &cp, &sp);
    const uint2 codes = *reinterpret_cast<const uint2 *>(cp);
    const uint32_t s2 = e4m3x2_to_f16x2(*sp * 0x0101u);
    const float g = is_v ? P.v_scale : P.k_scale;
    float y[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t r[4];
        e2m1x8_to_f16(i ? codes.y : codes.x, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = f16x2_mul(r[j], s2);
            float lo, hi;
            asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                : "=f"(lo), "=f"(hi)
                : "r"(v));
            y[8 * i + 2 * j] = lo * g;
            y[8 * i + 2 * j + 1] = hi * g;
        }
    }
    const uint64_t at = (static_cast<uint64_t>(t) * P.n_heads + h) * D + b * kKv4Group;
    if constexpr (FP32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(dst) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    } else {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(y[8 * i + 2 * j], y[8 * i + 2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&p);
            }
            o[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

Kv4Params params(const df11_kv4_cache &c, const int64_t *slots, int n_tokens, int *err) {
    Kv4Params P{};
    P.pages = static_cast<uint8_t *>(c.pages);
    P.n_slots = c.n_pages * static_cast<uint64_t>(c.page_size);
    P.n_heads = static_cast<uint32_t>(c.n_heads);
    while ((1 << P.page_shift) < c.page_size) ++P.page_shift;
    P.block = kv4_block(c.page_size, c.head_dim);
    P.k_scale = c.k_scale;
    P.v_scale = c.v_scale;
    P.slots = slots;
    P.n_tokens = n_tokens;
    P.err = err;
    return P;
}

// units of K or V, the tokens rounded up to whole groups of 4
dim3 grid_of(const df11_kv4_cache &c, int n_tokens) {
    const uint64_t units = (static_cast<uint64_t>(n_tokens) + 3) / 4 * 4 * c.n_heads * (c.head_dim / kKv4Group);
    return dim3(static_cast<unsigned>((units + kKv4Threads - 1) / kKv4Threads), 2);
}

}  // namespace

LaunchStatus launch_kv4_append(const df11_kv4_cache &c, const void *k, uint64_t k_stride, const void *v,
                               uint64_t v_stride, const int64_t *slots, int n_tokens, bool fp32, int *err,
                               cudaStream_t s) {
    Kv4Params P = params(c, slots, n_tokens, err);
    P.k = k;
    P.v = v;
    P.k_stride = k_stride;
    P.v_stride = v_stride;
    const dim3 grid = grid_of(c, n_tokens);
    if (c.head_dim == 128)
        fp32 ? kv4_append_kernel<true, 128><<<grid, kKv4Threads, 0, s>>>(P)
             : kv4_append_kernel<false, 128><<<grid, kKv4Threads, 0, s>>>(P);
    else
        fp32 ? kv4_append_kernel<true, 64><<<grid, kKv4Threads, 0, s>>>(P)
             : kv4_append_kernel<false, 64><<<grid, kKv4Threads, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

LaunchStatus launch_kv4_gather(const df11_kv4_cache &c, const int64_t *slots, int n_tokens, void *k_out, void *v_out,
                               bool fp32, int *err, cudaStream_t s) {
    Kv4Params P = params(c, slots, n_tokens, err);
    P.k_out = k_out;
    P.v_out = v_out;
    const dim3 grid = grid_of(c, n_tokens);
    if (c.head_dim == 128)
        fp32 ? kv4_gather_kernel<true, 128><<<grid, kKv4Threads, 0, s>>>(P)
             : kv4_gather_kernel<false, 128><<<grid, kKv4Threads, 0, s>>>(P);
    else
        fp32 ? kv4_gather_kernel<true, 64><<<grid, kKv4Threads, 0, s>>>(P)
             : kv4_gather_kernel<false, 64><<<grid, kKv4Threads, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

}  // namespace df11
