// kv4.cu -- writing and reading the paged 4-bit key/value cache (layout and
// number format in df11.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "df11.h"
#include "kv4.cuh"
#include "packed.cuh"
#include "serve.h"

namespace df11 {
namespace {

// A CTA takes 4 tokens, a thread 16 elements of one of them at a time, of K
// and of V: one scale, 8 code bytes each, both loads in flight together.
// Neighbouring threads take the 4 tokens (whose 8-byte pieces of V codes and
// bytes of V scales are neighbours where the tokens are), then the blocks of a
// row, which are contiguous in the rows and, within a head, in the K codes.
// 16,384 tokens of 8 heads of 128 (86 MB each way) appended and then gathered
// take 33 us, 5.2 TB/s; each again and again, its data partly in L2, 16 and 13.
// Append is bound by latency and instructions (61 % of the issue slots, the
// quotients most of them).  CTAs of 128 threads took 0.7 us less of the two, and a
// step of 64 tokens 5.6 us, not 4.4.
constexpr int kKv4Threads = 256;
constexpr int kKv4Tokens = 4;

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
    float k_inv, v_inv;  // of the scales, correctly rounded; 0: far from 1
    uint64_t k_stride, v_stride;
    void *k_out, *v_out;  // gather
};

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

// Slot of token t: false past the tokens, for a negative one, and (flagged) past the cache.
__device__ __forceinline__ bool slot_of(const Kv4Params &P, int64_t t, uint64_t &slot) {
    if (t >= P.n_tokens) return false;
    const int64_t s = __ldg(P.slots + t);
    if (s < 0) return false;
    slot = static_cast<uint64_t>(s);
    if (slot < P.n_slots) return true;
    if (P.err) atomicOr(P.err, static_cast<int>(DF11_DEV_ERR_PAGES));
    return false;
}

// 32 bytes, a whole sector, in one instruction where the address allows it
// (rows need only be 16-byte aligned; where strides are multiples of 32 bytes the
// branch is the same for all threads).
__device__ __forceinline__ void load32(const void *p, uint32_t *w) {
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(static_cast<const uint4 *>(p)), b = __ldg(static_cast<const uint4 *>(p) + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
}

__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Sixteen elements as they lie in memory.
template <bool FP32>
struct Sixteen {
    uint32_t w[FP32 ? 16 : 8];
    __device__ __forceinline__ void load(const void *p, uint64_t i) {
        const uint8_t *q = static_cast<const uint8_t *>(p) + i * (FP32 ? 4 : 2);
#pragma unroll
        for (int j = 0; j < (FP32 ? 2 : 1); ++j) load32(q + 32 * j, w + 8 * j);
    }
    // as BF16 values
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < (FP32 ? 16 : 8); ++i) {
            if constexpr (FP32) {
                x[i] = __bfloat162float(__float2bfloat16_rn(__uint_as_float(w[i])));
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
};

// x / d correctly rounded, from r = 1 / d correctly rounded, by one residual
// step (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", theorem on division with a correct reciprocal), for
// |x / d| <= 8 and d well inside the exponent range.
__device__ __forceinline__ float quotient(float x, float d, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, d, x), r, q);
}

__device__ __forceinline__ uint64_t quotient2(uint64_t x, float d, float r) {
    const uint64_t r2 = pair(r, r), q = mul2(x, r2);
    return fma2(fma2(q, pair(-d, -d), x), r2, q);
}

// The scale and the codes follow the definition step by step with correctly
// rounded quotients: a block's scale has 4 significant bits and an element 8,
// so quotients fall exactly on the borders between levels often, and a
// reciprocal's last bit would move them.  rg is 1 / g correctly rounded, or 0
// where g is far from 1.  16,384 tokens of 8 heads of 128 took 34 us with a
// division for each quotient, 21 with divisions for the scale's two.
__device__ __forceinline__ void quantize(const float (&x)[16], float g, float rg, uint2 &codes, uint32_t &scale) {
    float top = 0.0f;  // NaN left out
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max3(top, fabsf(x[i]), fabsf(x[i + 1]));
    const float wanted = rg > 0.0f && top > 0x1p-60f && top < 0x1p60f
                             ? quotient(quotient(top, 6.0f, 1.0f / 6.0f), g, rg)
                             : __fdiv_rn(__fdiv_rn(top, 6.0f), g);
    scale = f32_to_e4m3(fminf(wanted, 448.0f));
    const uint32_t sh = e4m3x2_to_f16x2(scale);
    float s;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(s) : "r"(sh));
    const float step = s * g;
    codes = make_uint2(0u, 0u);
    if (!(step > 0.0f)) return;
    float y[2][8];
    if (step > 0x1p-100f && step < 0x1p100f) {
        const float r = __frcp_rn(step), most = 8.0f * step;
        if (top <= most) {
            // (a NaN beside them stays one, and its code is that of +6)
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const uint64_t q = quotient2(pair(x[i], x[i + 1]), step, r);
                y[i / 8][i % 8] = low(q), y[i / 8][i % 8 + 1] = high(q);
            }
        } else {
            // what saturates anyway is brought to 8 steps first; a NaN goes with the positive ones
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i / 8][i % 8] = quotient(fmaxf(fminf(x[i], most), -most), step, r);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i / 8][i % 8] = __fdiv_rn(x[i], step);
    }
    codes = make_uint2(f32x8_to_e2m1(y[0]), f32x8_to_e2m1(y[1]));
}

template <bool FP32, int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Params P) {
    constexpr uint32_t NB = D / kKv4Group;
    const uint32_t units = kKv4Tokens * NB * P.n_heads;
    for (uint32_t u = threadIdx.x; u < units; u += blockDim.x) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * kKv4Tokens + u % kKv4Tokens;
        const uint32_t hb = u / kKv4Tokens;  // block of the row
        if (t >= P.n_tokens) continue;
        // the row is on its way while its slot is read, for nothing if it has none
        Sixteen<FP32> rk, rv;
        rk.load(P.k, t * P.k_stride + hb * kKv4Group);
        rv.load(P.v, t * P.v_stride + hb * kKv4Group);
        uint64_t slot;
        if (!slot_of(P, t, slot)) continue;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
            float x[16];
            (is_v ? rv : rk).get(x);
            uint2 codes;
            uint32_t scale;
            quantize(x, is_v ? P.v_scale : P.k_scale, is_v ? P.v_inv : P.k_inv, codes, scale);
            uint8_t *cp, *sp;
            place<D>(P, is_v, slot, hb / NB, hb % NB, &cp, &sp);
            *reinterpret_cast<uint2 *>(cp) = codes;
            *sp = static_cast<uint8_t>(scale);
        }
    }
}

// level * s is exact in FP16 (2 and 4 significant bits, at most 6 * 448); the
// product with the cache's scale is rounded to FP32 and then to the output.
template <bool FP32, int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_gather_kernel(const Kv4Params P) {
    constexpr uint32_t NB = D / kKv4Group;
    const uint32_t units = kKv4Tokens * NB * P.n_heads;
    for (uint32_t u = threadIdx.x; u < units; u += blockDim.x) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * kKv4Tokens + u % kKv4Tokens;
        const uint32_t hb = u / kKv4Tokens;
        uint64_t slot;
        if (!slot_of(P, t, slot)) continue;
        uint2 codes[2];
        uint32_t scale[2];
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
            if (!(is_v ? P.v_out : P.k_out)) continue;
            uint8_t *cp, *sp;
            place<D>(P, is_v, slot, hb / NB, hb % NB, &cp, &sp);
            codes[is_v] = *reinterpret_cast<const uint2 *>(cp);
            scale[is_v] = *sp;
        }
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
            void *dst = is_v ? P.v_out : P.k_out;
            if (!dst) continue;
            const uint32_t s2 = e4m3x2_to_f16x2(scale[is_v] * 0x0101u);
            const float g = is_v ? P.v_scale : P.k_scale;
            float y[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t r[4];
                e2m1x8_to_f16(i ? codes[is_v].y : codes[is_v].x, r);
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
            const uint64_t at = (static_cast<uint64_t>(t) * P.n_heads * NB + hb) * kKv4Group;
            uint32_t w[FP32 ? 16 : 8];
#pragma unroll
            for (int i = 0; i < (FP32 ? 16 : 8); ++i) {
                if constexpr (FP32) {
                    w[i] = __float_as_uint(y[i]);
                } else {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t *>(&p);
                }
            }
            uint8_t *o = static_cast<uint8_t *>(dst) + at * (FP32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < (FP32 ? 2 : 1); ++i) store32(o + 32 * i, w + 8 * i);
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

unsigned ctas_of(int n_tokens) { return static_cast<unsigned>((static_cast<int64_t>(n_tokens) + kKv4Tokens - 1) / kKv4Tokens); }

// A thread per unit of the CTA's tokens, in whole warps, as far as they go.
unsigned threads_of(const df11_kv4_cache &c) {
    const unsigned units = kKv4Tokens * static_cast<unsigned>(c.n_heads) * (c.head_dim / kKv4Group);
    return units < kKv4Threads ? (units + 31) / 32 * 32 : kKv4Threads;
}

// 1 / g where the quotients by it need no special cases, else 0.
float inverse(float g) { return g > 0x1p-60f && g < 0x1p60f ? 1.0f / g : 0.0f; }

}  // namespace

LaunchStatus launch_kv4_append(const df11_kv4_cache &c, const void *k, uint64_t k_stride, const void *v,
                               uint64_t v_stride, const int64_t *slots, int n_tokens, bool fp32, int *err,
                               cudaStream_t s) {
    Kv4Params P = params(c, slots, n_tokens, err);
    P.k = k;
    P.k_inv = inverse(c.k_scale);
    P.v_inv = inverse(c.v_scale);
    P.v = v;
    P.k_stride = k_stride;
    P.v_stride = v_stride;
    const unsigned grid = ctas_of(n_tokens), threads = threads_of(c);
    if (c.head_dim == 128)
        fp32 ? kv4_append_kernel<true, 128><<<grid, threads, 0, s>>>(P)
             : kv4_append_kernel<false, 128><<<grid, threads, 0, s>>>(P);
    else
        fp32 ? kv4_append_kernel<true, 64><<<grid, threads, 0, s>>>(P)
             : kv4_append_kernel<false, 64><<<grid, threads, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

LaunchStatus launch_kv4_gather(const df11_kv4_cache &c, const int64_t *slots, int n_tokens, void *k_out, void *v_out,
                               bool fp32, int *err, cudaStream_t s) {
    Kv4Params P = params(c, slots, n_tokens, err);
    P.k_out = k_out;
    P.v_out = v_out;
    const unsigned grid = ctas_of(n_tokens), threads = threads_of(c);
    if (c.head_dim == 128)
        fp32 ? kv4_gather_kernel<true, 128><<<grid, threads, 0, s>>>(P)
             : kv4_gather_kernel<false, 128><<<grid, threads, 0, s>>>(P);
    else
        fp32 ? kv4_gather_kernel<true, 64><<<grid, threads, 0, s>>>(P)
             : kv4_gather_kernel<false, 64><<<grid, threads, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? LaunchStatus::kOk : LaunchStatus::kCuda;
}

}  // namespace df11
