// serve.h -- host entry points of the serving operators: the step's pages and
// slots (serve.cu), norm and rotation of queries and keys (serve.cu), the
// 4-bit key/value cache (kv4.cu) and the attention over it (kv4_attention.cu).
// Every argument was checked by the caller (capi.cpp).
#pragma once

#include <cuda_runtime_api.h>

#include <cstdint>

#include "df11.h"
#include "launch.h"

namespace df11 {

constexpr int kKv4Group = 16;  // elements that share a scale

// One head's block of a page (layout in df11.h): byte offsets of its sections.
struct Kv4Block {
    uint32_t k_codes, k_scales, v_codes, v_scales, bytes;
};

#ifdef __CUDACC__
__host__ __device__
#endif
inline constexpr Kv4Block kv4_block(uint32_t page_size, uint32_t head_dim) {
    const uint32_t codes = page_size * head_dim / 2, scales = page_size * head_dim / kKv4Group;
    return Kv4Block{0, codes, codes + scales, 2 * codes + scales, 2 * (codes + scales)};
}

inline bool kv4_supported(int page_size, int head_dim) {
    return (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128) &&
           (head_dim == 64 || head_dim == 128);
}

LaunchStatus launch_kv_extend(const df11_kv_extend_args &a, int *err, cudaStream_t s);
LaunchStatus launch_qk_norm_rope(const df11_qk_norm_rope_args &a, cudaStream_t s);
LaunchStatus launch_kv4_append(const df11_kv4_cache &c, const void *k, uint64_t k_stride, const void *v,
                               uint64_t v_stride, const int64_t *slots, int n_tokens, bool fp32, int *err,
                               cudaStream_t s);
LaunchStatus launch_kv4_gather(const df11_kv4_cache &c, const int64_t *slots, int n_tokens, void *k_out, void *v_out,
                               bool fp32, int *err, cudaStream_t s);
LaunchStatus kv4_attention_workspace(const df11_kv4_cache &c, const df11_kv4_attention_args &a, uint64_t *bytes);
LaunchStatus launch_kv4_attention(const df11_kv4_cache &c, const df11_kv4_attention_args &a, int *err, cudaStream_t s);

}  // namespace df11
