// kv.hpp -- the key/value-cache operators' launchers and the device helpers
// they share.
#pragma once

#include <type_traits>

#include "../../include/nvfp4.h"
#include "common.hpp"
#include "device.hpp"

namespace nvfp4 {

hipError_t launch_kv_plan(const nvfp4_kv_plan_args& a, hipStream_t s);
hipError_t launch_qk_norm_rope(const nvfp4_qk_args& a, hipStream_t s);
hipError_t launch_qk_norm_rope_bwd(const nvfp4_qk_args& a, const uint16_t* gq, int64_t gq_stride,
                                   const uint16_t* gk, int64_t gk_stride, float* dqw, float* dkw,
                                   uint8_t* ws, hipStream_t s);
size_t qk_norm_rope_bwd_workspace(int head_dim);
hipError_t launch_kv_append(const nvfp4_kv_append_args& a, hipStream_t s);
hipError_t launch_kv_read(const nvfp4_kv_cache& c, const int64_t* slots, int64_t tokens,
                          uint16_t* k_out, uint16_t* v_out, hipStream_t s);
constexpr int64_t kAttnMaxGroups = (1 << 24) - 1;

// Launch shape of an attention call, from its sizes alone.
struct AttnPlan {
  int nq;           // 16-row tiles of a wavefront
  bool rows_split;  // wavefronts take rows of their own (else every fourth key tile)
  int rows;         // rows of a workgroup
  int splits;       // most workgroups over one tile's keys
  bool join;        // pieces are joined in the same launch
  int chunk;        // keys a workgroup is meant to take
  int64_t tiles;    // row tiles over all requests, at most
  int64_t grid;
  size_t bytes;     // of workspace
};

AttnPlan kv_attention_plan(const nvfp4_kv_attention_args& a);
hipError_t launch_kv_attention(const nvfp4_kv_attention_args& a, const AttnPlan& p, hipStream_t s);

// Byte offsets of one token's codes and scales of a head.  page < 2^31,
// heads <= 2^10, page_size <= 2^10 and D/2 <= 2^7: the products stay below
// 2^58, in 64 bits.
struct KvAddr {
  int64_t page_heads;  // page * kv_heads + head
  int off, page_size, D;
  __device__ __forceinline__ int64_t k_code() const { return (page_heads * page_size + off) * (D / 2); }
  __device__ __forceinline__ int64_t k_scale() const { return (page_heads * page_size + off) * (D / 16); }
  // of byte j of the token: + 8 * j
  __device__ __forceinline__ int64_t v_code() const {
    return (page_heads * page_size + (off & ~7)) * (D / 2) + (off & 7);
  }
  __device__ __forceinline__ int64_t v_scale() const {
    return (page_heads * page_size + (off & ~7)) * (D / 16) + (off & 7);
  }
};

// two binary32 values -> two bf16 patterns, nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

}  // namespace nvfp4
