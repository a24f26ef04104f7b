// kv_attention.hip -- attention of a step's queries over the paged NVFP4
// cache.
#include "kv.hpp"

namespace nvfp4 {

size_t kv_attention_workspace(const nvfp4_kv_attention_args&) { return 0; }

// One wavefront per query row (token, head).  64 keys at a time: each lane
// takes one key's dot product with the row in LDS, the running maximum and
// sum of the softmax are kept per row, then each lane adds the weighted
// values of its D / 64 value pairs.
template <int D>
__global__ void __launch_bounds__(64) kv_attention_kernel(nvfp4_kv_attention_args a) {
  __shared__ float q[D];
  __shared__ float p[64];
  __shared__ int64_t at[64];  // page * kv_heads + head of the tile's keys, -1: not attended
  const nvfp4_kv_cache& c = a.cache;
  const int lane = threadIdx.x;
  const int64_t token = blockIdx.x / a.q_heads;
  const int h = (int)(blockIdx.x - token * a.q_heads), kvh = h / (a.q_heads / c.kv_heads);
  // the request of this row
  int64_t len = 0, pos = -1;
  int64_t b = -1;
  if (!a.cu_q) {
    b = token;
    len = a.seq_lens[b];
    pos = len - 1;
  } else {
    for (int64_t i = 0; i < a.batch; ++i)
      if (token >= a.cu_q[i] && token < a.cu_q[i + 1]) {
        b = i;
        len = a.seq_lens[b];
        pos = len - (a.cu_q[i + 1] - token);
        break;
      }
  }
  const int shift = __builtin_ctz((unsigned)c.page_size);
  const int64_t room = a.table_width << shift;
  const int64_t hi0 = len < room ? len : room;
  const int64_t hi = a.causal ? (hi0 < pos + 1 ? hi0 : pos + 1) : hi0;
  int64_t lo = a.window > 0 ? pos - a.window + 1 : 0;
  lo = lo < 0 ? 0 : lo;
  for (int i = lane; i < D; i += 64)
    q[i] = __uint_as_float((uint32_t)a.q[token * a.q_stride + (int64_t)h * D + i] << 16);
  const float ks = outer_alpha(c.k_amax[kvh], c.global_fp8_max) * a.scale;
  float m = -__builtin_inff(), l = 0.0f, o[D / 32] = {};
  __syncthreads();
  for (int64_t k0 = lo; k0 < hi; k0 += 64) {
    const int64_t key = k0 + lane;
    float s = -__builtin_inff();
    int64_t ph = -1;
    if (key < hi) {
      const int64_t page = a.block_table[b * a.table_width + (key >> shift)];
      if (page >= 0 && page < c.num_pages) {
        ph = page * c.kv_heads + kvh;
        const KvAddr k = {ph, (int)(key & (c.page_size - 1)), c.page_size, D};
        const uint32_t* w = reinterpret_cast<const uint32_t*>(c.k_codes + k.k_code());
        const uint8_t* sc = c.k_scales + k.k_scale();
        float dot = 0.0f;
        for (int i = 0; i < D / 8; ++i) {
          float v[8];
          e2m1_unpack8(w[i], v);
          float part = 0.0f;
          for (int j = 0; j < 8; ++j) part = __builtin_fmaf(v[j], q[8 * i + j], part);
          dot = __builtin_fmaf(part, decode_scale(FMT_E4M3, sc[i / 2]), dot);
        }
        s = dot * ks;
      }
    }
    const bool any = ph >= 0;
    float mt = s;
    for (int d = 1; d < 64; d <<= 1) mt = __builtin_fmaxf(mt, __shfl_xor(mt, d));
    const float mn = __builtin_fmaxf(m, mt);
    const float base = mn == -__builtin_inff() ? 0.0f : mn;
    const float e = any ? __expf(s - base) : 0.0f;
    float lt = e;
    for (int d = 1; d < 64; d <<= 1) lt += __shfl_xor(lt, d);
    const float keep = m == -__builtin_inff() ? 0.0f : __expf(m - base);
    l = l * keep + lt;
    m = mn;
    __syncthreads();
    p[lane] = e;
    at[lane] = ph;
    __syncthreads();
    for (int i = 0; i < D / 32; ++i) o[i] *= keep;
    const int n = (int)(hi - k0 < 64 ? hi - k0 : 64);
    for (int j = 0; j < n; ++j) {
      if (at[j] < 0) continue;
      const KvAddr k = {at[j], (int)((k0 + j) & (c.page_size - 1)), c.page_size, D};
      for (int i = 0; i < (D + 127) / 128; ++i) {
        const int e2 = 2 * (lane + 64 * i);  // first value of the pair
        if (e2 >= D) break;
        const f32x2 v = NVFP4_DEC_PK_FP4((uint32_t)c.v_codes[k.v_code() + 8 * (e2 / 2)], 0);
        const float f = decode_scale(FMT_E4M3, c.v_scales[k.v_scale() + 8 * (e2 / 16)]);
        o[2 * i] = __builtin_fmaf(p[j], v[0] * f, o[2 * i]);
        o[2 * i + 1] = __builtin_fmaf(p[j], v[1] * f, o[2 * i + 1]);
      }
    }
    __syncthreads();
  }
  const float va = outer_alpha(c.v_amax[kvh], c.global_fp8_max);
  const bool empty = m == -__builtin_inff() && l == 0.0f;
  const float inv = empty ? 0.0f : va / l;
  uint16_t* out = a.out + (token * a.q_heads + h) * D;
  for (int i = 0; i < (D + 127) / 128; ++i) {
    const int e2 = 2 * (lane + 64 * i);
    if (e2 >= D) break;
    reinterpret_cast<uint32_t*>(out)[e2 / 2] = empty ? 0u : bf16_pair(o[2 * i] * inv, o[2 * i + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[token * a.q_heads + h] = empty ? -__builtin_inff() : m + __logf(l);
}

hipError_t launch_kv_attention(const nvfp4_kv_attention_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.tokens * a.q_heads));
  switch (a.cache.head_dim) {
    case 64: hipLaunchKernelGGL(kv_attention_kernel<64>, grid, dim3(64), 0, s, a); break;
    case 128: hipLaunchKernelGGL(kv_attention_kernel<128>, grid, dim3(64), 0, s, a); break;
    case 192: hipLaunchKernelGGL(kv_attention_kernel<192>, grid, dim3(64), 0, s, a); break;
    default: hipLaunchKernelGGL(kv_attention_kernel<256>, grid, dim3(64), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
