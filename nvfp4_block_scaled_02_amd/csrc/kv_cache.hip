// kv_cache.hip -- writing a step's keys and values into the paged NVFP4 cache
// (with the norm and rotation of queries and keys in the same pass), and
// reading them back.
#include "qk_row.hpp"

namespace nvfp4 {

// Value of lane i of the quad (a compile-time i).
template <int I>
__device__ __forceinline__ float quad_lane(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), I * 0x55, 0xF, 0xF, false));
}

// Encodes the 16-value blocks that a quad of lanes holds, one per group (x[0
// .. 3] group 0, x[4 .. 7] group 1): bits 0 .. 15 of codes[g] are the lane's
// four nibbles, scale[g] the block's byte.  The steps are those of
// nvfp4_quantize in their order (fmaf chain per four values, then (P0 + P1) +
// (P2 + P3): lane pairs add in that order).  All lanes of the quad call it.
template <int SELECT>
__device__ __forceinline__ void quad_quantize(const float (&x)[8], const TensorScale& ts,
                                              uint32_t (&codes)[2], uint32_t (&scale)[2]) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float* v = x + 4 * g;
    float a = __builtin_elementwise_maximum(
        __builtin_elementwise_maximum(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])),
        __builtin_elementwise_maximum(__builtin_fabsf(v[2]), __builtin_fabsf(v[3])));
    a = __builtin_elementwise_maximum(a, __uint_as_float(xor1_u32(__float_as_uint(a))));
    a = __builtin_elementwise_maximum(a, __uint_as_float(xor2_u32(__float_as_uint(a))));
    const bool nan = ts.nan || a != a;
    auto encode = [&](const f32x2& t) {
      uint32_t w = NVFP4_CVT_PK_FP4(0u, v[0] * t[1], v[1] * t[1], 0);
      return NVFP4_CVT_PK_FP4(w, v[2] * t[1], v[3] * t[1], 1) & 0xFFFFu;
    };
    if constexpr (SELECT == SELECT_6) {
      const uint32_t c6 = e4m3_encode_pair(a * ts.k6, 0.0f) & 0xFFu;
      codes[g] = encode(scale_entry(FMT_E4M3, c6, ts.alpha));
      scale[g] = c6;
    } else {
      const uint32_t cc = e4m3_encode_pair(a * ts.k6, a * ts.k4);
      const f32x2 t6 = scale_entry(FMT_E4M3, cc & 0xFFu, ts.alpha);
      const f32x2 t4 = scale_entry(FMT_E4M3, cc >> 8, ts.alpha);
      const uint32_t w6 = encode(t6), w4 = encode(t4);
      auto error = [&](uint32_t w, float S) {
        const f32x2 q0 = NVFP4_DEC_PK_FP4(w, 0), q1 = NVFP4_DEC_PK_FP4(w, 1);
        float d = __builtin_fmaf(-q0[0], S, v[0]), p = __builtin_fmaf(d, d, 0.0f);
        d = __builtin_fmaf(-q0[1], S, v[1]); p = __builtin_fmaf(d, d, p);
        d = __builtin_fmaf(-q1[0], S, v[2]); p = __builtin_fmaf(d, d, p);
        d = __builtin_fmaf(-q1[1], S, v[3]); p = __builtin_fmaf(d, d, p);
        p = p + __uint_as_float(xor1_u32(__float_as_uint(p)));
        return p + __uint_as_float(xor2_u32(__float_as_uint(p)));
      };
      const bool four = error(w4, t4[0]) < error(w6, t6[0]);
      codes[g] = four ? w4 : w6;
      scale[g] = four ? cc >> 8 : cc & 0xFFu;
    }
    if (nan) {
      codes[g] = 0;
      scale[g] = 0x7Fu;
    }
  }
}

// Heads of a token: queries (normed, rotated, returned), keys (normed,
// rotated, quantized), values (quantized).
template <int LPH, int PAIRS, int SELECT>
__global__ void __launch_bounds__(kRowThreads)
kv_append_kernel(nvfp4_kv_append_args p, int64_t tasks, int per_token) {
  const nvfp4_qk_args& a = p.qk;
  const nvfp4_kv_cache& c = p.cache;
  const int D = a.head_dim;
  const RowMap<LPH> m(D, a.rot_dim, PAIRS);
  const int heads = a.q_heads + 2 * a.k_heads;
  const double inv_d = 1.0 / D;
  const int64_t slots_end = c.num_pages * c.page_size;
  const int shift = __builtin_ctz((unsigned)c.page_size);
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < tasks; w += (int64_t)gridDim.x * 4) {
    const RowTask t = row_task<LPH>(w, per_token);
    const bool isq = t.head < a.q_heads, isv = t.head >= a.q_heads + a.k_heads;
    const int h = isq ? t.head : isv ? t.head - a.q_heads - a.k_heads : t.head - a.q_heads;
    RowMap<LPH> mm = m;
    mm.active = m.active && t.head < heads;
    const int64_t at = (int64_t)h * D;
    float x[8];
    row_load((isq ? a.q + t.token * a.q_stride : isv ? p.v + t.token * p.v_stride
                                                     : a.k + t.token * a.k_stride) + at, mm, x);
    if (!isv) {
      const RowAngles g = row_angles(a, mm, t.token);
      uint2 o0, o1;
      row_norm_rope<LPH, PAIRS>(x, mm, isq ? a.q_weight : a.k_weight, a.eps, inv_d, g, o0, o1);
      if (isq) row_store(a.q_out + t.token * a.q_out_stride + at, mm, o0, o1);
      x[0] = bf16_lo(o0.x); x[1] = bf16_hi(o0.x); x[2] = bf16_lo(o0.y); x[3] = bf16_hi(o0.y);
      x[4] = bf16_lo(o1.x); x[5] = bf16_hi(o1.x); x[6] = bf16_lo(o1.y); x[7] = bf16_hi(o1.y);
    }
    // the lanes of a head leave together, and quads exchange inside a head
    if (isq || t.head >= heads) continue;
    const int64_t slot = p.slots[t.token];
    if (slot < 0 || slot >= slots_end) continue;
    const TensorScale ts = tensor_scale((isv ? c.v_amax : c.k_amax)[h], c.global_fp8_max);
    uint32_t codes[2], scale[2];
    quad_quantize<SELECT>(x, ts, codes, scale);
    if (!mm.active) continue;
    const KvAddr k = {(slot >> shift) * c.kv_heads + h, (int)(slot & (c.page_size - 1)), c.page_size, D};
    if (!isv) {
      uint8_t* kc = c.k_codes + k.k_code();
      *reinterpret_cast<uint16_t*>(kc + mm.e0 / 2) = (uint16_t)codes[0];
      *reinterpret_cast<uint16_t*>(kc + mm.e1 / 2) = (uint16_t)codes[1];
      if ((threadIdx.x & 3) == 0) {
        uint8_t* ks = c.k_scales + k.k_scale();
        ks[mm.e0 / 16] = (uint8_t)scale[0];
        ks[mm.e1 / 16] = (uint8_t)scale[1];
      }
    } else {
      uint8_t* vc = c.v_codes + k.v_code();
      vc[8 * (mm.e0 / 2)] = (uint8_t)codes[0];
      vc[8 * (mm.e0 / 2 + 1)] = (uint8_t)(codes[0] >> 8);
      vc[8 * (mm.e1 / 2)] = (uint8_t)codes[1];
      vc[8 * (mm.e1 / 2 + 1)] = (uint8_t)(codes[1] >> 8);
      if ((threadIdx.x & 3) == 0) {
        uint8_t* vs = c.v_scales + k.v_scale();
        vs[8 * (mm.e0 / 16)] = (uint8_t)scale[0];
        vs[8 * (mm.e1 / 16)] = (uint8_t)scale[1];
      }
    }
  }
}

template <int LPH, int PAIRS>
static hipError_t launch_append(const nvfp4_kv_append_args& a, hipStream_t s) {
  const int per_token = (a.qk.q_heads + 2 * a.qk.k_heads + 64 / LPH - 1) / (64 / LPH);
  const int64_t tasks = a.qk.tokens * per_token;
  if (a.select == NVFP4_SELECT_6)
    hipLaunchKernelGGL((kv_append_kernel<LPH, PAIRS, SELECT_6>), dim3(row_grid(tasks)),
                       dim3(kRowThreads), 0, s, a, tasks, per_token);
  else
    hipLaunchKernelGGL((kv_append_kernel<LPH, PAIRS, SELECT_4OVER6>), dim3(row_grid(tasks)),
                       dim3(kRowThreads), 0, s, a, tasks, per_token);
  return hipGetLastError();
}

template <int LPH>
static hipError_t launch_append(const nvfp4_kv_append_args& a, hipStream_t s) {
  return a.qk.pairs == NVFP4_PAIRS_HALVES ? launch_append<LPH, NVFP4_PAIRS_HALVES>(a, s)
                                          : launch_append<LPH, NVFP4_PAIRS_NEIGHBOURS>(a, s);
}

hipError_t launch_kv_append(const nvfp4_kv_append_args& a, hipStream_t s) {
  switch (lanes_per_head(a.qk.head_dim)) {
    case 8: return launch_append<8>(a, s);
    case 16: return launch_append<16>(a, s);
    default: return launch_append<32>(a, s);
  }
}

// ---------------------------------------------------------------- read
template <int LPH>
__global__ void __launch_bounds__(kRowThreads)
kv_read_kernel(nvfp4_kv_cache c, const int64_t* slots, int64_t tasks, int per_token,
               uint16_t* k_out, uint16_t* v_out) {
  const int D = c.head_dim;
  const RowMap<LPH> m(D, D, NVFP4_PAIRS_HALVES);
  const int first = k_out ? 0 : c.kv_heads, heads = v_out ? 2 * c.kv_heads : c.kv_heads;
  const int64_t slots_end = c.num_pages * c.page_size;
  const int shift = __builtin_ctz((unsigned)c.page_size);
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < tasks; w += (int64_t)gridDim.x * 4) {
    RowTask t = row_task<LPH>(w, per_token);
    t.head += first;
    if (t.head >= heads || !m.active) continue;
    const bool isv = t.head >= c.kv_heads;
    const int h = isv ? t.head - c.kv_heads : t.head;
    const int64_t slot = slots[t.token];
    uint32_t w0 = 0, w1 = 0, s0 = 0, s1 = 0;
    if (slot >= 0 && slot < slots_end) {
      const KvAddr k = {(slot >> shift) * c.kv_heads + h, (int)(slot & (c.page_size - 1)), c.page_size, D};
      if (!isv) {
        const uint8_t* kc = c.k_codes + k.k_code();
        const uint8_t* ks = c.k_scales + k.k_scale();
        w0 = *reinterpret_cast<const uint16_t*>(kc + m.e0 / 2);
        w1 = *reinterpret_cast<const uint16_t*>(kc + m.e1 / 2);
        s0 = ks[m.e0 / 16];
        s1 = ks[m.e1 / 16];
      } else {
        const uint8_t* vc = c.v_codes + k.v_code();
        const uint8_t* vs = c.v_scales + k.v_scale();
        w0 = vc[8 * (m.e0 / 2)] | (uint32_t)vc[8 * (m.e0 / 2 + 1)] << 8;
        w1 = vc[8 * (m.e1 / 2)] | (uint32_t)vc[8 * (m.e1 / 2 + 1)] << 8;
        s0 = vs[8 * (m.e0 / 16)];
        s1 = vs[8 * (m.e1 / 16)];
      }
    }
    const float alpha = outer_alpha((isv ? c.v_amax : c.k_amax)[h], c.global_fp8_max);
    // E2M1 x E4M3 is exact in binary32; times alpha rounds once
    const float f0 = decode_scale(FMT_E4M3, s0), f1 = decode_scale(FMT_E4M3, s1);
    const f32x2 a0 = NVFP4_DEC_PK_FP4(w0, 0), a1 = NVFP4_DEC_PK_FP4(w0, 1);
    const f32x2 b0 = NVFP4_DEC_PK_FP4(w1, 0), b1 = NVFP4_DEC_PK_FP4(w1, 1);
    uint2 o0 = make_uint2(bf16_pair(a0[0] * f0 * alpha, a0[1] * f0 * alpha),
                          bf16_pair(a1[0] * f0 * alpha, a1[1] * f0 * alpha));
    uint2 o1 = make_uint2(bf16_pair(b0[0] * f1 * alpha, b0[1] * f1 * alpha),
                          bf16_pair(b1[0] * f1 * alpha, b1[1] * f1 * alpha));
    if (slot < 0 || slot >= slots_end) o0 = o1 = make_uint2(0, 0);  // also under an unusable amax
    row_store((isv ? v_out : k_out) + (t.token * c.kv_heads + h) * D, m, o0, o1);
  }
}

template <int LPH>
static hipError_t launch_read(const nvfp4_kv_cache& c, const int64_t* slots, int64_t tokens,
                              uint16_t* k_out, uint16_t* v_out, hipStream_t s) {
  const int heads = ((k_out != nullptr) + (v_out != nullptr)) * c.kv_heads;
  const int per_token = (heads + 64 / LPH - 1) / (64 / LPH);
  const int64_t tasks = tokens * per_token;
  hipLaunchKernelGGL((kv_read_kernel<LPH>), dim3(row_grid(tasks)), dim3(kRowThreads), 0, s, c,
                     slots, tasks, per_token, k_out, v_out);
  return hipGetLastError();
}

hipError_t launch_kv_read(const nvfp4_kv_cache& c, const int64_t* slots, int64_t tokens,
                          uint16_t* k_out, uint16_t* v_out, hipStream_t s) {
  switch (lanes_per_head(c.head_dim)) {
    case 8: return launch_read<8>(c, slots, tokens, k_out, v_out, s);
    case 16: return launch_read<16>(c, slots, tokens, k_out, v_out, s);
    default: return launch_read<32>(c, slots, tokens, k_out, v_out, s);
  }
}

}  // namespace nvfp4
