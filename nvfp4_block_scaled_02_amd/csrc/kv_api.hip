// kv_api.hip -- the extern "C" entry points of the key/value-cache operators
// (include/nvfp4.h): host-side validation and dispatch.  Nothing here
// allocates device memory or synchronizes.
#include <math.h>

#include "kv.hpp"

namespace nvfp4 {

static bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
static bool given(const void* p, unsigned n) { return p != nullptr && aligned(p, n); }
static int status_of(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }
constexpr int64_t kMax32 = INT32_MAX;

// rows * cols of a strided tensor stay within NVFP4_MAX_ELEMENTS
static bool extent_ok(int64_t rows, int64_t stride) {
  return rows >= 0 && stride >= 0 && (stride == 0 || rows <= NVFP4_MAX_ELEMENTS / stride);
}

static int cache_ok(const nvfp4_kv_cache& c) {
  if (!given(c.k_codes, 16) || !given(c.k_scales, 16) || !given(c.v_codes, 16) ||
      !given(c.v_scales, 16) || !given(c.k_amax, 4) || !given(c.v_amax, 4))
    return NVFP4_ERR_INVALID;
  if (c.num_pages < 1 || c.num_pages > kMax32 || c.kv_heads < 1 || c.kv_heads > NVFP4_KV_MAX_HEADS)
    return NVFP4_ERR_INVALID;
  if (c.page_size < 8 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)))
    return NVFP4_ERR_INVALID;
  if (!(c.global_fp8_max > 0.0f) || isinf(c.global_fp8_max)) return NVFP4_ERR_INVALID;
  if (c.head_dim <= 0 || c.head_dim % 16) return NVFP4_ERR_INVALID;
  if (!extent_ok(c.num_pages, (int64_t)c.kv_heads * c.page_size * c.head_dim)) return NVFP4_ERR_INVALID;
  if (c.head_dim % 64 || c.head_dim > 256) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

// the rules of one side (queries or keys) of nvfp4_qk_args
static bool side_ok(const uint16_t* x, const uint16_t* out, int64_t tokens, int heads, int D,
                    int64_t stride, int64_t out_stride, const uint16_t* w) {
  if (!aligned(w, 8)) return false;
  if (heads == 0) return true;
  if (!extent_ok(tokens, stride) || !extent_ok(tokens, out_stride)) return false;
  if (stride < (int64_t)heads * D || out_stride < (int64_t)heads * D || stride % 4 || out_stride % 4)
    return false;
  return tokens == 0 || (given(x, 8) && given(out, 8));
}

static int qk_ok(const nvfp4_qk_args& a, bool k_out_used) {
  if (a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0 || a.q_heads > NVFP4_KV_MAX_HEADS ||
      a.k_heads > NVFP4_KV_MAX_HEADS || a.q_heads + a.k_heads == 0)
    return NVFP4_ERR_INVALID;
  if (a.head_dim <= 0 || a.head_dim % 16 || a.rot_dim < 0 || a.rot_dim > a.head_dim)
    return NVFP4_ERR_INVALID;
  if (a.pairs != NVFP4_PAIRS_HALVES && a.pairs != NVFP4_PAIRS_NEIGHBOURS) return NVFP4_ERR_INVALID;
  if (!(a.eps >= 0.0f) || isinf(a.eps)) return NVFP4_ERR_INVALID;
  if (!side_ok(a.q, a.q_out, a.tokens, a.q_heads, a.head_dim, a.q_stride, a.q_out_stride, a.q_weight))
    return NVFP4_ERR_INVALID;
  if (!side_ok(a.k, k_out_used ? a.k_out : a.k, a.tokens, a.k_heads, a.head_dim, a.k_stride,
               k_out_used ? a.k_out_stride : a.k_stride, a.k_weight))
    return NVFP4_ERR_INVALID;
  if (a.rot_dim > 0 && a.tokens > 0) {
    if (a.max_pos < 1 || !extent_ok(a.max_pos, a.rot_dim) || !given(a.positions, 4) ||
        !given(a.cos, 16) || !given(a.sin, 16))
      return NVFP4_ERR_INVALID;
  }
  if (a.head_dim % 32 || a.rot_dim % 32 || a.head_dim > 256) return NVFP4_ERR_UNSUPPORTED;
  return NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_kv_plan(const nvfp4_kv_plan_args* p, hipStream_t stream) {
  if (!p) return NVFP4_ERR_INVALID;
  const nvfp4_kv_plan_args& a = *p;
  if (a.batch < 0 || a.batch > kMax32 || a.tokens < 0 || a.tokens > kMax32 || a.table_width < 0 ||
      a.table_width > kMax32 || a.num_pages < 1 || a.num_pages > kMax32)
    return NVFP4_ERR_INVALID;
  if (a.page_size < 8 || a.page_size > 1024 || (a.page_size & (a.page_size - 1)))
    return NVFP4_ERR_INVALID;
  if (!extent_ok(a.batch, a.table_width)) return NVFP4_ERR_INVALID;
  if (a.batch > 0 && (!given(a.ctx_lens, 4) || !given(a.new_lens, 4) || !given(a.seq_lens, 4) ||
                      (a.table_width > 0 && !given(a.block_table, 4))))
    return NVFP4_ERR_INVALID;
  if (a.tokens > 0 && (!given(a.positions, 4) || !given(a.slots, 8))) return NVFP4_ERR_INVALID;
  if (!given(a.free_pages, 4) || !given(a.free_count, 4) || !given(a.cu_new, 4) ||
      !given(a.free_count_out, 4) || !given(a.refused, 4))
    return NVFP4_ERR_INVALID;
  // one workgroup writes while another one still reads the inputs
  const void* const in[] = {a.ctx_lens, a.new_lens, a.free_pages, a.free_count, a.block_table};
  const void* const out[] = {a.cu_new, a.seq_lens, a.positions, a.slots, a.free_count_out, a.refused};
  for (const void* o : out)
    for (const void* i : in)
      if (o && o == i) return NVFP4_ERR_INVALID;
  return status_of(launch_kv_plan(a, stream));
}

int nvfp4_qk_norm_rope(const nvfp4_qk_args* args, hipStream_t stream) {
  if (!args) return NVFP4_ERR_INVALID;
  const int st = qk_ok(*args, true);
  if (st != NVFP4_OK) return st;
  if (args->tokens == 0) return NVFP4_OK;
  return status_of(launch_qk_norm_rope(*args, stream));
}

size_t nvfp4_qk_norm_rope_bwd_workspace_bytes(int head_dim) {
  return head_dim <= 0 || head_dim > 256 ? 0 : qk_norm_rope_bwd_workspace(head_dim);
}

int nvfp4_qk_norm_rope_bwd(const nvfp4_qk_args* args, const uint16_t* dq_out, int64_t gq_stride,
                           const uint16_t* dk_out, int64_t gk_stride, float* dq_weight,
                           float* dk_weight, void* workspace, hipStream_t stream) {
  if (!args) return NVFP4_ERR_INVALID;
  const nvfp4_qk_args& a = *args;
  const int st = qk_ok(a, true);
  if (st == NVFP4_ERR_INVALID) return st;
  if (!side_ok(dq_out, dq_out, a.tokens, a.q_heads, a.head_dim, gq_stride, gq_stride, nullptr) ||
      !side_ok(dk_out, dk_out, a.tokens, a.k_heads, a.head_dim, gk_stride, gk_stride, nullptr))
    return NVFP4_ERR_INVALID;
  const bool wq = a.q_weight && a.q_heads, wk = a.k_weight && a.k_heads;
  if (wq != (dq_weight != nullptr) || wk != (dk_weight != nullptr) || !aligned(dq_weight, 4) ||
      !aligned(dk_weight, 4))
    return NVFP4_ERR_INVALID;
  if ((wq || wk) && !given(workspace, 16)) return NVFP4_ERR_INVALID;
  if (st != NVFP4_OK) return st;
  if (a.tokens == 0 && !wq && !wk) return NVFP4_OK;
  return status_of(launch_qk_norm_rope_bwd(a, dq_out, gq_stride, dk_out, gk_stride, dq_weight,
                                           dk_weight, static_cast<uint8_t*>(workspace), stream));
}

int nvfp4_kv_append(const nvfp4_kv_append_args* args, hipStream_t stream) {
  if (!args) return NVFP4_ERR_INVALID;
  const nvfp4_kv_append_args& a = *args;
  const int st = qk_ok(a.qk, false), sc = cache_ok(a.cache);
  if (st == NVFP4_ERR_INVALID || sc == NVFP4_ERR_INVALID) return NVFP4_ERR_INVALID;
  if (a.qk.k_heads != a.cache.kv_heads || a.qk.head_dim != a.cache.head_dim) return NVFP4_ERR_INVALID;
  if (a.select < NVFP4_SELECT_6 || a.select > NVFP4_SELECT_SWEEP) return NVFP4_ERR_INVALID;
  if (!side_ok(a.v, a.v, a.qk.tokens, a.qk.k_heads, a.qk.head_dim, a.v_stride, a.v_stride, nullptr))
    return NVFP4_ERR_INVALID;
  if (a.qk.tokens > 0 && !given(a.slots, 8)) return NVFP4_ERR_INVALID;
  if (st != NVFP4_OK || sc != NVFP4_OK) return NVFP4_ERR_UNSUPPORTED;
  if (a.select != NVFP4_SELECT_6 && a.select != NVFP4_SELECT_4OVER6) return NVFP4_ERR_UNSUPPORTED;
  if (a.qk.tokens == 0) return NVFP4_OK;
  return status_of(launch_kv_append(a, stream));
}

int nvfp4_kv_read(const nvfp4_kv_cache* cache, const int64_t* slots, int64_t tokens,
                  uint16_t* k_out, uint16_t* v_out, hipStream_t stream) {
  if (!cache) return NVFP4_ERR_INVALID;
  const int st = cache_ok(*cache);
  if (st == NVFP4_ERR_INVALID) return st;
  if (tokens < 0 || !extent_ok(tokens, 2 * (int64_t)cache->kv_heads * cache->head_dim))
    return NVFP4_ERR_INVALID;
  if (!aligned(k_out, 8) || !aligned(v_out, 8)) return NVFP4_ERR_INVALID;
  if (tokens > 0 && (!given(slots, 8) || (!k_out && !v_out))) return NVFP4_ERR_INVALID;
  if (st != NVFP4_OK) return st;
  if (tokens == 0) return NVFP4_OK;
  return status_of(launch_kv_read(*cache, slots, tokens, k_out, v_out, stream));
}

static int attention_ok(const nvfp4_kv_attention_args& a, AttnPlan& plan) {
  const int st = cache_ok(a.cache);
  if (st == NVFP4_ERR_INVALID) return st;
  if (a.tokens < 0 || a.tokens > kMax32 || a.batch < 0 || a.batch > kMax32 || a.table_width < 0 ||
      a.table_width > kMax32 || a.max_seq_len < 0 || a.max_seq_len > kMax32 || a.window < 0)
    return NVFP4_ERR_INVALID;
  if (a.q_heads < 1 || a.q_heads > NVFP4_KV_MAX_HEADS || a.q_heads % a.cache.kv_heads)
    return NVFP4_ERR_INVALID;
  if (a.q_stride < (int64_t)a.q_heads * a.cache.head_dim || a.q_stride % 8 ||
      !extent_ok(a.tokens, a.q_stride) || !extent_ok(a.batch, a.table_width))
    return NVFP4_ERR_INVALID;
  if (!a.cu_q && a.tokens != a.batch) return NVFP4_ERR_INVALID;
  if (!isfinite(a.scale)) return NVFP4_ERR_INVALID;
  // key positions, and their sums with a tile's width, and rows stay in 32 bits
  if (st == NVFP4_OK && (a.table_width > ((int64_t)1 << 30) / a.cache.page_size ||
                         a.tokens > ((int64_t)1 << 31) / a.q_heads))
    return NVFP4_ERR_UNSUPPORTED;
  if (st != NVFP4_OK) return st;
  plan = kv_attention_plan(a);
  // threads of one launch stay in 32 bits
  return plan.grid > kAttnMaxGroups ? NVFP4_ERR_UNSUPPORTED : NVFP4_OK;
}

size_t nvfp4_kv_attention_workspace_bytes(const nvfp4_kv_attention_args* args) {
  AttnPlan plan = {};
  return !args || attention_ok(*args, plan) != NVFP4_OK ? 0 : plan.bytes;
}

int nvfp4_kv_attention(const nvfp4_kv_attention_args* args, hipStream_t stream) {
  if (!args) return NVFP4_ERR_INVALID;
  const nvfp4_kv_attention_args& a = *args;
  AttnPlan plan = {};
  const int st = attention_ok(a, plan);
  if (st == NVFP4_ERR_INVALID) return st;
  if (a.tokens > 0 && (!given(a.q, 16) || !given(a.out, 16))) return NVFP4_ERR_INVALID;
  if (!aligned(a.lse, 4) || !aligned(a.cu_q, 4) || !aligned(a.workspace, 16) || !aligned(a.counters, 16))
    return NVFP4_ERR_INVALID;
  if (a.batch > 0 && (!given(a.seq_lens, 4) || (a.table_width > 0 && !given(a.block_table, 4))))
    return NVFP4_ERR_INVALID;
  if (st != NVFP4_OK) return st;
  if (a.tokens == 0) return NVFP4_OK;
  if (plan.bytes != 0 && !a.workspace) return NVFP4_ERR_INVALID;
  return status_of(launch_kv_attention(a, plan, stream));
}

}  // extern "C"
