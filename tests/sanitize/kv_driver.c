/* Sanitizer driver for the host side of the key/value-cache entry points
 * (test infrastructure only): valid calls launch with plausible shapes, broken
 * ones launch nothing, and sizes up to the limits stay inside 64-bit
 * arithmetic.  Linked like abi_driver.c; the pointers are never dereferenced. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "nvfp4.h"

extern unsigned long stub_launches, stub_bad_launches;

static int failures = 0;
static unsigned long launches_before;

static void check(int got, int want, const char *what, int line) {
  const unsigned long n = stub_launches - launches_before;
  if (got != want || (want != NVFP4_OK && n > 0)) {
    fprintf(stderr, "FAIL line %d (%s): status %d, expected %d; %lu launches\n", line, what, got, want, n);
    ++failures;
  }
}
#define CALL(want, expr)                   \
  do {                                     \
    launches_before = stub_launches;       \
    check((expr), (want), #expr, __LINE__); \
  } while (0)
#define OK(expr) CALL(NVFP4_OK, expr)
#define BAD(expr) CALL(NVFP4_ERR_INVALID, expr)
#define UNS(expr) CALL(NVFP4_ERR_UNSUPPORTED, expr)

static _Alignas(256) unsigned char pool[1 << 16];
#define P(T, off) ((T *)(pool + (off)))

static nvfp4_kv_cache cache_of(int64_t pages, int heads, int page, int d) {
  nvfp4_kv_cache c;
  memset(&c, 0, sizeof c);
  c.k_codes = P(uint8_t, 0);
  c.k_scales = P(uint8_t, 256);
  c.v_codes = P(uint8_t, 512);
  c.v_scales = P(uint8_t, 768);
  c.k_amax = P(const float, 1024);
  c.v_amax = P(const float, 1280);
  c.num_pages = pages;
  c.kv_heads = heads;
  c.page_size = page;
  c.head_dim = d;
  c.global_fp8_max = 256.0f;
  return c;
}

static nvfp4_qk_args qk_of(int64_t tokens, int hq, int hk, int d, int rot) {
  nvfp4_qk_args a;
  memset(&a, 0, sizeof a);
  a.q = P(const uint16_t, 2048);
  a.k = P(const uint16_t, 2304);
  a.tokens = tokens;
  a.q_heads = hq;
  a.k_heads = hk;
  a.head_dim = d;
  a.q_stride = a.q_out_stride = (int64_t)hq * d;
  a.k_stride = a.k_out_stride = (int64_t)hk * d;
  a.positions = P(const int32_t, 2560);
  a.cos = P(const float, 2816);
  a.sin = P(const float, 4352);
  a.max_pos = 1000;
  a.rot_dim = rot;
  a.q_weight = P(const uint16_t, 3328);
  a.k_weight = P(const uint16_t, 3584);
  a.eps = 1e-6f;
  a.q_out = P(uint16_t, 3840);
  a.k_out = P(uint16_t, 4096);
  return a;
}

static void plan_calls(void) {
  nvfp4_kv_plan_args a;
  memset(&a, 0, sizeof a);
  a.ctx_lens = a.new_lens = P(const int32_t, 0);
  a.block_table = P(int32_t, 256);
  a.free_pages = a.free_count = P(const int32_t, 512);
  a.cu_new = a.seq_lens = a.positions = a.free_count_out = a.refused = P(int32_t, 1024);
  a.slots = P(int64_t, 2048);
  const int64_t tokens[] = {0, 1, 1024, 1025, INT32_MAX}, batches[] = {0, 1, 3000, 1 << 20};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < 4; ++j)
      for (int page = 8; page <= 1024; page *= 2) {
        a.tokens = tokens[i];
        a.batch = batches[j];
        a.table_width = 64;
        a.num_pages = INT32_MAX;
        a.page_size = page;
        OK(nvfp4_kv_plan(&a, 0));
      }
  a.batch = a.table_width = INT32_MAX;
  BAD(nvfp4_kv_plan(&a, 0));
  a.batch = 4; a.table_width = -1; BAD(nvfp4_kv_plan(&a, 0));
  a.table_width = 64; a.page_size = 12; BAD(nvfp4_kv_plan(&a, 0));
  a.page_size = INT32_MIN; BAD(nvfp4_kv_plan(&a, 0));
}

static void rope_calls(void) {
  const int64_t tokens[] = {0, 1, 7, 8192, (int64_t)1 << 24, (int64_t)1 << 31};
  for (int i = 0; i < 6; ++i)
    for (int d = 32; d <= 256; d += 32)
      for (int rot = 0; rot <= d; rot += 32)
        for (int pairs = 0; pairs < 2; ++pairs) {
          nvfp4_qk_args a = qk_of(tokens[i], 16, 4, d, rot);
          a.pairs = pairs;
          OK(nvfp4_qk_norm_rope(&a, 0));
          OK(nvfp4_qk_norm_rope_bwd(&a, P(const uint16_t, 0), a.q_stride, P(const uint16_t, 0), a.k_stride,
                                    P(float, 0), P(float, 256), pool, 0));
        }
  nvfp4_qk_args a = qk_of((int64_t)1 << 33, 16, 4, 256, 256);
  BAD(nvfp4_qk_norm_rope(&a, 0)); /* more than 2^44 elements */
  a = qk_of(INT64_MAX, 16, 4, 128, 128); BAD(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, 16, 4, 128, 128); a.q_stride = INT64_MAX - 3; BAD(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, 16, 4, 128, 128); a.max_pos = INT64_MAX; BAD(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, INT32_MAX, 4, 128, 128); BAD(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, 16, 4, INT32_MAX - 15, 128); UNS(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, 1024, 1024, 256, 256); OK(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, 16, 4, 144, 32); UNS(nvfp4_qk_norm_rope(&a, 0));
  a = qk_of(8, 16, 0, 64, 0); a.k = NULL; a.k_out = NULL; a.k_weight = NULL; OK(nvfp4_qk_norm_rope(&a, 0));
  for (int d = -1; d <= 300; ++d) (void)nvfp4_qk_norm_rope_bwd_workspace_bytes(d);
}

static void cache_calls(void) {
  const int dims[] = {64, 128, 192, 256};
  const int64_t tokens[] = {0, 1, 1000, (int64_t)1 << 24};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      for (int select = 0; select < 2; ++select) {
        nvfp4_kv_append_args a;
        memset(&a, 0, sizeof a);
        a.qk = qk_of(tokens[j], 32, 8, dims[i], dims[i] / 64 * 32);
        a.cache = cache_of((int64_t)1 << 20, 8, 64, dims[i]);
        a.v = P(const uint16_t, 0);
        a.v_stride = 8 * dims[i];
        a.slots = P(const int64_t, 0);
        a.select = select;
        OK(nvfp4_kv_append(&a, 0));
        OK(nvfp4_kv_read(&a.cache, a.slots, tokens[j], P(uint16_t, 0), j % 2 ? NULL : P(uint16_t, 256), 0));
      }
  nvfp4_kv_cache c = cache_of(INT32_MAX, 1024, 1024, 256);
  BAD(nvfp4_kv_read(&c, P(const int64_t, 0), 1, P(uint16_t, 0), NULL, 0));
  c = cache_of(INT32_MAX, 8, 16, 64);
  BAD(nvfp4_kv_read(&c, P(const int64_t, 0), INT64_MAX, P(uint16_t, 0), NULL, 0));
  OK(nvfp4_kv_read(&c, P(const int64_t, 0), (int64_t)1 << 32, P(uint16_t, 0), NULL, 0));
}

static void attention_calls(void) {
  const int dims[] = {64, 128, 192, 256}, heads[][2] = {{1, 1}, {32, 8}, {64, 1}, {40, 8}, {1024, 1024}};
  const int64_t batches[] = {0, 1, 64, 5000}, per[] = {1, 3, 200};
  const int64_t lens[] = {0, 1, 129, 100000, INT32_MAX}, windows[] = {0, 1, 4096, INT64_MAX};
  for (int i = 0; i < 4; ++i)
    for (int h = 0; h < 5; ++h)
      for (int b = 0; b < 4; ++b)
        for (int t = 0; t < 3; ++t)
          for (int l = 0; l < 5; ++l)
            for (int w = 0; w < 4; ++w) {
              nvfp4_kv_attention_args a;
              memset(&a, 0, sizeof a);
              a.cache = cache_of(1 << 20, heads[h][1], 16, dims[i]);
              a.q = P(const uint16_t, 0);
              a.q_heads = heads[h][0];
              a.tokens = batches[b] * per[t];
              a.q_stride = (int64_t)a.q_heads * dims[i];
              a.block_table = a.seq_lens = P(const int32_t, 0);
              a.cu_q = per[t] > 1 ? P(const int32_t, 0) : NULL;
              a.batch = batches[b];
              a.table_width = 1000;
              a.max_seq_len = lens[l];
              a.window = windows[w];
              a.scale = 0.1f;
              a.out = P(uint16_t, 0);
              a.workspace = NULL;
              const size_t bytes = nvfp4_kv_attention_workspace_bytes(&a);
              if (bytes && a.tokens) BAD(nvfp4_kv_attention(&a, 0));
              a.workspace = pool;
              OK(nvfp4_kv_attention(&a, 0));
              a.counters = pool;
              OK(nvfp4_kv_attention(&a, 0));
            }
  nvfp4_kv_attention_args a;
  memset(&a, 0, sizeof a);
  a.cache = cache_of(1 << 20, 8, 16, 128);
  a.q = P(const uint16_t, 0); a.q_heads = 32; a.tokens = a.batch = 4; a.q_stride = 4096;
  a.block_table = a.seq_lens = P(const int32_t, 0); a.table_width = 10; a.scale = 1.0f; a.out = P(uint16_t, 0);
  a.workspace = pool;
  OK(nvfp4_kv_attention(&a, 0));
  a.scale = NAN; BAD(nvfp4_kv_attention(&a, 0)); a.scale = 1.0f;
  a.q_heads = 12; BAD(nvfp4_kv_attention(&a, 0)); a.q_heads = 32;
  a.window = INT64_MIN; BAD(nvfp4_kv_attention(&a, 0)); a.window = 0;
  a.q_stride = INT64_MAX - 7; BAD(nvfp4_kv_attention(&a, 0)); a.q_stride = 4096;
  a.table_width = INT32_MAX; UNS(nvfp4_kv_attention(&a, 0)); a.table_width = 10;
  a.tokens = a.batch = (int64_t)1 << 21; UNS(nvfp4_kv_attention(&a, 0));
  a.tokens = --a.batch; OK(nvfp4_kv_attention(&a, 0));
  a.tokens = a.batch = (int64_t)1 << 27; UNS(nvfp4_kv_attention(&a, 0));
}

int main(void) {
  plan_calls();
  rope_calls();
  cache_calls();
  attention_calls();
  if (stub_bad_launches) {
    fprintf(stderr, "%lu launches with an implausible shape\n", stub_bad_launches);
    ++failures;
  }
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("kv driver: %lu launches, every status as expected\n", stub_launches);
  return 0;
}
