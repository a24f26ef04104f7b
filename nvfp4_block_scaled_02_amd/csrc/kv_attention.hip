// kv_attention.hip -- attention of a step's queries over the paged NVFP4
// cache.
//
// The products run on the matrix units in binary16: E2M1 x E4M3 has 6
// significant bits between 2^-10 and 2688, so a dequantized key or value
// (without its outer scale) is a binary16 number exactly, and a query row is
// scaled by a power of two to its largest value in [1, 2).  The outer scales,
// the softmax scale, log2(e) and that power of two are one binary32 factor per
// query row; the value's outer scale goes into the final division.
//
// A wavefront takes 16 * NQ query rows (token, head of one key/value head's
// group) and walks tiles of 32 keys.  Per tile, with r = lane % 16, g = lane /
// 16:
//   S^T = K Q^T   two 16 x 16 products over D: lane (r, g) reads key 8 (r/4) +
//     4 t + r % 4 and its values [g D/4, (g+1) D/4): whole 16-byte loads, and
//     lane (n, g) receives the scores of query n with keys 8 g + 4 t + 0..3
//   softmax       per lane, in the exponent of 2: weights are 2^(s - m) with m
//     set kLift below the largest score so far, and m moves only when a score
//     passes it by more than 15 (weights stay within binary16's 2^15), so a tile
//     usually needs no exchange between lanes and no rescaling; the weights'
//     sum is one more product, with ones
//   O^T += V^T P^T  lane (m, g) reads keys 8 g .. 8 g + 7 of 4 value columns
//     as the cache holds them (8 tokens side by side); lane (n, g)'s weights
//     of keys 8 g .. 8 g + 7 are already the product's other operand.
// Nothing is transposed between lanes.
//
// Few rows (decoding, drafted tokens): the four wavefronts of a workgroup
// take every fourth tile and join through LDS, and long key ranges are split
// over workgroups whose partial results (binary32) are joined in order, by the
// last of them or by a second launch.  Many rows (prompts): each
// wavefront has rows of its own, and the workgroup dequantizes each block of
// keys once, into LDS.
//
// Measured with 32 query and 8 key heads of 128 values: 64 requests of 8191
// keys 112 .. 115 us (5.3 TB/s, the rate of a copy), of up to 8192 78 .. 84
// (341 MB, 66 us at that rate; vector units 59 % busy, matrix units 16), one of
// 8191 keys 10.5; 2 x 2048 tokens behind 6000 cached ones 353 .. 362 us, 880 to
// 900 TFLOP/s (263 us at the rate of a large product; vector units 54 % busy
// with softmax and dequantization, matrix units 41: a wavefront runs scores,
// softmax and products one after the other, and a SIMD has two of them to
// overlap), a prompt of 8191 tokens 572 .. 582.
#include <math.h>

#include "kv.hpp"

namespace nvfp4 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnThreads = 256;
constexpr int kMaxSplits = 128;
constexpr int kManyPieces = 16;
constexpr int kJoinCounters = NVFP4_KV_COUNTER_BYTES / 128;
constexpr int kSlabStride = 68;  // floats of a 64-column slab row: 4 apart in the banks
constexpr float kLog2e = 1.44269504088896340736f;
// The largest weight of a row is 2^kLift and more: what binary16 rounds to 0
// is below 2^-(25 + kLift) of it.  The rest up to 2^15 is how far the scores
// may climb before a tile rescales its sums (11 and 4 instead of 7 and 8 take
// 0.6 % longer in prompt chunks).
constexpr float kLift = 7.0f;

struct AttnArgs {
  nvfp4_kv_attention_args a;
  int rows, splits, chunk, shift, group;
  uint32_t tiles, tiles_per_request;
  int join;  // the last workgroup of a tile to finish joins its pieces
};

// ---------------------------------------------------------------- lanes
__device__ __forceinline__ uint32_t u32(float v) { return __float_as_uint(v); }

// max over the four lanes of a query (lane % 16 equal), in all of them
__device__ __forceinline__ float max_over_g(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(u32(v), u32(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(u32(v), u32(v), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ f16x2 fp4_pair(uint32_t w, int sel) {
  switch (sel) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
  }
}
// two E4M3 bytes (the low or the high half of a word), 0x7F = NaN
__device__ __forceinline__ f16x2 fp8_lo(uint32_t w) { return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false); }
__device__ __forceinline__ f16x2 fp8_hi(uint32_t w) { return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true); }
__device__ __forceinline__ f16x8 join8(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// largest of three, NaN if any is (v_maximum3_f32).  A builtin, not assembly:
// the compiler has to see the read of a matrix result to wait for it.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// The tile as it lies in memory, for one lane.
template <int D>
struct Raw {
  static constexpr int NCH = D / 32;  // 8-value pieces of a key, and value pairs, per lane
  uint32_t k[2][NCH];
  uint32_t ks[2];    // block scales of the lane's pieces, one byte per two
  uint4 v[NCH / 2];
  uint2 vs[NCH / 2];
  bool ok;           // the lane's 8 value tokens lie on a page of the cache
};

// Pages of the lane's key group and value group of a tile; -1: none.
struct Pages {
  int k, v;
};

// A byte holds two columns of one token; the products want 8 tokens of one
// column, in any order that the weights share.  x, y: the bytes of tokens 0..3
// and 4..7 of a column pair; one column's nibbles of y move beside x's, and a
// conversion takes tokens i and i + 4 at once: the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ void value_columns(uint32_t x, uint32_t y, const f16x2 (&f)[4], f16x8& even, f16x8& odd) {
  const uint32_t M = 0x0F0F0F0Fu;
  const uint32_t e = (x & M) | ((y << 4) & ~M), o = ((x >> 4) & M) | (y & ~M);
  even = join8(fp4_pair(e, 0) * f[0], fp4_pair(e, 1) * f[1], fp4_pair(e, 2) * f[2], fp4_pair(e, 3) * f[3]);
  odd = join8(fp4_pair(o, 0) * f[0], fp4_pair(o, 1) * f[1], fp4_pair(o, 2) * f[2], fp4_pair(o, 3) * f[3]);
}
// The tokens' block scales in that order.
__device__ __forceinline__ void value_scales(uint2 s, f16x2 (&f)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(s.y, s.x, 0x05010400u), b = __builtin_amdgcn_perm(s.y, s.x, 0x07030602u);
  f[0] = fp8_lo(a); f[1] = fp8_hi(a); f[2] = fp8_lo(b); f[3] = fp8_hi(b);
}

// Byte mask of the keys key0 .. key0 + 7 that lie in [lo, hi), on a page of
// the cache.
__device__ __forceinline__ uint64_t keys_in(int key0, int lo, int hi, bool ok) {
  const int a = lo - key0, b = hi - key0;
  const uint64_t in = b <= 0 || !ok ? 0 : b >= 8 ? ~0ull : (1ull << (8 * b)) - 1;
  return in & (a <= 0 ? ~0ull : a >= 8 ? 0 : ~((1ull << (8 * a)) - 1));
}
// Top bit of every byte that is the E4M3 NaN, 0x7F (a byte below never
// carries into the next: 0x7F + 1).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t s) { return ((s & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// A workgroup's place: its request and rows.
// Rows (token x head of a group) and positions stay in 32 bits: the entry point
// refuses more than 2^31 rows and 2^30 keys a request.
struct Place {
  int b;           // request (batch: rows that belong to none)
  int begin, end;  // its rows of q
  int row0;        // first row of the workgroup, in the request
  int count;       // rows of the workgroup; 0: nothing to do
  int len;         // keys [0, len)
  int pos0;        // position of the request's first query
};

// Keys that a row attends, [lo, hi).  Both ascend with the row.
__device__ __forceinline__ void bounds_of(const AttnArgs& args, const Place& at, int row, int& lo, int& hi) {
  const nvfp4_kv_attention_args& a = args.a;
  const int64_t p = (int64_t)at.pos0 + (uint32_t)row / (uint32_t)args.group;
  const int64_t h = a.causal && p + 1 < at.len ? p + 1 : at.len;
  const int64_t w = a.window > 0 ? p - a.window + 1 : 0;
  hi = (int)(h < 0 ? 0 : h);
  lo = (int)(w < 0 ? 0 : w > at.len ? at.len : w);
}

__device__ __forceinline__ Place place_of(const AttnArgs& args, uint32_t tile, int lane) {
  const nvfp4_kv_attention_args& a = args.a;
  Place p;
  int local;
  p.count = 0;
  if (!a.cu_q) {
    p.b = (int)(tile / args.tiles_per_request);
    local = (int)(tile - (uint32_t)p.b * args.tiles_per_request);
    p.begin = p.b;
    p.end = p.b + 1;
  } else {
    // request b's tiles begin at floor(cu_q[b] * group / rows) + b; rows past
    // cu_q[batch] count as a request of length 0.  64 probes at a time.
    const int tokens = (int)a.tokens, batch = (int)a.batch;
    const auto cu = [&](int i) {
      const int v = a.cu_q[i];
      return v < 0 ? 0 : v < tokens ? v : tokens;
    };
    const auto start = [&](int i) { return (uint32_t)cu(i) * (uint32_t)args.group / (uint32_t)args.rows + (uint32_t)i; };
    int lo = 0, n = batch + 1;
    while (n > 1) {
      const int step = (n - 1) / 64 + 1, i = lane * step;
      const bool before = i < n && start(lo + i) <= tile;
      const int hits = __popcll(__ballot(before));
      const int k = hits > 0 ? hits - 1 : 0;
      lo += k * step;
      n = n - k * step < step ? n - k * step : step;
    }
    p.b = __builtin_amdgcn_readfirstlane(lo);
    local = (int)(tile - start(p.b));
    if (local < 0) return p;
    p.begin = cu(p.b);
    p.end = p.b < batch ? cu(p.b + 1) : tokens;
    p.end = p.end < p.begin ? p.begin : p.end;
  }
  const uint32_t rows = (uint32_t)(p.end - p.begin) * (uint32_t)args.group, row0 = (uint32_t)local * (uint32_t)args.rows;
  if (row0 >= rows) return p;
  p.row0 = (int)row0;
  p.count = rows - row0 < (uint32_t)args.rows ? (int)(rows - row0) : args.rows;
  const int seq = p.b < (int)a.batch ? a.seq_lens[p.b] : 0;
  const int room = (int)a.table_width << args.shift;
  p.len = seq < 0 ? 0 : seq < room ? seq : room;
  p.pos0 = seq - (p.end - p.begin);
  return p;
}

// Row of out (token * q_heads + head) of a workgroup's row.
__device__ __forceinline__ int64_t out_row(const AttnArgs& args, const Place& at, int kvh, int row) {
  const uint32_t rr = (uint32_t)(at.row0 + row), token = rr / (uint32_t)args.group;
  return (int64_t)(at.begin + (int)token) * args.a.q_heads + kvh * args.group + (int)(rr - token * (uint32_t)args.group);
}

// Where a lane reads.  The four pointers hold what does not change from tile
// to tile (array, head, the lane's place among 32 tokens); a tile adds its
// page and, in pages of more than 32 tokens, its place in the page: two
// instructions a pointer.  The table entry of a group past the last key is
// that of the last one (its tokens are masked).
template <int D>
struct Reader {
  static constexpr int NCH = D / 32;
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t* table;  // of the request
  int last;              // last table entry that may be read
  int shift, r, g;
  uint32_t pages_end, page_tokens;  // pages; tokens of a page over all heads
  __device__ __forceinline__ Reader(const AttnArgs& args, const Place& at, int kvh, int r_, int g_) : r(r_), g(g_) {
    const nvfp4_kv_cache& c = args.a.cache;
    shift = args.shift;
    table = args.a.block_table + (int64_t)at.b * args.a.table_width;
    last = at.len > 0 ? (at.len - 1) >> shift : 0;
    pages_end = (uint32_t)c.num_pages;
    page_tokens = (uint32_t)c.kv_heads << shift;  // <= 2^20
    const int mask = (1 << shift) - 1;
    const int64_t kt = ((int64_t)kvh << shift) + ((8 * (r >> 2)) & mask) + (r & 3);
    const int64_t vt = ((int64_t)kvh << shift) + ((8 * g) & mask);
    kc = c.k_codes + kt * (D / 2) + g * (D / 8);
    ks = c.k_scales + kt * (D / 16) + g * (NCH / 2);
    vc = c.v_codes + vt * (D / 2) + 16 * r;
    vs = c.v_scales + vt * (D / 16) + 8 * (r >> 2);
  }
  // Loads return in order, so these go ahead of the tile loads they will be
  // used after; and without a branch or a scalar load for tiles in one page,
  // either of which makes the compiler wait for all that is in flight (64
  // requests of up to 8192 keys: 93 us so, 89 as it is).
  __device__ __forceinline__ Pages pages(int tile0) const {
    const int ik = (tile0 + 8 * (r >> 2)) >> shift, iv = (tile0 + 8 * g) >> shift;
    return Pages{table[ik < last ? ik : last], table[iv < last ? iv : last]};
  }
  // bytes from a lane's pointer to its tokens of a tile, at `per` bytes a token
  __device__ __forceinline__ uint64_t ahead(int tile0, uint32_t page, int per) const {
    const uint32_t in_page = (uint32_t)tile0 & ((1u << shift) - 1) & ~31u;
    return (uint64_t)page * (page_tokens * (uint32_t)per) + in_page * (uint32_t)per;
  }
  // Codes and scales of one 16-key product (t of the tile): D / 8 bytes and D /
  // 64 scale bytes of the lane's key.
  __device__ __forceinline__ void load_keys(int tile0, int t, uint32_t page, uint32_t (&k)[NCH], uint32_t& sc) const {
    const uint8_t* p = kc + ahead(tile0, page, D / 2) + 4 * t * (D / 2);
    const uint8_t* s = ks + ahead(tile0, page, D / 16) + 4 * t * (D / 16);
    if constexpr (NCH % 4 == 0) {
#pragma unroll
      for (int i = 0; i < NCH / 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 16 * i);
        k[4 * i] = x.x; k[4 * i + 1] = x.y; k[4 * i + 2] = x.z; k[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NCH / 2; ++i) {
        const uint2 x = *reinterpret_cast<const uint2*>(p + 8 * i);
        k[2 * i] = x.x; k[2 * i + 1] = x.y;
      }
    }
    if constexpr (NCH == 2) sc = s[0];
    else if constexpr (NCH == 4) sc = *reinterpret_cast<const uint16_t*>(s);
    else if constexpr (NCH == 6) sc = s[0] | (uint32_t)s[1] << 8 | (uint32_t)s[2] << 16;
    else sc = *reinterpret_cast<const uint32_t*>(s);
  }
  __device__ __forceinline__ uint32_t usable(int page) const { return (uint32_t)page < pages_end ? (uint32_t)page : 0u; }
  // Product t of the tile's keys, half h (one column pair of two) of its values.
  template <class Q>
  __device__ __forceinline__ void load_quarter(int tile0, int sub, const Pages& p, Q& x) const {
    load_keys(tile0, sub, usable(p.k), x.k, x.ks);
    x.ok = (uint32_t)p.v < pages_end;
    const uint8_t* c = vc + ahead(tile0, usable(p.v), D / 2) + 8 * sub;
    const uint8_t* s = vs + ahead(tile0, usable(p.v), D / 16);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      x.v[j] = *reinterpret_cast<const uint2*>(c + 256 * j);
      x.vs[j] = *reinterpret_cast<const uint2*>(s + 32 * j);
    }
  }
  __device__ __forceinline__ void load(int tile0, const Pages& p, Raw<D>& w) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) load_keys(tile0, t, usable(p.k), w.k[t], w.ks[t]);
    w.ok = (uint32_t)p.v < pages_end;
    const uint8_t* c = vc + ahead(tile0, usable(p.v), D / 2);
    const uint8_t* s = vs + ahead(tile0, usable(p.v), D / 16);
#pragma unroll
    for (int j = 0; j < NCH / 2; ++j) {
      w.v[j] = *reinterpret_cast<const uint4*>(c + 256 * j);
      w.vs[j] = *reinterpret_cast<const uint2*>(s + 32 * j);
    }
  }
};

// ---------------------------------------------------------------- one tile
template <int D, int NQ>
struct Walk {
  static constexpr int NCH = D / 32, NJ = D / 64;
  f16x8 q[NQ][NCH];
  f32x4 o[NQ][NJ][4];  // [j][e][i]: query n, column 64 j + 16 g + 4 i + e
  float factor[NQ];    // binary32 factor of a row's scores
  float m[NQ];         // exponent that the row's weights and sums are scaled by
  float thr[NQ];       // largest score that m may stay for
  f32x4 l[NQ];         // sum of a row's weights, four times
  int lo[NQ], hi[NQ];  // keys that the row attends

  // partial: some row does not attend some key of the tile.
  __device__ __forceinline__ void tile(Raw<D>& w, int tile0, int g, int lo_any, int hi_any, bool partial) {
    f32x4 s[NQ][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const f16x2 s01 = fp8_lo(w.ks[t]), s23 = fp8_hi(w.ks[t]);
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const _Float16 b = c / 2 == 0 ? s01[0] : c / 2 == 1 ? s01[1] : c / 2 == 2 ? s23[0] : s23[1];
        const f16x2 f = {b, b};
        const uint32_t x = w.k[t][c];
        const f16x8 k = join8(fp4_pair(x, 0) * f, fp4_pair(x, 1) * f, fp4_pair(x, 2) * f, fp4_pair(x, 3) * f);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          s[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][c], c == 0 ? f32x4{0, 0, 0, 0} : s[n][t], 0, 0, 0);
      }
    }
    const int key0 = tile0 + 8 * g;
    if (partial) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!attends(n, key0 + i, w.ok)) s[n][i / 4][i % 4] = -__builtin_inff();
      hide_values(w, key0, lo_any, hi_any);
    }
    float top[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) top[n] = top_of(n, s[n][0], s[n][1]);
    raise(top);
    f16x8 p[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) p[n] = weights(n, s[n][0], s[n][1]);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      f16x2 f[4];
      value_scales(w.vs[j], f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f16x8 ve, vo;
        value_columns(h ? w.v[j].z : w.v[j].x, h ? w.v[j].w : w.v[j].y, f, ve, vo);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          o[n][j][2 * h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ve, p[n], o[n][j][2 * h], 0, 0, 0);
          o[n][j][2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vo, p[n], o[n][j][2 * h + 1], 0, 0, 0);
        }
      }
    }
  }

  // Largest score of query n among a lane's eight of a tile, as the exponent's
  // argument (factor >= 0: the largest product is that of the largest score).
  __device__ __forceinline__ float top_of(int n, const f32x4& s0, const f32x4& s1) const {
    return factor[n] * max3(max3(s0[0], s0[1], s0[2]), max3(s0[3], s1[0], s1[1]), max3(s1[2], s1[3], s1[3]));
  }
  // Moves the exponents of all rows where a score passes one by more than 15.
  // A NaN score never does; its weight and the row become NaN.  One branch for
  // all rows, so that what surrounds it stays in long runs that the matrix and
  // the vector units share.
  __device__ __forceinline__ void raise(const float (&top)[NQ]) {
    bool passed = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) passed |= top[n] > thr[n];
    if (!__any(passed)) return;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float was = m[n];
      m[n] = __builtin_fmaxf(m[n], max_over_g(top[n]) - kLift);
      // less by a step of m, so that where scores past 2^20 make steps of an
      // eighth and more, no sum rounds up past 15
      thr[n] = m[n] + __builtin_fmaf(__builtin_fabsf(m[n]), -0x1p-23f, 15.0f);
      const float keep = was == m[n] || was == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(was - m[n]);
      l[n] *= keep;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] *= keep;
    }
  }
  // The softmax weights of query n's scores of a tile (binary16, in the order of
  // value_columns), added to its sum.
  __device__ __forceinline__ f16x8 weights(int n, const f32x4& s0, const f32x4& s1) {
    const float base = m[n] == -__builtin_inff() ? 0.0f : -m[n];
    f16x8 p, ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = (_Float16)__builtin_amdgcn_exp2f(__builtin_fmaf(i % 2 == 0 ? s0[i / 2] : s1[i / 2], factor[n], base));
      ones[i] = (_Float16)1.0f;
    }
    // the sum over the tile's keys, of the weights as they are used
    l[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p, l[n], 0, 0, 0);
    return p;
  }

  // Query rows [first, first + 16 NQ) of the workgroup (the spare ones repeat
  // the last one): their bf16 patterns as they lie in memory ...
  struct RawQ {
    uint4 x[NQ][NCH];
  };
  __device__ __forceinline__ void load_queries(const AttnArgs& args, const Place& at, int kvh, int first, int r, int g,
                                               RawQ& raw) {
    const nvfp4_kv_attention_args& a = args.a;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      int row = first + 16 * n + r;
      row = at.row0 + (row < at.count ? row : at.count - 1);
      bounds_of(args, at, row, lo[n], hi[n]);
      const uint32_t token = (uint32_t)row / (uint32_t)args.group;
      const int head = kvh * args.group + (int)((uint32_t)row - token * (uint32_t)args.group);
      const uint16_t* src = a.q + (int64_t)(at.begin + (int)token) * a.q_stride + head * D + g * (D / 4);
#pragma unroll
      for (int i = 0; i < NCH; ++i) raw.x[n][i] = *reinterpret_cast<const uint4*>(src + 8 * i);
    }
  }
  // ... and in binary16, each row scaled by a power of two.
  __device__ __forceinline__ void start(const AttnArgs& args, int kvh, const RawQ& raw) {
    const nvfp4_kv_attention_args& a = args.a;
    float common = outer_alpha(a.cache.k_amax[kvh], a.cache.global_fp8_max) * __builtin_fabsf(a.scale) * kLog2e;
    // An unusable amax makes the queries NaN, not the factor: a score that a
    // mask has replaced by -infinity is multiplied by the factor too.
    const bool unusable = common != common;
    common = unusable ? 1.0f : common;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const uint32_t t = chunk_abs_max_bits(raw.x[n][i]);
        top = top > t ? top : t;
      }
      // the row's largest magnitude: bf16 patterns order like their values
      // (infinity for a NaN too)
      const float topf = max_over_g(__uint_as_float((top < 0x7F80u ? top : 0x7F80u) << 16));
      int e = 254 - (int)(u32(topf) >> 23);  // exponent field of 2^-floor(log2 top)
      e = topf == 0.0f ? 127 : e < 1 ? 1 : e > 254 ? 254 : e;
      // Against an infinite value every key's score is infinite or NaN, and a
      // softmax of infinities of either sign is NaN: so is the row, then.
      const bool nan = unusable || topf == __builtin_inff();
      // a negative scale turns the row's sign, so that factor >= 0
      const float up = nan ? __builtin_nanf("") : __builtin_copysignf(__uint_as_float((uint32_t)e << 23), a.scale);
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const uint32_t x[4] = {raw.x[n][i].x, raw.x[n][i].y, raw.x[n][i].z, raw.x[n][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q[n][i][2 * k] = (_Float16)(bf16_lo(x[k]) * up);
          q[n][i][2 * k + 1] = (_Float16)(bf16_hi(x[k]) * up);
        }
      }
      factor[n] = __builtin_ldexpf(common, 127 - e);
      // a score of -inf stays below every other one
      factor[n] = factor[n] == 0.0f ? 0x1p-126f : factor[n];
      m[n] = thr[n] = -__builtin_inff();
      l[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) o[n][j][e2] = f32x4{0, 0, 0, 0};
    }
  }

  // No key seen.
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n] = -__builtin_inff();
      l[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = f32x4{0, 0, 0, 0};
    }
  }

  __device__ __forceinline__ bool attends(int n, int key, bool ok) const {
    return ok && key >= lo[n] && key < hi[n];
  }

  // In a tile that some rows attend in part: the scales of values that no row
  // attends (which may be anything) become 0; a NaN scale becomes 0 too, and
  // the rows that attend it get their NaN here.
  __device__ __forceinline__ void hide_values(Raw<D>& w, int key0, int lo_any, int hi_any) {
    const uint64_t in = keys_in(key0, lo_any, hi_any, w.ok);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t s[2] = {w.vs[j].x & (uint32_t)in, w.vs[j].y & (uint32_t)(in >> 32)};
      const uint32_t nan0 = nan_bytes(s[0]), nan1 = nan_bytes(s[1]);
      if (__any((nan0 | nan1) != 0)) {
        f16x8 nan;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          nan[i] = ((i < 4 ? nan0 : nan1) >> (8 * (i % 4)) & 0x80u) ? (_Float16)1.0f : (_Float16)0.0f;
        s[0] &= ~((nan0 >> 7) * 0xFFu);
        s[1] &= ~((nan1 >> 7) * 0xFFu);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          f16x8 seen;
#pragma unroll
          for (int i = 0; i < 8; ++i) seen[i] = attends(n, key0 + i, w.ok) ? (_Float16)1.0f : (_Float16)0.0f;
          const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x32_f16(nan, seen, f32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][j][e][i] = hit[i] > 0.0f ? __builtin_nanf("") : o[n][j][e][i];
        }
      }
      w.vs[j] = make_uint2(s[0], s[1]);
    }
  }
};

// ---------------------------------------------------------------- workspace
// Partial results of split tiles: per (tile, head) group and split, rows x D
// accumulated values, and behind all of those a (maximum, sum) pair per row.
struct Parts {
  float* o;
  float2* ml;
};
template <int D, int RW>
__device__ __forceinline__ Parts parts_of(const AttnArgs& args, uint32_t tile, uint32_t kvh) {
  const uint64_t first = ((uint64_t)tile * (uint32_t)args.a.cache.kv_heads + kvh) * (uint32_t)args.splits * RW;
  const uint64_t all = (uint64_t)args.tiles * (uint32_t)args.a.cache.kv_heads * (uint32_t)args.splits * RW;
  float* o = static_cast<float*>(args.a.workspace);
  return Parts{o + first * D, reinterpret_cast<float2*>(o + all * D) + first};
}

// How the keys [k0, k1) of a tile are cut up: `n` pieces of `each`.
struct Cut {
  int n, each;
};
__device__ __forceinline__ Cut cut_of(const AttnArgs& args, int k0, int k1) {
  if (args.splits == 1) return Cut{1, 0};
  const int keys = k1 > k0 ? k1 - k0 : 0;
  int n = (keys + args.chunk - 1) / args.chunk;
  n = n < 1 ? 1 : n < args.splits ? n : args.splits;
  const int each = ((keys + n - 1) / n + 127) & ~127;
  n = each > 0 ? (keys + each - 1) / each : 1;
  return Cut{n < 1 ? 1 : n, each};
}

// weight of a partial result with maximum m under the joint maximum M
__device__ __forceinline__ float join_weight(float m, float M) {
  return m == M ? 1.0f : __builtin_amdgcn_exp2f(m - M);
}

// The weights of a row's pieces: lane i those of pieces i and i + 64, from
// their (maximum, sum) pairs.
struct Weights {
  float f0, f1, M, L;
  __device__ __forceinline__ Weights(float2 x0, float2 x1, int lane, int n) {
    x0 = lane < n ? x0 : make_float2(-__builtin_inff(), 0.0f);
    x1 = lane + 64 < n ? x1 : make_float2(-__builtin_inff(), 0.0f);
    M = __builtin_fmaxf(x0.x, x1.x);
    for (int d = 1; d < 64; d <<= 1) M = __builtin_fmaxf(M, __shfl_xor(M, d));
    f0 = join_weight(x0.x, M);
    f1 = join_weight(x1.x, M);
    L = f0 * x0.y + f1 * x1.y;
    for (int d = 1; d < 64; d <<= 1) L += __shfl_xor(L, d);
  }
  __device__ __forceinline__ float operator()(int i) const {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)u32(i < 64 ? f0 : f1), i & 63));
  }
};
// A joined row (columns C lane ..) and its lse.
template <int D>
__device__ __forceinline__ void put_row(const AttnArgs& args, const Place& at_, uint32_t kvh, int row, int lane,
                                        const float (&o)[D / 64], const Weights& w) {
  const nvfp4_kv_attention_args& a = args.a;
  constexpr int C = D / 64;
  const bool empty = w.M == -__builtin_inff() && w.L == 0.0f;
  const float inv = empty ? 0.0f : outer_alpha(a.cache.v_amax[kvh], a.cache.global_fp8_max) / w.L;
  const int64_t to = out_row(args, at_, (int)kvh, row);
  uint16_t* dst = a.out + to * D + C * lane;
#pragma unroll
  for (int k = 0; k < C; ++k) dst[k] = empty ? (uint16_t)0 : (uint16_t)bf16_pair(o[k] * inv, 0.0f);
  if (a.lse && lane == 0) a.lse[to] = empty ? -__builtin_inff() : (w.M + __builtin_log2f(w.L)) / kLog2e;
}

// Values that another workgroup of the launch reads: written and read at the
// level that the whole GPU sees, so no cache is written back or emptied.
__device__ __forceinline__ void put_shared(float* p, float x, float y) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)u32(y) << 32 | u32(x), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get_shared(const float2* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float get_shared(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// After a workgroup's piece is on its way: true in the last of a tile's n to
// arrive, which then sees all of them.  Nobody waits for anybody.
__device__ __forceinline__ bool last_piece(const AttnArgs& args, uint32_t tile, uint32_t kvh, int n) {
  __shared__ bool last;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the piece has arrived
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t* c = static_cast<uint32_t*>(args.a.counters) + 32 * (size_t)(tile * (uint32_t)args.a.cache.kv_heads + kvh);
    last = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)n - 1;
    if (last) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return last;
}

// Joins a tile's n pieces, a wavefront per row, in the order of the kernel
// below: SUMS sums of every SUMS-th piece.
template <int D, int RW, int SUMS>
__device__ __forceinline__ void join_here(const AttnArgs& args, const Place& at_, uint32_t kvh, const Parts& parts, int n) {
  constexpr int C = D / 64;
  const int lane = threadIdx.x & 63;
  for (int row = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); row < at_.count; row += 4) {
    const auto pair = [&](int i) { return get_shared(parts.ml + (size_t)(i < n ? i : n - 1) * RW + row); };
    const float2 x0 = pair(lane), x1 = pair(lane + 64);
    const float* src = parts.o + (size_t)row * D + C * lane;
    const auto value = [&](int i, float (&y)[C]) {
      const float* p = src + (size_t)(i < n ? i : n - 1) * (RW * D);
      if constexpr (C % 2 == 0) {
#pragma unroll
        for (int k = 0; k < C; k += 2) {
          const float2 v = get_shared(reinterpret_cast<const float2*>(p + k));
          y[k] = v.x; y[k + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < C; ++k) y[k] = get_shared(p + k);
      }
    };
    constexpr int AHEAD = 8;
    static_assert(AHEAD % SUMS == 0, "piece i belongs to sum i % SUMS");
    float y[AHEAD][C], o[SUMS][C] = {};
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) value(u, y[u]);
    const Weights w(x0, x1, lane, n);
    for (int i = 0; i < n; i += AHEAD) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        if (i + u < n) {
          const float f = w(i + u);
#pragma unroll
          for (int k = 0; k < C; ++k) o[u % SUMS][k] = __builtin_fmaf(f, y[u][k], o[u % SUMS][k]);
        }
      }
      if (i + AHEAD < n)
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) value(i + AHEAD + u, y[u]);
    }
#pragma unroll
    for (int v = 1; v < SUMS; ++v)
#pragma unroll
      for (int k = 0; k < C; ++k) o[0][k] += o[v][k];
    put_row<D>(args, at_, kvh, row, lane, o[0], w);
  }
}

// Wavefronts of a SIMD that the registers are shared out for: as many as fit
// without spilling (512 registers a lane at one wavefront).
constexpr int attn_waves(int D, int NQ) {
  return D * NQ <= 64 ? 4 : D * NQ <= 128 ? 3 : D * NQ <= 256 ? 2 : 1;
}

// Most 16-row tiles of a wavefront of the kernel below.  Four of D = 128 (two
// of 256) spill and leave one wavefront a SIMD: 64 rows of 8 requests over up to 8192 keys
// take 97 us that way and 44 us as two tiles of 32.
constexpr int keys_nq_most(int D) { return D == 64 ? 4 : D <= 192 ? 2 : 1; }

// Few rows: the wavefronts of a workgroup take every fourth key tile.
template <int D, int NQ>
__global__ void __launch_bounds__(kAttnThreads, attn_waves(D, NQ))
kv_attention_keys_kernel(AttnArgs args) {
  constexpr int NJ = D / 64, RW = 16 * NQ, SLOTS = 2;
  const nvfp4_kv_attention_args& a = args.a;
  const nvfp4_kv_cache& c = a.cache;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  // the workgroup's head, split and row tile; later tiles (whose causal key
  // range is longer) first
  const uint32_t kvh = blockIdx.x % (uint32_t)c.kv_heads;
  uint32_t rest = blockIdx.x / (uint32_t)c.kv_heads;
  const uint32_t split = rest % (uint32_t)args.splits;
  rest /= (uint32_t)args.splits;
  const uint32_t tile = args.tiles - 1 - rest;
  const Place at_ = place_of(args, tile, lane);
  if (at_.count == 0) return;
  const int count = at_.count;
  // keys that any row attends, and those that all attend
  int lo_any, hi_any, lo_all, hi_all;
  bounds_of(args, at_, at_.row0, lo_any, hi_all);
  bounds_of(args, at_, at_.row0 + count - 1, lo_all, hi_any);
  // this workgroup's share
  int k0 = lo_any & ~31, k1 = hi_any;
  const Cut cut = cut_of(args, k0, k1);
  const int nsplit = cut.n;
  if ((int)split >= nsplit) return;
  if (nsplit > 1) {
    k0 += (int)split * cut.each;
    k1 = k1 - k0 < cut.each ? k1 : k0 + cut.each;
  }

  // the walk: the next tile's bytes are in flight while one is computed (the
  // first tile's while the queries are made ready), and the table entries of
  // the one after
  Walk<D, NQ> w;
  typename Walk<D, NQ>::RawQ rq;
  constexpr int STEP = 128, S = SLOTS;
  const int t0 = k0 + 32 * __builtin_amdgcn_readfirstlane(wave);
  const bool any = t0 < k1;
  const Reader<D> rd(args, at_, (int)kvh, r, g);
  const auto at = [&](int i) {  // i tiles ahead, the last one again past the end
    const int t = t0 + i * STEP;
    return t < k1 ? t : t0 + (k1 - 1 - t0) / STEP * STEP;
  };
  Raw<D> raw[S];
  Pages p = {-1, -1};
  if (any) {
    p = rd.pages(t0);
#pragma unroll
    for (int u = 0; u < S - 1; ++u) {
      const Pages pn = rd.pages(at(u + 1));
      if (u == 0) w.load_queries(args, at_, (int)kvh, 0, r, g, rq);
      rd.load(at(u), p, raw[u]);
      p = pn;
    }
    w.start(args, (int)kvh, rq);
    for (int i = 0; t0 + i * STEP < k1; i += S) {
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int t = t0 + (i + u) * STEP;
        if (u > 0 && t >= k1) break;
        const Pages pn = rd.pages(at(i + u + S));
        rd.load(at(i + u + S - 1), p, raw[(u + S - 1) % S]);
        p = pn;
        Raw<D>& cur = raw[u];
        const bool whole = t >= lo_all && t + 32 <= hi_all && __all(cur.ok);
        w.tile(cur, t, g, lo_any, hi_any, !whole);
      }
    }
  } else {
    w.none();
  }
  const float av = outer_alpha(c.v_amax[kvh], c.global_fp8_max);
  {
    // join the four wavefronts: their maxima and sums, then 64 columns at a time
    __shared__ __align__(16) float slab[4 * RW * kSlabStride];
    __shared__ float ms[4][RW], ls[4][RW];
    if (g == 0) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        ms[wave][16 * n + r] = w.m[n];
        ls[wave][16 * n + r] = w.l[n][0];
      }
    }
    __syncthreads();
    const Parts parts = parts_of<D, RW>(args, tile, kvh);
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = 16 * n + r;
      const float M = __builtin_fmaxf(__builtin_fmaxf(ms[0][row], ms[1][row]), __builtin_fmaxf(ms[2][row], ms[3][row]));
      const float f = join_weight(w.m[n], M);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) w.o[n][j][e] *= f;
    }
    const int col = 4 * (threadIdx.x & 15);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j) __syncthreads();
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float* dst = slab + ((wave * RW) + 16 * n + r) * kSlabStride + 16 * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(dst + 4 * i) =
              make_float4(w.o[n][j][0][i], w.o[n][j][1][i], w.o[n][j][2][i], w.o[n][j][3][i]);
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int row = 16 * n + (threadIdx.x >> 4);
        if (row >= count) continue;
        float M = ms[0][row];
#pragma unroll
        for (int v = 1; v < 4; ++v) M = __builtin_fmaxf(M, ms[v][row]);
        float L = 0.0f;
        float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          L += ls[v][row] * join_weight(ms[v][row], M);
          const float4 y = *reinterpret_cast<const float4*>(slab + (v * RW + row) * kSlabStride + col);
          x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        if (nsplit == 1) {
          const bool empty = M == -__builtin_inff() && L == 0.0f;
          const float inv = empty ? 0.0f : av / L;
          const int64_t at = out_row(args, at_, (int)kvh, row);
          uint2 y = make_uint2(bf16_pair(x.x * inv, x.y * inv), bf16_pair(x.z * inv, x.w * inv));
          if (empty) y = make_uint2(0, 0);
          *reinterpret_cast<uint2*>(a.out + at * D + 64 * j + col) = y;
          if (a.lse && j == 0 && col == 0) a.lse[at] = empty ? -__builtin_inff() : (M + __builtin_log2f(L)) / kLog2e;
        } else {
          const int at = (int)split * RW + row;
          float* dst = parts.o + (size_t)at * D + 64 * j + col;
          if (args.join) {
            put_shared(dst, x.x, x.y);
            put_shared(dst + 2, x.z, x.w);
            if (j == 0 && col == 0) put_shared(reinterpret_cast<float*>(parts.ml + at), M, L);
          } else {
            *reinterpret_cast<float4*>(dst) = x;
            if (j == 0 && col == 0) parts.ml[at] = make_float2(M, L);
          }
        }
      }
    }
    if (args.join && nsplit > 1 && last_piece(args, tile, kvh, nsplit)) {
      if (args.splits >= kManyPieces) join_here<D, RW, 4>(args, at_, kvh, parts, nsplit);
      else join_here<D, RW, 1>(args, at_, kvh, parts, nsplit);
    }
  }
}

// Joins the pieces of split tiles, in order: a wavefront per row, or, of many
// pieces, a workgroup per row, each wavefront taking every fourth piece (16 of
// them and more: one token over 8191 13.6 -> 11.9 us, 3 x 4 drafted tokens over
// up to 131072 99 -> 90; 8 x 8 over up to 8192, few pieces, 40 against 52 the
// other way).  A launch of its own, where there are no counters or much to
// join: by the last workgroup of a tile to arrive, the pieces of one tile pass
// through one CU (32 rows x 128 pieces: 257 us in all against 119).  What a
// piece holds is asked for before it is known how many there are (the
// workspace has room for the most), so one memory latency covers both.
template <int D, int RW, int WAVES>
__global__ void __launch_bounds__(kAttnThreads) kv_attention_join_kernel(AttnArgs args, int rows) {
  __shared__ float part[WAVES == 1 ? 1 : WAVES][D];
  const nvfp4_kv_attention_args& a = args.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int ROWS = 4 / WAVES;  // of a workgroup
  const int first = WAVES == 1 ? 0 : wave;
  const uint32_t per = (uint32_t)(rows + ROWS - 1) / ROWS;  // workgroups a tile
  const uint32_t rest = blockIdx.x / per, tile = rest / (uint32_t)a.cache.kv_heads;
  const uint32_t kvh = rest - tile * (uint32_t)a.cache.kv_heads;
  const int row = (int)(blockIdx.x - rest * per) * ROWS + (WAVES == 1 ? wave : 0);
  if (row >= rows) return;
  const Parts parts = parts_of<D, RW>(args, tile, kvh);
  constexpr int C = D / 64, AHEAD = 4;  // columns C lane .. of a lane; pieces asked for ahead
  const float2* ml = parts.ml + row;
  const float* src = parts.o + (size_t)row * D + C * lane;
  const auto piece = [&](int i) { return (size_t)(i < args.splits ? i : args.splits - 1); };
  static_assert(kMaxSplits == 128, "two pieces a lane");
  float2 x0 = ml[piece(lane) * RW], x1 = ml[piece(lane + 64) * RW];
  float ahead[AHEAD][C];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
#pragma unroll
    for (int k = 0; k < C; ++k) ahead[i][k] = src[piece(first + WAVES * i) * (RW * D) + k];
  const Place at_ = place_of(args, tile, lane);
  if (row >= at_.count) return;
  int lo_any, hi_any, other;
  bounds_of(args, at_, at_.row0, lo_any, other);
  bounds_of(args, at_, at_.row0 + at_.count - 1, other, hi_any);
  const int n = cut_of(args, lo_any & ~31, hi_any).n;
  if (n == 1) return;  // its workgroup has written the result
  const Weights weight(x0, x1, lane, n);
  float o[C] = {};
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (first + WAVES * i < n) {
      const float f = weight(first + WAVES * i);
#pragma unroll
      for (int k = 0; k < C; ++k) o[k] = __builtin_fmaf(f, ahead[i][k], o[k]);
    }
#pragma unroll 8
  for (int i = first + WAVES * AHEAD; i < n; i += WAVES) {
    const float f = weight(i);
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] = __builtin_fmaf(f, src[(size_t)i * (RW * D) + k], o[k]);
  }
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int k = 0; k < C; ++k) part[wave][C * lane + k] = o[k];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int v = 1; v < WAVES; ++v) o[k] += part[v][C * lane + k];
  }
  put_row<D>(args, at_, kvh, row, lane, o, weight);
}

// ---------------------------------------------------------------- many rows
// Rows of a wavefront of the kernel below, in 16s: accumulators of D * NQ / 4
// registers a lane beside D * NQ / 8 of queries, two wavefronts a SIMD up to
// D = 192 (one at 256).
constexpr int rows_nq(int D) { return D == 64 ? 4 : 2; }

// Many rows: each wavefront has 16 NQ rows of its own and all four walk the
// same keys, 64 at a time.  The bytes of a block are dequantized once for the
// workgroup (each wavefront a quarter) into LDS, as the operands the matrix
// units take (64 lanes x 16 bytes in lane order, read without conflicts): a
// wavefront's share of the vector work drops by four, and what is left is the
// softmax.  Two buffers: a block is written while the one before is used, one
// barrier a block.
template <int D, int NQ>
__global__ void __launch_bounds__(kAttnThreads, D <= 192 ? 2 : 1)
kv_attention_rows_kernel(AttnArgs args) {
  constexpr int NCH = D / 32, NJ = D / 64, RW = 16 * NQ, BLOCK = 64;
  __shared__ f16x8 ks[2][2][2][NCH][64];  // [buffer][32 keys][t][piece][lane]
  __shared__ f16x8 vs[2][2][NJ][4][64];   // [buffer][32 keys][j][e][lane]
  __shared__ int flags[2][4];             // per wavefront: 1 a NaN scale was hidden, 2 a page is missing
  const nvfp4_kv_attention_args& a = args.a;
  const nvfp4_kv_cache& c = a.cache;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t kvh = blockIdx.x % (uint32_t)c.kv_heads;
  const uint32_t tile = args.tiles - 1 - blockIdx.x / (uint32_t)c.kv_heads;
  const Place at_ = place_of(args, tile, lane);
  if (at_.count == 0) return;
  const int count = at_.count, first = wave * RW;
  const bool mine = first < count;  // the wavefront has rows
  // the workgroup's keys, and the wavefront's
  int lo_wg, hi_wg, lo_wg_all, hi_wg_all, lo_any, hi_any, lo_all, hi_all;
  bounds_of(args, at_, at_.row0, lo_wg, hi_wg_all);
  bounds_of(args, at_, at_.row0 + count - 1, lo_wg_all, hi_wg);
  bounds_of(args, at_, at_.row0 + (mine ? first : 0), lo_any, hi_all);
  bounds_of(args, at_, at_.row0 + (mine && first + RW < count ? first + RW : count) - 1, lo_all, hi_any);

  Walk<D, NQ> w;
  {
    typename Walk<D, NQ>::RawQ rq;
    w.load_queries(args, at_, (int)kvh, mine ? first : 0, r, g, rq);
    w.start(args, (int)kvh, rq);
  }

  const int k0 = lo_wg & ~(BLOCK - 1), k1 = hi_wg;
  if (k0 < k1) {
    const Reader<D> rd(args, at_, (int)kvh, r, g);
    const int half = wave >> 1, sub = wave & 1;  // the wavefront's 32 keys of a block; t of its keys, h of its values
    // a block's quarter: NCH key pieces of 16 keys, NJ x 2 value columns of 32
    struct Quarter {
      uint32_t k[NCH], ks;
      uint2 v[NJ], vs[NJ];
      bool ok;
    };
    const auto load = [&](int t0, const Pages& p, Quarter& x) { rd.load_quarter(t0 + 32 * half, sub, p, x); };
    const auto put = [&](Quarter& x, int t0, int buf) {
      const f16x2 s01 = fp8_lo(x.ks), s23 = fp8_hi(x.ks);
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const _Float16 b = i / 2 == 0 ? s01[0] : i / 2 == 1 ? s01[1] : i / 2 == 2 ? s23[0] : s23[1];
        const f16x2 f = {b, b};
        ks[buf][half][sub][i][lane] =
            join8(fp4_pair(x.k[i], 0) * f, fp4_pair(x.k[i], 1) * f, fp4_pair(x.k[i], 2) * f, fp4_pair(x.k[i], 3) * f);
      }
      // where some row does not attend some key of the block: scales of keys
      // that no row attends, and NaN ones, become 0
      bool nan = false;
      if (!(t0 >= lo_wg_all && t0 + BLOCK <= hi_wg_all && __all(x.ok))) {
        const uint64_t in = keys_in(t0 + 32 * half + 8 * g, lo_wg, hi_wg, x.ok);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          x.vs[j].x &= (uint32_t)in;
          x.vs[j].y &= (uint32_t)(in >> 32);
          const uint32_t n0 = nan_bytes(x.vs[j].x), n1 = nan_bytes(x.vs[j].y);
          nan |= (n0 | n1) != 0;
          x.vs[j].x &= ~((n0 >> 7) * 0xFFu);
          x.vs[j].y &= ~((n1 >> 7) * 0xFFu);
        }
      }
      const int flag = (__any(nan) ? 1 : 0) | (__all(x.ok) ? 0 : 2);
      if (lane == 0) flags[buf][wave] = flag;
  #pragma unroll
      for (int j = 0; j < NJ; ++j) {
        f16x2 f[4];
        value_scales(x.vs[j], f);
        f16x8 even, odd;
        value_columns(x.v[j].x, x.v[j].y, f, even, odd);
        vs[buf][half][j][2 * sub][lane] = even;
        vs[buf][half][j][2 * sub + 1][lane] = odd;
      }
    };
    Quarter x;
    Pages p = rd.pages(k0 + 32 * half);
    const Pages p1 = rd.pages((k0 + BLOCK < k1 ? k0 + BLOCK : k0) + 32 * half);
    load(k0, p, x);
    p = p1;
    put(x, k0, 0);
    lds_sync();
    int buf = 0;
    for (int t = k0; t < k1; t += BLOCK, buf ^= 1) {
      const int tn = t + BLOCK < k1 ? t + BLOCK : t;
      const Pages pn = rd.pages((tn + BLOCK < k1 ? tn + BLOCK : tn) + 32 * half);
      load(tn, p, x);
      p = pn;
      if (mine && t < hi_any && t + BLOCK > lo_any) {
        const int flag = __builtin_amdgcn_readfirstlane(flags[buf][0] | flags[buf][1] | flags[buf][2] | flags[buf][3]);
        constexpr int U = D * NQ <= 256 ? 2 : 1;  // 32-key tiles whose scores are held at once
#pragma unroll
        for (int u0 = 0; u0 < 2; u0 += U) {
          f32x4 s[U][NQ][2];
#pragma unroll
          for (int v = 0; v < U; ++v)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < NCH; ++i) {
                const f16x8 key = ks[buf][u0 + v][k][i][lane];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                  s[v][n][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, w.q[n][i], i == 0 ? f32x4{0, 0, 0, 0} : s[v][n][k], 0, 0, 0);
              }
          const int tu = t + 32 * u0;
          if (!(tu >= lo_all && tu + 32 * U <= hi_all) || flag) {
#pragma unroll
            for (int v = 0; v < U; ++v) {
              const int tv = tu + 32 * v, key0 = tv + 8 * g;
              const Pages pv = rd.pages(tv);
              const bool ok = (uint32_t)pv.v < (uint32_t)c.num_pages;
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (!w.attends(n, key0 + i, ok)) s[v][n][i / 4][i % 4] = -__builtin_inff();
              if (flag & 1) {  // NaN values: the rows that attend them
                Raw<D> raw;
                rd.load(tv, pv, raw);
                w.hide_values(raw, key0, lo_any, hi_any);
              }
            }
          }
          float top[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            top[n] = w.top_of(n, s[0][n][0], s[0][n][1]);
            if constexpr (U == 2) top[n] = __builtin_elementwise_maximum(top[n], w.top_of(n, s[U - 1][n][0], s[U - 1][n][1]));
          }
          w.raise(top);
          f16x8 pw[U][NQ];
#pragma unroll
          for (int v = 0; v < U; ++v)
#pragma unroll
            for (int n = 0; n < NQ; ++n) pw[v][n] = w.weights(n, s[v][n][0], s[v][n][1]);
#pragma unroll
          for (int v = 0; v < U; ++v)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const f16x8 value = vs[buf][u0 + v][j][e][lane];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                  w.o[n][j][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(value, pw[v][n], w.o[n][j][e], 0, 0, 0);
              }
        }
      }
      put(x, tn, buf ^ 1);
      lds_sync();
    }
  }
  if (!mine) return;

  const float av = outer_alpha(c.v_amax[kvh], c.global_fp8_max);
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float l = w.l[n][0];
    const int row = first + 16 * n + r;
    if (row >= count) continue;
    const bool empty = w.m[n] == -__builtin_inff() && l == 0.0f;
    const float inv = empty ? 0.0f : av / l;
    const int64_t at = out_row(args, at_, (int)kvh, row);
    if (a.lse && g == 0) a.lse[at] = empty ? -__builtin_inff() : (w.m[n] + __builtin_log2f(l)) / kLog2e;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = empty ? 0u : bf16_pair(w.o[n][j][0][i] * inv, w.o[n][j][1][i] * inv);
        y[2 * i + 1] = empty ? 0u : bf16_pair(w.o[n][j][2][i] * inv, w.o[n][j][3][i] * inv);
      }
      uint4* dst = reinterpret_cast<uint4*>(a.out + at * D + 64 * j + 16 * g);
      dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
      dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// ---------------------------------------------------------------- host
AttnPlan kv_attention_plan(const nvfp4_kv_attention_args& a) {
  AttnPlan p = {};
  const int D = a.cache.head_dim, group = a.q_heads / a.cache.kv_heads;
  // Rows of an average request decide the form; every form is right for all.
  // Many rows: 2 x 2048 tokens behind 6000 cached ones 392 us against 801 in
  // the other form.  That form never cuts the keys, though, so few tiles over a
  // long axis cost what one workgroup takes to walk it: 31 tokens (124 rows)
  // behind 32768 keys of 8 heads 46 us, 32 tokens 863 and 256 tokens 878.  And
  // one form serves a whole call: 64 single tokens over 4096 keys beside a
  // chunk of 2048 take 246 us, one after the other 56 and 134.
  const int64_t batch = a.batch > 0 ? a.batch : 1;
  const int64_t rows = a.cu_q ? (a.tokens * group + batch - 1) / batch : group;
  const int nq_most = keys_nq_most(D);
  p.rows_split = rows >= 128;
  p.nq = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  p.nq = p.rows_split ? rows_nq(D) : p.nq < nq_most ? p.nq : nq_most;
  p.rows = 16 * p.nq * (p.rows_split ? 4 : 1);
  p.tiles = a.cu_q ? a.tokens * group / p.rows + a.batch + 1
                   : a.batch * ((group + p.rows - 1) / p.rows);
  const int64_t groups = p.tiles * a.cache.kv_heads;
  int64_t keys = a.max_seq_len;
  const int64_t reach = p.rows / group + 64;  // of a tile's rows and blocks, beyond the window
  if (a.window > 0 && a.window < keys - reach) keys = a.window + reach;
  p.splits = 1;
  p.chunk = 0x7FFFFF80;
  if (!p.rows_split && keys > 128) {
    // Pieces a tile's keys are cut into: the least of a small model of the
    // launch, in microseconds, over full requests and over requests of part of
    // the bound; the join is a second launch, or in the first one a memory
    // latency for every eight pieces of four rows.
    // 16 rows a wavefront: the keys come at the speed of the card (CARD a CU)
    // or, where the pieces are spread unevenly, at that of the CU with the most
    // of them (WG); each piece a CU takes costs its start and end; of uneven
    // requests part of the longest piece runs alone.  Fitted to 28 shapes timed
    // with 1 to 96 pieces (3 % over the best of them on average; at most
    // 25 %, 2 tokens each of 32 requests of 3000 keys), e.g. 64 requests of 8191 keys and 8 heads: 1 piece
    // 113 us, 2 120, 5 122; 32 of up to 8000: 1 piece 53, 2 44, 6 48; 4 of
    // 32000: 8 pieces 31, 16 33; 16 of up to 2000: 1 piece 16.8, 4 13.5, 8 17.4.
    // More rows: bound by their arithmetic, so rounds of resident workgroups,
    // each with its start and end and its keys (70 us for 3 requests of 4 drafted
    // tokens over up to 131072 where the model above takes 73 to 85).
    // Joined in the first launch against a second one: 4 rows of 1 request over
    // 8191 keys 10.8 us against 11.5, 8 rows of 32 over up to 4000 28.0 against
    // 30.4, 32 rows of 8 over up to 8192 33.3 against 28.9.
    const double cus = device_cu_count(), resident = cus * attn_waves(D, p.nq);
    const double CARD = 140.0 * 128 / D, WG = (p.nq > 1 ? 60.0 : 200.0) * 128 / D;
    // tiles that an even batch has (p.tiles has room for any)
    const int64_t even = a.tokens * group / p.rows;
    const double likely = (double)((even > a.batch ? even : a.batch) * a.cache.kv_heads);
    // rows of an average tile, and whether there is a counter for each of the
    // most tiles; the same with and without cu_q, and whether counters are
    // given or not, so that the pieces and with them the bits are the same
    const int64_t joined = rows < p.rows ? rows : p.rows;
    const bool counters = (even + a.batch + 1) * a.cache.kv_heads <= kJoinCounters;
    double best = 0;
    // past 64 pieces a CU there is nothing left to even out, only workspace to fill
    for (int n = 1; n == 1 || (n <= kMaxSplits && (n - 1) * (int64_t)128 < keys && likely * n <= 64 * cus); ++n) {
      const int64_t each = ((keys + n - 1) / n + 127) & ~(int64_t)127;
      if (n > 1 && (keys + each - 1) / each != n) continue;  // as fewer pieces
      const double piece = (double)(each < keys ? each : keys) / WG;
      double cost;
      if (p.nq > 1) {
        cost = (ceil(likely * n / resident) + ceil(0.6 * likely * n / resident)) * (5 + piece);
      } else {
        const double all = likely * (double)keys / (cus * CARD);
        const double most = ceil(likely * n / cus), some = likely * (n * 0.8 > 1 ? n * 0.8 : 1) / cus;
        const double fewer = some > 1 ? some : 1;
        cost = (all > most * piece ? all : most * piece) + 3 * most +
               (0.8 * all > fewer * piece ? 0.8 * all : fewer * piece) + 3 * fewer + 0.6 * piece;
      }
      const int64_t trips = (joined + 3) / 4 * ((n + 7) / 8);
      const double second = 7 + 0.1 * n, here = counters ? 2 + 1.5 * (double)trips : second;
      cost += n == 1 ? 0 : here < second ? here : second;
      if (n == 1 || cost < best) {
        best = cost;
        p.splits = n;
        p.join = a.counters && n > 1 && here < second;
      }
    }
    p.chunk = (int)((keys + p.splits - 1) / p.splits);
  }
  p.grid = groups * p.splits;
  p.bytes = p.splits > 1 ? (size_t)groups * p.splits * p.rows * (D + 2) * sizeof(float) : 0;
  return p;
}

template <int D>
static void launch_dim(const AttnArgs& x, const AttnPlan& p, hipStream_t s) {
  constexpr int MOST = keys_nq_most(D);
  const dim3 grid((unsigned)p.grid), block(kAttnThreads);
  if (p.rows_split) {
    hipLaunchKernelGGL((kv_attention_rows_kernel<D, rows_nq(D)>), grid, block, 0, s, x);
    return;
  }
  // rows that a tile can have
  const int rows = !x.a.cu_q && x.group < p.rows ? x.group : p.rows;
  const auto launch = [&](auto nq) {
    constexpr int NQ = decltype(nq)::value;
    hipLaunchKernelGGL((kv_attention_keys_kernel<D, NQ>), grid, block, 0, s, x);
    if (p.splits == 1 || p.join) return;
    const int64_t tiles = p.tiles * x.a.cache.kv_heads;
    if (p.splits >= kManyPieces)
      hipLaunchKernelGGL((kv_attention_join_kernel<D, 16 * NQ, 4>), dim3((unsigned)(tiles * rows)), block, 0, s, x, rows);
    else
      hipLaunchKernelGGL((kv_attention_join_kernel<D, 16 * NQ, 1>), dim3((unsigned)(tiles * ((rows + 3) / 4))), block, 0,
                         s, x, rows);
  };
  if (p.nq == 1) launch(std::integral_constant<int, 1>{});
  if constexpr (MOST >= 2) {
    if (p.nq == 2) launch(std::integral_constant<int, 2>{});
  }
  if constexpr (MOST >= 4) {
    if (p.nq == 4) launch(std::integral_constant<int, 4>{});
  }
}

hipError_t launch_kv_attention(const nvfp4_kv_attention_args& a, const AttnPlan& p, hipStream_t s) {
  AttnArgs x = {};
  x.a = a;
  if (x.a.window > INT32_MAX) x.a.window = 0;  // reaches past every position
  x.rows = p.rows;
  x.splits = p.splits;
  x.join = p.join;
  x.chunk = p.chunk;
  x.shift = __builtin_ctz((unsigned)a.cache.page_size);
  x.group = a.q_heads / a.cache.kv_heads;
  x.tiles = (uint32_t)p.tiles;
  x.tiles_per_request = (uint32_t)((x.group + p.rows - 1) / p.rows);
  switch (a.cache.head_dim) {
    case 64: launch_dim<64>(x, p, s); break;
    case 128: launch_dim<128>(x, p, s); break;
    case 192: launch_dim<192>(x, p, s); break;
    default: launch_dim<256>(x, p, s); break;
  }
  return hipGetLastError();
}

}  // namespace nvfp4
