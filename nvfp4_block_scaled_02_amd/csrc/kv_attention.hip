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
//   softmax       per lane, in the exponent of 2: the running maximum moves
//     only when a score passes it by more than 2^8 (weights stay below 2^8,
//     far inside binary16), so a tile usually needs no exchange between lanes
//     and no rescaling; the sums stay per lane until the end
//   O^T += V^T P^T  lane (m, g) reads keys 8 g .. 8 g + 7 of 4 value columns
//     as the cache holds them (8 tokens side by side); lane (n, g)'s weights
//     of keys 8 g .. 8 g + 7 are already the product's other operand.
// Nothing is transposed between lanes.
//
// Few rows (decoding, drafted tokens): the four wavefronts of a workgroup
// take every fourth tile and join through LDS, and long key ranges are split
// over workgroups whose partial results (binary32) meet in the workspace; the
// last workgroup to arrive joins them in order.  Many rows (prompts): each
// wavefront has rows of its own, and the workgroup dequantizes each block of
// keys once, into LDS.
#include "kv.hpp"

namespace nvfp4 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnThreads = 256;
constexpr int kMaxSplits = 128;
constexpr int kMaxGroups = NVFP4_KV_ATTENTION_COUNTER_BYTES / 4;
constexpr int kSlabStride = 68;  // floats of a 64-column slab row: 4 apart in the banks
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnPlan {
  int nq;           // 16-row tiles of a wavefront
  bool rows_split;  // wavefronts take rows of their own (else every fourth key tile)
  int rows;         // rows of a workgroup
  int splits;       // most workgroups over one tile's keys
  int chunk;        // keys a workgroup is meant to take
  int64_t tiles;    // row tiles over all requests, at most
  int64_t grid;
  size_t bytes;     // of workspace
};

struct AttnArgs {
  nvfp4_kv_attention_args a;
  int rows, splits, chunk, shift, group;
  uint32_t tiles, tiles_per_request;
};

// ---------------------------------------------------------------- lanes
__device__ __forceinline__ uint32_t u32(float v) { return __float_as_uint(v); }

// max / sum over the four lanes of a query (lane % 16 equal), in all of them
__device__ __forceinline__ float max_over_g(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(u32(v), u32(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(u32(v), u32(v), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_g(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(u32(v), u32(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(u32(v), u32(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
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

// One tile's worth of addresses.  The table entry of a group past the last
// key is that of the last one (its tokens are masked).
struct Reader {
  const nvfp4_kv_cache& c;
  const int32_t* table;  // of the request
  int last;              // last table entry that may be read
  int shift, kvh, r, g;
  __device__ __forceinline__ Pages pages(int tile0) const {
    Pages p;
    if (shift >= 5) {  // the tile lies in one page: a scalar load
      const int i = tile0 >> shift;
      p.k = p.v = table[i < last ? i : last];
    } else {
      const int ik = (tile0 + 8 * (r >> 2)) >> shift, iv = (tile0 + 8 * g) >> shift;
      p.k = table[ik < last ? ik : last];
      p.v = table[iv < last ? iv : last];
    }
    return p;
  }
  // Codes and scales of one 16-key product (t of the tile): D / 8 bytes and D /
  // 64 scale bytes of the lane's key.
  template <int D>
  __device__ __forceinline__ void load_keys(int tile0, int t, uint32_t page, uint32_t (&k)[D / 32], uint32_t& sc) const {
    constexpr int NCH = D / 32;
    // tokens from the start of the cache (page < 2^31, heads and page size <= 2^10)
    const uint64_t kt = (uint64_t)page * (uint32_t)(c.kv_heads << shift) + ((uint64_t)kvh << shift) +
                        (((uint32_t)tile0 + 8 * (r >> 2)) & ((1u << shift) - 1)) + (r & 3) + 4 * t;
    const uint8_t* p = c.k_codes + kt * (D / 2) + g * (D / 8);
    const uint8_t* s = c.k_scales + kt * (D / 16) + g * (NCH / 2);
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
  __device__ __forceinline__ uint64_t value_tokens(int tile0, uint32_t page) const {
    return (uint64_t)page * (uint32_t)(c.kv_heads << shift) + ((uint64_t)kvh << shift) +
           (((uint32_t)tile0 + 8 * g) & ((1u << shift) - 1));
  }
  // Product t of the tile's keys, half h (one column pair of two) of its values.
  template <int D, class Q>
  __device__ __forceinline__ void load_quarter(int tile0, int sub, const Pages& p, Q& x) const {
    const uint32_t n = (uint32_t)c.num_pages;
    load_keys<D>(tile0, sub, (uint32_t)p.k < n ? (uint32_t)p.k : 0u, x.k, x.ks);
    x.ok = (uint32_t)p.v < n;
    const uint64_t vt = value_tokens(tile0, x.ok ? (uint32_t)p.v : 0u);
    const uint8_t* vc = c.v_codes + vt * (D / 2) + 16 * r + 8 * sub;
    const uint8_t* vs = c.v_scales + vt * (D / 16) + 8 * (r >> 2);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      x.v[j] = *reinterpret_cast<const uint2*>(vc + 256 * j);
      x.vs[j] = *reinterpret_cast<const uint2*>(vs + 32 * j);
    }
  }
  template <int D>
  __device__ __forceinline__ void load(int tile0, const Pages& p, Raw<D>& w) const {
    constexpr int NCH = Raw<D>::NCH;
    const uint32_t n = (uint32_t)c.num_pages;
    const uint32_t pk = (uint32_t)p.k < n ? (uint32_t)p.k : 0u;
#pragma unroll
    for (int t = 0; t < 2; ++t) load_keys<D>(tile0, t, pk, w.k[t], w.ks[t]);
    w.ok = (uint32_t)p.v < n;
    const uint64_t vt = value_tokens(tile0, w.ok ? (uint32_t)p.v : 0u);
    const uint8_t* vc = c.v_codes + vt * (D / 2) + 16 * r;
    const uint8_t* vs = c.v_scales + vt * (D / 16) + 8 * (r >> 2);
#pragma unroll
    for (int j = 0; j < NCH / 2; ++j) {
      w.v[j] = *reinterpret_cast<const uint4*>(vc + 256 * j);
      w.vs[j] = *reinterpret_cast<const uint2*>(vs + 32 * j);
    }
  }
};

// A byte holds two columns of one token; the products want 8 tokens of one
// column.  x, y: the bytes of tokens 0..3 and 4..7 of a column pair; nibbles of
// neighbouring bytes change places, and a conversion takes two tokens at once.
__device__ __forceinline__ void value_columns(uint32_t x, uint32_t y, const f16x2 (&f)[4], f16x8& even, f16x8& odd) {
  const uint32_t M = 0x000F000Fu;
  const uint32_t x4 = x >> 4, y4 = y >> 4, x8 = x >> 8, y8 = y >> 8;
  const uint32_t xe = (x & M) | (x4 & ~M), ye = (y & M) | (y4 & ~M);
  const uint32_t xo = (x4 & M) | (x8 & ~M), yo = (y4 & M) | (y8 & ~M);
  even = join8(fp4_pair(xe, 0) * f[0], fp4_pair(xe, 2) * f[1], fp4_pair(ye, 0) * f[2], fp4_pair(ye, 2) * f[3]);
  odd = join8(fp4_pair(xo, 0) * f[0], fp4_pair(xo, 2) * f[1], fp4_pair(yo, 0) * f[2], fp4_pair(yo, 2) * f[3]);
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

// Row of a request -> its token among the request's, and its head in the group.
__device__ __forceinline__ int64_t split_row(int64_t row, int group, int64_t& head) {
  const uint32_t r = (uint32_t)row;
  if ((uint64_t)row >> 32) {
    const int64_t t = row / group;
    head = row - t * group;
    return t;
  }
  head = r % (uint32_t)group;
  return r / (uint32_t)group;
}

// A workgroup's place: its request and rows.
struct Place {
  int64_t b;           // request (batch: rows that belong to none)
  int64_t begin, end;  // its rows of q
  int64_t row0;        // first row (token x head of the group) of the workgroup
  int count;           // rows of the workgroup; 0: nothing to do
  int len;             // keys [0, len)
  int64_t pos0;        // position of the request's first query
  __device__ __forceinline__ void bounds(const nvfp4_kv_attention_args& a, int group, int64_t row, int& lo,
                                         int& hi) const {
    int64_t head;
    const int64_t p = pos0 + split_row(row, group, head);
    const int64_t h = a.causal && p + 1 < len ? p + 1 : len;
    const int64_t w = a.window > 0 ? p - a.window + 1 : 0;
    hi = (int)(h < 0 ? 0 : h);
    lo = (int)(w < 0 ? 0 : w > len ? len : w);
  }
};

__device__ __forceinline__ Place place_of(const AttnArgs& args, uint32_t tile, int lane) {
  const nvfp4_kv_attention_args& a = args.a;
  Place p;
  int64_t local;
  p.count = 0;
  if (!a.cu_q) {
    p.b = tile / args.tiles_per_request;
    local = tile - (uint32_t)p.b * args.tiles_per_request;
    p.begin = p.b;
    p.end = p.b + 1;
  } else {
    // request b's tiles begin at floor(cu_q[b] * group / rows) + b; rows past
    // cu_q[batch] count as a request of length 0.  64 probes at a time.
    const auto cu = [&](int64_t i) {
      const int64_t v = a.cu_q[i];
      return v < 0 ? 0 : v < a.tokens ? v : a.tokens;
    };
    const auto start = [&](int64_t i) { return (uint64_t)cu(i) * (uint32_t)args.group / (uint32_t)args.rows + i; };
    int64_t lo = 0, n = a.batch + 1;
    while (n > 1) {
      const int64_t step = (n + 63) / 64, i = lane * step;
      const bool before = i < n && start(lo + i) <= tile;
      const int hits = __popcll(__ballot(before));
      const int64_t k = hits > 0 ? hits - 1 : 0;
      lo += k * step;
      n = n - k * step < step ? n - k * step : step;
    }
    p.b = lo;
    local = (int64_t)tile - (int64_t)start(lo);
    if (local < 0) return p;
    p.begin = cu(lo);
    p.end = lo < a.batch ? cu(lo + 1) : a.tokens;
    p.end = p.end < p.begin ? p.begin : p.end;
  }
  const int64_t rows = (p.end - p.begin) * args.group;
  p.row0 = local * args.rows;
  if (p.row0 >= rows) return p;
  p.count = (int)(rows - p.row0 < args.rows ? rows - p.row0 : args.rows);
  const int64_t seq = p.b < a.batch ? a.seq_lens[p.b] : 0;
  const int64_t room = a.table_width << args.shift;
  p.len = (int)(seq < 0 ? 0 : seq < room ? seq : room);
  p.pos0 = seq - (p.end - p.begin);
  return p;
}

// ---------------------------------------------------------------- one tile
template <int D, int NQ>
struct Walk {
  static constexpr int NCH = D / 32, NJ = D / 64;
  f16x8 q[NQ][NCH];
  f32x4 o[NQ][NJ][4];  // [j][e][i]: query n, column 64 j + 16 g + 4 i + e
  float factor[NQ];    // binary32 factor of a row's scores
  float m[NQ], thr[NQ], l[NQ];
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
    f16x8 p[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) p[n] = weights(n, s[n][0], s[n][1]);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint2 vs = w.vs[j];
      const f16x2 f[4] = {fp8_lo(vs.x), fp8_hi(vs.x), fp8_lo(vs.y), fp8_hi(vs.y)};
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

  // The softmax weights of query n's scores of a tile (binary16), added to
  // its sum; its maximum moves first where a score passes it by 2^8.
  __device__ __forceinline__ f16x8 weights(int n, const f32x4& s0, const f32x4& s1) {
    // factor >= 0: the largest product is that of the largest score.  A NaN
    // score never moves the maximum; its weight and the row become NaN.
    const float top = factor[n] * max3(max3(s0[0], s0[1], s0[2]), max3(s0[3], s1[0], s1[1]), max3(s1[2], s1[3], s1[3]));
    if (__any(top > thr[n])) {
      const float was = m[n];
      m[n] = __builtin_fmaxf(m[n], max_over_g(top));
      thr[n] = m[n] + 8.0f;
      const float keep = was == m[n] || was == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(was - m[n]);
      l[n] *= keep;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] *= keep;
    }
    const float base = m[n] == -__builtin_inff() ? 0.0f : -m[n];
    float t[8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(i < 4 ? s0[i % 4] : s1[i % 4], factor[n], base));
      sum += t[i];
    }
    l[n] += sum;
    f16x8 p;
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (_Float16)t[i];
    return p;
  }

  // Query rows [first, first + 16 NQ) of the workgroup's `count` (the spare
  // ones repeat the last) into binary16, each scaled by a power of two.
  template <class RowAt, class Bounds>
  __device__ __forceinline__ void start(const nvfp4_kv_attention_args& a, int group, int kvh, int first, int count,
                                        int r, int g, const RowAt& row_at, const Bounds& bounds,
                                        int64_t begin) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      int row = first + 16 * n + r;
      row = row < count ? row : count - 1;
      const int64_t rr = row_at(row);
      bounds(rr, lo[n], hi[n]);
      int64_t head;
      const int64_t token = split_row(rr, group, head);
      const uint16_t* src = a.q + (begin + token) * a.q_stride + ((int64_t)kvh * group + head) * D + g * (D / 4);
      uint4 raw[NCH];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        raw[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
        const uint32_t t = chunk_abs_max_bits(raw[i]);
        top = top > t ? top : t;
      }
      // the row's largest magnitude: bf16 patterns order like their values
      float topf = __uint_as_float(top << 16);
      topf = top >= 0x7F80u ? 1.0f : topf;  // infinities and NaN travel as they are
      topf = max_over_g(topf);
      int e = 254 - (int)(u32(topf) >> 23);  // exponent field of 2^-floor(log2 top)
      e = topf == 0.0f ? 127 : e < 1 ? 1 : e > 254 ? 254 : e;
      // a negative scale turns the row's sign, so that factor >= 0
      const float up = __builtin_copysignf(__uint_as_float((uint32_t)e << 23), a.scale);
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q[n][i][2 * k] = (_Float16)(bf16_lo(x[k]) * up);
          q[n][i][2 * k + 1] = (_Float16)(bf16_hi(x[k]) * up);
        }
      }
      factor[n] = __builtin_ldexpf(outer_alpha(a.cache.k_amax[kvh], a.cache.global_fp8_max) *
                                       __builtin_fabsf(a.scale) * kLog2e, 127 - e);
      // a score of -inf stays below every other one
      factor[n] = factor[n] == 0.0f ? 0x1p-126f : factor[n];
      m[n] = thr[n] = -__builtin_inff();
      l[n] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e2 = 0; e2 < 4; ++e2) o[n][j][e2] = f32x4{0, 0, 0, 0};
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
// Partial results of a split tile: per (tile, head) group and split, rows x
// (D values, then maximum and sum), written and read where the whole GPU sees
// them (no cache holds a stale copy).
__device__ __forceinline__ void put2(float* p, float a, float b) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), (uint64_t)u32(b) << 32 | u32(a), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// weight of a partial result with maximum m under the joint maximum M
__device__ __forceinline__ float join_weight(float m, float M) {
  return m == M ? 1.0f : __builtin_amdgcn_exp2f(m - M);
}

// Wavefronts of a SIMD that the registers are shared out for: as many as fit
// without spilling (512 registers a lane at one wavefront).
constexpr int attn_waves(int D, int NQ) {
  return D * NQ <= 64 ? 4 : D * NQ <= 128 ? 3 : D * NQ <= 256 ? 2 : 1;
}

// Few rows: the wavefronts of a workgroup take every fourth key tile.
template <int D, int NQ>
__global__ void __launch_bounds__(kAttnThreads, attn_waves(D, NQ))
kv_attention_keys_kernel(AttnArgs args) {
  constexpr int NJ = D / 64, RW = 16 * NQ;
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
  const auto bounds = [&](int64_t row, int& lo, int& hi) { at_.bounds(a, args.group, row, lo, hi); };
  // keys that any row attends, and those that all attend: bounds ascend with the row
  int lo_any, hi_any, lo_all, hi_all;
  bounds(at_.row0, lo_any, hi_all);
  bounds(at_.row0 + count - 1, lo_all, hi_any);
  // this workgroup's share
  int k0 = lo_any & ~31, k1 = hi_any, nsplit = 1;
  if (args.splits > 1) {
    const int keys = k1 > k0 ? k1 - k0 : 0;
    nsplit = (keys + args.chunk - 1) / args.chunk;
    nsplit = nsplit < 1 ? 1 : nsplit < args.splits ? nsplit : args.splits;
    const int each = ((keys + nsplit - 1) / nsplit + 127) & ~127;
    nsplit = each > 0 ? (keys + each - 1) / each : 1;
    nsplit = nsplit < 1 ? 1 : nsplit;
    if ((int)split >= nsplit) return;
    k0 += (int)split * each;
    k1 = k1 - k0 < each ? k1 : k0 + each;
  }

  Walk<D, NQ> w;
  w.start(a, args.group, (int)kvh, 0, count, r, g, [&](int row) { return at_.row0 + row; }, bounds,
          at_.begin);

  // the walk: the next tile's bytes are in flight while one is computed, and
  // the table entries of the one after
  {
    constexpr int STEP = 128;
    const int t0 = k0 + 32 * __builtin_amdgcn_readfirstlane(wave);
    if (t0 < k1) {
      const Reader rd = {c, a.block_table + at_.b * a.table_width, (at_.len - 1) >> args.shift, args.shift,
                         (int)kvh, r, g};
      Raw<D> cur, nxt;
      Pages p = rd.pages(t0);
      rd.load(t0, p, cur);
      p = rd.pages(t0 + STEP < k1 ? t0 + STEP : t0);
      for (int t = t0; t < k1; t += STEP) {
        const int tn = t + STEP < k1 ? t + STEP : t;
        rd.load(tn, p, nxt);
        p = rd.pages(tn + STEP < k1 ? tn + STEP : tn);
        const bool whole = t >= lo_all && t + 32 <= hi_all && __all(cur.ok);
        w.tile(cur, t, g, lo_any, hi_any, !whole);
        cur = nxt;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n) w.l[n] = sum_over_g(w.l[n]);

  const float av = outer_alpha(c.v_amax[kvh], c.global_fp8_max);
  const auto out_row = [&](int row) {  // token * q_heads + head
    int64_t head;
    const int64_t token = split_row(at_.row0 + row, args.group, head);
    return (at_.begin + token) * a.q_heads + (int64_t)kvh * args.group + head;
  };
  {
    // join the four wavefronts: their maxima and sums, then 64 columns at a time
    __shared__ __align__(16) float slab[4 * RW * kSlabStride];
    __shared__ float ms[4][RW], ls[4][RW];
    __shared__ bool last;
    if (g == 0) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        ms[wave][16 * n + r] = w.m[n];
        ls[wave][16 * n + r] = w.l[n];
      }
    }
    __syncthreads();
    const size_t row_floats = D + 2;
    const uint64_t group_at = (uint64_t)tile * (uint32_t)c.kv_heads + kvh;
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + NVFP4_KV_ATTENTION_COUNTER_BYTES) +
                   group_at * args.splits * RW * row_floats;
    float* mine = parts + (size_t)split * RW * row_floats;
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
          const int64_t at = out_row(row);
          uint2 y = make_uint2(bf16_pair(x.x * inv, x.y * inv), bf16_pair(x.z * inv, x.w * inv));
          if (empty) y = make_uint2(0, 0);
          *reinterpret_cast<uint2*>(a.out + at * D + 64 * j + col) = y;
          if (a.lse && j == 0 && col == 0) a.lse[at] = empty ? -__builtin_inff() : (M + __builtin_log2f(L)) / kLog2e;
        } else {
          float* dst = mine + (size_t)row * row_floats;
          put2(dst + 64 * j + col, x.x, x.y);
          put2(dst + 64 * j + col + 2, x.z, x.w);
          if (j == 0 && col == 0) put2(dst + D, M, L);
        }
      }
    }
    if (nsplit == 1) return;
    // arrive once the partial result has reached the level that all see
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    uint32_t* counter = static_cast<uint32_t*>(a.workspace) + group_at;
    if (threadIdx.x == 0) {
      last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)nsplit - 1;
      if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!last) return;
    // the last workgroup joins the splits in order: weights first (in the
    // slab: at most 128 splits x 16 rows per pass), then the columns
    float* wt = slab;  // [16 rows][kMaxSplits]
#pragma unroll 1
    for (int n = 0; n < NQ; ++n) {
      const int row = 16 * n + (threadIdx.x >> 4), sub = threadIdx.x & 15;
      const bool on = row < count;
      const float* src = parts + (size_t)(on ? row : 0) * row_floats;
      const size_t next = RW * row_floats;
      float M = -__builtin_inff();
      for (int s = sub; s < nsplit; s += 16) M = __builtin_fmaxf(M, get2(src + s * next + D).x);
      M = __builtin_fmaxf(M, __uint_as_float(xor1_u32(u32(M))));
      M = __builtin_fmaxf(M, __uint_as_float(xor2_u32(u32(M))));
      M = __builtin_fmaxf(M, __uint_as_float(xor4_u32(u32(M))));
      M = __builtin_fmaxf(M, __uint_as_float(xor8_u32(u32(M))));
      float L = 0.0f;
      __syncthreads();
      for (int s = sub; s < nsplit; s += 16) {
        const float2 ml = get2(src + s * next + D);
        const float f = join_weight(ml.x, M);
        wt[(threadIdx.x >> 4) * kMaxSplits + s] = f;
        L += f * ml.y;
      }
      L += __uint_as_float(xor1_u32(u32(L)));
      L += __uint_as_float(xor2_u32(u32(L)));
      L += __uint_as_float(xor4_u32(u32(L)));
      L += __uint_as_float(xor8_u32(u32(L)));
      __syncthreads();
      if (!on) continue;
      const bool empty = M == -__builtin_inff() && L == 0.0f;
      const float inv = empty ? 0.0f : av / L;
      const int64_t at = out_row(row);
      if (a.lse && sub == 0) a.lse[at] = empty ? -__builtin_inff() : (M + __builtin_log2f(L)) / kLog2e;
      const float* f = wt + (threadIdx.x >> 4) * kMaxSplits;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        float4 x = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int s = 0; s < nsplit; ++s) {
          const float2 y = get2(src + s * next + 64 * j + col), z = get2(src + s * next + 64 * j + col + 2);
          x.x += f[s] * y.x; x.y += f[s] * y.y; x.z += f[s] * z.x; x.w += f[s] * z.y;
        }
        uint2 y = make_uint2(bf16_pair(x.x * inv, x.y * inv), bf16_pair(x.z * inv, x.w * inv));
        if (empty) y = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(a.out + at * D + 64 * j + col) = y;
      }
    }
  }
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
  const auto bounds = [&](int64_t row, int& lo, int& hi) { at_.bounds(a, args.group, row, lo, hi); };
  // bounds ascend with the row: the workgroup's keys, and the wavefront's
  int lo_wg, hi_wg, lo_wg_all, hi_wg_all, lo_any, hi_any, lo_all, hi_all;
  bounds(at_.row0, lo_wg, hi_wg_all);
  bounds(at_.row0 + count - 1, lo_wg_all, hi_wg);
  bounds(at_.row0 + (mine ? first : 0), lo_any, hi_all);
  bounds(at_.row0 + (mine && first + RW < count ? first + RW : count) - 1, lo_all, hi_any);

  Walk<D, NQ> w;
  w.start(a, args.group, (int)kvh, mine ? first : 0, count, r, g, [&](int row) { return at_.row0 + row; },
          bounds, at_.begin);

  const int k0 = lo_wg & ~(BLOCK - 1), k1 = hi_wg;
  if (k0 < k1) {
    const Reader rd = {c, a.block_table + at_.b * a.table_width, (at_.len - 1) >> args.shift, args.shift,
                       (int)kvh, r, g};
    const int half = wave >> 1, sub = wave & 1;  // the wavefront's 32 keys of a block; t of its keys, h of its values
    // a block's quarter: NCH key pieces of 16 keys, NJ x 2 value columns of 32
    struct Quarter {
      uint32_t k[NCH], ks;
      uint2 v[NJ], vs[NJ];
      bool ok;
    };
    const auto load = [&](int t0, const Pages& p, Quarter& x) { rd.template load_quarter<D>(t0 + 32 * half, sub, p, x); };
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
        const f16x2 f[4] = {fp8_lo(x.vs[j].x), fp8_hi(x.vs[j].x), fp8_lo(x.vs[j].y), fp8_hi(x.vs[j].y)};
        f16x8 even, odd;
        value_columns(x.v[j].x, x.v[j].y, f, even, odd);
        vs[buf][half][j][2 * sub][lane] = even;
        vs[buf][half][j][2 * sub + 1][lane] = odd;
      }
    };
    Quarter x;
    Pages p = rd.pages(k0 + 32 * half);
    load(k0, p, x);
    p = rd.pages((k0 + BLOCK < k1 ? k0 + BLOCK : k0) + 32 * half);
    put(x, k0, 0);
    lds_sync();
    int buf = 0;
    for (int t = k0; t < k1; t += BLOCK, buf ^= 1) {
      const int tn = t + BLOCK < k1 ? t + BLOCK : t;
      load(tn, p, x);
      p = rd.pages((tn + BLOCK < k1 ? tn + BLOCK : tn) + 32 * half);
      if (mine && t < hi_any && t + BLOCK > lo_any) {
        const int flag = __builtin_amdgcn_readfirstlane(flags[buf][0] | flags[buf][1] | flags[buf][2] | flags[buf][3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tu = t + 32 * u, key0 = tu + 8 * g;
          f32x4 s[NQ][2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
              const f16x8 key = ks[buf][u][k][i][lane];
#pragma unroll
              for (int n = 0; n < NQ; ++n)
                s[n][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key, w.q[n][i], i == 0 ? f32x4{0, 0, 0, 0} : s[n][k], 0, 0, 0);
            }
          if (!(tu >= lo_all && tu + 32 <= hi_all) || flag) {
            const Pages pu = rd.pages(tu);
            const bool ok = (uint32_t)pu.v < (uint32_t)c.num_pages;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (!w.attends(n, key0 + i, ok)) s[n][i / 4][i % 4] = -__builtin_inff();
            if (flag & 1) {  // NaN values: the rows that attend them
              Raw<D> raw;
              rd.load(tu, pu, raw);
              w.hide_values(raw, key0, lo_any, hi_any);
            }
          }
          f16x8 pw[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) pw[n] = w.weights(n, s[n][0], s[n][1]);
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f16x8 v = vs[buf][u][j][e][lane];
#pragma unroll
              for (int n = 0; n < NQ; ++n)
                w.o[n][j][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pw[n], w.o[n][j][e], 0, 0, 0);
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
    const float l = sum_over_g(w.l[n]);
    const int row = first + 16 * n + r;
    if (row >= count) continue;
    const bool empty = w.m[n] == -__builtin_inff() && l == 0.0f;
    const float inv = empty ? 0.0f : av / l;
    int64_t head;
    const int64_t token = split_row(at_.row0 + row, args.group, head);
    const int64_t at = (at_.begin + token) * a.q_heads + (int64_t)kvh * args.group + head;
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
static AttnPlan plan_of(const nvfp4_kv_attention_args& a) {
  AttnPlan p = {};
  const int D = a.cache.head_dim, group = a.q_heads / a.cache.kv_heads;
  // rows of an average request decide the form; every form is right for all
  const int64_t batch = a.batch > 0 ? a.batch : 1;
  const int64_t rows = a.cu_q ? (a.tokens * group + batch - 1) / batch : group;
  const int nq_most = D <= 128 ? 4 : 2;  // registers: NQ * D accumulator values a lane / 16
  p.rows_split = rows >= 128;
  p.nq = p.rows_split ? rows_nq(D) : rows <= 16 ? 1 : rows <= 32 ? 2 : nq_most;
  p.rows = 16 * p.nq * (p.rows_split ? 4 : 1);
  p.tiles = a.cu_q ? a.tokens * group / p.rows + a.batch + 1
                   : a.batch * ((group + p.rows - 1) / p.rows);
  const int64_t groups = p.tiles * a.cache.kv_heads;
  int64_t keys = a.max_seq_len;
  if (a.window > 0 && a.window + p.rows / group + 64 < keys) keys = a.window + p.rows / group + 64;
  p.splits = 1;
  p.chunk = 0x7FFFFF80;
  if (!p.rows_split && groups <= kMaxGroups && keys > 128) {
    // keys a workgroup takes: halved from 4096 until four workgroups for each
    // compute unit have work at the bound, 128 (one tile a wavefront) at least
    const int64_t want = 4 * (int64_t)device_cu_count();
    int64_t chunk = 4096;
    while (chunk > 128 && groups * ((keys + chunk - 1) / chunk) < want) chunk /= 2;
    int64_t splits = (keys + chunk - 1) / chunk;
    if (splits > kMaxSplits) splits = kMaxSplits;
    p.splits = (int)splits;
    p.chunk = (int)chunk;
  }
  p.grid = groups * p.splits;
  p.bytes = p.splits > 1 ? NVFP4_KV_ATTENTION_COUNTER_BYTES +
                               (size_t)groups * p.splits * 16 * p.nq * (D + 2) * sizeof(float)
                         : 0;
  return p;
}

size_t kv_attention_workspace(const nvfp4_kv_attention_args& a) { return plan_of(a).bytes; }

template <int D>
static void launch_dim(const AttnArgs& x, const AttnPlan& p, hipStream_t s) {
  constexpr int MOST = D <= 128 ? 4 : 2;
  const dim3 grid((unsigned)p.grid), block(kAttnThreads);
  if (p.rows_split) hipLaunchKernelGGL((kv_attention_rows_kernel<D, rows_nq(D)>), grid, block, 0, s, x);
  else if (p.nq == 1) hipLaunchKernelGGL((kv_attention_keys_kernel<D, 1>), grid, block, 0, s, x);
  else if (p.nq == 2) hipLaunchKernelGGL((kv_attention_keys_kernel<D, 2>), grid, block, 0, s, x);
  else hipLaunchKernelGGL((kv_attention_keys_kernel<D, MOST>), grid, block, 0, s, x);
}

hipError_t launch_kv_attention(const nvfp4_kv_attention_args& a, hipStream_t s) {
  const AttnPlan p = plan_of(a);
  if (p.grid > INT32_MAX) return hipErrorInvalidValue;
  AttnArgs x = {};
  x.a = a;
  x.rows = p.rows;
  x.splits = p.splits;
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
