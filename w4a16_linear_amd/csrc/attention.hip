// Attention of one token, or of a tree of drafted tokens, per sequence over a
// paged cache, straight from the cache's codes:
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  lse = ln sum_j exp(scale q . k_j).
//
// One pass over the keys with the running maximum and sum of the softmax, in
// base 2: m = max s_j, l = sum 2^(s_j - m), o = sum 2^(s_j - m) v_j with
// s_j = scale log2(e) (q . code_j) kscale_j; results of different keys join by
// rescaling to the common maximum.
//
// Everything between the cache and the accumulators stays in registers.  A wave
// takes 32 keys at a time and v_mfma_f32_16x16x32_bf16 (lane 16 g + c holds
// rows/columns c at k = 8 g .. 8 g + 7 of its operands, and rows 4 g .. 4 g + 3 of
// column c of the result):
//   S^T = K Q^T: K the A operand, so each lane loads the codes of one key
//     (row c of a 16-key tile) and needs no exchange; the order of the head's
//     dimensions within the products is free, and is the one that makes these
//     loads wide (`KeyTile::dim_at`);
//   O^T = V^T P^T: a lane of S^T holds, of query c, keys 4 g .. 4 g + 3 of both
//     16-key tiles: exactly a B operand if the keys of the product are taken in
//     that order.  The A operand then is dimension c' of those eight keys: a
//     lane loads dim/16 consecutive dimensions of its eight keys and turns them
//     by byte permutes; of result tile j the lane's row c is dimension
//     dim/16 * c + j, so a lane ends with consecutive dimensions of its query.
// Codes become bfloat16 exactly (e4m3 by conversion, OPQ by the level planes);
// the rows' scales multiply the scores and, for values, the weights p.
//
// Query heads that share a kv head, times the drafted tokens, are the rows of Q
// (1 to 4 tiles of 16 in a workgroup); the four waves of a workgroup take every
// fourth 32 keys and join at its end; long sequences are split over workgroups
// and joined by a second kernel.
#include "attention_internal.hpp"
#include "decode.hpp"

namespace opq {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kStep = 32;             // keys a wave takes at a time
constexpr int kRound = kWaves * kStep;  // keys a workgroup takes at a time
constexpr float kLowest = -3.0e38f;     // running maximum of a row that saw nothing
// The maximum is raised only when a score exceeds it by more than this (in powers
// of two): the weights then stay below 2^8, which float32 sums and bfloat16
// weights hold as well as weights below 1, and most steps skip the rescaling.
constexpr float kSlack = 8.0f;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float floatx2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const floatx2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}
__device__ __forceinline__ bf16x8_t frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, u32x4_t{a, b, c, d});
}
template <bool kHigh>
__device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, kHigh));
}

template <int N>
struct Words {
  uint32_t w[N];
};
// N words at p, which is aligned to 4 N bytes (16 at most).
template <int N>
__device__ __forceinline__ Words<N> load_words(const char* p) {
  Words<N> r;
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4_t v = reinterpret_cast<const u32x4_t*>(p)[i];
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
    static_assert(N == 1, "");
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}

template <int FMT, int D>
constexpr int kRowBytes = FMT == OPQ_CACHE_BF16 ? 2 * D : FMT == OPQ_CACHE_FP8 ? D : D / 2;

// One lane's part of a 16-key tile of K: a quarter (g) of key c's dimensions.
template <int FMT, int D>
struct KeyTile;

template <int D>
struct KeyTile<OPQ_CACHE_BF16, D> {
  Words<D / 8> raw;
  // first of the eight dimensions that lane quarter g holds in product step s
  __device__ static int dim_at(int s, int g) { return 32 * s + 8 * g; }
  __device__ __forceinline__ void load(const char* row, const char*, int g) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const Words<4> t = load_words<4>(row + 64 * s + 16 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) raw.w[4 * s + i] = t.w[i];
    }
  }
  __device__ __forceinline__ bf16x8_t at(int s, const RowLut&) const {
    return frag(raw.w[4 * s], raw.w[4 * s + 1], raw.w[4 * s + 2], raw.w[4 * s + 3]);
  }
};

template <int D>
struct KeyTile<OPQ_CACHE_FP8, D> {
  Words<D / 16> raw;
  __device__ static int dim_at(int s, int g) { return 64 * (s >> 1) + 16 * g + 8 * (s & 1); }
  __device__ __forceinline__ void load(const char* row, const char*, int g) {
#pragma unroll
    for (int s = 0; s < D / 64; ++s) {
      const Words<4> t = load_words<4>(row + 64 * s + 16 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) raw.w[4 * s + i] = t.w[i];
    }
  }
  __device__ __forceinline__ bf16x8_t at(int s, const RowLut&) const {
    const uint32_t a = raw.w[2 * s], b = raw.w[2 * s + 1];
    return frag(from_e4m3<false>(a), from_e4m3<true>(a), from_e4m3<false>(b), from_e4m3<true>(b));
  }
};

template <int D>
struct KeyTile<OPQ_CACHE_OPQ4, D> {
  static constexpr int kSteps = D / 32;
  Words<kSteps> raw;
  uint64_t sign;  // byte s: signs of step s
  __device__ static int dim_at(int s, int g) { return 8 * (kSteps * g + s); }
  __device__ __forceinline__ void load(const char* row, const char* signs, int g) {
    raw = load_words<kSteps>(row + 4 * kSteps * g);
    const char* p = signs + kSteps * g;
    if (kSteps == 2) sign = *reinterpret_cast<const uint16_t*>(p);
    else if (kSteps == 4) sign = *reinterpret_cast<const uint32_t*>(p);
    else sign = *reinterpret_cast<const uint64_t*>(p);
  }
  __device__ __forceinline__ bf16x8_t at(int s, const RowLut& lut) const {
    uint32_t o[4];
    decode_word_split(raw.w[s], (uint32_t)(sign >> (8 * s)) & 0xFFu, lut, o);
    return frag(o[0], o[1], o[2], o[3]);
  }
};

// One lane's part of 32 keys of V: dimensions D/16 * c .. of its eight keys, key
// i of the lane in element i.
template <int FMT, int D>
struct ValueTile;

// Result tiles 2 t and 2 t + 1 from pairs of dimensions of eight keys.
__device__ __forceinline__ void turn_pairs(const uint32_t (&p)[8], bf16x8_t& even, bf16x8_t& odd) {
  uint32_t e[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
    o[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
  }
  even = frag(e[0], e[1], e[2], e[3]);
  odd = frag(o[0], o[1], o[2], o[3]);
}

template <int D>
struct ValueTile<OPQ_CACHE_BF16, D> {
  static constexpr int kWords = D / 32;
  static constexpr int kTogether = 2;  // result tiles that one call of tiles() gives
  Words<kWords> raw[8];
  __device__ __forceinline__ void load(int i, const char* row, const char*, int c) {
    raw[i] = load_words<kWords>(row + 4 * kWords * c);
  }
  __device__ __forceinline__ void tiles(int t, const RowLut&, bf16x8_t (&v)[kTogether]) const {
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = raw[i].w[t];
    turn_pairs(p, v[0], v[1]);
  }
};

template <int D>
struct ValueTile<OPQ_CACHE_FP8, D> {
  static constexpr int kWords = D / 64;
  static constexpr int kTogether = 4;
  Words<kWords> raw[8];
  __device__ __forceinline__ void load(int i, const char* row, const char*, int c) {
    raw[i] = load_words<kWords>(row + 4 * kWords * c);
  }
  __device__ __forceinline__ void tiles(int t, const RowLut&, bf16x8_t (&v)[kTogether]) const {
    uint32_t o[kTogether][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes of two keys, dimension by dimension: each half converts to one pair
      const uint32_t a = raw[2 * i].w[t], b = raw[2 * i + 1].w[t];
      const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x05010400u);
      const uint32_t hi = __builtin_amdgcn_perm(b, a, 0x07030602u);
      o[0][i] = from_e4m3<false>(lo);
      o[1][i] = from_e4m3<true>(lo);
      o[2][i] = from_e4m3<false>(hi);
      o[3][i] = from_e4m3<true>(hi);
    }
#pragma unroll
    for (int j = 0; j < kTogether; ++j) v[j] = frag(o[j][0], o[j][1], o[j][2], o[j][3]);
  }
};

template <int D>
struct ValueTile<OPQ_CACHE_OPQ4, D> {
  static constexpr int kWords = D / 128;  // codes of dim/16 dimensions (D = 64: half a word)
  static constexpr int kTogether = 8;
  Words<kWords> raw[8];
  uint32_t sign[8];
  __device__ __forceinline__ void load(int i, const char* row, const char* signs, int c) {
    raw[i] = load_words<kWords>(row + 4 * kWords * c);
    if (kWords == 1) sign[i] = reinterpret_cast<const uint8_t*>(signs)[c];
    else sign[i] = reinterpret_cast<const uint16_t*>(signs)[c];
  }
  __device__ __forceinline__ void tiles(int t, const RowLut& lut, bf16x8_t (&v)[kTogether]) const {
    uint32_t o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      decode_word_split(raw[i].w[t], (sign[i] >> (8 * t)) & 0xFFu, lut, o[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = o[i][j];
      turn_pairs(p, v[2 * j], v[2 * j + 1]);
    }
  }
};

template <>
struct ValueTile<OPQ_CACHE_OPQ4, 64> {
  static constexpr int kTogether = 4;
  uint32_t raw[8];   // four codes
  uint32_t sign[8];  // four signs
  int shift;
  __device__ __forceinline__ void load(int i, const char* row, const char* signs, int c) {
    raw[i] = reinterpret_cast<const uint16_t*>(row)[c];
    sign[i] = reinterpret_cast<const uint8_t*>(signs)[c >> 1];
    shift = 4 * (c & 1);
  }
  __device__ __forceinline__ void tiles(int, const RowLut& lut, bf16x8_t (&v)[kTogether]) const {
    uint32_t o[4][4];  // of keys 2 i and 2 i + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t s0 = (sign[2 * i] >> shift) & 15u, s1 = (sign[2 * i + 1] >> shift) & 15u;
      decode_word_split(raw[2 * i] | (raw[2 * i + 1] << 16), s0 | (s1 << 4), lut, o[i]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t p[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[2 * i] = o[i][j];
        p[2 * i + 1] = o[i][2 + j];
      }
      turn_pairs(p, v[2 * j], v[2 * j + 1]);
    }
  }
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// Tokens of sequence b before its drafted ones, its drafted ones that count, and
// the end of the keys that rows up to `last` of a kv head can see.
struct Extent {
  int64_t len, count, end;
};
__device__ __forceinline__ Extent extent(const AttentionArgs& a, int b, int last_row) {
  Extent e;
  e.len = clamp64(a.lens[b], 0, a.capacity);
  e.count = a.counts ? clamp64(a.counts[b], 0, a.draft) : a.draft;
  e.end = e.len + e.count;
  if (!a.mask) {  // a chain: nothing past the last row's own token
    const int64_t seen = e.len + last_row / a.share + 1;
    e.end = seen < e.end ? seen : e.end;
  }
  e.end = e.end < a.capacity ? e.end : a.capacity;
  return e;
}

// ------------------------------------------------------------------ the kernel

template <int FMT, int D, int NT>
__global__ __launch_bounds__(kThreads) void attend(AttentionArgs a) {
  constexpr int kSteps = D / 32;  // product steps of a score
  constexpr int kTiles = D / 16;  // result tiles, and dimensions of a value lane
  constexpr int kRow = kRowBytes<FMT, D>;
  typedef ValueTile<FMT, D> V;

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave, c = lane & 15, g = lane >> 4;

  // Workgroups that read the same keys for different query rows sit on one XCD
  // (blockIdx % 8), next to each other, and share its L2.
  int unit, rg;
  if (a.groups == 1) {
    unit = (int)blockIdx.x;
    rg = 0;
  } else {
    const int xcd = (int)blockIdx.x & 7, j = (int)blockIdx.x >> 3;
    rg = j % a.groups;
    unit = (j / a.groups) * 8 + xcd;
    if (unit >= a.batch * a.kv_heads * a.splits) return;
  }
  const int split = unit % a.splits, bh = unit / a.splits;
  const int kvh = bh % a.kv_heads, b = bh / a.kv_heads;

  const int r0 = rg * NT * 16;
  const int r_last = (r0 + NT * 16 < a.rows ? r0 + NT * 16 : a.rows) - 1;
  const Extent ex = extent(a, b, r_last);
  const int64_t k0 = (int64_t)split * a.chunk;
  if (split > 0 && k0 >= ex.end) return;
  // the last piece takes what a sequence has past max_len
  const int64_t k1 = split + 1 < a.splits && k0 + a.chunk < ex.end ? k0 + a.chunk : ex.end;
  const bool direct = a.splits == 1 || ex.end <= a.chunk;  // sees all of its rows' keys

  RowLut lut;
  if (FMT == OPQ_CACHE_OPQ4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { lut.lo[i] = a.lp.lo[i]; lut.hi[i] = a.lp.hi[i]; }
  }

  // Q, the B operand: row c of each tile
  bf16x8_t q[NT][kSteps];
  int token[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + 16 * n + c, t = r / a.share;
    token[n] = t;
    const uint16_t* p = a.q + (int64_t)b * a.q_batch + (int64_t)t * a.q_token +
                        (int64_t)(kvh * a.share + (r - t * a.share)) * a.q_head;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (r < a.rows) w = *reinterpret_cast<const u32x4_t*>(p + KeyTile<FMT, D>::dim_at(s, g));
      q[n][s] = __builtin_bit_cast(bf16x8_t, w);
    }
  }

  floatx4_t o[NT][kTiles];
  float m[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = kLowest;
    l[n] = 0.0f;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[n][j] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int32_t* table = a.page_table + (int64_t)b * a.max_pages;
  const int64_t page_mask = ((int64_t)1 << a.page_shift) - 1;

  for (int64_t kk = k0 + wave * kStep; kk < k1; kk += kRound) {
    // the two 16-key tiles, each inside one page; a tile past the end is read
    // from the last tile instead, rows past it from the last row
    KeyTile<FMT, D> kt[2];
    V vt;
    floatx4_t ks[2], vs[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int64_t base = kk + 16 * u;
      const int64_t last_tile = (k1 - 1) & ~(int64_t)15;
      base = base < last_tile ? base : last_tile;
      const int left = (int)(k1 - 1 - base < 15 ? k1 - 1 - base : 15);  // last row that counts
      uint32_t page = (uint32_t)table[base >> a.page_shift];
      const bool lost = page >= a.pages;
      page = lost ? 0u : page;
      const int64_t row0 = ((((int64_t)page * a.kv_heads + kvh) << a.page_shift) + (base & page_mask));
      const int kc = c < left ? c : left;
      kt[u].load(a.k + (row0 + kc) * kRow,
                 reinterpret_cast<const char*>(a.k_sign) + (row0 + kc) * (D / 8), g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int vc = 4 * g + i < left ? 4 * g + i : left;
        vt.load(4 * u + i, a.v + (row0 + vc) * kRow,
                reinterpret_cast<const char*>(a.v_sign) + (row0 + vc) * (D / 8), c);
      }
      ks[u] = *reinterpret_cast<const floatx4_t*>(a.k_scale + row0 + 4 * g);
      vs[u] = *reinterpret_cast<const floatx4_t*>(a.v_scale + row0 + 4 * g);
      const float sc = lost ? __builtin_nanf("") : a.scale_log2;
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[u][i] *= sc;
    }

    floatx4_t st[2][NT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) st[u][n] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const bf16x8_t k = kt[u].at(s, lut);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          st[u][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[n][s], st[u][n], 0, 0, 0);
      }
    }

    // Masks touch only the steps that reach past the cached tokens: bit 4 u + i
    // of `hidden` is the lane's key i of tile u.
    const bool masked = kk + kStep > (ex.len < k1 ? ex.len : k1);
    uint32_t hidden[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) hidden[n] = 0u;
    if (masked) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool counts = token[n] < ex.count;
        const uint32_t* row =
            a.mask ? a.mask + (int64_t)b * a.mask_batch + (int64_t)token[n] * a.mask_words : nullptr;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t key = kk + 16 * (i >> 2) + 4 * g + (i & 3), j = key - ex.len;
          bool seen = key < k1 && counts;
          if (seen && j >= 0) seen = row ? (row[j >> 5] >> (j & 31)) & 1u : j <= token[n];
          hidden[n] |= seen ? 0u : 1u << i;
        }
        // opaque: eight bits in a register, not eight lane masks in scalar ones
        asm volatile("" : "+v"(hidden[n]));
      }
    }

    bf16x8_t p[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float s[8], top = kLowest;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = st[i >> 2][n][i & 3] * ks[i >> 2][i & 3];
      if (masked) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = (hidden[n] >> i) & 1u ? -__builtin_inff() : s[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, s[i]);
      if (__builtin_amdgcn_ballot_w64(top > m[n] + kSlack)) {
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float raised = fmaxf(m[n], top), f = __builtin_amdgcn_exp2f(m[n] - raised);
        m[n] = raised;
        l[n] *= f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][i] *= f;
      }
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = __builtin_amdgcn_exp2f(s[i] - m[n]);
        l[n] += e;
        w[i] = e * vs[i >> 2][i & 3];
      }
      if (masked) {  // a hidden token's scale may be NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (hidden[n] >> i) & 1u ? 0.0f : w[i];
      }
      p[n] = frag(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]),
                  pack_bf16(w[6], w[7]));
    }

#pragma unroll
    for (int t = 0; t < kTiles / V::kTogether; ++t) {
      bf16x8_t v[V::kTogether];
      vt.tiles(t, lut, v);
#pragma unroll
      for (int j = 0; j < V::kTogether; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          o[n][t * V::kTogether + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              v[j], p[n], o[n][t * V::kTogether + j], 0, 0, 0);
    }
  }

  // Join the four waves: the rows' common maximum, then one tile of rows (in two
  // parts for wide heads) at a time through LDS.  A lane holds dimensions
  // kTiles (4 g + i) + j of row c; part p has those with i / kSpan = p.
  constexpr int kParts = D > 128 ? 2 : 1, kSpan = 4 / kParts;
  constexpr int kCols = D / kParts, kOwn = kCols / 16;
  __shared__ float m_all[kWaves][NT * 16], l_all[kWaves][NT * 16];
  __shared__ float o_all[kWaves][16][kCols + 4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += __shfl_xor(l[n], 16, kWave);
    l[n] += __shfl_xor(l[n], 32, kWave);
    if (g == 0) {
      m_all[wave][16 * n + c] = m[n];
      l_all[wave][16 * n + c] = l[n];
    }
  }
  __syncthreads();
  // this thread's row of a tile and its first column of a part
  const int rr = threadIdx.x >> 4, col = (threadIdx.x & 15) * kOwn;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float top = m_all[0][16 * n + c], mt = m_all[0][16 * n + rr], lt = 0.0f;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      top = fmaxf(top, m_all[w][16 * n + c]);
      mt = fmaxf(mt, m_all[w][16 * n + rr]);
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      lt += l_all[w][16 * n + rr] * __builtin_amdgcn_exp2f(m_all[w][16 * n + rr] - mt);
    const float f = __builtin_amdgcn_exp2f(m[n] - top);
    const int r = r0 + 16 * n + rr, t = r / a.share, h = kvh * a.share + (r - t * a.share);
    const bool none = lt == 0.0f || t >= ex.count;
    const float inv = none ? 0.0f : 1.0f / lt;
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      if (n + part > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < kSpan; ++i)
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
          o_all[wave][c][kTiles * (kSpan * g + i) + j] = o[n][j][kSpan * part + i] * f;
      __syncthreads();
      if (r >= a.rows) continue;
      float v[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        v[j] = o_all[0][rr][col + j];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v[j] += o_all[w][rr][col + j];
      }
      const int dim = kParts == 1 ? col : col / (kSpan * kTiles) * (4 * kTiles) +
                                              part * (kSpan * kTiles) + col % (kSpan * kTiles);
      if (direct) {
        const int64_t at = ((int64_t)b * a.draft + t) * a.heads + h;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.out + at * D + dim);
#pragma unroll
        for (int j = 0; j < kOwn / 2; ++j)
          out[j] = none ? 0u : pack_bf16(v[2 * j] * inv, v[2 * j + 1] * inv);
        if (a.lse && col == 0 && part == 0)
          a.lse[at] = none ? -__builtin_inff() : (mt + log2f(lt)) * 0.69314718055994531f;
      } else {
        const int64_t at = (((int64_t)split * a.batch + b) * a.kv_heads + kvh) * a.rows + r;
        float* po = a.part_o + at * D + dim;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) po[j] = v[j];
        if (col == 0 && part == 0) {
          a.part_ml[2 * at] = mt;
          a.part_ml[2 * at + 1] = lt;
        }
      }
    }
  }
}

// Join the pieces of the keys: one wave per row.  Lane i first weighs piece i, then
// each lane sums dim/64 dimensions over the pieces in order.
template <int D>
__global__ __launch_bounds__(kThreads) void join_pieces(AttentionArgs a, int group_rows) {
  constexpr int kPer = D / kWave;
  const int lane = threadIdx.x % kWave;
  const int64_t row = (int64_t)blockIdx.x * kWaves + threadIdx.x / kWave;
  const int64_t all = (int64_t)a.batch * a.kv_heads * a.rows;
  if (row >= all) return;
  const int r = (int)(row % a.rows);
  const int64_t bh = row / a.rows;
  const int kvh = (int)(bh % a.kv_heads), b = (int)(bh / a.kv_heads);
  int r_last = (r / group_rows + 1) * group_rows;
  r_last = (r_last < a.rows ? r_last : a.rows) - 1;
  const Extent ex = extent(a, b, r_last);
  if (ex.end <= a.chunk) return;  // one workgroup saw all of it and wrote the result
  const int64_t needed = (ex.end + a.chunk - 1) / a.chunk;
  const int pieces = needed < a.splits ? (int)needed : a.splits;
  const int t = r / a.share, h = kvh * a.share + (r - t * a.share);
  float m = kLowest, l = 0.0f;
  if (lane < pieces) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (lane * all + row));
    m = ml.x;
    l = ml.y;
  }
  const float top = wave_max(m);
  const float w = __builtin_amdgcn_exp2f(m - top);
  l *= w;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) l += __shfl_xor(l, off, kWave);
  float v[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) v[j] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const float wi = readlane_f(w, i);
    const float* p = a.part_o + (i * all + row) * D + lane * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] += p[j] * wi;
  }
  const bool none = l == 0.0f || t >= ex.count;
  const float inv = none ? 0.0f : 1.0f / l;
  const int64_t at = ((int64_t)b * a.draft + t) * a.heads + h;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    a.out[at * D + lane * kPer + j] =
        none ? (uint16_t)0 : __builtin_bit_cast(uint16_t, (__bf16)(v[j] * inv));
  if (a.lse && lane == 0)
    a.lse[at] = none ? -__builtin_inff() : (top + log2f(l)) * 0.69314718055994531f;
}

template <int FMT, int D, int NT>
hipError_t go(const AttentionArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.batch * a.kv_heads * a.splits;
  const int64_t blocks = a.groups == 1 ? units : (units + 7) / 8 * 8 * a.groups;
  hipLaunchKernelGGL((attend<FMT, D, NT>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
  hipLaunchKernelGGL((join_pieces<D>), dim3((unsigned)((rows + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, stream, a, NT * 16);
  return hipGetLastError();
}

template <int FMT>
hipError_t go_format(const AttentionArgs& a, int dim, int tiles, hipStream_t stream) {
  if (dim == 64) {
    if (tiles == 1) return go<FMT, 64, 1>(a, stream);
    if (tiles == 2) return go<FMT, 64, 2>(a, stream);
    return go<FMT, 64, 4>(a, stream);
  }
  if (dim == 128) {
    if (tiles == 1) return go<FMT, 128, 1>(a, stream);
    if (tiles == 2) return go<FMT, 128, 2>(a, stream);
    return go<FMT, 128, 4>(a, stream);
  }
  if (tiles == 1) return go<FMT, 256, 1>(a, stream);
  return go<FMT, 256, 2>(a, stream);
}

}  // namespace

AttentionPlan attention_plan(int64_t batch, int64_t draft, int64_t heads, int64_t kv_heads,
                             int64_t dim, int64_t max_len) {
  AttentionPlan p;
  const int64_t rows = draft * (heads / kv_heads);
  const int most = dim == 256 ? 2 : 4;
  p.tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : most;
  p.groups = (int)((rows + 16 * p.tiles - 1) / (16 * p.tiles));
  // Two workgroups for each of the 256 CUs, and at least one round of keys each.
  const int64_t units = batch * kv_heads * p.groups, keys = max_len + draft;
  int64_t splits = (512 + units - 1) / units;
  const int64_t rounds = (keys + kRound - 1) / kRound;
  splits = splits < rounds ? splits : rounds;
  splits = splits < 64 ? splits : 64;
  splits = splits < 1 ? 1 : splits;
  p.chunk = ((keys + splits - 1) / splits + kRound - 1) / kRound * kRound;
  if (p.chunk < kRound) p.chunk = kRound;
  p.splits = (int)((keys + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  p.workspace = 0;
  if (p.splits > 1)
    p.workspace = ((size_t)p.splits * (size_t)(batch * kv_heads * rows) * (size_t)(dim + 2) * 4u + 255u) &
                  ~(size_t)255u;
  return p;
}

hipError_t launch_attention(const AttentionArgs& a, int format, int dim, int tiles,
                            hipStream_t stream) {
  if (format == OPQ_CACHE_BF16) return go_format<OPQ_CACHE_BF16>(a, dim, tiles, stream);
  if (format == OPQ_CACHE_FP8) return go_format<OPQ_CACHE_FP8>(a, dim, tiles, stream);
  return go_format<OPQ_CACHE_OPQ4>(a, dim, tiles, stream);
}

}  // namespace opq
