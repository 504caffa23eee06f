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
// (1 or 2 tiles of 16 in a workgroup); the four waves of a workgroup take every
// fourth 32 keys and join at its end; long sequences are split over workgroups
// and joined by a second kernel.
//
// Bounds.  Few rows: memory, at the rate of a large copy.  32 sequences of up to
// 8191 tokens, 32 query and 8 kv heads of 128, fp8: 61 us, 4.7 TB/s; 2 of 200000
// tokens, 64 query heads, opq4: 116 us (108 at best), 4.6 TB/s.  Many rows: the instructions and
// waits of a step, as every 32 rows walk over the keys again from the L2 (81 % hits).
// Trees of 48 tokens on 8 sequences of up to 6001 tokens, bf16: 88 us, 12 % of the
// matrix cores' and 29 % of the VALU's time; 3 of up to 4093 tokens, 16 heads of 256,
// 21 tokens each, fp8: 22 us.  One sequence of 1000 tokens: 6.5 us, and 3.3 for the join.
// A prompt of 8192 tokens, 32 query and 8 kv heads of 128, bf16: 1330 us, 413 TFLOP/s.
//
// Measured and not taken: waves that share decoded keys in LDS and split the rows
// (4 or 8 waves, 91 to 146 us where this takes 70 to 98); four tiles of rows to a
// workgroup, one workgroup a CU (the trees above: 91 us, and 94 for 67 from an fp8
// cache); the product with the values after the next step's scores, so that values have
// longer to arrive (trees 92 us, the batch above 71 for 65: registers for it cost waves).
#include "attention_internal.hpp"
#include "decode.hpp"

namespace opq {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kStep = 32;             // keys a wave takes at a time
constexpr int kRound = kWaves * kStep;  // keys a workgroup takes at a time
constexpr float kLowest = -3.0e38f;     // running maximum of a row that saw nothing
// The running maximum is kept this much (in powers of two) above the largest score seen
// when it was last raised, and raised again only when a score exceeds it: no weight
// exceeds 1, float32 sums and bfloat16 weights hold weights of 2^-8 as well as of 1,
// and most steps skip the rescaling.
constexpr float kSlack = 8.0f;
// Up to this magnitude of the running maximum a score's rounding (half an ulp, 4) stays
// below kSlack, and the unrounded product may stand in the exponent.
constexpr float kFine = 0x1p26f;

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

// OPQ codes are looked up two at a time: entry (two sign bits, code byte) of a table
// in LDS is the pair as bfloat16, so eight codes take four reads and twelve
// VALU instructions (the permutes of decode.hpp take 34, which bounded this
// kernel).  4 KB.
// The entries of one sign pair are kSignStride apart, not 256: magnitudes crowd
// around a few codes, and without the shift their banks coincide for all four
// sign pairs (9.2 cycles a read measured, 6.3 with it).
constexpr int kSignStride = 276, kPairs = 4 * kSignStride;
typedef const uint32_t* PairTable;

__device__ __forceinline__ void build_pairs(const LevelPlanes& lp, uint32_t* pairs) {
  RowLut t;
#pragma unroll
  for (int i = 0; i < 4; ++i) { t.lo[i] = lp.lo[i]; t.hi[i] = lp.hi[i]; }
  if (threadIdx.x >= 256) return;  // a code byte a thread
#pragma unroll
  for (uint32_t sign = 0; sign < 4; ++sign) {
    uint32_t o[4];
    decode_word_split(threadIdx.x, sign, t, o);
    pairs[sign * kSignStride + threadIdx.x] = o[0];
  }
}
// Pairs 0..3 of word w with the signs in bits 0..7 of sb.
__device__ __forceinline__ void decode_pairs(uint32_t w, uint32_t sb, PairTable t, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = t[((w >> (8 * i)) & 0xFFu) + __umul24((sb >> (2 * i)) & 3u, kSignStride)];
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
  __device__ __forceinline__ void load(const char* rows, const char*, uint32_t r, int g) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const Words<4> t = load_words<4>(rows + (r * 2 * D + 64 * s + 16 * g));
#pragma unroll
      for (int i = 0; i < 4; ++i) raw.w[4 * s + i] = t.w[i];
    }
  }
  __device__ __forceinline__ bf16x8_t at(int s, PairTable) const {
    return frag(raw.w[4 * s], raw.w[4 * s + 1], raw.w[4 * s + 2], raw.w[4 * s + 3]);
  }
};

template <int D>
struct KeyTile<OPQ_CACHE_FP8, D> {
  Words<D / 16> raw;
  __device__ static int dim_at(int s, int g) { return 64 * (s >> 1) + 16 * g + 8 * (s & 1); }
  __device__ __forceinline__ void load(const char* rows, const char*, uint32_t r, int g) {
#pragma unroll
    for (int s = 0; s < D / 64; ++s) {
      const Words<4> t = load_words<4>(rows + (r * D + 64 * s + 16 * g));
#pragma unroll
      for (int i = 0; i < 4; ++i) raw.w[4 * s + i] = t.w[i];
    }
  }
  __device__ __forceinline__ bf16x8_t at(int s, PairTable) const {
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
  __device__ __forceinline__ void load(const char* rows, const char* signs, uint32_t r, int g) {
    raw = load_words<kSteps>(rows + (r * (D / 2) + 4 * kSteps * g));
    const char* p = signs + (r * (D / 8) + kSteps * g);
    if (kSteps == 2) sign = *reinterpret_cast<const uint16_t*>(p);
    else if (kSteps == 4) sign = *reinterpret_cast<const uint32_t*>(p);
    else sign = *reinterpret_cast<const uint64_t*>(p);
  }
  __device__ __forceinline__ bf16x8_t at(int s, PairTable lut) const {
    uint32_t o[4];
    decode_pairs(raw.w[s], (uint32_t)(sign >> (8 * s)), lut, o);
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
  __device__ __forceinline__ void load(int i, const char* rows, const char*, uint32_t r, int c) {
    raw[i] = load_words<kWords>(rows + (r * 2 * D + 4 * kWords * c));
  }
  __device__ __forceinline__ void tiles(int t, PairTable, bf16x8_t (&v)[kTogether]) const {
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
  __device__ __forceinline__ void load(int i, const char* rows, const char*, uint32_t r, int c) {
    raw[i] = load_words<kWords>(rows + (r * D + 4 * kWords * c));
  }
  __device__ __forceinline__ void tiles(int t, PairTable, bf16x8_t (&v)[kTogether]) const {
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
  __device__ __forceinline__ void load(int i, const char* rows, const char* signs, uint32_t r, int c) {
    raw[i] = load_words<kWords>(rows + (r * (D / 2) + 4 * kWords * c));
    const char* p = signs + (r * (D / 8) + kWords * c);
    if (kWords == 1) sign[i] = *reinterpret_cast<const uint8_t*>(p);
    else sign[i] = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void tiles(int t, PairTable lut, bf16x8_t (&v)[kTogether]) const {
    uint32_t o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      decode_pairs(raw[i].w[t], sign[i] >> (8 * t), lut, o[i]);
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
  __device__ __forceinline__ void load(int i, const char* rows, const char* signs, uint32_t r, int c) {
    raw[i] = *reinterpret_cast<const uint16_t*>(rows + (r * 32 + 2 * c));
    sign[i] = *reinterpret_cast<const uint8_t*>(signs + (r * 8 + (c >> 1)));
    shift = 4 * (c & 1);
  }
  __device__ __forceinline__ void tiles(int, PairTable lut, bf16x8_t (&v)[kTogether]) const {
    uint32_t o[4][4];  // of keys 2 i and 2 i + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t s0 = (sign[2 * i] >> shift) & 15u, s1 = (sign[2 * i + 1] >> shift) & 15u;
      decode_pairs(raw[2 * i] | (raw[2 * i + 1] << 16), s0 | (s1 << 4), lut, o[i]);
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

// Which piece of which sequence's keys, for which group of query rows, a workgroup has.
struct Task {
  int split, b, kvh, rg;
};
__device__ __forceinline__ bool task_of(const AttentionArgs& a, Task& t) {
  // Workgroups that read the same keys for different query rows sit on one XCD
  // (blockIdx % 8), next to each other, and share its L2.
  int unit;
  if (a.groups == 1) {
    unit = (int)blockIdx.x;
    t.rg = 0;
  } else {
    const int xcd = (int)blockIdx.x & 7, j = (int)blockIdx.x >> 3;
    t.rg = j % a.groups;
    unit = (j / a.groups) * 8 + xcd;
    if (unit >= a.batch * a.kv_heads * a.splits) return false;
  }
  // Pieces of one sequence are far apart: the ones that a short sequence does not
  // have would otherwise be every blockIdx of some XCDs, which then stand idle
  // (32 sequences of half the longest length: 83 against 58 us).
  const int pairs = a.batch * a.kv_heads, bh = unit % pairs;
  t.split = unit / pairs;
  t.b = bh / a.kv_heads;
  t.kvh = bh - t.b * a.kv_heads;
  return true;
}

// A wave's walk over the keys k0 .. k1 of one sequence and kv head, 32 at a time.
template <int FMT, int D>
struct Walk {
  static constexpr int kRow = kRowBytes<FMT, D>;
  // Rows past the last one that counts may hold NaN codes, which no weight of 0
  // takes away; OPQ codes have none.
  static constexpr bool kClamp = FMT != OPQ_CACHE_OPQ4;
  struct Place {
    int64_t row;  // first row of a 16-key tile
    int left;     // last row of the tile that counts
    bool lost;    // the page id names no page
  };
  const AttentionArgs& a;
  const int32_t* table;
  int64_t k1, last_tile, held;
  uint32_t ids;  // lane i: id of page `held + i`
  int kvh, lane, c, g;
  KeyTile<FMT, D> kt[2];
  ValueTile<FMT, D> vt;
  floatx4_t ks[2], vs[2];
  Place at[2];

  __device__ __forceinline__ Walk(const AttentionArgs& args, const Task& t, int64_t k0, int64_t end,
                                  int lane_)
      : a(args), table(args.page_table + (int64_t)t.b * args.max_pages), k1(end),
        last_tile((end - 1) & ~(int64_t)15), held(k0 >> args.page_shift), ids(0u), kvh(t.kvh),
        lane(lane_), c(lane_ & 15), g(lane_ >> 4) {}

  __device__ __forceinline__ void hold(int64_t first) {
    held = first;
    const int64_t p = first + lane;
    if (p < a.max_pages) ids = (uint32_t)table[p];
    // waited for here (vmcnt(0)), where it happens once in many steps: left to its
    // use, every step would wait for all of its requests in flight
    __builtin_amdgcn_s_waitcnt(0x0F70);
  }
  // Finds the two 16-key tiles at `key`, each inside one page.  A tile past the end
  // is read from the last tile instead, and rows past it from the last row.
  __device__ __forceinline__ void find(int64_t key) {
    const int64_t page_mask = ((int64_t)1 << a.page_shift) - 1;
    if (((key + 16 < last_tile ? key + 16 : last_tile) >> a.page_shift) - held >= kWave)
      hold((key < last_tile ? key : last_tile) >> a.page_shift);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t base = key + 16 * u < last_tile ? key + 16 * u : last_tile;
      const int64_t index = (base >> a.page_shift) - held;
      const uint32_t id = (uint32_t)__builtin_amdgcn_readlane((int)ids, (int)index);
      at[u].lost = id >= a.pages;
      at[u].row = (((int64_t)(at[u].lost ? 0u : id) * a.kv_heads + kvh) << a.page_shift) +
                  (base & page_mask);
      at[u].left = (int)(k1 - 1 - base < 15 ? k1 - 1 - base : 15);
    }
  }
  __device__ __forceinline__ static uint32_t row_of(int r, int left) {
    return (uint32_t)(!kClamp || r < left ? r : left);
  }
  __device__ __forceinline__ void load_keys() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kt[u].load(a.k + at[u].row * kRow,
                 reinterpret_cast<const char*>(a.k_sign) + at[u].row * (D / 8),
                 row_of(c, at[u].left), g);
      ks[u] = *reinterpret_cast<const floatx4_t*>(a.k_scale + at[u].row + 4 * g);
    }
  }
  __device__ __forceinline__ void load_values() {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // unclamped rows differ by a constant from the lane's first
        const int64_t first = at[u].row + (kClamp ? 0 : i);
        vt.load(4 * u + i, a.v + first * kRow,
                reinterpret_cast<const char*>(a.v_sign) + first * (D / 8),
                kClamp ? row_of(4 * g + i, at[u].left) : 4u * g, c);
      }
      vs[u] = *reinterpret_cast<const floatx4_t*>(a.v_scale + at[u].row + 4 * g);
    }
  }
  // the loaded keys' scales, times scale log2(e); NaN for a page that is none
  __device__ __forceinline__ floatx4_t key_scale(int u) const {
    const float sc = at[u].lost ? __builtin_nanf("") : a.scale_log2;
    floatx4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ks[u][i] * sc;
    return r;
  }
};

// Which of a lane's eight keys (bit 4 u + i: key kk + 16 u + 4 g + i) its query
// row, of drafted token `token`, does not see.
__device__ __forceinline__ uint32_t hidden_keys(const AttentionArgs& a, const Extent& ex, int b,
                                                int token, int64_t kk, int64_t k1, int g) {
  const bool counts = token < ex.count;
  uint32_t seen = 0u;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    // drafted index of the lane's first key of the tile, and how many of its four
    // keys there are
    const int64_t key = kk + 16 * u + 4 * g;
    const int j0 = (int)(key - ex.len < -kStep ? -kStep : key - ex.len);
    const int there = (int)clamp64(k1 - key, 0, 4);
    uint32_t four;
    if (a.mask) {
      // the row's bits j0 .. j0 + 3, those before the draft set
      const uint32_t* row = a.mask + (int64_t)b * a.mask_batch +
                            (int64_t)(counts ? token : 0) * a.mask_words;
      const int last = (int)a.mask_words - 1, j = j0 < 0 ? 0 : j0;
      const int w0 = j >> 5 < last ? j >> 5 : last, w1 = w0 < last ? w0 + 1 : last;
      const uint64_t bits = ((uint64_t)row[w1] << 32 | row[w0]) >> (j & 31);
      const int before = j - j0 < 4 ? j - j0 : 4;
      four = ((uint32_t)bits << before | ((1u << before) - 1u)) & 15u;
    } else {
      const int upto = token + 1 - j0;  // a chain: j <= token
      four = (1u << (upto < 0 ? 0 : upto > 4 ? 4 : upto)) - 1u;
    }
    four &= (1u << there) - 1u;
    seen |= four << (4 * u);
  }
  uint32_t hidden = counts ? ~seen : 255u;
  // opaque: eight bits in a register, not eight lane masks in scalar ones
  asm volatile("" : "+v"(hidden));
  return hidden;
}

// A score as float32 holds it (not fused into what uses it).
__device__ __forceinline__ float score(float acc, float kscale) {
#pragma clang fp contract(off)
  return acc * kscale;
}

// A 16-row tile of queries: lane 16 g + c has the running maximum of row c, its own
// keys' part of the sum, and dimensions kTiles (4 g + i) + j in o[j][i].
template <int kTiles>
struct Rows {
  floatx4_t o[kTiles];
  float m, l;
  bool coarse;  // of the wave: some row's m is larger than kFine
  __device__ __forceinline__ void clear() {
    m = kLowest;
    l = 0.0f;
    coarse = false;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) o[j] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // Takes the products of 32 keys in and gives their weights, times the values'
  // scales, as the B operand of the second product.  No score of the lane's keys
  // exceeds max(acc, 0) * scale_top (the largest of kscale): while that stays below
  // the running maximum (tested exactly, by the sign of a fused multiply-add), the
  // scores themselves are formed only inside the exponent, one fused multiply-add each.
  // Past kFine such a product would keep what the score's rounding took off the maximum,
  // whole powers of two either way (2^9 of them at 2^33): there scores are rounded first,
  // as the maximum was.  Rounding all of them measures 101 us for 92 on the trees above.
  // `rest`, where it is asked for (kTwo), is what their rounding to bfloat16 left.
  template <bool kTwo>
  __device__ __forceinline__ bf16x8_t weigh(const floatx4_t& s0, const floatx4_t& s1,
                                            const floatx4_t (&kscale)[2], float scale_top,
                                            const floatx4_t (&vs)[2], bool masked,
                                            uint32_t hidden, bf16x8_t& rest) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i] = s0[i];
      acc[4 + i] = s1[i];
    }
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, acc[i]);
    if (__builtin_amdgcn_ballot_w64(__builtin_fmaf(most, scale_top, -m) > 0.0f)) {
      float top = kLowest;
      // an opaque copy, here and below: the tests of its bits stay on these rare ways
      uint32_t h = hidden;
      asm volatile("" : "+v"(h));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = score(acc[i], kscale[i >> 2][i & 3]);
        top = fmaxf(top, (h >> i) & 1u ? kLowest : s);
      }
      if (__builtin_amdgcn_ballot_w64(top >= m && top > kLowest)) {
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float raised = fmaxf(m, top + kSlack), f = __builtin_amdgcn_exp2f(m - raised);
        m = raised;
        coarse = __builtin_amdgcn_ballot_w64(fabsf(m) > kFine && m > kLowest) != 0;
        l *= f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] *= f;
      }
    }
    float x[8], e[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __builtin_fmaf(acc[i], kscale[i >> 2][i & 3], -m);
    if (__builtin_expect(coarse, 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        asm volatile("" : "+v"(acc[i]));  // stays a branch: both ways at once cost 24 registers
        x[i] = score(acc[i], kscale[i >> 2][i & 3]) - m;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = __builtin_amdgcn_exp2f(x[i]);
      w[i] = e[i] * vs[i >> 2][i & 3];
    }
    if (masked) {  // a hidden token may hold anything
      uint32_t h = hidden;
      asm volatile("" : "+v"(h));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool hide = (h >> i) & 1u;
        e[i] = hide ? 0.0f : e[i];
        w[i] = hide ? 0.0f : w[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) l += e[i];
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack_bf16(w[2 * i], w[2 * i + 1]);
    if (kTwo) {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = pack_bf16(w[2 * i] - __uint_as_float(p[i] << 16),
                         w[2 * i + 1] - __uint_as_float(p[i] & 0xFFFF0000u));
      rest = frag(r[0], r[1], r[2], r[3]);
    }
    return frag(p[0], p[1], p[2], p[3]);
  }
};
__device__ __forceinline__ float top_of(const floatx4_t (&k)[2]) {
  float t = fmaxf(k[0][0], k[1][0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) t = fmaxf(t, fmaxf(k[0][i], k[1][i]));
  return t;
}

// Row r of a kv head's queries: 16 bytes at dimension d, or zeros past the last row.
__device__ __forceinline__ bf16x8_t query_at(const AttentionArgs& a, const Task& k, int r, int d) {
  const int t = r / a.share;
  const uint16_t* p = a.q + (int64_t)k.b * a.q_batch + (int64_t)t * a.q_token +
                      (int64_t)(k.kvh * a.share + (r - t * a.share)) * a.q_head;
  u32x4_t w = {0u, 0u, 0u, 0u};
  if (r < a.rows) w = *reinterpret_cast<const u32x4_t*>(p + d);
  return __builtin_bit_cast(bf16x8_t, w ^ a.q_flip);
}

// ------------------------------------------------------------------ the kernel

// Workgroups a CU's registers have to hold.  Two, so that one computes while the
// other waits, is what everything but a wide bfloat16 tile fits in; one tile of narrow
// heads has registers for three (32 sequences of 8191 tokens, 8 kv heads of 64, opq4, with
// the join: 57 us, 60 with two; fp8 57 both ways; at 128 dimensions there is no difference).
template <int FMT, int D, int NT>
constexpr int kOccupancy = FMT == OPQ_CACHE_BF16 && D == 256 ? 1 : NT * D == 64 ? 3 : 2;

template <int FMT, int D, int NT>
__global__ __launch_bounds__(kThreads, (kOccupancy<FMT, D, NT>)) void attend(AttentionArgs a) {
  constexpr int kSteps = D / 32;  // product steps of a score
  constexpr int kTiles = D / 16;  // result tiles, and dimensions of a value lane
  typedef ValueTile<FMT, D> V;
  // One tile of rows leaves the matrix cores idle: the weights then go in twice, as
  // their bfloat16 and what that left out, so that only the result is rounded (free
  // on fp8 and bfloat16 caches; 5 % on OPQ ones, whose 4-bit codes are far coarser).
  constexpr bool kTwo = NT == 1 && FMT != OPQ_CACHE_OPQ4;

  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave, c = lane & 15, g = lane >> 4;

  Task k;
  if (!task_of(a, k)) return;
  const int r0 = k.rg * NT * 16;
  const int r_last = (r0 + NT * 16 < a.rows ? r0 + NT * 16 : a.rows) - 1;
  const Extent ex = extent(a, k.b, r_last);
  const int64_t k0 = (int64_t)k.split * a.chunk;
  if (k.split > 0 && k0 >= ex.end) return;
  // the last piece takes what a sequence has past max_len
  const int64_t k1 = k.split + 1 < a.splits && k0 + a.chunk < ex.end ? k0 + a.chunk : ex.end;
  const bool direct = a.splits == 1 || ex.end <= a.chunk;  // sees all of its rows' keys

  __shared__ uint32_t lut[FMT == OPQ_CACHE_OPQ4 ? kPairs : 1];
  if (FMT == OPQ_CACHE_OPQ4) {
    build_pairs(a.lp, lut);
    __syncthreads();
  }

  // Q, the B operand: row c of each tile.  Where registers are short the
  // workgroup's waves share one copy in LDS, in the order of their reads.
  constexpr bool kShareQ = FMT == OPQ_CACHE_BF16 && D == 128 && NT == 2;
  __shared__ bf16x8_t q_all[kShareQ ? NT : 1][kShareQ ? kSteps : 1][kShareQ ? kWave : 1];
  bf16x8_t q[kShareQ ? 1 : NT][kShareQ ? 1 : kSteps];
  int token[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + 16 * n + c;
    token[n] = r / a.share;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (kShareQ && s % kWaves != wave) continue;
      const bf16x8_t v = query_at(a, k, r, KeyTile<FMT, D>::dim_at(s, g));
      if constexpr (kShareQ) q_all[n][s][lane] = v;
      else q[n][s] = v;
    }
  }
  if (kShareQ) __syncthreads();
  auto q_at = [&](int n, int s) {
    if constexpr (kShareQ) return q_all[n][s][lane];
    else return q[n][s];
  };

  Rows<kTiles> rows[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) rows[n].clear();

  // Software pipeline: a step's keys are requested before the softmax of the step
  // before it, its values before its own scores.  The requests past the last step
  // repeat its rows: without a condition around them, the loop waits for nothing
  // but what it uses.
  Walk<FMT, D> w(a, k, k0, k1, lane);
  int64_t kk = k0 + wave * kStep;
  if (kk < k1) {
    w.hold(w.held);
    w.find(kk);
    w.load_keys();
  }
  for (; kk < k1; kk += kRound) {
    w.load_values();
    // 2 NT sums side by side: each product of a sum waits for the one before it
    floatx4_t st[2][NT], kscale[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n) st[u][n] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const bf16x8_t key[2] = {w.kt[0].at(s, lut), w.kt[1].at(s, lut)};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bf16x8_t query = q_at(n, s);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          st[u][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(key[u], query, st[u][n], 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kscale[u] = w.key_scale(u);
      // made here, before the next step's scales are requested: kept for later, the
      // old and the new scales would change places in registers at the loop's end,
      // which waits for the new ones
      asm volatile("" : "+v"(kscale[u]));
    }
    w.find(kk + kRound);
    w.load_keys();

    // masks touch only the steps that reach past the cached tokens
    const bool masked = kk + kStep > (ex.len < k1 ? ex.len : k1);
    const float scale_top = top_of(kscale);
    bf16x8_t p[NT], rest[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t hidden = 0u;
      if (masked) hidden = hidden_keys(a, ex, k.b, token[n], kk, k1, g);
      p[n] = rows[n].template weigh<kTwo>(st[0][n], st[1][n], kscale, scale_top, w.vs, masked, hidden,
                                          rest[n]);
    }
#pragma unroll
    for (int t = 0; t < kTiles / V::kTogether; ++t) {
      bf16x8_t v[V::kTogether];
      w.vt.tiles(t, lut, v);
#pragma unroll
      for (int j = 0; j < V::kTogether; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          floatx4_t& o = rows[n].o[t * V::kTogether + j];
          if (kTwo) o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[j], rest[n], o, 0, 0, 0);
          o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[j], p[n], o, 0, 0, 0);
        }
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
    float l = rows[n].l;
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
    if (g == 0) {
      m_all[wave][16 * n + c] = rows[n].m;
      l_all[wave][16 * n + c] = l;
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
    const float f = __builtin_amdgcn_exp2f(rows[n].m - top);
    const int r = r0 + 16 * n + rr, t = r / a.share, h = k.kvh * a.share + (r - t * a.share);
    const bool none = lt == 0.0f || t >= ex.count;
    const float inv = none ? 0.0f : 1.0f / lt;
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      if (n + part > 0) __syncthreads();
#pragma unroll
      for (int i = 0; i < kSpan; ++i)
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
          o_all[wave][c][kTiles * (kSpan * g + i) + j] = rows[n].o[j][kSpan * part + i] * f;
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
        const int64_t at = ((int64_t)k.b * a.draft + t) * a.heads + h;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.out + at * D + dim);
#pragma unroll
        for (int j = 0; j < kOwn / 2; ++j)
          out[j] = none ? 0u : pack_bf16(v[2 * j] * inv, v[2 * j + 1] * inv);
        if (a.lse && col == 0 && part == 0)
          a.lse[at] = none ? -__builtin_inff() : (mt + log2f(lt)) * 0.69314718055994531f;
      } else {
        const int64_t at = (((int64_t)k.split * a.batch + k.b) * a.kv_heads + k.kvh) * a.rows + r;
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

// ------------------------------------------------------------------ joining pieces

// Join the pieces of the keys.  A wave holds 256 / D pieces at a time, 16 bytes a
// lane, and merges them into a running result as the kernel above merges keys; a
// piece's partial result and its (m, l) are requested together, so nothing waits
// for a maximum over all pieces first.  kTeam waves share a row (4 where a row has
// many pieces) and meet in LDS.
template <int D, int kTeam>
__global__ __launch_bounds__(kThreads) void join_pieces(AttentionArgs a) {
  constexpr int kLanes = D / 4, kTogether = kWave / kLanes, kUnroll = 4;
  const int lane = threadIdx.x % kWave, sub = lane / kLanes, d = (lane % kLanes) * 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int all = a.batch * a.kv_heads * a.rows;  // at most 2^22
  const int row = (int)blockIdx.x * (kWaves / kTeam) + wave / kTeam;
  if (row >= all) return;  // all waves of a team
  const int bh = row / a.rows, r = row - bh * a.rows;
  const int b = bh / a.kv_heads, kvh = bh - b * a.kv_heads;
  int r_last = (r / a.group_rows + 1) * a.group_rows;
  r_last = (r_last < a.rows ? r_last : a.rows) - 1;
  const Extent ex = extent(a, b, r_last);
  if (ex.end <= a.chunk) return;  // one workgroup saw all of it and wrote the result
  const int64_t needed = (ex.end + a.chunk - 1) / a.chunk;
  const int pieces = needed < a.splits ? (int)needed : a.splits;

  float m = kLowest, l = 0.0f;
  floatx4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
  auto merge = [&](float mi, float li, floatx4_t vi) {
    const float top = fmaxf(m, mi);
    const float f = __builtin_amdgcn_exp2f(m - top), fi = __builtin_amdgcn_exp2f(mi - top);
    m = top;
    l = l * f + li * fi;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = v[j] * f + vi[j] * fi;
  };
  for (int i0 = wave % kTeam * kTogether; i0 < pieces; i0 += kTeam * kTogether * kUnroll) {
    float2 ml[kUnroll];
    floatx4_t po[kUnroll];
    bool there[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * kTeam * kTogether + sub;
      there[k] = i < pieces;
      const int64_t at = (int64_t)(there[k] ? i : 0) * all + row;
      ml[k] = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
      po[k] = *reinterpret_cast<const floatx4_t*>(a.part_o + at * D + d);
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (there[k]) merge(ml[k].x, ml[k].y, po[k]);
  }
#pragma unroll
  for (int off = kLanes; off < kWave; off *= 2) {
    floatx4_t vo;
#pragma unroll
    for (int j = 0; j < 4; ++j) vo[j] = __shfl_xor(v[j], off, kWave);
    merge(__shfl_xor(m, off, kWave), __shfl_xor(l, off, kWave), vo);
  }
  if (kTeam > 1) {
    __shared__ floatx4_t v_all[kTeam][kLanes];
    __shared__ float m_all[kTeam], l_all[kTeam];
    if (lane < kLanes) v_all[wave][lane] = v;
    if (lane == 0) {
      m_all[wave] = m;
      l_all[wave] = l;
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < kTeam; ++w) merge(m_all[w], l_all[w], v_all[w][lane % kLanes]);
  }
  if (sub > 0) return;
  const int t = r / a.share, h = kvh * a.share + (r - t * a.share);
  const bool none = l == 0.0f || t >= ex.count;
  const float inv = none ? 0.0f : 1.0f / l;
  const int64_t at = ((int64_t)b * a.draft + t) * a.heads + h;
  const uint2 w = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
  *reinterpret_cast<uint2*>(a.out + at * D + d) = none ? make_uint2(0u, 0u) : w;
  if (a.lse && lane == 0)
    a.lse[at] = none ? -__builtin_inff() : (m + log2f(l)) * 0.69314718055994531f;
}

template <int FMT, int D, int NT>
hipError_t go(const AttentionArgs& a, hipStream_t stream) {
  const int64_t units = (int64_t)a.batch * a.kv_heads * a.splits;
  const int64_t blocks = a.groups == 1 ? units : (units + 7) / 8 * 8 * a.groups;
  hipLaunchKernelGGL((attend<FMT, D, NT>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  // A wave merges 4 x 256 / D pieces in one trip to memory; rows with more, where
  // rows are few, get a workgroup each
  // (one sequence of 16000 tokens, 32 query heads, fp8: 12.4 us, 13.8 with a wave a
  // row; trees of 48 tokens on 8 sequences of 4000, bf16: 76 us with a wave, 87 with
  // a workgroup).
  const int64_t rows = (int64_t)a.batch * a.kv_heads * a.rows;
  if (a.splits > 4 * (256 / D) && rows <= 8192)
    hipLaunchKernelGGL((join_pieces<D, kWaves>), dim3((unsigned)rows), dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((join_pieces<D, 1>), dim3((unsigned)((rows + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <int FMT, int D>
hipError_t go_tiles(const AttentionArgs& a, int tiles, hipStream_t stream) {
  if constexpr (D < 256) {
    if (tiles == 2) return go<FMT, D, 2>(a, stream);
  }
  return go<FMT, D, 1>(a, stream);
}

template <int FMT>
hipError_t go_format(const AttentionArgs& a, int dim, int tiles, hipStream_t stream) {
  if (dim == 64) return go_tiles<FMT, 64>(a, tiles, stream);
  if (dim == 128) return go_tiles<FMT, 128>(a, tiles, stream);
  return go_tiles<FMT, 256>(a, tiles, stream);
}

}  // namespace

AttentionPlan attention_plan(int64_t batch, int64_t draft, int64_t heads, int64_t kv_heads,
                             int64_t dim, int64_t max_len) {
  AttentionPlan p;
  const int64_t rows = draft * (heads / kv_heads);
  const int64_t tiles = (rows + 15) / 16;
  p.tiles = dim == 256 || tiles == 1 ? 1 : 2;
  p.groups = (int)((tiles + p.tiles - 1) / p.tiles);
  p.group_rows = 16 * p.tiles;
  const int64_t units = batch * kv_heads * p.groups, keys = max_len + draft;
  const int64_t rounds = (keys + kRound - 1) / kRound;
  // About 1024 workgroups: four for each of the 256 CUs, so that the last ones to
  // run are a small part of the whole (32 sequences of up to 8191 tokens: 67 us, 76
  // with 512, 69 with 2048).  But a piece has to be worth its partial result: 4
  // rounds of keys where that is 16 rows (8 sequences of 2000 tokens: 13 us in 4
  // pieces, 16 to 18 in 8 or 16), 12 where a workgroup has 32 (8 sequences of 1000
  // tokens with 192 rows: 32 us in one piece, 43 in three).  Shorter ones, down to
  // two rounds, only for workgroups that would leave CUs empty (one sequence of 1000
  // tokens: 9.4 us in 4 pieces, 11.2 in one).  Joining costs more than splitting up
  // to 4 rounds saves (16 sequences of 500 tokens: 9.2 us in one, 12.8 in two).
  const int64_t worth = p.tiles == 1 ? 4 : 12, by_length = rounds / worth;
  int64_t splits = (1024 + units - 1) / units, fill = (256 + units - 1) / units;
  fill = fill < rounds / 2 ? fill : rounds / 2;
  const int64_t bound = rounds <= 4 ? 1 : by_length > fill ? by_length : fill;
  splits = splits < bound ? splits : bound;
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
