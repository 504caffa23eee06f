// A paged cache of keys and values, quantized as it is written.
//
// A row is the `dim` values of one token and kv head; it gets one float32 scale
// from its largest magnitude m:
//   bf16: code bf16(x), scale 1;
//   fp8:  s = m / 448 (the largest e4m3 value), code e4m3(x / s);
//   opq4: u = |x| / m, q = nearest(15 u^alpha), a nibble and a sign bit, as
//         opq_quantize stores a row of weights (model card "OPQ INT4 Z-Image",
//         "OPQ 原理" and "技术细节 / 存储格式"), scale m.
// A row with a NaN or an infinity gets scale NaN and codes 0.
//
// A group of dim/8 lanes holds a row, eight values a lane (16 bytes of bf16), so
// the maximum is a few lane exchanges and nothing is read twice.  With few tokens
// the launch bounds both ways (48 tokens of 8 heads of 128, fp8: 2.8 us to write, 2.5
// to read).  Reading long histories is bound by memory: 131072 tokens of 8 heads of 128
// from opq4, 133 us, 5.3 TB/s.  Writing 32768 such tokens takes 48 us for opq4 (3.7
// TB/s), bound by the VALU (a logarithm and an exponential, each four issue slots, of
// some twenty a value); fp8 and bf16 by memory: 37 and 44 us, 5.5 and 6.1 TB/s.
#include "attention_internal.hpp"
#include "decode.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;
constexpr float kSmallest = 0x1p-100f;  // rows below it are stored as zeros

typedef float floatx2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const floatx2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight raw values of a row.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  uint32_t w[4];
  // `wide`: p is a multiple of 16 bytes
  __device__ __forceinline__ void load(const uint16_t* p, bool wide) {
    if (wide) {
      const u32x4_t v = load_stream16(p);
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = low_half(w[i]);
      x[2 * i + 1] = high_half(w[i]);
    }
  }
  // bits of the largest magnitude, as binary32 (NaN above infinity above the rest)
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t = __builtin_bit_cast(uint32_t,
                             __builtin_elementwise_max(
                                 __builtin_bit_cast(u16x2_t, t),
                                 __builtin_bit_cast(u16x2_t, w[i] & 0x7FFF7FFFu)));
    return max(t << 16, t & 0xFFFF0000u);
  }
};
template <>
struct Eight<float> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p, bool wide) {
    if (wide) {
      const u32x4_t a = load_stream16(p), b = load_stream16(p + 4);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(p[i]);
    }
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, w[i] & 0x7FFFFFFFu);
    return t;
  }
};

// Largest of v over each group of kLanes (8, 16 or 32) lanes, in every lane of
// it.  Within four lanes by quad permutes; then the mirrored halves of eight and
// of sixteen lanes hold the other part's result.
template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
  if (kLanes >= 16) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));
  if (kLanes >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16, kWave));
  return v;
}

// Code of magnitude a in a row with maximum m: the number of decision points
// not above the correctly rounded quotient.
__device__ uint32_t code_exact(float a, float m, const CacheCodes& cc) {
  const float u = a / m;
  uint32_t q = 0u;
#pragma unroll
  for (int i = 0; i < 15; ++i) q += u >= cc.t[i] ? 1u : 0u;
  return q;
}

// Nibbles of eight magnitudes.  15 u^alpha comes from the hardware's log2 and exp2
// on |x| * fl(1/m): its error is far below cc.guard, so the nearest integer is the
// exact code unless a half-integer is within the guard; those few (and every row
// whose 1/m is not a normal number) are decided by code_exact.  The conversion to
// a byte rounds to nearest; codes gather in bytes, which costs an instruction a value
// less than shifting nibbles together (16384 tokens of 8 heads of 128: 27 us, 30).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float m, const CacheCodes& cc) {
  constexpr float kLog15 = 3.90689059560851853f;
  const float r = __builtin_amdgcn_rcpf(m);
  uint32_t even = 0u, odd = 0u;  // codes 0 2 4 6 and 1 3 5 7, a byte each
  float nearest = 1.0f;          // smallest distance from a half-integer
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lg = __builtin_amdgcn_logf(fabsf(x[i]) * r);
    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(cc.alpha, lg, kLog15));
    nearest = fminf(nearest, fabsf(__builtin_amdgcn_fractf(p) - 0.5f));
    uint32_t& bytes = i & 1 ? odd : even;
    bytes = __builtin_amdgcn_cvt_pk_u8_f32(p, i >> 1, bytes);
  }
  uint32_t word = even | odd << 4;
  if (!(nearest > cc.guard && r >= 0x1p-126f)) {
    word = 0u;
#pragma unroll 1
    for (int i = 7; i >= 0; --i) {
      float v = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) v = i == j ? x[j] : v;
      word = (word << 4) + code_exact(fabsf(v), m, cc);
    }
  }
  return word;
}

// x / s, correctly rounded, from ri = fl(1/s): q = fl(x ri) is within an ulp, its
// remainder x - q s is exact in a fused multiply-add, and fl(q + rem ri) is then the
// rounded quotient (Markstein's theorem; it needs s's significand not to be all
// ones, and no underflow, which only quotients far below the smallest code have).
__device__ __forceinline__ float quotient(float x, float s, float ri) {
  const float q = x * ri;
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), ri, q);
}

struct WriteArgs {
  CacheRows side[2];
  const int32_t* slots;
  uint32_t tokens;  // of this launch
  uint32_t heads;
  uint32_t slot_end;  // pages * page
  int page_shift;
  bool wide;
};

// One row: eight values a lane; `at` is its place in the cache.
template <typename T, int FMT, int D>
__device__ __forceinline__ void write_row(const Eight<T>& raw, const CacheRows& s, int64_t at,
                                          int lane, const CacheCodes& cc) {
  constexpr int kLanes = D / 8;
  float x[8];
  raw.values(x);
  if (FMT == OPQ_CACHE_BF16) {
    uint32_t w[4], top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    }
    const bool bad = group_max<kLanes>(top) >= 0x7F80u;
    const u32x4_t o = bad ? u32x4_t{0u, 0u, 0u, 0u} : u32x4_t{w[0], w[1], w[2], w[3]};
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(s.codes) + at * D + lane * 8) = o;
    if (lane == 0) s.scale[at] = bad ? __builtin_nanf("") : 1.0f;
    return;
  }
  const uint32_t top = group_max<kLanes>(raw.top());
  const bool bad = top >= 0x7F800000u;
  const float m = __uint_as_float(top);
  const bool zero = !bad && m < kSmallest;
  if (__builtin_amdgcn_ballot_w64(bad || zero)) {  // rare: no selects on every row's way
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bad || zero ? 0.0f : x[i];
  }
  const float mm = bad || zero ? 1.0f : m;  // what the codes are taken against
  if (FMT == OPQ_CACHE_FP8) {
    const float sc = mm / 448.0f, ri = 1.0f / sc;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = quotient(x[i], sc, ri);
    if ((__float_as_uint(sc) & 0x7FFFFFu) == 0x7FFFFFu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i] / sc;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -448.0f, 448.0f);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], v, true);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.codes) + at * D + lane * 8) =
        make_uint2(w[0], w[1]);
    if (lane == 0) s.scale[at] = bad ? __builtin_nanf("") : zero ? 0.0f : sc;
    return;
  }
  static_cast<uint32_t*>(s.codes)[at * (D / 8) + lane] = encode8(x, mm, cc);
  uint32_t sb = 0u;
#pragma unroll
  for (int i = 7; i >= 0; --i) sb = sb + sb + (x[i] < 0.0f ? 1u : 0u);
  uint32_t s32 = sb << (8 * (lane & 3));
  // OR over each group of four lanes (quad permutes 1,0,3,2 and 2,3,0,1)
  s32 |= (uint32_t)__builtin_amdgcn_mov_dpp((int)s32, 0xB1, 0xF, 0xF, false);
  s32 |= (uint32_t)__builtin_amdgcn_mov_dpp((int)s32, 0x4E, 0xF, 0xF, false);
  if ((lane & 3) == 0) s.sign[at * (D / 32) + (lane >> 2)] = s32;
  if (lane == 0) s.scale[at] = bad ? __builtin_nanf("") : zero ? 0.0f : m;
}

// A group of dim/8 lanes: HPT heads of one token, of keys (blockIdx.y = 0) or
// values (1).  A workgroup's groups are consecutive tokens of the same heads: a page
// keeps a head's tokens together, so codes, signs and scales leave as runs and not
// as lines that several XCDs write parts of (32768 tokens of 8 heads of 128, bf16:
// 41 us, 44 with consecutive heads; 5 heads, opq4: 33 and 39).
template <typename T, int FMT, int D, int HPT>
__global__ __launch_bounds__(kThreads) void write_rows(WriteArgs a, CacheCodes cc) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x % kLanes;
  const uint32_t per = (a.heads + HPT - 1) / HPT, tile = blockIdx.x / per;
  const uint32_t token = tile * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (token >= a.tokens) return;  // whole groups of lanes
  const uint32_t head = (blockIdx.x - tile * per) * HPT;
  const uint32_t slot = (uint32_t)a.slots[token];
  const CacheRows s = blockIdx.y ? a.side[1] : a.side[0];
  const T* x = static_cast<const T*>(s.x) + token * s.token_stride + lane * 8;
  Eight<T> raw[HPT];
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (head + h < a.heads) raw[h].load(x + (int64_t)(head + h) * s.head_stride, a.wide);
  if (slot >= a.slot_end) return;  // -1 among them
  const int64_t row0 = (int64_t)(slot >> a.page_shift) * a.heads + head;
  const uint32_t in_page = slot & ((1u << a.page_shift) - 1u);
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (head + h < a.heads)
      write_row<T, FMT, D>(raw[h], s, ((row0 + h) << a.page_shift) + in_page, lane, cc);
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  store_stream16(p, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  store_stream16(p, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                 __float_as_uint(v[3]));
  store_stream16(p + 4, __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                 __float_as_uint(v[7]));
}

struct ReadArgs {
  CacheRows side[2];  // x: the output
  const int32_t* slots;
  uint32_t tokens, heads, slot_end;
  int page_shift;
};

// One lane's stored part of a row.
template <int FMT, int D>
struct Stored {
  uint32_t w[FMT == OPQ_CACHE_BF16 ? 4 : 2];  // OPQ: code word and sign byte
  float scale;
  __device__ __forceinline__ void load(const CacheRows& s, int64_t at, int lane) {
    scale = s.scale[at];
    if constexpr (FMT == OPQ_CACHE_BF16) {
      const u32x4_t c = *reinterpret_cast<const u32x4_t*>(
          static_cast<const uint16_t*>(s.codes) + at * D + lane * 8);
      w[0] = c.x; w[1] = c.y; w[2] = c.z; w[3] = c.w;
    } else if constexpr (FMT == OPQ_CACHE_FP8) {
      const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.codes) +
                                                      at * D + lane * 8);
      w[0] = c.x; w[1] = c.y;
    } else {
      w[0] = static_cast<const uint32_t*>(s.codes)[at * (D / 8) + lane];
      w[1] = reinterpret_cast<const uint8_t*>(s.sign + at * (D / 32))[lane];
    }
  }
  __device__ __forceinline__ void values(const RowLut& lut, float (&v)[8]) const {
    if constexpr (FMT == OPQ_CACHE_FP8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const floatx2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const floatx2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = a.x * scale;
        v[4 * i + 1] = a.y * scale;
        v[4 * i + 2] = b.x * scale;
        v[4 * i + 3] = b.y * scale;
      }
    } else {
      uint32_t o[4];
      if constexpr (FMT == OPQ_CACHE_BF16) {
        o[0] = w[0]; o[1] = w[1]; o[2] = w[2]; o[3] = w[3];
      } else {
        decode_word_split(w[0], w[1], lut, o);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = low_half(o[i]) * scale;
        v[2 * i + 1] = high_half(o[i]) * scale;
      }
    }
  }
};

template <typename T, int FMT, int D, int HPT>
__global__ __launch_bounds__(kThreads) void read_rows(ReadArgs a, LevelPlanes lp) {
  constexpr int kLanes = D / 8;
  const uint32_t group = (blockIdx.x * (uint32_t)kThreads + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  const uint32_t per = (a.heads + HPT - 1) / HPT, token = group / per;
  if (token >= a.tokens) return;
  const uint32_t head = (group - token * per) * HPT;
  const uint32_t slot = (uint32_t)a.slots[token];
  const CacheRows s = blockIdx.y ? a.side[1] : a.side[0];
  T* out = static_cast<T*>(const_cast<void*>(s.x)) + ((int64_t)token * a.heads + head) * D + lane * 8;
  const bool there = slot < a.slot_end;
  const int64_t row0 = (int64_t)(slot >> a.page_shift) * a.heads + head;
  const uint32_t in_page = slot & ((1u << a.page_shift) - 1u);
  Stored<FMT, D> row[HPT];
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (there && head + h < a.heads) row[h].load(s, ((row0 + h) << a.page_shift) + in_page, lane);
  RowLut lut;
#pragma unroll
  for (int i = 0; i < 4; ++i) { lut.lo[i] = lp.lo[i]; lut.hi[i] = lp.hi[i]; }
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (head + h < a.heads) {
      float v[8];
      if (there) {
        row[h].values(lut, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      }
      store8(out + h * D, v);
    }
}

struct MoveArgs {
  CacheRows side[2];
  const int32_t* src;
  const int32_t* dst;
  uint32_t count, heads, slot_end;
  int page_shift, row_chunks, sign_words;  // of a row: 16-byte chunks of codes, words of signs
};

// One sequence (blockIdx.x), head (y) and side (z).  All of its rows are in the
// workgroup's registers before the barrier, and written after it.  A few KB a
// workgroup: the launch and two trips to memory bound it (32 sequences,
// 8 rows of 8 heads each: 4 us).
__global__ __launch_bounds__(kThreads) void move_rows(MoveArgs a) {
  constexpr int kChunks = (int)kMaxMoves * 32 / kThreads, kSigns = (int)kMaxMoves * 8 / kThreads;
  const int32_t* src = a.src + (int64_t)blockIdx.x * a.count;
  const int32_t* dst = a.dst + (int64_t)blockIdx.x * a.count;
  const CacheRows s = blockIdx.z ? a.side[1] : a.side[0];
  auto row_of = [&](uint32_t slot) {
    return (((int64_t)(slot >> a.page_shift) * a.heads + blockIdx.y) << a.page_shift) +
           (slot & ((1u << a.page_shift) - 1u));
  };
  // item `e` of `per` a row: its move, or none
  auto moves = [&](uint32_t e, uint32_t per, int64_t& from, int64_t& to) {
    const uint32_t i = e / per;
    if (i >= a.count) return false;
    const uint32_t f = (uint32_t)src[i], t = (uint32_t)dst[i];
    if (f >= a.slot_end || t >= a.slot_end) return false;
    from = row_of(f) * per + (e - i * per);
    to = row_of(t) * per + (e - i * per);
    return true;
  };
  u32x4_t code[kChunks];
  uint32_t sign[kSigns];
  float scale = 0.0f;
  int64_t from, to;
#pragma unroll
  for (int k = 0; k < kChunks; ++k)
    if (moves(threadIdx.x + k * kThreads, a.row_chunks, from, to))
      code[k] = static_cast<const u32x4_t*>(s.codes)[from];
  if (s.sign) {
#pragma unroll
    for (int k = 0; k < kSigns; ++k)
      if (moves(threadIdx.x + k * kThreads, a.sign_words, from, to)) sign[k] = s.sign[from];
  }
  if (moves(threadIdx.x, 1, from, to)) scale = s.scale[from];
  // every load has come back before any wave stores
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kChunks; ++k)
    if (moves(threadIdx.x + k * kThreads, a.row_chunks, from, to))
      static_cast<u32x4_t*>(s.codes)[to] = code[k];
  if (s.sign) {
#pragma unroll
    for (int k = 0; k < kSigns; ++k)
      if (moves(threadIdx.x + k * kThreads, a.sign_words, from, to)) s.sign[to] = sign[k];
  }
  if (moves(threadIdx.x, 1, from, to)) s.scale[to] = scale;
}

int page_shift_of(int64_t page) {
  int s = 0;
  while ((int64_t(1) << s) < page) ++s;
  return s;
}

template <typename F>
hipError_t in_launches(int64_t tokens, int64_t step, F one) {
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    one(t0, tokens - t0 < step ? tokens - t0 : step);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// Several heads to a group of lanes (two to write, four to read) share one look at the
// token's slot and keep that many requests in flight; with few rows a head each spreads
// the launch wider.  Rows of 8 heads of 128 from bfloat16, several and one: writing opq4
// 512 tokens 6.1 and 5.0 us, 4096 tokens 10.4 and 10.5, 32768 tokens 47 and 53 (fp8 37
// and 40, bf16 41 and 43); reading opq4 4096 tokens 4.4 and 5.0, 32768 tokens 28 and 33.
bool many_rows(const opq_cache& c, int64_t tokens) {
  return tokens * c.heads * (c.dim / 8) >= int64_t(1) << 19;
}

template <typename T, int FMT, int D, int HPT>
hipError_t write_all(const CacheRows (&side)[2], const opq_cache& c, int64_t tokens,
                     const int32_t* slots, const CacheCodes& cc, hipStream_t stream) {
  bool wide = true;
  for (const CacheRows& s : side)
    wide = wide && reinterpret_cast<uintptr_t>(s.x) % 16 == 0 &&
           s.token_stride % (int64_t)(16 / sizeof(T)) == 0 &&
           s.head_stride % (int64_t)(16 / sizeof(T)) == 0;
  // whole tiles of tokens per launch, so that its work-items count below 2^31
  const int64_t per = (c.heads + HPT - 1) / HPT, tile = kThreads / (D / 8);
  return in_launches(tokens, kMaxLaunchThreads / kThreads / per * tile, [&](int64_t t0, int64_t n) {
    const dim3 grid((unsigned)((n + tile - 1) / tile * per), 2);
    WriteArgs a{{side[0], side[1]}, slots + t0, (uint32_t)n, (uint32_t)c.heads,
                (uint32_t)(c.pages * c.page), page_shift_of(c.page), wide};
    for (CacheRows& s : a.side) s.x = static_cast<const T*>(s.x) + t0 * s.token_stride;
    hipLaunchKernelGGL((write_rows<T, FMT, D, HPT>), grid, dim3(kThreads), 0, stream, a, cc);
  });
}

template <typename T, int FMT, int D, int HPT>
hipError_t read_all(const CacheRows (&side)[2], const opq_cache& c, int64_t tokens,
                    const int32_t* slots, const LevelPlanes& lp, hipStream_t stream) {
  // whole tokens per launch, so that its work-items count below 2^31
  const int64_t per = (c.heads + HPT - 1) / HPT * (D / 8);
  return in_launches(tokens, (kMaxLaunchThreads - kThreads) / per, [&](int64_t t0, int64_t n) {
    const dim3 grid((unsigned)((n * per + kThreads - 1) / kThreads), 2);
    ReadArgs a{{side[0], side[1]}, slots + t0, (uint32_t)n, (uint32_t)c.heads,
               (uint32_t)(c.pages * c.page), page_shift_of(c.page)};
    for (CacheRows& s : a.side)
      s.x = static_cast<const T*>(s.x) + t0 * c.heads * (int64_t)D;
    hipLaunchKernelGGL((read_rows<T, FMT, D, HPT>), grid, dim3(kThreads), 0, stream, a, lp);
  });
}

template <typename T, int FMT, int D, typename... A>
hipError_t write_heads(const CacheRows (&side)[2], const opq_cache& c, int64_t tokens, A... a) {
  if (c.heads > 1 && many_rows(c, tokens))
    return write_all<T, FMT, D, 2>(side, c, tokens, a...);
  return write_all<T, FMT, D, 1>(side, c, tokens, a...);
}
template <typename T, int FMT, int D, typename... A>
hipError_t read_heads(const CacheRows (&side)[2], const opq_cache& c, int64_t tokens, A... a) {
  if (c.heads > 1 && many_rows(c, tokens))
    return read_all<T, FMT, D, 4>(side, c, tokens, a...);
  return read_all<T, FMT, D, 1>(side, c, tokens, a...);
}

template <typename T, int FMT, typename... A>
hipError_t write_dim(const CacheRows (&side)[2], const opq_cache& c, A... a) {
  if (c.dim == 64) return write_heads<T, FMT, 64>(side, c, a...);
  if (c.dim == 128) return write_heads<T, FMT, 128>(side, c, a...);
  return write_heads<T, FMT, 256>(side, c, a...);
}
template <typename T, int FMT, typename... A>
hipError_t read_dim(const CacheRows (&side)[2], const opq_cache& c, A... a) {
  if (c.dim == 64) return read_heads<T, FMT, 64>(side, c, a...);
  if (c.dim == 128) return read_heads<T, FMT, 128>(side, c, a...);
  return read_heads<T, FMT, 256>(side, c, a...);
}
template <typename T, typename... A>
hipError_t write_format(const CacheRows (&side)[2], const opq_cache& c, A... a) {
  if (c.format == OPQ_CACHE_BF16) return write_dim<T, OPQ_CACHE_BF16>(side, c, a...);
  if (c.format == OPQ_CACHE_FP8) return write_dim<T, OPQ_CACHE_FP8>(side, c, a...);
  return write_dim<T, OPQ_CACHE_OPQ4>(side, c, a...);
}
template <typename T, typename... A>
hipError_t read_format(const CacheRows (&side)[2], const opq_cache& c, A... a) {
  if (c.format == OPQ_CACHE_BF16) return read_dim<T, OPQ_CACHE_BF16>(side, c, a...);
  if (c.format == OPQ_CACHE_FP8) return read_dim<T, OPQ_CACHE_FP8>(side, c, a...);
  return read_dim<T, OPQ_CACHE_OPQ4>(side, c, a...);
}

}  // namespace

hipError_t launch_cache_write(const CacheRows (&side)[2], const opq_cache& c, bool bf16,
                              int64_t tokens, const int32_t* slots, const CacheCodes& cc,
                              hipStream_t stream) {
  return bf16 ? write_format<uint16_t>(side, c, tokens, slots, cc, stream)
              : write_format<float>(side, c, tokens, slots, cc, stream);
}

hipError_t launch_cache_move(const CacheRows (&side)[2], const opq_cache& c, int64_t batch,
                             int64_t count, const int32_t* src, const int32_t* dst,
                             hipStream_t stream) {
  const int64_t bytes = c.format == OPQ_CACHE_BF16 ? 2 * c.dim
                        : c.format == OPQ_CACHE_FP8 ? c.dim : c.dim / 2;
  const MoveArgs a{{side[0], side[1]}, src, dst, (uint32_t)count, (uint32_t)c.heads,
                   (uint32_t)(c.pages * c.page), page_shift_of(c.page), (int)(bytes / 16),
                   (int)(c.dim / 32)};
  hipLaunchKernelGGL(move_rows, dim3((unsigned)batch, (unsigned)c.heads, 2), dim3(kThreads), 0,
                     stream, a);
  return hipGetLastError();
}

namespace {

// One of the cache's arrays: what a page holds of it, in 16-byte units and in chunks.
struct PageArray {
  uint4* base;
  int64_t units;
  int chunks;
};
struct CopyArgs {
  PageArray array[6];
  const int32_t* src;
  const int32_t* dst;
  int count, chunks;  // pairs; chunks of a page over all arrays
  uint32_t pages;
};
constexpr int kCopyUnits = 4;  // 16-byte units of a lane: 4 KB a chunk

// Pages copied: a wave a chunk of a pair (4 KB, so that small pages fill waves too), all its
// loads out before the first store.  (The units are held in variables of their own: an
// array of them filled under conditions became LDS, and finding its place in it a read of the
// dispatch packet in host memory: 12 us a launch.)
__global__ __launch_bounds__(kThreads) void copy_pages(CopyArgs a) {
  int chunk = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave);
  if (chunk >= a.chunks) return;
  uint4* base = a.array[0].base;
  int64_t units = a.array[0].units;
  int held = a.array[0].chunks;
#pragma unroll
  for (int i = 1; i < 6; ++i)
    if (chunk >= held) {
      chunk -= held;
      base = a.array[i].base;
      units = a.array[i].units;
      held = a.array[i].chunks;
    }
  const int64_t last = units - 1;
  const int64_t at = (int64_t)chunk * (kWave * kCopyUnits) + (threadIdx.x & (kWave - 1));
  for (int pair = blockIdx.y; pair < a.count; pair += gridDim.y) {
    const int32_t src = a.src[pair], dst = a.dst[pair];
    if ((uint32_t)src >= a.pages || (uint32_t)dst >= a.pages || src == dst) continue;
    const uint4* from = base + src * units;
    uint4* to = base + dst * units;
    const uint4 v0 = from[min(at, last)], v1 = from[min(at + kWave, last)];
    const uint4 v2 = from[min(at + 2 * kWave, last)], v3 = from[min(at + 3 * kWave, last)];
    if (at <= last) to[at] = v0;
    if (at + kWave <= last) to[at + kWave] = v1;
    if (at + 2 * kWave <= last) to[at + 2 * kWave] = v2;
    if (at + 3 * kWave <= last) to[at + 3 * kWave] = v3;
  }
}

}  // namespace

hipError_t launch_cache_copy_pages(const CacheRows (&side)[2], const opq_cache& c, int64_t count,
                                   const int32_t* src, const int32_t* dst, hipStream_t stream) {
  const int64_t rows = c.heads * c.page;
  const int64_t bytes = c.format == OPQ_CACHE_BF16 ? 2 * c.dim
                        : c.format == OPQ_CACHE_FP8 ? c.dim : c.dim / 2;
  CopyArgs a{};
  for (int i = 0; i < 2; ++i) {
    void* const base[3] = {side[i].codes, side[i].sign, side[i].scale};
    const int64_t units[3] = {rows * bytes / 16, side[i].sign ? rows * (c.dim / 32) / 4 : 0, rows / 4};
    for (int j = 0; j < 3; ++j) {
      const int chunks = (int)((units[j] + kWave * kCopyUnits - 1) / (kWave * kCopyUnits));
      a.array[3 * i + j] = {static_cast<uint4*>(base[j]), units[j], chunks};
      a.chunks += chunks;
    }
  }
  a.src = src;
  a.dst = dst;
  a.count = (int)count;
  a.pages = (uint32_t)c.pages;
  const unsigned x = (unsigned)((a.chunks + kThreads / kWave - 1) / (kThreads / kWave));
  hipLaunchKernelGGL(copy_pages, dim3(x, (unsigned)(count < 4096 ? count : 4096)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheRows (&side)[2], const opq_cache& c, bool bf16,
                             int64_t tokens, const int32_t* slots, const LevelPlanes& lp,
                             hipStream_t stream) {
  return bf16 ? read_format<uint16_t>(side, c, tokens, slots, lp, stream)
              : read_format<float>(side, c, tokens, slots, lp, stream);
}

}  // namespace opq
