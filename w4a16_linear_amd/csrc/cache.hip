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
// the maximum is a few lane exchanges and nothing is read twice.  Bound by
// memory for long prompts (2 bytes in, 0.66 to 2 out per value), by the launch for a
// few tokens.
#include "attention_internal.hpp"
#include "decode.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;
constexpr float kSmallest = 0x1p-100f;  // rows below it are stored as zeros

typedef float floatx2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const floatx2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
}
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Eight values of a row; `wide` when their address is a multiple of 16 bytes.
__device__ __forceinline__ void load8(const uint16_t* p, bool wide, float (&x)[8]) {
  uint32_t w[4];
  if (wide) {
    const u32x4_t v = load_stream16(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = low_half(w[i]);
    x[2 * i + 1] = high_half(w[i]);
  }
}
__device__ __forceinline__ void load8(const float* p, bool wide, float (&x)[8]) {
  if (wide) {
    const u32x4_t a = load_stream16(p), b = load_stream16(p + 4);
    x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
    x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
    x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
    x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p[i];
  }
}

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

// Nibbles of eight magnitudes.  The power comes from the hardware's log2 and exp2
// on |x| * fl(1/m): its error is far below cc.guard, so a result farther than
// that from a half-integer rounds to the exact code, and the few others (and
// every row whose 1/m is not a normal number) are decided by code_exact.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float m, const CacheCodes& cc) {
  const float r = __builtin_amdgcn_rcpf(m);
  uint32_t word = 0u;
  bool sure = r >= 0x1p-126f;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    const float lg = __builtin_amdgcn_logf(fabsf(x[i]) * r);
    const float p = fminf(15.0f * __builtin_amdgcn_exp2f(cc.alpha * lg), 15.0f);
    const float n = __builtin_rintf(p);
    sure = sure && fabsf(p - n) < 0.5f - cc.guard;
    word = (word << 4) + (uint32_t)n;
  }
  if (!sure) {
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

struct WriteArgs {
  CacheRows side[2];
  const int32_t* slots;
  uint32_t rows;  // tokens * heads of this launch
  uint32_t heads;
  uint32_t slot_end;  // pages * page
  int page_shift;
  bool wide;
};

// Row (token, head) of keys (blockIdx.y = 0) or values (1).
template <typename T, int FMT, int D>
__global__ __launch_bounds__(kThreads) void write_rows(WriteArgs a, CacheCodes cc) {
  constexpr int kLanes = D / 8;
  const uint32_t row = (blockIdx.x * (uint32_t)kThreads + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (row >= a.rows) return;  // whole groups of lanes
  const uint32_t token = row / a.heads, head = row - token * a.heads;
  const uint32_t slot = (uint32_t)a.slots[token];
  if (slot >= a.slot_end) return;  // -1 among them
  const CacheRows s = blockIdx.y ? a.side[1] : a.side[0];
  float x[8];
  load8(static_cast<const T*>(s.x) + token * s.token_stride + head * s.head_stride + lane * 8,
        a.wide, x);
  const uint32_t page = slot >> a.page_shift;
  const int64_t at = ((((int64_t)page * a.heads + head) << a.page_shift) +
                      (slot & ((1u << a.page_shift) - 1u)));

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
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = group_max<kLanes>(top);
  const bool bad = top >= 0x7F800000u;
  const float m = __uint_as_float(top);
  const bool zero = !bad && m < kSmallest;
  if (bad || zero) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  }
  const float mm = bad || zero ? 1.0f : m;  // what the codes are taken against
  if (FMT == OPQ_CACHE_FP8) {
    const float sc = mm / 448.0f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(x[i] / sc, -448.0f, 448.0f);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], v, true);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(s.codes) + at * D + lane * 8) =
        make_uint2(w[0], w[1]);
    if (lane == 0) s.scale[at] = bad ? __builtin_nanf("") : zero ? 0.0f : sc;
    return;
  }
  const uint32_t word = encode8(x, mm, cc);
  static_cast<uint32_t*>(s.codes)[at * (D / 8) + lane] = word;
  uint32_t sb = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) sb |= (x[i] < 0.0f ? 1u : 0u) << i;
  uint32_t s32 = sb << (8 * (lane & 3));
  // OR over each group of four lanes (quad permutes 1,0,3,2 and 2,3,0,1)
  s32 |= (uint32_t)__builtin_amdgcn_mov_dpp((int)s32, 0xB1, 0xF, 0xF, false);
  s32 |= (uint32_t)__builtin_amdgcn_mov_dpp((int)s32, 0x4E, 0xF, 0xF, false);
  if ((lane & 3) == 0) s.sign[at * (D / 32) + (lane >> 2)] = s32;
  if (lane == 0) s.scale[at] = bad ? __builtin_nanf("") : zero ? 0.0f : m;
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
  uint32_t rows, heads, slot_end;
  int page_shift;
};

template <typename T, int FMT, int D>
__global__ __launch_bounds__(kThreads) void read_rows(ReadArgs a, LevelPlanes lp) {
  constexpr int kLanes = D / 8;
  const uint32_t row = (blockIdx.x * (uint32_t)kThreads + threadIdx.x) / kLanes;
  const int lane = threadIdx.x % kLanes;
  if (row >= a.rows) return;
  const uint32_t token = row / a.heads, head = row - token * a.heads;
  const uint32_t slot = (uint32_t)a.slots[token];
  const CacheRows s = blockIdx.y ? a.side[1] : a.side[0];
  T* out = static_cast<T*>(const_cast<void*>(s.x)) + (int64_t)row * D + lane * 8;
  float v[8];
  if (slot >= a.slot_end) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    store8(out, v);
    return;
  }
  const uint32_t page = slot >> a.page_shift;
  const int64_t at = ((((int64_t)page * a.heads + head) << a.page_shift) +
                      (slot & ((1u << a.page_shift) - 1u)));
  const float sc = s.scale[at];
  if (FMT == OPQ_CACHE_FP8) {
    const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(s.codes) + at * D +
                                                    lane * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const floatx2_t f = (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)(i < 2 ? c.x : c.y), true)
                                  : __builtin_amdgcn_cvt_pk_f32_fp8((int)(i < 2 ? c.x : c.y), false);
      v[2 * i] = f.x * sc;
      v[2 * i + 1] = f.y * sc;
    }
  } else {
    uint32_t w[4];
    if (FMT == OPQ_CACHE_BF16) {
      const u32x4_t c = *reinterpret_cast<const u32x4_t*>(
          static_cast<const uint16_t*>(s.codes) + at * D + lane * 8);
      w[0] = c.x; w[1] = c.y; w[2] = c.z; w[3] = c.w;
    } else {
      const uint32_t code = static_cast<const uint32_t*>(s.codes)[at * (D / 8) + lane];
      const uint32_t sb = reinterpret_cast<const uint8_t*>(s.sign + at * (D / 32))[lane];
      RowLut t;
#pragma unroll
      for (int i = 0; i < 4; ++i) { t.lo[i] = lp.lo[i]; t.hi[i] = lp.hi[i]; }
      decode_word_split(code, sb, t, w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = low_half(w[i]) * sc;
      v[2 * i + 1] = high_half(w[i]) * sc;
    }
  }
  store8(out, v);
}

int page_shift_of(int64_t page) {
  int s = 0;
  while ((int64_t(1) << s) < page) ++s;
  return s;
}

// Whole tokens per launch, so that its work-items count below 2^31.
template <typename F>
hipError_t in_launches(const opq_cache& c, int64_t tokens, F one) {
  const int64_t per = c.heads * (c.dim / 8);
  const int64_t step = (kMaxLaunchThreads - kThreads) / per;
  for (int64_t t0 = 0; t0 < tokens; t0 += step) {
    const int64_t n = tokens - t0 < step ? tokens - t0 : step;
    one(t0, n, dim3((unsigned)((n * per + kThreads - 1) / kThreads), 2));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int FMT, int D>
hipError_t write_all(const CacheRows (&side)[2], const opq_cache& c, int64_t tokens,
                     const int32_t* slots, const CacheCodes& cc, hipStream_t stream) {
  bool wide = true;
  for (const CacheRows& s : side)
    wide = wide && reinterpret_cast<uintptr_t>(s.x) % 16 == 0 &&
           s.token_stride % (int64_t)(16 / sizeof(T)) == 0 &&
           s.head_stride % (int64_t)(16 / sizeof(T)) == 0;
  return in_launches(c, tokens, [&](int64_t t0, int64_t n, dim3 grid) {
    WriteArgs a{{side[0], side[1]}, slots + t0, (uint32_t)(n * c.heads), (uint32_t)c.heads,
                (uint32_t)(c.pages * c.page), page_shift_of(c.page), wide};
    for (CacheRows& s : a.side) s.x = static_cast<const T*>(s.x) + t0 * s.token_stride;
    hipLaunchKernelGGL((write_rows<T, FMT, D>), grid, dim3(kThreads), 0, stream, a, cc);
  });
}

template <typename T, int FMT, int D>
hipError_t read_all(const CacheRows (&side)[2], const opq_cache& c, int64_t tokens,
                    const int32_t* slots, const LevelPlanes& lp, hipStream_t stream) {
  return in_launches(c, tokens, [&](int64_t t0, int64_t n, dim3 grid) {
    ReadArgs a{{side[0], side[1]}, slots + t0, (uint32_t)(n * c.heads), (uint32_t)c.heads,
               (uint32_t)(c.pages * c.page), page_shift_of(c.page)};
    for (CacheRows& s : a.side)
      s.x = static_cast<const T*>(s.x) + t0 * c.heads * (int64_t)D;
    hipLaunchKernelGGL((read_rows<T, FMT, D>), grid, dim3(kThreads), 0, stream, a, lp);
  });
}

template <typename T, int FMT, typename... A>
hipError_t write_dim(const CacheRows (&side)[2], const opq_cache& c, A... a) {
  if (c.dim == 64) return write_all<T, FMT, 64>(side, c, a...);
  if (c.dim == 128) return write_all<T, FMT, 128>(side, c, a...);
  return write_all<T, FMT, 256>(side, c, a...);
}
template <typename T, int FMT, typename... A>
hipError_t read_dim(const CacheRows (&side)[2], const opq_cache& c, A... a) {
  if (c.dim == 64) return read_all<T, FMT, 64>(side, c, a...);
  if (c.dim == 128) return read_all<T, FMT, 128>(side, c, a...);
  return read_all<T, FMT, 256>(side, c, a...);
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

hipError_t launch_cache_read(const CacheRows (&side)[2], const opq_cache& c, bool bf16,
                             int64_t tokens, const int32_t* slots, const LevelPlanes& lp,
                             hipStream_t stream) {
  return bf16 ? read_format<uint16_t>(side, c, tokens, slots, lp, stream)
              : read_format<float>(side, c, tokens, slots, lp, stream);
}

}  // namespace opq
