// Rotary positions: a pair (a, b) of a head's dimensions is turned by an angle
// that grows with the token's position, a' = a c - b s, b' = a s + b c, with
// (c, s) = table[position][pair].  The turn is orthogonal (times the table's
// amplitude), so its gradient is the turn by the opposite angle.
//
// Bound by memory: every element is read and written once.  The table's row
// (8 bytes a pair) is shared by all heads of a token, so a thread keeps its
// pairs' (c, s) in registers and walks several heads with it.
#include "attention_internal.hpp"
#include "device_common.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;

// N consecutive elements aligned to A elements (16 bytes at most): loaded and
// stored with accesses as wide as that.
template <typename T, int N, int A = N>
struct alignas(sizeof(T) * A < 16 ? sizeof(T) * A : 16) Pack {
  T v[N];
};

// The stores of a large call carry the nontemporal hint: 4096 tokens of 60 heads of
// 128 from rows of 90, three axes, bfloat16, 25.1 us a call without and 21.9 with it
// (5.7 TB/s read and written); with a cache write of the result behind it 46.2 and 44.5
// together, in place 23.8 and 21.6.
template <bool kStream, typename P>
__device__ __forceinline__ void put(void* p, const P& v) {
  if constexpr (kStream && sizeof(P) == 16) {
    const u32x4_t w = __builtin_bit_cast(u32x4_t, v);
    store_stream16(p, w.x, w.y, w.z, w.w);
  } else {
    *static_cast<P*>(p) = v;
  }
}

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float widen(float f) { return f; }
__device__ __forceinline__ void narrow(float f, float& o) { o = f; }
__device__ __forceinline__ void narrow(float f, uint16_t& o) {
  o = __builtin_bit_cast(uint16_t, (__bf16)f);
}

// Elements that one thread holds of a head: VE of each half (half layout) or VE
// consecutive ones (interleaved).  Without alignment (AE = 1) a thread turns
// one pair, and what is not turned is copied element by element, so no boundary
// has to be a multiple of anything.
template <int VE, int AE>
constexpr int kTail = AE == 1 ? 1 : VE;

// One thread: one chunk of HPT heads of one token.  Items of a token's head: the
// turned chunks first, then the chunks of rot..dim-1, which are copied.
template <typename T, int VE, int AE, bool kInter, int HPT>
__global__ __launch_bounds__(kThreads) void rotary_rows(RotaryArgs a) {
  constexpr int kPairs = kInter ? VE / 2 : VE;
  constexpr int TE = kTail<VE, AE>;
  constexpr bool kStream = HPT > 1;  // the large calls
  typedef Pack<T, VE, AE> P;
  typedef Pack<T, TE, AE> Q;
  const uint32_t turned = (uint32_t)(a.rot / 2 / kPairs);
  const uint32_t items = turned + (uint32_t)((a.dim - a.rot) / TE);
  const uint32_t hgroups = (uint32_t)((a.heads + HPT - 1) / HPT);
  const uint32_t idx = blockIdx.x * (uint32_t)kThreads + threadIdx.x;  // below 2^31
  const uint32_t per = items * hgroups;  // work items of a token
  const uint32_t tk = idx / per;
  const int64_t token = tk;
  if (token >= a.tokens) return;
  const uint32_t rest = idx - tk * per;
  const uint32_t hg = rest / items, item = rest - hg * items;
  const int h0 = (int)hg * HPT;
  const T* x = static_cast<const T*>(a.x) + token * a.x_token + h0 * a.x_head;
  T* out = static_cast<T*>(a.out) + token * a.out_token + h0 * a.out_head;

  if (item >= turned) {  // not turned: copied
    const int at = a.rot + (int)(item - turned) * TE;
    Q t[HPT];
#pragma unroll
    for (int h = 0; h < HPT; ++h)
      if (h0 + h < a.heads) t[h] = *reinterpret_cast<const Q*>(x + h * a.x_head + at);
#pragma unroll
    for (int h = 0; h < HPT; ++h)
      if (h0 + h < a.heads) put<kStream>(out + h * a.out_head + at, t[h]);
    return;
  }

  const int p0 = (int)item * kPairs;
  const int lo = kInter ? 2 * p0 : p0;
  const int hi = a.rot / 2 + p0;  // half layout only
  P u[HPT], w[HPT];
#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (h0 + h < a.heads) {
      u[h] = *reinterpret_cast<const P*>(x + h * a.x_head + lo);
      if (!kInter) w[h] = *reinterpret_cast<const P*>(x + h * a.x_head + hi);
    }

  // a chunk's pairs share an axis: the sections are multiples of kPairs
  int axis = 0;
#pragma unroll
  for (int i = 0; i + 1 < kMaxAxes; ++i) axis += (i + 1 < a.axes && p0 >= a.end[i]) ? 1 : 0;
  const int64_t pos = a.positions[token * a.axes + axis];
  const bool inside = pos >= 0 && pos < a.table_len;
  Pack<float, 2 * kPairs> cs;
  if (inside)
    cs = *reinterpret_cast<const Pack<float, 2 * kPairs>*>(a.table + pos * a.rot + 2 * p0);
  else
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) cs.v[i] = __builtin_nanf("");

#pragma unroll
  for (int h = 0; h < HPT; ++h)
    if (h0 + h < a.heads) {
      P r, s;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float c = cs.v[2 * i], sn = cs.v[2 * i + 1] * a.turn;
        const float p = widen(kInter ? u[h].v[2 * i] : u[h].v[i]);
        const float q = widen(kInter ? u[h].v[2 * i + 1] : w[h].v[i]);
        const float np = p * c - q * sn, nq = p * sn + q * c;
        if (kInter) {
          narrow(np, r.v[2 * i]);
          narrow(nq, r.v[2 * i + 1]);
        } else {
          narrow(np, r.v[i]);
          narrow(nq, s.v[i]);
        }
      }
      put<kStream>(out + h * a.out_head + lo, r);
      if (!kInter) put<kStream>(out + h * a.out_head + hi, s);
    }
}

// Positions `first` .. first + len - 1, into `table` from its start.
__global__ __launch_bounds__(kThreads) void rotary_table(const double* __restrict__ freq,
                                                         int pairs, int64_t first, int64_t len,
                                                         double amplitude,
                                                         float* __restrict__ table) {
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t at = idx / pairs;
  if (at >= len) return;
  const int i = (int)(idx - at * pairs);
  // turns of the angle pos * f, the whole ones dropped.  r is within 2^-53 of
  // itself relative, so a context of 10^6 keeps 1e-10 of a turn.
  const double turns = (double)(first + at) * (freq[i] * 0.15915494309189533577);
  const double r = turns - rint(turns);
  double s, c;
  sincospi(2.0 * r, &s, &c);
  *reinterpret_cast<float2*>(table + 2 * idx) =
      make_float2((float)(c * amplitude), (float)(s * amplitude));
}

template <typename T, int VE, int AE, bool kInter, int HPT>
hipError_t go(const RotaryArgs& a, hipStream_t stream) {
  const int pairs = kInter ? VE / 2 : VE;
  const int64_t per = (int64_t)(a.rot / 2 / pairs + (a.dim - a.rot) / kTail<VE, AE>) *
                      ((a.heads + HPT - 1) / HPT);
  // whole tokens per launch, within the 32-bit count of work-items
  const int64_t step = kMaxLaunchThreads / per;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += step) {
    RotaryArgs p = a;
    p.x = static_cast<const T*>(a.x) + t0 * a.x_token;
    p.out = static_cast<T*>(a.out) + t0 * a.out_token;
    p.positions = a.positions + t0 * a.axes;
    p.tokens = a.tokens - t0 < step ? a.tokens - t0 : step;
    const dim3 grid((unsigned)((p.tokens * per + kThreads - 1) / kThreads));
    hipLaunchKernelGGL((rotary_rows<T, VE, AE, kInter, HPT>), grid, dim3(kThreads), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Several heads per thread share one read of the table's row and keep more
// requests in flight; with few tokens the launch is latency-bound and a head per
// thread spreads it wider.  32 heads of 128, bfloat16: 512 tokens 4.0 us by four,
// 3.5 singly; 1024 tokens 5.1 and 5.6; 4096 tokens 11.9 and 15.1; 16384 tokens 50
// and 52 (5.4 TB/s).
template <typename T, int VE, int AE, bool kInter>
hipError_t go_heads(const RotaryArgs& a, hipStream_t stream) {
  const int64_t threads = a.tokens * a.heads * (int64_t)(a.dim / (2 * VE) + 1);
  if (threads >= int64_t(1) << 18) return go<T, VE, AE, kInter, 4>(a, stream);
  return go<T, VE, AE, kInter, 1>(a, stream);
}

// Can chunks of VE elements tile every boundary, and is every access aligned?
template <typename T>
bool fits(const RotaryArgs& a, bool inter, int ve) {
  const uintptr_t bytes = sizeof(T) * (uintptr_t)ve;
  if (reinterpret_cast<uintptr_t>(a.x) % bytes || reinterpret_cast<uintptr_t>(a.out) % bytes)
    return false;
  if (a.x_token % ve || a.x_head % ve || a.out_token % ve || a.out_head % ve) return false;
  if (a.dim % ve || a.rot % ve || (!inter && (a.rot / 2) % ve)) return false;
  const int pairs = inter ? ve / 2 : ve;
  for (int i = 0; i < a.axes; ++i)
    if (a.end[i] % pairs) return false;
  return true;
}

template <typename T>
hipError_t pick(const RotaryArgs& a, bool inter, hipStream_t stream) {
  constexpr int kWide = 16 / sizeof(T);
  if (inter) {
    if (fits<T>(a, true, kWide)) return go_heads<T, kWide, kWide, true>(a, stream);
    return go_heads<T, 2, 1, true>(a, stream);
  }
  if (fits<T>(a, false, kWide)) return go_heads<T, kWide, kWide, false>(a, stream);
  return go_heads<T, 1, 1, false>(a, stream);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, bool bf16, bool interleaved, hipStream_t stream) {
  return bf16 ? pick<uint16_t>(a, interleaved, stream) : pick<float>(a, interleaved, stream);
}

hipError_t launch_rotary_table(const double* freq, int64_t pairs, int64_t len, double amplitude,
                               float* table, hipStream_t stream) {
  // whole positions per launch, within the 32-bit count of work-items
  const int64_t step = kMaxLaunchThreads / pairs;
  for (int64_t p0 = 0; p0 < len; p0 += step) {
    const int64_t n = len - p0 < step ? len - p0 : step;
    const dim3 grid((unsigned)((n * pairs + kThreads - 1) / kThreads));
    hipLaunchKernelGGL(rotary_table, grid, dim3(kThreads), 0, stream, freq, (int)pairs, p0, n,
                       amplitude, table + 2 * p0 * pairs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace opq
