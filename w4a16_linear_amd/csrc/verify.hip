// Drafted tokens verified against the target's probabilities (include/opq_attention.h).
//
// What decides is little: one probability (two with a draft model's) a tested token.  What
// has to be read is the one row that `next` is drawn from, all of the vocabulary (and q's
// row with it): the floor.  Two kernels: verify_sums, a workgroup a piece of the row, each
// finding the last kept token by itself (one wave; the whole walk is a few
// gathers and register steps), then adding its piece; verify_draw, a workgroup a
// sequence, finds the piece that u0 falls into and the token in it.
//
// Sums are float64: a float32 sum over 10^5 weights is off by 10^-6 of the whole, the
// weight of many tokens of a long tail.  u q is a product of two float32 values in float64,
// which is exact; Z, a float64 sum of float32 values, and u Z are rounded.
#include <algorithm>

#include "attention_internal.hpp"
#include "device_common.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDraft = 1024;
constexpr int kPiece = 4096;   // tokens of a piece, as long as there are pieces enough
constexpr int kSmall = 1024;   // tokens of a piece of few and short rows
constexpr int kMaxPieces = 1024;

enum Mode { kAll = 0, kLessDraft = 1, kLessTested = 2 };  // weights of the last draw

struct Found {  // what verify_sums leaves a sequence for verify_draw
  int node, mode;
};

// A probability as it counts.
__device__ __forceinline__ float proper(float v) { return v > 0.0f && v < __builtin_inff() ? v : 0.0f; }

template <typename T> __device__ __forceinline__ float as_float(T v);
template <> __device__ __forceinline__ float as_float<float>(float v) { return v; }
template <> __device__ __forceinline__ float as_float<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Four neighbours at an element's alignment: rows start anywhere.
template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) Four { T v[4]; };

// The walk, by one wave: kept tokens go to `kept` (or nowhere), the return value is
// their number; found tells what the last draw needs.
template <typename T>
__device__ int walk(const VerifyArgs& a, int b, int count, int32_t* kept, Found* found) {
  const int lane = threadIdx.x & (kWave - 1);
  const int32_t* tokens = a.tokens + (int64_t)b * a.draft;
  const int32_t* parents = a.parents ? a.parents + (int64_t)b * a.draft : nullptr;
  const float* uniforms = a.uniforms + (int64_t)b * a.draft;
  const T* p = static_cast<const T*>(a.p) + b * a.p_batch;
  const T* q = static_cast<const T*>(a.q) + (a.q ? b * a.q_batch : 0);
  int node = 0, number = 1, tested = 0;
  double left = 1.0;
  if (kept && lane == 0) kept[0] = 0;
  for (int t0 = 0; t0 < count; t0 += kWave) {
    const int t = t0 + lane;
    const bool in = t > 0 && t < count;
    const int parent = in ? (parents ? parents[t] : t - 1) : -1;
    const int token = in ? tokens[t] : -1;
    const float u = in ? uniforms[t] : 0.0f;
    const bool real = in && parent >= 0 && parent < t && token >= 0 && token < a.vocab;
    float px = 0.0f, qx = 0.0f;
    if (real) {
      px = proper(as_float<T>(p[parent * a.p_token + token]));
      if (a.q) qx = proper(as_float<T>(q[(t - 1) * a.q_token + token]));
    }
    uint64_t todo = ~uint64_t(0);
    while (true) {
      const uint64_t children = __ballot(in && parent == node) & todo;
      if (!children) break;
      const int at = __ffsll((unsigned long long)children) - 1;
      todo = at == 63 ? 0 : ~uint64_t(0) << (at + 1);
      double pd = readlane_f(px, at);
      const double ud = readlane_f(u, at), qd = readlane_f(qx, at);
      if (!a.q && tested) {  // an earlier sibling's token again counts nothing; siblings come after the node
        const int x = __builtin_amdgcn_readlane(token, at);
        bool again = __ballot(in && t > node && lane < at && parent == node && token == x);
        for (int s0 = node / kWave * kWave; s0 < t0 && !again; s0 += kWave) {
          const int s = s0 + lane;
          again = __ballot(s > node && (parents ? parents[s] : s - 1) == node && tokens[s] == x);
        }
        if (again) pd = 0.0;
      }
      if (pd > 0.0 && ud * (a.q ? qd : left) < pd) {
        node = t0 + at;
        left = 1.0;
        tested = 0;
        if (kept && lane == 0) kept[number] = node;
        ++number;
      } else {
        left -= pd;
        tested = 1;
      }
    }
  }
  if (kept)
    for (int t = number + lane; t < a.draft; t += kWave) kept[t] = -1;
  found->node = node;
  found->mode = !tested ? kAll : a.q ? kLessDraft : kLessTested;
  return number;
}

__device__ __forceinline__ int counted(const VerifyArgs& a, int b) {
  return a.counts ? max(0, min(a.counts[b], a.draft)) : a.draft;
}

// Bits of the tokens of a piece that were tested under `node`.
template <int PIECE>
__device__ void tested_bits(const VerifyArgs& a, int b, int count, int node, int v0, uint32_t* bits) {
  for (int w = threadIdx.x; w < PIECE / 32; w += kThreads) bits[w] = 0;
  __syncthreads();
  const int32_t* tokens = a.tokens + (int64_t)b * a.draft;
  const int32_t* parents = a.parents ? a.parents + (int64_t)b * a.draft : nullptr;
  for (int t = node + 1 + threadIdx.x; t < count; t += kThreads)
    if ((parents ? parents[t] : t - 1) == node) {
      const int at = tokens[t] - v0;
      if (tokens[t] >= 0 && at >= 0 && at < PIECE) atomicOr(bits + at / 32, 1u << (at % 32));
    }
  __syncthreads();
}

// Weights of tokens v0 + at .. + 3 (0 past the vocabulary).
template <typename T>
__device__ __forceinline__ void weights(const T* p, const T* q, const uint32_t* bits, int v0, int at, int vocab,
                                        double (&w)[4]) {
  float pv[4] = {}, qv[4] = {};
  if (v0 + at + 4 <= vocab) {
    const Four<T> f = *reinterpret_cast<const Four<T>*>(p + v0 + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) pv[i] = as_float<T>(f.v[i]);
    if (q) {
      const Four<T> g = *reinterpret_cast<const Four<T>*>(q + v0 + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = as_float<T>(g.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v0 + at + i < vocab) {
        pv[i] = as_float<T>(p[v0 + at + i]);
        if (q) qv[i] = as_float<T>(q[v0 + at + i]);
      }
  }
  const uint32_t gone = bits ? bits[at / 32] >> (at % 32) : 0u;  // at is a multiple of 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double d = (double)proper(pv[i]) - (double)proper(qv[i]);
    w[i] = d > 0.0 && !(gone >> i & 1u) ? d : 0.0;
  }
}

// The rows that the last draw's weights come from.
template <typename T>
__device__ __forceinline__ void rows_of(const VerifyArgs& a, int b, Found f, const T** p, const T** q) {
  *p = static_cast<const T*>(a.p) + b * a.p_batch + f.node * a.p_token;
  *q = f.mode == kLessDraft ? static_cast<const T*>(a.q) + b * a.q_batch + f.node * a.q_token : nullptr;
}

// Workgroup (piece, sequence): the sum of the piece's weights.
template <typename T, int PIECE>
__global__ __launch_bounds__(kThreads) void verify_sums(VerifyArgs a, double* sums, Found* founds) {
  __shared__ Found s_found;
  __shared__ uint32_t s_bits[PIECE / 32];
  __shared__ double s_sum[kThreads / kWave];
  const int b = blockIdx.y, piece = blockIdx.x, pieces = gridDim.x;
  const int count = counted(a, b);
  if (threadIdx.x < kWave) {
    Found f{0, kAll};
    int32_t* kept = piece == 0 ? a.kept + (int64_t)b * a.draft : nullptr;
    int number = 0;
    if (count > 0) {
      number = walk<T>(a, b, count, kept, &f);
    } else if (kept) {
      for (int t = threadIdx.x; t < a.draft; t += kWave) kept[t] = -1;
    }
    if (threadIdx.x == 0) {
      s_found = f;
      if (piece == 0) {
        founds[b] = f;
        a.count[b] = number;
      }
    }
  }
  __syncthreads();
  if (count == 0) return;
  const Found f = s_found;
  const T *p, *q;
  rows_of<T>(a, b, f, &p, &q);
  const int v0 = piece * PIECE;
  const uint32_t* bits = nullptr;
  if (f.mode == kLessTested) {
    tested_bits<PIECE>(a, b, count, f.node, v0, s_bits);
    bits = s_bits;
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PIECE / (4 * kThreads); ++i) {
    double w[4];
    weights<T>(p, q, bits, v0, (i * kThreads + threadIdx.x) * 4, a.vocab, w);
    sum += (w[0] + w[1]) + (w[2] + w[3]);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  if ((threadIdx.x & (kWave - 1)) == 0) s_sum[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) sums[(int64_t)b * pieces + piece] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

// This thread's value added over the threads up to and with it, in a fixed order.
__device__ __forceinline__ double scan(double v, double* s_sum, double* all) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  for (int off = 1; off < kWave; off <<= 1) {
    const double o = __shfl_up(v, off, kWave);
    if (lane >= off) v += o;
  }
  __syncthreads();
  if (lane == kWave - 1) s_sum[wave] = v;
  __syncthreads();
  double before = 0.0, total = 0.0;
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w < wave) before += s_sum[w];
    total += s_sum[w];
  }
  *all = total;
  return before + v;
}

// The lowest `first` and the highest `last` of the workgroup: a wave's lowest is that of its
// lowest lane that has one, so one lane a wave goes to LDS.
__device__ __forceinline__ void note(int first, int last, int* s_first, int* s_last) {
  const uint64_t some = __ballot(last >= 0), past = __ballot(first != 0x7FFFFFFF);
  const int lane = threadIdx.x & (kWave - 1);
  if (past && lane == __ffsll((unsigned long long)past) - 1) atomicMin(s_first, first);
  if (some && lane == 63 - __clzll((long long)some)) atomicMax(s_last, last);
}

// Workgroup = sequence: the piece, then the token.
template <typename T, int PIECE>
__global__ __launch_bounds__(kThreads) void verify_draw(VerifyArgs a, const double* sums, const Found* founds,
                                                        int pieces) {
  __shared__ uint32_t s_bits[PIECE / 32];
  __shared__ double s_sum[kThreads / kWave];
  __shared__ double s_before;
  __shared__ int s_first, s_last;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int count = counted(a, b);
  if (count == 0) {
    if (tid == 0) a.next[b] = -1;
    return;
  }
  if (tid == 0) {
    s_first = 0x7FFFFFFF;
    s_last = -1;
  }
  const int per = (pieces + kThreads - 1) / kThreads;
  double mine = 0.0, all;
  for (int i = tid * per; i < min(pieces, (tid + 1) * per); ++i) mine += sums[(int64_t)b * pieces + i];
  const double to = scan(mine, s_sum, &all);
  const double aim = (double)a.uniforms[(int64_t)b * a.draft] * all;
  {
    double at = to - mine;
    int first = 0x7FFFFFFF, last = -1;
    for (int i = tid * per; i < min(pieces, (tid + 1) * per); ++i) {
      const double s = sums[(int64_t)b * pieces + i];
      if (s > 0.0) {
        last = i;
        if (at + s > aim) first = min(first, i);
      }
      at += s;
    }
    note(first, last, &s_first, &s_last);
  }
  __syncthreads();
  if (s_last < 0) {  // nothing to draw from
    if (tid == 0) a.next[b] = -1;
    return;
  }
  const int piece = min(s_first, s_last);
  if (piece / per == tid) {  // what the pieces before it hold
    double at = to - mine;
    for (int i = tid * per; i < piece; ++i) at += sums[(int64_t)b * pieces + i];
    s_before = at;
  }
  __syncthreads();
  if (tid == 0) {
    s_first = 0x7FFFFFFF;
    s_last = -1;
  }
  const Found f = founds[b];
  const T *p, *q;
  rows_of<T>(a, b, f, &p, &q);
  const int v0 = piece * PIECE;
  const uint32_t* bits = nullptr;
  if (f.mode == kLessTested) {
    tested_bits<PIECE>(a, b, count, f.node, v0, s_bits);
    bits = s_bits;
  }
  constexpr int kRun = PIECE / kThreads;  // tokens of a thread, one after the other
  double w[kRun], own = 0.0;
#pragma unroll
  for (int i = 0; i < kRun; i += 4) {
    double four[4];
    weights<T>(p, q, bits, v0, tid * kRun + i, a.vocab, four);
#pragma unroll
    for (int e = 0; e < 4; ++e) own += w[i + e] = four[e];
  }
  double at = s_before + (scan(own, s_sum, &all) - own);
  int first = 0x7FFFFFFF, last = -1;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    at += w[i];
    if (w[i] > 0.0) {
      last = v0 + tid * kRun + i;
      if (at > aim) first = min(first, last);
    }
  }
  note(first, last, &s_first, &s_last);
  __syncthreads();
  if (tid == 0) a.next[b] = min(s_first, s_last);
}

struct VerifyPlan {
  bool small;
  int64_t pieces;
};
// Long pieces, unless they would make fewer than 512 workgroups (long / short, us in a graph: 8 rows of
// 131072 9.9/9.0, 64 of 32000, 512 workgroups, 11.6/10.4, 128 of them 13.9/14.3, 64 of 131072 17.8/23.2).
VerifyPlan verify_plan(int64_t batch, int64_t vocab) {
  const int64_t big = (vocab + kPiece - 1) / kPiece;
  if (batch * big >= 512 || vocab > (int64_t)kMaxPieces * kSmall) return {false, big};
  return {true, (vocab + kSmall - 1) / kSmall};
}

template <typename T, int PIECE>
hipError_t launch_of(const VerifyArgs& a, int64_t pieces, double* sums, Found* founds, hipStream_t stream) {
  hipLaunchKernelGGL((verify_sums<T, PIECE>), dim3((unsigned)pieces, (unsigned)a.batch), dim3(kThreads), 0, stream,
                     a, sums, founds);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((verify_draw<T, PIECE>), dim3((unsigned)a.batch), dim3(kThreads), 0, stream, a, sums, founds,
                     (int)pieces);
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace_bytes(int64_t batch, int64_t vocab) {
  const VerifyPlan p = verify_plan(batch, vocab);
  const size_t sums = ((size_t)batch * p.pieces * 8 + 255) & ~size_t(255);
  return sums + (((size_t)batch * sizeof(Found) + 255) & ~size_t(255));
}

hipError_t launch_verify(const VerifyArgs& a, bool bf16, hipStream_t stream) {
  const VerifyPlan p = verify_plan(a.batch, a.vocab);
  double* sums = static_cast<double*>(a.workspace);
  Found* founds = reinterpret_cast<Found*>(static_cast<char*>(a.workspace) +
                                           (((size_t)a.batch * p.pieces * 8 + 255) & ~size_t(255)));
  if (bf16)
    return p.small ? launch_of<uint16_t, kSmall>(a, p.pieces, sums, founds, stream)
                   : launch_of<uint16_t, kPiece>(a, p.pieces, sums, founds, stream);
  return p.small ? launch_of<float, kSmall>(a, p.pieces, sums, founds, stream)
                 : launch_of<float, kPiece>(a, p.pieces, sums, founds, stream);
}

}  // namespace opq
