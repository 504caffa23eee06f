// Low-rank adapters of many requests beside one shared projection, and their
// gradients (include/opq_adapters.h).
//
// Everything is three products with a stack P [count][rank][d] (`down` with
// d = k, `up` with d = n), token t using its adapter i = index[t]:
//   shrink  c_t = P_i v_t              (rank sums over d: h from x, e from dy)
//   expand  o_t = b_t + s_i P_i^T c_t  (d sums over rank)
//   grad    dP_i = sum_t c_t v_t^T     (rank x d sums over the adapter's tokens)
//   forward   c = shrink(down, x);  out = expand(up, c) + y
//   backward  h = shrink(down, x), e = shrink(up, dy);  dx += expand(down, e),
//             d_down = grad(s e, x), d_up = grad(s h, dy)
// Both stacks keep d as the dense dimension, so that one kernel serves either
// side and every load of a stack, a token matrix or an output is of 16 bytes
// along d.  All run on v_mfma_f32_16x16x32_bf16; few operations per byte, so
// memory (and, for few tokens, latency) bounds them.
//
// Operands whose contraction runs along a strided dimension (expand: rank,
// grad: tokens) are transposed in registers: a lane loads an 8 x 8 block (8 rows
// of 16 bytes) and v_perm pairs rows, 32 of them for the eight operands of the
// eight columns; nothing goes through LDS.
//
// Tokens are grouped by adapter where they are used.  Forward, each workgroup
// sorts the (up to 256) tokens of its block in LDS, stably, into tiles of equal
// adapters; a call needs no plan and no launch for it.  A tile's columns are
// independent in the matrix product, so what is in another token's row never
// reaches a token.
//
// Rounding: c is float32.  Entering a second product it is cut into bfloat16
// parts: two (16 bits) where the result is bfloat16 itself, three (24 bits, all
// of it) where it is float32.  Parts are cut by truncation, so none overflows;
// the last one is rounded.
#include <algorithm>

#include "adapters_internal.hpp"
#include "device_common.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kBlockTokens = 256;  // tokens a workgroup sorts: one a thread
constexpr int kNone = 0x7FFFFFFE;  // sorts behind every adapter

// -------------------------------------------------------------- token tiles

// The block's tokens in the order of their adapters, cut into tiles of at most
// TILE tokens of one adapter.
template <int TILE>
struct Tiles {
  int id[kBlockTokens];
  uint16_t order[kBlockTokens];  // token (of the block) at each sorted place
  uint16_t first[kBlockTokens];  // sorted place of each tile's first token
  int adapter[kBlockTokens];     // adapter of each tile, or kNone
  uint8_t starts[kBlockTokens];
  int count;                     // tiles
  int same;
  int sums[kWaves];
  __device__ int size(int tile, int cnt) const {
    return (tile + 1 < count ? first[tile + 1] : cnt) - first[tile];
  }
};

template <int TILE>
__device__ __forceinline__ void make_tiles(Tiles<TILE>& s, const int32_t* index, int cnt, int64_t adapters) {
  const int t = threadIdx.x;
  int id = 0x7FFFFFFF;  // past the block: behind everything
  if (t < cnt) {
    id = index[t];
    if (id < 0 || id >= adapters) id = kNone;
  }
  s.id[t] = id;
  if (t == 0) s.same = 1;
  __syncthreads();
  if (t < cnt && id != s.id[0]) s.same = 0;
  __syncthreads();
  // place: tokens of lower adapters, and earlier ones of the same; rank: among the same
  int place = t, rank = t;
  if (!s.same) {
    place = rank = 0;
    for (int o = 0; o < cnt; ++o) {
      const int other = s.id[o];
      place += other < id;
      rank += other == id && o < t;
    }
    place += rank;
  }
  if (t < cnt) {
    s.order[place] = (uint16_t)t;
    s.starts[place] = rank % TILE == 0;
  }
  __syncthreads();
  const int lane = t & (kWave - 1), wave = t / kWave;
  const bool start = t < cnt && s.starts[t];
  const uint64_t mask = __ballot(start);
  if (lane == 0) s.sums[wave] = __popcll(mask);
  __syncthreads();
  int before = __popcll(mask & ((uint64_t(1) << lane) - 1));
  int total = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += s.sums[w];
    total += s.sums[w];
  }
  if (start) {
    s.first[before] = (uint16_t)t;
    s.adapter[before] = s.id[s.order[t]];
  }
  if (t == 0) s.count = total;
  __syncthreads();
}

// ------------------------------------------------------------------- helpers

__device__ __forceinline__ bf16x8_t operand(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }
__device__ __forceinline__ uint4 zero16() { return make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Eight rows of eight columns -> the eight columns, each of eight rows.
__device__ __forceinline__ void transpose8(const uint4 (&r)[8], uint4 (&c)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t a = q == 0 ? r[2 * t].x : q == 1 ? r[2 * t].y : q == 2 ? r[2 * t].z : r[2 * t].w;
      const uint32_t b = q == 0 ? r[2 * t + 1].x : q == 1 ? r[2 * t + 1].y : q == 2 ? r[2 * t + 1].z : r[2 * t + 1].w;
      lo[t] = __builtin_amdgcn_perm(b, a, 0x05040100u);
      hi[t] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
    c[2 * q] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    c[2 * q + 1] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

// v as a sum of PARTS bfloat16 values, the first ones cut off (an infinity or NaN is
// all in the first), the last one rounded.
template <int PARTS>
__device__ __forceinline__ void split(float v, uint32_t (&part)[PARTS]) {
  const bool finite = (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
#pragma unroll
  for (int p = 0; p < PARTS - 1; ++p) {
    uint32_t b = __float_as_uint(v) & 0xFFFF0000u;
    if (p == 0 && v != v) b = 0x7FC00000u;
    part[p] = b >> 16;
    v = finite ? v - __uint_as_float(b) : 0.0f;
  }
  part[PARTS - 1] = bf16_rne(v);
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 a = load16(static_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// A NaN stays one: bf16_rne is for numbers.
__device__ __forceinline__ uint32_t bf16_any(float f) { return f == f ? bf16_rne(f) : 0x7FC0u; }

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_any(v[2 * i]) | bf16_any(v[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// -------------------------------------------------------------------- shrink

struct ShrinkSide {
  const uint16_t* p;  // [count][rank][d]
  const uint16_t* v;  // [m][stride]
  int64_t stride;
  float* part;        // [slices][m][rank]
  int d, slices;
};
struct ShrinkArgs {
  ShrinkSide side[2];  // workgroups x < side[0].slices take the first, the rest the second
  const int32_t* index;
  int64_t m, count;
  int rank;
};

// Workgroup (slice of d, share of the block's tiles, block of tokens).  A wave
// takes every fourth 32-wide step of the slice for a tile of up to 32 tokens and
// all rank rows; the waves' sums meet in LDS, the slices' in the reader.
// RT: 16-row tiles of the rank.
template <int RT>
__global__ __launch_bounds__(kThreads) void lowrank_shrink(ShrinkArgs a) {
  constexpr int kTile = 32;
  constexpr int kDepth = RT >= 8 ? 1 : RT >= 4 ? 2 : 4;  // steps whose loads are out together
  __shared__ Tiles<kTile> s;
  __shared__ float s_red[kWaves * RT * 2 * 4 * kWave];
  const ShrinkSide& g = a.side[blockIdx.x >= (unsigned)a.side[0].slices];
  const int slice = blockIdx.x - (blockIdx.x >= (unsigned)a.side[0].slices ? a.side[0].slices : 0);
  const int64_t t0 = (int64_t)blockIdx.z * kBlockTokens;
  const int cnt = (int)min((int64_t)kBlockTokens, a.m - t0);
  make_tiles(s, a.index + t0, cnt, a.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int steps = (g.d + 31) / 32;
  const int per = (steps + g.slices - 1) / g.slices;
  const int begin = slice * per, end = min(steps, begin + per);

  for (int tile = blockIdx.y; tile < s.count; tile += gridDim.y) {
    const int id = s.adapter[tile];
    if (id == kNone) break;  // they come last
    const int size = s.size(tile, cnt), first = s.first[tile];
    const uint16_t* p = g.p + (int64_t)id * a.rank * g.d + q * 8;
    uint32_t row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = (uint32_t)min(i * 16 + c, a.rank - 1) * (uint32_t)g.d;
    const uint16_t* v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = g.v + (t0 + s.order[first + min(h * 16 + c, size - 1)]) * g.stride + q * 8;
    floatx4_t acc[2][RT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[h][i] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    auto walk = [&](auto halves) __attribute__((always_inline)) {
      constexpr int H = decltype(halves)::value;
      int at = begin + wave;
      auto some = [&](auto depth) __attribute__((always_inline)) {
        constexpr int D = decltype(depth)::value;
        uint4 vv[D][H], pp[D][RT];
#pragma unroll
        for (int u = 0; u < D; ++u) {
          const int e = (at + u * kWaves) * 32;
          const bool in = e + q * 8 < g.d;  // d is a multiple of 8
#pragma unroll
          for (int h = 0; h < H; ++h) vv[u][h] = in ? load16(v[h] + e) : zero16();
#pragma unroll
          for (int i = 0; i < RT; ++i) pp[u][i] = in ? load16(p + row[i] + e) : zero16();
        }
#pragma unroll
        for (int u = 0; u < D; ++u)
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < RT; ++i)
              acc[h][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(pp[u][i]), operand(vv[u][h]),
                                                                  acc[h][i], 0, 0, 0);
        at += D * kWaves;
      };
      while (at + (kDepth - 1) * kWaves < end) some(std::integral_constant<int, kDepth>{});
      while (at < end) some(std::integral_constant<int, 1>{});
    };
    if (size > 16) walk(std::integral_constant<int, 2>{});
    else walk(std::integral_constant<int, 1>{});

    // [wave][half][row tile][lane][4]
    float4* red = reinterpret_cast<float4*>(s_red);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < RT; ++i)
        red[((wave * 2 + h) * RT + i) * kWave + lane] =
            make_float4(acc[h][i][0], acc[h][i][1], acc[h][i][2], acc[h][i][3]);
    __syncthreads();
    for (int o = threadIdx.x; o < 2 * RT * kWave; o += kThreads) {
      const int ln = o % kWave, i = o / kWave % RT, h = o / kWave / RT;
      const int token = h * 16 + (ln & 15), r = i * 16 + (ln >> 4) * 4;  // rank is a multiple of 8
      if (token < size && r < a.rank) {
        float4 sum = red[o];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
          const float4 add = red[w * 2 * RT * kWave + o];
          sum.x += add.x; sum.y += add.y; sum.z += add.z; sum.w += add.w;
        }
        const int64_t t = t0 + s.order[first + token];
        *reinterpret_cast<float4*>(g.part + ((int64_t)slice * a.m + t) * a.rank + r) = sum;
      }
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------------- expand

struct ExpandArgs {
  const uint16_t* p;   // [count][rank][d]
  const float* scale;
  const float* part;   // [slices][m][rank]
  const int32_t* index;
  const void* base;    // [m][base_stride], or nullptr
  void* out;           // [m][out_stride]
  int64_t base_stride, out_stride, m, count;
  int rank, d, slices, block;  // block: tokens of a workgroup, <= kBlockTokens
};

// Workgroup (512 columns, share of the block's tiles, block of tokens), a wave
// 128 columns.  The tiles' operands (s c, in parts) are made once in LDS for the
// four waves, kMade tiles at a time.  Of lane (c, q) = (l % 16, l / 16) the
// stack's block is rank rows 32 s + 8 q ..., columns 8 pi(c) ... with pi(4 i + j)
// = 4 j + i: the accumulators of a lane are then, for i = 0..3, the eight columns
// 8 (4 i + q) ..., so that in a load or store of 16 bytes a token's four lanes
// touch 64 bytes in a row.
template <int RS, bool BASE_BF16, bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void lowrank_expand(ExpandArgs a) {
  constexpr int PARTS = OUT_BF16 ? 2 : 3;
  constexpr int kMade = RS * PARTS <= 4 ? 16 : RS * PARTS <= 8 ? 8 : 4;
  __shared__ Tiles<16> s;
  __shared__ uint4 s_c[kMade * RS * PARTS * kWave];
  const int64_t t0 = (int64_t)blockIdx.z * a.block;
  const int cnt = (int)min((int64_t)a.block, a.m - t0);
  make_tiles(s, a.index + t0, cnt, a.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 512 + wave * 128;
  const int mine = n0 + ((c & 3) * 4 + (c >> 2)) * 8;  // first column of the lane's block
  uint4 p[RS][8];
  int held = -1;  // adapter in p

  // this workgroup's tiles: consecutive ones, so that neighbours share an adapter
  const int share = (s.count + gridDim.y - 1) / gridDim.y;
  const int last = min(s.count, ((int)blockIdx.y + 1) * share);
  for (int from = blockIdx.y * share; from < last; from += kMade) {
    const int made = min(kMade, last - from);
    for (int w = wave; w < made * RS; w += kWaves) {
      const int tile = from + w / RS, rs = w % RS;
      const int id = s.adapter[tile];
      uint32_t cut[8][PARTS];
      float v[8] = {};
      const int r = rs * 32 + q * 8;
      if (id != kNone && c < s.size(tile, cnt) && r < a.rank) {
        const float* f = a.part + (t0 + s.order[s.first[tile] + c]) * a.rank + r;
        const int64_t plane = a.m * a.rank;
#pragma unroll 4
        for (int k = 0; k < a.slices; ++k) {
          float add[8];
          load8<false>(f, k * plane, add);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += add[e];
        }
        const float by = a.scale[id];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= by;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) split<PARTS>(v[e], cut[e]);
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
        s_c[(w * PARTS + k) * kWave + lane] =
            make_uint4(cut[0][k] | cut[1][k] << 16, cut[2][k] | cut[3][k] << 16,
                       cut[4][k] | cut[5][k] << 16, cut[6][k] | cut[7][k] << 16);
    }
    __syncthreads();
    for (int w = 0; w < made && n0 < a.d; ++w) {
      const int tile = from + w, id = __builtin_amdgcn_readfirstlane(s.adapter[tile]);
      const int size = s.size(tile, cnt);
      if (id == kNone && a.base == a.out) break;  // nothing to copy, and they come last
      if (id != held && id != kNone) {
        held = id;
#pragma unroll
        for (int k = 0; k < RS; ++k) {
          const int r = k * 32 + q * 8;
          const bool in = r < a.rank && mine < a.d;
          const uint16_t* at = a.p + ((int64_t)id * a.rank + r) * a.d + mine;
          uint4 rows[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) rows[e] = in ? load16(at + (int64_t)e * a.d) : zero16();
          transpose8(rows, p[k]);
        }
      }
      floatx4_t acc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
      if (id != kNone) {
#pragma unroll
        for (int k = 0; k < RS; ++k)
#pragma unroll
          for (int e = 0; e < PARTS; ++e) {
            const bf16x8_t h = operand(s_c[((w * RS + k) * PARTS + e) * kWave + lane]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(p[k][j]), h, acc[j], 0, 0, 0);
          }
      }
      if (c < size) {
        const int64_t t = t0 + s.order[s.first[tile] + c];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + (i * 4 + q) * 8;
          if (n < a.d) {
            float v[8] = {};
            if (a.base) load8<BASE_BF16>(a.base, t * a.base_stride + n, v);
            if (id != kNone) {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += acc[j][i];
            }
            store8<OUT_BF16>(a.out, t * a.out_stride + n, v);
          }
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ launches

// 16-row tiles of the rank, as an instance has them.
int rank_tiles(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

struct ShrinkPlan {
  int slices, shares;
  int64_t blocks;
};

// About 512 workgroups, as long as a wave has a step of its own; shares: workgroups
// over a block's tiles.  Both follow from m and d alone: the host does not know how
// many adapters a call meets.
ShrinkPlan shrink_plan(int64_t m, int64_t d) {
  ShrinkPlan p;
  m = std::max<int64_t>(m, 1);
  p.blocks = (m + kBlockTokens - 1) / kBlockTokens;
  p.shares = (int)(m > kBlockTokens ? 8 : std::min<int64_t>(m, 32));
  const int64_t steps = (d + 31) / 32;
  const int64_t want = (512 + p.blocks * p.shares - 1) / (p.blocks * p.shares);
  p.slices = (int)std::max<int64_t>(1, std::min<int64_t>({want, (steps + 3) / 4, 16}));
  const int64_t per = (steps + p.slices - 1) / p.slices;
  p.slices = (int)std::max<int64_t>(1, (steps + per - 1) / per);  // none without steps
  return p;
}

size_t up256(size_t b) { return (b + 255u) & ~size_t(255); }

hipError_t launch_shrink(const ShrinkArgs& a, const ShrinkPlan& plan, hipStream_t stream) {
  const dim3 grid((unsigned)(a.side[0].slices + a.side[1].slices), (unsigned)plan.shares, (unsigned)plan.blocks);
  switch (rank_tiles(a.rank)) {
    case 1: hipLaunchKernelGGL(lowrank_shrink<1>, grid, dim3(kThreads), 0, stream, a); break;
    case 2: hipLaunchKernelGGL(lowrank_shrink<2>, grid, dim3(kThreads), 0, stream, a); break;
    case 4: hipLaunchKernelGGL(lowrank_shrink<4>, grid, dim3(kThreads), 0, stream, a); break;
    default: hipLaunchKernelGGL(lowrank_shrink<8>, grid, dim3(kThreads), 0, stream, a); break;
  }
  return hipGetLastError();
}

template <int RS>
void launch_expand_of(const ExpandArgs& a, bool base_bf16, bool out_bf16, dim3 grid, hipStream_t stream) {
  if (base_bf16 && out_bf16)
    hipLaunchKernelGGL((lowrank_expand<RS, true, true>), grid, dim3(kThreads), 0, stream, a);
  else if (base_bf16)
    hipLaunchKernelGGL((lowrank_expand<RS, true, false>), grid, dim3(kThreads), 0, stream, a);
  else if (out_bf16)
    hipLaunchKernelGGL((lowrank_expand<RS, false, true>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((lowrank_expand<RS, false, false>), grid, dim3(kThreads), 0, stream, a);
}

hipError_t launch_expand(ExpandArgs a, bool base_bf16, bool out_bf16, hipStream_t stream) {
  a.block = a.m <= 256 ? 256 : 128;
  const int64_t shares = a.m > 256 ? 1 : std::min<int64_t>(a.m, 64);
  const dim3 grid((unsigned)((a.d + 511) / 512), (unsigned)shares, (unsigned)((a.m + a.block - 1) / a.block));
  if (a.rank <= 32) launch_expand_of<1>(a, base_bf16, out_bf16, grid, stream);
  else if (a.rank <= 64) launch_expand_of<2>(a, base_bf16, out_bf16, grid, stream);
  else launch_expand_of<4>(a, base_bf16, out_bf16, grid, stream);
  return hipGetLastError();
}

}  // namespace

size_t lowrank_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank) {
  (void)n;
  return up256((size_t)shrink_plan(m, k).slices * (size_t)m * (size_t)rank * 4u);
}

hipError_t launch_lowrank_add(const LowrankAdd& c, hipStream_t stream) {
  const ShrinkPlan plan = shrink_plan(c.m, c.a.k);
  ShrinkArgs s{};
  s.side[0] = {c.a.down, c.x, c.x_stride, static_cast<float*>(c.workspace), (int)c.a.k, plan.slices};
  s.index = c.index;
  s.m = c.m;
  s.count = c.a.count;
  s.rank = (int)c.a.rank;
  const hipError_t e = launch_shrink(s, plan, stream);
  if (e != hipSuccess) return e;
  ExpandArgs x{};
  x.p = c.a.up;
  x.scale = c.a.scale;
  x.part = static_cast<const float*>(c.workspace);
  x.index = c.index;
  x.base = c.y;
  x.out = c.out;
  x.base_stride = c.y_stride;
  x.out_stride = c.out_stride;
  x.m = c.m;
  x.count = c.a.count;
  x.rank = (int)c.a.rank;
  x.d = (int)c.a.n;
  x.slices = plan.slices;
  return launch_expand(x, c.y_bf16, c.out_bf16, stream);
}

// ------------------------------------------------------------------ backward

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;

// A backward pass' tokens in the order of their adapters, each adapter's from a multiple
// of 32 on, and the items of work: up to `seg` tokens of one adapter.  An adapter with one
// item has its gradient written by it; the items of the others leave theirs in
// slots, which are added in order.
struct GradPlan {
  int32_t* order;    // [cap] token at each place, -1 for padding
  int32_t* places;   // [1] places in use
  int32_t* items;    // [1] items
  int32_t* adapter;  // [item cap]
  int32_t* from;     // [item cap] first place
  int32_t* length;   // [item cap] tokens
  int32_t* slot;     // [item cap] slot, or -1
  int32_t* slots;    // [count][2] first slot and number of them; -1: a single item
};

struct PlanArgs {
  GradPlan g;
  const int32_t* index;
  int64_t m;
  int count, seg;
};

// One workgroup: a stable counting sort, every wave over a run of the tokens of its own.
__global__ __launch_bounds__(kPlanThreads) void lowrank_plan(PlanArgs a) {
  __shared__ int s_count[kPlanWaves * kMaxTrained];
  __shared__ int s_scan[3][kPlanWaves];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int i = tid; i < kPlanWaves * a.count; i += kPlanThreads) s_count[i] = 0;
  __syncthreads();
  const int64_t per = ((a.m + kPlanWaves - 1) / kPlanWaves + kWave - 1) / kWave * kWave;
  const int64_t begin = min(a.m, wave * per), end = min(a.m, begin + per);
  int* mine = s_count + wave * a.count;
  for (int64_t t = begin + lane; t < end; t += kWave) {
    const int id = a.index[t];
    if (id >= 0 && id < a.count) atomicAdd(mine + id, 1);
  }
  __syncthreads();
  // thread = adapter: the waves' counts become offsets in the adapter's run
  int total = 0;
  if (tid < a.count)
    for (int w = 0; w < kPlanWaves; ++w) {
      const int n = s_count[w * a.count + tid];
      s_count[w * a.count + tid] = total;
      total += n;
    }
  const int items = (total + a.seg - 1) / a.seg;
  int own[3] = {(total + 31) & ~31, items, items > 1 ? items : 0}, at[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int v = own[i];
    for (int off = 1; off < kWave; off <<= 1) {
      const int up = __shfl_up(v, off, kWave);
      if (lane >= off) v += up;
    }
    if (lane == kWave - 1) s_scan[i][wave] = v;
    at[i] = v - own[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (int w = 0; w < wave; ++w) at[i] += s_scan[i][w];
  if (tid == kPlanThreads - 1) {
    *a.g.places = at[0] + own[0];
    *a.g.items = at[1] + own[1];
  }
  if (tid < a.count) {
    a.g.slots[2 * tid] = items == 1 ? -1 : at[2];
    a.g.slots[2 * tid + 1] = own[2];
    for (int i = 0; i < items; ++i) {
      a.g.adapter[at[1] + i] = tid;
      a.g.from[at[1] + i] = at[0] + i * a.seg;
      a.g.length[at[1] + i] = min(a.seg, total - i * a.seg);
      a.g.slot[at[1] + i] = items > 1 ? at[2] + i : -1;
    }
    for (int i = total; i < own[0]; ++i) a.g.order[at[0] + i] = -1;
    for (int w = 0; w < kPlanWaves; ++w) s_count[w * a.count + tid] += at[0];
  }
  __syncthreads();
  for (int64_t t0 = begin; t0 < end; t0 += kWave) {
    const int64_t t = t0 + lane;
    int id = t < end ? a.index[t] : -1;
    if (id >= a.count) id = -1;
    uint64_t left = __ballot(id >= 0);
    while (left) {  // one turn an adapter met
      const int who = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
      const uint64_t same = __ballot(id == who);
      const int place = mine[who];
      if (id == who) a.g.order[place + __popcll(same & ((uint64_t(1) << lane) - 1))] = (int32_t)t;
      wave_lds_sync();
      if (lane == 0) mine[who] = place + __popcll(same);
      wave_lds_sync();
      left &= ~same;
    }
  }
}

struct OperandArgs {
  GradPlan g;
  const float* part[2];  // [slices][m][rank]
  int slices[2];
  uint16_t* out[2];      // [parts][rank][cap]
  const float* scale;
  const int32_t* index;
  int64_t m, cap;
  int rank;
};

// s c in bfloat16 parts, transposed: what the rows of grad's products read along the
// tokens.  A thread makes eight ranks of one place.
template <int PARTS>
__global__ __launch_bounds__(kThreads) void lowrank_operands(OperandArgs a) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= *a.g.places) return;
  const int side = blockIdx.z, r = blockIdx.y * 8;
  const int t = a.g.order[j];
  float v[8] = {};
  if (t >= 0) {
    const float* f = a.part[side] + (int64_t)t * a.rank + r;
    for (int k = 0; k < a.slices[side]; ++k) {
      float add[8];
      load8<false>(f, (int64_t)k * a.m * a.rank, add);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += add[e];
    }
    const float by = a.scale[a.index[t]];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= by;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t cut[PARTS];
    split<PARTS>(v[e], cut);
#pragma unroll
    for (int k = 0; k < PARTS; ++k)
      a.out[side][((int64_t)k * a.rank + r + e) * a.cap + j] = (uint16_t)cut[k];
  }
}

struct GradSide {
  const uint16_t* v;  // [m][stride]
  const uint16_t* c;  // [parts][rank][cap]
  int64_t stride;
  float* part;        // [slots][rank][d]
  void* out;          // [count][rank][d]
  int d, blocks;
};
struct GradArgs {
  GradPlan g;
  GradSide side[2];  // workgroups x < side[0].blocks take the first, the rest the second
  int64_t cap;
  int rank;
};

// Workgroup (512 columns, item, 64 rows of the rank), a wave 128 columns: lane (c, q) holds
// columns 8 c ... of eight tokens, 8 q ... of each 32, and after the transposition is column
// 8 c + j of the j-th product.  RT: 16-row tiles of the rank, at most 4 (rank 128 takes two
// workgroups, by registers).
template <int RT, bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void lowrank_grad(GradArgs a) {
  constexpr int PARTS = OUT_BF16 ? 2 : 3;
  const int item = blockIdx.y;
  if (item >= *a.g.items) return;
  const bool second = blockIdx.x >= (unsigned)a.side[0].blocks;
  const GradSide& g = a.side[second];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int n0 = ((int)blockIdx.x - (second ? a.side[0].blocks : 0)) * 512 + wave * 128;
  if (n0 >= g.d) return;
  const int n = n0 + c * 8, r0 = blockIdx.z * 64;
  const int from = a.g.from[item], length = a.g.length[item];
  const uint16_t* v = g.v + (n < g.d ? n : 0);
  const uint16_t* row[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) row[i] = g.c + (int64_t)min(r0 + i * 16 + c, a.rank - 1) * a.cap + from + q * 8;
  floatx4_t acc[RT][8];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  for (int at = 0; at < length; at += 32) {
    const int4* o = reinterpret_cast<const int4*>(a.g.order + from + at + q * 8);
    const int4 o0 = o[0], o1 = o[1];
    const int t[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
    uint4 rows[8], cols[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rows[e] = t[e] >= 0 ? load16(v + t[e] * g.stride) : zero16();
    bf16x8_t h[RT][PARTS];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int k = 0; k < PARTS; ++k) h[i][k] = operand(load16(row[i] + (int64_t)k * a.rank * a.cap + at));
    transpose8(rows, cols);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h[i][k], operand(cols[j]), acc[i][j], 0, 0, 0);
  }
  if (n >= g.d) return;
  const int slot = a.g.slot[item];
  const int64_t first = slot < 0 ? (int64_t)a.g.adapter[item] * a.rank : (int64_t)slot * a.rank;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + i * 16 + q * 4 + e;
      if (r < a.rank) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = acc[i][j][e];
        const int64_t to = (first + r) * g.d + n;
        if (slot < 0) store8<OUT_BF16>(g.out, to, w);
        else store8<false>(g.part, to, w);
      }
    }
}

struct JoinArgs {
  const int32_t* slots;  // [count][2]
  const float* part[2];
  void* out[2];
  int64_t size[2];       // rank * d
};

// The slots of an adapter's items added in order; zeros for an adapter without tokens.
template <bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void lowrank_join(JoinArgs a) {
  const int id = blockIdx.y, side = blockIdx.z;
  const int first = a.slots[2 * id], count = a.slots[2 * id + 1];
  if (first < 0) return;
  const int64_t size = a.size[side];
  for (int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; at < size;
       at += (int64_t)gridDim.x * kThreads * 8) {
    float v[8] = {};
    for (int s = 0; s < count; ++s) {
      float add[8];
      load8<false>(a.part[side], (first + s) * size + at, add);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += add[e];
    }
    store8<OUT_BF16>(a.out[side], id * size + at, v);
  }
}

struct BackwardPlan {
  ShrinkPlan h, e;
  int64_t cap, items, slots;
  int seg;
  size_t part_h, part_e, operand_h, operand_e, sums_down, sums_up, lists, bytes;
};

BackwardPlan backward_plan(int64_t m, int64_t k, int64_t n, int64_t rank, int64_t count) {
  BackwardPlan b{};
  b.h = shrink_plan(m, k);
  b.e = shrink_plan(m, n);
  // about 2048 waves in grad, each of at least 32 tokens
  const int64_t columns = (k + 127) / 128 + (n + 127) / 128;
  const int64_t seg = (m * columns / 2048 + 31) / 32 * 32;
  b.seg = (int)std::max<int64_t>(32, seg);
  const int64_t met = std::min(m, count);
  b.cap = (m + 32 * met + 63) / 64 * 64;
  b.items = (m + b.seg - 1) / b.seg + met;
  // an adapter of q > 1 items has more than (q - 1) seg tokens, and q <= 2 (q - 1)
  b.slots = 2 * (m / b.seg);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  b.part_h = take((size_t)b.h.slices * m * rank * 4);
  b.part_e = take((size_t)b.e.slices * m * rank * 4);
  b.operand_h = take((size_t)3 * rank * b.cap * 2);
  b.operand_e = take((size_t)3 * rank * b.cap * 2);
  b.sums_down = take((size_t)b.slots * rank * k * 4);
  b.sums_up = take((size_t)b.slots * rank * n * 4);
  b.lists = take((size_t)(b.cap + 64 + 4 * b.items + 2 * count) * 4);
  b.bytes = at;
  return b;
}

template <int RT>
void launch_grad_of(const GradArgs& g, bool bf16, dim3 grid, hipStream_t stream) {
  if (bf16) hipLaunchKernelGGL((lowrank_grad<RT, true>), grid, dim3(kThreads), 0, stream, g);
  else hipLaunchKernelGGL((lowrank_grad<RT, false>), grid, dim3(kThreads), 0, stream, g);
}

}  // namespace

size_t lowrank_backward_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank, int64_t count) {
  return backward_plan(m, k, n, rank, count).bytes;
}

hipError_t launch_lowrank_backward(const LowrankBackward& c, hipStream_t stream) {
  const int64_t k = c.a.k, n = c.a.n, rank = c.a.rank;
  const BackwardPlan b = backward_plan(c.m, k, n, rank, c.a.count);
  char* ws = static_cast<char*>(c.workspace);
  float* part_h = reinterpret_cast<float*>(ws + b.part_h);
  float* part_e = reinterpret_cast<float*>(ws + b.part_e);
  const bool grads = c.d_down != nullptr;
  hipError_t err;

  ShrinkArgs s{};
  const ShrinkSide down{c.a.down, c.x, c.x_stride, part_h, (int)k, b.h.slices};
  const ShrinkSide up{c.a.up, c.dy, c.dy_stride, part_e, (int)n, b.e.slices};
  s.side[0] = up;
  if (grads) s.side[1] = down;
  s.index = c.index;
  s.m = c.m;
  s.count = c.a.count;
  s.rank = (int)rank;
  if (c.m > 0 && (err = launch_shrink(s, b.e, stream)) != hipSuccess) return err;

  if (c.dx_out) {
    ExpandArgs x{};
    x.p = c.a.down;
    x.scale = c.a.scale;
    x.part = part_e;
    x.index = c.index;
    x.base = c.dx;
    x.out = c.dx_out;
    x.base_stride = c.dx_stride;
    x.out_stride = c.dx_out_stride;
    x.m = c.m;
    x.count = c.a.count;
    x.rank = (int)rank;
    x.d = (int)k;
    x.slices = b.e.slices;
    if ((err = launch_expand(x, c.dx_bf16, c.dx_bf16, stream)) != hipSuccess) return err;
  }
  if (!grads) return hipSuccess;

  GradPlan g;
  int32_t* list = reinterpret_cast<int32_t*>(ws + b.lists);
  g.order = list;
  g.places = list + b.cap;
  g.items = g.places + 1;
  g.adapter = list + b.cap + 64;
  g.from = g.adapter + b.items;
  g.length = g.from + b.items;
  g.slot = g.length + b.items;
  g.slots = g.slot + b.items;
  PlanArgs p{g, c.index, c.m, (int)c.a.count, b.seg};
  hipLaunchKernelGGL(lowrank_plan, dim3(1), dim3(kPlanThreads), 0, stream, p);
  if ((err = hipGetLastError()) != hipSuccess) return err;

  OperandArgs o{};
  o.g = g;
  o.part[0] = part_e;
  o.part[1] = part_h;
  o.slices[0] = b.e.slices;
  o.slices[1] = b.h.slices;
  o.out[0] = reinterpret_cast<uint16_t*>(ws + b.operand_e);
  o.out[1] = reinterpret_cast<uint16_t*>(ws + b.operand_h);
  o.scale = c.a.scale;
  o.index = c.index;
  o.m = c.m;
  o.cap = b.cap;
  o.rank = (int)rank;
  // no tokens: no places and no items, and the join below writes zeros
  const dim3 og((unsigned)((b.cap + kThreads - 1) / kThreads), (unsigned)(rank / 8), 2);
  if (c.m > 0) {
    if (c.grad_bf16) hipLaunchKernelGGL(lowrank_operands<2>, og, dim3(kThreads), 0, stream, o);
    else hipLaunchKernelGGL(lowrank_operands<3>, og, dim3(kThreads), 0, stream, o);
  }
  if ((err = hipGetLastError()) != hipSuccess) return err;

  GradArgs ga{};
  ga.g = g;
  ga.side[0] = {c.x, o.out[0], c.x_stride, reinterpret_cast<float*>(ws + b.sums_down), c.d_down, (int)k,
                (int)((k + 511) / 512)};
  ga.side[1] = {c.dy, o.out[1], c.dy_stride, reinterpret_cast<float*>(ws + b.sums_up), c.d_up, (int)n,
                (int)((n + 511) / 512)};
  ga.cap = b.cap;
  ga.rank = (int)rank;
  const dim3 gg((unsigned)(ga.side[0].blocks + ga.side[1].blocks), (unsigned)b.items, (unsigned)(rank > 64 ? 2 : 1));
  if (c.m == 0) {
  } else if (rank <= 16) launch_grad_of<1>(ga, c.grad_bf16, gg, stream);
  else if (rank <= 32) launch_grad_of<2>(ga, c.grad_bf16, gg, stream);
  else launch_grad_of<4>(ga, c.grad_bf16, gg, stream);
  if ((err = hipGetLastError()) != hipSuccess) return err;

  JoinArgs j{};
  j.slots = g.slots;
  j.part[0] = ga.side[0].part;
  j.part[1] = ga.side[1].part;
  j.out[0] = c.d_down;
  j.out[1] = c.d_up;
  j.size[0] = rank * k;
  j.size[1] = rank * n;
  const int64_t widest = std::max(j.size[0], j.size[1]);
  const dim3 jg((unsigned)std::min<int64_t>((widest / 8 + kThreads - 1) / kThreads, 1024), (unsigned)c.a.count, 2);
  if (c.grad_bf16) hipLaunchKernelGGL(lowrank_join<true>, jg, dim3(kThreads), 0, stream, j);
  else hipLaunchKernelGGL(lowrank_join<false>, jg, dim3(kThreads), 0, stream, j);
  return hipGetLastError();
}

}  // namespace opq
