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
// Tokens are grouped by adapter where they are used: each wave looks at the 64
// tokens of its block, one a lane, and finds tiles of equal adapters with ballots, in
// registers; a forward call needs no plan, no launch and no barrier for it.  A tile's
// columns are independent in the matrix product, so what is in another token's row
// never reaches a token.
//
// Rounding: c is float32.  Entering a second product it is cut into three bfloat16
// parts, all of its 24 bits, whatever the result's type: a bfloat16 result is the float32
// one rounded.  (With two parts, 16 bits: 4096 tokens, 3840 -> 20480, rank 64 99 us for
// 102; one token, rank 8 7.7 for 8.0; gradients of one adapter 77 for 77.6.)  Parts are
// cut by truncation, so none overflows; the last one is rounded.  A later part may be zero where
// c is not, and zero times an infinite weight or gradient is NaN.  A sum that comes out NaN
// has an infinity or NaN among its operands, so the definition makes it one too, and
// the first parts alone, which have c's sign, say which: such sums are made of those.
#include <algorithm>

#include "adapters_internal.hpp"
#include "device_common.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kBlockTokens = kWave;  // tokens a wave groups: one a lane
constexpr int kNoAdapter = -1, kNoToken = -2;
constexpr int kCuts = 3;  // bfloat16 parts of a float32

// -------------------------------------------------------------- token tiles

// The adapter of the block's token `lane`.
__device__ __forceinline__ int block_id(const int32_t* index, int cnt, int64_t adapters) {
  const int lane = threadIdx.x & (kWave - 1);
  if (lane >= cnt) return kNoToken;
  const int id = index[lane];
  return id >= 0 && id < adapters ? id : kNoAdapter;
}

__device__ __forceinline__ uint64_t below(int lane) { return (uint64_t(1) << lane) - 1; }
__device__ __forceinline__ int first_of(uint64_t mask) { return __ffsll((unsigned long long)mask) - 1; }

// Tokens that lead a tile: every TILE-th of an adapter's.
template <int TILE>
__device__ __forceinline__ uint64_t leaders(int id, int lowest) {
  const int lane = threadIdx.x & (kWave - 1);
  uint64_t left = __ballot(id >= lowest), lead = 0;
  while (left) {  // a turn an adapter
    const int who = __builtin_amdgcn_readlane(id, first_of(left));
    const uint64_t same = __ballot(id == who);
    lead |= __ballot(id == who && __popcll(same & below(lane)) % TILE == 0);
    left &= ~same;
  }
  return lead;
}

struct Tile {
  int id, size;
  int token;  // of lane s: the tile's s-th token
};

template <int TILE>
__device__ __forceinline__ bool leads(int id, int lane) {
  const int who = __builtin_amdgcn_readlane(id, lane);
  return __popcll(__ballot(id == who) & below(lane)) % TILE == 0;
}

template <int TILE>
__device__ __forceinline__ Tile tile_of(int id, int leader) {
  const int lane = threadIdx.x & (kWave - 1);
  Tile t;
  t.id = __builtin_amdgcn_readlane(id, leader);
  const uint64_t same = __ballot(id == t.id);
  const int before = __popcll(same & below(leader));
  t.size = min(TILE, __popcll(same) - before);
  const int place = __popcll(same & below(lane)) - before;
  const bool in = id == t.id && place >= 0 && place < TILE;
  // Every lane sends its number to its place, those outside the tile to the last lane, which is
  // asked only for a tile of all 64: then none is outside.
  t.token = __builtin_amdgcn_ds_permute((in ? place : kWave - 1) * 4, lane);
  return t;
}

// ------------------------------------------------------------------- helpers

__device__ __forceinline__ bf16x8_t operand(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }
__device__ __forceinline__ uint4 zero16() { return make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Rows are loaded as memory wants them: lane l has chunk l % 4 (16 bytes) of row l / 4, four lanes
// 64 bytes in a row.  (The matrix operands' own order, rows in neighbouring lanes, makes
// every lane an access of its own: 64 a load, which bound these kernels at a quarter of
// L1's rate.)  This moves them to the operands' order: lane (c, q) gets chunk q of row c.
__device__ __forceinline__ uint4 to_operand(uint4 v) {
  const int lane = threadIdx.x & (kWave - 1);
  const int from = ((lane & 15) * 4 + (lane >> 4)) * 4;
  return make_uint4((uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.x), (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.y),
                    (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.z), (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)v.w));
}

// Whether a sum of the wave's may be NaN (it is one, or two are opposite infinities).
__device__ __forceinline__ bool some_nan(const floatx4_t (&acc)[8]) {
  float all = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) all += (acc[j][0] + acc[j][1]) + (acc[j][2] + acc[j][3]);
  return __ballot(all != all);
}

// NaN in sums replaced by what `first` gives for operand j, the product of the first parts.
template <typename F>
__device__ __forceinline__ void mend(floatx4_t (&acc)[8], F first) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const floatx4_t by = first(j);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = acc[j][i] != acc[j][i] ? by[i] : acc[j][i];
    __builtin_amdgcn_sched_barrier(0);  // rarely run: registers count here, not time
  }
}

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

// v as a sum of bfloat16 values, the first ones cut off (an infinity or NaN is all in
// the first), the last one rounded.
__device__ __forceinline__ void split(float v, uint32_t (&part)[kCuts]) {
  const bool finite = (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
#pragma unroll
  for (int p = 0; p < kCuts - 1; ++p) {
    uint32_t b = __float_as_uint(v) & 0xFFFF0000u;
    if (p == 0 && v != v) b = 0x7FC00000u;
    part[p] = b >> 16;
    v = finite ? v - __uint_as_float(b) : 0.0f;
  }
  part[kCuts - 1] = bf16_rne(v);
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

// Two values rounded to bfloat16 (nearest even; a NaN stays one), by one instruction of this part.
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{a, b}), bf16x2_t));
}

// Sixteen bytes read or written once (STREAM: around the caches' other contents).
template <bool STREAM>
__device__ __forceinline__ uint4 load_once(const char* p) {
  const u32x4_t* v = reinterpret_cast<const u32x4_t*>(p);
  if constexpr (STREAM) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(v));
  return __builtin_bit_cast(uint4, *v);
}
template <bool STREAM>
__device__ __forceinline__ void store_once(void* p, u32x4_t v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<u32x4_t*>(p));
  else *static_cast<u32x4_t*>(p) = v;
}

template <bool BF16, bool STREAM>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    store_once<STREAM>(static_cast<uint16_t*>(p) + at, u32x4_t{w[0], w[1], w[2], w[3]});
  } else {
    float* f = static_cast<float*>(p) + at;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      store_once<STREAM>(f + 4 * i, u32x4_t{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                            __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])});
  }
}

// -------------------------------------------------------------- training's plan

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

template <int W> constexpr int plan_bytes() { return (W * (int)kMaxTrained + 3 * W) * 4; }

// One workgroup of W waves: a stable counting sort, every wave over a run of the tokens of its own.
template <int W>
__device__ void plan_tokens(const PlanArgs& a, int* s) {
  constexpr int kWaves = W, kThreads = W * kWave;
  constexpr int kPlanAdapters = (int)kMaxTrained / kThreads;  // adapters of a thread
  constexpr int kAhead = 8;  // vectors of 64 tokens requested together
  int* s_scan = s + kWaves * kMaxTrained;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  for (int i = tid; i < kWaves * a.count; i += kThreads) s[i] = 0;
  __syncthreads();
  const int64_t per = ((a.m + kWaves - 1) / kWaves + kWave - 1) / kWave * kWave;
  const int64_t begin = min(a.m, wave * per), end = min(a.m, begin + per);
  int* mine = s + wave * a.count;
  auto each = [&](auto&& what) __attribute__((always_inline)) {
    for (int64_t t0 = begin; t0 < end; t0 += kAhead * kWave) {
      int id[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t t = t0 + i * kWave + lane;
        id[i] = a.index[min(t, end - 1)];
        if (t >= end || id[i] >= a.count) id[i] = -1;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        uint64_t left = __ballot(id[i] >= 0);
        while (left) {  // a turn an adapter met
          const int who = __builtin_amdgcn_readlane(id[i], first_of(left));
          const uint64_t same = __ballot(id[i] == who);
          what(t0 + i * kWave + lane, who, id[i] == who, same);
          left &= ~same;
        }
      }
    }
  };
  each([&](int64_t, int who, bool, uint64_t same) __attribute__((always_inline)) {
    if (lane == 0) mine[who] += __popcll(same);
  });
  __syncthreads();
  // the thread's adapters: the waves' counts become offsets in an adapter's run
  int total[kPlanAdapters], own[3] = {0, 0, 0}, at[3];
#pragma unroll
  for (int i = 0; i < kPlanAdapters; ++i) {
    const int id = tid * kPlanAdapters + i;
    total[i] = 0;
    if (id < a.count)
      for (int w = 0; w < kWaves; ++w) {
        const int n = s[w * a.count + id];
        s[w * a.count + id] = total[i];
        total[i] += n;
      }
    const int items = (total[i] + a.seg - 1) / a.seg;
    own[0] += (total[i] + 31) & ~31;
    own[1] += items;
    own[2] += items > 1 ? items : 0;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int v = own[i];
    for (int off = 1; off < kWave; off <<= 1) {
      const int up = __shfl_up(v, off, kWave);
      if (lane >= off) v += up;
    }
    if (lane == kWave - 1) s_scan[i * kWaves + wave] = v;
    at[i] = v - own[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (int w = 0; w < wave; ++w) at[i] += s_scan[i * kWaves + w];
  if (tid == kThreads - 1) {
    *a.g.places = at[0] + own[0];
    *a.g.items = at[1] + own[1];
  }
#pragma unroll
  for (int k = 0; k < kPlanAdapters; ++k) {
    const int id = tid * kPlanAdapters + k;
    if (id >= a.count) break;
    const int items = (total[k] + a.seg - 1) / a.seg, padded = (total[k] + 31) & ~31;
    a.g.slots[2 * id] = items == 1 ? -1 : at[2];
    a.g.slots[2 * id + 1] = items > 1 ? items : 0;
    for (int i = 0; i < items; ++i) {
      a.g.adapter[at[1] + i] = id;
      a.g.from[at[1] + i] = at[0] + i * a.seg;
      a.g.length[at[1] + i] = min(a.seg, total[k] - i * a.seg);
      a.g.slot[at[1] + i] = items > 1 ? at[2] + i : -1;
    }
    for (int i = total[k]; i < padded; ++i) a.g.order[at[0] + i] = -1;
    for (int w = 0; w < kWaves; ++w) s[w * a.count + id] += at[0];
    at[0] += padded;
    at[1] += items;
    at[2] += items > 1 ? items : 0;
  }
  __syncthreads();
  each([&](int64_t t, int who, bool in, uint64_t same) __attribute__((always_inline)) {
    const int place = mine[who];
    if (in) a.g.order[place + __popcll(same & below(lane))] = (int32_t)t;
    wave_lds_sync();
    if (lane == 0) mine[who] = place + __popcll(same);
    wave_lds_sync();
  });
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
  bool single;  // workgroup y takes the tile that token y leads, if it leads one
};

// Tokens of a shrink's tile.  Each tile reads the adapter's rows, mostly from L2: past rank 32
// that costs more than the fewer workgroups of larger tiles do.
constexpr int shrink_tile(int64_t rank) { return rank > 32 ? kBlockTokens : kBlockTokens / 2; }

// Workgroup (slice of d, share of the block's tiles, block of tokens).  A wave
// takes its share of the slice's 32-wide steps for a tile, all tokens of the block that use
// one adapter, and all rank rows; the waves' sums meet in LDS, the slices' in the
// reader.  (The two sides of 4096 tokens, 3840 -> 11520, rank 16: 33 us, where reading the
// tokens alone takes 27.)
// RT: 16-row tiles of the rank.  PLAN: the workgroup past the slices sorts the tokens for
// the gradients, which wait for this launch anyway (9 us as a launch of its own).
template <int RT, int W, bool PLAN>
__global__ __launch_bounds__(W * kWave) void lowrank_shrink(ShrinkArgs a, PlanArgs plan) {
  constexpr int kWaves = W;
  constexpr int kTile = shrink_tile(RT * 16), kParts = kTile / 16;
  constexpr int kDepth = RT >= 8 ? 1 : RT >= 4 ? 2 : 4;  // steps whose loads are out together
  constexpr int kSums = kWaves * RT * 2 * 4 * kWave;
  __shared__ float s_red[PLAN && kSums * 4 < plan_bytes<W>() ? plan_bytes<W>() / 4 : kSums];
  if (PLAN && (int)blockIdx.x == a.side[0].slices + a.side[1].slices) {
    if (blockIdx.y == 0 && blockIdx.z == 0) plan_tokens<W>(plan, reinterpret_cast<int*>(s_red));
    return;
  }
  const bool second = (int)blockIdx.x >= a.side[0].slices;
  const ShrinkSide& g = a.side[second];
  const int slice = blockIdx.x - (second ? a.side[0].slices : 0);
  const int64_t t0 = (int64_t)blockIdx.z * kBlockTokens;
  const int id = block_id(a.index + t0, (int)min((int64_t)kBlockTokens, a.m - t0), a.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int lr = lane >> 2, lc = lane & 3;  // row and 16-byte chunk of a load
  uint64_t lead;
  if (a.single) {
    if (__builtin_amdgcn_readlane(id, blockIdx.y) < 0 || !leads<kTile>(id, blockIdx.y)) return;
    lead = uint64_t(1) << blockIdx.y;
  } else {
    lead = leaders<kTile>(id, 0);
    for (unsigned i = 0; i < blockIdx.y; ++i) lead &= lead - 1;  // tiles y, y + shares, ...
  }
  const int whole = g.d / 32, steps = (g.d + 31) / 32;
  const int per = (steps + g.slices - 1) / g.slices;
  const int begin = slice * per, end = min(steps, begin + per);
  const int run = per >= kWaves * kDepth ? kDepth : 1;

  while (lead) {
    const Tile tile = tile_of<kTile>(id, first_of(lead));
    for (unsigned i = 0; i < gridDim.y; ++i) lead &= lead - 1;
    if (a.single) lead = 0;
    const uint16_t* p = g.p + (int64_t)tile.id * a.rank * g.d;
    uint32_t row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) row[i] = (uint32_t)min(i * 16 + lr, a.rank - 1) * (uint32_t)g.d;
    const uint16_t* v[kParts];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      v[h] = g.v + (t0 + __shfl(tile.token, min(h * 16 + lr, tile.size - 1), kWave)) * g.stride;
    floatx4_t acc[kParts][RT];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[h][i] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    auto walk = [&](auto parts) __attribute__((always_inline)) {
      constexpr int H = decltype(parts)::value;  // sixteenths of tokens
      // a wave takes runs of steps, so that it reads up to 256 bytes of a row in a row
      auto some = [&](int at, auto depth, bool full) __attribute__((always_inline)) {
        constexpr int D = decltype(depth)::value;
        uint4 vv[D][H], pp[D][RT];
#pragma unroll
        for (int u = 0; u < D; ++u) {
          const int e = (at + u) * 32 + lc * 8;
          const bool in = full || e < g.d;  // d is a multiple of 8
          const int col = in ? e : 0;       // past d the row's first columns are read, and dropped
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const uint4 x = load16(v[h] + col);
            vv[u][h] = in ? x : zero16();
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const uint4 x = load16(p + row[i] + col);
            pp[u][i] = in ? x : zero16();
          }
        }
#pragma unroll
        for (int u = 0; u < D; ++u) {
#pragma unroll
          for (int h = 0; h < H; ++h) vv[u][h] = to_operand(vv[u][h]);
#pragma unroll
          for (int i = 0; i < RT; ++i) pp[u][i] = to_operand(pp[u][i]);
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < RT; ++i)
              acc[h][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(pp[u][i]), operand(vv[u][h]),
                                                                  acc[h][i], 0, 0, 0);
        }
      };
      // Whole runs first, then what is left, as two loops.  (As two branches of one they made the
      // compiler copy the sums from turn to turn, for ranks up to 16 five wait states behind the
      // matrix instruction that writes them, where eight are needed: it copied what was there before.)
      const int stop = min(end, whole);
      int at = begin + wave * run;
      if (run == kDepth)
        for (; at + kDepth <= stop; at += kWaves * kDepth) some(at, std::integral_constant<int, kDepth>{}, true);
      for (; at < end; at += kWaves * run)
        for (int u = at; u < min(end, at + run); ++u) some(u, std::integral_constant<int, 1>{}, u < whole);
    };
    if (kParts > 2 && tile.size > 32) walk(std::integral_constant<int, kParts>{});
    else if (tile.size > 16) walk(std::integral_constant<int, 2>{});
    else walk(std::integral_constant<int, 1>{});

    // [wave][part of two][row tile][lane][4]
    float4* red = reinterpret_cast<float4*>(s_red);
#pragma unroll
    for (int two = 0; two < kParts; two += 2) {
      if (two * 16 >= tile.size) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          red[((wave * 2 + h) * RT + i) * kWave + lane] = make_float4(
              acc[two + h][i][0], acc[two + h][i][1], acc[two + h][i][2], acc[two + h][i][3]);
      __syncthreads();
      for (int o = wave; o < 2 * RT; o += kWaves) {
        const int i = o % RT, h = o / RT;
        const int token = (two + h) * 16 + c, r = i * 16 + q * 4;  // rank is a multiple of 8
        const int64_t t = t0 + __shfl(tile.token, token, kWave);
        if (token < tile.size && r < a.rank) {
          float4 sum = red[o * kWave + lane];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) {
            const float4 add = red[(w * 2 * RT + o) * kWave + lane];
            sum.x += add.x; sum.y += add.y; sum.z += add.z; sum.w += add.w;
          }
          *reinterpret_cast<float4*>(g.part + ((int64_t)slice * a.m + t) * a.rank + r) = sum;
        }
      }
      __syncthreads();
    }
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
  int rank, d, slices;
};

// Eight sums of the slices of c, in order, times the adapter's scale: the loads of four
// slices are out together.
__device__ __forceinline__ void scaled(const float* part, int64_t plane, int slices, float by, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
  for (int k = 0; k < slices; k += 4) {
    float add[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) load8<false>(part, min(k + i, slices - 1) * plane, add[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += k + i < slices ? add[i][e] : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= by;
}

// What a lane adds to of one tile: eight columns of four tokens, as they are stored.
template <bool BF16> struct Base { uint4 v[BF16 ? 4 : 8]; };

template <bool BF16>
__device__ __forceinline__ void unpack(const Base<BF16>& b, int i, float (&v)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {b.v[i].x, b.v[i].y, b.v[i].z, b.v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 a = b.v[2 * i + k];
      v[4 * k] = __uint_as_float(a.x);
      v[4 * k + 1] = __uint_as_float(a.y);
      v[4 * k + 2] = __uint_as_float(a.z);
      v[4 * k + 3] = __uint_as_float(a.w);
    }
  }
}

constexpr int kMade = 4;  // tiles whose operands are in LDS together: one a wave
template <int RS>
struct ExpandShared {
  uint4 c[kMade][RS][kCuts][kWave];
};

// Workgroup (512 columns, share of the block's tiles, block of tokens), a wave
// 128 columns.  The tiles' operands (s c, in parts) are made once in LDS, a tile a wave,
// for the four waves.  Lane (c, q) = (l % 16, l / 16) loads rank rows 32 s + 8 q ... of
// columns 8 c ..., which after the transposition are the product's j-th columns 8 c + j;
// tokens are its rows, so a lane's accumulators are eight columns in a row of four tokens,
// and in every load and store sixteen lanes touch 256 bytes in a row.  What the tiles add
// to is requested with the stack's block before the operands are made.  It and the result
// pass the caches by, which are for the stack and c (4096 tokens, 3840 -> 20480, rank 64:
// 113 us with ordinary loads and stores, 103 so); one block of tokens is small enough for both.
template <int RS, bool BASE_BF16, bool OUT_BF16, bool SINGLE>
__device__ __forceinline__ void expand(const ExpandArgs& a, ExpandShared<RS>& s, int bx, int by, int bz) {
  constexpr int kAhead = SINGLE ? 1 : RS > 1 && BASE_BF16 ? 4 : 2;  // by registers
  const int64_t t0 = (int64_t)bz * kBlockTokens;
  const int id = block_id(a.index + t0, (int)min((int64_t)kBlockTokens, a.m - t0), a.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int lowest = a.base == a.out ? 0 : kNoAdapter;  // in place, tokens without an adapter are done
  uint64_t lead;
  if constexpr (SINGLE) {
    if (__builtin_amdgcn_readlane(id, by) < lowest || !leads<16>(id, by)) return;
    lead = uint64_t(1) << by;
  } else {
    lead = leaders<16>(id, lowest);
  }
  const int n0 = bx * 512 + wave * 128;
  const int mine = n0 + c * 8;  // the lane's first column
  const int64_t plane = a.m * a.rank;
  uint4 p[RS][8];
  int held = kNoToken;  // adapter in p

  auto load_p = [&](int who) __attribute__((always_inline)) {
    if (who == held || who < 0) return;
    held = who;
#pragma unroll
    for (int k = 0; k < RS; ++k) {
      const int r = k * 32 + q * 8;
      const bool in = r < a.rank && mine < a.d;
      const uint16_t* at = a.p + ((int64_t)who * a.rank + r) * a.d + mine;
      uint4 rows[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) rows[e] = in ? load16(at + (int64_t)e * a.d) : zero16();
      transpose8(rows, p[k]);
    }
  };
  // places past d or the tile read the first place of a token of it
  auto load_base = [&](const Tile& t, Base<BASE_BF16>& b) __attribute__((always_inline)) {
    const int n = mine < a.d ? mine : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t token = t0 + __shfl(t.token, min(q * 4 + i, t.size - 1), kWave);
      const char* from = static_cast<const char*>(a.base) + (token * a.base_stride + n) * (BASE_BF16 ? 2 : 4);
      if constexpr (BASE_BF16) {
        b.v[i] = load_once<!SINGLE>(from);
      } else {
        b.v[2 * i] = load_once<!SINGLE>(from);
        b.v[2 * i + 1] = load_once<!SINGLE>(from + 16);
      }
    }
  };

  while (lead) {
    // the next tiles, and what they add to, as far ahead as registers allow
    Tile t[kMade];
    int made = 0, own = -1;
#pragma unroll
    for (int w = 0; w < kMade; ++w)
      if (lead) {
        const int at = first_of(lead);
        if (w == wave) own = at;
        t[w] = tile_of<16>(id, at);
        lead &= lead - 1;
        ++made;
      } else {
        t[w] = Tile{kNoToken, 0, 0};
      }
    if (SINGLE) lead = 0;
    Base<BASE_BF16> base[kAhead] = {};
    if (n0 < a.d) {
      if (a.base) {
#pragma unroll
        for (int w = 0; w < kAhead; ++w)
          if (w < made) load_base(t[w], base[w]);
      }
      load_p(t[0].id);
    }
    if (own >= 0) {
      const Tile o = tile_of<16>(id, own);
      const int64_t token = t0 + __shfl(o.token, min(c, o.size - 1), kWave);
      const float scale = o.id >= 0 ? a.scale[o.id] : 0.0f;
#pragma unroll
      for (int k = 0; k < RS; ++k) {
        const int r = k * 32 + q * 8;
        uint32_t cut[8][kCuts];
        float v[8] = {};
        if (o.id >= 0 && c < o.size && r < a.rank)
          scaled(a.part + token * a.rank + r, plane, a.slices, scale, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) split(v[e], cut[e]);
#pragma unroll
        for (int e = 0; e < kCuts; ++e)
          s.c[wave][k][e][lane] = make_uint4(cut[0][e] | cut[1][e] << 16, cut[2][e] | cut[3][e] << 16,
                                             cut[4][e] | cut[5][e] << 16, cut[6][e] | cut[7][e] << 16);
      }
    }
    lds_barrier();
#pragma unroll
    for (int w = 0; w < kMade; ++w) {
      if (w >= made || n0 >= a.d) break;
      const int who = t[w].id;
      if (w > 0) load_p(who);
      floatx4_t acc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
      if (who >= 0) {
#pragma unroll
        for (int k = 0; k < RS; ++k)
#pragma unroll
          for (int e = 0; e < kCuts; ++e) {
            const bf16x8_t h = operand(s.c[w][k][e][lane]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, operand(p[k][j]), acc[j], 0, 0, 0);
          }
        if (some_nan(acc))
          mend(acc, [&](int j) __attribute__((always_inline)) {
            floatx4_t by = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < RS; ++k)
              by = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(s.c[w][k][0][lane]), operand(p[k][j]), by, 0, 0, 0);
            return by;
          });
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t token = t0 + __shfl(t[w].token, q * 4 + i, kWave);
        float v[8] = {};
        if (a.base) unpack<BASE_BF16>(base[w % kAhead], i, v);
        if (who >= 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += acc[j][i];
        }
        if (q * 4 + i < t[w].size && mine < a.d) store8<OUT_BF16, !SINGLE>(a.out, token * a.out_stride + mine, v);
      }
      if (SINGLE) return;
      if (w + kAhead < kMade && w + kAhead < made && a.base) load_base(t[w + kAhead], base[w % kAhead]);
    }
    if (lead) lds_barrier();  // the operands are made anew
  }
}

// Waves of a SIMD that the registers are to leave room for: the loads of several hide each
// other's waits.
template <int RS, bool BASE_BF16, bool SINGLE>
constexpr int expand_waves() {
  return RS == 1 ? (SINGLE ? 4 : BASE_BF16 ? 3 : 2) : RS == 2 ? (SINGLE ? 3 : 2) : 1;
}

// SINGLE: one block of tokens, whose workgroup y takes the tile that token y leads, if any.
template <int RS, bool BASE_BF16, bool OUT_BF16, bool SINGLE>
__global__ __launch_bounds__(kThreads, (expand_waves<RS, BASE_BF16, SINGLE>())) void lowrank_expand(ExpandArgs a) {
  __shared__ ExpandShared<RS> s;
  expand<RS, BASE_BF16, OUT_BF16, SINGLE>(a, s, blockIdx.x, blockIdx.y, blockIdx.z);
}

// ---------------------------------------------------------- few tokens, one launch

constexpr int kFewWaves = 16, kFewThreads = kFewWaves * kWave;
struct FewArgs {
  const uint16_t* down;
  const uint16_t* up;
  const float* scale;
  const uint16_t* x;
  const int32_t* index;
  const void* base;  // or nullptr
  void* out;
  int64_t x_stride, base_stride, out_stride, count;
  int m, rank, k, n;
};

// One block of tokens.  Workgroup (a token that leads a tile, 2048 columns of the output): its
// sixteen waves take up to four of the shrink's steps at a time and meet in LDS; then each
// expands 128 columns, whose rows of the stack and tokens to add to were requested first.
// Every workgroup of a tile makes the tile's c anew, from rows of `down` that are in L2
// after the first: workgroups of one tile are a multiple of 8 apart, on one XCD.
// Bound by latency: index, rows, their sums, the product and the store follow one another
// (3840 -> 3840, rank 8, 1 token: 8.1 us, of which the second round of loads is 2).
template <int RT, bool BASE_BF16, bool OUT_BF16>
__global__ __launch_bounds__(kFewThreads) void lowrank_add_few(FewArgs a) {
  constexpr int kDepth = BASE_BF16 ? 4 : 2;  // by registers
  __shared__ float4 s_red[kFewWaves][RT][kWave];
  __shared__ float4 s_sum[RT][kWave];
  const int id = block_id(a.index, a.m, a.count);
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int lowest = a.base == a.out ? 0 : kNoAdapter;  // in place, tokens without an adapter are done
  if (__builtin_amdgcn_readlane(id, blockIdx.x) < lowest || !leads<16>(id, blockIdx.x)) return;
  const Tile tile = tile_of<16>(id, blockIdx.x);
  const bool has = tile.id >= 0;
  const int mine = blockIdx.y * (kFewWaves * 128) + wave * 128 + c * 8;  // the lane's first column
  const int at = mine < a.n ? mine : 0;
  const float scale = has ? a.scale[tile.id] : 0.0f;
  Base<BASE_BF16> base{};
  auto load_base = [&]() __attribute__((always_inline)) {
    if (!a.base) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t token = __shfl(tile.token, min(q * 4 + i, tile.size - 1), kWave);
      const char* from = static_cast<const char*>(a.base) + (token * a.base_stride + at) * (BASE_BF16 ? 2 : 4);
      if constexpr (BASE_BF16) {
        base.v[i] = load_once<false>(from);
      } else {
        base.v[2 * i] = load_once<false>(from);
        base.v[2 * i + 1] = load_once<false>(from + 16);
      }
    }
  };
  if (BASE_BF16 || !has) load_base();  // float32 has to wait for registers
  floatx4_t acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  if (has) {
    uint4 rows[8], p[8];
    {
      const uint16_t* from = a.up + ((int64_t)tile.id * a.rank + min(q * 8, a.rank - 8)) * a.n + at;
#pragma unroll
      for (int e = 0; e < 8; ++e) rows[e] = load16(from + (int64_t)e * a.n);
    }
    const int lr = lane >> 2, lc = lane & 3;  // row and 16-byte chunk of a load
    const uint16_t* x = a.x + (int64_t)__shfl(tile.token, min(lr, tile.size - 1), kWave) * a.x_stride;
    const uint16_t* down = a.down + (int64_t)tile.id * a.rank * a.k;
    floatx4_t sum[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) sum[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    for (int step = wave * kDepth; step * 32 < a.k; step += kFewWaves * kDepth) {
      uint4 v[kDepth], w[kDepth][RT];
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int e = (step + u) * 32 + lc * 8;
        const bool in = e < a.k;      // k is a multiple of 8
        const int col = in ? e : 0;   // past k the row's first columns are read, and dropped
        const uint4 y = load16(x + col);
        v[u] = in ? y : zero16();
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint4 z = load16(down + (int64_t)min(i * 16 + lr, a.rank - 1) * a.k + col);
          w[u][i] = in ? z : zero16();
        }
      }
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const bf16x8_t y = operand(to_operand(v[u]));
#pragma unroll
        for (int i = 0; i < RT; ++i)
          sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(to_operand(w[u][i])), y, sum[i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) s_red[wave][i][lane] = make_float4(sum[i][0], sum[i][1], sum[i][2], sum[i][3]);
    __syncthreads();
    if (wave < RT) {
      float4 all = s_red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) {
        const float4 add = s_red[w][wave][lane];
        all.x += add.x; all.y += add.y; all.z += add.z; all.w += add.w;
      }
      s_sum[wave][lane] = all;
    }
    __syncthreads();
    // lane (c, q): ranks 8 q ... of token c, which lanes c + 16 (2 q % 4) and the next sixteen hold
    uint32_t cut[8][kCuts];
    auto cuts = [&]() __attribute__((always_inline)) {
      float v[8] = {};
      if (q / 2 < RT && q * 8 < a.rank && c < tile.size) {
        const float4 lo = s_sum[q / 2][c + 32 * (q & 1)], hi = s_sum[q / 2][c + 32 * (q & 1) + 16];
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) split(v[e] * scale, cut[e]);
    };
    auto part = [&](int e) __attribute__((always_inline)) {
      return operand(make_uint4(cut[0][e] | cut[1][e] << 16, cut[2][e] | cut[3][e] << 16,
                                cut[4][e] | cut[5][e] << 16, cut[6][e] | cut[7][e] << 16));
    };
    cuts();
#pragma unroll
    for (int e = 0; e < 8; ++e) rows[e] = q * 8 < a.rank ? rows[e] : zero16();
    transpose8(rows, p);
    if (!BASE_BF16) {
      __builtin_amdgcn_sched_barrier(0);  // neither sooner nor later: by registers
      load_base();
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int e = 0; e < kCuts; ++e) {
      const bf16x8_t h = part(e);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, operand(p[j]), acc[j], 0, 0, 0);
    }
    if (some_nan(acc)) {
      __builtin_amdgcn_sched_barrier(0);
      cuts();  // made anew: kept, they would cost registers
      const bf16x8_t h = part(0);
      mend(acc, [&](int j) __attribute__((always_inline)) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(h, operand(p[j]), floatx4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      });
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t token = __shfl(tile.token, min(q * 4 + i, tile.size - 1), kWave);
    float v[8] = {};
    if (a.base) unpack<BASE_BF16>(base, i, v);
    if (has) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += acc[j][i];
    }
    if (q * 4 + i < tile.size && mine < a.n) store8<OUT_BF16, false>(a.out, token * a.out_stride + mine, v);
  }
}

// ------------------------------------------------------------------ launches

int64_t blocks_of(int64_t m) { return (m + kBlockTokens - 1) / kBlockTokens; }
// One block of tokens: a workgroup a token, those that lead no tile end at once.  More blocks have work
// enough as long as a block meets few adapters (3840 -> 11520, rank 16: 128 tokens of one adapter
// 14.5 us); tokens of as many adapters are walked tile by tile by few workgroups (65 to 256
// of them 210 us, where calls of 64 take 24 to 63).
bool single_block(int64_t m) { return m <= kBlockTokens; }

struct ShrinkPlan {
  int slices, shares;
};

// About `groups_wanted` workgroups, as long as a wave has a step of its own.  Shares of a block's
// tiles: two, for its two tiles or for the block in which one adapter's run ends and another's
// begins.  Backward 512: dy comes from memory (8192 tokens of 10240, rank 64: 144 us, with 256
// 237).  Forward 256, x was made a moment ago and is in cache; 128 past rank 32, where every
// workgroup of the expand adds as many slices of longer rows (4096 tokens, 3840 -> 20480,
// rank 64: 102 us, with 256 104; 2047 tokens, 10240 -> 3840, rank 32: 42, with 256 33).
constexpr int kBackwardGroups = 512;
constexpr int forward_groups(int64_t rank) { return rank > 32 ? 128 : 256; }
ShrinkPlan shrink_plan(int64_t m, int64_t d, int64_t rank, int64_t groups_wanted) {
  ShrinkPlan p;
  m = std::max<int64_t>(m, 1);
  p.shares = (int)(single_block(m) ? m : 2);
  const int64_t steps = (d + 31) / 32;
  const int64_t groups = single_block(m) ? m : blocks_of(m) * (kBlockTokens / shrink_tile(rank));
  const int64_t want = (groups_wanted + groups - 1) / groups;
  p.slices = (int)std::max<int64_t>(1, std::min<int64_t>({want, (steps + 3) / 4, 16}));
  const int64_t per = (steps + p.slices - 1) / p.slices;
  p.slices = (int)((steps + per - 1) / per);  // none without steps
  return p;
}

size_t up256(size_t b) { return (b + 255u) & ~size_t(255); }

template <int W, bool PLAN>
hipError_t launch_shrink_of(const ShrinkArgs& a, const PlanArgs& plan, dim3 grid, hipStream_t stream) {
  const dim3 threads(W * kWave);
  if (a.rank <= 16) hipLaunchKernelGGL((lowrank_shrink<1, W, PLAN>), grid, threads, 0, stream, a, plan);
  else if (a.rank <= 32) hipLaunchKernelGGL((lowrank_shrink<2, W, PLAN>), grid, threads, 0, stream, a, plan);
  else if (a.rank <= 64) hipLaunchKernelGGL((lowrank_shrink<4, W, PLAN>), grid, threads, 0, stream, a, plan);
  else if constexpr (W == 4) hipLaunchKernelGGL((lowrank_shrink<8, W, PLAN>), grid, threads, 0, stream, a, plan);
  return hipGetLastError();
}

template <bool PLAN>
hipError_t launch_shrink(const ShrinkArgs& a, const PlanArgs& plan, int shares, hipStream_t stream) {
  const dim3 grid((unsigned)(a.side[0].slices + a.side[1].slices + PLAN), (unsigned)shares,
                  (unsigned)std::max<int64_t>(1, blocks_of(a.m)));
  // eight waves a workgroup where registers allow: half the slices for the reader to add
  return a.single || a.rank > 64 ? launch_shrink_of<4, PLAN>(a, plan, grid, stream)
                                 : launch_shrink_of<8, PLAN>(a, plan, grid, stream);
}

template <int RS, bool SINGLE>
hipError_t launch_expand_of(const ExpandArgs& a, bool base_bf16, bool out_bf16, hipStream_t stream) {
  const dim3 grid((unsigned)((a.d + 511) / 512), (unsigned)(SINGLE ? a.m : 1), (unsigned)blocks_of(a.m));
  if (base_bf16 && out_bf16)
    hipLaunchKernelGGL((lowrank_expand<RS, true, true, SINGLE>), grid, dim3(kThreads), 0, stream, a);
  else if (base_bf16)
    hipLaunchKernelGGL((lowrank_expand<RS, true, false, SINGLE>), grid, dim3(kThreads), 0, stream, a);
  else if (out_bf16)
    hipLaunchKernelGGL((lowrank_expand<RS, false, true, SINGLE>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((lowrank_expand<RS, false, false, SINGLE>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <bool SINGLE>
hipError_t launch_expand_as(const ExpandArgs& a, bool base_bf16, bool out_bf16, hipStream_t stream) {
  return a.rank <= 32 ? launch_expand_of<1, SINGLE>(a, base_bf16, out_bf16, stream)
         : a.rank <= 64 ? launch_expand_of<2, SINGLE>(a, base_bf16, out_bf16, stream)
                        : launch_expand_of<4, SINGLE>(a, base_bf16, out_bf16, stream);
}
hipError_t launch_expand(const ExpandArgs& a, bool base_bf16, bool out_bf16, hipStream_t stream) {
  return single_block(a.m) ? launch_expand_as<true>(a, base_bf16, out_bf16, stream)
                           : launch_expand_as<false>(a, base_bf16, out_bf16, stream);
}

}  // namespace

namespace {

// Adapters small enough to be read anew by every workgroup, and no more of those than the card
// takes at once (calls in a graph, this kernel / both, us: 3840 -> 3840, rank 16, 1 token
// 8.3/8.4, 48 tokens 9.2/10.9; 1024 -> 1024, 48 tokens 6.4/8.6; past the rules rank 32 of
// 3840 -> 3840, 1 token 9.7/8.7, and 48 tokens of 3840 -> 11520, rank 16, 17.4/15.3).
constexpr int64_t kFewElements = 1 << 16, kFewGroups = 256;
bool few(int64_t m, int64_t k, int64_t n, int64_t rank) {
  return single_block(m) && rank <= 32 && k * rank <= kFewElements &&
         m * ((n + kFewWaves * 128 - 1) / (kFewWaves * 128)) <= kFewGroups;
}

template <int RT>
hipError_t launch_few_of(const FewArgs& a, bool base_bf16, bool out_bf16, hipStream_t stream) {
  const dim3 grid((unsigned)(a.m + 7) / 8 * 8, (unsigned)(a.n + kFewWaves * 128 - 1) / (kFewWaves * 128));
  auto kernel = base_bf16 ? out_bf16 ? lowrank_add_few<RT, true, true> : lowrank_add_few<RT, true, false>
                : out_bf16 ? lowrank_add_few<RT, false, true> : lowrank_add_few<RT, false, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kFewThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t lowrank_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank) {
  (void)n;
  return up256((size_t)shrink_plan(m, k, rank, forward_groups(rank)).slices * (size_t)m * (size_t)rank * 4u);
}

hipError_t launch_lowrank_add(const LowrankAdd& c, hipStream_t stream) {
  if (few(c.m, c.a.k, c.a.n, c.a.rank)) {
    FewArgs f{};
    f.down = c.a.down;
    f.up = c.a.up;
    f.scale = c.a.scale;
    f.x = c.x;
    f.index = c.index;
    f.base = c.y;
    f.out = c.out;
    f.x_stride = c.x_stride;
    f.base_stride = c.y_stride;
    f.out_stride = c.out_stride;
    f.count = c.a.count;
    f.m = (int)c.m;
    f.rank = (int)c.a.rank;
    f.k = (int)c.a.k;
    f.n = (int)c.a.n;
    return c.a.rank <= 16 ? launch_few_of<1>(f, c.y_bf16, c.out_bf16, stream)
                          : launch_few_of<2>(f, c.y_bf16, c.out_bf16, stream);
  }
  const ShrinkPlan plan = shrink_plan(c.m, c.a.k, c.a.rank, forward_groups(c.a.rank));
  ShrinkArgs s{};
  s.side[0] = {c.a.down, c.x, c.x_stride, static_cast<float*>(c.workspace), (int)c.a.k, plan.slices};
  s.index = c.index;
  s.m = c.m;
  s.count = c.a.count;
  s.rank = (int)c.a.rank;
  s.single = single_block(c.m);
  const hipError_t e = launch_shrink<false>(s, PlanArgs{}, plan.shares, stream);
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

// Element of part k, rank r, place j among grad's operands.
__device__ __forceinline__ int64_t operand_at(int rank, int64_t cap, int k, int r, int64_t j) {
  const int tiles = (rank + 15) / 16;
  return (((k * tiles + r / 16) * (cap / 32) + j / 32) * kWave + j % 32 / 8 * 16 + r % 16) * 8 + j % 8;
}

struct OperandArgs {
  GradPlan g;
  const float* part[2];  // [slices][m][rank]
  int slices[2];
  uint16_t* out[2];      // [parts][16-row tiles of the rank][cap / 32][64 lanes][8]
  const float* scale;
  const int32_t* index;
  int64_t m, cap;
  int rank;
};

// s c in bfloat16 parts, transposed, in the order of grad's operands: of 32 places and 16
// ranks, lane (c, q) has rank c, places 8 q ..., and its 16 bytes lie beside its neighbours'.
// A thread makes eight ranks of one place; `group`: 256 places of eight ranks and a side.
__device__ __forceinline__ void operands(const OperandArgs& a, int64_t group) {
  const int64_t groups = (a.cap + kThreads - 1) / kThreads;
  const int64_t j = group % groups * kThreads + threadIdx.x;
  const int which = (int)(group / groups);
  const int side = which / (a.rank / 8), r = which % (a.rank / 8) * 8;
  if (side > 1 || j >= *a.g.places) return;
  const int t = a.g.order[j];
  float v[8] = {};
  if (t >= 0)
    scaled(a.part[side] + (int64_t)t * a.rank + r, a.m * a.rank, a.slices[side], a.scale[a.index[t]], v);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t cut[kCuts];
    split(v[e], cut);
#pragma unroll
    for (int k = 0; k < kCuts; ++k) a.out[side][operand_at(a.rank, a.cap, k, r + e, j)] = (uint16_t)cut[k];
  }
}

__global__ __launch_bounds__(kThreads) void lowrank_operands(OperandArgs a) { operands(a, blockIdx.x); }

// The input's gradient and the operands of the adapters' own: workgroups x < columns expand,
// the others make operands (a launch less).
template <int RS, bool BF16>
__global__ __launch_bounds__(kThreads, (expand_waves<RS, BF16, false>())) void lowrank_expand_operands(
    ExpandArgs a, OperandArgs o, int columns) {
  __shared__ ExpandShared<RS> s;
  if ((int)blockIdx.x < columns) {
    expand<RS, BF16, BF16, false>(a, s, blockIdx.x, 0, blockIdx.y);
    return;
  }
  operands(o, (int64_t)blockIdx.y * ((int)gridDim.x - columns) + ((int)blockIdx.x - columns));
}

struct GradSide {
  const uint16_t* v;  // [m][stride]
  const uint16_t* c;  // the operands
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

// Workgroup (128 columns, item, 64 rows of the rank): its waves take every fourth 32 tokens and
// meet in LDS, so that an item may be four times as long as one wave's share (with a wave
// for 128 columns each and items a quarter as long, the slots of a single adapter of 4096 tokens
// were 16 MB to write and join).  Lane (c, q) holds columns 8 c ... of eight tokens, 8 q ... of
// each 32, and after the transposition is column 8 c + j of the j-th product.  RT: 16-row
// tiles of the rank, at most 4 (rank 128 takes two workgroups, by registers).
template <int RT, bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void lowrank_grad(GradArgs a) {
  constexpr int kOnce = RT < 2 ? RT : 2;  // row tiles in LDS together
  __shared__ float s_red[kWaves][kOnce][8][4][kWave];
  const int item = blockIdx.y;
  if (item >= *a.g.items) return;
  const bool second = blockIdx.x >= (unsigned)a.side[0].blocks;
  const GradSide& g = a.side[second];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int n = ((int)blockIdx.x - (second ? a.side[0].blocks : 0)) * 128 + c * 8, r0 = blockIdx.z * 64;
  const int from = a.g.from[item], length = a.g.length[item];
  const uint16_t* v = g.v + (n < g.d ? n : 0);
  const int tiles = (a.rank + 15) / 16;
  const int64_t plane = (int64_t)tiles * a.cap * 16;  // elements of a part
  const uint16_t* row[RT];  // a tile past the rank reads the last one, and is dropped
#pragma unroll
  for (int i = 0; i < RT; ++i)
    row[i] = g.c + ((int64_t)min(r0 / 16 + i, tiles - 1) * a.cap + from) * 16 + lane * 8;
  floatx4_t acc[RT][8];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  for (int at = wave * 32; at < length; at += kWaves * 32) {
    const int4* o = reinterpret_cast<const int4*>(a.g.order + from + at + q * 8);
    const int4 o0 = o[0], o1 = o[1];
    const int t[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
    uint4 rows[8], cols[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rows[e] = t[e] >= 0 ? load16(v + t[e] * g.stride) : zero16();
    bf16x8_t h[RT][kCuts];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int k = 0; k < kCuts; ++k) h[i][k] = operand(load16(row[i] + k * plane + at * 16));
    transpose8(rows, cols);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int k = 0; k < kCuts; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(h[i][k], operand(cols[j]), acc[i][j], 0, 0, 0);
  }
  const int slot = a.g.slot[item];
  const int64_t first = slot < 0 ? (int64_t)a.g.adapter[item] * a.rank : (int64_t)slot * a.rank;
#pragma unroll
  for (int i0 = 0; i0 < RT; i0 += kOnce) {
    if (i0) __syncthreads();  // the last tiles are read
#pragma unroll
    for (int i = 0; i < kOnce; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_red[wave][i][j][e][lane] = acc[i0 + i][j][e];
    __syncthreads();
    // wave e adds the rows 4 q + e
#pragma unroll
    for (int i = 0; i < kOnce; ++i) {
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = s_red[0][i][j][wave][lane];
#pragma unroll
        for (int k = 1; k < kWaves; ++k) w[j] += s_red[k][i][j][wave][lane];
      }
      const int r = r0 + (i0 + i) * 16 + q * 4 + wave;
      if (r < a.rank && n < g.d) {
        float all = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) all += w[j];
        if (all != all) {  // NaN: the item's sums of the first parts, token by token
          float by[8] = {};
#pragma unroll 1
          for (int at = from; at < from + length; ++at) {
            const float c0 = __uint_as_float((uint32_t)g.c[operand_at(a.rank, a.cap, 0, r, at)] << 16);
            float x[8];
            load8<true>(v, a.g.order[at] * g.stride, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) by[j] += c0 * x[j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = w[j] != w[j] ? by[j] : w[j];
        }
        const int64_t to = (first + r) * g.d + n;
        if (slot < 0) store8<OUT_BF16, false>(g.out, to, w);
        else store8<false, false>(g.part, to, w);
      }
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
    store8<OUT_BF16, false>(a.out[side], id * size + at, v);
  }
}

constexpr int kGradGroups = 512;
struct BackwardPlan {
  ShrinkPlan h, e;
  int64_t cap, items, slots;
  int seg;
  size_t part_h, part_e, operand_h, operand_e, sums_down, sums_up, lists, bytes;
};

BackwardPlan backward_plan(int64_t m, int64_t k, int64_t n, int64_t rank, int64_t count) {
  BackwardPlan b{};
  b.h = shrink_plan(m, k, rank, kBackwardGroups);
  b.e = shrink_plan(m, n, rank, kBackwardGroups);
  // about 512 workgroups in grad, each wave of at least 32 tokens
  const int64_t columns = (k + 127) / 128 + (n + 127) / 128;
  const int64_t seg = (m * columns / kGradGroups + 127) / 128 * 128;
  b.seg = (int)std::max<int64_t>(128, seg);
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
  const size_t ranks = (size_t)(rank + 15) / 16 * 16;  // whole tiles
  b.operand_h = take(kCuts * ranks * b.cap * 2);
  b.operand_e = take(kCuts * ranks * b.cap * 2);
  b.sums_down = take((size_t)b.slots * rank * k * 4);
  b.sums_up = take((size_t)b.slots * rank * n * 4);
  b.lists = take((size_t)(b.cap + 64 + 4 * b.items + 2 * count) * 4);
  b.bytes = at;
  return b;
}

template <int RT>
hipError_t launch_grad_of(const GradArgs& g, bool bf16, dim3 grid, hipStream_t stream) {
  if (bf16) hipLaunchKernelGGL((lowrank_grad<RT, true>), grid, dim3(kThreads), 0, stream, g);
  else hipLaunchKernelGGL((lowrank_grad<RT, false>), grid, dim3(kThreads), 0, stream, g);
  return hipGetLastError();
}

hipError_t launch_grad(const GradArgs& g, bool bf16, int64_t items, hipStream_t stream) {
  const dim3 grid((unsigned)(g.side[0].blocks + g.side[1].blocks), (unsigned)items, (unsigned)(g.rank > 64 ? 2 : 1));
  return g.rank <= 16 ? launch_grad_of<1>(g, bf16, grid, stream)
         : g.rank <= 32 ? launch_grad_of<2>(g, bf16, grid, stream) : launch_grad_of<4>(g, bf16, grid, stream);
}

template <int RS>
hipError_t launch_both_of(const ExpandArgs& a, const OperandArgs& o, bool bf16, dim3 grid, int columns,
                          hipStream_t stream) {
  if (bf16) hipLaunchKernelGGL((lowrank_expand_operands<RS, true>), grid, dim3(kThreads), 0, stream, a, o, columns);
  else hipLaunchKernelGGL((lowrank_expand_operands<RS, false>), grid, dim3(kThreads), 0, stream, a, o, columns);
  return hipGetLastError();
}

hipError_t launch_both(const ExpandArgs& a, const OperandArgs& o, bool bf16, int64_t groups, hipStream_t stream) {
  const int columns = (a.d + 511) / 512;
  const int64_t blocks = blocks_of(a.m);
  const dim3 grid((unsigned)(columns + (groups + blocks - 1) / blocks), (unsigned)blocks);
  return a.rank <= 32 ? launch_both_of<1>(a, o, bf16, grid, columns, stream)
         : a.rank <= 64 ? launch_both_of<2>(a, o, bf16, grid, columns, stream)
                        : launch_both_of<4>(a, o, bf16, grid, columns, stream);
}

}  // namespace

size_t lowrank_backward_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank, int64_t count) {
  return backward_plan(m, k, n, rank, count).bytes;
}

// Four launches: both shrinks and the plan; dx and the operands; both gradients; their slots
// joined.
hipError_t launch_lowrank_backward(const LowrankBackward& c, hipStream_t stream) {
  const int64_t k = c.a.k, n = c.a.n, rank = c.a.rank;
  const BackwardPlan b = backward_plan(c.m, k, n, rank, c.a.count);
  char* ws = static_cast<char*>(c.workspace);
  float* part_h = reinterpret_cast<float*>(ws + b.part_h);
  float* part_e = reinterpret_cast<float*>(ws + b.part_e);
  const bool grads = c.d_down != nullptr;
  hipError_t err;

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

  ShrinkArgs s{};
  s.side[0] = {c.a.up, c.dy, c.dy_stride, part_e, (int)n, b.e.slices};
  if (grads) s.side[1] = {c.a.down, c.x, c.x_stride, part_h, (int)k, b.h.slices};
  s.index = c.index;
  s.m = c.m;
  s.count = c.a.count;
  s.rank = (int)rank;
  s.single = single_block(c.m);
  err = grads ? launch_shrink<true>(s, PlanArgs{g, c.index, c.m, (int)c.a.count, b.seg}, b.e.shares, stream)
              : launch_shrink<false>(s, PlanArgs{}, b.e.shares, stream);
  if (err != hipSuccess) return err;

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
  if (!grads) return launch_expand(x, c.dx_bf16, c.dx_bf16, stream);

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
  GradArgs ga{};
  ga.g = g;
  ga.side[0] = {c.x, o.out[0], c.x_stride, reinterpret_cast<float*>(ws + b.sums_down), c.d_down, (int)k,
                (int)((k + 127) / 128)};
  ga.side[1] = {c.dy, o.out[1], c.dy_stride, reinterpret_cast<float*>(ws + b.sums_up), c.d_up, (int)n,
                (int)((n + 127) / 128)};
  ga.cap = b.cap;
  ga.rank = (int)rank;
  if (c.m > 0) {  // else there is no item, and the join writes zeros
    const int64_t groups = (b.cap + kThreads - 1) / kThreads * (rank / 8) * 2;
    if (c.dx_out) {
      err = launch_both(x, o, c.dx_bf16, groups, stream);
    } else {
      hipLaunchKernelGGL(lowrank_operands, dim3((unsigned)groups), dim3(kThreads), 0, stream, o);
      err = hipGetLastError();
    }
    if (err != hipSuccess) return err;
    if ((err = launch_grad(ga, c.grad_bf16, b.items, stream)) != hipSuccess) return err;
  }

  JoinArgs j{};
  j.slots = g.slots;
  for (int i = 0; i < 2; ++i) {
    j.part[i] = ga.side[i].part;
    j.out[i] = ga.side[i].out;
    j.size[i] = rank * ga.side[i].d;
  }
  const int64_t widest = std::max(j.size[0], j.size[1]);
  const dim3 grid((unsigned)std::min<int64_t>((widest / 8 + kThreads - 1) / kThreads, 1024), (unsigned)c.a.count, 2);
  if (c.grad_bf16) hipLaunchKernelGGL(lowrank_join<true>, grid, dim3(kThreads), 0, stream, j);
  else hipLaunchKernelGGL(lowrank_join<false>, grid, dim3(kThreads), 0, stream, j);
  return hipGetLastError();
}

}  // namespace opq
