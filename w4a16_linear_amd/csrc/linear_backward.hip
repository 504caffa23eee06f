// The parts of the gradient through a quantized projection that are its own: the dense
// product contracts along the weights' rows, and its operand has that dimension dense.
#include <algorithm>

#include "adapters_internal.hpp"
#include "decode.hpp"
#include "device_common.hpp"
#include "group.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;
constexpr int kMidThreads = 512;

// Eight columns of eight rows each, from eight rows of eight bfloat16: v_perm pairs rows.
__device__ __forceinline__ void store_columns(const uint32_t (&row)[8][4], uint16_t* to, int64_t ld) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = __builtin_amdgcn_perm(row[2 * i + 1][q], row[2 * i][q], 0x05040100u);
      hi[i] = __builtin_amdgcn_perm(row[2 * i + 1][q], row[2 * i][q], 0x07060302u);
    }
    *reinterpret_cast<uint4*>(to + (int64_t)(2 * q) * ld) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(to + (int64_t)(2 * q + 1) * ld) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

// Eight columns of a token's dx, or of the slice's plane of sums.
__device__ __forceinline__ void store_row(const float (&v)[8], int token, int col, int m, int k, void* out,
                                          int out_bf16, float* part) {
  if (part) {
    float4* to = reinterpret_cast<float4*>(part + ((int64_t)blockIdx.y * m + token) * k + col);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else if (out_bf16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + (int64_t)token * k + col) =
        make_uint4(bf16_rne(v[0]) | bf16_rne(v[1]) << 16, bf16_rne(v[2]) | bf16_rne(v[3]) << 16,
                   bf16_rne(v[4]) | bf16_rne(v[5]) << 16, bf16_rne(v[6]) | bf16_rne(v[7]) << 16);
  } else {
    float4* to = reinterpret_cast<float4*>(static_cast<float*>(out) + (int64_t)token * k + col);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Few tokens: dx straight from the 4-bit codes, which are read once and W' nowhere written.
// Workgroup (128 columns of k, a slice of the weights' rows), 16 MT tokens.  Of 32 rows, lane
// (c, q) = (l % 16, l / 16) decodes the word of columns 8 c ... of rows 8 q ... and turns
// the 8 x 8 block in registers: it is column 8 c + j of the j-th product, tokens are the
// rows.  The rows' tables (16 bfloat16 entries as byte planes, one for each group in the
// columns) are made in LDS for 256 rows at a time, while the codes of those rows are on
// their way; a wave takes two of their eight steps.  The waves' sums meet in LDS, the
// slices' in linear.hip's split reduction.  Bound by the decoder's VALU work (20480 x 3840 at
// 8 tokens: 49 MB of codes in 33 us and 5 for the slices' sums).  Up to 64 tokens; with 65
// backward_mid takes 20 us where this takes 26 (3840 x 3840), and 40 for 43 (11520 x 3840).
template <int MT, int GS>
__global__ __launch_bounds__(kThreads) void backward_short(
    const uint16_t* __restrict__ dy, int64_t ldy, const uint32_t* __restrict__ packed,
    const uint32_t* __restrict__ sign, const float* __restrict__ scale, const uint16_t* __restrict__ scale16,
    int m, int n, int n_read, int k, Levels lv, int slice_rows, void* __restrict__ out, int out_bf16,
    float* __restrict__ part) {
  constexpr int kWaves = kThreads / kWave, kChunk = 256, kMine = kChunk / 32 / kWaves;
  constexpr int G = GS == 0 || GS >= 128 ? 1 : 128 / GS;  // tables of a row
  __shared__ __attribute__((aligned(16))) uint32_t s_tab[kChunk * G * 8];
  __shared__ float s_red[kWaves][8][4][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int k0 = blockIdx.x * 128, col = k0 + c * 8, kk = min(col, k - 8);
  const int begin = blockIdx.y * slice_rows, end = min(n, begin + slice_rows);
  const int group = GS == 0 || GS >= 128 ? 0 : c * 8 / (GS ? GS : 1);
  floatx4_t acc[MT][8];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[t][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  for (int r0 = begin; r0 < end; r0 += kChunk) {
    uint32_t word[kMine][8], sg[kMine][8];
    uint4 a[kMine][MT];
#pragma unroll
    for (int s = 0; s < kMine; ++s) {
      const int r = r0 + (wave + s * kWaves) * 32 + q * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t at = min(r + e, n - 1);
        word[s][e] = packed[at * (k / 8) + kk / 8];
        sg[s][e] = sign[at * (k / 32) + kk / 32] >> (8 * (c & 3));
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint4 v = *reinterpret_cast<const uint4*>(dy + (int64_t)min(t * 16 + c, m - 1) * ldy +
                                                        min(r, n_read - 8));
        a[s][t] = r < min(end, n_read) ? v : make_uint4(0u, 0u, 0u, 0u);  // rows past the slice count nothing
      }
    }
    if (r0 > begin) __syncthreads();  // the last rows' tables are read
    {
      const int64_t r = min(r0 + (int)threadIdx.x, n - 1);
      const bool past = r0 + (int)threadIdx.x >= n;  // the last row's codes with tables of zeros
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float top;
        if constexpr (GS > 0) top = f16_value(scale16[r * (k / (GS ? GS : 1)) + min(k0 / (GS ? GS : 1) + g, k / (GS ? GS : 1) - 1)]);
        else top = scale[r];
        const RowLut t = make_row_lut(lv, past ? 0.f : top);
        uint32_t* to = s_tab + (threadIdx.x * G + g) * 8;
        *reinterpret_cast<uint4*>(to) = make_uint4(t.lo[0], t.lo[1], t.lo[2], t.lo[3]);
        *reinterpret_cast<uint4*>(to + 4) = make_uint4(t.hi[0], t.hi[1], t.hi[2], t.hi[3]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kMine; ++s) {
      const int local = (wave + s * kWaves) * 32 + q * 8;
      if (r0 + (wave + s * kWaves) * 32 >= end) continue;
      uint32_t row[8][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(s_tab + ((local + e) * G + group) * 8);
        const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(s_tab + ((local + e) * G + group) * 8 + 4);
        RowLut t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t.lo[i] = lo[i];
          t.hi[i] = hi[i];
        }
        decode_word_split(word[s][e], sg[s][e], t, row[e]);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __builtin_amdgcn_perm(row[2 * i + 1][p], row[2 * i][p], 0x05040100u);
          hi[i] = __builtin_amdgcn_perm(row[2 * i + 1][p], row[2 * i][p], 0x07060302u);
        }
        const bf16x8_t w0 = __builtin_bit_cast(bf16x8_t, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        const bf16x8_t w1 = __builtin_bit_cast(bf16x8_t, make_uint4(hi[0], hi[1], hi[2], hi[3]));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const bf16x8_t x = __builtin_bit_cast(bf16x8_t, a[s][t]);
          acc[t][2 * p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w0, acc[t][2 * p], 0, 0, 0);
          acc[t][2 * p + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w1, acc[t][2 * p + 1], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (t) __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s_red[wave][j][e][lane] = acc[t][j][e];
    __syncthreads();
    // wave e adds the tokens 4 q + e
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = s_red[0][j][wave][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v[j] += s_red[w][j][wave][lane];
    }
    const int token = t * 16 + q * 4 + wave;
    if (token < m && col < k) store_row(v, token, col, m, k, out, out_bf16, part);
  }
}

// Some hundred tokens: the same product with the decoding shared.  Workgroup (128 columns of k,
// a slice of the weights' rows), all tokens: of 256 rows each of eight waves decodes 32
// into the products' operands in LDS, then every wave takes all of them for its tokens,
// sixteen rows in eight tiles apart, so sums stay in one wave.  dy is loaded in memory's order
// (four lanes 64 bytes of a row), some steps ahead, and permuted; the next rows' codes are on
// their way during the products.  Bound by the latency of a chunk's phases (codes and tables, two
// barriers, the products' operands from LDS, 64 KB a chunk to each wave): 333 tokens,
// 3840 x 3840: 27 us and 7 for the sums of eight slices; dy one step ahead 30.
template <int MT, int GS>
__global__ __launch_bounds__(kMidThreads) void backward_mid(
    const uint16_t* __restrict__ dy, int64_t ldy, const uint32_t* __restrict__ packed,
    const uint32_t* __restrict__ sign, const float* __restrict__ scale, const uint16_t* __restrict__ scale16,
    int m, int n, int n_read, int k, Levels lv, int slice_rows, void* __restrict__ out, int out_bf16,
    float* __restrict__ part) {
  constexpr int kWaves = kMidThreads / kWave, kChunk = 32 * kWaves;
  constexpr int G = GS == 0 || GS >= 128 ? 1 : 128 / GS;  // tables of a row
  constexpr int kGroup = GS ? GS : 1;
  constexpr int kAhead = MT == 1 ? 8 : MT == 2 ? 6 : MT == 3 ? 3 : 2;  // steps of dy, by registers
  __shared__ __attribute__((aligned(16))) uint32_t s_tab[kChunk * G * 8];
  __shared__ uint4 s_op[kWaves][8][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, q = lane >> 4;
  const int k0 = blockIdx.x * 128, col = k0 + c * 8, kk = min(col, k - 8);
  const int begin = blockIdx.y * slice_rows, end = min(n, begin + slice_rows);
  const int group = GS == 0 || GS >= 128 ? 0 : c * 8 / kGroup;
  const uint16_t* from[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
    from[t] = dy + (int64_t)min((wave + t * kWaves) * 16 + (lane >> 2), m - 1) * ldy;
  floatx4_t acc[MT][8];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[t][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
  uint32_t word[8], sg[8];
  auto codes = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t at = min(r0 + wave * 32 + q * 8 + e, n - 1);
      word[e] = packed[at * (k / 8) + kk / 8];
      sg[e] = sign[at * (k / 32) + kk / 32] >> (8 * (c & 3));
    }
  };
  // rows past the slice count nothing
  auto tokens = [&](int r, uint4 (&x)[MT]) __attribute__((always_inline)) {
    const int at = r + (lane & 3) * 8;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint4 v = *reinterpret_cast<const uint4*>(from[t] + min(at, n_read - 8));
      x[t] = at < min(end, n_read) ? v : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  codes(begin);
  for (int r0 = begin; r0 < end; r0 += kChunk) {
    uint4 x[kAhead][MT];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) tokens(r0 + s * 32, x[s]);
    for (int i = threadIdx.x; i < kChunk * G; i += kMidThreads) {
      const int64_t r = min(r0 + i / G, n - 1);
      float top;
      if constexpr (GS > 0) top = f16_value(scale16[r * (k / kGroup) + min(k0 / kGroup + i % G, k / kGroup - 1)]);
      else top = scale[r];
      const RowLut t = make_row_lut(lv, r0 + i / G < n ? top : 0.f);  // rows past n: tables of zeros
      uint32_t* to = s_tab + i * 8;
      *reinterpret_cast<uint4*>(to) = make_uint4(t.lo[0], t.lo[1], t.lo[2], t.lo[3]);
      *reinterpret_cast<uint4*>(to + 4) = make_uint4(t.hi[0], t.hi[1], t.hi[2], t.hi[3]);
    }
    __syncthreads();  // the tables are made, and the last rows' operands read
    {
      uint32_t row[8][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t* at = s_tab + ((wave * 32 + q * 8 + e) * G + group) * 8;
        const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(at);
        const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(at + 4);
        RowLut t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t.lo[i] = lo[i];
          t.hi[i] = hi[i];
        }
        decode_word_split(word[e], sg[e], t, row[e]);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __builtin_amdgcn_perm(row[2 * i + 1][p], row[2 * i][p], 0x05040100u);
          hi[i] = __builtin_amdgcn_perm(row[2 * i + 1][p], row[2 * i][p], 0x07060302u);
        }
        s_op[wave][2 * p][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        s_op[wave][2 * p + 1][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
    }
    if (r0 + kChunk < end) codes(r0 + kChunk);
    __syncthreads();
    const int steps = min(kWaves, (end - r0 + 31) / 32);
#pragma unroll
    for (int s = 0; s < kWaves; ++s) {
      if (s >= steps) break;
      bf16x8_t a[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int at = ((lane & 15) * 4 + (lane >> 4)) * 4;  // chunk q of row c
        a[t] = __builtin_bit_cast(bf16x8_t, make_uint4((uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)x[s % kAhead][t].x),
                                                       (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)x[s % kAhead][t].y),
                                                       (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)x[s % kAhead][t].z),
                                                       (uint32_t)__builtin_amdgcn_ds_bpermute(at, (int)x[s % kAhead][t].w)));
      }
      if (s + kAhead < kWaves) tokens(r0 + (s + kAhead) * 32, x[s % kAhead]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bf16x8_t w = __builtin_bit_cast(bf16x8_t, s_op[s][j][lane]);
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t], w, acc[t][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int token = (wave + t * kWaves) * 16 + q * 4 + e;
      if (token >= m || col >= k) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[t][j][e];
      store_row(v, token, col, m, k, out, out_bf16, part);
    }
}

// dst [k][ld] = W' transposed, straight from 4-bit codes: 0.625 B read and 2 B written a
// weight, where the dequantizer and a transposition move another 4 (11520 x 3840: 57 us).
// A lane decodes 32 k of eight rows, 8 k at a time, and turns each 8 x 8 block in
// registers.  Lane (a, b) = (l % 8, l / 8) of a wave: k 32 a ..., rows 8 b ... of the
// workgroup's 64, so that eight lanes read 128 bytes of a row's codes and eight others write
// 128 bytes of a column.  Rows past n give zeros (the product's padding).
// GS 0: a row's table as byte planes in LDS, a thread making four entries; otherwise the
// group form's tables from the significand table (group.hpp).
template <int GS>
__global__ __launch_bounds__(kThreads) void dequantize_transposed(
    const uint32_t* __restrict__ packed, const uint32_t* __restrict__ sign, const float* __restrict__ scale,
    const uint16_t* __restrict__ scale16, int64_t n, int k, Levels lv, uint16_t* __restrict__ dst, int64_t ld,
    int row_blocks, int k_blocks) {
  constexpr int kRows = 64, kWide = 32 * 8 * (kThreads / kWave);  // rows and k of a workgroup's tile
  __shared__ __attribute__((aligned(16))) uint32_t s_tab[GS ? kMantissas * 8 : kRows * 8];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int a = lane & 7, b = lane >> 3;
  if constexpr (GS > 0) {
    build_mant_table(lv, s_tab);
    __syncthreads();
  }
  for (int tile = blockIdx.x; tile < row_blocks * k_blocks; tile += gridDim.x) {
    const int64_t row0 = (int64_t)(tile / k_blocks) * kRows;
    const int k0 = tile % k_blocks * kWide + wave * 256 + a * 32;
    const int64_t r0 = row0 + b * 8;
    const bool in = k0 < k && r0 < ld;
    uint4 codes[8];
    uint32_t signs[8], tops[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = min(r0 + i, n - 1);
      const int kk = in ? k0 : 0;
      codes[i] = *reinterpret_cast<const uint4*>(packed + r * (k / 8) + kk / 8);
      signs[i] = sign[r * (k / 32) + kk / 32];
      if constexpr (GS > 0) tops[i] = scale16[r * (k / (GS ? GS : 1)) + kk / (GS ? GS : 1)];
      if (r0 + i >= n) {
        codes[i] = make_uint4(0u, 0u, 0u, 0u);
        signs[i] = 0u;
        tops[i] = 0u;
      }
    }
    if constexpr (GS == 0) {
      // entry q of row t / 4 as bytes of the planes: thread t makes q = 4 (t % 4) ...
      const int t = threadIdx.x, j = t & 3;
      const float top = row0 + (t >> 2) < n ? scale[row0 + (t >> 2)] : 0.f;
      uint32_t lo = 0u, hi = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t e = lut_entry(lv, 4 * j + i, top);
        lo |= (e & 0xFFu) << (8 * i);
        hi |= (e >> 8) << (8 * i);
      }
      __syncthreads();  // the tables of the last tile are read
      s_tab[(t >> 2) * 8 + j] = lo;
      s_tab[(t >> 2) * 8 + 4 + j] = hi;
      __syncthreads();
    }
    if (!in) continue;
    RowLut lut[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (GS > 0) {
        lut[i] = group_lut(s_tab, tops[i]);
      } else {
        const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(s_tab + (b * 8 + i) * 8);
        const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(s_tab + (b * 8 + i) * 8 + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lut[i].lo[e] = lo[e];
          lut[i].hi[e] = hi[e];
        }
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t row[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = s == 0 ? codes[i].x : s == 1 ? codes[i].y : s == 2 ? codes[i].z : codes[i].w;
        decode_word_split(w, signs[i] >> (8 * s), lut[i], row[i]);
      }
      store_columns(row, dst + (int64_t)(k0 + 8 * s) * ld + r0, ld);
    }
  }
}

// dst [k][ld] = w [n][k] transposed, columns n..ld-1 zero (codes of other widths).  A lane turns an 8 x 8 block in
// registers (v_perm pairs rows); the eight lanes of a row of blocks read, and the
// eight of a column write, 128 bytes in a row.
__global__ __launch_bounds__(kThreads) void transpose_bf16(const uint16_t* __restrict__ w, int64_t n, int64_t k,
                                                           uint16_t* __restrict__ dst, int64_t ld) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t c = (int64_t)blockIdx.x * 64 + (lane & 7) * 8;                       // along k
  const int64_t r = ((int64_t)blockIdx.y * (kThreads / kWave) + wave) * 64 + (lane >> 3) * 8;  // along n
  if (c >= k || r >= ld) return;  // k and ld are multiples of 8
  uint32_t row[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4 v = r + i < n ? *reinterpret_cast<const uint4*>(w + (r + i) * k + c) : make_uint4(0u, 0u, 0u, 0u);
    row[i][0] = v.x;
    row[i][1] = v.y;
    row[i][2] = v.z;
    row[i][3] = v.w;
  }
  store_columns(row, dst + c * ld + r, ld);
}

__global__ __launch_bounds__(kThreads) void pad_rows(const uint16_t* __restrict__ src, int64_t m, int64_t n,
                                                     uint16_t* __restrict__ dst, int64_t ld) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < m * ld; i += (int64_t)gridDim.x * kThreads) {
    const int64_t c = i % ld;
    dst[i] = c < n ? src[i / ld * n + c] : (uint16_t)0;
  }
}

}  // namespace

namespace {

constexpr int kShortTokens = 64;  // of backward_short

template <int GS>
hipError_t short_of(int tiles, dim3 grid, const uint16_t* dy, int64_t ldy, const uint32_t* packed,
                    const uint32_t* sign, const float* scale, const uint16_t* scale16, int m, int n, int n_read,
                    int k, const Levels& lv, int rows, void* out, int bf16, float* part, hipStream_t stream) {
  auto kernel = tiles == 1   ? backward_short<1, GS>
                : tiles == 2 ? backward_short<2, GS>
                : tiles == 4 ? backward_short<4, GS>
                : tiles == 8 ? backward_mid<1, GS>
                : tiles == 16 ? backward_mid<2, GS>
                : tiles == 24 ? backward_mid<3, GS>
                              : backward_mid<4, GS>;
  hipLaunchKernelGGL(kernel, grid, dim3(tiles > 4 ? kMidThreads : kThreads), 0, stream, dy, ldy, packed, sign, scale, scale16, m, n, n_read, k,
                     lv, rows, out, bf16, part);
  return hipGetLastError();
}

}  // namespace

// Slices of about 512 workgroups in all (up to 256 of the larger kernel's, which fill a CU: 128 take
// 40 us and 512 34, for 34, at 333 tokens of 3840 x 3840; 93 and 84, for 64, at 11520 x 3840), each of
// at least 256 rows, their sums at most 64 MB.
BackwardShort backward_short_plan(int64_t m, int64_t n, int64_t k) {
  BackwardShort p{};
  p.taken = m > 0 && n > 0 && m <= kBackwardShortTokens;
  if (!p.taken) return p;
  const bool mid = m > kShortTokens;
  const int64_t groups = (k + 127) / 128;
  int64_t s = std::min(mid ? std::max<int64_t>(1, 256 / groups) : (512 + groups - 1) / groups, (n + 255) / 256);
  s = std::max<int64_t>(1, std::min<int64_t>(s, (int64_t(64) << 20) / (m * k * 4)));
  p.rows = ((n + s - 1) / s + 255) / 256 * 256;
  p.slices = (n + p.rows - 1) / p.rows;
  p.part_bytes = p.slices > 1 ? (size_t)p.slices * m * k * 4 : 0;
  return p;
}

hipError_t launch_backward_short(const uint16_t* dy, int64_t ldy, const uint32_t* packed, const uint32_t* sign,
                                 const float* scale, const uint16_t* scale16, int64_t m, int64_t n, int64_t k,
                                 int gs, const Levels& lv, void* out, bool bf16, float* part, hipStream_t stream) {
  const BackwardShort p = backward_short_plan(m, n, k);
  const int tiles = m <= 16 ? 1 : m <= 32 ? 2 : m <= kShortTokens ? 4 : m <= 128 ? 8 : m <= 256 ? 16 : m <= 384 ? 24 : 32;
  const dim3 grid((unsigned)((k + 127) / 128), (unsigned)p.slices);
  const int n_read = (int)(ldy > n ? ldy : n);  // dy's rows are zeros past n where they are longer
  if (p.slices == 1) part = nullptr;
  hipError_t e = hipErrorInvalidValue;
#define OPQ_SHORT(G)                                                                                        \
  case G:                                                                                                   \
    e = short_of<G>(tiles, grid, dy, ldy, packed, sign, scale, scale16, (int)m, (int)n, n_read, (int)k, lv, \
                    (int)p.rows, out, (int)bf16, part, stream);                                             \
    break;
  switch (gs) {
    OPQ_SHORT(0)
    OPQ_SHORT(32)
    OPQ_SHORT(64)
    OPQ_SHORT(128)
    OPQ_SHORT(256)
  }
#undef OPQ_SHORT
  if (e != hipSuccess || !part) return e;
  return launch_split_sums(part, (int)p.slices, m, k, out, bf16, stream);
}

hipError_t launch_dequantize_transposed(const uint32_t* packed, const uint32_t* sign, const float* scale,
                                        const uint16_t* scale16, int64_t n, int64_t k, int gs, const Levels& lv,
                                        uint16_t* dst, int64_t ld, hipStream_t stream) {
  const int rows = (int)((ld + 63) / 64), wide = (int)((k + 1023) / 1024);
  // group form: a workgroup makes the significand table once and goes on with it
  const int blocks = gs ? std::min(rows * wide, 1024) : rows * wide;
#define OPQ_TRANSPOSED(G)                                                                                   \
  hipLaunchKernelGGL(dequantize_transposed<G>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, packed, sign, \
                     scale, scale16, n, (int)k, lv, dst, ld, rows, wide);                                   \
  break
  switch (gs) {
    case 0: OPQ_TRANSPOSED(0);
    case 32: OPQ_TRANSPOSED(32);
    case 64: OPQ_TRANSPOSED(64);
    case 128: OPQ_TRANSPOSED(128);
    case 256: OPQ_TRANSPOSED(256);
    default: return hipErrorInvalidValue;
  }
#undef OPQ_TRANSPOSED
  return hipGetLastError();
}

hipError_t launch_transpose(const uint16_t* w, int64_t n, int64_t k, uint16_t* dst, int64_t ld,
                            hipStream_t stream) {
  const dim3 grid((unsigned)((k + 63) / 64), (unsigned)((ld + 255) / 256));
  hipLaunchKernelGGL(transpose_bf16, grid, dim3(kThreads), 0, stream, w, n, k, dst, ld);
  return hipGetLastError();
}

hipError_t launch_pad_rows(const uint16_t* src, int64_t m, int64_t n, uint16_t* dst, int64_t ld,
                           hipStream_t stream) {
  const int64_t blocks = (m * ld + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(pad_rows, dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(kThreads), 0, stream,
                     src, m, n, dst, ld);
  return hipGetLastError();
}

}  // namespace opq
