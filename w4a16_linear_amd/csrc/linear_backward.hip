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
      }
    }
    if constexpr (GS == 0) {
      // entry q of row t / 4 as bytes of the planes: thread t makes q = 4 (t % 4) ...
      const int t = threadIdx.x, j = t & 3;
      const float top = scale[min(row0 + (t >> 2), n - 1)];
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
