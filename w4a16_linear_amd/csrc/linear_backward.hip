// The parts of the gradient through a quantized projection that are its own: the dense
// product contracts along the weights' rows, and its operand has that dimension dense.
#include "adapters_internal.hpp"
#include "device_common.hpp"

namespace opq {
namespace {

constexpr int kThreads = 256;

// dst [k][ld] = w [n][k] transposed, columns n..ld-1 zero.  A lane turns an 8 x 8 block in
// registers (v_perm pairs rows); the eight lanes of a row of blocks read, and the
// eight of a column write, 128 bytes in a row.
__global__ __launch_bounds__(kThreads) void transpose_bf16(const uint16_t* __restrict__ w, int64_t n, int64_t k,
                                                           uint16_t* __restrict__ dst, int64_t ld) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t c = (int64_t)blockIdx.x * 64 + (lane & 7) * 8;                       // along k
  const int64_t r = ((int64_t)blockIdx.y * (kThreads / kWave) + wave) * 64 + (lane >> 3) * 8;  // along n
  if (c >= k || r >= ld) return;  // k and ld are multiples of 8
  uint4 row[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    row[i] = r + i < n ? *reinterpret_cast<const uint4*>(w + (r + i) * k + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = q == 0 ? row[2 * i].x : q == 1 ? row[2 * i].y : q == 2 ? row[2 * i].z : row[2 * i].w;
      const uint32_t b = q == 0 ? row[2 * i + 1].x : q == 1 ? row[2 * i + 1].y : q == 2 ? row[2 * i + 1].z : row[2 * i + 1].w;
      lo[i] = __builtin_amdgcn_perm(b, a, 0x05040100u);
      hi[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    }
    *reinterpret_cast<uint4*>(dst + (c + 2 * q) * ld + r) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(dst + (c + 2 * q + 1) * ld + r) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

__global__ __launch_bounds__(kThreads) void pad_rows(const uint16_t* __restrict__ src, int64_t m, int64_t n,
                                                     uint16_t* __restrict__ dst, int64_t ld) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < m * ld; i += (int64_t)gridDim.x * kThreads) {
    const int64_t c = i % ld;
    dst[i] = c < n ? src[i / ld * n + c] : (uint16_t)0;
  }
}

}  // namespace

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
