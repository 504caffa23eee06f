// Internal interface between the C ABI of the adapters (adapters_api.cpp) and
// their kernel launchers.  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "opq_adapters.h"
#include "opq_internal.hpp"

namespace opq {

// lowrank.hip
struct LowrankAdd {
  opq_lowrank a;
  const uint16_t* x;
  int64_t x_stride;
  const int32_t* index;
  int64_t m;
  const void* y;  // or nullptr
  int64_t y_stride;
  bool y_bf16;
  void* out;
  int64_t out_stride;
  bool out_bf16;
  void* workspace;
};
size_t lowrank_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank);
hipError_t launch_lowrank_add(const LowrankAdd& c, hipStream_t stream);

constexpr int64_t kMaxTrained = 1024;  // adapters of a backward pass: its counts are held in LDS
struct LowrankBackward {
  opq_lowrank a;
  const uint16_t* dy;
  int64_t dy_stride;
  const uint16_t* x;
  int64_t x_stride;
  const int32_t* index;
  int64_t m;
  const void* dx;  // or nullptr
  int64_t dx_stride;
  bool dx_bf16;
  void* dx_out;  // or nullptr
  int64_t dx_out_stride;
  void* d_down;  // both or neither
  void* d_up;
  bool grad_bf16;
  void* workspace;
};
size_t lowrank_backward_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank, int64_t count);
hipError_t launch_lowrank_backward(const LowrankBackward& c, hipStream_t stream);

// linear_backward.hip: the gradient of few tokens straight from 4-bit codes.  dy has rows of ldy
// elements, n rounded up to 8 at least, zeros past n; part: the plan's bytes.  Up to 512 tokens,
// the most that one workgroup holds sums of; a call takes (so / W' transposed and the dense product,
// us) at 8, 64, 128, 333 and 512 tokens: 3840 x 3840 16/23, 26/29, 23/42, 34/41, 43/46; 11520 x 3840
// 27/38, 43/51, 44/80, 64/88, 79/92; 20480 x 3840 38/73, 61/95, 67/143, 96/133, 119/142; with fewer
// slices 3840 x 10240 23/38, 41/56, 39/92, 58/101, 72/103; 3840 x 20480 34/68, 67/102, 78/115,
// 111/131, 135/133.  Two workgroups' tokens decode twice: 1024 would take twice the 512, against 60,
// 120 and 217
constexpr int64_t kBackwardShortTokens = 512;
struct BackwardShort {
  bool taken;
  int64_t rows, slices;  // weight rows of a slice
  size_t part_bytes;
};
BackwardShort backward_short_plan(int64_t m, int64_t n, int64_t k);
hipError_t launch_backward_short(const uint16_t* dy, int64_t ldy, const uint32_t* packed, const uint32_t* sign,
                                 const float* scale, const uint16_t* scale16, int64_t m, int64_t n, int64_t k,
                                 int gs, const Levels& lv, void* out, bool bf16, float* part, hipStream_t stream);
// linear.hip: out [m][n] = the sums of `split` float32 planes of `part`, in order
hipError_t launch_split_sums(const float* part, int split, int64_t m, int64_t n, void* out, bool bf16,
                             hipStream_t stream);
// dst [k][ld] = W' (bfloat16) transposed, columns n..ld-1 zero, from 4-bit
// codes with one max a row (gs 0: scale) or a group (scale16)
hipError_t launch_dequantize_transposed(const uint32_t* packed, const uint32_t* sign, const float* scale,
                                        const uint16_t* scale16, int64_t n, int64_t k, int gs, const Levels& lv,
                                        uint16_t* dst, int64_t ld, hipStream_t stream);
// dst [k][ld] = the transpose of w [n][k] (bfloat16), columns n..ld-1 zero
hipError_t launch_transpose(const uint16_t* w, int64_t n, int64_t k, uint16_t* dst, int64_t ld,
                            hipStream_t stream);
// dst [m][ld] = src [m][n], columns n..ld-1 zero
hipError_t launch_pad_rows(const uint16_t* src, int64_t m, int64_t n, uint16_t* dst, int64_t ld,
                           hipStream_t stream);

}  // namespace opq
