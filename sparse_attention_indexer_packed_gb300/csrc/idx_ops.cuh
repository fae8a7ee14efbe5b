// Declarations shared by the store of keys and values, the norm and the C ABI
// layer: argument blocks, and the e4m3 rule with one fp32 scale a group.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace idx {

// e4m3 with a scale: a = max(max |x|, 2^-96); scale = a / 448; code =
// e4m3(x * (448 * (1 / a))).  The floor keeps 1 / a finite and the scale a normal
// number; a group below it (all zeros, above all) gets small or zero codes.
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 1.262177448e-29f;  // 2^-96
constexpr int kMaxNormDim = 32768;

// max that keeps a NaN
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 448 * (1 / a), each step rounded once
__device__ __forceinline__ float e4m3_up(float a) { return __fmul_rn(kE4m3Max, __frcp_rn(a)); }

// Two e4m3 codes, round to nearest even, saturating at 448: lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

struct NormArgs {
  const uint16_t* x;         // bf16 [rows][dim], x_stride elements between rows
  const uint16_t* residual;  // bf16, residual_stride between rows; or nullptr
  const uint16_t* weight;    // bf16 [dim]
  uint8_t* out;              // e4m3 [rows][dim]
  float* out_scale;          // [rows][groups]
  uint16_t* out_residual;    // bf16 [rows][dim] or nullptr
  long long rows, x_stride, residual_stride;
  int dim, group;            // group: 128, or 0 for the whole row
  float eps;
};
cudaError_t launch_add_rmsnorm(const NormArgs& args, cudaStream_t stream);

struct StoreArgs {
  const uint16_t* src[2];    // bf16 keys / values [tokens][heads][128]
  long long stride[2];       // elements between tokens
  uint8_t* payload[2];
  float* scale[2];
  const int64_t* slots;      // [tokens]: page * 64 + offset
  long long tokens, num_slots;
  int heads, planes;
};
cudaError_t launch_store_kv(int key_format, const StoreArgs& args, cudaStream_t stream);

}  // namespace idx
