// elem_io.cuh -- the element types of the entry points that take a cla_dtype
// (fp32, bf16, fp16): stores from fp32 registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace cla {
namespace {

template <typename E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

}  // namespace

inline size_t dtype_bytes(int dtype) { return dtype == CLA_F32 ? 4 : (dtype == CLA_BF16 || dtype == CLA_F16) ? 2 : 0; }

}  // namespace cla
