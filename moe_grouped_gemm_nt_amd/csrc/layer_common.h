// layer_common.h - what the kernels around the grouped products share (include/mgg/layer_ops.h):
// error text, element conversion, and reductions over groups of lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mgg/layer_ops.h"

// Sets the calling thread's error text (library.hip).
extern "C" void mgg_set_last_error(const char* text) __attribute__((visibility("hidden")));

namespace mgg_layer {

inline mgg_status fail(mgg_status s, const char* text) {
  mgg_set_last_error(text);
  return s;
}

// The status of a call whose kernels have just been enqueued.
inline mgg_status launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MGG_OK : fail(MGG_EHIP, hipGetErrorString(e));
}

inline bool aligned(const void* p, size_t n) { return (uintptr_t)p % n == 0; }
inline size_t elem_bytes(mgg_act dt) { return dt == MGG_ACT_BF16 ? 2 : 4; }
inline bool known(mgg_act dt) { return dt == MGG_ACT_BF16 || dt == MGG_ACT_F32; }
constexpr size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }
constexpr int cdiv(int a, int b) { return (a + b - 1) / b; }

struct bf16_t {
  uint16_t bits;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }

// Round to nearest even; NaN stays a quiet NaN.
__device__ __forceinline__ uint16_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  if (f != f) return 0x7fc0u;
  return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

template <class T>
__device__ __forceinline__ T from_f32(float f);
template <>
__device__ __forceinline__ float from_f32<float>(float f) { return f; }
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float f) { return bf16_t{bf16_bits(f)}; }

// e^x for x <= 0 (NaN stays NaN): 2^(x log2 e) with the rounding of the product put back, so
// that the relative error does not grow with |x|.
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -150.f ? -150.f : x;  // also -inf; e^-150 is below the smallest float
  const float t = x * 1.44269504f;
  const float r = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  return __builtin_amdgcn_exp2f(t) * fmaf(r, 0.69314718f, 1.f);
}

// sigmoid(v) and 1 - sigmoid(v), each to full relative precision.
__device__ __forceinline__ void sigmoid_parts(float v, float& q, float& one_minus_q) {
  const float a = exp_neg(-fabsf(v)), r = 1.f / (1.f + a);
  q = v >= 0.f ? r : a * r;
  one_minus_q = v >= 0.f ? a * r : r;
}

// Sum, or another associative operation, over the L lanes (a power of two up to 64) that
// share a row; every lane gets the result.
template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v = op(v, __shfl_xor(v, off, 64));
  return v;
}
template <int L, class T>
__device__ __forceinline__ T lanes_sum(T v) {
  return lanes_reduce<L>(v, [](T a, T b) { return a + b; });
}

}  // namespace mgg_layer
