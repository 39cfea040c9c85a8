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

constexpr int kMaxRows = 1 << 30;  // row numbers plus a grid's worth of rows stay below 2^31

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
__host__ __device__ constexpr int cdiv(int a, int b) { return (a + b - 1) / b; }

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

// e^x for x <= 0 (0 for -inf, NaN for NaN), as 2^(x log2 e): the product's rounding is a relative
// error of |x| 2^-24, the same as that of the difference that x usually is.
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504f);
}

// 1 / x to within one unit in the last place, for x in a float's normal range.
__device__ __forceinline__ float reciprocal(float x) { return __builtin_amdgcn_rcpf(x); }

// sigmoid(v) and 1 - sigmoid(v), each to the relative precision of exp_neg.
__device__ __forceinline__ void sigmoid_parts(float v, float& q, float& one_minus_q) {
  const float a = exp_neg(-fabsf(v)), r = reciprocal(1.f + a);
  q = v >= 0.f ? r : a * r;
  one_minus_q = v >= 0.f ? a * r : r;
}

// op of the lane's own value and its partner's, OFF = 1, 2, 4, 8, 16 or 32 lanes away, for a
// commutative op. The partner is lane ^ OFF for 1, 2, 16 and 32, and the mirrored lane of its
// eight or sixteen for 4 and 8: the same thing once a reduction has made smaller groups of lanes
// equal. These are lane permutations of the vector unit; a shuffle goes through LDS and takes
// many times as long.
template <int OFF>
__device__ __forceinline__ void pair_bits(uint32_t v, uint32_t& a, uint32_t& b) {
  if constexpr (OFF == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0], b = r[1];
  } else if constexpr (OFF == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0], b = r[1];
  } else {
    // quad_perm [1,0,3,2], quad_perm [2,3,0,1], row_half_mirror, row_mirror
    constexpr int CTRL = OFF == 1 ? 0xb1 : OFF == 2 ? 0x4e : OFF == 4 ? 0x141 : 0x140;
    a = v, b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
  }
}
template <int OFF, class T, class Op>
__device__ __forceinline__ T with_partner(T v, Op op) {
  if constexpr (sizeof(T) == 4) {
    uint32_t a, b;
    pair_bits<OFF>(__builtin_bit_cast(uint32_t, v), a, b);
    return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  } else {
    const uint64_t bits = __builtin_bit_cast(uint64_t, v);
    uint32_t al, bl, ah, bh;
    pair_bits<OFF>((uint32_t)bits, al, bl);
    pair_bits<OFF>((uint32_t)(bits >> 32), ah, bh);
    return op(__builtin_bit_cast(T, al | (uint64_t)ah << 32),
              __builtin_bit_cast(T, bl | (uint64_t)bh << 32));
  }
}

// Sum, or another associative and commutative operation, over the L lanes (a power of two up to
// 64) that share a row; every lane gets the same result.
template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
  if constexpr (L > 1) v = with_partner<1>(v, op);
  if constexpr (L > 2) v = with_partner<2>(v, op);
  if constexpr (L > 4) v = with_partner<4>(v, op);
  if constexpr (L > 8) v = with_partner<8>(v, op);
  if constexpr (L > 16) v = with_partner<16>(v, op);
  if constexpr (L > 32) v = with_partner<32>(v, op);
  return v;
}
template <int L, class T>
__device__ __forceinline__ T lanes_sum(T v) {
  return lanes_reduce<L>(v, [](T a, T b) { return a + b; });
}

// Inclusive prefix sum over the L lanes that share a row.
template <int L>
__device__ __forceinline__ int lanes_prefix(int v) {
  static_assert(L >= 16, "whole rows of 16 lanes");
  // row_shr 1, 2, 4, 8: zeros come in from outside the 16 lanes
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  const int lane = threadIdx.x & 63;
  if constexpr (L >= 32) {
    const int before = __shfl(v, (lane & 32) + 15, 64);
    v += (lane & 16) ? before : 0;
  }
  if constexpr (L >= 64) {
    const int before = __shfl(v, 31, 64);
    v += (lane & 32) ? before : 0;
  }
  return v;
}

// LDS accesses of a wave take effect in program order; this keeps the program's order where
// lanes of one wave exchange values through LDS without a barrier.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace mgg_layer
