// linear_common.h - what the parts of the dense products share (linear.hip, linear_forward.hip,
// linear_backward.hip): the epilogue's arithmetic, and what a product in tiles is asked for with.
#pragma once

#include "mgg/linear.h"

#include "linear_tile.h"
#include "row_stream.h"

namespace mgg_dense {

constexpr int kMaxSide = 1 << 20;

// ---------------------------------------------------------------------------- epilogue

struct Emit {
  void* out;
  const void* bias;
  const void* residual;
  int64_t ld_res;
  void* z;
  int rows;         // of the output
  int N, C;         // columns of z and of the output
  mgg_func func;
  bool out_f32, bias_f32, z_f32;
};

// Up to V elements from `at` on, `n` of which exist; their order in memory is the vector's.
template <int V>
__device__ __forceinline__ void load_values(const void* p, bool f32, int64_t at, int n,
                                            float (&v)[V]) {
  if (f32) {
    const float* s = reinterpret_cast<const float*>(p) + at;
    if (n >= V) {
      __builtin_memcpy(v, s, 4 * V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = i < n ? s[i] : 0.f;
    }
  } else {
    const bf16_t* s = reinterpret_cast<const bf16_t*>(p) + at;
    bf16_t b[V];
    if (n >= V) {
      __builtin_memcpy(b, s, 2 * V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = i < n ? s[i] : bf16_t{0};
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(b[i]);
  }
}

template <int V>
__device__ __forceinline__ void store_values(void* p, bool f32, int64_t at, int n,
                                             const float (&v)[V]) {
  if (f32) {
    float* s = reinterpret_cast<float*>(p) + at;
    if (n >= V) {
      __builtin_memcpy(s, v, 4 * V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) s[i] = v[i];
    }
  } else {
    __bf16* s = reinterpret_cast<__bf16*>(p) + at;
    __bf16 b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = (__bf16)v[i];  // one instruction rounds two to nearest even
    if (n >= V) {
      __builtin_memcpy(s, b, 2 * V);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) s[i] = b[i];
    }
  }
}

// The normal distribution's tail Phi(-a) = t q(t) e^(-a^2 / 2) for a >= 0, with t = 1 / (1 + a / 4)
// and q the polynomial of degree 9 nearest to erfcx(a / sqrt 2) / (2 t) on (0, 1] in relative error
// (a least-squares fit in Chebyshev polynomials, reweighted until its errors were level: 3.4e-8);
// in float32 it is within 7 roundings, and those of the exponential's argument. A fit in a itself
// or by erfc of the device library takes several times the instructions and registers.
__device__ __forceinline__ float normal_tail(float a, float exponential) {
  const float t = reciprocal(fmaf(a, 0.25f, 1.f));
  float q = 0.019782206f;
  q = fmaf(q, t, -0.080878088f);
  q = fmaf(q, t, 0.095598333f);
  q = fmaf(q, t, -0.031718582f);
  q = fmaf(q, t, 0.063699625f);
  q = fmaf(q, t, 0.058975011f);
  q = fmaf(q, t, 0.081603132f);
  q = fmaf(q, t, 0.093466356f);
  q = fmaf(q, t, 0.09973643f);
  q = fmaf(q, t, 0.099735565f);
  return q * t * exponential;
}
// Phi(v), and e^(-v^2 / 2).
__device__ __forceinline__ float normal_cdf(float v, float& exponential) {
  exponential = exp_neg(-0.5f * v * v);
  const float tail = normal_tail(fabsf(v), exponential);
  return v >= 0.f ? 1.f - tail : tail;
}

__device__ __forceinline__ float sigmoid(float v) {
  float q, rest;
  sigmoid_parts(v, q, rest);
  return q;
}

__device__ __forceinline__ float func_of(mgg_func f, float z) {
  switch (f) {
    case MGG_FUNC_RELU: return z > 0.f ? z : z != z ? z : 0.f;  // NaN stays
    case MGG_FUNC_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case MGG_FUNC_SILU: return z * sigmoid(z);
    default: return z;
  }
}

// V consecutive columns n .. of row m: z (and of the pair `u`, up, for the gated unit) without bias
// in, outputs stored.
template <int V, bool PAIRS>
__device__ __forceinline__ void emit(const Emit& e, int64_t m, int n, float (&v)[V],
                                     float (&u)[PAIRS ? V : 1]) {
  const int have = e.C - n;
  if (m >= e.rows || have <= 0) return;
  float t[V];
  if (e.bias) {
    load_values<V>(e.bias, e.bias_f32, n, have, t);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += t[i];
    if constexpr (PAIRS) {
      load_values<V>(e.bias, e.bias_f32, e.C + n, have, t);
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] += t[i];
    }
  }
  if (e.z) {
    store_values<V>(e.z, e.z_f32, m * e.N + n, have, v);
    if constexpr (PAIRS) store_values<V>(e.z, e.z_f32, m * e.N + e.C + n, have, u);
  }
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
  } else if (e.func != MGG_FUNC_NONE) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = func_of(e.func, v[i]);
  }
  if (e.residual) {
    load_values<V>(e.residual, e.out_f32, m * e.ld_res + n, have, t);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += t[i];
  }
  store_values<V>(e.out, e.out_f32, m * e.C + n, have, v);
}

// ------------------------------------------------------------------------------- tiles

// Which tiles a launch has: `whole` of them one to a workgroup at a time, the rest cut along K into
// `parts` of `part_k`, whose sums go to the workspace and are joined by a second kernel.
struct Deal {
  int tiles_m, tiles_n, whole, parts, part_k;
  __host__ __device__ int tiles() const { return tiles_m * tiles_n; }
  __host__ __device__ int items() const { return whole + (tiles() - whole) * parts; }
};

struct TileArgs {
  Side x, w;
  int64_t second;  // bytes from a gate row of w to its up row
  int K;
  Deal deal;
  float* sums;     // [rest][parts][waves][blocks][4][64] of four floats
  Emit e;
};

constexpr int kCus = 256;

// Whether tiles take a matrix as it lies: whole aligned pieces of 16 bytes, rows whose
// distances stay below 2 GiB within a tile.
inline bool in_pieces(const void* p, int64_t ld, int cols, size_t elem) {
  return aligned(p, 16) && ld * (int64_t)elem % 16 == 0 && cols * elem % 16 == 0 && ld <= kMaxSide;
}

enum FormName { kLarge, kSmall, kNarrow };

struct Product {
  FormName form;
  Deal deal;
  size_t bytes;   // of the parts' sums
  bool counted;   // false: more tiles than an int counts
};

// Enqueues the product; its instantiations are in linear_forward.hip and linear_backward.hip.
template <bool F32, bool TURN_X, bool TURN_W, bool PAIRS>
mgg_status run_product(const Product& p, TileArgs a, hipStream_t stream)
    __attribute__((visibility("hidden")));

}  // namespace mgg_dense
