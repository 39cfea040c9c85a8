// row_stream.h - products of few rows with weights that stream from memory once: the part that
// the MoE layer for few tokens (few_tokens.hip) and the dense product (linear.hip) share.
//
// A wave multiplies 16 weight rows with up to 64 token rows over a range of K. Weights go
// straight from memory to the registers of the lane that multiplies them - no other wave wants
// them - and feed a matrix instruction's first operand; the token rows, few and in cache, feed
// its second. Lane l = 16 q + r holds weight row r and token row r; of every block of K elements
// it takes the q-th quarter, a contiguous run of 32 bytes of 8-bit weights or more. Both
// operands number K alike, so that the instruction's own order does not matter. Results: lane
// 16 q + r holds weight rows 4 q .. 4 q + 3 of token r.
#pragma once

#include "layer_common.h"

namespace mgg_layer {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

enum WeightForm { kBf16Weights, kFp8Weights, kFp4Weights, kF32Weights };
enum ScaleForm { kNoScales, kF32Scales, kByteScales };
enum ScaleSpan { kPerBlock, kPerChannel };  // FP8: 128 x 128 weights or 1 x 128 to a scale

// What a weight element's storage means: K elements to a block and to a lane's run of it.
template <WeightForm W>
struct Form {
  static constexpr int BLOCK = W == kF32Weights ? 32 : W == kBf16Weights ? 64 : 128;
  static constexpr int RUN = BLOCK / 4;
  static constexpr int RUN_BYTES = W == kFp4Weights ? 16 : 32;
  static constexpr int LOADS = RUN_BYTES / 16;
  static constexpr int X_BYTES = W == kF32Weights ? 32 : RUN * 2;  // the run of a token row
  static constexpr int X_LOADS = X_BYTES / 16;
};
__host__ __device__ constexpr int block_elements(WeightForm w) {
  return w == kF32Weights ? 32 : w == kBf16Weights ? 64 : 128;
}

__device__ __forceinline__ float byte_scale(uint32_t u) {  // 2^(u - 127); 255: NaN
  return __uint_as_float(u == 0 ? 0x00400000u : u == 255 ? 0x7fc00000u : u << 23);
}

__device__ __forceinline__ uint4 load16(const void* p) {  // any alignment
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// The first `bytes` of up to 16 at p, zeros behind them.
template <int ELEM>
__device__ __forceinline__ uint4 load16_part(const void* p, int bytes) {
  uint32_t w[4] = {0, 0, 0, 0};
  if constexpr (ELEM == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * i < bytes) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (2 * i < bytes)
        w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's view of its operands, at K = 0 of its own run.
template <int RT>
struct StreamRows {
  const uint8_t* w;             // its weight row
  const void* scale;            // FP8: of its result rows; FP4: of its weight row
  int64_t scale_step;           // elements from one block of 128 K to the next
  const uint8_t* x[RT];         // its token rows; null: no row, zeros
  const uint8_t* x_low[RT];     // the low halves of token rows held as two bfloat16
};

// One block of K in registers.
template <WeightForm W, int RT, bool LOW>
struct StreamBlock {
  uint4 w[Form<W>::LOADS];
  float scale[4];
  uint32_t scale_bits;
  uint4 x[RT][Form<W>::X_LOADS];
  uint4 x_low[LOW ? RT : 1][Form<W>::X_LOADS];
};

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int RT, bool LOW>
__device__ __forceinline__ void load_block(StreamBlock<W, RT, LOW>& b, const StreamRows<RT>& rows,
                                           int block, int K) {
  using F = Form<W>;
  const int q = (threadIdx.x >> 4) & 3;
  const int64_t w_at = (int64_t)block * (4 * F::RUN_BYTES), x_at = (int64_t)block * (4 * F::X_BYTES);
  // FP8 and FP4 rows are whole blocks; the others may end inside one
  constexpr bool TAIL = W == kBf16Weights || W == kF32Weights;
  constexpr int ELEM = W == kF32Weights ? 4 : 2;
  if (!TAIL || (block + 1) * F::BLOCK <= K) {
#pragma unroll
    for (int i = 0; i < F::LOADS; ++i) b.w[i] = load16(rows.w + w_at + 16 * i);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < F::X_LOADS; ++i) {
        b.x[t][i] = make_uint4(0, 0, 0, 0);
        if (rows.x[t]) b.x[t][i] = load16(rows.x[t] + x_at + 16 * i);
        if constexpr (LOW) {
          b.x_low[t][i] = make_uint4(0, 0, 0, 0);
          if (rows.x[t]) b.x_low[t][i] = load16(rows.x_low[t] + x_at + 16 * i);
        }
      }
  } else {
    const int left = (K - block * F::BLOCK - q * F::RUN) * ELEM;  // bytes of its run that exist
#pragma unroll
    for (int i = 0; i < F::LOADS; ++i)
      b.w[i] = load16_part<ELEM>(rows.w + w_at + 16 * i, left - 16 * i);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < F::X_LOADS; ++i) {
        b.x[t][i] = make_uint4(0, 0, 0, 0);
        if (rows.x[t]) b.x[t][i] = load16_part<ELEM>(rows.x[t] + x_at + 16 * i, left - 16 * i);
        if constexpr (LOW) {
          b.x_low[t][i] = make_uint4(0, 0, 0, 0);
          if (rows.x[t])
            b.x_low[t][i] = load16_part<ELEM>(rows.x_low[t] + x_at + 16 * i, left - 16 * i);
        }
      }
  }
  if constexpr (W == kFp4Weights) {
    b.scale_bits = reinterpret_cast<const uint8_t*>(rows.scale)[block * rows.scale_step];
  } else if constexpr (W == kFp8Weights) {
    const int64_t at = block * rows.scale_step;
    if constexpr (SF == kF32Scales) {
      const float* s = reinterpret_cast<const float*>(rows.scale) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) b.scale[i] = s[SPAN == kPerChannel ? i : 0];
    } else {
      const uint8_t* s = reinterpret_cast<const uint8_t*>(rows.scale) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) b.scale[i] = byte_scale(s[SPAN == kPerChannel ? i : 0]);
    }
  }
}

__device__ __forceinline__ v8bf as_bf16(const uint4& v) { return __builtin_bit_cast(v8bf, v); }

// Eight E4M3 codes as bfloat16, exactly.
__device__ __forceinline__ v8bf from_e4m3(uint32_t a, uint32_t b) {
  uint4 v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true));
  v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false));
  v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true));
  return as_bf16(v);
}

// Eight E2M1 codes times a power of two as bfloat16, exactly (beyond bfloat16's largest: infinite).
__device__ __forceinline__ v8bf from_e2m1(uint32_t a, float scale) {
  uint4 v;
  v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 0));
  v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 1));
  v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 2));
  v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, scale, 3));
  return as_bf16(v);
}

// acc += the block's products. FP8 scales multiply each block's float32 sum; FP4 scales, powers
// of two, go into the conversion.
template <WeightForm W, int RT, bool LOW>
__device__ __forceinline__ void multiply_block(const StreamBlock<W, RT, LOW>& b, v4f (&acc)[RT]) {
  using F = Form<W>;
  if constexpr (W == kF32Weights) {
    float w[8];
    __builtin_memcpy(w, b.w, 32);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float x[8];
      __builtin_memcpy(x, b.x[t], 32);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i], x[i], acc[t], 0, 0, 0);
    }
  } else {
    v8bf w[F::X_LOADS];
    if constexpr (W == kBf16Weights) {
#pragma unroll
      for (int i = 0; i < F::X_LOADS; ++i) w[i] = as_bf16(b.w[i]);
    } else if constexpr (W == kFp8Weights) {
      const uint32_t* c = reinterpret_cast<const uint32_t*>(b.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = from_e4m3(c[2 * i], c[2 * i + 1]);
    } else {
      const uint32_t* c = reinterpret_cast<const uint32_t*>(b.w);
      // 255 (NaN) and 0 (2^-127) go through the exponent field as they are
      const float scale = __uint_as_float(b.scale_bits << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = from_e2m1(c[i], scale);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      v4f sum = W == kFp8Weights ? v4f{0.f, 0.f, 0.f, 0.f} : acc[t];
#pragma unroll
      for (int i = 0; i < F::X_LOADS; ++i) {
        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], as_bf16(b.x[t][i]), sum, 0, 0, 0);
        if constexpr (LOW)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], as_bf16(b.x_low[t][i]), sum, 0, 0, 0);
      }
      if constexpr (W == kFp8Weights) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(sum[e], b.scale[e], acc[t][e]);
      } else {
        acc[t] = sum;
      }
    }
  }
}

// acc += products over the blocks [from, to) of K elements.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int RT, bool LOW>
__device__ __forceinline__ void stream_rows(const StreamRows<RT>& rows, int from, int to, int K,
                                            v4f (&acc)[RT]) {
  for (int b = from; b < to; ++b) {
    StreamBlock<W, RT, LOW> block;
    load_block<W, SF, SPAN>(block, rows, b, K);
    multiply_block<W, RT, LOW>(block, acc);
  }
}

}  // namespace mgg_layer
