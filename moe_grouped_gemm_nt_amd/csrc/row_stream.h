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

// One block of K in registers: a lane's weights and the scales that go with them, and its runs of
// token rows.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN>
struct WeightBlock {
  static constexpr int SCALES = W == kFp8Weights && SF == kF32Scales && SPAN == kPerChannel ? 4 : 1;
  uint4 w[Form<W>::LOADS];
  uint32_t scale[SCALES];  // as stored; the bytes of four rows in one word
};
// A token row may be the sum of PLANES rows of bfloat16.
template <WeightForm W, int RT, int PLANES>
struct TokenBlock {
  uint4 x[PLANES][RT][Form<W>::X_LOADS];
};

// FP8 and FP4 rows are whole blocks of K; the others may end inside one.
template <WeightForm W>
struct Tail {
  static constexpr bool POSSIBLE = W == kBf16Weights || W == kF32Weights;
  static constexpr int ELEM = W == kF32Weights ? 4 : 2;
  // whether block `block` is whole, and else how many bytes of the lane's run exist
  static __device__ __forceinline__ bool whole(int block, int K) {
    return !POSSIBLE || (block + 1) * Form<W>::BLOCK <= K;
  }
  static __device__ __forceinline__ int left(int block, int K) {
    const int q = (threadIdx.x >> 4) & 3;
    return (K - block * Form<W>::BLOCK - q * Form<W>::RUN) * ELEM;
  }
};

// A piece of a run that may end in it, `left` bytes from its start. PIECES: rows are whole pieces.
template <WeightForm W, bool PIECES>
__device__ __forceinline__ uint4 load_end(const uint8_t* p, int left) {
  if constexpr (PIECES) return left >= 16 ? load16(p) : make_uint4(0, 0, 0, 0);
  else return load16_part<Tail<W>::ELEM>(p, left);
}

// `w`, `scale`: the lane's weight row at K = 0 of its own run, and its scales there.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, bool PIECES>
__device__ __forceinline__ void load_weights(WeightBlock<W, SF, SPAN>& b, const uint8_t* w,
                                             const void* scale, int64_t scale_step, int block,
                                             int K) {
  using F = Form<W>;
  w += (int64_t)block * (4 * F::RUN_BYTES);
  if (Tail<W>::whole(block, K)) {
#pragma unroll
    for (int i = 0; i < F::LOADS; ++i) b.w[i] = load16(w + 16 * i);
  } else {
    const int left = Tail<W>::left(block, K);
#pragma unroll
    for (int i = 0; i < F::LOADS; ++i)
      b.w[i] = load_end<W, PIECES>(w + 16 * i, left - 16 * i);
  }
  if constexpr (W == kFp8Weights || W == kFp4Weights) {
    constexpr int BYTES = SF == kF32Scales ? 4 : 1;
    const uint8_t* s = reinterpret_cast<const uint8_t*>(scale) + block * scale_step * BYTES;
    b.scale[0] = 0;
    __builtin_memcpy(b.scale, s, W == kFp8Weights && SPAN == kPerChannel ? 4 * BYTES : BYTES);
  }
}

// A run of a token row at block `block`; a null row is zeros.
template <WeightForm W, bool PIECES>
__device__ __forceinline__ void load_tokens(uint4 (&x)[Form<W>::X_LOADS], const uint8_t* row,
                                            int block, int K) {
  using F = Form<W>;
#pragma unroll
  for (int i = 0; i < F::X_LOADS; ++i) x[i] = make_uint4(0, 0, 0, 0);
  if (!row) return;
  row += (int64_t)block * (4 * F::X_BYTES);
  if (Tail<W>::whole(block, K)) {
#pragma unroll
    for (int i = 0; i < F::X_LOADS; ++i) x[i] = load16(row + 16 * i);
  } else {
    const int left = Tail<W>::left(block, K);
#pragma unroll
    for (int i = 0; i < F::X_LOADS; ++i)
      x[i] = load_end<W, PIECES>(row + 16 * i, left - 16 * i);
  }
}

// Scale of the lane's i-th result row (FP8).
template <ScaleForm SF, ScaleSpan SPAN, class Block>
__device__ __forceinline__ float scale_of(const Block& b, int i) {
  if constexpr (SF == kF32Scales) return __uint_as_float(b.scale[SPAN == kPerChannel ? i : 0]);
  return byte_scale(b.scale[0] >> (SPAN == kPerChannel ? 8 * i : 0) & 255);
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

// A block's weights as the first operands of its matrix instructions (8- and 4-bit forms: exactly;
// FP4 scales, powers of two, go into the conversion).
template <WeightForm W, class Block>
__device__ __forceinline__ void operands_of(const Block& b, v8bf (&w)[Form<W>::X_LOADS]) {
  using F = Form<W>;
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
    const float scale = __uint_as_float(b.scale[0] << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = from_e2m1(c[i], scale);
  }
}

// acc += the block's products. FP8 scales multiply each block's float32 sum. `x(p, t, i)` is the i-th
// 16 bytes of the lane's run of plane p of its t-th token row.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int RT, int PLANES, class Block, class X>
__device__ __forceinline__ void multiply_block(const Block& b, v4f (&acc)[RT], X x) {
  using F = Form<W>;
  if constexpr (W == kF32Weights) {
    float w[8];
    __builtin_memcpy(w, b.w, 32);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4f v = __builtin_bit_cast(v4f, x(0, t, h));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[4 * h + i], v[i], acc[t], 0, 0, 0);
      }
  } else {
    v8bf w[F::X_LOADS];
    operands_of<W>(b, w);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      v4f sum = W == kFp8Weights ? v4f{0.f, 0.f, 0.f, 0.f} : acc[t];
#pragma unroll
      for (int p = 0; p < PLANES; ++p)
#pragma unroll
        for (int i = 0; i < F::X_LOADS; ++i)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], as_bf16(x(p, t, i)), sum, 0, 0, 0);
      if constexpr (W == kFp8Weights) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[t][e] = fmaf(sum[e], scale_of<SF, SPAN>(b, e), acc[t][e]);
      } else {
        acc[t] = sum;
      }
    }
  }
}

// acc += products over the blocks [from, to) of K elements, token rows from memory. AHEAD blocks
// are on their way at a time: loads return in the order in which they were issued, so a block's
// token rows are asked for together with its weights.
template <WeightForm W, int RT, int AHEAD>
__device__ __forceinline__ void stream_rows(const uint8_t* w, const uint8_t* const (&x)[RT],
                                            int from, int to, int K, v4f (&acc)[RT]) {
  WeightBlock<W, kNoScales, kPerBlock> weights[AHEAD];
  TokenBlock<W, RT, 1> tokens[AHEAD];
  auto load = [&](int i, int b) {
    load_weights<W, kNoScales, kPerBlock, false>(weights[i], w, nullptr, 0, b, K);
#pragma unroll
    for (int t = 0; t < RT; ++t) load_tokens<W, false>(tokens[i].x[0][t], x[t], b, K);
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (from + i < to) load(i, from + i);
  for (int b = from; b < to; b += AHEAD)
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (b + i < to) {
        auto x_of = [&](int, int t, int j) { return tokens[i].x[0][t][j]; };
        multiply_block<W, kNoScales, kPerBlock, RT, 1>(weights[i], acc, x_of);
        if (b + i + AHEAD < to) load(i, b + i + AHEAD);
      }
}

}  // namespace mgg_layer
