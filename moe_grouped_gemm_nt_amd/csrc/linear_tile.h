// linear_tile.h - one output tile of a dense product: operands from memory to LDS, matrix
// instructions, sums in registers. linear.hip makes its three products of it.
//
// C[m][n] = sum_k X(m, k) W(n, k). An operand is "long" when memory holds [row][k] (K
// contiguous) and "turned" when it holds [k][row]:
//   forward  x w^T     both long
//   d_x      dz w      dz long, w turned
//   d_w      dz^T x    both turned
// A slice is SLICE bytes of K of every row: 64 (or 32) bfloat16, half as many float32. Slices go
// straight from memory to a ring of LDS stages; the rows of a long slice are stored one after
// another, the k of a turned one. 16-byte pieces change places by row (long) or 64-byte pieces by k
// (turned) so that the lanes a read serves at once meet different banks; the copies apply that to
// the address they read, as a copy's lanes write consecutive bytes of LDS.
//
// A step is 32 bytes of K of a long row: one 32 x 32 x 16 instruction in bfloat16, four of
// 32 x 32 x 2 in float32 (lanes 0-31 hold the lower half of the step's K, lanes 32-63 the
// upper; both operands number K alike). Turned bfloat16 operands are read by the LDS's
// transposing reads, four k of one row a lane. W's rows are the instruction's first operand, its
// rows permuted so that a lane ends up with 16 consecutive n of one m.
#pragma once

#include "gemm_engine.h"
#include "layer_common.h"

namespace mgg_dense {

using namespace mgg_layer;
using mgg::v16f;
using mgg::v4i;
using mgg::v8bf;
typedef short v4s __attribute__((ext_vector_type(4)));

struct Side {
  const uint8_t* p;
  int64_t ld;   // bytes from one memory row to the next, a multiple of 16
  int rows;     // of this operand, m or n
};

// WI x WJ waves of (32 RI) x (32 RJ) results; S stages of SLICE bytes of K, whose copies are dealt
// to WINDOW steps.
template <bool F32_, bool TURN_X_, bool TURN_W_, bool PAIRS_, int WI_, int WJ_, int RI_, int RJ_,
          int S_, int SLICE_, int WINDOW_>
struct TileForm {
  // PAIRS: W's 32-row blocks alternate between two matrices of equal height (gate and up rows)
  static constexpr bool PAIRS = PAIRS_;
  static constexpr bool F32 = F32_, TURN_X = TURN_X_, TURN_W = TURN_W_;
  static constexpr int WI = WI_, WJ = WJ_, RI = RI_, RJ = RJ_, S = S_, SLICE = SLICE_;
  static constexpr int WINDOW = WINDOW_;
  static constexpr int WAVES = WI * WJ, THREADS = 64 * WAVES;
  static constexpr int BM = 32 * RI * WI, BN = 32 * RJ * WJ;
  static constexpr int ELEM = F32 ? 4 : 2, SLICE_K = SLICE / ELEM, STEPS = SLICE / 32;
  static constexpr int X_BYTES = BM * SLICE, W_BYTES = BN * SLICE, STAGE = X_BYTES + W_BYTES;
  static constexpr int X_COPIES = X_BYTES / (1024 * WAVES), W_COPIES = W_BYTES / (1024 * WAVES);
  static constexpr int COPIES = X_COPIES + W_COPIES;
  static constexpr int LDS = S * STAGE;
  static_assert(X_COPIES * 1024 * WAVES == X_BYTES && W_COPIES * 1024 * WAVES == W_BYTES,
                "whole copies, the same number for each wave");
  static_assert((RI & (RI - 1)) == 0 && (RJ & (RJ - 1)) == 0, "powers of two");
  static_assert(SLICE == 128 || SLICE == 64, "slice");
  static_assert(LDS <= 160 * 1024, "LDS");
  static_assert(!PAIRS || (!TURN_W && RJ % 2 == 0), "a wave has both of a pair");
  static constexpr int COLUMNS = PAIRS ? BN / 2 : BN;  // of the output
};

// Row of a 32-row block that row i of the instruction's first operand is: its results, rows
// 8 t + 4 g + e of the lanes of half g, are then columns 16 g + 4 t + e of the block.
__device__ __forceinline__ int first_operand_row(int i) {
  return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
}

// A copy's lane: where it reads, from the operand's first row of the tile and k = 0 of the slice.
struct CopyLane {
  uint32_t off;  // kOOB: no such row
  int k;         // bytes of K before it (long), k before it (turned)
};

// Lane of the u-th KB of an operand of ROWS rows. `row_of` maps a tile's row to the operand's
// row from the tile's first (or a negative number for none).
template <class T, bool TURN, int ROWS, class RowOf>
__device__ __forceinline__ CopyLane copy_lane(const Side& s, int u, int lane, RowOf row_of) {
  CopyLane c;
  if constexpr (!TURN) {
    constexpr int PIECES = T::SLICE / 16;
    const int row = u * (64 / PIECES) + lane / PIECES;
    const int sw = T::SLICE == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
    c.k = ((lane % PIECES) ^ sw) * 16;
    const int r = row_of(row);
    c.off = r < 0 ? mgg::kOOB : (uint32_t)(r * s.ld + c.k);
  } else {
    constexpr int RB = ROWS * T::ELEM;  // bytes of one k
    const int at = u * 1024 + lane * 16;
    const int k = at / RB;
    int b = at % RB;
    if constexpr (T::F32) b ^= ((k >> 2) & 1 & (RB / 128 - 1)) << 7;
    else b ^= (k & 3 & (RB / 64 - 1)) << 6;
    c.k = k;
    const int r = row_of(b / T::ELEM);
    c.off = r < 0 ? mgg::kOOB : (uint32_t)(k * s.ld + (int64_t)r * T::ELEM);
  }
  return c;
}

// Fragments of one step: 16 bytes a lane for each 32 rows.
typedef uint4 Frag;

template <class T, bool TURN, bool FIRST, int ROWS>
struct FragReader {
  uint32_t base;  // of the lane, in the operand's part of a stage
  __device__ __forceinline__ FragReader(int part, int lane) {
    if constexpr (!TURN) {
      const int row = part + (FIRST ? first_operand_row(lane & 31) : lane & 31);
      const int sw = T::SLICE == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
      base = row * T::SLICE + ((lane >> 5) ^ sw) * 16;
    } else if constexpr (T::F32) {
      constexpr int RB = ROWS * 4;
      const int col = FIRST ? first_operand_row(lane & 31) : lane & 31;
      const int f = (lane >> 5) & (RB / 128 - 1);
      base = 4 * (lane >> 5) * RB + (((part >> 5) ^ f) << 7) + col * 4;
    } else {
      constexpr int RB = ROWS * 2;
      const int kk = (lane & 15) >> 2, quad = 4 * ((lane >> 4) & 1) + (lane & 3);
      const int col = FIRST ? 16 * (quad & 1) + 4 * (quad >> 1) : 4 * quad;
      base = (8 * (lane >> 5) + kk) * RB + (((part >> 5) ^ (kk & (RB / 64 - 1))) << 6) + col * 2;
    }
  }
  // 32 rows further i times, at step `step` of the slice
  __device__ __forceinline__ Frag read(const uint8_t* stage, int i, int step) const {
    if constexpr (!TURN) {
      return *reinterpret_cast<const Frag*>(stage + (base ^ (step << 5)) + i * 32 * T::SLICE);
    } else if constexpr (T::F32) {
      constexpr int RB = ROWS * 4;
      const uint8_t* p = stage + (base ^ (i << 7)) + step * 8 * RB;
      Frag v;
      v.x = *reinterpret_cast<const uint32_t*>(p);
      v.y = *reinterpret_cast<const uint32_t*>(p + RB);
      v.z = *reinterpret_cast<const uint32_t*>(p + 2 * RB);
      v.w = *reinterpret_cast<const uint32_t*>(p + 3 * RB);
      return v;
    } else {
      constexpr int RB = ROWS * 2;
      using Lds = __attribute__((address_space(3))) v4s*;
      const uint8_t* p = stage + (base ^ (i << 6)) + step * 16 * RB;
      const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p));
      const uint2 hi =
          __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * RB)));
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
};

template <bool F32>
__device__ __forceinline__ v16f multiply(const Frag& w, const Frag& x, v16f acc) {
  if constexpr (F32) {
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w.x), __uint_as_float(x.x), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w.y), __uint_as_float(x.y), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w.z), __uint_as_float(x.z), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w.w), __uint_as_float(x.w), acc, 0, 0, 0);
    return acc;
  } else {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w),
                                                   __builtin_bit_cast(v8bf, x), acc, 0, 0, 0);
  }
}

// acc = the tile's sums over K elements from k0 on, `k_len` of them (any number, also none). x and
// w stand at the tile's first row (long) or column (turned) and at k0, and have `rows` rows from
// there on; PAIRS: so does the second matrix, `second` bytes behind w.
template <class T>
__device__ __forceinline__ void tile_sums(const Side& x, const Side& w, int64_t second, int k_len,
                                          uint8_t* lds, v16f (&acc)[T::RI][T::RJ]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto x_row = [&](int r) { return r < x.rows ? r : -1; };
  const auto w_row = [&](int r) {
    if constexpr (T::PAIRS) r = (r >> 6) * 32 + (r & 31);
    return r < w.rows ? r : -1;
  };
  CopyLane cx[T::X_COPIES], cw[T::W_COPIES];
#pragma unroll
  for (int q = 0; q < T::X_COPIES; ++q)
    cx[q] = copy_lane<T, T::TURN_X, T::BM>(x, q * T::WAVES + wave, lane, x_row);
#pragma unroll
  for (int q = 0; q < T::W_COPIES; ++q)
    cw[q] = copy_lane<T, T::TURN_W, T::BN>(w, q * T::WAVES + wave, lane, w_row);

  const uint32_t lds0 = mgg::lds_addr(lds) + wave * 1024;
  const int slices = (k_len + T::SLICE_K - 1) / T::SLICE_K;
  // Copies go slice by slice. Those past the last slice read nothing and write zeros, so that the
  // number of copies under way is the same in every slice.
  int left_x = T::TURN_X ? k_len : k_len * T::ELEM, left_w = T::TURN_W ? k_len : k_len * T::ELEM;
  const uint8_t *px = x.p, *pw = w.p;
  v4i rx, rw, rw2;
  int to_stage = 0;
  auto begin_slice = [&]() {
    rx = mgg::make_rsrc(px, 0x7fffffffu);
    rw = mgg::make_rsrc(pw, 0x7fffffffu);
    mgg::pin_sgpr(rx);
    mgg::pin_sgpr(rw);
    if constexpr (T::PAIRS) {
      rw2 = mgg::make_rsrc(pw + second, 0x7fffffffu);
      mgg::pin_sgpr(rw2);
    }
    mgg::dma_fence();
  };
  auto copy = [&](int q) {  // the q-th of COPIES
    if (q < T::X_COPIES) {
      const CopyLane& c = cx[q < T::X_COPIES ? q : 0];
      const uint32_t off = c.k < left_x ? c.off : mgg::kOOB;
      mgg::dma_x4(lds0 + to_stage * T::STAGE + q * T::WAVES * 1024, rx, off);
    } else {
      const int qw = q - T::X_COPIES;
      const CopyLane& c = cw[qw >= 0 && qw < T::W_COPIES ? qw : 0];
      const uint32_t off = c.k < left_w ? c.off : mgg::kOOB;
      const uint32_t at = lds0 + to_stage * T::STAGE + T::X_BYTES + qw * T::WAVES * 1024;
      if constexpr (T::PAIRS) {
        // the KB's rows are all of one matrix
        const bool up = ((qw * T::WAVES + wave) * (1024 / T::SLICE) >> 5) & 1;
        if (up) mgg::dma_x4(at, rw2, off);
        else mgg::dma_x4(at, rw, off);
      } else {
        mgg::dma_x4(at, rw, off);
      }
    }
  };
  auto end_slice = [&]() {
    px += T::TURN_X ? T::SLICE_K * x.ld : T::SLICE;
    pw += T::TURN_W ? T::SLICE_K * w.ld : T::SLICE;
    left_x -= T::TURN_X ? T::SLICE_K : T::SLICE;
    left_w -= T::TURN_W ? T::SLICE_K : T::SLICE;
    to_stage = to_stage + 1 == T::S ? 0 : to_stage + 1;
  };

#pragma unroll
  for (int i = 0; i < T::RI; ++i)
#pragma unroll
    for (int j = 0; j < T::RJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  if (slices <= 0) return;

  const int wi = wave / T::WJ * 32 * T::RI, wj = wave % T::WJ * 32 * T::RJ;
  const FragReader<T, T::TURN_X, false, T::BM> read_x(wi, lane);
  const FragReader<T, T::TURN_W, true, T::BN> read_w(wj, lane);
  struct Step {
    Frag x[T::RI], w[T::RJ];
  };
  constexpr int READS = T::RI + T::RJ;
  auto read = [&](Step& f, int n, int stage, int step) {  // the n-th of READS
    const uint8_t* base = lds + stage * T::STAGE;
    if (n < T::RJ) f.w[n < T::RJ ? n : 0] = read_w.read(base + T::X_BYTES, n, step);
    else f.x[n < T::RJ ? 0 : n - T::RJ] = read_x.read(base, n - T::RJ, step);
  };

  // The copies of a slice are dealt to WINDOW steps: the last step of the slice S before it, whose
  // stage it takes, and the ones after that.
  constexpr int WINDOW = T::STEPS < T::WINDOW ? T::STEPS : T::WINDOW;
  auto copies = [&](int pos, int i) {  // with the i-th of RI groups of products
#pragma unroll
    for (int q = 0; q < T::COPIES; ++q)
      if (q * WINDOW * T::RI / T::COPIES == pos * T::RI + i) copy(q);
  };
  for (int s = 0; s < T::S - 1; ++s) {
    begin_slice();
#pragma unroll
    for (int q = 0; q < T::COPIES; ++q) copy(q);
    end_slice();
  }
  mgg::vm_wait_imm<(T::S - 2) * T::COPIES>();
  mgg::lds_barrier();
  begin_slice();
#pragma unroll
  for (int i = 0; i < T::RI; ++i) copies(0, i);
  Step now, next;
#pragma unroll
  for (int n = 0; n < READS; ++n) read(now, n, 0, 0);
  int stage = 0;
  for (int s = 0; s < slices; ++s) {
    const int then = stage + 1 == T::S ? 0 : stage + 1;
#pragma unroll
    for (int step = 0; step < T::STEPS; ++step) {
      const bool last = step == T::STEPS - 1;
      if (last) {
        // The next slice has landed, and everyone has read this one to its end.
        end_slice();
        mgg::vm_wait_imm<(T::S - 2) * T::COPIES>();
        mgg::lds_barrier();
        begin_slice();
      }
#pragma unroll
      for (int i = 0; i < T::RI; ++i) {
#pragma unroll
        for (int j = 0; j < T::RJ; ++j)
          acc[i][j] = multiply<T::F32>(now.w[j], now.x[i], acc[i][j]);
#pragma unroll
        for (int n = 0; n < READS; ++n)
          if (n * T::RI / READS == i) read(next, n, last ? then : stage, last ? 0 : step + 1);
        if (last) copies(0, i);
        else if (step + 1 < WINDOW) copies(step + 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      now = next;
    }
    stage = then;
  }
  mgg::vm_wait_imm<0>();
  mgg::lds_barrier();  // LDS is free, nothing is on its way into it
}

}  // namespace mgg_dense
