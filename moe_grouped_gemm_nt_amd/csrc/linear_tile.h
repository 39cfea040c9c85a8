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
// rows permuted so that a lane ends up with runs of 8 consecutive n of one m.
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
// 8 t + 4 g + e in register 4 t + e of the lanes of half g, are then columns
// 16 (t / 2) + 8 g + 4 (t % 2) + e of the block.
__device__ __forceinline__ int first_operand_row(int i) {
  return 16 * (i >> 4) + 8 * ((i >> 2) & 1) + 4 * ((i >> 3) & 1) + (i & 3);
}

// A lane's part in an operand's copies. A wave's q-th copy of a slice is the KB q * WAVES + wave of
// the operand's stage; from one of a lane's pieces to the next is a fixed distance, the same for
// all lanes, so that one offset serves them all.
template <class T, bool TURN, bool PAIRS, int ROWS>
struct CopyLane {
  // rows (long) or k (turned) from one copy of a wave to its next
  static constexpr int FURTHER = TURN ? T::WAVES * 1024 / (ROWS * T::ELEM) : T::WAVES * 1024 / T::SLICE;
  static_assert(!TURN || FURTHER % (T::F32 ? 8 : 4) == 0, "pieces change places alike in all copies");
  static_assert(TURN || FURTHER % (T::SLICE == 128 ? 16 : 4) == 0, "as above");
  // PAIRS: 32 rows of one matrix, then 32 of the other. A KB is of one of them; which one goes by
  // the wave (a round of copies has 64 rows) or by the copy (32 rows).
  static constexpr bool BY_WAVE = FURTHER == 64;
  static_assert(!PAIRS || FURTHER == 64 || FURTHER == 32, "whole blocks of 32 rows");
  static constexpr int shared(int q) {  // rows or k before copy q
    return !PAIRS ? q * FURTHER : BY_WAVE ? q * 32 : q / 2 * 32;
  }
  uint32_t off;  // of its first piece, from the tile's first row and the slice's first k
  int at;        // row (long) or k (turned) of its first piece
  int other;     // its bytes of K (long) or its row (turned)

  __device__ __forceinline__ CopyLane(int64_t ld, int wave, int lane) {
    if constexpr (!TURN) {
      constexpr int PIECES = T::SLICE / 16;
      const int row = wave * (64 / PIECES) + lane / PIECES;
      const int sw = T::SLICE == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
      other = ((lane % PIECES) ^ sw) * 16;
      at = PAIRS ? row % 32 : row;
      off = (uint32_t)(at * ld + other);
    } else {
      constexpr int RB = ROWS * T::ELEM;  // bytes of one k
      const int k = (wave * 1024 + lane * 16) / RB;
      int b = (wave * 1024 + lane * 16) % RB;
      if constexpr (T::F32) b ^= ((k >> 2) & 1 & (RB / 128 - 1)) << 7;
      else b ^= (k & 3 & (RB / 64 - 1)) << 6;
      other = b / T::ELEM;
      at = k;
      off = (uint32_t)(k * ld + b);
    }
  }
  // Offset of the lane's piece of copy q, less that of the shared(q) rows or k.
  __device__ __forceinline__ uint32_t offset(int q, int rows, int left) const {
    const bool there = TURN ? at < left - shared(q) && other < rows
                            : at < rows - shared(q) && other < left;
    return there ? off : mgg::kOOB;
  }
};

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
      const int col = FIRST ? first_operand_row(4 * quad) : 4 * quad;
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

// acc[j] += w[j] x^T over a step. Float32 takes four instructions a block; those of one block depend
// on each other, so they alternate between the blocks.
template <bool F32, int RJ>
__device__ __forceinline__ void multiply(const Frag (&w)[RJ], const Frag& x, v16f (&acc)[RJ]) {
  if constexpr (F32) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(ws[e]), __uint_as_float(xs[e]),
                                                      acc[j], 0, 0, 0);
      }
  } else {
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(v8bf, w[j]), __builtin_bit_cast(v8bf, x), acc[j], 0, 0, 0);
  }
}

// Slices of a tile: one at least, so that a sum of nothing is a tile like others.
template <class T>
__device__ __forceinline__ int slices_of(int k_len) {
  return max(1, (k_len - 1) / T::SLICE_K + 1);
}

// Where a tile's operands start and what is left of them: x and w stand at the tile's first row
// (long) or column (turned) and at its first k, and have `rows` rows from there on; PAIRS: so does
// the second matrix of w, `second` bytes behind it.
struct TileAt {
  const uint8_t *x, *w;
  int rows_x, rows_w, k_len;
};

// The tiles of a workgroup one after another. `at(n, TileAt&)` tells where its n-th tile is, or
// returns false behind the last; `done(n, acc)` takes the tile's sums. Slices of all tiles are one
// stream: a tile's first ones are on their way while the tile before is finished and handed over.
template <class T, class At, class Done>
__device__ __forceinline__ void tile_stream(const Side& x, const Side& w, int64_t second,
                                            uint8_t* lds, At at, Done done) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = mgg::lds_addr(lds) + wave * 1024;

  // ---- copies: the tile that they are at, and the slice of it
  const CopyLane<T, T::TURN_X, false, T::BM> cx(x.ld, wave, lane);
  const CopyLane<T, T::TURN_W, T::PAIRS, T::BN> cw(w.ld, wave, lane);
  const uint8_t *px, *pw;
  int left_x, left_w;       // of K: bytes (long) or elements (turned)
  int rows_x, rows_w;
  int copy_tile = 0, copy_left;  // slices of that tile to come
  int to_stage = 0;
  v4i rx, rw, rw2;
  auto begin_tile = [&]() {
    TileAt t;
    if (!at(copy_tile, t)) {
      // behind the last tile nothing is read, zeros are written: the number of copies under way
      // is the same in every slice
      t.x = x.p, t.w = w.p;
      t.rows_x = t.rows_w = 0;
      t.k_len = INT32_MAX / 8;
    }
    px = t.x, pw = t.w;
    rows_x = t.rows_x, rows_w = t.rows_w;
    left_x = T::TURN_X ? t.k_len : t.k_len * T::ELEM;
    left_w = T::TURN_W ? t.k_len : t.k_len * T::ELEM;
    copy_left = slices_of<T>(t.k_len);
  };
  auto begin_slice = [&]() {
    rx = mgg::make_rsrc(px, 0x7fffffffu);
    rw = mgg::make_rsrc(pw + (T::PAIRS && cw.BY_WAVE && wave >= 4 ? second : 0), 0x7fffffffu);
    mgg::pin_sgpr(rx);
    mgg::pin_sgpr(rw);
    if constexpr (T::PAIRS && !cw.BY_WAVE) {
      rw2 = mgg::make_rsrc(pw + second, 0x7fffffffu);
      mgg::pin_sgpr(rw2);
    }
    mgg::dma_fence();
  };
  auto copy = [&](int q) {  // the q-th of COPIES
    if (q < T::X_COPIES) {
      mgg::dma_x4_so(lds0 + to_stage * T::STAGE + q * T::WAVES * 1024, rx,
                     cx.offset(q, rows_x, left_x), (uint32_t)(cx.shared(q) * x.ld));
    } else {
      const int qw = q - T::X_COPIES;
      mgg::dma_x4_so(lds0 + to_stage * T::STAGE + T::X_BYTES + qw * T::WAVES * 1024,
                     T::PAIRS && !cw.BY_WAVE && qw % 2 ? rw2 : rw,
                     cw.offset(qw, rows_w, left_w), (uint32_t)(cw.shared(qw) * w.ld));
    }
  };
  auto end_slice = [&]() {
    to_stage = to_stage + 1 == T::S ? 0 : to_stage + 1;
    if (--copy_left == 0) {
      ++copy_tile;
      begin_tile();
    } else {
      px += T::TURN_X ? T::SLICE_K * x.ld : T::SLICE;
      pw += T::TURN_W ? T::SLICE_K * w.ld : T::SLICE;
      left_x -= T::TURN_X ? T::SLICE_K : T::SLICE;
      left_w -= T::TURN_W ? T::SLICE_K : T::SLICE;
    }
  };

  // ---- products
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

  begin_tile();
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
  int stage = 0;
  TileAt t;
  for (int tile = 0; at(tile, t); ++tile) {
    v16f acc[T::RI][T::RJ];
#pragma unroll
    for (int i = 0; i < T::RI; ++i)
#pragma unroll
      for (int j = 0; j < T::RJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    // read here and not at the end of the tile before: no registers of it while that is handed over
    Step now, next;
#pragma unroll
    for (int n = 0; n < READS; ++n) read(now, n, stage, 0);
    const int slices = slices_of<T>(t.k_len);
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
          multiply<T::F32>(now.w, now.x[i], acc[i]);
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
    done(tile, acc);
  }
  mgg::vm_wait_imm<0>();  // nothing is on its way into LDS when the workgroup ends
}

}  // namespace mgg_dense
