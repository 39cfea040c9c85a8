// linear_products.h - the dense products in tiles: which tile a workgroup takes, and how its sums
// get to the outputs.
#pragma once

#include "linear_common.h"

namespace mgg_dense {

// Tile of a workgroup. Workgroups go to the eight dies in turn, so each die gets a run of
// consecutive tiles; a run goes down eight tiles of m, then to the next of n, so that the tiles a
// die has under way share their operand rows in its L2.
__device__ __forceinline__ void tile_place(int b, int tiles_m, int tiles_n, int& i, int& j) {
  const int tiles = tiles_m * tiles_n, per = tiles / 8, whole = per * 8;
  const int t = b < whole ? (b & 7) * per + (b >> 3) : b;
  constexpr int DOWN = 8;
  const int band = t / (DOWN * tiles_n), in = t - band * DOWN * tiles_n;
  const int height = min(DOWN, tiles_m - band * DOWN);
  i = band * DOWN + in % height;
  j = in / height;
}

// The results of a wave's tile. A lane's results of a 32 x 32 block are runs of eight columns of one
// row: lane (m, h) has columns 8 h .. (registers 0-7) and 16 + 8 h .. (8-15) of row m. Bias and
// function are applied there; then 128 bytes of each of 32 rows - two blocks in bfloat16, one in
// float32 - turn in 4 KB of LDS of the wave's own, so that eight lanes side by side store 128
// bytes of a row. Lanes that are not side by side have their 16 bytes stored one by one, which
// took the epilogue of a 256 x 256 tile three times as long. A residual comes in the same way.
// 16-byte pieces change places by row, so that lanes that are served at once meet different banks.
struct Turn {
  uint8_t* lds;
  int lane;
  __device__ __forceinline__ uint4* at(int row, int piece) const {
    return reinterpret_cast<uint4*>(lds + row * 128 + (piece ^ ((row >> 1) & 7)) * 16);
  }
  // the lane's k-th piece of four among the eight of its row
  template <bool F32>
  __device__ __forceinline__ int own(int k) const {
    return F32 ? 4 * (k >> 1) + 2 * (lane >> 5) + (k & 1) : 2 * k + (lane >> 5);
  }
  // pieces of the lane's own row -> pieces lane & 7 of rows 8 k + (lane >> 3), and back
  template <bool F32>
  __device__ __forceinline__ void to_lines(uint4 (&p)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) *at(lane & 31, own<F32>(k)) = p[k];
    wave_order();
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = *at(8 * k + (lane >> 3), lane & 7);
    wave_order();
  }
  template <bool F32>
  __device__ __forceinline__ void to_rows(uint4 (&p)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) *at(8 * k + (lane >> 3), lane & 7) = p[k];
    wave_order();
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = *at(lane & 31, own<F32>(k));
    wave_order();
  }
};

// A matrix of whole aligned 16-byte pieces that tiles store to or load from: element (0, 0) of the
// tile's first row and column, and how much there is from there on.
struct Lines {
  v4i rsrc;
  int ld, rows, bytes;
  __device__ __forceinline__ Lines(const void* base, bool f32, int64_t ld_, int64_t m, int n,
                                   int64_t rows_, int cols) {
    const int elem = f32 ? 4 : 2;
    ld = (int)ld_ * elem;
    rows = (int)min((int64_t)INT32_MAX, rows_ - m);
    bytes = (cols - n) * elem;
    rsrc = mgg::make_rsrc(reinterpret_cast<const uint8_t*>(base) + (m * ld_ + n) * elem, 0x7fffffffu);
  }
  // the piece `at` bytes along row `row` of the tile; nothing is outside
  __device__ __forceinline__ uint32_t offset(int row, int at) const {
    return row < rows && at < bytes ? (uint32_t)(row * ld + at) : mgg::kOOB;
  }
};

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {  // one instruction
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, v2{(__bf16)a, (__bf16)b});
}

// Stores NB blocks of 32 columns (at columns `at` .. of the lines) of 32 rows (from `row` on): two, or
// one in float32.
template <bool F32, int NB>
__device__ __forceinline__ void store_blocks(const Lines& to, int row, int at,
                                             const float (&v)[NB][16], const Turn& turn) {
  static_assert(F32 || NB == 2, "lines of 128 bytes");
  const int r = row + (turn.lane >> 3), c = (turn.lane & 7) * 16;
  uint4 p[4];
#pragma unroll
  for (int b = 0; b < (F32 ? NB : 1); ++b) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32) {
        p[k] = __builtin_bit_cast(uint4, v4f{v[b][4 * k], v[b][4 * k + 1], v[b][4 * k + 2], v[b][4 * k + 3]});
      } else {
        const float* s = v[k >> 1] + 8 * (k & 1);
        p[k] = make_uint4(two_bf16(s[0], s[1]), two_bf16(s[2], s[3]), two_bf16(s[4], s[5]),
                          two_bf16(s[6], s[7]));
      }
    }
    turn.to_lines<F32>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mgg::store_b128(to.rsrc, to.offset(r + 8 * k, (at + 32 * b) * (F32 ? 4 : 2) + c),
                      __builtin_bit_cast(v4i, p[k]));
  }
}

// Such blocks on their way, as pieces of lines.
template <bool F32, int NB>
__device__ __forceinline__ void load_blocks(const Lines& from, int row, int at, int lane,
                                            uint4 (&p)[F32 ? 4 * NB : 4]) {
  const int r = row + (lane >> 3), c = (lane & 7) * 16;
#pragma unroll
  for (int k = 0; k < (F32 ? 4 * NB : 4); ++k)
    p[k] = __builtin_bit_cast(
        uint4, mgg::load_b128(from.rsrc, from.offset(r + 8 * (k & 3),
                                                     (at + 32 * (k >> 2)) * (F32 ? 4 : 2) + c)));
}
// v += those.
template <bool F32, int NB>
__device__ __forceinline__ void add_blocks(const uint4 (&lines)[F32 ? 4 * NB : 4],
                                           float (&v)[NB][16], const Turn& turn) {
#pragma unroll
  for (int b = 0; b < (F32 ? NB : 1); ++b) {
    uint4 p[4] = {lines[4 * b], lines[4 * b + 1], lines[4 * b + 2], lines[4 * b + 3]};
    turn.to_rows<F32>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {p[k].x, p[k].y, p[k].z, p[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (F32) {
          v[b][4 * k + e] += __uint_as_float(w[e]);
        } else {
          v[k >> 1][8 * (k & 1) + 2 * e] += __uint_as_float(w[e] << 16);
          v[k >> 1][8 * (k & 1) + 2 * e + 1] += __uint_as_float(w[e] & 0xffff0000u);
        }
      }
    }
  }
}

// v += the bias of a lane's results of the block at column n, of which `have` columns exist.
__device__ __forceinline__ void add_bias(const Emit& e, int n, int have, int lane, float (&v)[16]) {
  const int h = 8 * (lane >> 5);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float t[8];
    const int left = have - 16 * c - h;
    load_values<8>(e.bias, e.bias_f32, left > 0 ? n + 16 * c + h : 0, left, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * c + i] += t[i];
  }
}

// What the tiles' outputs are: matrices of whole aligned pieces in one of the types (`out` and the
// residual; z, if any, is whole too), or anything, stored element by element where it has to be.
enum OutForm { kOutBf16, kOutF32, kOutAny };

// Takes a tile's sums to its outputs; `lds`: 4 KB for each wave (kOutAny: none).
template <class T, OutForm OUT>
__device__ __forceinline__ void finish_tile(const Emit& e, int64_t m0, int64_t n0, uint8_t* lds,
                                            v16f (&acc)[T::RI][T::RJ]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr bool EPILOGUE = !T::TURN_W;  // gradients are stored as they are
  const int row0 = wave / T::WJ * 32 * T::RI, col0 = wave % T::WJ * (T::COLUMNS / T::WJ);
  // two blocks of columns at a time, if a wave has two; PAIRS: of gate columns and their up columns
  constexpr int P = T::PAIRS ? 2 : 1, NB = T::RJ >= 2 * P ? 2 : 1;
  if constexpr (OUT == kOutAny) {
#pragma unroll
    for (int j = 0; j < T::RJ; j += P)
#pragma unroll
      for (int i = 0; i < T::RI; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v[8], u[T::PAIRS ? 8 : 1];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            v[r] = acc[i][j][8 * c + r];
            if constexpr (T::PAIRS) u[r] = acc[i][j + 1][8 * c + r];
          }
          emit<8, T::PAIRS>(e, m0 + row0 + 32 * i + (lane & 31),
                            (int)n0 + col0 + j / P * 32 + 16 * c + 8 * (lane >> 5), v, u);
        }
  } else {
    constexpr bool F32 = OUT == kOutF32;
    const Turn turn{lds + wave * 4096, lane};
    const Lines out(e.out, F32, e.C, m0, (int)n0, e.rows, e.C);
    const Lines z(e.z, T::F32, e.N, m0, (int)n0, e.rows, e.C);
    const Lines z_up(reinterpret_cast<uint8_t*>(e.z) + (int64_t)e.C * T::ELEM, T::F32, e.N, m0,
                     (int)n0, e.rows, e.C);
    const Lines res(e.residual, F32, e.ld_res, m0, (int)n0, e.rows, e.C);
    // the residual of the next blocks is on its way while these are turned
    uint4 ahead[F32 ? 4 * NB : 4];
    if (EPILOGUE && e.residual) load_blocks<F32, NB>(res, row0, col0, lane, ahead);
#pragma unroll
    for (int j = 0; j < T::RJ; j += NB * P)
#pragma unroll
      for (int i = 0; i < T::RI; ++i) {
        const int row = row0 + 32 * i, col = col0 + j / P * 32, n = (int)n0 + col;
        float v[P][NB][16];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[p][b][r] = acc[i][j + P * b + p][r];
        if (EPILOGUE && e.bias) {
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int b = 0; b < NB; ++b)
              add_bias(e, p * e.C + n + 32 * b, e.C - n - 32 * b, lane, v[p][b]);
        }
        if (EPILOGUE && e.z) {
          store_blocks<T::F32, NB>(z, row, col, v[0], turn);
          if constexpr (T::PAIRS) store_blocks<T::F32, NB>(z_up, row, col, v[P - 1], turn);
        }
        if constexpr (T::PAIRS) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[0][b][r] *= sigmoid(v[0][b][r]) * v[P - 1][b][r];
        } else if (EPILOGUE && e.func != MGG_FUNC_NONE) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[0][b][r] = func_of(e.func, v[0][b][r]);
        }
        if (EPILOGUE && e.residual) {
          add_blocks<F32, NB>(ahead, v[0], turn);
          if (i + 1 < T::RI) load_blocks<F32, NB>(res, row + 32, col, lane, ahead);
          else if (j + NB * P < T::RJ) load_blocks<F32, NB>(res, row0, col + 32 * NB, lane, ahead);
        }
        store_blocks<F32, NB>(out, row, col, v[0], turn);
        __builtin_amdgcn_sched_barrier(0);
      }
  }
}

template <class T>
__device__ __forceinline__ void tile_origin(const Deal& d, int tile, int64_t& m0, int64_t& n0) {
  int ti, tj;
  tile_place(tile, d.tiles_m, d.tiles_n, ti, tj);
  m0 = (int64_t)ti * T::BM, n0 = (int64_t)tj * T::COLUMNS;
}

template <class T>
__device__ __forceinline__ float* part_sums(const TileArgs& a, int part) {
  return a.sums + (size_t)part * (T::BM * T::BN) +
         (threadIdx.x >> 6) * (T::RI * T::RJ * 1024) + (threadIdx.x & 63) * 4;
}

// A workgroup takes every gridDim.x-th item: whole tiles first, then parts of the others.
//
// Bound by the matrix cores, at the clock that the power limit leaves (1.85 GHz for bfloat16, where
// they are busy 60 % of the cycles). In the large tile the LDS moves what it can: a slice of
// 256 x 256 is 192 KB read and 64 KB written in the 2048 cycles that its products take. Measured with
// 8192 x 4096 x 4096 in bfloat16: x w^T 219 us (1255 TFLOP/s; a library product 210), dz w 222 (237),
// dz^T x 224 (253); 16384 x 7168 x 2048 386 us (339). Without storing anything the first takes 203 us,
// without copies and storing 165.
template <class T, OutForm OUT>
__global__ __launch_bounds__(T::THREADS) void linear_tile(TileArgs a) {
  extern __shared__ __align__(16) uint8_t s_lds[];
  const int items = a.deal.items();
  auto at = [&](int n, mgg_dense::TileAt& t) {
    const int64_t item = blockIdx.x + (int64_t)n * gridDim.x;
    if (item >= items) return false;
    const int part = (int)item - a.deal.whole;
    const int tile = part < 0 ? (int)item : a.deal.whole + part / a.deal.parts;
    const int k0 = part < 0 ? 0 : part % a.deal.parts * a.deal.part_k;
    int64_t m0, n0;
    tile_origin<T>(a.deal, tile, m0, n0);
    t.x = a.x.p + (T::TURN_X ? m0 * T::ELEM + k0 * a.x.ld : m0 * a.x.ld + (int64_t)k0 * T::ELEM);
    t.w = a.w.p + (T::TURN_W ? n0 * T::ELEM + k0 * a.w.ld : n0 * a.w.ld + (int64_t)k0 * T::ELEM);
    t.rows_x = a.x.rows - (int)m0;
    t.rows_w = a.w.rows - (int)n0;
    t.k_len = part < 0 ? a.K : min(a.deal.part_k, a.K - k0);
    return true;
  };
  auto done = [&](int n, v16f (&acc)[T::RI][T::RJ]) {
    const int item = (int)(blockIdx.x + (int64_t)n * gridDim.x);
    if (item < a.deal.whole) {
      int64_t m0, n0;
      tile_origin<T>(a.deal, item, m0, n0);
      finish_tile<T, OUT>(a.e, m0, n0, s_lds + T::LDS, acc);
      return;
    }
    float* to = part_sums<T>(a, item - a.deal.whole);
#pragma unroll
    for (int i = 0; i < T::RI; ++i)
#pragma unroll
      for (int j = 0; j < T::RJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<v4f*>(to + ((i * T::RJ + j) * 4 + q) * 256) =
              v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  };
  mgg_dense::tile_stream<T>(a.x, a.w, a.second, s_lds, at, done);
}

// Adds a cut tile's parts, in order, and takes them to the outputs.
template <class T, OutForm OUT>
__global__ __launch_bounds__(T::THREADS) void linear_join(TileArgs a) {
  extern __shared__ __align__(16) uint8_t s_lds[];
  v16f acc[T::RI][T::RJ];
#pragma unroll
  for (int i = 0; i < T::RI; ++i)
#pragma unroll
    for (int j = 0; j < T::RJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  for (int p = 0; p < a.deal.parts; ++p) {
    const float* from = part_sums<T>(a, blockIdx.x * a.deal.parts + p);
#pragma unroll
    for (int i = 0; i < T::RI; ++i)
#pragma unroll
      for (int j = 0; j < T::RJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f v = *reinterpret_cast<const v4f*>(from + ((i * T::RJ + j) * 4 + q) * 256);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
        }
  }
  int64_t m0, n0;
  tile_origin<T>(a.deal, a.deal.whole + blockIdx.x, m0, n0);
  finish_tile<T, OUT>(a.e, m0, n0, s_lds, acc);
}
template <class T, OutForm OUT>
mgg_status launch_tiles(const TileArgs& a, hipStream_t stream) {
  constexpr int TURN = OUT == kOutAny ? 0 : T::WAVES * 4096, LDS = T::LDS + TURN;
  static_assert(LDS <= 160 * 1024, "LDS");
  const auto kernel = linear_tile<T, OUT>;
  if (LDS > 64 * 1024 &&
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, LDS) !=
          hipSuccess)
    return fail(MGG_EHIP, "hipFuncSetAttribute failed");
  const int at_once = kCus * std::max(1, 160 * 1024 / LDS);
  kernel<<<std::min(a.deal.items(), at_once), T::THREADS, LDS, stream>>>(a);
  if (const int rest = a.deal.tiles() - a.deal.whole)
    linear_join<T, OUT><<<rest, T::THREADS, TURN, stream>>>(a);
  return MGG_OK;
}

template <class T>
mgg_status run_tiles(const TileArgs& a, hipStream_t stream) {
  const Emit& e = a.e;
  auto whole = [&](const void* p, int64_t ld, bool f32) {
    return !p || in_pieces(p, ld, e.C, f32 ? 4 : 2);
  };
  if (!whole(e.out, e.C, e.out_f32) || !whole(e.z, e.N, e.z_f32) ||
      !whole(e.residual, e.ld_res, e.out_f32))
    return launch_tiles<T, kOutAny>(a, stream);
  if (e.out_f32) return launch_tiles<T, kOutF32>(a, stream);
  // float32 operands with bfloat16 results are rare: the plain way of storing is enough
  return launch_tiles<T, T::F32 ? kOutAny : kOutBf16>(a, stream);
}

template <bool F32, bool TURN_X, bool TURN_W, bool PAIRS>
mgg_status run_product(const Product& p, TileArgs a, hipStream_t stream) {
  if (!p.counted) return fail(MGG_EUNSUPPORTED, "more tiles than are counted");
  a.deal = p.deal;
  // forms: waves along m and n, 32 x 32 blocks of a wave, stages, bytes of a slice, steps that
  // its copies are dealt to
  if (p.form == kLarge)
    return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 2, 2, 4, 2, 128, 3>>(a, stream);
  if constexpr (F32 && !PAIRS)
    if (p.form == kNarrow)
      return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 2, 1, 1, 3, 128, 2>>(a, stream);
  if constexpr (PAIRS)  // gate and up columns of a pair of blocks in one wave
    return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 1, 1, 4, 2, 128, 2>>(a, stream);
  else
    return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 2, 1, 2, 3, 128, 2>>(a, stream);
}
}  // namespace mgg_dense
