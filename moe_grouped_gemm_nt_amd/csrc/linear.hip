// linear.hip - dense products with bias, activation and residual in their epilogue, and their
// gradients (C ABI in include/mgg/linear.h: linear_act, linear_act_backward).
//
// Forward: out = f(x w^T + b) + r; the gated unit's tiles hold the same columns of gate and up.
// Few rows of x are multiplied as weights stream by (row_stream.h); more of them in tiles
// (linear_tile.h). Backward: one pass over d_out and z makes dz = d_out f'(z), rounded to the
// operands' type as every operand of a matrix instruction is, and the column sums that are the
// bias's gradient before that rounding; then d_x = dz w and d_w = dz^T x in tiles, whose turned
// operands are read as they lie in memory.

#include "mgg/linear.h"

#include "linear_tile.h"
#include "row_stream.h"

namespace {

using namespace mgg_layer;
using mgg::v16f;
using mgg::v4i;
using mgg_dense::Side;
using mgg_dense::TileForm;

constexpr int kMaxSide = 1 << 20;
constexpr int kFewRows = 64;  // up to here the weights stream past the rows

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

// Stores two blocks of 32 columns (at columns `at` .. of the lines) of 32 rows (from `row` on).
template <bool F32>
__device__ __forceinline__ void store_blocks(const Lines& to, int row, int at,
                                             const float (&v)[2][16], const Turn& turn) {
  const int r = row + (turn.lane >> 3), c = (turn.lane & 7) * 16;
  uint4 p[4];
#pragma unroll
  for (int b = 0; b < (F32 ? 2 : 1); ++b) {
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

// Two such blocks on their way, as pieces of lines.
template <bool F32>
__device__ __forceinline__ void load_blocks(const Lines& from, int row, int at, int lane,
                                            uint4 (&p)[F32 ? 8 : 4]) {
  const int r = row + (lane >> 3), c = (lane & 7) * 16;
#pragma unroll
  for (int k = 0; k < (F32 ? 8 : 4); ++k)
    p[k] = __builtin_bit_cast(
        uint4, mgg::load_b128(from.rsrc, from.offset(r + 8 * (k & 3),
                                                     (at + 32 * (k >> 2)) * (F32 ? 4 : 2) + c)));
}
// v += those.
template <bool F32>
__device__ __forceinline__ void add_blocks(const uint4 (&lines)[F32 ? 8 : 4], float (&v)[2][16],
                                           const Turn& turn) {
#pragma unroll
  for (int b = 0; b < (F32 ? 2 : 1); ++b) {
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
  // two blocks of columns at a time; PAIRS: two of gate columns and their up columns
  constexpr int P = T::PAIRS ? 2 : 1;
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
    uint4 ahead[F32 ? 8 : 4];
    if (EPILOGUE && e.residual) load_blocks<F32>(res, row0, col0, lane, ahead);
#pragma unroll
    for (int j = 0; j < T::RJ; j += 2 * P)
#pragma unroll
      for (int i = 0; i < T::RI; ++i) {
        const int row = row0 + 32 * i, col = col0 + j / P * 32, n = (int)n0 + col;
        float v[P][2][16];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[p][b][r] = acc[i][j + P * b + p][r];
        if (EPILOGUE && e.bias) {
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              add_bias(e, p * e.C + n + 32 * b, e.C - n - 32 * b, lane, v[p][b]);
        }
        if (EPILOGUE && e.z) {
          store_blocks<T::F32>(z, row, col, v[0], turn);
          if constexpr (T::PAIRS) store_blocks<T::F32>(z_up, row, col, v[P - 1], turn);
        }
        if constexpr (T::PAIRS) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[0][b][r] *= sigmoid(v[0][b][r]) * v[P - 1][b][r];
        } else if (EPILOGUE && e.func != MGG_FUNC_NONE) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) v[0][b][r] = func_of(e.func, v[0][b][r]);
        }
        if (EPILOGUE && e.residual) {
          add_blocks<F32>(ahead, v[0], turn);
          if (i + 1 < T::RI) load_blocks<F32>(res, row + 32, col, lane, ahead);
          else if (j + 2 * P < T::RJ) load_blocks<F32>(res, row0, col + 64, lane, ahead);
        }
        store_blocks<F32>(out, row, col, v[0], turn);
        __builtin_amdgcn_sched_barrier(0);
      }
  }
}

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

constexpr int kCus = 256;

// Whether tiles take a matrix as it lies: whole aligned pieces of 16 bytes, rows whose
// distances stay below 2 GiB within a tile.
bool in_pieces(const void* p, int64_t ld, int cols, size_t elem) {
  return aligned(p, 16) && ld * (int64_t)elem % 16 == 0 && cols * elem % 16 == 0 && ld <= kMaxSide;
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

// The tile forms of a product, and what they are chosen by: how long one tile takes a CU that has
// it alone (time for 2^20 multiply-adds, and for starting and storing a tile).
//   large   256 x 256 by eight waves of 64 x 128: 1250 TFLOP/s in bfloat16 (8192 x 4096 x 4096), 144
//           in float32 (4096 x 4096 x 4096)
//   small   128 x 128 by eight waves of 32 x 64: 910 and 137
//   narrow  128 x 64 by four waves of 32 x 64, float32: 118
enum FormName { kLarge, kSmall, kNarrow };
struct FormCost {
  int bm, bn;
  double us_per_m, us_fixed;
};
constexpr FormCost kBf16Forms[] = {{256, 256, 0.43, 6.0}, {128, 128, 0.59, 4.0}};
constexpr FormCost kF32Forms[] = {{256, 256, 3.73, 8.0}, {128, 128, 3.92, 5.0}, {128, 64, 4.55, 4.0}};

struct Product {
  FormName form;
  Deal deal;
  size_t bytes;   // of the parts' sums
  bool counted;   // false: more tiles than an int counts
};

// Tiles of [rows][cols] sums over K: the form, and how its tiles are dealt to the CUs, that cost
// least. A last round of few tiles leaves CUs idle; its tiles are cut along K so that it fills
// them, where that gains more than the join costs (a launch, and the sums written and read).
Product plan_product(bool f32, bool pairs, int64_t rows, int cols, int K) {
  Product best{};
  double best_us = 0;
  // a narrow tile has no room for blocks of gate and of up columns
  for (int f = 0; f < (f32 && !pairs ? 3 : 2); ++f) {
    const FormCost& c = f32 ? kF32Forms[f] : kBf16Forms[f];
    const int64_t m = (rows + c.bm - 1) / c.bm, n = cdiv(cols, c.bn);
    Product p{};
    p.form = (FormName)f;
    p.counted = m * n < INT32_MAX / 64;
    const int slice = f32 ? 32 : 64, slices = std::max(1, cdiv(K, slice));
    const int64_t tiles = m * n;
    const int rest = (int)(tiles % kCus);
    const double tile_us = c.us_per_m * c.bm * c.bn * (double)K / (1 << 20) + c.us_fixed;
    double us = tile_us * (double)((tiles + kCus - 1) / kCus);
    p.deal = Deal{(int)m, (int)n, (int)tiles, 1, K};
    if (rest > 0 && p.counted) {
      int parts = std::min(kCus / rest, slices / 4);
      if (parts > 1) {
        const int part_k = cdiv(slices, parts) * slice;
        parts = cdiv(K, part_k);
        const size_t bytes = (size_t)rest * parts * c.bm * c.bn * 4;
        const double cut = tile_us * (double)(tiles / kCus) +
                           (tile_us - c.us_fixed) * part_k / K + c.us_fixed + 8.0 + bytes * 4e-7;
        if (cut < us) {
          us = cut;
          p.deal.whole = (int)tiles - rest;
          p.deal.parts = parts;
          p.deal.part_k = part_k;
          p.bytes = bytes;
        }
      }
    }
    if (f == 0 || us < best_us) best = p, best_us = us;
  }
  return best;
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
      return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 1, 1, 2, 2, 128, 2>>(a, stream);
  if constexpr (PAIRS)  // gate and up columns of a pair of blocks in one wave
    return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 1, 1, 4, 2, 128, 2>>(a, stream);
  else
    return run_tiles<TileForm<F32, TURN_X, TURN_W, PAIRS, 4, 2, 1, 2, 3, 128, 2>>(a, stream);
}

// ---------------------------------------------------------------------------- few rows

constexpr int kRowWaves = 8, kRowThreads = 64 * kRowWaves, kPartLd = 20;

struct RowArgs {
  const uint8_t *x, *w;
  int64_t ldx, ldw;  // bytes
  int M, K;
  Emit e;
};

// 16 weight rows (PAIRS: 8 gate rows and their 8 up rows) times all rows of x; the waves share K.
template <bool F32, bool PAIRS, int RT>
__global__ __launch_bounds__(kRowThreads) void linear_rows(RowArgs a) {
  constexpr WeightForm W = F32 ? kF32Weights : kBf16Weights;
  using F = Form<W>;
  constexpr int COLS = PAIRS ? 8 : 16;
  __shared__ __align__(16) float s_part[kRowWaves * RT * 16 * kPartLd];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * COLS;
  const int n = min(n0 + (PAIRS ? r & 7 : r), a.e.C - 1) + (PAIRS && r >= 8 ? a.e.C : 0);
  const uint8_t* x[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int m = 16 * t + r;
    x[t] = m < a.M ? a.x + m * a.ldx + q * F::X_BYTES : nullptr;
  }
  v4f acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int blocks = cdiv(a.K, F::BLOCK);
  stream_rows<W, RT, RT == 1 ? 6 : RT == 2 ? 4 : 2>(
      a.w + n * a.ldw + q * F::RUN_BYTES, x, blocks * wave / kRowWaves,
      blocks * (wave + 1) / kRowWaves, a.K, acc);
#pragma unroll
  for (int t = 0; t < RT; ++t)
    *reinterpret_cast<v4f*>(s_part + ((wave * RT + t) * 16 + r) * kPartLd + 4 * q) = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * 16 * COLS; i += kRowThreads) {
    const int m = i / COLS, c = i % COLS;
    float v[1] = {0.f}, u[1] = {0.f};
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) {
      const float* s = s_part + (w * RT * 16 + m) * kPartLd + c;
      v[0] += s[0];
      if constexpr (PAIRS) u[0] += s[8];
    }
    emit<1, PAIRS>(a.e, m, n0 + c, v, u);
  }
}

template <bool F32, bool PAIRS>
void run_rows(const RowArgs& a, hipStream_t stream) {
  const int grid = cdiv(a.e.C, PAIRS ? 8 : 16);
  if (a.M <= 16) linear_rows<F32, PAIRS, 1><<<grid, kRowThreads, 0, stream>>>(a);
  else if (a.M <= 32) linear_rows<F32, PAIRS, 2><<<grid, kRowThreads, 0, stream>>>(a);
  else linear_rows<F32, PAIRS, 4><<<grid, kRowThreads, 0, stream>>>(a);
}

// -------------------------------------------------------------------- passes over operands

// Rows of an operand that are not whole aligned pieces of 16 bytes, copied to rows that are;
// elements past a row's end are 0.
struct PackArgs {
  const uint8_t* from;
  uint8_t* to;
  int64_t ld_from, rows;  // bytes
  int bytes, ld_to;
};
template <int ELEM>
__global__ __launch_bounds__(256) void linear_pack(PackArgs a) {
  const int pieces = a.ld_to / 16;
  const int64_t total = a.rows * pieces, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
    const int64_t row = i / pieces;
    const int at = (int)(i - row * pieces) * 16;
    const uint8_t* p = a.from + row * a.ld_from + at;
    const uint4 v = at + 16 <= a.bytes ? load16(p) : load16_part<ELEM>(p, a.bytes - at);
    *reinterpret_cast<uint4*>(a.to + row * a.ld_to + at) = v;
  }
}

struct GradArgs {
  const void *z, *d;
  int64_t ldz, ldd;
  void* dz;        // rows of `ld`, zeros behind the N-th; null: column sums alone
  int ld;
  float* sums;     // [strips][N], or null
  int64_t rows, strip;
  int N, C;
  mgg_func func;
  bool f32, d_f32;
};

__device__ __forceinline__ float grad_of(mgg_func f, float z, float d) {
  switch (f) {
    case MGG_FUNC_RELU: return z > 0.f ? d : z != z ? z : 0.f;
    case MGG_FUNC_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      return d * fmaf(z * 0.39894228f, e, cdf);
    }
    case MGG_FUNC_SILU: {
      float q, rest;
      sigmoid_parts(z, q, rest);
      return d * (q * fmaf(z, rest, 1.f));
    }
    default: return d;
  }
}

// dz and its column sums: a workgroup takes a strip of rows of 512 columns of d_out, eight columns
// a lane, its four waves row by row in turn.
constexpr int kGradColumns = 512, kGradWaves = 4;
template <bool PAIRS>
__global__ __launch_bounds__(64 * kGradWaves) void linear_grad(GradArgs a) {
  constexpr int P = PAIRS ? 2 : 1;
  __shared__ float s_sum[P][kGradWaves][kGradColumns];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * kGradColumns + lane * 8;
  const int have = a.C - c;
  const int64_t r0 = blockIdx.y * a.strip, r1 = min(a.rows, r0 + a.strip);
  float sum[P][8] = {};
  // a gated unit's dz has its up columns right behind its gate columns; only there the end of the
  // rows, with zeros up to `ld`
  const int room = PAIRS ? have : a.ld - c;
  if (room > 0) {
    for (int64_t r = r0 + wave; r < r1; r += kGradWaves) {
      float d[8], z[8], u[P == 2 ? 8 : 1], g[8];
      load_values<8>(a.d, a.d_f32, r * a.ldd + c, have, d);
      if (a.func != MGG_FUNC_NONE) load_values<8>(a.z, a.f32, r * a.ldz + c, have, z);
      if constexpr (PAIRS) {
        load_values<8>(a.z, a.f32, r * a.ldz + a.C + c, have, u);
        float gu[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float q, rest;
          sigmoid_parts(z[i], q, rest);
          g[i] = d[i] * u[i] * (q * fmaf(z[i], rest, 1.f));
          gu[i] = d[i] * (z[i] * q);
          if (i < have) sum[1][i] += gu[i];
        }
        if (a.dz) store_values<8>(a.dz, a.f32, r * a.ld + a.C + c, have, gu);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          g[i] = i < have ? (a.func == MGG_FUNC_NONE ? d[i] : grad_of(a.func, z[i], d[i])) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < have) sum[0][i] += g[i];
      if (a.dz) store_values<8>(a.dz, a.f32, r * a.ld + c, room, g);
    }
  }
  if (PAIRS && a.dz && blockIdx.x == 0 && a.ld > a.N) {
    const float zeros[8] = {};
    for (int64_t r = r0 + threadIdx.x; r < r1; r += 64 * kGradWaves)
      store_values<8>(a.dz, a.f32, r * a.ld + a.N, a.ld - a.N, zeros);
  }
  if (!a.sums) return;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[p][wave][lane * 8 + i] = sum[p][i];
  __syncthreads();
  for (int i = threadIdx.x; i < P * kGradColumns; i += 64 * kGradWaves) {
    const int p = i / kGradColumns, at = i % kGradColumns, col = blockIdx.x * kGradColumns + at;
    if (col >= a.C) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kGradWaves; ++w) v += s_sum[p][w][at];
    a.sums[(int64_t)blockIdx.y * a.N + p * a.C + col] = v;
  }
}

// d_bias from the strips' sums, in order: 64 columns a workgroup, its waves share the strips.
constexpr int kSumWaves = 8;
__global__ __launch_bounds__(64 * kSumWaves) void linear_bias_sum(const float* sums, int strips,
                                                                   int N, float* d_bias) {
  __shared__ float s_sum[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  float v = 0.f;
  if (col < N) {
#pragma unroll 8
    for (int s = wave; s < strips; s += kSumWaves) v += sums[(int64_t)s * N + col];
  }
  s_sum[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < N) {
    for (int w = 1; w < kSumWaves; ++w) v += s_sum[w][lane];
    d_bias[col] = v;
  }
}

// ---------------------------------------------------------------------------- host side

bool func_known(mgg_func f) { return f >= MGG_FUNC_NONE && f <= MGG_FUNC_SWIGLU; }

int packed_ld(int cols, size_t elem) { return (int)round_up(cols, 16 / elem); }

// An operand of the tiles, [rows][cols], and its packed copy where it needs one.
struct Operand {
  const void* p;
  int64_t ld, rows;
  int cols;
  size_t elem;
  bool packed;
  Operand(const void* p_, int64_t ld_, int64_t rows_, int cols_, size_t elem_)
      : p(p_), ld(ld_), rows(rows_), cols(cols_), elem(elem_),
        packed(!in_pieces(p_, ld_, cols_, elem_)) {}
  size_t bytes() const { return packed ? (size_t)rows * packed_ld(cols, elem) * elem : 0; }
  // Enqueues the copy to `room`, if any, and returns where the tiles read.
  Side place(char* room, int64_t side_rows, hipStream_t stream) const {
    if (!packed) return Side{(const uint8_t*)p, ld * (int64_t)elem, (int)side_rows};
    const int to = packed_ld(cols, elem);
    const PackArgs a{(const uint8_t*)p, (uint8_t*)room, ld * (int64_t)elem, rows,
                     (int)(cols * elem), (int)(to * elem)};
    const int64_t pieces = rows * a.ld_to / 16;
    const int blocks = (int)std::min<int64_t>(4096, (pieces + 255) / 256);
    if (blocks > 0) {
      if (elem == 2) linear_pack<2><<<blocks, 256, 0, stream>>>(a);
      else linear_pack<4><<<blocks, 256, 0, stream>>>(a);
    }
    return Side{(const uint8_t*)room, to * (int64_t)elem, (int)side_rows};
  }
};

mgg_status check(const mgg_linear* l) {
  if (!l) return fail(MGG_EINVAL, "null pointer");
  if (!known(l->dtype) || !known(l->out_dt) || !known(l->bias_dt))
    return fail(MGG_EINVAL, "unknown element type");
  if (!func_known(l->func)) return fail(MGG_EINVAL, "unknown function");
  if (l->M < 0 || l->M > kMaxRows) return fail(MGG_EINVAL, "M must be in [0, 2^30]");
  if (l->N < 1 || l->N > kMaxSide || l->K < 1 || l->K > kMaxSide)
    return fail(MGG_EINVAL, "N and K must be in [1, 2^20]");
  if (l->func == MGG_FUNC_SWIGLU && l->N % 2) return fail(MGG_EINVAL, "SwiGLU needs an even N");
  if (l->ldx < l->K || l->ldw < l->K)
    return fail(MGG_EINVAL, "a row stride is smaller than the row");
  const size_t b = elem_bytes(l->dtype);
  if (!aligned(l->x, b) || !aligned(l->w, b))
    return fail(MGG_EINVAL, "tensors must be aligned to their element");
  return MGG_OK;
}

int out_columns(const mgg_linear* l) { return l->func == MGG_FUNC_SWIGLU ? l->N / 2 : l->N; }

// The parts of a call's workspace, each 256-byte aligned.
struct Room {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes = round_up(bytes + n, 256);
    return at;
  }
};

struct ForwardPlan {
  Operand x, w;
  bool few;
  Product product{};
  Room room;
  size_t at_x = 0, at_w = 0, at_parts = 0;
  explicit ForwardPlan(const mgg_linear* l)
      : x(l->x, l->ldx, l->M, l->K, elem_bytes(l->dtype)),
        w(l->w, l->ldw, l->N, l->K, elem_bytes(l->dtype)), few(l->M <= kFewRows) {
    if (few) return;
    // both have whole pieces along K, or neither: zeros behind a row's end meet zeros
    at_x = room.take(x.bytes());
    at_w = room.take(w.bytes());
    product = plan_product(l->dtype == MGG_ACT_F32, l->func == MGG_FUNC_SWIGLU, l->M, l->N, l->K);
    at_parts = room.take(product.bytes);
  }
};

constexpr int kMaxStrips = 128;

struct BackwardPlan {
  bool dz_pass;      // dz is made, not d_out itself
  int ld_dz, strips;
  int64_t strip;
  Operand dz, w, x;
  Product by_x{}, by_w{};
  Room room;
  size_t at_dz, at_sums, at_w, at_x, at_parts;
  static bool needs_pass(const mgg_linear* l, const void* d, int64_t ldd) {
    return l->func != MGG_FUNC_NONE || l->out_dt != l->dtype ||
           !in_pieces(d, ldd, l->N, elem_bytes(l->dtype));
  }
  BackwardPlan(const mgg_linear* l, const void* d, int64_t ldd, bool want_x, bool want_w,
               bool want_bias)
      : dz_pass((want_x || want_w) && needs_pass(l, d, ldd)),
        ld_dz(packed_ld(l->N, elem_bytes(l->dtype))),
        dz(dz_pass ? nullptr : d, dz_pass ? ld_dz : ldd, l->M, dz_pass ? ld_dz : l->N,
           elem_bytes(l->dtype)),
        w(l->w, l->ldw, l->N, l->K, elem_bytes(l->dtype)),
        x(l->x, l->ldx, l->M, l->K, elem_bytes(l->dtype)) {
    strip = std::max<int64_t>(16, ((int64_t)l->M + kMaxStrips - 1) / kMaxStrips);
    strips = (int)((l->M + strip - 1) / strip);
    at_dz = room.take(dz_pass ? (size_t)l->M * ld_dz * elem_bytes(l->dtype) : 0);
    at_sums = room.take(want_bias ? (size_t)strips * l->N * 4 : 0);
    at_w = room.take(want_x ? w.bytes() : 0);
    at_x = room.take(want_w ? x.bytes() : 0);
    // one product after the other: their parts' sums share a place
    if (want_x) by_x = plan_product(l->dtype == MGG_ACT_F32, false, l->M, l->K, l->N);
    if (want_w) by_w = plan_product(l->dtype == MGG_ACT_F32, false, l->N, l->K, l->M);
    at_parts = room.take(std::max(by_x.bytes, by_w.bytes));
  }
};

mgg_status check_workspace(const void* workspace, size_t have, size_t need, const char* text) {
  if (need == 0) return MGG_OK;
  if (!workspace || have < need) return fail(MGG_EINVAL, text);
  if (!aligned(workspace, 256)) return fail(MGG_EINVAL, "the workspace must be 256-byte aligned");
  return MGG_OK;
}

mgg_status check_backward(const mgg_linear* l, const void* z, int64_t ldz, const void* d_out,
                          int64_t ldd, const void* d_x, const void* d_w, const float* d_bias) {
  if (const mgg_status s = check(l)) return s;
  if (!d_x && !d_w && !d_bias && l->M > 0)
    return fail(MGG_EINVAL, "one of d_x, d_w and d_bias must be given");
  if (l->M > 0) {
    if ((z != nullptr) != (l->func != MGG_FUNC_NONE))
      return fail(MGG_EINVAL, "z goes with a function, and only with one");
    if (!d_out || (d_x && !l->w) || (d_w && !l->x)) return fail(MGG_EINVAL, "null pointer");
    if (ldd < out_columns(l) || (z && ldz < l->N))
      return fail(MGG_EINVAL, "a row stride is smaller than the row");
  }
  if (!aligned(z, elem_bytes(l->dtype)) || !aligned(d_out, elem_bytes(l->out_dt)) ||
      !aligned(d_x, elem_bytes(l->dtype)) || !aligned(d_bias, 4))
    return fail(MGG_EINVAL, "tensors must be aligned to their element");
  return MGG_OK;
}

}  // namespace

extern "C" {

size_t linear_act_workspace(const mgg_linear* l) {
  return check(l) == MGG_OK ? ForwardPlan(l).room.bytes : 0;
}

mgg_status linear_act(const mgg_linear* l, void* out, void* z, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  mgg_set_last_error("");
  if (const mgg_status s = check(l)) return s;
  if (l->M == 0) return MGG_OK;
  if (!l->x || !l->w || !out) return fail(MGG_EINVAL, "null pointer");
  const int C = out_columns(l);
  if (l->residual && l->ld_res < C)
    return fail(MGG_EINVAL, "a row stride is smaller than the row");
  if (!aligned(out, elem_bytes(l->out_dt)) || !aligned(l->residual, elem_bytes(l->out_dt)) ||
      !aligned(z, elem_bytes(l->dtype)) || !aligned(l->bias, elem_bytes(l->bias_dt)))
    return fail(MGG_EINVAL, "tensors must be aligned to their element");
  const ForwardPlan plan(l);
  if (const mgg_status s =
          check_workspace(workspace, workspace_bytes, plan.room.bytes,
                          "the workspace is smaller than linear_act_workspace says"))
    return s;
  const bool f32 = l->dtype == MGG_ACT_F32, pairs = l->func == MGG_FUNC_SWIGLU;
  const Emit e{out, l->bias, l->residual, l->ld_res, z, l->M, l->N, C, l->func,
               l->out_dt == MGG_ACT_F32, l->bias_dt == MGG_ACT_F32, f32};
  if (plan.few) {
    const int64_t b = (int64_t)elem_bytes(l->dtype);
    const RowArgs a{(const uint8_t*)l->x, (const uint8_t*)l->w, l->ldx * b, l->ldw * b,
                    l->M, l->K, e};
    if (f32) pairs ? run_rows<true, true>(a, stream) : run_rows<true, false>(a, stream);
    else pairs ? run_rows<false, true>(a, stream) : run_rows<false, false>(a, stream);
    return launched();
  }
  char* base = reinterpret_cast<char*>(workspace);
  TileArgs a{};
  a.x = plan.x.place(base + plan.at_x, l->M, stream);
  a.w = plan.w.place(base + plan.at_w, C, stream);
  a.second = (int64_t)C * a.w.ld;
  a.K = l->K;
  a.sums = reinterpret_cast<float*>(base + plan.at_parts);
  a.e = e;
  const Product& p = plan.product;
  const mgg_status s = f32 ? pairs ? run_product<true, false, false, true>(p, a, stream)
                                   : run_product<true, false, false, false>(p, a, stream)
                       : pairs ? run_product<false, false, false, true>(p, a, stream)
                               : run_product<false, false, false, false>(p, a, stream);
  return s ? s : launched();
}

size_t linear_act_backward_workspace(const mgg_linear* l, const void* z, int64_t ldz,
                                     const void* d_out, int64_t ld_dout, const void* d_x,
                                     const void* d_w, const float* d_bias) {
  if (check_backward(l, z, ldz, d_out, ld_dout, d_x, d_w, d_bias) != MGG_OK) return 0;
  return BackwardPlan(l, d_out, ld_dout, d_x, d_w, d_bias).room.bytes;
}

mgg_status linear_act_backward(const mgg_linear* l, const void* z, int64_t ldz,
                               const void* d_out, int64_t ld_dout, void* d_x, void* d_w,
                               mgg_act dw_dt, float* d_bias, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  mgg_set_last_error("");
  if (const mgg_status s = check_backward(l, z, ldz, d_out, ld_dout, d_x, d_w, d_bias)) return s;
  if (d_w && !known(dw_dt)) return fail(MGG_EINVAL, "unknown element type");
  if (d_w && !aligned(d_w, elem_bytes(dw_dt)))
    return fail(MGG_EINVAL, "tensors must be aligned to their element");
  const BackwardPlan plan(l, d_out, ld_dout, d_x, d_w, d_bias);
  if (const mgg_status s =
          check_workspace(workspace, workspace_bytes, plan.room.bytes,
                          "the workspace is smaller than linear_act_backward_workspace says"))
    return s;
  char* base = reinterpret_cast<char*>(workspace);
  const bool f32 = l->dtype == MGG_ACT_F32;
  const int C = out_columns(l);
  float* sums = reinterpret_cast<float*>(base + plan.at_sums);
  if (l->M > 0 && (plan.dz_pass || d_bias)) {
    const GradArgs g{z, d_out, ldz, ld_dout, plan.dz_pass ? base + plan.at_dz : nullptr,
                     plan.ld_dz, d_bias ? sums : nullptr, l->M, plan.strip, l->N, C, l->func,
                     f32, l->out_dt == MGG_ACT_F32};
    const dim3 grid(cdiv(l->func == MGG_FUNC_SWIGLU ? C : plan.ld_dz, kGradColumns), plan.strips);
    if (l->func == MGG_FUNC_SWIGLU) linear_grad<true><<<grid, 64 * kGradWaves, 0, stream>>>(g);
    else linear_grad<false><<<grid, 64 * kGradWaves, 0, stream>>>(g);
  }
  if (d_bias)
    linear_bias_sum<<<cdiv(l->N, 64), 64 * kSumWaves, 0, stream>>>(sums, plan.strips, l->N, d_bias);
  const int64_t b = (int64_t)elem_bytes(l->dtype);
  const uint8_t* dz = plan.dz_pass ? (const uint8_t*)base + plan.at_dz : (const uint8_t*)d_out;
  const int64_t ld_dz = (plan.dz_pass ? plan.ld_dz : ld_dout) * b;
  if (d_x && l->M > 0) {
    TileArgs a{};
    a.x = Side{dz, ld_dz, l->M};
    a.w = plan.w.place(base + plan.at_w, l->K, stream);
    a.K = l->N;
    a.e = Emit{d_x, nullptr, nullptr, 0, nullptr, l->M, l->K, l->K, MGG_FUNC_NONE, f32, f32, f32};
    a.sums = reinterpret_cast<float*>(base + plan.at_parts);
    if (const mgg_status s = f32 ? run_product<true, false, true, false>(plan.by_x, a, stream)
                                 : run_product<false, false, true, false>(plan.by_x, a, stream))
      return s;
  }
  if (d_w) {
    TileArgs a{};
    a.x = Side{dz, ld_dz, l->N};
    a.w = plan.x.place(base + plan.at_x, l->K, stream);
    a.K = l->M;
    a.e = Emit{d_w, nullptr, nullptr, 0, nullptr, l->N, l->K, l->K, MGG_FUNC_NONE,
               dw_dt == MGG_ACT_F32, f32, f32};
    a.sums = reinterpret_cast<float*>(base + plan.at_parts);
    if (const mgg_status s = f32 ? run_product<true, true, true, false>(plan.by_w, a, stream)
                                 : run_product<false, true, true, false>(plan.by_w, a, stream))
      return s;
  }
  return launched();
}

}  // extern "C"
