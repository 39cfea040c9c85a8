// linear.hip - dense products with bias, activation and residual in their epilogue, and their
// gradients (C ABI in include/mgg/linear.h: linear_act, linear_act_backward).
//
// Forward: out = f(x w^T + b) + r; the gated unit's tiles hold the same columns of gate and up.
// Few rows of x are multiplied as weights stream by (row_stream.h); more of them in tiles
// (linear_tile.h). Backward: one pass over d_out and z makes dz = d_out f'(z), rounded to the
// operands' type as every operand of a matrix instruction is, and the column sums that are the
// bias's gradient before that rounding; then d_x = dz w and d_w = dz^T x in tiles, whose turned
// operands are read as they lie in memory.

#include "linear_common.h"

namespace {

using namespace mgg_dense;

constexpr int kFewRows = 64;  // up to here the weights stream past the rows (linear_rows)

// The tile forms of a product, and what they are chosen by: how long one tile takes a CU that has
// it alone (time for 2^20 multiply-adds, and for starting and storing a tile).
//   large   256 x 256 by eight waves of 64 x 128: 1250 TFLOP/s in bfloat16 (8192 x 4096 x 4096), 144
//           in float32 (4096 x 4096 x 4096)
//   small   128 x 128 by eight waves of 32 x 64: 910 and 137
//   narrow  128 x 64 by eight waves of 32 x 32, float32: 125
struct FormCost {
  int bm, bn;
  double us_per_m, us_fixed;
};
constexpr FormCost kBf16Forms[] = {{256, 256, 0.43, 6.0}, {128, 128, 0.59, 4.0}};
constexpr FormCost kF32Forms[] = {{256, 256, 3.73, 8.0}, {128, 128, 3.92, 5.0}, {128, 64, 4.3, 4.0}};

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

// ---------------------------------------------------------------------------- few rows

constexpr int kRowWaves = 8, kRowThreads = 64 * kRowWaves, kPartLd = 20;

struct RowArgs {
  const uint8_t *x, *w;
  int64_t ldx, ldw;  // bytes
  int M, K;
  Emit e;
};

// 16 weight rows (PAIRS: 8 gate rows and their 8 up rows) times all rows of x; the waves share K.
// Bound by the weights' way from HBM, with more rows by that of x from L2, which every workgroup reads
// whole. Measured in bfloat16: one row, 7168 x 2048: 29 MB in 7.9 us; 48 rows, 4096 x 4096 with SwiGLU
// 16.7 us, where tiles cut along K take 20 (33 to 128 rows: 19 to 23 us).
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

// dz and its column sums, bound by HBM (8192 x 4096 bfloat16: 201 MB in 53 us): a workgroup takes a strip of rows of 512 columns of d_out, eight columns
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
