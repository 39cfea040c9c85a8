// newton_schulz.hip - orthogonalised updates of many matrices at once by Newton-Schulz
// products (C ABI in include/mgg/layer_ops.h: grouped_newton_schulz).
//
// X [m][n], m <= n (a taller matrix is handled transposed), is scaled to Frobenius norm 1.
// One step is three products:
//   A  = X X^T                      symmetric: tiles on and above the diagonal, mirrored
//   P  = a I + b A + c A A          symmetric likewise (A A = A A^T)
//   X' = P X = P (X^T)^T
// so with X^T kept beside X every product has both operands with K contiguous (NT).
//
// Number format. The products have to be of float32 grade: the map amplifies small singular
// values several hundred times in five steps, and an error of 16-bit size, spread over all
// directions, with them. Matrix instructions take 16-bit operands, so a value v is held as
// two fp16 numbers, hi = fp16(v * 2^s) and lo = fp16(v * 2^s - hi), together 22 bits, and a
// product is hi hi + hi lo + lo hi in one float32 accumulator (lo lo is below 2^-22 of it).
// The power of two keeps hi and lo out of fp16's subnormal range: |X| <= 4 and |A| <= 16 take
// 2^12, |P| <= 64 takes 2^10.

#include "layer_common.h"

namespace {

using namespace mgg_layer;

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTile = 128;   // rows and columns of an output tile; operands are padded to it
constexpr int kSlice = 32;   // K elements staged at once
constexpr int kMaxSide = 32768, kMaxMatrices = 4096, kMaxSteps = 32;
constexpr int kNormBlocks = 64;  // partial sums of squares per matrix
constexpr float kScaleX = 4096.f, kScaleA = 4096.f, kScaleP = 1024.f;

// A matrix as its two fp16 halves, each [rows][ld], `group` elements from one matrix to the
// next.
struct Split {
  _Float16 *hi, *lo;
  int ld;
  size_t group;
};

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

struct NsArgs {
  const void* in;
  void* out;
  int in_bf16, out_bf16;
  int M, N;        // as the caller's
  int tall;        // M > N: rows of X are the caller's columns
  float eps, scale;
  double* norms;   // [G][kNormBlocks]
};

__global__ __launch_bounds__(kThreads) void ns_norm(NsArgs a) {
  __shared__ double s_sum[kThreads / 64];
  const size_t size = (size_t)a.M * a.N, base = size * blockIdx.y;
  const size_t per = (size + kNormBlocks - 1) / kNormBlocks;
  const size_t lo = per * blockIdx.x, hi = min(lo + per, size);
  double sum = 0.0;
  for (size_t i = lo + threadIdx.x; i < hi; i += kThreads) {
    const float v = a.in_bf16 ? to_f32(reinterpret_cast<const bf16_t*>(a.in)[base + i])
                              : reinterpret_cast<const float*>(a.in)[base + i];
    sum += (double)v * (double)v;
  }
  sum = lanes_sum<64>(sum);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 64; ++w) sum += s_sum[w];
    a.norms[(size_t)blockIdx.y * kNormBlocks + blockIdx.x] = sum;
  }
}

constexpr int kSplitTile = 64;

// Scales a matrix to norm 1 and writes X and X^T in halves, padded with zeros.
__global__ __launch_bounds__(kThreads) void ns_split(NsArgs a, Split x, Split xt) {
  __shared__ float s_tile[kSplitTile][kSplitTile + 1];
  double sum = 0.0;
  for (int i = 0; i < kNormBlocks; ++i) sum += a.norms[(size_t)blockIdx.z * kNormBlocks + i];
  const double inv = (double)kScaleX / (sqrt(sum) + (double)a.eps);
  // the caller's rows run along tile rows here
  const int r0 = blockIdx.y * kSplitTile, c0 = blockIdx.x * kSplitTile;
  const int col = threadIdx.x % kSplitTile, row = threadIdx.x / kSplitTile;
  const size_t base = (size_t)a.M * a.N * blockIdx.z;
  // in the caller's orientation, `direct` has the input's rows as rows
  const Split direct = a.tall ? xt : x, turned = a.tall ? x : xt;
  for (int r = row; r < kSplitTile; r += kThreads / kSplitTile) {
    const int i = r0 + r, j = c0 + col;
    float v = 0.f;
    if (i < a.M && j < a.N) {
      const size_t at = base + (size_t)i * a.N + j;
      v = a.in_bf16 ? to_f32(reinterpret_cast<const bf16_t*>(a.in)[at])
                    : reinterpret_cast<const float*>(a.in)[at];
      v = (float)((double)v * inv);
    }
    s_tile[r][col] = v;
    _Float16 hi, lo;
    split(v, hi, lo);
    const size_t to = blockIdx.z * direct.group + (size_t)i * direct.ld + j;
    direct.hi[to] = hi;
    direct.lo[to] = lo;
  }
  __syncthreads();
  for (int r = row; r < kSplitTile; r += kThreads / kSplitTile) {
    _Float16 hi, lo;
    split(s_tile[col][r], hi, lo);
    const size_t to = blockIdx.z * turned.group + (size_t)(c0 + r) * turned.ld + r0 + col;
    turned.hi[to] = hi;
    turned.lo[to] = lo;
  }
}

enum Product { kGram, kPoly, kApply, kLast };

struct ProductArgs {
  Split left, right;  // both [rows][K]: C = left right^T
  int K;
  int tiles_i, tiles_j;
  float to_value;     // accumulator -> value: the operands' powers of two taken back
  Split c, ct;        // the result and its transpose (symmetric results: the same matrix)
  // kPoly: P = ca I + cb A + cc A A
  Split a;
  float ca, cb, cc;
  NsArgs ns;          // kLast
};

// C = left right^T for one 128 x 128 tile: four waves of 64 x 64 in 32 x 32 x 16 MFMAs, three
// to a K step (hi hi, hi lo, lo hi). The right operand's rows are the instruction's first
// operand, so a lane ends up with runs of four consecutive columns of one row of C.
template <Product WHAT>
__global__ __launch_bounds__(kThreads) void ns_product(ProductArgs p) {
  constexpr bool SYM = WHAT == kGram || WHAT == kPoly;
  // [operand half: left hi, left lo, right hi, right lo][row][K], the 16-byte pieces of a row
  // exchanged by its number so that eight consecutive rows meet different banks
  __shared__ _Float16 s_op[4][kTile][kSlice];
  int ti, tj;
  if constexpr (SYM) {  // the b-th pair i <= j, rows of the triangle one after another
    int b = blockIdx.x;
    ti = 0;
    for (int len = p.tiles_i; b >= len; --len) {
      b -= len;
      ++ti;
    }
    tj = ti + b;
  } else {
    ti = blockIdx.x / p.tiles_j;
    tj = blockIdx.x % p.tiles_j;
  }
  const int i0 = ti * kTile, j0 = tj * kTile;
  const size_t g = blockIdx.y;
  const _Float16* src[4] = {p.left.hi + g * p.left.group + (size_t)i0 * p.left.ld,
                            p.left.lo + g * p.left.group + (size_t)i0 * p.left.ld,
                            p.right.hi + g * p.right.group + (size_t)j0 * p.right.ld,
                            p.right.lo + g * p.right.group + (size_t)j0 * p.right.ld};
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wi = (wave >> 1) * 64, wj = (wave & 1) * 64;  // the wave's place in the tile
  v16f acc[2][2];  // [i][j]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  auto piece = [](int row, int c) { return c ^ ((row >> 1) & 3); };
  for (int k0 = 0; k0 < p.K; k0 += kSlice) {
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int ld = h < 2 ? p.left.ld : p.right.ld;
#pragma unroll
      for (int q = 0; q < kTile * 4 / kThreads; ++q) {
        const int at = q * kThreads + threadIdx.x, row = at >> 2, c = at & 3;
        *reinterpret_cast<v8h*>(&s_op[h][row][piece(row, c) * 8]) =
            *reinterpret_cast<const v8h*>(src[h] + (size_t)row * ld + k0 + c * 8);
      }
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kSlice / 16; ++kk) {
      v8h l[2][2], r[2][2];  // [half][32-row part]
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int c = kk * 2 + (lane >> 5);
          const int li = wi + t * 32 + (lane & 31), ri = wj + t * 32 + (lane & 31);
          l[h][t] = *reinterpret_cast<const v8h*>(&s_op[h][li][piece(li, c) * 8]);
          r[h][t] = *reinterpret_cast<const v8h*>(&s_op[2 + h][ri][piece(ri, c) * 8]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(r[0][j], l[0][i], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(r[1][j], l[0][i], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(r[0][j], l[1][i], acc[i][j], 0, 0, 0);
        }
    }
  }

  // lane: row i0 + wi + 32 i + (lane & 31); registers 4 q .. 4 q + 3: columns
  // j0 + wj + 32 j + 8 q + 4 (lane >> 5) ..
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = i0 + wi + 32 * i + (lane & 31);
        const int col = j0 + wj + 32 * j + 8 * q + 4 * (lane >> 5);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e] * p.to_value;
        if constexpr (WHAT == kLast) {
          const NsArgs& n = p.ns;
          const int rows = n.tall ? n.N : n.M, cols = n.tall ? n.M : n.N;
          const size_t base = (size_t)n.M * n.N * g;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (row < rows && col + e < cols) {
              const size_t at = base + (n.tall ? (size_t)(col + e) * n.N + row
                                               : (size_t)row * n.N + col + e);
              const float o = v[e] * n.scale;
              if (n.out_bf16) reinterpret_cast<bf16_t*>(n.out)[at] = from_f32<bf16_t>(o);
              else reinterpret_cast<float*>(n.out)[at] = o;
            }
        } else {
          float power = WHAT == kGram ? kScaleA : WHAT == kPoly ? kScaleP : kScaleX;
          if constexpr (WHAT == kPoly) {
            const size_t at = g * p.a.group + (size_t)row * p.a.ld + col;
            const v4h hi = *reinterpret_cast<const v4h*>(p.a.hi + at);
            const v4h lo = *reinterpret_cast<const v4h*>(p.a.lo + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float av = ((float)hi[e] + (float)lo[e]) * (1.f / kScaleA);
              v[e] = fmaf(p.cc, v[e], p.cb * av) + (row == col + e ? p.ca : 0.f);
            }
          }
          v4h hi, lo;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            _Float16 h, l;
            split(v[e] * power, h, l);
            hi[e] = h;
            lo[e] = l;
          }
          const size_t at = g * p.c.group + (size_t)row * p.c.ld + col;
          *reinterpret_cast<v4h*>(p.c.hi + at) = hi;
          *reinterpret_cast<v4h*>(p.c.lo + at) = lo;
          if (!SYM || ti != tj) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const size_t mirrored = g * p.ct.group + (size_t)(col + e) * p.ct.ld + row;
              p.ct.hi[mirrored] = hi[e];
              p.ct.lo[mirrored] = lo[e];
            }
          }
        }
      }
}

struct Workspace {
  int m, n, mp, np;
  size_t x, xt[2], a, p, norms, bytes;
  Workspace(int G, int M, int N) {
    m = std::min(M, N);
    n = std::max(M, N);
    mp = cdiv(m, kTile) * kTile;
    np = cdiv(n, kTile) * kTile;
    const size_t big = (size_t)G * mp * np * 2 * sizeof(_Float16);
    const size_t small = (size_t)G * mp * mp * 2 * sizeof(_Float16);
    x = 0;
    xt[0] = x + big;
    xt[1] = xt[0] + big;
    a = xt[1] + big;
    p = a + small;
    norms = p + small;
    bytes = round_up(norms + (size_t)G * kNormBlocks * sizeof(double), 256);
  }
  Split at(void* base, size_t off, int G, int rows, int ld) const {
    _Float16* hi = reinterpret_cast<_Float16*>((char*)base + off);
    return Split{hi, hi + (size_t)G * rows * ld, ld, (size_t)rows * ld};
  }
};

// The largest |x p(x^2)| that the steps reach from singular values in [0, 1], and of the
// polynomial P that multiplies X: a bound from the ends and the stationary points.
bool stays_in_range(int steps, const float* coeffs) {
  double top = 1.0;
  for (int s = 0; s < steps; ++s) {
    const double a = coeffs[3 * s], b = coeffs[3 * s + 1], c = coeffs[3 * s + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
    auto poly = [&](double t) { return a + t * (b + t * c); };  // t = x^2
    double next = top * std::fabs(poly(top * top));
    double p_top = std::max(std::fabs(poly(0.0)), std::fabs(poly(top * top)));
    // d/dx (a x + b x^3 + c x^5) = a + 3 b t + 5 c t^2
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (disc >= 0.0) {
      for (double sign : {-1.0, 1.0}) {
        const double t = c != 0.0 ? (-3.0 * b + sign * std::sqrt(disc)) / (10.0 * c)
                                  : (b != 0.0 ? -a / (3.0 * b) : -1.0);
        if (t > 0.0 && t < top * top) next = std::max(next, std::sqrt(t) * std::fabs(poly(t)));
      }
    }
    if (c != 0.0) {
      const double t = -b / (2.0 * c);
      if (t > 0.0 && t < top * top) p_top = std::max(p_top, std::fabs(poly(t)));
    }
    if (!(next <= 3.9) || !(p_top <= 60.0)) return false;
    top = std::max(next, 1e-3);
  }
  return true;
}

}  // namespace

extern "C" {

size_t grouped_newton_schulz_workspace(int G, int M, int N) {
  if (G < 1 || G > kMaxMatrices || M < 1 || N < 1 || M > kMaxSide || N > kMaxSide) return 0;
  return Workspace(G, M, N).bytes;
}

mgg_status grouped_newton_schulz(mgg_act dt, mgg_act out_dt, int G, int M, int N,
                                 const void* X, void* out, int steps, const float* coeffs,
                                 float eps, float scale, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  mgg_set_last_error("");
  if (!known(dt) || !known(out_dt)) return fail(MGG_EINVAL, "unknown element type");
  if (G < 1 || G > kMaxMatrices) return fail(MGG_EINVAL, "G must be in [1, 4096]");
  if (M < 1 || N < 1 || M > kMaxSide || N > kMaxSide)
    return fail(MGG_EINVAL, "M and N must be in [1, 32768]");
  if (steps < 1 || steps > kMaxSteps) return fail(MGG_EINVAL, "steps must be in [1, 32]");
  if (!X || !out || !coeffs) return fail(MGG_EINVAL, "null pointer");
  if (!aligned(X, elem_bytes(dt)) || !aligned(out, elem_bytes(out_dt)))
    return fail(MGG_EINVAL, "X and out must be aligned to their element");
  if (!(eps > 0.f) || !std::isfinite(eps) || !std::isfinite(scale))
    return fail(MGG_EINVAL, "eps must be positive, eps and scale finite");
  if (!stays_in_range(steps, coeffs))
    return fail(MGG_EUNSUPPORTED, "the coefficients send singular values out of range");
  const Workspace ws(G, M, N);
  if (!workspace || workspace_bytes < ws.bytes)
    return fail(MGG_EINVAL, "the workspace is smaller than grouped_newton_schulz_workspace says");
  if (!aligned(workspace, 256)) return fail(MGG_EINVAL, "the workspace must be 256-byte aligned");

  const int mp = ws.mp, np = ws.np;
  const Split x = ws.at(workspace, ws.x, G, mp, np);
  Split xt = ws.at(workspace, ws.xt[0], G, np, mp), xt_next = ws.at(workspace, ws.xt[1], G, np, mp);
  const Split a = ws.at(workspace, ws.a, G, mp, mp), p = ws.at(workspace, ws.p, G, mp, mp);
  const NsArgs ns{X, out, dt == MGG_ACT_BF16, out_dt == MGG_ACT_BF16, M, N, M > N, eps, scale,
                  reinterpret_cast<double*>((char*)workspace + ws.norms)};
  ns_norm<<<dim3(kNormBlocks, G), kThreads, 0, stream>>>(ns);
  const int rows = M > N ? np : mp, cols = M > N ? mp : np;
  ns_split<<<dim3(cols / kSplitTile, rows / kSplitTile, G), kThreads, 0, stream>>>(ns, x, xt);
  const int tm = mp / kTile, tn = np / kTile;
  for (int s = 0; s < steps; ++s) {
    ProductArgs gram{x, x, np, tm, tm, 1.f / (kScaleX * kScaleX), a, a, a, 0.f, 0.f, 0.f, ns};
    ns_product<kGram><<<dim3(tm * (tm + 1) / 2, G), kThreads, 0, stream>>>(gram);
    ProductArgs poly{a, a, mp, tm, tm, 1.f / (kScaleA * kScaleA), p, p, a,
                     coeffs[3 * s], coeffs[3 * s + 1], coeffs[3 * s + 2], ns};
    ns_product<kPoly><<<dim3(tm * (tm + 1) / 2, G), kThreads, 0, stream>>>(poly);
    ProductArgs apply{p, xt, mp, tm, tn, 1.f / (kScaleP * kScaleX), x, xt_next, a,
                      0.f, 0.f, 0.f, ns};
    if (s + 1 < steps) ns_product<kApply><<<dim3(tm * tn, G), kThreads, 0, stream>>>(apply);
    else ns_product<kLast><<<dim3(tm * tn, G), kThreads, 0, stream>>>(apply);
    std::swap(xt, xt_next);
  }
  return launched();
}

}  // extern "C"
