// block_norm.hip - the norms before and after a block, fused with the block's gate, residual
// scale and residual sum, forward and backward (C ABI in include/mgg/layer_ops.h).
//
// TPR threads hold one row of each tensor in registers (NV 16-byte pieces a thread), so each
// tensor is read once and written once whatever the number of reductions over the row. The
// kernels are bound by HBM. The backward recomputes both norms' statistics from the rows it
// reads anyway; its sums over rows (norm weights, residual scale) are kept in registers per
// column while a workgroup walks its rows, written once per row group and added in a fixed
// order by a second kernel.

#include "layer_common.h"

namespace {

using namespace mgg_layer;

constexpr int kMaxH = 32768;

struct NormArgs {
  int T, H;
  const void *x, *y, *gate;
  int64_t ldx, ldy, ld_gate;
  int gate_kind, param_bf16;
  const void *scale, *w_after, *w_before;
  float alpha, beta, eps;
  void *x_out, *u;
  // backward
  const void *d_x, *d_u;
  int64_t ld_dx, ld_du;
  void *d_x_in, *d_y, *d_gate;
  float *part_before, *part_block;  // [row groups][H]
};

template <class T>
constexpr int kVec = 16 / sizeof(T);

// 16 bytes of a row as they are stored; rows may start at any element.
template <class T>
struct Piece {
  uint32_t w[4];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// `n`: elements of the row that are left at p.
template <class T>
__device__ __forceinline__ Piece<T> load_piece(const T* p, int n) {
  Piece<T> r{{0u, 0u, 0u, 0u}};
  if (n >= kVec<T>) {
    __builtin_memcpy(&r, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) {
      if (i < n) {
        if constexpr (sizeof(T) == 4) r.w[i] = __float_as_uint(p[i]);
        else r.w[i / 2] |= (uint32_t)p[i].bits << (i & 1 ? 16 : 0);
      }
    }
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store_piece(T* p, int n, const float (&v)[kVec<T>]) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_bits(v[2 * i]) | (uint32_t)bf16_bits(v[2 * i + 1]) << 16;
  }
  if (n >= kVec<T>) {
    __builtin_memcpy(p, w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// VEC values of a parameter vector from column `c` (n left); `missing` where there is none.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, int bf16, int c, int n, float missing,
                                           float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = missing;
  if (p == nullptr) return;
  if (bf16) {
    const bf16_t* q = reinterpret_cast<const bf16_t*>(p) + c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = i < n ? to_f32(q[i]) : 0.f;
  } else {
    const float* q = reinterpret_cast<const float*>(p) + c;
    if (n >= VEC) {
      __builtin_memcpy(v, q, VEC * 4);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = i < n ? q[i] : 0.f;
    }
  }
}

// Sums of N values over the TPR threads of a row, in a fixed order. `s` holds
// [2][N][waves] floats; `turn` alternates its halves, so one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* s, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum<64>(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* half = s + turn * (N * W);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) half[i * W + threadIdx.x / 64] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = half[i * W];
#pragma unroll
      for (int w = 1; w < W; ++w) v[i] += half[i * W + w];
    }
  }
}

constexpr int block_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <class T, int TPR, int NV, bool BLOCK>
__global__ __launch_bounds__(block_threads(TPR)) void norm_forward(NormArgs a) {
  constexpr int VEC = kVec<T>;
  __shared__ float s_sum[2 * TPR / 64];
  int turn = 0;
  const int tid = threadIdx.x & (TPR - 1);
  const int t = blockIdx.x * (block_threads(TPR) / TPR) + threadIdx.x / TPR;
  if (t >= a.T) return;  // whole waves, and whole workgroups where a barrier follows
  const int H = a.H;
  const T* xr = reinterpret_cast<const T*>(a.x) + (size_t)t * a.ldx;
  float out[NV][VEC];
  if constexpr (BLOCK) {
    const T* yr = reinterpret_cast<const T*>(a.y) + (size_t)t * a.ldy;
    const T* gr = reinterpret_cast<const T*>(a.gate) + (size_t)t * a.ld_gate;
    Piece<T> xs[NV], ys[NV], gs[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      ys[c] = load_piece(yr + col, H - col);
      xs[c] = load_piece(xr + col, H - col);
      if (a.gate_kind == MGG_GATE_ELEMENT) gs[c] = load_piece(gr + col, H - col);
    }
    float row = a.beta;  // what a whole row is multiplied with
    if (a.gate_kind == MGG_GATE_TOKEN) {
      float q, not_q;
      sigmoid_parts(to_f32(*gr), q, not_q);
      row *= q;
    }
    if (a.w_after != nullptr) {
      float sum[1] = {0.f};
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[0] += ys[c].at(i) * ys[c].at(i);
      row_sums<TPR>(sum, s_sum, turn);
      row *= 1.f / sqrtf(sum[0] / (float)H + a.eps);
    }
    T* outr = reinterpret_cast<T*>(a.x_out) + (size_t)t * H;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      float wa[VEC], sc[VEC];
      load_param(a.w_after, a.param_bf16, col, H - col, 1.f, wa);
      load_param(a.scale, a.param_bf16, col, H - col, 1.f, sc);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float g = row * sc[i] * wa[i];
        if (a.gate_kind == MGG_GATE_ELEMENT) {
          float q, not_q;
          sigmoid_parts(gs[c].at(i), q, not_q);
          g *= q;
        }
        out[c][i] = fmaf(ys[c].at(i), g, a.alpha * xs[c].at(i));
      }
      store_piece(outr + col, H - col, out[c]);
    }
    if (a.w_before == nullptr) return;
  } else {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      const Piece<T> xs = load_piece(xr + col, H - col);
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[c][i] = xs.at(i);
    }
  }
  float sum[1] = {0.f};
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum[0] += out[c][i] * out[c][i];
  row_sums<TPR>(sum, s_sum, turn);
  const float r = 1.f / sqrtf(sum[0] / (float)H + a.eps);
  T* ur = reinterpret_cast<T*>(a.u) + (size_t)t * H;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int col = (c * TPR + tid) * VEC;
    float wb[VEC];
    load_param(a.w_before, a.param_bf16, col, H - col, 1.f, wb);
#pragma unroll
    for (int i = 0; i < VEC; ++i) out[c][i] *= r * wb[i];
    store_piece(ur + col, H - col, out[c]);
  }
}

// With xhat = x rx, yhat = y ry (or y), w = beta scale w_after and g the gate:
//   D    = d_x + rx (du w_before - xhat mean(du w_before xhat))
//   d_y  = ry (D w g - yhat mean(D w g yhat))      (without a norm after: D w g)
//   d_gate = (1 - g) sum(D w g yhat) per token, (1 - g) D w g yhat per element
//   column sums: du xhat (d_w_before); D g yhat (d_scale and d_w_after, scaled at the end)
template <class T, int TPR, int NV, bool BLOCK>
__global__ __launch_bounds__(block_threads(TPR)) void norm_backward(NormArgs a) {
  constexpr int VEC = kVec<T>, GROUPS = block_threads(TPR) / TPR;
  __shared__ float s_sum[2 * 3 * TPR / 64], s_sum2[2 * TPR / 64];
  int turn = 0, turn2 = 0;
  const int tid = threadIdx.x & (TPR - 1);
  const int group = blockIdx.x * GROUPS + threadIdx.x / TPR;
  const int H = a.H;
  const float inv_h = 1.f / (float)H;
  const bool before = a.w_before != nullptr, after = BLOCK && a.w_after != nullptr;
  float c_before[NV][VEC], c_block[NV][VEC];
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < VEC; ++i) c_before[c][i] = c_block[c][i] = 0.f;

  for (int t = group; t < a.T; t += (int)gridDim.x * GROUPS) {
    const T* xr = reinterpret_cast<const T*>(a.x) + (size_t)t * a.ldx;
    const T* yr = reinterpret_cast<const T*>(a.y) + (size_t)t * a.ldy;
    const T* gr = reinterpret_cast<const T*>(a.gate) + (size_t)t * a.ld_gate;
    const T* dxr = reinterpret_cast<const T*>(a.d_x) + (size_t)t * a.ld_dx;
    const T* dur = reinterpret_cast<const T*>(a.d_u) + (size_t)t * a.ld_du;
    Piece<T> xs[NV], ys[NV], dxs[NV], dus[NV];
    float sums[3] = {0.f, 0.f, 0.f};  // x x, du w_before x, y y
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if (before) {
        xs[c] = load_piece(xr + col, H - col);
        dus[c] = load_piece(dur + col, H - col);
      }
      dxs[c] = a.d_x != nullptr ? load_piece(dxr + col, H - col) : Piece<T>{{0u, 0u, 0u, 0u}};
      if constexpr (BLOCK) ys[c] = load_piece(yr + col, H - col);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if (before) {
        float wb[VEC];
        load_param(a.w_before, a.param_bf16, col, H - col, 1.f, wb);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          sums[0] += xs[c].at(i) * xs[c].at(i);
          sums[1] += dus[c].at(i) * wb[i] * xs[c].at(i);
        }
      }
      if (after) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) sums[2] += ys[c].at(i) * ys[c].at(i);
      }
    }
    row_sums<TPR>(sums, s_sum, turn);
    const float rx = 1.f / sqrtf(sums[0] * inv_h + a.eps);
    const float mx = rx * rx * sums[1] * inv_h;  // mean(du w xhat) = rx sums[1] / H
    const float ry = after ? 1.f / sqrtf(sums[2] * inv_h + a.eps) : 1.f;
    float gate = 1.f, not_gate = 0.f;
    if (BLOCK && a.gate_kind == MGG_GATE_TOKEN) sigmoid_parts(to_f32(*gr), gate, not_gate);

    float d[NV][VEC];  // D, then D w g
    float dot[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) d[c][i] = dxs[c].at(i);
      if (before) {
        float wb[VEC];
        load_param(a.w_before, a.param_bf16, col, H - col, 1.f, wb);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float x = xs[c].at(i), du = dus[c].at(i);
          d[c][i] += rx * (du * wb[i] - x * mx);
          c_before[c][i] += du * (x * rx);
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = a.alpha * d[c][i];
      store_piece(reinterpret_cast<T*>(a.d_x_in) + (size_t)t * H + col, H - col, o);
      if constexpr (BLOCK) {
        float wa[VEC], sc[VEC], dg[VEC];
        load_param(a.w_after, a.param_bf16, col, H - col, 1.f, wa);
        load_param(a.scale, a.param_bf16, col, H - col, 1.f, sc);
        Piece<T> gs;
        if (a.gate_kind == MGG_GATE_ELEMENT) gs = load_piece(gr + col, H - col);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (a.gate_kind == MGG_GATE_ELEMENT) sigmoid_parts(gs.at(i), gate, not_gate);
          const float yhat = ys[c].at(i) * ry;
          c_block[c][i] += d[c][i] * gate * yhat;
          d[c][i] *= a.beta * sc[i] * wa[i] * gate;
          dot[0] += d[c][i] * yhat;
          dg[i] = not_gate * (d[c][i] * yhat);
        }
        if (a.gate_kind == MGG_GATE_ELEMENT)
          store_piece(reinterpret_cast<T*>(a.d_gate) + (size_t)t * H + col, H - col, dg);
      }
    }
    if constexpr (BLOCK) {
      row_sums<TPR>(dot, s_sum2, turn2);
      if (a.gate_kind == MGG_GATE_TOKEN && tid == 0)
        reinterpret_cast<T*>(a.d_gate)[t] = from_f32<T>(not_gate * dot[0]);
      const float my = after ? ry * dot[0] * inv_h : 0.f;  // times y: yhat mean / 1
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int col = (c * TPR + tid) * VEC;
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = ry * (d[c][i] - ys[c].at(i) * my);
        store_piece(reinterpret_cast<T*>(a.d_y) + (size_t)t * H + col, H - col, o);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int col = (c * TPR + tid) * VEC + i;
      if (col < H) {
        if (before) a.part_before[(size_t)group * H + col] = c_before[c][i];
        if constexpr (BLOCK)
          if (a.part_block != nullptr) a.part_block[(size_t)group * H + col] = c_block[c][i];
      }
    }
}

constexpr int kSumCols = 16, kSumStrips = 16;

// Adds the row groups' column sums. blockIdx.y: 0 the norm before, 1 the block's.
__global__ __launch_bounds__(kSumCols* kSumStrips) void norm_column_sums(
    NormArgs a, int groups, float* d_scale, float* d_w_after, float* d_w_before) {
  __shared__ double s_part[kSumStrips][kSumCols];
  const float* part = blockIdx.y == 0 ? a.part_before : a.part_block;
  if (part == nullptr) return;
  const int col = threadIdx.x % kSumCols, strip = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + col;
  double sum = 0.0;
  if (c < a.H)
    for (int g = strip; g < groups; g += kSumStrips) sum += (double)part[(size_t)g * a.H + c];
  s_part[strip][col] = sum;
  __syncthreads();
  if (strip != 0 || c >= a.H) return;
  for (int i = 1; i < kSumStrips; ++i) sum += s_part[i][col];
  if (blockIdx.y == 0) {
    d_w_before[c] = (float)sum;
    return;
  }
  float sc[1], wa[1];
  load_param(a.scale, a.param_bf16, c, 1, 1.f, sc);
  load_param(a.w_after, a.param_bf16, c, 1, 1.f, wa);
  if (d_scale != nullptr) d_scale[c] = (float)(sum * (double)a.beta * (double)wa[0]);
  if (d_w_after != nullptr) d_w_after[c] = (float)(sum * (double)a.beta * (double)sc[0]);
}

// Row groups of the backward kernel, each with its own column sums: enough to fill the chip,
// and at least eight rows each where there are as many, so that the sums' traffic stays small
// next to the rows'.
// A whole number of workgroups' groups: the last may have no rows.
int row_groups(int T, int tpr) {
  const int per = block_threads(tpr) / tpr;
  const int most = tpr == 64 ? 2048 : tpr == 256 ? 512 : 256;
  return cdiv(std::max(1, std::min(most, cdiv(T, 8))), per) * per;
}

// Threads to a row: a wave up to four pieces a lane, then 256 threads, then 1024.
int threads_per_row(int H, int vec) {
  return H <= 64 * vec * 4 ? 64 : H <= 256 * vec * 4 ? 256 : 1024;
}

template <class F>
void with_shape(int H, int vec, F f) {
  using std::integral_constant;
  const int tpr = threads_per_row(H, vec), nv = cdiv(H, tpr * vec);
#define MGG_SHAPE(TPR, NV) \
  if (tpr == TPR && nv <= NV) return f(integral_constant<int, TPR>{}, integral_constant<int, NV>{})
  MGG_SHAPE(64, 1);
  MGG_SHAPE(64, 2);
  MGG_SHAPE(64, 4);
  MGG_SHAPE(256, 2);
  MGG_SHAPE(256, 4);
  MGG_SHAPE(1024, 2);
  MGG_SHAPE(1024, 4);
  MGG_SHAPE(1024, 8);
#undef MGG_SHAPE
}

const char* check_block(const NormArgs& a, mgg_act dt, mgg_act param, bool block) {
  if (!known(dt) || !known(param)) return "unknown element type";
  if (a.T < 0) return "T must not be negative";
  if (a.H < 1 || a.H > kMaxH) return "H must be in [1, 32768]";
  if (!(a.eps > 0.f) || !std::isfinite(a.eps)) return "eps must be positive and finite";
  if (!std::isfinite(a.alpha) || !std::isfinite(a.beta)) return "alpha and beta must be finite";
  const size_t e = elem_bytes(dt), p = elem_bytes(param);
  if (a.T > 0 && !a.x) return "null pointer";
  if (a.ldx < a.H) return "row strides must be at least H";
  if (!aligned(a.x, e) || !aligned(a.y, e) || !aligned(a.gate, e) || !aligned(a.d_x, e) ||
      !aligned(a.d_u, e) || !aligned(a.x_out, e) || !aligned(a.u, e) || !aligned(a.d_x_in, e) ||
      !aligned(a.d_y, e) || !aligned(a.d_gate, e))
    return "tensors must be aligned to their element";
  if (!aligned(a.scale, p) || !aligned(a.w_after, p) || !aligned(a.w_before, p))
    return "parameters must be aligned to their element";
  if (!block) return nullptr;
  if (a.gate_kind < MGG_GATE_NONE || a.gate_kind > MGG_GATE_ELEMENT) return "unknown gate kind";
  if (a.T > 0 && (!a.y || (a.gate_kind != MGG_GATE_NONE && !a.gate))) return "null pointer";
  if (a.ldy < a.H || (a.gate_kind == MGG_GATE_ELEMENT && a.ld_gate < a.H) ||
      (a.gate_kind == MGG_GATE_TOKEN && a.ld_gate < 1))
    return "row strides must be at least H (a token gate's step at least 1)";
  return nullptr;
}

NormArgs args_of(const mgg_block& b) {
  NormArgs a{};
  a.T = b.T;
  a.H = b.H;
  a.x = b.x;
  a.ldx = b.ldx;
  a.y = b.y;
  a.ldy = b.ldy;
  a.gate_kind = b.gate_kind;
  a.gate = b.gate;
  a.ld_gate = b.ld_gate;
  a.param_bf16 = b.param == MGG_ACT_BF16;
  a.scale = b.scale;
  a.w_after = b.w_after;
  a.w_before = b.w_before;
  a.alpha = b.alpha;
  a.beta = b.beta;
  a.eps = b.eps;
  return a;
}

template <bool BLOCK>
mgg_status run_forward(mgg_act dt, const NormArgs& a, hipStream_t stream) {
  if (a.T == 0) return MGG_OK;
  auto go = [&](auto elem) {
    with_shape(a.H, kVec<decltype(elem)>, [&](auto tpr, auto nv) {
      constexpr int threads = block_threads(tpr());
      norm_forward<decltype(elem), tpr(), nv(), BLOCK>
          <<<cdiv(a.T, threads / tpr()), threads, 0, stream>>>(a);
    });
  };
  if (dt == MGG_ACT_BF16) go(bf16_t{});
  else go(0.f);
  return launched();
}

template <bool BLOCK>
mgg_status run_backward(mgg_act dt, NormArgs a, float* d_scale, float* d_w_after,
                        float* d_w_before, void* workspace, size_t workspace_bytes,
                        hipStream_t stream) {
  const bool sums = d_scale || d_w_after || d_w_before;
  if (sums) {
    if (!workspace || workspace_bytes < block_residual_norm_backward_workspace(a.T, a.H))
      return fail(MGG_EINVAL, "the workspace is smaller than the workspace function says");
    if (!aligned(workspace, 256)) return fail(MGG_EINVAL, "the workspace must be 256-byte aligned");
  }
  int groups = 0;
  auto go = [&](auto elem) {
    constexpr int vec = kVec<decltype(elem)>;
    groups = row_groups(a.T, threads_per_row(a.H, vec));
    float* part = (float*)workspace;
    if (d_w_before) a.part_before = part;
    if (d_scale || d_w_after) a.part_block = part + round_up((size_t)groups * a.H, 64);
    if (a.T == 0) return;
    with_shape(a.H, vec, [&](auto tpr, auto nv) {
      constexpr int threads = block_threads(tpr());
      norm_backward<decltype(elem), tpr(), nv(), BLOCK>
          <<<groups / (threads / tpr()), threads, 0, stream>>>(a);
    });
  };
  if (dt == MGG_ACT_BF16) go(bf16_t{});
  else go(0.f);
  if (sums)
    norm_column_sums<<<dim3(cdiv(a.H, kSumCols), BLOCK ? 2 : 1), kSumCols * kSumStrips, 0,
                       stream>>>(a, a.T == 0 ? 0 : groups, d_scale, d_w_after, d_w_before);
  return launched();
}

}  // namespace

extern "C" {

mgg_status block_residual_norm(const mgg_block* block, void* x_out, void* u,
                               hipStream_t stream) {
  mgg_set_last_error("");
  if (!block) return fail(MGG_EINVAL, "null pointer");
  NormArgs a = args_of(*block);
  a.x_out = x_out;
  a.u = u;
  if (const char* err = check_block(a, block->dtype, block->param, true))
    return fail(MGG_EINVAL, err);
  if (a.T > 0 && !x_out) return fail(MGG_EINVAL, "null pointer");
  if (a.T > 0 && (u != nullptr) != (a.w_before != nullptr))
    return fail(MGG_EINVAL, "u and w_before go together");
  return run_forward<true>(block->dtype, a, stream);
}

size_t block_residual_norm_backward_workspace(int T, int H) {
  if (T < 0 || H < 1 || H > kMaxH) return 0;
  size_t bytes = 0;
  for (int vec : {kVec<bf16_t>, kVec<float>}) {
    const size_t groups = (size_t)row_groups(T, threads_per_row(H, vec));
    bytes = std::max(bytes, 2 * round_up(groups * H, 64) * 4);
  }
  return round_up(bytes, 256);
}

mgg_status block_residual_norm_backward(const mgg_block* block, const void* d_x, int64_t ld_dx,
                                        const void* d_u, int64_t ld_du, void* d_x_in,
                                        void* d_y, void* d_gate, float* d_scale,
                                        float* d_w_after, float* d_w_before, void* workspace,
                                        size_t workspace_bytes, hipStream_t stream) {
  mgg_set_last_error("");
  if (!block) return fail(MGG_EINVAL, "null pointer");
  NormArgs a = args_of(*block);
  a.d_x = d_x;
  a.ld_dx = ld_dx;
  a.d_u = d_u;
  a.ld_du = ld_du;
  a.d_x_in = d_x_in;
  a.d_y = d_y;
  a.d_gate = d_gate;
  if (const char* err = check_block(a, block->dtype, block->param, true))
    return fail(MGG_EINVAL, err);
  if (a.T > 0 && (!d_x_in || !d_y || (!d_x && !d_u))) return fail(MGG_EINVAL, "null pointer");
  if ((d_x && ld_dx < a.H) || (d_u && ld_du < a.H))
    return fail(MGG_EINVAL, "row strides must be at least H");
  if (a.T > 0 && (d_u != nullptr) != (a.w_before != nullptr))
    return fail(MGG_EINVAL, "d_u and w_before go together");
  if ((a.T > 0 && (d_gate != nullptr) != (a.gate_kind != MGG_GATE_NONE)) ||
      (d_scale != nullptr) != (a.scale != nullptr) ||
      (d_w_after != nullptr) != (a.w_after != nullptr) ||
      (d_w_before != nullptr) != (a.w_before != nullptr))
    return fail(MGG_EINVAL, "a gradient is given exactly when its input is");
  if (!aligned(d_scale, 4) || !aligned(d_w_after, 4) || !aligned(d_w_before, 4))
    return fail(MGG_EINVAL, "parameter gradients must be 4-byte aligned");
  return run_backward<true>(block->dtype, a, d_scale, d_w_after, d_w_before, workspace,
                            workspace_bytes, stream);
}

mgg_status block_norm(mgg_act dt, mgg_act param, int T, int H, const void* x, int64_t ldx,
                      const void* w, float eps, void* u, hipStream_t stream) {
  mgg_set_last_error("");
  NormArgs a{};
  a.T = T;
  a.H = H;
  a.x = x;
  a.ldx = ldx;
  a.param_bf16 = param == MGG_ACT_BF16;
  a.w_before = w;
  a.eps = eps;
  a.alpha = 1.f;
  a.u = u;
  if (const char* err = check_block(a, dt, param, false)) return fail(MGG_EINVAL, err);
  if (!w || (T > 0 && !u)) return fail(MGG_EINVAL, "null pointer");
  return run_forward<false>(dt, a, stream);
}

mgg_status block_norm_backward(mgg_act dt, mgg_act param, int T, int H, const void* x,
                               int64_t ldx, const void* w, float eps, const void* d_x,
                               int64_t ld_dx, const void* d_u, int64_t ld_du, void* d_x_in,
                               float* d_w, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  mgg_set_last_error("");
  NormArgs a{};
  a.T = T;
  a.H = H;
  a.x = x;
  a.ldx = ldx;
  a.param_bf16 = param == MGG_ACT_BF16;
  a.w_before = w;
  a.eps = eps;
  a.alpha = 1.f;
  a.d_x = d_x;
  a.ld_dx = ld_dx;
  a.d_u = d_u;
  a.ld_du = ld_du;
  a.d_x_in = d_x_in;
  if (const char* err = check_block(a, dt, param, false)) return fail(MGG_EINVAL, err);
  if (!w || !d_w || (T > 0 && (!d_u || !d_x_in))) return fail(MGG_EINVAL, "null pointer");
  if ((d_x && ld_dx < H) || (d_u && ld_du < H))
    return fail(MGG_EINVAL, "row strides must be at least H");
  if (!aligned(d_w, 4)) return fail(MGG_EINVAL, "parameter gradients must be 4-byte aligned");
  return run_backward<false>(dt, a, nullptr, nullptr, d_w, workspace, workspace_bytes, stream);
}

}  // extern "C"
