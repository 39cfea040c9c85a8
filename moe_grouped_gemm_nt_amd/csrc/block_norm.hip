// block_norm.hip - the norms before and after a block, fused with the block's gate, residual
// scale and residual sum, forward and backward (C ABI in include/mgg/layer_ops.h).
//
// TPR threads hold one row of each tensor in registers (NV 16-byte pieces a thread), so each
// tensor is read once and written once whatever the number of reductions over the row; the
// next row is loaded while one is worked on. The backward recomputes both norms' statistics
// from the rows it reads anyway; its sums over rows (norm weights, residual scale) are kept in
// registers per column while a workgroup walks its rows, written once per workgroup and added
// in a fixed order by a second kernel.
//
// Bound by HBM. Measured for 16384 rows of 7168 in bf16, gated per token, with both norms:
// forward 190 us, 4.9 TB/s; backward 310 us, 4.5 TB/s (a large copy reaches 5.2 TB/s). Streaming
// cache policies on its loads and stores gained 5 % there and lost as much or more on tensors
// that the last-level cache holds. Rows of more than two pieces for each of 1024 threads (bf16 above
// 16384 columns, float32 above 8192) spill registers, backward most: 2048 x 12288 in float32 181 us,
// where the bytes take 116, 2048 x 32768 in bf16 598 us, where they take 155. So do the kernels for
// a few rows of 1024 threads whose length is not whole pieces (forward, 600 rows of bf16: 12288 columns
// 18 us, 8193 columns 87 us), by the tails of three parameter vectors.

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
  float *part_before, *part_block;  // [workgroups][H]
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

// The piece at column `c` of a row of H. Rows are the wave's (a scalar address), columns the
// lane's (a 32-bit offset to it). WHOLE: H is a multiple of the piece. Otherwise the last piece
// is read so that it ends with the row, and settle() shifts it into place - later, where the
// piece is used: the wave that holds it would otherwise wait here for each of its loads. Rows
// shorter than a piece go by elements.
template <bool WHOLE, class T>
__device__ __forceinline__ Piece<T> load_piece(const T* row, int c, int H) {
  constexpr int VEC = kVec<T>;
  const char* base = reinterpret_cast<const char*>(row);
  Piece<T> r{{0u, 0u, 0u, 0u}};
  if (c >= H) return r;
  if (WHOLE || H >= VEC) {
    const int from = WHOLE ? c : min(c, H - VEC);
    __builtin_memcpy(&r, base + (uint32_t)from * (uint32_t)sizeof(T), 16);
  } else {
    uint64_t half[2] = {0, 0};
#pragma unroll 1
    for (int i = 0; i < H - c; ++i) {
      uint64_t bits = 0;
      __builtin_memcpy(&bits, base + (size_t)(c + i) * sizeof(T), sizeof(T));
      const int at = i * (int)sizeof(T) * 8;
      half[0] |= at < 64 ? bits << at : 0;
      half[1] |= at < 64 ? 0 : bits << (at - 64);
    }
    __builtin_memcpy(&r, half, 16);
  }
  return r;
}
template <bool WHOLE, class T>
__device__ __forceinline__ void settle(Piece<T>& r, int c, int H) {
  if constexpr (!WHOLE) {
    if (H < kVec<T> || c >= H || c + kVec<T> <= H) return;
    const uint32_t by = (uint32_t)(c + kVec<T> - H) * (uint32_t)sizeof(T) * 8;  // bits, below 128
    if (by & 64) r = Piece<T>{{r.w[2], r.w[3], 0u, 0u}};
    if (by & 32) r = Piece<T>{{r.w[1], r.w[2], r.w[3], 0u}};
    if (by & 16)
      r = Piece<T>{{r.w[0] >> 16 | r.w[1] << 16, r.w[1] >> 16 | r.w[2] << 16,
                    r.w[2] >> 16 | r.w[3] << 16, r.w[3] >> 16}};
  }
}

template <bool WHOLE, class T>
__device__ __forceinline__ void store_piece(T* row, int c, int H, const float (&v)[kVec<T>]) {
  constexpr int VEC = kVec<T>;
  if (c >= H) return;
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_bits(v[2 * i]) | (uint32_t)bf16_bits(v[2 * i + 1]) << 16;
  }
  char* to = reinterpret_cast<char*>(row) + (uint32_t)c * (uint32_t)sizeof(T);
  if (WHOLE || H - c >= VEC) {
    __builtin_memcpy(to, w, 16);
    return;
  }
  // the row's last few: eight, four and two bytes as its length asks for them
  const int n = (H - c) * (int)sizeof(T);
  uint32_t a = w[0], b = w[1];
  if (n & 8) {
    __builtin_memcpy(to, w, 8);
    to += 8;
    a = w[2], b = w[3];
  }
  if (n & 4) {
    __builtin_memcpy(to, &a, 4);
    to += 4;
    a = b;
  }
  if (n & 2) {
    const uint16_t last = (uint16_t)a;
    __builtin_memcpy(to, &last, 2);
  }
}

// VEC values of a parameter vector of H from column `c`; `missing` where there is no vector, anything
// finite past its end. WHOLE: H and c are multiples of VEC.
template <bool WHOLE, int VEC>
__device__ __forceinline__ void load_param(const void* p, int bf16, int c, int H, float missing,
                                           float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = missing;
  if (p == nullptr || (WHOLE && c >= H)) return;
  const char* base = reinterpret_cast<const char*>(p);
  if (WHOLE || c + VEC <= H) {
    if (bf16) {
      uint16_t bits[VEC];
      __builtin_memcpy(bits, base + (uint32_t)c * 2u, VEC * 2);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = to_f32(bf16_t{bits[i]});
    } else {
      __builtin_memcpy(v, base + (uint32_t)c * 4u, VEC * 4);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const uint32_t at = (uint32_t)min(c + i, H - 1);
    v[i] = bf16 ? to_f32(reinterpret_cast<const bf16_t*>(p)[at])
                : reinterpret_cast<const float*>(p)[at];
  }
}

// Sums of N values over the TPR threads of a row, in a fixed order. `s` holds
// [2][N][waves] floats; `turn` alternates its halves, so one barrier a sum is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* s, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lanes_sum<TPR < 64 ? TPR : 64>(v[i]);
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
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<W>(half[i * W + (threadIdx.x & (W - 1))]);
  }
}

// Workgroups hold several rows of a wave or less, or one row.
constexpr int block_threads(int tpr) { return tpr <= 64 ? 256 : tpr; }

// The thread's row group in its workgroup: the same for a whole wave from 64 threads a row on.
template <int TPR>
__device__ __forceinline__ int group_of() {
  if constexpr (TPR < 64) return threadIdx.x / TPR;
  return __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
}

// What multiplies the columns of a row: `block` = scale * w_after and `before` = w_before, 1
// where there is none. STAGED: a workgroup that takes many rows keeps both in LDS as float32
// (two vectors of Hp floats); read again for every row from memory they are several times the
// bytes of a bf16 row.
template <int VEC, bool STAGED, bool WHOLE>
struct Columns {
  const NormArgs& a;
  const float* lds;
  int Hp;
  __device__ __forceinline__ void stage(float* to) const {
    for (int c = threadIdx.x * VEC; c < Hp; c += blockDim.x * VEC) {
      float wa[VEC], sc[VEC], wb[VEC];
      from_memory(a.w_after, c, wa);
      from_memory(a.scale, c, sc);
      from_memory(a.w_before, c, wb);
#pragma unroll
      for (int i = 0; i < VEC; ++i) wa[i] *= sc[i];
      __builtin_memcpy(__builtin_assume_aligned(to + c, 16), wa, VEC * 4);
      __builtin_memcpy(__builtin_assume_aligned(to + Hp + c, 16), wb, VEC * 4);
    }
    __syncthreads();
  }
  __device__ __forceinline__ void from_memory(const void* p, int c, float (&v)[VEC]) const {
    load_param<WHOLE>(p, a.param_bf16, c, a.H, 1.f, v);
  }
  // Read anew for every row: kept in registers over the rows they cost more in occupancy (and, with
  // a gate per element, spills) than they save.
  __device__ __forceinline__ void from_lds(int c, float (&v)[VEC]) const {
    asm volatile("" ::: "memory");
    __builtin_memcpy(v, __builtin_assume_aligned(lds + c, 16), VEC * 4);
  }
  // for VEC columns from `c`; columns past the row give anything finite
  __device__ __forceinline__ void block(int c, float (&v)[VEC]) const {
    if constexpr (STAGED) {
      from_lds(min(c, Hp - VEC), v);
    } else {
      float sc[VEC];
      from_memory(a.w_after, c, v);
      from_memory(a.scale, c, sc);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] *= sc[i];
    }
  }
  __device__ __forceinline__ void before(int c, float (&v)[VEC]) const {
    if constexpr (STAGED) from_lds(Hp + min(c, Hp - VEC), v);
    else from_memory(a.w_before, c, v);
  }
};

template <class T>
__device__ __forceinline__ const T* row_of(const void* p, int64_t ld, int t) {
  return reinterpret_cast<const T*>(p) + (size_t)t * ld;
}

// Row groups (TPR threads) take rows group, group + groups, ...; the next row's loads are under
// way while one is worked on.
template <class T, int TPR, int NV, bool BLOCK, bool STAGED, bool WHOLE>
__global__ __launch_bounds__(block_threads(TPR)) void norm_forward(NormArgs a) {
  constexpr int VEC = kVec<T>, GROUPS = block_threads(TPR) / TPR;
  __shared__ float s_sum[cdiv(2 * TPR, 64)];
  extern __shared__ __align__(16) float s_columns[];
  const int H = a.H;
  const Columns<VEC, STAGED, WHOLE> columns{a, s_columns, (H + VEC - 1) / VEC * VEC};
  if constexpr (STAGED) columns.stage(s_columns);
  int turn = 0;
  const int tid = threadIdx.x & (TPR - 1);
  const int stride = (int)gridDim.x * GROUPS;
  struct Row {
    Piece<T> x[NV], y[NV];
  };
  auto load = [&](int t) {
    Row r;
    const T *x = row_of<T>(a.x, a.ldx, t), *y = row_of<T>(a.y, a.ldy, t);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if constexpr (BLOCK) r.y[c] = load_piece<WHOLE>(y, col, H);
      r.x[c] = load_piece<WHOLE>(x, col, H);
    }
    return r;
  };
  int t = blockIdx.x * GROUPS + group_of<TPR>();
  if (t >= a.T) return;  // whole waves, and whole workgroups where a barrier follows
  Row next = load(t);
  for (; t < a.T; t += stride) {
    Row in = next;
    if (t + stride < a.T) next = load(t + stride);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if constexpr (BLOCK) settle<WHOLE>(in.y[c], col, H);
      settle<WHOLE>(in.x[c], col, H);
    }
    float out[NV][VEC];
    if constexpr (BLOCK) {
      const T* gr = row_of<T>(a.gate, a.ld_gate, t);
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
          for (int i = 0; i < VEC; ++i) sum[0] += in.y[c].at(i) * in.y[c].at(i);
        row_sums<TPR>(sum, s_sum, turn);
        row *= 1.f / sqrtf(sum[0] / (float)H + a.eps);
      }
      T* outr = reinterpret_cast<T*>(a.x_out) + (size_t)t * H;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int col = (c * TPR + tid) * VEC;
        float w[VEC];
        columns.block(col, w);
        Piece<T> gs;
        if (a.gate_kind == MGG_GATE_ELEMENT) {
          gs = load_piece<WHOLE>(gr, col, H);
          settle<WHOLE>(gs, col, H);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float g = row * w[i];
          if (a.gate_kind == MGG_GATE_ELEMENT) {
            float q, not_q;
            sigmoid_parts(gs.at(i), q, not_q);
            g *= q;
          }
          out[c][i] = fmaf(in.y[c].at(i), g, a.alpha * in.x[c].at(i));
        }
        store_piece<WHOLE>(outr, col, H, out[c]);
      }
      if (a.w_before == nullptr) continue;
    } else {
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) out[c][i] = in.x[c].at(i);
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
      columns.before(col, wb);
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[c][i] *= r * wb[i];
      store_piece<WHOLE>(ur, col, H, out[c]);
    }
  }
}

// With xhat = x rx, yhat = y ry (or y), w = beta scale w_after and g the gate:
//   D    = d_x + rx (du w_before - xhat mean(du w_before xhat))
//   d_y  = ry (D w g - yhat mean(D w g yhat))      (without a norm after: D w g)
//   d_gate = (1 - g) sum(D w g yhat) per token, (1 - g) D w g yhat per element
//   column sums: du xhat (d_w_before); D g yhat (d_scale and d_w_after, scaled at the end)
// BLOCK: 0 the norm before a block alone, 1 with a block, 2 with a block gated per element.
template <class T, int TPR, int NV, int BLOCK, bool STAGED, bool WHOLE>
__global__ __launch_bounds__(block_threads(TPR)) void norm_backward(NormArgs a) {
  constexpr int VEC = kVec<T>, GROUPS = block_threads(TPR) / TPR;
  constexpr bool ELEMENT = BLOCK == 2;
  __shared__ float s_sum[cdiv(2 * 3 * TPR, 64)], s_sum2[cdiv(2 * TPR, 64)];
  extern __shared__ __align__(16) float s_columns[];
  int turn = 0, turn2 = 0;
  const int tid = threadIdx.x & (TPR - 1);
  const int group = blockIdx.x * GROUPS + group_of<TPR>();
  const int H = a.H;
  const Columns<VEC, STAGED, WHOLE> columns{a, s_columns, (H + VEC - 1) / VEC * VEC};
  if constexpr (STAGED) columns.stage(s_columns);
  const float inv_h = 1.f / (float)H;
  const bool before = a.w_before != nullptr, after = BLOCK != 0 && a.w_after != nullptr;
  float c_before[NV][VEC], c_block[NV][VEC];
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < VEC; ++i) c_before[c][i] = c_block[c][i] = 0.f;

  // with one piece of each tensor a thread there are registers for the next row's
  constexpr bool AHEAD = NV == 1;
  struct Row {
    Piece<T> x[NV], y[NV], dx[NV], du[NV];
  };
  auto load = [&](int t) {
    Row r;
    const T *x = row_of<T>(a.x, a.ldx, t), *y = row_of<T>(a.y, a.ldy, t);
    const T *dx = row_of<T>(a.d_x, a.ld_dx, t), *du = row_of<T>(a.d_u, a.ld_du, t);
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if (before) {
        r.x[c] = load_piece<WHOLE>(x, col, H);
        r.du[c] = load_piece<WHOLE>(du, col, H);
      }
      if constexpr (BLOCK != 0) r.y[c] = load_piece<WHOLE>(y, col, H);
      r.dx[c] = a.d_x != nullptr ? load_piece<WHOLE>(dx, col, H) : Piece<T>{{0u, 0u, 0u, 0u}};
    }
    return r;
  };
  const int stride = (int)gridDim.x * GROUPS;
  Row next;
  if (AHEAD && group < a.T) next = load(group);
  for (int t = group; t < a.T; t += stride) {
    Row in;
    if constexpr (AHEAD) {
      in = next;
      if (t + stride < a.T) next = load(t + stride);
    } else {
      in = load(t);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if (before) {
        settle<WHOLE>(in.x[c], col, H);
        settle<WHOLE>(in.du[c], col, H);
      }
      if constexpr (BLOCK != 0) settle<WHOLE>(in.y[c], col, H);
      settle<WHOLE>(in.dx[c], col, H);
    }
    const Piece<T>(&xs)[NV] = in.x, (&ys)[NV] = in.y, (&dxs)[NV] = in.dx, (&dus)[NV] = in.du;
    const T* gr = row_of<T>(a.gate, a.ld_gate, t);
    float sums[3] = {0.f, 0.f, 0.f};  // x x, du w_before x, y y
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int col = (c * TPR + tid) * VEC;
      if (before) {
        float wb[VEC];
        columns.before(col, wb);
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
    if (BLOCK == 1 && a.gate_kind == MGG_GATE_TOKEN) sigmoid_parts(to_f32(*gr), gate, not_gate);

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
        columns.before(col, wb);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float x = xs[c].at(i), du = dus[c].at(i);
          d[c][i] += rx * (du * wb[i] - x * mx);
          c_before[c][i] += du * (x * rx);
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = a.alpha * d[c][i];
      store_piece<WHOLE>(reinterpret_cast<T*>(a.d_x_in) + (size_t)t * H, col, H, o);
      if constexpr (BLOCK != 0) {
        float w[VEC], dg[VEC];
        columns.block(col, w);
        Piece<T> gs;
        if constexpr (ELEMENT) {
          gs = load_piece<WHOLE>(gr, col, H);
          settle<WHOLE>(gs, col, H);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if constexpr (ELEMENT) sigmoid_parts(gs.at(i), gate, not_gate);
          const float yhat = ys[c].at(i) * ry;
          c_block[c][i] += d[c][i] * gate * yhat;
          d[c][i] *= a.beta * w[i] * gate;
          const float dy = d[c][i] * yhat;
          dot[0] += dy;
          dg[i] = not_gate * dy;
        }
        if constexpr (ELEMENT)
          store_piece<WHOLE>(reinterpret_cast<T*>(a.d_gate) + (size_t)t * H, col, H, dg);
      }
    }
    if constexpr (BLOCK != 0) {
      row_sums<TPR>(dot, s_sum2, turn2);
      if (BLOCK == 1 && a.gate_kind == MGG_GATE_TOKEN && tid == 0)
        reinterpret_cast<T*>(a.d_gate)[t] = from_f32<T>(not_gate * dot[0]);
      const float my = after ? ry * dot[0] * inv_h : 0.f;  // yhat mean(..) = y my
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int col = (c * TPR + tid) * VEC;
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = ry * (d[c][i] - ys[c].at(i) * my);
        store_piece<WHOLE>(reinterpret_cast<T*>(a.d_y) + (size_t)t * H, col, H, o);
      }
    }
  }
  // the workgroup's sums: those of its groups, one after another
  auto write_sums = [&](float (&sums)[NV][VEC], float* part) {
    if constexpr (GROUPS == 1) {
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int col = (c * TPR + tid) * VEC + i;
          if (col < H) part[(size_t)blockIdx.x * H + col] = sums[c][i];
        }
    } else {
      __shared__ float s_part[TPR * NV * VEC];
      for (int g = 0; g < GROUPS; ++g) {
        __syncthreads();
        if ((int)threadIdx.x / TPR == g) {
#pragma unroll
          for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              float& at = s_part[(c * TPR + tid) * VEC + i];
              at = g == 0 ? sums[c][i] : at + sums[c][i];
            }
        }
      }
      __syncthreads();
      for (int col = threadIdx.x; col < H; col += block_threads(TPR))
        part[(size_t)blockIdx.x * H + col] = s_part[col];
    }
  };
  if (before) write_sums(c_before, a.part_before);
  if (BLOCK != 0 && a.part_block != nullptr) write_sums(c_block, a.part_block);
}

constexpr int kSumCols = 16, kSumStrips = 64, kSumFold = 8;

// Adds the workgroups' column sums. blockIdx.y: 0 the norm before, 1 the block's.
__global__ __launch_bounds__(kSumCols* kSumStrips) void norm_column_sums(
    NormArgs a, int blocks, float* d_scale, float* d_w_after, float* d_w_before) {
  __shared__ double s_part[kSumStrips][kSumCols];
  const float* part = blockIdx.y == 0 ? a.part_before : a.part_block;
  if (part == nullptr) return;
  const int col = threadIdx.x % kSumCols, strip = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + col;
  double sum = 0.0;
  if (c < a.H)
#pragma unroll 8
    for (int g = strip; g < blocks; g += kSumStrips) sum += (double)part[(size_t)g * a.H + c];
  s_part[strip][col] = sum;
  __syncthreads();
  if (strip < kSumStrips / kSumFold) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kSumFold; ++i) sum += s_part[strip * kSumFold + i][col];
  }
  __syncthreads();
  if (strip < kSumStrips / kSumFold) s_part[strip][col] = sum;
  __syncthreads();
  if (strip != 0 || c >= a.H) return;
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kSumStrips / kSumFold; ++i) sum += s_part[i][col];
  if (blockIdx.y == 0) {
    d_w_before[c] = (float)sum;
    return;
  }
  float sc[1], wa[1];
  load_param<false>(a.scale, a.param_bf16, c, a.H, 1.f, sc);
  load_param<false>(a.w_after, a.param_bf16, c, a.H, 1.f, wa);
  if (d_scale != nullptr) d_scale[c] = (float)(sum * (double)a.beta * (double)wa[0]);
  if (d_w_after != nullptr) d_w_after[c] = (float)(sum * (double)a.beta * (double)sc[0]);
}

// Threads to a row. Short rows go to a half wave or a wave of their own. The forward kernels take two 16-byte
// pieces of each tensor a thread, the backward kernels one, which leaves registers to load the
// next row ahead, as long as a workgroup can hold the row so. Rows of 65 to 128 pieces are a wave's
// with two pieces in both: the backward kernels do without the next row's loads there (30000 x 777 in
// bf16 gated per token 89 us, where its bytes take 54).
int threads_forward(int H, int vec) {
  const int pieces = cdiv(H, vec);
  return pieces <= 32 ? 32 : pieces <= 128 ? 64 : pieces <= 512 ? 256 : pieces <= 1024 ? 512 : 1024;
}
int threads_backward(int H, int vec) {
  const int pieces = cdiv(H, vec);
  return pieces <= 32 ? 32 : pieces <= 128 ? 64 : pieces <= 256 ? 256 : pieces <= 512 ? 512 : 1024;
}

// Row groups when 1024 threads are resident on each of the 256 CUs, the most that the backward
// kernels' registers allow, and what the forward kernels' LDS leaves room for on wide rows.
int resident_groups(int tpr) { return 256 * 1024 / tpr; }

// Most workgroups of the forward kernels that do not keep the parameters: a launch holds fewer than
// 2^32 threads. Further rows are walked.
constexpr int kMostBlocks = 1 << 20;

// Workgroups of the backward kernel, each with its own column sums: one round of resident ones,
// with at least two rows for each of a workgroup's groups where there are as many, so that the
// sums' traffic stays small next to the rows'.
int row_blocks(int T, int tpr) {
  const int per = block_threads(tpr) / tpr;
  const int rows = std::max(2, cdiv(T, resident_groups(tpr)));
  return std::max(1, cdiv(T, rows * per));
}

// Whether workgroups keep the columns' parameters in LDS: when each takes several rows, and two
// workgroups' vectors fit a CU.
constexpr int kStagedH = 8192;
bool staged(int T, int H, int groups) { return H <= kStagedH && T >= 4 * groups; }
// Whether rows of a shape can be that short: those with more than one piece a thread hold more pieces
// than the shape with half as many.
constexpr bool may_stage(int tpr, int nv, int vec) { return nv == 1 || tpr * (nv / 2) * vec < kStagedH; }
size_t staged_bytes(int H, int vec) { return (size_t)cdiv(H, vec) * vec * 2 * sizeof(float); }

// Calls f(threads to a row, pieces a thread, whether H is whole pieces) as compile-time constants.
template <bool BACKWARD, int VEC, class F>
void with_shape(int H, F f) {
  using std::integral_constant;
  const int tpr = BACKWARD ? threads_backward(H, VEC) : threads_forward(H, VEC);
  const int nv = cdiv(H, tpr * VEC);
  const bool whole = H % VEC == 0;
#define MGG_SHAPE(TPR, NV)                                                                      \
  if (tpr == TPR && nv <= NV)                                                                   \
  return whole                                                                                  \
             ? f(integral_constant<int, TPR>{}, integral_constant<int, NV>{}, std::true_type{}) \
             : f(integral_constant<int, TPR>{}, integral_constant<int, NV>{}, std::false_type{})
  MGG_SHAPE(32, 1);
  MGG_SHAPE(64, 1);
  MGG_SHAPE(64, 2);
  MGG_SHAPE(256, 1);
  if constexpr (BACKWARD) {
    MGG_SHAPE(512, 1);
    MGG_SHAPE(1024, 1);
  } else {
    MGG_SHAPE(256, 2);
    MGG_SHAPE(512, 2);
  }
  MGG_SHAPE(1024, 2);
  MGG_SHAPE(1024, 4);
  if constexpr (1024 * 4 * VEC < kMaxH) {
    MGG_SHAPE(1024, 8);
  }
#undef MGG_SHAPE
}

// Launches a kernel with the columns staged or not.
template <class K>
bool launch(K kernel, int blocks, int threads, size_t lds, const NormArgs& a,
            hipStream_t stream) {
  if (lds > 60 * 1024 &&
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                          (int)lds) != hipSuccess)
    return false;
  kernel<<<blocks, threads, lds, stream>>>(a);
  return true;
}

const char* check_block(const NormArgs& a, mgg_act dt, mgg_act param, bool block) {
  if (!known(dt) || !known(param)) return "unknown element type";
  if (a.T < 0 || a.T > kMaxRows) return "T must be in [0, 2^30]";
  if (a.H < 1 || a.H > kMaxH) return "H must be in [1, 32768]";
  // from a subnormal eps on the square of 1 / sqrt(eps) is infinite
  if (!(a.eps >= 1.17549435e-38f) || !std::isfinite(a.eps))
    return "eps must be positive, normal and finite";
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
  bool ok = true;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    with_shape<false, kVec<T>>(a.H, [&](auto tpr, auto nv, auto whole) {
      constexpr int threads = block_threads(tpr()), per = threads / tpr();
      const int groups = resident_groups(tpr());
      if constexpr (may_stage(tpr(), nv(), kVec<T>)) {
        if (staged(a.T, a.H, groups)) {
          ok = launch(norm_forward<T, tpr(), nv(), BLOCK, true, whole()>, groups / per, threads,
                      staged_bytes(a.H, kVec<T>), a, stream);
          return;
        }
      }
      ok = launch(norm_forward<T, tpr(), nv(), BLOCK, false, whole()>,
                  std::min(cdiv(a.T, per), kMostBlocks), threads, 0, a, stream);
    });
  };
  if (dt == MGG_ACT_BF16) go(bf16_t{});
  else go(0.f);
  return ok ? launched() : fail(MGG_EHIP, "hipFuncSetAttribute failed");
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
  int blocks = 0;
  bool ok = true;
  auto go = [&](auto elem) {
    using T = decltype(elem);
    constexpr int vec = kVec<T>;
    blocks = row_blocks(a.T, threads_backward(a.H, vec));
    float* part = (float*)workspace;
    if (d_w_before) a.part_before = part;
    if (d_scale || d_w_after) a.part_block = part + round_up((size_t)blocks * a.H, 64);
    if (a.T == 0) return;
    with_shape<true, vec>(a.H, [&](auto tpr, auto nv, auto whole) {
      constexpr int threads = block_threads(tpr());
      auto go = [&](auto what) {
        if constexpr (may_stage(tpr(), nv(), vec)) {
          if (staged(a.T, a.H, blocks * (threads / tpr()))) {
            ok = launch(norm_backward<T, tpr(), nv(), what(), true, whole()>, blocks, threads,
                        staged_bytes(a.H, vec), a, stream);
            return;
          }
        }
        ok = launch(norm_backward<T, tpr(), nv(), what(), false, whole()>, blocks, threads, 0, a,
                    stream);
      };
      using std::integral_constant;
      if constexpr (!BLOCK) go(integral_constant<int, 0>{});
      else if (a.gate_kind == MGG_GATE_ELEMENT) go(integral_constant<int, 2>{});
      else go(integral_constant<int, 1>{});
    });
  };
  if (dt == MGG_ACT_BF16) go(bf16_t{});
  else go(0.f);
  if (!ok) return fail(MGG_EHIP, "hipFuncSetAttribute failed");
  if (sums)
    norm_column_sums<<<dim3(cdiv(a.H, kSumCols), BLOCK ? 2 : 1), kSumCols * kSumStrips, 0,
                       stream>>>(a, a.T == 0 ? 0 : blocks, d_scale, d_w_after, d_w_before);
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
  if (T < 0 || T > kMaxRows || H < 1 || H > kMaxH) return 0;
  size_t bytes = 0;
  for (int vec : {kVec<bf16_t>, kVec<float>}) {
    const size_t blocks = (size_t)row_blocks(T, threads_backward(H, vec));
    bytes = std::max(bytes, 2 * round_up(blocks * H, 64) * 4);
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
