// route.hip - top-k routing with per-expert counts and a balance loss, and the gradient of
// the logits (C ABI in include/mgg/layer_ops.h: route_topk, route_topk_backward).
//
// L lanes share a row, each holding V = ceil(G / L) logits in registers (expert e at lane
// e % L, slot e / L), so a row is read once and everything about it - its maximum, the sum
// of its exponentials, the k selections - is a reduction over registers and L lanes. Rows
// are dealt to workgroups in chunks of consecutive rows; a workgroup walks the sequences that
// its chunk meets and writes one partial (sum of p, counts) per chunk and sequence. Along
// that walk chunk + sequence strictly increases, so it numbers the partials without a table.
// A second kernel sums them in order of the chunks: float sums have one order, and the only
// atomics are integer counters.

#include "layer_common.h"

namespace {

using namespace mgg_layer;

constexpr int kThreads = 256;
constexpr int kMaxTopk = 32;
constexpr int kMaxExperts = 4096;
constexpr int kMaxSequences = 65535;  // grid.y of the summing kernel
// Workgroups that the rows of a large call are dealt to: four for each CU.
constexpr int kRowBlocks = 1024;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int T, G, k, S;
  int renormalize;
  float scale;
  const int32_t* seq_ends;
  int32_t* ids;
  float* weights;
  int rows_per_block;
  // partial sums, one row of G for each (chunk, sequence) pair; `counters`: column blocks of
  // the summing kernel that are done, per sequence
  float* part_prob;
  int32_t* part_count;
  int32_t* counters;
};

// What the row's scores are made of, from its maximum: `hat` is proportional to q within the
// row, and q = hat * to_q. Softmax: hat = e^(l - max). Sigmoid: q times e^-m with
// m = min(max, 0), so a row of very negative logits keeps its proportions.
template <bool SIGMOID>
struct Scores {
  float m, to_q;
  __device__ __forceinline__ explicit Scores(float row_max) {
    m = row_max == -INFINITY ? 0.f : (SIGMOID ? fminf(row_max, 0.f) : row_max);
    to_q = SIGMOID ? exp_neg(m) : 1.f;
  }
  __device__ __forceinline__ float hat(float l) const {
    if constexpr (!SIGMOID) return exp_neg(l - m);
    const float a = exp_neg(-fabsf(l));
    const float num = m < 0.f ? exp_neg(l - m) : (l < 0.f ? a : 1.f);
    return num / (1.f + a);
  }
  // 1 - sigmoid(l)
  __device__ __forceinline__ static float one_minus_q(float l) {
    const float a = exp_neg(-fabsf(l));
    return (l >= 0.f ? a : 1.f) / (1.f + a);
  }
};

// The smallest s >= from whose end lies past `row` (S if none). Ends raised to the largest
// earlier end keep the same answer, so they are compared as they stand. Called by the whole
// workgroup.
__device__ int sequence_of(const int32_t* ends, int S, int row, int from, int* s_found) {
  for (int base = from; base < S; base += kThreads) {
    const int s = base + (int)threadIdx.x;
    const bool past = s < S && ends[s] > row;
    const unsigned long long hit = __ballot(past);
    __syncthreads();  // the last reader of s_found is done
    if ((threadIdx.x & 63) == 0)
      s_found[threadIdx.x >> 6] = hit ? base + (int)threadIdx.x + __ffsll(hit) - 1 : INT32_MAX;
    __syncthreads();
    int first = INT32_MAX;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) first = min(first, s_found[w]);
    if (first != INT32_MAX) return first;
  }
  return S;
}

template <class T, int L, int V>
__device__ __forceinline__ void load_row(const T* row, int G, int lane, float (&l)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + L * v;
    l[v] = e < G ? to_f32(row[e]) : -INFINITY;
  }
}

template <int L, int V>
__device__ __forceinline__ float row_max(const float (&l)[V]) {
  float m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  return lanes_reduce<L>(m, [](float a, float b) { return fmaxf(a, b); });
}

// One row: probabilities p[v] (zero for padding slots), and ids and weights written.
// BIAS orders by q + bias in float64, where sums that float32 cannot tell apart still differ.
template <int L, int V, bool SIGMOID, bool BIAS>
__device__ __forceinline__ void route_row(const RouteArgs& a, int t, bool active, int lane,
                                          const float (&l)[V], float (&p)[V], int* s_count) {
  const Scores<SIGMOID> sc(row_max<L>(l));
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    p[v] = sc.hat(l[v]);
    sum += p[v];
  }
  sum = lanes_sum<L>(sum);
  const float inv_sum = sum == 0.f ? 0.f : 1.f / sum;

  using Key = std::conditional_t<BIAS, double, float>;
  Key key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (BIAS) {
      const int e = lane + L * v;
      const double q = 1.0 / (1.0 + exp(-(double)l[v]));
      key[v] = e < a.G && l[v] > -INFINITY ? q + (double)a.bias[e] : -INFINITY;
    } else {
      key[v] = l[v];
    }
  }
  int id[kMaxTopk / L > 0 ? cdiv(kMaxTopk, L) : 1];
  float w[kMaxTopk / L > 0 ? cdiv(kMaxTopk, L) : 1];
  float chosen = 0.f;
  for (int r = 0; r < a.k; ++r) {
    Key best = -INFINITY;
    int e = INT32_MAX;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool more = key[v] > best;  // false for NaN and -inf; the lower index wins a tie
      e = more ? lane + L * v : e;
      best = more ? key[v] : best;
    }
    const Key top = lanes_reduce<L>(best, [](Key x, Key y) { return x > y ? x : y; });
    e = lanes_reduce<L>(best == top ? e : INT32_MAX, [](int x, int y) { return min(x, y); });
    float hat = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + L * v == e) {
        hat = p[v];
        key[v] = -INFINITY;
      }
    hat = __shfl(hat, e & (L - 1), L);
    if (e == INT32_MAX) hat = 0.f;
    chosen += hat;
    if (s_count != nullptr && active && lane == 0 && e != INT32_MAX) atomicAdd(&s_count[e], 1);
    if ((r & (L - 1)) == lane) {
      id[r / L] = e == INT32_MAX ? -1 : e;
      w[r / L] = hat;
    }
  }
  const float to_w =
      a.scale * (a.renormalize ? (chosen == 0.f ? 0.f : 1.f / chosen)
                               : (SIGMOID ? sc.to_q : inv_sum));
  if (active) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(id) / sizeof(int)); ++i) {
      const int r = lane + L * i;
      if (r < a.k) {
        a.ids[(size_t)t * a.k + r] = id[i];
        a.weights[(size_t)t * a.k + r] = id[i] < 0 ? 0.f : w[i] * to_w;
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] *= inv_sum;
}

template <class T, int L, int V, bool SIGMOID, bool BIAS, bool STATS>
__global__ __launch_bounds__(kThreads) void route_rows(RouteArgs a) {
  extern __shared__ int s_dyn[];  // STATS: counts [G], sums [G]
  __shared__ int s_found[kThreads / 64];
  int* s_count = STATS ? s_dyn : nullptr;
  float* s_prob = reinterpret_cast<float*>(s_dyn + a.G);
  constexpr int RP = kThreads / L;  // rows at once
  const int lane = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  const int r0 = blockIdx.x * a.rows_per_block;
  const int r1 = min(a.T, r0 + a.rows_per_block);
  if constexpr (STATS)
    if (blockIdx.x == 0)
      for (int s = threadIdx.x; s < a.S; s += kThreads) a.counters[s] = 0;

  int row = r0, s = -1;
  while (row < r1) {
    int end = r1;
    if (a.seq_ends == nullptr) {
      s = 0;
    } else {
      s = sequence_of(a.seq_ends, a.S, row, s + 1, s_found);
      if (s == a.S) break;
      end = min(a.seq_ends[s], r1);
    }
    float acc[V];
    if constexpr (STATS) {
      __syncthreads();
      for (int e = threadIdx.x; e < a.G; e += kThreads) s_count[e] = 0;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.f;
    }
    for (int base = row; base < end; base += RP) {
      const int t = base + grp;
      const bool active = t < end;
      float l[V], p[V];
      load_row<T, L>(reinterpret_cast<const T*>(a.logits) + (size_t)min(t, end - 1) * a.ld,
                     a.G, lane, l);
      route_row<L, V, SIGMOID, BIAS>(a, t, active, lane, l, p, s_count);
      if constexpr (STATS) {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += active ? p[v] : 0.f;
      }
    }
    if constexpr (STATS) {
      // the groups' sums, added in the order of the groups
      for (int g = 0; g < RP; ++g) {
        __syncthreads();
        if (grp == g) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int e = lane + L * v;
            if (e < a.G) s_prob[e] = g == 0 ? acc[v] : s_prob[e] + acc[v];
          }
        }
      }
      __syncthreads();
      const size_t slot = (size_t)(blockIdx.x + s) * a.G;
      for (int e = threadIdx.x; e < a.G; e += kThreads) {
        a.part_prob[slot + e] = s_prob[e];
        a.part_count[slot + e] = s_count[e];
      }
    }
    row = end;
  }
  for (size_t i = (size_t)row * a.k + threadIdx.x; i < (size_t)r1 * a.k; i += kThreads) {
    a.ids[i] = -1;
    a.weights[i] = 0.f;
  }
}

constexpr int kSumCols = 16, kSumStrips = kThreads / kSumCols;

// Sums the partials of 16 experts of one sequence and dots counts with probabilities; the
// last of a sequence's workgroups to finish adds the dots in order and writes the loss.
__global__ __launch_bounds__(kThreads) void route_balance(RouteArgs a, int32_t* counts,
                                                          int32_t* tokens, float* balance,
                                                          double* dots) {
  __shared__ double s_prob[kSumStrips][kSumCols];
  __shared__ int s_count[kSumStrips][kSumCols];
  __shared__ int s_tmp[kThreads / 64];
  const int s = blockIdx.y;
  int start = 0, end = a.T;
  if (a.seq_ends != nullptr) {
    int before = 0;
    for (int i = threadIdx.x; i < s; i += kThreads) before = max(before, a.seq_ends[i]);
    before = lanes_reduce<64>(before, [](int x, int y) { return max(x, y); });
    if ((threadIdx.x & 63) == 0) s_tmp[threadIdx.x >> 6] = before;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) start = max(start, s_tmp[w]);
    start = min(start, a.T);
    end = min(max(a.seq_ends[s], start), a.T);
  }
  const int col = threadIdx.x % kSumCols, strip = threadIdx.x / kSumCols;
  const int e = blockIdx.x * kSumCols + col;
  double prob = 0.0;
  int count = 0;
  if (end > start && e < a.G) {
    const int last = (end - 1) / a.rows_per_block;
    for (int c = start / a.rows_per_block + strip; c <= last; c += kSumStrips) {
      const size_t slot = (size_t)(c + s) * a.G + e;
      prob += (double)a.part_prob[slot];
      count += a.part_count[slot];
    }
  }
  s_prob[strip][col] = prob;
  s_count[strip][col] = count;
  __syncthreads();
  if (threadIdx.x < kSumCols) {
    for (int i = 1; i < kSumStrips; ++i) {
      prob += s_prob[i][col];
      count += s_count[i][col];
    }
    if (e < a.G) counts[(size_t)s * a.G + e] = count;
    const double dot = lanes_sum<kSumCols>((double)count * prob);
    if (threadIdx.x == 0) {
      double* at = dots + (size_t)s * gridDim.x;
      __hip_atomic_store(at + blockIdx.x, dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const int done = __hip_atomic_fetch_add(a.counters + s, 1, __ATOMIC_ACQ_REL,
                                              __HIP_MEMORY_SCOPE_AGENT);
      if (done == (int)gridDim.x - 1) {
        double sum = 0.0;
        for (unsigned i = 0; i < gridDim.x; ++i)
          sum += __hip_atomic_load(at + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int n = end - start;
        const double nn = (double)n * (double)n;
        balance[s] = n > 0 ? (float)(sum * ((double)a.G / (double)a.k) / nn) : 0.f;
        tokens[s] = n;
      }
    }
  }
}

struct RouteGradArgs {
  const void* logits;
  int64_t ld;
  int T, G, k, S;
  int renormalize;
  float scale;
  const int32_t* seq_ends;
  const int32_t* ids;
  const int32_t* counts;
  const int32_t* tokens;
  const float* d_weights;
  const float* d_balance;
  void* d_logits;
  int rows_per_block;
};

// d_l = p (b - sum p b) [(1 - q) for sigmoid], b_e = d_balance G c_e / (k n^2), plus on the
// chosen experts the gradient that reaches them through the weights: with pi = hat / Q the
// shares of the chosen (Q the sum of their hats),
//   renormalised: scale * pi * (dw - sum pi dw)    [(1 - q) for sigmoid]
//   otherwise:    scale * dw enters b (softmax), or scale * dw q (1 - q) (sigmoid).
template <class T, int L, int V, bool SIGMOID>
__global__ __launch_bounds__(kThreads) void route_grad(RouteGradArgs a) {
  __shared__ int s_found[kThreads / 64];
  constexpr int RP = kThreads / L;
  const int lane = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  const int r0 = blockIdx.x * a.rows_per_block;
  const int r1 = min(a.T, r0 + a.rows_per_block);
  T* out = reinterpret_cast<T*>(a.d_logits);
  int row = r0, s = -1;
  while (row < r1) {
    int end = r1;
    if (a.seq_ends == nullptr) {
      s = 0;
    } else {
      s = sequence_of(a.seq_ends, a.S, row, s + 1, s_found);
      if (s == a.S) break;
      end = min(a.seq_ends[s], r1);
    }
    float b0[V];
    float per_count = 0.f;
    if (a.d_balance != nullptr) {
      const float n = (float)a.tokens[s];
      per_count = n > 0.f ? a.d_balance[s] * ((float)a.G / (float)a.k) / n / n : 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane + L * v;
      b0[v] = a.d_balance != nullptr && e < a.G
                  ? per_count * (float)a.counts[(size_t)s * a.G + e] : 0.f;
    }
    for (int base = row; base < end; base += RP) {
      const int t = base + grp;
      const bool active = t < end;
      const size_t tr = (size_t)min(t, end - 1);
      float l[V], h[V], g[V];
      load_row<T, L>(reinterpret_cast<const T*>(a.logits) + tr * a.ld, a.G, lane, l);
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] = 0.f;
      uint64_t chosen = 0;  // bit v: slot v is among the row's choices
      if (a.d_weights != nullptr) {
        for (int r = 0; r < a.k; ++r) {
          const int id = a.ids[tr * a.k + r];
          const float dw = a.d_weights[tr * a.k + r];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const bool is = lane + L * v == id && id < a.G;
            g[v] = is ? dw : g[v];
            chosen |= is ? 1ull << v : 0;
          }
        }
      }
      const Scores<SIGMOID> sc(row_max<L>(l));
      float sum = 0.f, q_sum = 0.f, q_dw = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[v] = sc.hat(l[v]);
        sum += h[v];
        q_sum += chosen >> v & 1 ? h[v] : 0.f;
        q_dw += chosen >> v & 1 ? h[v] * g[v] : 0.f;
      }
      sum = lanes_sum<L>(sum);
      q_sum = lanes_sum<L>(q_sum);
      q_dw = lanes_sum<L>(q_dw);
      const float inv_sum = sum == 0.f ? 0.f : 1.f / sum;
      const float inv_q = q_sum == 0.f ? 0.f : 1.f / q_sum;
      // g becomes what each chosen expert's hat is multiplied with
      const float mean_dw = a.renormalize ? q_dw * inv_q : 0.f;
      const float to_g = a.scale * (a.renormalize ? inv_q : (SIGMOID ? sc.to_q : inv_sum));
      // softmax without renormalisation: the weights are p themselves and share its sum rule
      const bool shared = !SIGMOID && !a.renormalize;
      float mean_b = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        g[v] = chosen >> v & 1 ? to_g * (g[v] - mean_dw) : 0.f;
        mean_b += h[v] * (b0[v] * inv_sum + (shared ? g[v] : 0.f));
      }
      mean_b = lanes_sum<L>(mean_b);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + L * v;
        float d = h[v] * ((b0[v] - mean_b) * inv_sum + g[v]);
        if constexpr (SIGMOID) d *= Scores<SIGMOID>::one_minus_q(l[v]);
        if (active && e < a.G) out[tr * a.G + e] = from_f32<T>(d);
      }
    }
    row = end;
  }
  for (size_t i = (size_t)row * a.G + threadIdx.x; i < (size_t)r1 * a.G; i += kThreads)
    out[i] = from_f32<T>(0.f);
}

// Rows a workgroup takes: whole passes of kThreads / L rows, and no more workgroups than
// kRowBlocks, so that partials stay few next to the logits.
int rows_per_block(int T, int G) {
  const int pass = G <= 320 ? 16 : G <= 512 ? 8 : 4;
  const int per = cdiv(T > 0 ? T : 1, kRowBlocks);
  return cdiv(per, pass) * pass;
}
int row_blocks(int T, int G) { return T > 0 ? cdiv(T, rows_per_block(T, G)) : 1; }

// Calls f(L, V) as compile-time constants: the fewest slots that hold G. Up to 320 experts 16
// lanes share a row (four rows to a wave); beyond that a row takes more lanes, so that its
// logits still fit the registers.
template <class F>
void with_shape(int G, F f) {
  using std::integral_constant;
#define MGG_SHAPE(MAX, L, V) \
  if (G <= MAX) return f(integral_constant<int, L>{}, integral_constant<int, V>{})
  MGG_SHAPE(64, 16, 4);
  MGG_SHAPE(128, 16, 8);
  MGG_SHAPE(256, 16, 16);
  MGG_SHAPE(320, 16, 20);
  MGG_SHAPE(512, 32, 16);
  MGG_SHAPE(1024, 64, 16);
  MGG_SHAPE(2048, 64, 32);
  MGG_SHAPE(4096, 64, 64);
#undef MGG_SHAPE
}

struct Workspace {
  size_t prob, count, dots, counters, bytes;
  Workspace(int T, int G, int S) {
    const size_t slots = (size_t)row_blocks(T, G) + S;
    prob = 0;
    count = round_up(prob + slots * G * 4, 256);
    dots = round_up(count + slots * G * 4, 256);
    counters = round_up(dots + (size_t)S * cdiv(G, kSumCols) * 8, 256);
    bytes = round_up(counters + (size_t)S * 4, 256);
  }
};

const char* check_route(mgg_act dt, int T, int G, int k, const void* logits, int64_t ld,
                        mgg_score score, float scale, int S, const int32_t* ends) {
  if (!known(dt)) return "unknown element type";
  if (score != MGG_SCORE_SOFTMAX && score != MGG_SCORE_SIGMOID) return "unknown score function";
  if (T < 0) return "T must not be negative";
  if (G < 1 || G > kMaxExperts) return "G must be in [1, 4096]";
  if (k < 1 || k > G || k > kMaxTopk) return "k must be in [1, min(G, 32)]";
  if (T > 0 && !logits) return "null pointer";
  if (ld < G) return "the row stride must be at least G";
  if (!aligned(logits, elem_bytes(dt))) return "logits must be aligned to their element";
  if (!std::isfinite(scale)) return "scale must be finite";
  if (S < 1 || S > kMaxSequences) return "S must be in [1, 65535]";
  if (!ends && S != 1) return "several sequences need seq_ends";
  if (!aligned(ends, 4)) return "seq_ends must be 4-byte aligned";
  return nullptr;
}

}  // namespace

extern "C" {

size_t route_topk_workspace(int T, int G, int S) {
  if (T < 0 || G < 1 || G > kMaxExperts || S < 1 || S > kMaxSequences) return 0;
  return Workspace(T, G, S).bytes;
}

mgg_status route_topk(mgg_act dt, int T, int G, int k, const void* logits, int64_t ld,
                      const float* bias, mgg_score score, int renormalize, float scale, int S,
                      const int32_t* seq_ends, int32_t* ids, float* weights, int32_t* counts,
                      int32_t* tokens, float* balance, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  mgg_set_last_error("");
  if (const char* err = check_route(dt, T, G, k, logits, ld, score, scale, S, seq_ends))
    return fail(MGG_EINVAL, err);
  if (bias && score != MGG_SCORE_SIGMOID)
    return fail(MGG_EUNSUPPORTED, "a selection bias goes with sigmoid scores");
  if (T > 0 && (!ids || !weights)) return fail(MGG_EINVAL, "null pointer");
  if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(bias, 4))
    return fail(MGG_EINVAL, "ids, weights and bias must be 4-byte aligned");
  const bool stats = counts || tokens || balance;
  if (stats && (!counts || !tokens || !balance))
    return fail(MGG_EINVAL, "counts, tokens and balance are given together");
  if (!aligned(counts, 4) || !aligned(tokens, 4) || !aligned(balance, 4))
    return fail(MGG_EINVAL, "counts, tokens and balance must be 4-byte aligned");
  RouteArgs a{logits, ld,       bias, T,       G,          k,       S, renormalize,
              scale,  seq_ends, ids,  weights, rows_per_block(T, G), nullptr, nullptr, nullptr};
  double* dots = nullptr;
  if (stats) {
    const Workspace ws(T, G, S);
    if (!workspace || workspace_bytes < ws.bytes)
      return fail(MGG_EINVAL, "the workspace is smaller than route_topk_workspace says");
    if (!aligned(workspace, 256)) return fail(MGG_EINVAL, "the workspace must be 256-byte aligned");
    char* base = (char*)workspace;
    a.part_prob = (float*)(base + ws.prob);
    a.part_count = (int32_t*)(base + ws.count);
    a.counters = (int32_t*)(base + ws.counters);
    dots = (double*)(base + ws.dots);
  } else if (T == 0) {
    return MGG_OK;
  }
  const dim3 grid((unsigned)row_blocks(T, G));
  const size_t lds = stats ? (size_t)G * 8 : 0;
  const bool sigmoid = score == MGG_SCORE_SIGMOID;
  with_shape(G, [&](auto L, auto V) {
    auto go = [&](auto elem, auto sig, auto biased, auto with_stats) {
      route_rows<decltype(elem), L(), V(), sig(), biased(), with_stats()>
          <<<grid, kThreads, lds, stream>>>(a);
    };
    auto by_stats = [&](auto elem, auto sig, auto biased) {
      if (stats) go(elem, sig, biased, std::true_type{});
      else go(elem, sig, biased, std::false_type{});
    };
    auto by_score = [&](auto elem) {
      if (!sigmoid) by_stats(elem, std::false_type{}, std::false_type{});
      else if (!bias) by_stats(elem, std::true_type{}, std::false_type{});
      else by_stats(elem, std::true_type{}, std::true_type{});
    };
    if (dt == MGG_ACT_BF16) by_score(bf16_t{});
    else by_score(0.f);
  });
  if (stats)
    route_balance<<<dim3(cdiv(G, kSumCols), S), kThreads, 0, stream>>>(a, counts, tokens,
                                                                       balance, dots);
  return launched();
}

mgg_status route_topk_backward(mgg_act dt, int T, int G, int k, const void* logits, int64_t ld,
                               mgg_score score, int renormalize, float scale, int S,
                               const int32_t* seq_ends, const int32_t* ids,
                               const int32_t* counts, const int32_t* tokens,
                               const float* d_weights, const float* d_balance,
                               void* d_logits, hipStream_t stream) {
  mgg_set_last_error("");
  if (const char* err = check_route(dt, T, G, k, logits, ld, score, scale, S, seq_ends))
    return fail(MGG_EINVAL, err);
  if (!d_weights && !d_balance)
    return fail(MGG_EINVAL, "one of d_weights and d_balance must be given");
  if (T > 0 && (!d_logits || (d_weights && !ids))) return fail(MGG_EINVAL, "null pointer");
  if (d_balance && (!counts || !tokens))
    return fail(MGG_EINVAL, "d_balance needs counts and tokens");
  if (!aligned(d_logits, elem_bytes(dt)))
    return fail(MGG_EINVAL, "d_logits must be aligned to its element");
  if (!aligned(ids, 4) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(d_weights, 4) ||
      !aligned(d_balance, 4))
    return fail(MGG_EINVAL, "ids, counts, tokens and gradients must be 4-byte aligned");
  if (T == 0) return MGG_OK;
  const RouteGradArgs a{logits, ld,     T,      G,         k,         S,        renormalize,
                        scale,  seq_ends, ids,  counts,    tokens,    d_weights, d_balance,
                        d_logits, rows_per_block(T, G)};
  const dim3 grid((unsigned)row_blocks(T, G));
  with_shape(G, [&](auto L, auto V) {
    auto by_score = [&](auto elem) {
      if (score == MGG_SCORE_SIGMOID)
        route_grad<decltype(elem), L(), V(), true><<<grid, kThreads, 0, stream>>>(a);
      else
        route_grad<decltype(elem), L(), V(), false><<<grid, kThreads, 0, stream>>>(a);
    };
    if (dt == MGG_ACT_BF16) by_score(bf16_t{});
    else by_score(0.f);
  });
  return launched();
}

}  // extern "C"
