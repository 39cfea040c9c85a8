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
// atomics on sums are integer counters.
//
// The forward kernel is bound by its vector operations, about 500 for four rows of 288 experts (66 %
// of the busy time), and with few passes a workgroup by waiting for each pass's logits, which are not
// loaded ahead; the backward one by HBM with softmax, by its operations with sigmoid. Measured for
// 65536 rows of 288 logits, 8 chosen, 16 sequences, other inputs in each call: selection alone 19 us
// (float32 and bf16); with counts and losses 30 us and 7 us for the sums (both); backward 38 us,
// 4.1 TB/s (float32), with sigmoid scores 45 us (both).

#include "layer_common.h"

namespace {

using namespace mgg_layer;

constexpr int kThreads = 256;
constexpr int kMaxTopk = 32;
constexpr int kMaxExperts = 4096;
constexpr int kMaxSequences = 65535;  // grid.y of the summing kernel
// Most workgroups that rows are dealt to: four for each of the 256 CUs, or two in a forward kernel with
// counts whose registers leave room for fewer than four waves a SIMD. 65536 rows with two and with four:
// selection with counts of 128 by softmax 27 and 23 us, of 288 36 and 31; by sigmoid with bias of
// 128 42 and 33, of 288 (three waves) 53 and 56, 16384 rows 25 and 31. In the gradient's kernels with
// three waves neither is better throughout (288 by sigmoid: 16384 rows of float32 16 and 19 us,
// 131072 of bf16 73 and 67).
constexpr int kRowBlocks = 1024, kRowBlocksFew = 512;

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
    return (m < 0.f ? exp_neg(l - m) : (l < 0.f ? a : 1.f)) * reciprocal(1.f + a);
  }
  // of a whole row: the shifted exponentials only where the row has no logit above 0
  template <int V>
  __device__ __forceinline__ void hats(const float (&l)[V], float (&h)[V]) const {
    if constexpr (!SIGMOID) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = exp_neg(l[v] - m);
    } else if (m < 0.f) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        h[v] = exp_neg(l[v] - m) * reciprocal(1.f + exp_neg(-fabsf(l[v])));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float a = exp_neg(-fabsf(l[v]));
        h[v] = (l[v] < 0.f ? a : 1.f) * reciprocal(1.f + a);
      }
    }
  }
  // 1 - sigmoid(l)
  __device__ __forceinline__ static float one_minus_q(float l) {
    const float a = exp_neg(-fabsf(l));
    return (l >= 0.f ? a : 1.f) * reciprocal(1.f + a);
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

// How a row is laid over lanes: L lanes, V slots each, of which the first FULL hold an expert in
// every lane for all G that take this shape.
template <int L_, int V_, int FULL_>
struct ShapeOf {
  static constexpr int L = L_, V = V_, FULL = FULL_;
};

template <class SHAPE, class T>
__device__ __forceinline__ void load_row(const T* row, int G, int lane, float (&l)[SHAPE::V]) {
#pragma unroll
  for (int v = 0; v < SHAPE::V; ++v) {
    const int e = lane + SHAPE::L * v;
    l[v] = v < SHAPE::FULL || e < G ? to_f32(row[e]) : -INFINITY;
  }
}

template <int L, int V>
__device__ __forceinline__ float row_max(const float (&l)[V]) {
  float m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  return lanes_reduce<L>(m, [](float a, float b) { return fmaxf(a, b); });
}

// Candidates that a row's selection keeps, in LDS, two to a lane.
template <int L>
constexpr int kCandidates = 2 * L;

// The chosen of a row as a lane holds them: `id` at place `rank` (>= k: none), with its hat, or with
// its logit where a bias chose it.
template <int L>
struct Chosen {
  static constexpr int N = 2;  // places lane and lane + L; kMaxTopk <= 2 L
  int rank[N], id[N];
  float hat[N];
};

// Value of a lane's maximum as an integer of the same order.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((int)b < 0 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ ((int)u < 0 ? 0x80000000u : 0xffffffffu));
}

// Selection key of expert e: its logit, or q + bias in float64, where sums that float32 cannot
// tell apart still differ.
template <bool BIAS>
using KeyOf = std::conditional_t<BIAS, double, float>;
template <bool BIAS>
__device__ __forceinline__ KeyOf<BIAS> key_of(float l, const float* bias, int e) {
  if constexpr (BIAS) return 1.0 / (1.0 + exp(-(double)l)) + (double)bias[e];
  else return l;
}

// The k first experts by key, one after another: every round takes the largest key that is left
// (the lower index among equals; never NaN or -inf). For any row, at about 5 k V operations.
// With a bias it goes over the row in memory: its float64 keys would cost every row registers.
template <class T, int L, int V, bool BIAS, class Hat>
__device__ __forceinline__ Chosen<L> choose_by_rounds(const RouteArgs& a, const T* row, int lane,
                                                      const float (&l)[V], Hat hat_of) {
  using Key = KeyOf<BIAS>;
  uint64_t taken = 0;  // slots
  Chosen<L> c;
#pragma unroll
  for (int i = 0; i < c.N; ++i) c.rank[i] = lane + L * i, c.id[i] = -1, c.hat[i] = 0.f;
  for (int r = 0; r < a.k; ++r) {
    Key best = -INFINITY;
    int e = INT32_MAX;
    float logit = 0.f;
    auto see = [&](int v, float value) {
      const int at = lane + L * v;
      if (value > -INFINITY && !(taken >> v & 1)) {
        const Key key = key_of<BIAS>(value, a.bias, at);
        if (key > best) best = key, e = at, logit = value;
      }
    };
    if constexpr (BIAS) {
#pragma unroll 1
      for (int v = 0; lane + L * v < a.G; ++v) see(v, to_f32(row[lane + L * v]));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) see(v, l[v]);
    }
    const Key top = lanes_reduce<L>(best, [](Key x, Key y) { return x > y ? x : y; });
    const int first = lanes_reduce<L>(best == top ? e : INT32_MAX,
                                      [](int x, int y) { return min(x, y); });
    if (first == INT32_MAX) break;  // the same for all lanes of the row
    logit = __shfl(logit, first & (L - 1), L);
    if ((first & (L - 1)) == lane) taken |= 1ull << (first / L);
    const float hat = hat_of(logit);
#pragma unroll
    for (int i = 0; i < c.N; ++i)
      if (lane + L * i == r) c.id[i] = first, c.hat[i] = hat;
  }
  return c;
}

// A candidate's place in the order as one integer: by key, then by the lower index. Zeros of
// either sign are equal.
__device__ __forceinline__ uint64_t order_of(float key, int e) {
  return (uint64_t)ordered(key + 0.f) << 32 | (uint32_t)~e;
}

// The same by candidates. The k-th largest of the lanes' own maxima is a bound that at least k
// keys reach; the few that do (11 of 288 for k = 8) are gathered in LDS and ranked against each
// other, a sixth of the work of k rounds. With a bias the bound is taken on float32 sums and
// lowered by more than their error, and only candidates get a float64 key. Returns false where
// the candidates do not fit (equal logits, k next to or above the lanes): a matter of this row
// alone, so its result does not depend on its neighbours. Selection of 65536 x 288 takes 17, 19,
// 48, 94 and 161 us for k = 4, 8, 12, 16 and 32, with a bias (float64 keys in every round) 23, 31,
// 191, 668 and 1279 us.
template <class T, int L, int V, bool SIGMOID, bool BIAS, class Hat>
__device__ __forceinline__ bool choose_by_candidates(const RouteArgs& a, const T* row, int lane,
                                                     const float (&l)[V], const float (&hat)[V],
                                                     const float* bias, float to_q, Hat hat_of,
                                                     int* s_id, uint64_t* s_order,
                                                     Chosen<L>& c) {
  float rough[V];  // what the bound is taken on
  float most = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (BIAS) rough[v] = l[v] > -INFINITY ? fmaf(hat[v], to_q, bias[v]) : -INFINITY;
    else rough[v] = l[v];
    most = fmaxf(most, rough[v]);
  }
  // lanes apart by their number in the last bits: k rounds take k lanes
  uint32_t left = (ordered(most) & ~(uint32_t)(L - 1)) | (uint32_t)lane, bound = 0;
  for (int r = 0; r < a.k; ++r) {
    bound = lanes_reduce<L>(left, [](uint32_t x, uint32_t y) { return max(x, y); });
    left = left == bound ? 0u : left;
  }
  // ordered(-inf) is 0x007fffff: no k lanes have anything to take
  float least = bound <= 0x00800000u ? -INFINITY : from_ordered(bound & ~(uint32_t)(L - 1));
  if (BIAS && least < INFINITY) least -= 4e-6f * (1.f + fabsf(least));
  least = fmaxf(least, -3.402823466e38f);  // -inf itself is no candidate
  using Bits = std::conditional_t<(V > 32), uint64_t, uint32_t>;
  Bits slots = 0;
#pragma unroll
  for (int v = V - 1; v >= 0; --v) slots = slots + slots + (rough[v] >= least ? 1 : 0);
  const int mine = V > 32 ? __popcll(slots) : __popc((uint32_t)slots);
  const int upto = lanes_prefix<L>(mine);
  const int total = __shfl(upto, L - 1, L);
  if (total > kCandidates<L>) return false;
  for (int at = upto - mine; slots != 0; slots &= slots - 1, ++at)
    s_id[at] = lane + L * (V > 32 ? __ffsll((unsigned long long)slots) - 1
                                  : __ffs((uint32_t)slots) - 1);
  wave_order();
  uint64_t mine_at[c.N];
  auto take = [&](int i) {
    const int n = lane + L * i;
    c.rank[i] = n, c.id[i] = -1, c.hat[i] = 0.f;
    mine_at[i] = ~0ull;
    if (n < total) {
      const int e = s_id[n];
      const float logit = to_f32(row[e]);
      c.id[i] = e;
      c.hat[i] = hat_of(logit);
      if constexpr (BIAS) {
        // doubles order as integers once negative ones are turned round; equal ones are told
        // apart by the lanes that hold them, below
        const int64_t b = __builtin_bit_cast(int64_t, key_of<BIAS>(logit, a.bias, e) + 0.0);
        mine_at[i] = (uint64_t)(b ^ (b >> 63 & 0x7fffffffffffffffll)) ^ 0x8000000000000000ull;
      } else {
        mine_at[i] = order_of(logit, e);
      }
      s_order[n] = mine_at[i];
    }
  };
  auto rank = [&](int i) {
    if (c.id[i] < 0) return;
    int before = 0;
#pragma unroll 4
    for (int n = 0; n < total; ++n) {
      const uint64_t other = s_order[n];
      before += other > mine_at[i] ? 1 : 0;
      if constexpr (BIAS) before += other == mine_at[i] && s_id[n] < c.id[i] ? 1 : 0;
    }
    c.rank[i] = before;
  };
  take(0);
  take(1);
  wave_order();
  rank(0);
  if (total > L) rank(1);
  wave_order();  // the next row's candidates may come
  return true;
}

// One row: ids and weights written, its probabilities added to `acc` where `active`.
template <class T, class SHAPE, bool SIGMOID, bool BIAS, bool STATS>
__device__ __forceinline__ void route_row(const RouteArgs& a, const T* row, int t, bool active,
                                          int lane, const float (&l)[SHAPE::V],
                                          const float* bias, float (&acc)[SHAPE::V],
                                          int* s_count, int* s_id, uint64_t* s_order) {
  constexpr int L = SHAPE::L, V = SHAPE::V;
  const Scores<SIGMOID> sc(row_max<L>(l));
  float hat[V], sum = 0.f;
  sc.hats(l, hat);
#pragma unroll
  for (int v = 0; v < V; ++v) sum += hat[v];
  sum = lanes_sum<L>(sum);
  const float inv_sum = sum == 0.f ? 0.f : 1.f / sum;
  if constexpr (STATS) {
    if (active) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(hat[v], inv_sum, acc[v]);
    }
  }
  auto hat_of = [&](float logit) { return BIAS ? logit : sc.hat(logit); };
  Chosen<L> c;
  if (!choose_by_candidates<T, L, V, SIGMOID, BIAS>(a, row, lane, l, hat, bias, sc.to_q, hat_of,
                                                    s_id, s_order, c))
    c = choose_by_rounds<T, L, V, BIAS>(a, row, lane, l, hat_of);
  float to_q = sc.to_q;
  if constexpr (BIAS) {
    // a bias may choose experts so far below the row's best that nothing is left of their hats:
    // their shares come from their own best
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < c.N; ++i)
      if (c.rank[i] < a.k && c.id[i] >= 0) top = fmaxf(top, c.hat[i]);
    const Scores<SIGMOID> own(lanes_reduce<L>(top, [](float x, float y) { return fmaxf(x, y); }));
#pragma unroll
    for (int i = 0; i < c.N; ++i) c.hat[i] = c.id[i] < 0 ? 0.f : own.hat(c.hat[i]);
    to_q = own.to_q;
  }
  float chosen = 0.f;
#pragma unroll
  for (int i = 0; i < c.N; ++i) chosen += c.rank[i] < a.k ? c.hat[i] : 0.f;
  chosen = lanes_sum<L>(chosen);
  const float to_w =
      a.scale * (a.renormalize ? (chosen == 0.f ? 0.f : 1.f / chosen)
                               : (SIGMOID ? to_q : inv_sum));
#pragma unroll
  for (int i = 0; i < c.N; ++i)
    if (active && c.rank[i] < a.k) {
      a.ids[(size_t)t * a.k + c.rank[i]] = c.id[i];
      a.weights[(size_t)t * a.k + c.rank[i]] = c.id[i] < 0 ? 0.f : c.hat[i] * to_w;
      if (STATS && c.id[i] >= 0) atomicAdd(&s_count[c.id[i]], 1);
    }
}

template <class T, class SHAPE, bool SIGMOID, bool BIAS, bool STATS>
__global__ __launch_bounds__(kThreads) void route_rows(RouteArgs a) {
  extern __shared__ int s_dyn[];  // STATS: counts [G], sums [G]
  __shared__ int s_found[kThreads / 64];
  constexpr int L = SHAPE::L, V = SHAPE::V, RP = kThreads / L;  // RP rows at once
  __shared__ uint64_t s_order[RP][kCandidates<L>];
  __shared__ int s_id[RP][kCandidates<L>];
  int* s_count = STATS ? s_dyn : nullptr;
  float* s_prob = reinterpret_cast<float*>(s_dyn + a.G);
  const int lane = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  const int r0 = blockIdx.x * a.rows_per_block;
  const int r1 = min(a.T, r0 + a.rows_per_block);
  if constexpr (STATS)
    if (blockIdx.x == 0)
      for (int s = threadIdx.x; s < a.S; s += kThreads) a.counters[s] = 0;

  float bias[BIAS ? V : 1];  // -inf past the row, so that nothing is taken there
  if constexpr (BIAS) load_row<SHAPE>(a.bias, a.G, lane, bias);

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
    auto row_at = [&](int t) {
      return reinterpret_cast<const T*>(a.logits) + (size_t)min(t, end - 1) * a.ld;
    };
    for (int base = row; base < end; base += RP) {
      const int t = base + grp;
      float l[V];
      load_row<SHAPE>(row_at(t), a.G, lane, l);
      route_row<T, SHAPE, SIGMOID, BIAS, STATS>(a, row_at(t), t, t < end, lane, l, bias, acc,
                                                s_count, s_id[grp], s_order[grp]);
    }
    if constexpr (STATS) {
      // the sums of a wave's rows, then those of the waves one after another
      const auto add = [](float x, float y) { return x + y; };
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (L <= 16) acc[v] = with_partner<16>(acc[v], add);
        if constexpr (L <= 32) acc[v] = with_partner<32>(acc[v], add);
      }
      for (int w = 0; w < kThreads / 64; ++w) {
        __syncthreads();
        if ((int)threadIdx.x / 64 == w && (threadIdx.x & 63) < L) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int e = lane + L * v;
            if (e < a.G) s_prob[e] = w == 0 ? acc[v] : s_prob[e] + acc[v];
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
#pragma unroll 8
    for (int c = start / a.rows_per_block + strip; c <= last; c += kSumStrips) {
      const size_t slot = (size_t)(c + s) * a.G + e;
      prob += (double)a.part_prob[slot];
      count += a.part_count[slot];
    }
  }
  s_prob[strip][col] = prob;
  s_count[strip][col] = count;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  double dot = 0.0;
  if (threadIdx.x < kSumCols) {
    for (int i = 1; i < kSumStrips; ++i) {
      prob += s_prob[i][col];
      count += s_count[i][col];
    }
    if (e < a.G) counts[(size_t)s * a.G + e] = count;
    dot = (double)count * prob;
  }
  dot = lanes_sum<64>(dot);
  // The dot goes out by an exchange whose answer has to be back before the count goes up, and is
  // read by atomic loads: all of them act where the whole device sees them, and nothing else
  // passes between the workgroups. The order rests on the machine, not on a release: the asm takes
  // the exchange's answer, so the compiler waits for it there, and an exchange that has answered has
  // been done; the loads come after a branch on the count. (A release of the agent scope writes
  // back the die's whole L2 instead, 5 us here.)
  double* at = dots + (size_t)s * gridDim.x;
  int done = 0;
  if (threadIdx.x == 0) {
    const double before = __hip_atomic_exchange(at + blockIdx.x, dot, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::"v"(before) : "memory");
    done = __hip_atomic_fetch_add(a.counters + s, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (__builtin_amdgcn_readfirstlane(done) != (int)gridDim.x - 1) return;
  double sum = 0.0;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += 64)
    sum += __hip_atomic_load(at + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = lanes_sum<64>(sum);
  if (threadIdx.x == 0) {
    const int n = end - start;
    const double nn = (double)n * (double)n;
    balance[s] = n > 0 ? (float)(sum * ((double)a.G / (double)a.k) / nn) : 0.f;
    tokens[s] = n;
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

constexpr uint32_t kNone = 0xffffffffu;  // a NaN that no gradient is stored as

__device__ __forceinline__ uint32_t gradient_bits(float d) {
  return d != d ? 0x7fc00000u : __float_as_uint(d);
}

// d_l = p (b - sum p b) [(1 - q) for sigmoid], b_e = d_balance G c_e / (k n^2), plus on the
// chosen experts the gradient that reaches them through the weights: with pi = hat / Q the
// shares of the chosen (Q the sum of their hats),
//   renormalised: scale * pi * (dw - sum pi dw)    [(1 - q) for sigmoid]
//   otherwise:    scale * dw enters b (softmax), or scale * dw q (1 - q) (sigmoid).
// Waves for each SIMD that the compiler is held to: with sigmoid scores and 16 slots it would take 136
// registers and lose one of four.
constexpr int grad_waves(int V) { return V <= 8 ? 5 : V <= 16 ? 4 : V <= 20 ? 3 : 1; }

template <class T, class SHAPE, bool SIGMOID>
__global__ __launch_bounds__(kThreads, grad_waves(SHAPE::V)) void route_grad(RouteGradArgs a) {
  __shared__ int s_found[kThreads / 64];
  constexpr int L = SHAPE::L, V = SHAPE::V, RP = kThreads / L;
  // rows 16 words apart modulo the 64 banks
  __shared__ uint32_t s_dw[RP][L * V + (L < 64 ? 16 : 0)];
  const int lane = threadIdx.x & (L - 1), grp = threadIdx.x / L;
  if (a.d_weights != nullptr) {
#pragma unroll
    for (int v = 0; v < V; ++v) s_dw[grp][lane + L * v] = kNone;
    wave_order();
  }
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
    // a row's inputs: its logits, and the lane's share of its choices
    struct Row {
      float l[V];
      int id[2];
      float dw[2];
    };
    auto load = [&](int t) {
      Row r;
      const size_t tr = (size_t)min(t, end - 1);
      load_row<SHAPE>(reinterpret_cast<const T*>(a.logits) + tr * a.ld, a.G, lane, r.l);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = lane + L * i;
        const bool is = a.d_weights != nullptr && j < a.k;
        r.id[i] = is ? a.ids[tr * a.k + j] : -1;
        r.dw[i] = is ? a.d_weights[tr * a.k + j] : 0.f;
      }
      return r;
    };
    Row next = load(row + grp);
    for (int base = row; base < end; base += RP) {
      const int t = base + grp;
      const bool active = t < end;
      const size_t tr = (size_t)min(t, end - 1);
      const Row in = next;
      if (base + RP < end) next = load(t + RP);
      const float(&l)[V] = in.l;
      float h[V], g[V];
      uint64_t chosen = 0;  // bit v: slot v is among the row's choices
      if (a.d_weights != nullptr) {
        // the gradients go to their experts' lanes through LDS, which holds kNone elsewhere
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if ((unsigned)in.id[i] < (unsigned)a.G)
            s_dw[grp][in.id[i]] = gradient_bits(in.dw[i]);
        wave_order();
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint32_t bits = s_dw[grp][lane + L * v];
          g[v] = __uint_as_float(bits);
          chosen |= bits != kNone ? 1ull << v : 0;
        }
        wave_order();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if ((unsigned)in.id[i] < (unsigned)a.G) s_dw[grp][in.id[i]] = kNone;
        wave_order();
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = 0.f;
      }
      const Scores<SIGMOID> sc(row_max<L>(l));
      float sum = 0.f, q_sum = 0.f, q_dw = 0.f;
      sc.hats(l, h);
#pragma unroll
      for (int v = 0; v < V; ++v) {
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
        if (active && (v < SHAPE::FULL || e < a.G)) out[tr * a.G + e] = from_f32<T>(d);
      }
      // Chosen by a bias, far below the row's best: little or nothing may be left of their hats, and
      // their shares come from their own best. The same for all lanes of a row. The choices' lanes
      // write their experts' gradients again, after the slots' lanes of the same wave.
      if (SIGMOID && a.renormalize && a.d_weights != nullptr && q_sum < 0.0625f) {
        float own_l[2], own_h[2], top = -INFINITY, own_sum = 0.f, own_dw = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          own_l[i] = (unsigned)in.id[i] < (unsigned)a.G
                         ? to_f32(reinterpret_cast<const T*>(a.logits)[tr * a.ld + in.id[i]])
                         : -INFINITY;
          top = fmaxf(top, own_l[i]);
        }
        const Scores<SIGMOID> own(
            lanes_reduce<L>(top, [](float x, float y) { return fmaxf(x, y); }));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          own_h[i] = own.hat(own_l[i]);  // 0 where there is no choice
          own_sum += own_h[i];
          own_dw += own_h[i] * in.dw[i];
        }
        own_sum = lanes_sum<L>(own_sum);
        const float inv = own_sum == 0.f ? 0.f : 1.f / own_sum;
        own_dw = lanes_sum<L>(own_dw) * inv;
        wave_order();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!active || (unsigned)in.id[i] >= (unsigned)a.G) continue;
          const float b = a.d_balance != nullptr
                              ? per_count * (float)a.counts[(size_t)s * a.G + in.id[i]] : 0.f;
          const float d = sc.hat(own_l[i]) * ((b - mean_b) * inv_sum) +
                          a.scale * inv * own_h[i] * (in.dw[i] - own_dw);
          out[tr * a.G + in.id[i]] = from_f32<T>(d * Scores<SIGMOID>::one_minus_q(own_l[i]));
        }
        wave_order();
      }
    }
    row = end;
  }
  for (size_t i = (size_t)row * a.G + threadIdx.x; i < (size_t)r1 * a.G; i += kThreads)
    out[i] = from_f32<T>(0.f);
}

// Whether fewer than four waves a SIMD fit (128 registers each) a forward kernel: with counts it keeps
// two arrays of a row's V slots, and with a bias two more.
constexpr bool few_blocks(int V, bool biased, bool stats) { return stats && V > (biased ? 12 : 20); }

// Rows a workgroup takes: whole passes of kThreads / L rows, and no more workgroups than
// `most`, so that partials stay few next to the logits.
int rows_per_block(int T, int G, int most) {
  const int pass = G <= 320 ? 16 : G <= 512 ? 8 : 4;
  const int per = cdiv(T > 0 ? T : 1, most);
  return cdiv(per, pass) * pass;
}
int row_blocks(int T, int rows) { return T > 0 ? cdiv(T, rows) : 1; }

// Calls f with the shape that holds G in the fewest slots. Up to 320 experts 16 lanes share a row
// (four rows to a wave), with two slots more for every 32 experts; beyond that a row takes more
// lanes, so that its logits still fit the registers, and the slots double.
template <class F>
void with_shape(int G, F f) {
  if (G <= 32) return f(ShapeOf<16, 2, 0>{});
  if (G <= 64) return f(ShapeOf<16, 4, 2>{});
  if (G <= 96) return f(ShapeOf<16, 6, 4>{});
  if (G <= 128) return f(ShapeOf<16, 8, 6>{});
  if (G <= 160) return f(ShapeOf<16, 10, 8>{});
  if (G <= 192) return f(ShapeOf<16, 12, 10>{});
  if (G <= 224) return f(ShapeOf<16, 14, 12>{});
  if (G <= 256) return f(ShapeOf<16, 16, 14>{});
  if (G <= 288) return f(ShapeOf<16, 18, 16>{});
  if (G <= 320) return f(ShapeOf<16, 20, 18>{});
  if (G <= 512) return f(ShapeOf<32, 16, 10>{});
  if (G <= 1024) return f(ShapeOf<64, 16, 8>{});
  if (G <= 2048) return f(ShapeOf<64, 32, 16>{});
  f(ShapeOf<64, 64, 32>{});
}

struct Workspace {
  size_t prob, count, dots, counters, bytes;
  Workspace(int T, int G, int S) {
    const size_t slots = (size_t)row_blocks(T, rows_per_block(T, G, kRowBlocks)) + S;
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
  if (T < 0 || T > kMaxRows) return "T must be in [0, 2^30]";
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
  if (T < 0 || T > kMaxRows || G < 1 || G > kMaxExperts || S < 1 || S > kMaxSequences) return 0;
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
  RouteArgs a{logits, ld,       bias, T,       G, k,       S,       renormalize,
              scale,  seq_ends, ids,  weights, 0, nullptr, nullptr, nullptr};
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
  const size_t lds = stats ? (size_t)G * 8 : 0;
  const bool sigmoid = score == MGG_SCORE_SIGMOID;
  with_shape(G, [&](auto shape) {
    using SHAPE = decltype(shape);
    auto go = [&](auto elem, auto sig, auto biased, auto with_stats) {
      constexpr bool few = few_blocks(SHAPE::V, biased(), with_stats());
      a.rows_per_block = rows_per_block(T, G, few ? kRowBlocksFew : kRowBlocks);
      const dim3 grid((unsigned)row_blocks(T, a.rows_per_block));
      route_rows<decltype(elem), SHAPE, sig(), biased(), with_stats()>
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
  // without rows d_weights has no elements, and its address may be 0
  if (T > 0 && !d_weights && !d_balance)
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
  const int rows = rows_per_block(T, G, kRowBlocks);
  const RouteGradArgs a{logits,   ld,  T,      G,      k,         S,         renormalize, scale,
                        seq_ends, ids, counts, tokens, d_weights, d_balance, d_logits,    rows};
  const dim3 grid((unsigned)row_blocks(T, rows));
  with_shape(G, [&](auto shape) {
    using SHAPE = decltype(shape);
    auto by_score = [&](auto elem) {
      if (score == MGG_SCORE_SIGMOID)
        route_grad<decltype(elem), SHAPE, true><<<grid, kThreads, 0, stream>>>(a);
      else
        route_grad<decltype(elem), SHAPE, false><<<grid, kThreads, 0, stream>>>(a);
    };
    if (dt == MGG_ACT_BF16) by_score(bf16_t{});
    else by_score(0.f);
  });
  return launched();
}

}  // extern "C"
