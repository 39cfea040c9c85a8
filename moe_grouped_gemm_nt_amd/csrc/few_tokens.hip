// few_tokens.hip - a whole MoE layer for the few tokens of a decoding step (C ABI in
// include/mgg/few_tokens.h: moe_few_tokens).
//
// A slot is an expert that some token names: slot s is expert s where there are as many places
// as experts, and else the expert of place s, if no earlier place names it (a place is one of a
// token's k choices). Which tokens name it, each workgroup finds by itself from the ids, so
// nothing is sorted beforehand.
//   few_up     h = silu(g) u of some columns for all of a slot's tokens: a wave multiplies 8 gate
//              rows and their 8 up rows over a part of K, the slot's rows of x are in LDS;
//   few_down   16 columns of the output for all tokens: a workgroup goes through every slot, its
//              waves share the slots' K evenly, each with sums of its own for all tokens, which
//              are added in a fixed order at the end.
// Both are bound by reading the experts' weights once.

#include "mgg/few_tokens.h"
#include "row_stream.h"

namespace {

using namespace mgg_layer;

constexpr int kWaves = 8, kFewThreads = 64 * kWaves;
constexpr int kMaxTokens = 128, kMaxPlaces = 32, kMaxExperts = 4096, kMaxWidth = 1 << 16;
constexpr int kUpColumns = 8, kDownColumns = 16;
constexpr int kLdsBytes = 160 * 1024;
constexpr int kPartLd = 20;    // words from one token's 16 sums to the next: 16-byte aligned

struct FewArgs {
  int T, k, places, G, H, I, slots, by_expert;
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  const uint8_t *w13, *w2;
  const void *s13, *s2;
  int2* slot_meta;       // [slots]: tokens, expert
  int2* slot_rows;       // [slots][T]: for each token that names the expert its place (low 16 bits)
                         // and number, and what its output takes of the expert (float32 bits)
  uint16_t* h;           // [planes][places][I]: silu(g) u as one bfloat16, or as the sum of three
  int x_rows;            // few_up: rows of x in LDS at a time
  mgg_act out_dt;
  const void* residual;
  int64_t ld_res;
  void* out;
};

// The places that stand for the tokens of a slot, one a token, in ascending order, into `list`
// (LDS of the wave's own); returns their number, 0 for a slot that is none.
__device__ int find_rows(const FewArgs& a, int slot, int& expert, int32_t* list) {
  const int lane = threadIdx.x & 63;
  expert = a.by_expert ? slot : a.ids[slot];
  if (expert < 0 || expert >= a.G) return 0;
  int count = 0, last = -1;  // last: the token of the latest hit
  constexpr int AT_ONCE = 8;
  for (int c0 = 0; c0 < a.places; c0 += 64 * AT_ONCE) {
    int id[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int p = c0 + 64 * i + lane;
      id[i] = p < a.places ? a.ids[p] : -1;
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int c = c0 + 64 * i, p = c + lane;
      const bool hit = id[i] == expert;
      const uint64_t hits = __ballot(hit);
      if (hits == 0) continue;
      if (!a.by_expert && last < 0 && c + __builtin_ctzll(hits) != slot) return 0;
      // a token's places stand together: only its first one counts
      const uint64_t below = hits & ((1ull << lane) - 1);
      const int before = below ? (c + 63 - __builtin_clzll(below)) / a.k : last;
      const bool first = hit && p / a.k != before;
      const uint64_t firsts = __ballot(first);
      if (first) list[count + __popcll(firsts & ((1ull << lane) - 1))] = p;
      count += __popcll(firsts);
      last = (c + 63 - __builtin_clzll(hits)) / a.k;
    }
  }
  wave_order();
  return count;
}

// Rows of an expert's scales: where row n's stand at K = 0, and the step to the next 128 K.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN>
__device__ __forceinline__ void set_scale(const void* s, int expert, int N, int K, int n, int q,
                                          const void*& at, int64_t& step) {
  at = nullptr;
  step = 0;
  if constexpr (W == kFp4Weights) {
    at = reinterpret_cast<const uint8_t*>(s) + ((int64_t)expert * (K / 128) * N + n) * 4 + q;
    step = (int64_t)N * 4;
  } else if constexpr (W == kFp8Weights) {
    const int64_t i = SPAN == kPerChannel
                          ? (int64_t)expert * (K / 128) * N + n
                          : ((int64_t)expert * cdiv(N, 128) + n / 128) * (K / 128);
    at = reinterpret_cast<const uint8_t*>(s) + i * (SF == kF32Scales ? 4 : 1);
    step = SPAN == kPerChannel ? N : 1;
  }
}

template <WeightForm W>
__device__ __forceinline__ int64_t row_bytes(int K) {
  return W == kBf16Weights ? (int64_t)K * 2 : W == kFp8Weights ? K : K / 2;
}

__device__ __forceinline__ float silu(float g) {
  float q, rest;
  sigmoid_parts(g, q, rest);
  return g * q;
}

// A token row in LDS: whole blocks of K, and 16 bytes more so that rows start in different banks.
template <WeightForm W>
__host__ __device__ constexpr int x_row_bytes(int H) {
  return cdiv(H, Form<W>::BLOCK) * Form<W>::BLOCK * 2 + 16;
}

// [g; u] = W13[e] x, h = silu(g) u. Bound by the weights' way from HBM: what matters is that enough
// of them are under way, so each lane loads what it multiplies itself, AHEAD blocks early, straight
// into registers, and x, which every wave needs, is in LDS: its registers would halve the blocks
// (2 KB of weights a wave in FP8 against 4 KB of x). TILES: 8-column tiles of a workgroup, which
// shares K among kWaves / TILES waves for each. More tiles mean fewer copies of x into LDS and longer
// streams, fewer workgroups.
// Measured: 64 tokens, 8 of 288 experts of 4096 x 256 in FP8: 505 MB in 105 us, 4.8 TB/s (a large copy
// reaches 4.7); one token, 17 MB in 8.3 us: the ids, then the weights, each a trip to HBM.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int TILES>
__global__ __launch_bounds__(kFewThreads, 4) void few_up(FewArgs a) {
  using F = Form<W>;
  constexpr int PARTS = kWaves / TILES;
  // blocks of weights on their way, within the 128 registers that leave 16 waves to a CU
  constexpr int AHEAD = WeightBlock<W, SF, SPAN>::SCALES > 1 ? 3 : 4;
  extern __shared__ __align__(16) float s_few[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int slot = blockIdx.y, tile = blockIdx.x * TILES + wave % TILES, part = wave / TILES;
  const int x_ld = x_row_bytes<W>(a.H);
  uint8_t* s_x = reinterpret_cast<uint8_t*>(s_few);
  float* s_part = reinterpret_cast<float*>(s_x + a.x_rows * x_ld);
  int32_t* list = reinterpret_cast<int32_t*>(s_part + kWaves * 16 * kPartLd) + wave * a.T;
  int expert;
  const int count = find_rows(a, slot, expert, list);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.slot_meta[slot] = make_int2(count, expert);
  if (count == 0) return;

  const int i0 = tile * kUpColumns;
  const bool live = i0 < a.I;  // a wave behind the last column has nothing to multiply
  const int n = live ? (r < 8 ? 0 : a.I) + i0 + (r & 7) : 0;  // I is a multiple of 8
  const uint8_t* w = a.w13 + ((int64_t)expert * 2 * a.I + n) * row_bytes<W>(a.H) + q * F::RUN_BYTES;
  // FP8 scales multiply results, rows 4 q .. 4 q + 3 here; FP4 scales the lane's weights
  const int ns = W == kFp4Weights ? n : live ? (q < 2 ? 0 : a.I) + i0 + 4 * (q & 1) : 0;
  const void* scale;
  int64_t scale_step;
  set_scale<W, SF, SPAN>(a.s13, expert, 2 * a.I, a.H, ns, q, scale, scale_step);
  const int blocks = cdiv(a.H, F::BLOCK);
  const int from = blocks * part / PARTS, to = live ? blocks * (part + 1) / PARTS : from;

  for (int r0 = 0; r0 < count; r0 += a.x_rows) {
    const int rows = min(a.x_rows, count - r0);
    WeightBlock<W, SF, SPAN> ring[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (from + i < to) load_weights<W, SF, SPAN, true>(ring[i], w, scale, scale_step, from + i, a.H);
    if (r0 > 0) __syncthreads();  // everyone is done with the rows and sums before
    const int pieces = (x_ld - 16) / 16;
    for (int row = 0; row < rows; row += 4) {
      const uint16_t* from_x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        from_x[i] = a.x + (int64_t)(list[r0 + min(row + i, rows - 1)] / a.k) * a.ldx;
      for (int c = threadIdx.x; c < pieces; c += kFewThreads) {
        const int left = (a.H - 8 * c) * 2;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = left >= 16 ? load16(from_x[i] + 8 * c) : load16_part<2>(from_x[i] + 8 * c, left);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row + i < rows) *reinterpret_cast<uint4*>(s_x + (row + i) * x_ld + c * 16) = v[i];
      }
    }
    __syncthreads();
    v4f acc[1] = {v4f{0.f, 0.f, 0.f, 0.f}};
    // lanes without a row repeat the first one; nobody reads their results
    const uint8_t* xr = s_x + (r < rows ? r : 0) * x_ld + q * F::X_BYTES;
    for (int b = from; b < to; b += AHEAD)
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (b + i < to) {
          const uint8_t* xb = xr + (b + i) * (4 * F::X_BYTES);
          auto x = [&](int, int, int j) { return *reinterpret_cast<const uint4*>(xb + 16 * j); };
          multiply_block<W, SF, SPAN, 1, 1>(ring[i], acc, x);
          if (b + i + AHEAD < to)
            load_weights<W, SF, SPAN, true>(ring[i], w, scale, scale_step, b + i + AHEAD, a.H);
        }
    *reinterpret_cast<v4f*>(s_part + (wave * 16 + r) * kPartLd + 4 * q) = acc[0];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * TILES * kUpColumns; i += kFewThreads) {
      const int row = i / (TILES * kUpColumns), t = i / kUpColumns % TILES, c = i % kUpColumns;
      const int col = (blockIdx.x * TILES + t) * kUpColumns + c;
      if (col >= a.I) continue;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        const float* s = s_part + ((p * TILES + t) * 16 + row) * kPartLd + c;
        g += s[0];
        u += s[8];
      }
      // Bfloat16 outputs: as between the grouped products, h is rounded to their type. Float32
      // outputs: three bfloat16 are the 24 bits of h (an infinite one stays alone).
      float h = silu(g) * u;
      uint16_t* to = a.h + (int64_t)list[r0 + row] * a.I + col;
      const int64_t plane = (int64_t)a.places * a.I;
      for (int p = 0; p < (a.out_dt == MGG_ACT_F32 ? 3 : 1); ++p) {
        const uint16_t bits = bf16_bits(h);
        to[p * plane] = bits;
        const float held = to_f32(bf16_t{bits});
        h = fabsf(held) < INFINITY ? h - held : 0.f;
      }
    }
  }
  if (blockIdx.x == 0)  // what few_down needs to know of the slot
    for (int i = threadIdx.x; i < count; i += kFewThreads) {
      const int p = list[i], t = p / a.k;
      float sum = 0.f;
      for (int j = p; j < (t + 1) * a.k; ++j)
        if (a.ids[j] == expert) sum += a.weights[j];
      a.slot_rows[(int64_t)slot * a.T + i] = make_int2(p | t << 16, __float_as_int(sum));
    }
}

// A job of few_down is up to 16 tokens of a slot, in one word: the first of its rows in the list of
// all slots' rows, their number less 1, and the expert.
__device__ __forceinline__ uint32_t pack_job(int row, int count, int expert) {
  return (uint32_t)row | (uint32_t)(count - 1) << 16 | (uint32_t)expert << 20;
}
constexpr int kMaxJobs(int slots, int places) { return slots + places / 16; }

// out = residual + the weighted sums of W2[e] h over each token's experts. A workgroup owns 16 columns
// of all tokens, so that the sum over a token's experts stays in it: partial sums of experts in
// different workgroups would go through memory (four times the tokens' output in float32) and a third
// kernel. Its waves take equal runs of the units (16 tokens of an expert, a block of K), whatever
// expert they are of, as one stream with AHEAD units under way; where a job ends, its sums go into
// the wave's own [T][16] in LDS. Bound by the weights as above.
// Measured: the 64 tokens above, 252 MB in 57 us, 4.4 TB/s; one token, 8.4 MB in 5.4 us: the slots'
// rows, then weights and h.
template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int PLANES>
__global__ __launch_bounds__(kFewThreads, PLANES > 1 ? 2 : 4) void few_down(FewArgs a) {
  using F = Form<W>;
  constexpr int AHEAD = W == kBf16Weights ? 4 : PLANES > 1 ? 2 : 3;
  extern __shared__ __align__(16) float s_few[];
  __shared__ int2 s_total[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * kDownColumns;
  float* sums = s_few + wave * a.T * kDownColumns;
  int2* s_rows = reinterpret_cast<int2*>(s_few + kWaves * a.T * kDownColumns);
  uint32_t* s_jobs = reinterpret_cast<uint32_t*>(s_rows + a.places);
  for (int i = lane; i < a.T * kDownColumns; i += 64) sums[i] = 0.f;
  // the slots' rows one behind the other, and their jobs, in the order of the slots
  int rows = 0, jobs = 0;
  for (int s0 = 0; s0 < a.slots; s0 += kFewThreads) {
    const int slot = s0 + threadIdx.x;
    const int2 meta = slot < a.slots ? a.slot_meta[slot] : make_int2(0, 0);
    const int mine = cdiv(meta.x, 16);
    int before_r = lanes_prefix<64>(meta.x), before_j = lanes_prefix<64>(mine);
    if (lane == 63) s_total[wave] = make_int2(before_r, before_j);
    __syncthreads();
    before_r += rows - meta.x;
    before_j += jobs - mine;
    for (int w = 0; w < kWaves; ++w) {
      before_r += w < wave ? s_total[w].x : 0;
      before_j += w < wave ? s_total[w].y : 0;
      rows += s_total[w].x;
      jobs += s_total[w].y;
    }
    const int2* from = a.slot_rows + (int64_t)slot * a.T;
#pragma unroll 4
    for (int i = 0; i < meta.x; ++i) s_rows[before_r + i] = from[i];
    for (int j = 0; j < mine; ++j)
      s_jobs[before_j + j] = pack_job(before_r + 16 * j, min(16, meta.x - 16 * j), meta.y);
    __syncthreads();
  }

  const int blocks = cdiv(a.I, F::BLOCK);
  const int units = jobs * blocks;
  const int first = (int)((int64_t)units * wave / kWaves);
  const int end = (int)((int64_t)units * (wave + 1) / kWaves);
  const int n = min(n0 + r, a.H - 1), ns = W == kFp4Weights ? n : min(n0 + 4 * q, a.H - 4);
  WeightBlock<W, SF, SPAN> weights[AHEAD];
  TokenBlock<W, 1, PLANES> tokens[AHEAD];
  // the unit to load next: block `lb` of job `lj`
  int lj = first / blocks, lb = first % blocks;
  auto load = [&](int i) {
    const uint32_t job = s_jobs[lj];
    const int row = job & 0xffff, count = (job >> 16 & 15) + 1, expert = job >> 20;
    const uint8_t* w = a.w2 + ((int64_t)expert * a.H + n) * row_bytes<W>(a.I) + q * F::RUN_BYTES;
    const void* scale;
    int64_t step;
    set_scale<W, SF, SPAN>(a.s2, expert, a.H, a.I, ns, q, scale, step);
    load_weights<W, SF, SPAN, true>(weights[i], w, scale, step, lb, a.I);
    const int place = r < count ? s_rows[row + r].x & 0xffff : -1;
    const int64_t at = (int64_t)place * a.I * 2 + q * F::X_BYTES;
#pragma unroll
    for (int p = 0; p < PLANES; ++p)
      load_tokens<W, true>(tokens[i].x[p][0],
                           place < 0 ? nullptr
                                     : reinterpret_cast<const uint8_t*>(a.h) + at +
                                           p * ((int64_t)a.places * a.I * 2),
                           lb, a.I);
    if (++lb == blocks) lb = 0, ++lj;
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (first + i < end) load(i);
  v4f acc[1] = {v4f{0.f, 0.f, 0.f, 0.f}};
  int job_at = first / blocks, block_at = first % blocks;
  for (int u = first; u < end; u += AHEAD)
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (u + i < end) {
        auto x = [&](int p, int, int j) { return tokens[i].x[p][0][j]; };
        multiply_block<W, SF, SPAN, 1, PLANES>(weights[i], acc, x);
        if (u + i + AHEAD < end) load(i);
        if (++block_at == blocks || u + i + 1 == end) {
          // a wave's tokens of one job are different ones
          const uint32_t job = s_jobs[job_at];
          if (r < (int)(job >> 16 & 15) + 1) {
            const int2 row = s_rows[(job & 0xffff) + r];
            const float weight = __int_as_float(row.y);
            v4f* s = reinterpret_cast<v4f*>(sums + (row.x >> 16) * kDownColumns + 4 * q);
            v4f v = *s;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(weight, acc[0][e], v[e]);
            *s = v;
          }
          wave_order();
          acc[0] = v4f{0.f, 0.f, 0.f, 0.f};
          block_at = 0;
          ++job_at;
        }
      }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * kDownColumns; i += kFewThreads) {
    const int t = i / kDownColumns, col = n0 + i % kDownColumns;
    if (col >= a.H) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_few[w * a.T * kDownColumns + i];
    const int64_t at = (int64_t)t * a.H + col, res = t * a.ld_res + col;
    if (a.out_dt == MGG_ACT_BF16) {
      if (a.residual) v += to_f32(reinterpret_cast<const bf16_t*>(a.residual)[res]);
      reinterpret_cast<bf16_t*>(a.out)[at] = from_f32<bf16_t>(v);
    } else {
      if (a.residual) v += reinterpret_cast<const float*>(a.residual)[res];
      reinterpret_cast<float*>(a.out)[at] = v;
    }
  }
}

// Where the workspace's parts start.
struct FewWorkspace {
  size_t meta, rows, h, bytes;
  FewWorkspace(int T, int k, int G, int I) {
    const size_t places = (size_t)T * k, slots = std::min<size_t>(places, G);
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t here = at;
      at = round_up(at + n, 256);
      return here;
    };
    meta = take(slots * sizeof(int2));
    rows = take(slots * T * sizeof(int2));
    h = take(3 * places * I * 2);
    bytes = at;
  }
};

bool sizes_ok(int T, int k, int G, int I) {
  return T >= 0 && T <= kMaxTokens && k >= 1 && k <= kMaxPlaces && G >= 1 && G <= kMaxExperts &&
         I >= 1 && I <= kMaxWidth;
}

template <class F>
bool launch_few(F kernel, dim3 grid, size_t lds, const FewArgs& a, hipStream_t stream) {
  if (lds > 64 * 1024 &&
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                          (int)lds) != hipSuccess)
    return false;
  kernel<<<grid, kFewThreads, lds, stream>>>(a);
  return true;
}

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int TILES>
bool run_up(const FewArgs& a, hipStream_t stream) {
  const size_t lds = (size_t)a.x_rows * x_row_bytes<W>(a.H) +
                     ((size_t)kWaves * 16 * kPartLd + (size_t)kWaves * a.T) * 4;
  return launch_few(few_up<W, SF, SPAN, TILES>,
                    dim3(cdiv(cdiv(a.I, kUpColumns), TILES), a.slots), lds, a, stream);
}

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN>
bool run_few(FewArgs a, hipStream_t stream) {
  // Rows of x in LDS: what an expert can be expected to have twice over, in two workgroups to a
  // CU where that leaves four rows, else in one.
  const int mean = cdiv(a.places, a.G);
  const int want = a.T <= 4 ? a.T : mean <= 2 ? 4 : mean <= 4 ? 8 : 16;
  const int rest = (int)((size_t)kWaves * 16 * kPartLd + (size_t)kWaves * a.T) * 4;
  const int row = x_row_bytes<W>(a.H);
  const int half = (kLdsBytes / 2 - rest) / row, all = (kLdsBytes - rest) / row;
  a.x_rows = std::min(std::min(want, 16), half >= 4 || half >= want ? std::max(half, 1) : all);
  if (want > 8 && all >= 16) a.x_rows = 16;
  // Tiles of a workgroup: as many as leave a workgroup for each CU, and a block of K for each wave
  // (32 tokens over six FP4 experts of 256 tiles: 58, 50.5 and 49 us with one, two and four).
  const int64_t tiles = (int64_t)cdiv(a.I, kUpColumns) * std::min(a.slots, a.places);
  const int blocks = cdiv(a.H, Form<W>::BLOCK);
  const bool up = tiles >= 4 * 300 || blocks < 4 ? run_up<W, SF, SPAN, 4>(a, stream)
                  : tiles >= 2 * 300 || blocks < 8 ? run_up<W, SF, SPAN, 2>(a, stream)
                                                   : run_up<W, SF, SPAN, 1>(a, stream);
  const size_t lds = (size_t)kWaves * a.T * kDownColumns * 4 + a.places * sizeof(int2) +
                     kMaxJobs(a.slots, a.places) * 4;
  const dim3 grid(cdiv(a.H, kDownColumns));
  return up && (a.out_dt == MGG_ACT_F32 ? launch_few(few_down<W, SF, SPAN, 3>, grid, lds, a, stream)
                                        : launch_few(few_down<W, SF, SPAN, 1>, grid, lds, a, stream));
}

}  // namespace

extern "C" {

size_t moe_few_tokens_workspace(int T, int k, int G, int I) {
  return sizes_ok(T, k, G, I) ? FewWorkspace(T, k, G, I).bytes : 0;
}

mgg_status moe_few_tokens(mgg_weight wt, int T, int k, int G, int H, int I, const void* x,
                          int64_t ldx, const int32_t* ids, const float* weights,
                          const void* W13, const void* S13, const void* W2, const void* S2,
                          mgg_sf_fmt sf, mgg_sfb_gran gran, mgg_act out_dt,
                          const void* residual, int64_t ld_res, void* out, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  mgg_set_last_error("");
  if (wt != MGG_WEIGHT_BF16 && wt != MGG_WEIGHT_FP8 && wt != MGG_WEIGHT_FP4)
    return fail(MGG_EINVAL, "unknown weight type");
  if (!known(out_dt)) return fail(MGG_EINVAL, "unknown element type");
  if (T < 0 || T > kMaxTokens) return fail(MGG_EINVAL, "T must be in [0, 128]");
  if (k < 1 || k > kMaxPlaces) return fail(MGG_EINVAL, "k must be in [1, 32]");
  if (G < 1 || G > kMaxExperts) return fail(MGG_EINVAL, "G must be in [1, 4096]");
  const int unit = wt == MGG_WEIGHT_BF16 ? 8 : 128;
  if (H < 1 || H > kMaxWidth || H % unit || I < 1 || I > kMaxWidth || I % unit)
    return fail(MGG_EINVAL, "H and I must be in [1, 2^16] and multiples of 8 (BF16) or 128");
  const bool scaled = wt != MGG_WEIGHT_BF16;
  if (scaled) {
    if (sf != MGG_SF_F32 && sf != MGG_SF_UE8M0) return fail(MGG_EINVAL, "unknown scale format");
    if (wt == MGG_WEIGHT_FP4 && (sf != MGG_SF_UE8M0 || gran != MGG_SFB_BLOCK32))
      return fail(MGG_EUNSUPPORTED, "FP4 weights take UE8M0 scales per 32 elements");
    if (wt == MGG_WEIGHT_FP8 && gran != MGG_SFB_BLOCK128 && gran != MGG_SFB_CHANNEL)
      return fail(MGG_EUNSUPPORTED, "FP8 weights take scales per 128 x 128 block or per channel");
  }
  if ((S13 != nullptr) != scaled || (S2 != nullptr) != scaled)
    return fail(MGG_EINVAL, "scales go with FP8 and FP4 weights, and only with them");
  if (!W13 || !W2) return fail(MGG_EINVAL, "null pointer");
  if (!aligned(W13, 16) || !aligned(W2, 16))
    return fail(MGG_EINVAL, "weights must be 16-byte aligned");
  if (scaled && sf == MGG_SF_F32 && (!aligned(S13, 4) || !aligned(S2, 4)))
    return fail(MGG_EINVAL, "float32 scales must be 4-byte aligned");
  if (T == 0) return MGG_OK;
  if (!x || !ids || !weights || !out) return fail(MGG_EINVAL, "null pointer");
  if (ldx < H || (residual && ld_res < H))
    return fail(MGG_EINVAL, "a row stride is smaller than the row");
  if (!aligned(x, 2) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(residual, elem_bytes(out_dt)) || !aligned(out, elem_bytes(out_dt)))
    return fail(MGG_EINVAL, "tensors must be aligned to their element");
  const FewWorkspace ws(T, k, G, I);
  if (!workspace || workspace_bytes < ws.bytes)
    return fail(MGG_EINVAL, "the workspace is smaller than moe_few_tokens_workspace says");
  if (!aligned(workspace, 256)) return fail(MGG_EINVAL, "the workspace must be 256-byte aligned");

  char* base = reinterpret_cast<char*>(workspace);
  FewArgs a{};
  a.T = T, a.k = k, a.places = T * k, a.G = G, a.H = H, a.I = I;
  a.by_expert = a.places >= G;
  a.slots = a.by_expert ? G : a.places;
  a.x = reinterpret_cast<const uint16_t*>(x), a.ldx = ldx;
  a.ids = ids, a.weights = weights;
  a.w13 = reinterpret_cast<const uint8_t*>(W13), a.w2 = reinterpret_cast<const uint8_t*>(W2);
  a.s13 = S13, a.s2 = S2;
  a.slot_meta = reinterpret_cast<int2*>(base + ws.meta);
  a.slot_rows = reinterpret_cast<int2*>(base + ws.rows);
  a.h = reinterpret_cast<uint16_t*>(base + ws.h);
  a.out_dt = out_dt, a.residual = residual, a.ld_res = ld_res, a.out = out;

  bool ok;
  if (wt == MGG_WEIGHT_BF16) ok = run_few<kBf16Weights, kNoScales, kPerBlock>(a, stream);
  else if (wt == MGG_WEIGHT_FP4) ok = run_few<kFp4Weights, kByteScales, kPerChannel>(a, stream);
  else if (gran == MGG_SFB_BLOCK128)
    ok = sf == MGG_SF_F32 ? run_few<kFp8Weights, kF32Scales, kPerBlock>(a, stream)
                          : run_few<kFp8Weights, kByteScales, kPerBlock>(a, stream);
  else
    ok = sf == MGG_SF_F32 ? run_few<kFp8Weights, kF32Scales, kPerChannel>(a, stream)
                          : run_few<kFp8Weights, kByteScales, kPerChannel>(a, stream);
  if (!ok) return fail(MGG_EHIP, "hipFuncSetAttribute failed");
  return launched();
}

}  // extern "C"
