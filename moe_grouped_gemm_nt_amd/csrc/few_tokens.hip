// few_tokens.hip - a whole MoE layer for the few tokens of a decoding step (C ABI in
// include/mgg/few_tokens.h: moe_few_tokens).
//
// A slot is an expert that some token names: slot s is expert s where there are as many places
// as experts, and else the expert of place s, if no earlier place names it (a place is one of a
// token's k choices). Which tokens name it, each workgroup finds by itself from the ids, so
// nothing is sorted beforehand.
//   few_up     h = silu(g) u of 8 columns for all of a slot's tokens: a workgroup holds 8 gate
//              rows and their 8 up rows, its waves share K;
//   few_down   16 columns of the output for all tokens: a workgroup goes through every slot, its
//              waves share the slots' K evenly, each with sums of its own for all tokens, which
//              are added in a fixed order at the end.
// Both are bound by reading the experts' weights once.

#include "mgg/few_tokens.h"
#include "row_stream.h"

namespace {

using namespace mgg_layer;

constexpr int kWaves = 8, kFewThreads = 64 * kWaves;
constexpr int kMaxTokens = 256, kMaxPlaces = 32, kMaxExperts = 4096, kMaxWidth = 1 << 17;
constexpr int kRowTiles = 4;   // token rows that a wave holds at once, in sixteens
constexpr int kUpColumns = 8, kDownColumns = 16;
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
  int32_t* slot_rows;    // [slots][T]: the place of each token that names the expert
  float* place_weight;   // [places]: what that token's output takes of the expert
  uint16_t *h, *h_low;   // [places][I]: silu(g) u as two bfloat16
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
  for (int c = 0; c < a.places; c += 64) {
    const int p = c + lane;
    const bool hit = p < a.places && a.ids[p] == expert;
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

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int RT>
__device__ __forceinline__ void up_rows(const FewArgs& a, int expert, int tile,
                                        const int32_t* list, int count, float* s_part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  const int i0 = tile * kUpColumns;
  StreamRows<RT> rows;
  const int n = (r < 8 ? 0 : a.I) + i0 + (r & 7);  // I is a multiple of 8
  rows.w = a.w13 + ((int64_t)expert * 2 * a.I + n) * row_bytes<W>(a.H) + q * Form<W>::RUN_BYTES;
  // FP8 scales multiply results, rows 4 q .. 4 q + 3 here; FP4 scales the lane's weights
  const int ns = W == kFp4Weights ? n : (q < 2 ? 0 : a.I) + i0 + 4 * (q & 1);
  set_scale<W, SF, SPAN>(a.s13, expert, 2 * a.I, a.H, ns, q, rows.scale, rows.scale_step);
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int at = 16 * t + r;
    rows.x[t] = at < count ? reinterpret_cast<const uint8_t*>(a.x + (list[at] / a.k) * a.ldx) +
                                 q * Form<W>::X_BYTES
                           : nullptr;
  }
  v4f acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  const int blocks = cdiv(a.H, Form<W>::BLOCK);
  stream_rows<W, SF, SPAN, RT, false>(rows, blocks * wave / kWaves, blocks * (wave + 1) / kWaves,
                                      a.H, acc);
#pragma unroll
  for (int t = 0; t < RT; ++t)
    *reinterpret_cast<v4f*>(s_part + ((wave * RT + t) * 16 + r) * kPartLd + 4 * q) = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < RT * 16 * kUpColumns; i += kFewThreads) {
    const int row = i / kUpColumns, c = i % kUpColumns;
    if (row >= count) break;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float* s = s_part + (w * RT * 16 + row) * kPartLd + c;
      g += s[0];
      u += s[8];
    }
    const float h = silu(g) * u;
    const uint16_t hi = bf16_bits(h);
    const float high = to_f32(bf16_t{hi});
    const int64_t at = (int64_t)list[row] * a.I + i0 + c;
    a.h[at] = hi;
    a.h_low[at] = fabsf(high) < INFINITY ? bf16_bits(h - high) : 0;
  }
}

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN>
__global__ __launch_bounds__(kFewThreads) void few_up(FewArgs a) {
  extern __shared__ __align__(16) float s_few[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = blockIdx.x, slot = blockIdx.y;
  int32_t* list = reinterpret_cast<int32_t*>(s_few) + wave * a.T;
  float* s_part = s_few + round_up(kWaves * a.T, 4);
  int expert;
  const int count = find_rows(a, slot, expert, list);
  if (tile == 0 && threadIdx.x == 0) a.slot_meta[slot] = make_int2(count, expert);
  if (count == 0) return;
  if (tile == 0) {
    for (int i = threadIdx.x; i < count; i += kFewThreads) {
      const int p = list[i], end = (p / a.k + 1) * a.k;
      float sum = 0.f;
      for (int j = p; j < end; ++j)
        if (a.ids[j] == expert) sum += a.weights[j];
      a.slot_rows[(int64_t)slot * a.T + i] = p;
      a.place_weight[p] = sum;
    }
  }
  for (int r0 = 0; r0 < count; r0 += 16 * kRowTiles) {
    const int left = count - r0;
    if (r0 > 0) __syncthreads();  // everyone has read the sums before
    if (left <= 16) up_rows<W, SF, SPAN, 1>(a, expert, tile, list + r0, left, s_part);
    else if (left <= 32) up_rows<W, SF, SPAN, 2>(a, expert, tile, list + r0, left, s_part);
    else up_rows<W, SF, SPAN, 4>(a, expert, tile, list + r0, left, s_part);
  }
}

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN, int RT>
__device__ __forceinline__ void down_rows(const FewArgs& a, int expert, int n0,
                                          const int32_t* list, int count, int from, int to,
                                          float* sums) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  StreamRows<RT> rows;
  const int n = min(n0 + r, a.H - 1);
  rows.w = a.w2 + ((int64_t)expert * a.H + n) * row_bytes<W>(a.I) + q * Form<W>::RUN_BYTES;
  const int ns = W == kFp4Weights ? n : min(n0 + 4 * q, a.H - 4);
  set_scale<W, SF, SPAN>(a.s2, expert, a.H, a.I, ns, q, rows.scale, rows.scale_step);
  int place[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    place[t] = 16 * t + r < count ? list[16 * t + r] : -1;
    const int64_t at = ((int64_t)place[t] * a.I) * 2 + q * Form<W>::X_BYTES;
    rows.x[t] = place[t] < 0 ? nullptr : reinterpret_cast<const uint8_t*>(a.h) + at;
    rows.x_low[t] = reinterpret_cast<const uint8_t*>(a.h_low) + at;
  }
  v4f acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
  stream_rows<W, SF, SPAN, RT, true>(rows, from, to, a.I, acc);
#pragma unroll
  for (int t = 0; t < RT; ++t)
    if (place[t] >= 0) {
      const float weight = a.place_weight[place[t]];
      v4f* s = reinterpret_cast<v4f*>(sums + (place[t] / a.k) * kDownColumns + 4 * q);
      v4f v = *s;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = fmaf(weight, acc[t][e], v[e]);
      *s = v;
    }
}

// A slot with tokens in one word.
__device__ __forceinline__ uint32_t pack_slot(int slot, int count, int expert) {
  return (uint32_t)slot | (uint32_t)(count - 1) << 12 | (uint32_t)expert << 20;
}

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN>
__global__ __launch_bounds__(kFewThreads) void few_down(FewArgs a) {
  extern __shared__ __align__(16) float s_few[];
  __shared__ int s_count[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * kDownColumns;
  float* sums = s_few + wave * a.T * kDownColumns;
  uint32_t* s_slots = reinterpret_cast<uint32_t*>(s_few + kWaves * a.T * kDownColumns);
  for (int i = lane; i < a.T * kDownColumns; i += 64) sums[i] = 0.f;
  // the slots that have tokens, in order
  int active = 0;
  for (int s0 = 0; s0 < a.slots; s0 += kFewThreads) {
    const int slot = s0 + threadIdx.x;
    const int2 meta = slot < a.slots ? a.slot_meta[slot] : make_int2(0, 0);
    const uint64_t mask = __ballot(meta.x > 0);
    if (lane == 0) s_count[wave] = __popcll(mask);
    __syncthreads();
    int at = active + __popcll(mask & ((1ull << lane) - 1));
    for (int w = 0; w < kWaves; ++w) {
      at += w < wave ? s_count[w] : 0;
      active += s_count[w];
    }
    if (meta.x > 0) s_slots[at] = pack_slot(slot, meta.x, meta.y);
    __syncthreads();
  }
  const int blocks = cdiv(a.I, Form<W>::BLOCK), units = active * blocks;
  int u = (int)((int64_t)units * wave / kWaves);
  const int end = (int)((int64_t)units * (wave + 1) / kWaves);
  while (u < end) {
    const int from = u % blocks, to = min(blocks, from + end - u);
    const uint32_t packed = s_slots[u / blocks];
    const int slot = packed & 4095, count = ((packed >> 12) & 255) + 1, expert = packed >> 20;
    const int32_t* list = a.slot_rows + (int64_t)slot * a.T;
    for (int r0 = 0; r0 < count; r0 += 16 * kRowTiles) {
      const int left = count - r0;
      if (left <= 16)
        down_rows<W, SF, SPAN, 1>(a, expert, n0, list + r0, left, from, to, sums);
      else if (left <= 32)
        down_rows<W, SF, SPAN, 2>(a, expert, n0, list + r0, left, from, to, sums);
      else
        down_rows<W, SF, SPAN, 4>(a, expert, n0, list + r0, left, from, to, sums);
    }
    u += to - from;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * kDownColumns; i += kFewThreads) {
    const int t = i / kDownColumns, n = n0 + i % kDownColumns;
    if (n >= a.H) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_few[w * a.T * kDownColumns + i];
    const int64_t at = (int64_t)t * a.H + n, res = t * a.ld_res + n;
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
  size_t meta, rows, weight, h, h_low, bytes;
  FewWorkspace(int T, int k, int G, int I) {
    const size_t places = (size_t)T * k, slots = std::min<size_t>(places, G);
    size_t at = 0;
    auto take = [&](size_t n) {
      const size_t here = at;
      at = round_up(at + n, 256);
      return here;
    };
    meta = take(slots * sizeof(int2));
    rows = take(slots * T * 4);
    weight = take(places * 4);
    h = take(places * I * 2);
    h_low = take(places * I * 2);
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

template <WeightForm W, ScaleForm SF, ScaleSpan SPAN>
bool run_few(const FewArgs& a, hipStream_t stream) {
  const int tiles = std::min(kRowTiles, cdiv(a.T, 16)) == 3 ? 4 : std::min(kRowTiles, cdiv(a.T, 16));
  const size_t up = (round_up(kWaves * a.T, 4) + (size_t)kWaves * tiles * 16 * kPartLd) * 4;
  const size_t down = ((size_t)kWaves * a.T * kDownColumns + a.slots) * 4;
  return launch_few(few_up<W, SF, SPAN>, dim3(cdiv(a.I, kUpColumns), a.slots), up, a, stream) &&
         launch_few(few_down<W, SF, SPAN>, dim3(cdiv(a.H, kDownColumns)), down, a, stream);
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
  if (T < 0 || T > kMaxTokens) return fail(MGG_EINVAL, "T must be in [0, 256]");
  if (k < 1 || k > kMaxPlaces) return fail(MGG_EINVAL, "k must be in [1, 32]");
  if (G < 1 || G > kMaxExperts) return fail(MGG_EINVAL, "G must be in [1, 4096]");
  const int unit = wt == MGG_WEIGHT_BF16 ? 8 : 128;
  if (H < 1 || H > kMaxWidth || H % unit || I < 1 || I > kMaxWidth || I % unit)
    return fail(MGG_EINVAL, "H and I must be in [1, 2^17] and multiples of 8 (BF16) or 128");
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
  a.slot_rows = reinterpret_cast<int32_t*>(base + ws.rows);
  a.place_weight = reinterpret_cast<float*>(base + ws.weight);
  a.h = reinterpret_cast<uint16_t*>(base + ws.h);
  a.h_low = reinterpret_cast<uint16_t*>(base + ws.h_low);
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
