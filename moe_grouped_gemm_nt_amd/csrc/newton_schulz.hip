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
// The power of two keeps them below fp16's largest and a matrix as a whole, relative to its
// norm, clear of the 2^-24 at which fp16 ends below: |X| <= 4 and |A| <= 16 take 2^12, |P| <= 64
// takes 2^10. Where a matrix is small (its norm next to eps, or coefficients that shrink it) X is
// held 2^x times larger, A = X X^T by itself 2^2x times, and P 2^p times: x and p of each matrix
// and step come from bounds that hold before the steps run (Growth), and are 0 where the bounds
// are 1/2 or more.

#include "layer_common.h"

namespace {

using namespace mgg_layer;

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kSlice = 16;   // K elements of a slice (32 bytes of a row): one MFMA's
constexpr int kMaxSide = 32768, kMaxMatrices = 4096, kMaxSteps = 32;
constexpr int kNormBlocks = 256;  // most partial sums of squares per matrix
constexpr float kScaleX = 4096.f, kScaleA = 4096.f, kScaleP = 1024.f;

// A matrix [rows][K] as its two fp16 halves, `group` elements from one matrix to the next. Each
// half is stored slice by slice, [K / 16][rows][16]: a tile's slice is one contiguous run, which
// spreads over all memory channels whatever K is (rows a power of two apart would meet in one
// of them), and 32 x 32 results are stored as runs of 1 KB. The two 16-byte pieces of a row
// change places every eight rows, the order in which LDS holds them: the 16 lanes that a
// 16-byte LDS read serves at once (0-3, 12-15, 20-23, 24-27 and the other four fours) then
// meet 64 different banks.
struct Split {
  _Float16 *hi, *lo;
  int rows;
  size_t group;
  __device__ __forceinline__ size_t at(size_t g, int row, int k) const {
    return g * group + ((size_t)(k / kSlice) * rows + row) * kSlice +
           ((k / 8 & 1) ^ (row >> 3 & 1)) * 8 + k % 8;
  }
};

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// Copies 1 KB, 16 bytes a lane (lane_bytes = 16 * lane), from memory to LDS; both addresses are
// the wave's. The bytes are there after a wait for the copy and a barrier.
__device__ __forceinline__ void copy_to_lds(const void* from, void* lds, uint32_t lane_bytes) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(at), "v"(lane_bytes), "s"(from) : "memory");
}
// Waits until at most N of the wave's copies are under way.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

struct NsArgs {
  const void* in;
  void* out;
  int in_bf16, out_bf16;
  int M, N;        // as the caller's
  int tall;        // M > N: rows of X are the caller's columns
  float eps, scale;
  double* norms;   // [G][kNormBlocks], the first norm_blocks of each
  int norm_blocks;
  int2* bits;      // [G][kMaxSteps + 1]: x and p of each step's X and P (above)
};

// What the steps do to singular values: `a`, `b`, `c` the sizes of the coefficients, `most` the
// largest |P| and `top` the largest singular value that a step makes of those in its range.
struct Growth {
  int steps;
  float a[kMaxSteps], b[kMaxSteps], c[kMaxSteps], most[kMaxSteps], top[kMaxSteps];
};

// The powers of two that a matrix of this norm at most is held larger by (NaN: none). Below
// 2^-kMostBits nothing is left of a float32 result; P's factor stays a float.
constexpr int kMostBits = 300, kMostBitsP = 110;
__device__ __forceinline__ int spare_bits(double bound, int most) {
  if (!(bound > 0.0)) return 0;
  int exponent;
  (void)frexp(bound, &exponent);
  return min(max(-exponent, 0), most);
}

// Eight elements of the caller's matrix from `p`, which is aligned to an element only; `n` of them
// exist.
__device__ __forceinline__ void load_eight(const void* in, int bf16, size_t at, long n,
                                           float (&v)[8]) {
  if (bf16) {
    const bf16_t* p = reinterpret_cast<const bf16_t*>(in) + at;
    uint16_t bits[8];
    if (n >= 8) {
      __builtin_memcpy(bits, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) bits[i] = i < n ? p[i].bits : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(bf16_t{bits[i]});
  } else {
    const float* p = reinterpret_cast<const float*>(in) + at;
    if (n >= 8) {
      __builtin_memcpy(v, p, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    }
  }
}

// Sums of squares in float64: a float32 overflows above 1e19.
__global__ __launch_bounds__(kThreads) void ns_norm(NsArgs a) {
  __shared__ double s_sum[kThreads / 64];
  const size_t size = (size_t)a.M * a.N, base = size * blockIdx.y;
  double sum = 0.0;
  constexpr int AT_ONCE = 2;
  const size_t step = (size_t)gridDim.x * kThreads * 8;
  for (size_t i0 = ((size_t)blockIdx.x * kThreads + threadIdx.x) * 8; i0 < size;
       i0 += AT_ONCE * step) {
    float v[AT_ONCE][8];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const size_t i = i0 + u * step;
      load_eight(a.in, a.in_bf16, base + (i < size ? i : 0), i < size ? (long)(size - i) : 0, v[u]);
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += (double)v[u][e] * (double)v[u][e];
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

// Eight values as eight hi and eight lo.
__device__ __forceinline__ void store_eight(const Split& to, size_t at, const float (&v)[8]) {
  v8h hi, lo;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    _Float16 h, l;
    split(v[i], h, l);
    hi[i] = h;
    lo[i] = l;
  }
  *reinterpret_cast<v8h*>(to.hi + at) = hi;
  *reinterpret_cast<v8h*>(to.lo + at) = lo;
}

// Scales a matrix to norm 1 and writes X and X^T in halves, padded with zeros: 64 x 64 values a
// workgroup, eight of a row (then of a column, by way of LDS) a thread. One more row of workgroups
// (blockIdx.y) writes `bits`.
__global__ __launch_bounds__(kThreads) void ns_split(NsArgs a, Growth growth, Split x, Split xt) {
  // rows 65 words apart: the columns' readers meet different banks
  __shared__ float s_tile[kSplitTile][kSplitTile + 1];
  // every wave adds the partial sums in the same order
  double sum = 0.0;
  for (int i = threadIdx.x & 63; i < a.norm_blocks; i += 64)
    sum += a.norms[(size_t)blockIdx.z * kNormBlocks + i];
  sum = lanes_sum<64>(sum);
  const double norm = sqrt(sum), to_one = norm + (double)a.eps;
  const double inv = ldexp((double)kScaleX, spare_bits(norm / to_one, kMostBits)) / to_one;
  if (blockIdx.y == gridDim.y - 1) {
    // a workgroup of its own: the steps' bounds depend on each other
    if (blockIdx.x != 0 || threadIdx.x != 0) return;
    double bound = norm / to_one;  // of X's singular values before step s
    for (int s = 0; s < growth.steps; ++s) {
      const double t = bound * bound;
      const double p = fmin((double)growth.most[s],
                            growth.a[s] + t * (growth.b[s] + t * growth.c[s]));
      a.bits[(size_t)blockIdx.z * (kMaxSteps + 1) + s] =
          make_int2(spare_bits(bound, kMostBits), spare_bits(p, kMostBitsP));
      bound = fmin((double)growth.top[s], bound * p);
    }
    a.bits[(size_t)blockIdx.z * (kMaxSteps + 1) + growth.steps] = make_int2(0, 0);
    return;
  }
  // the caller's rows run along tile rows here; `direct` has them as rows
  const Split direct = a.tall ? xt : x, turned = a.tall ? x : xt;
  const int r0 = blockIdx.y * kSplitTile, c0 = blockIdx.x * kSplitTile;
  const size_t base = (size_t)a.M * a.N * blockIdx.z;
#pragma unroll
  for (int q = 0; q < kSplitTile * kSplitTile / (8 * kThreads); ++q) {
    const int at = q * kThreads + threadIdx.x, r = at / (kSplitTile / 8), c = at % (kSplitTile / 8) * 8;
    const int i = r0 + r, j = c0 + c;
    const bool in = i < a.M && j < a.N;
    float v[8];
    load_eight(a.in, a.in_bf16, in ? base + (size_t)i * a.N + j : 0, in ? a.N - j : 0, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = (float)((double)v[e] * inv);
      s_tile[r][c + e] = v[e];
    }
    store_eight(direct, direct.at(blockIdx.z, i, j), v);
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSplitTile * kSplitTile / (8 * kThreads); ++q) {
    const int at = q * kThreads + threadIdx.x, c = at % kSplitTile, r = at / kSplitTile * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s_tile[r + e][c];
    store_eight(turned, turned.at(blockIdx.z, c0 + c, r0 + r), v);
  }
}

enum Product { kGram, kPoly, kApply, kLast };

struct ProductArgs {
  Split left, right;  // both [rows][K]: C = left right^T
  int K;
  int tiles_i, tiles_j;  // of one matrix
  int whole;             // tiles of all matrices that are not cut into quarters
  // kGram: the parts that a tile's sum is cut into, of part_k elements of K (the last one may be
  // shorter), and where their sums go; one part: straight on to the result
  int part_k, parts;
  float* sums;
  float to_value;     // accumulator -> value: the operands' powers of two taken back
  Split c, ct;        // the result and its transpose (symmetric results: the same matrix)
  // kPoly: P = ca I + cb A + cc A A
  Split a;
  float ca, cb, cc;
  int step;
  NsArgs ns;
};

// A T x T output tile by WI x WJ waves of (32 RI) x (32 RJ), S slices in LDS.
template <int T_, int WI_, int WJ_, int S_>
struct TileOf {
  static constexpr int T = T_, WI = WI_, WJ = WJ_, S = S_, THREADS = 64 * WI * WJ;
  static constexpr int RI = T / (32 * WI), RJ = T / (32 * WJ);
  static constexpr int WAVES = WI * WJ;
  static constexpr int HALF = T * kSlice * 2;   // bytes of one operand half in a slice
  static constexpr int STAGE = 4 * HALF;        // left hi, left lo, right hi, right lo
  static constexpr int COPIES = STAGE / (WAVES * 1024);  // 1 KB copies a wave makes a slice
  // the epilogue's 32 x 32 words, one row apart by 36: rows and columns both spread over
  // the banks, rows stay 16-byte aligned
  static constexpr int TURN_LD = 36, TURN = 32 * TURN_LD * 4;
  static constexpr int LDS = S * STAGE > WAVES * TURN ? S * STAGE : WAVES * TURN;
  static_assert(HALF % 1024 == 0, "a copy stays in one operand half");
  static_assert(S == 4 || S == 8, "the last steps are written out for these");
};

// Which tile a workgroup takes. Workgroups go to the eight dies in turn, so each die gets a run
// of consecutive tiles, whose operand rows its L2 then shares.
__device__ __forceinline__ int tile_of_block(int b, int tiles) {
  const int per = tiles / 8, whole = per * 8;
  return b < whole ? (b & 7) * per + (b >> 3) : b;
}

// The two halves of a value in one word, hi in the lower.
__device__ __forceinline__ uint32_t pack_halves(float v) {
  _Float16 hi, lo;
  split(v, hi, lo);
  return (uint32_t)__builtin_bit_cast(uint16_t, hi) |
         (uint32_t)__builtin_bit_cast(uint16_t, lo) << 16;
}

// Stores the wave's 32 x 32 words at (row, col) of a split matrix.
__device__ __forceinline__ void store_split(const uint32_t* words, int ld_words, const Split& to,
                                            size_t g, int row, int col, int lane) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = half * 16 + (lane >> 2), c = (lane & 3) * 8;
    const uint4 a = *reinterpret_cast<const uint4*>(words + r * ld_words + c);
    const uint4 b = *reinterpret_cast<const uint4*>(words + r * ld_words + c + 4);
    uint4 hi, lo;
    hi.x = __builtin_amdgcn_perm(a.y, a.x, 0x05040100);
    hi.y = __builtin_amdgcn_perm(a.w, a.z, 0x05040100);
    hi.z = __builtin_amdgcn_perm(b.y, b.x, 0x05040100);
    hi.w = __builtin_amdgcn_perm(b.w, b.z, 0x05040100);
    lo.x = __builtin_amdgcn_perm(a.y, a.x, 0x07060302);
    lo.y = __builtin_amdgcn_perm(a.w, a.z, 0x07060302);
    lo.z = __builtin_amdgcn_perm(b.y, b.x, 0x07060302);
    lo.w = __builtin_amdgcn_perm(b.w, b.z, 0x07060302);
    const size_t at = to.at(g, row + r, col + c);
    *reinterpret_cast<uint4*>(to.hi + at) = hi;
    *reinterpret_cast<uint4*>(to.lo + at) = lo;
  }
}

// Stores the wave's 32 x 32 floats at (row, col) of the caller's [rows][cols] output.
__device__ __forceinline__ void store_out(const uint32_t* words, int ld_words, const NsArgs& n,
                                          size_t g, int row, int col, int lane) {
  const size_t base = (size_t)n.M * n.N * g;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = i * 2 + (lane >> 5), c = lane & 31;
    if (row + r < n.M && col + c < n.N) {
      const float v = __uint_as_float(words[r * ld_words + c]);
      const size_t at = base + (size_t)(row + r) * n.N + col + c;
      if (n.out_bf16) reinterpret_cast<bf16_t*>(n.out)[at] = from_f32<bf16_t>(v);
      else reinterpret_cast<float*>(n.out)[at] = v;
    }
  }
}

// C = left right^T for one T x T tile in 32 x 32 x 16 MFMAs, three to a slice of 16 K (hi hi,
// hi lo, lo hi). The right operand's rows are the instruction's first operand, so a lane ends
// up with runs of four consecutive columns of one row of C. Slices go straight from memory to
// a ring of LDS stages; each is read into registers one slice before it is multiplied. Results
// turn in LDS, so that both C and its transpose are written in 16-byte pieces of their rows.
//
// Measured on four 2048 x 2048 matrices: X' takes 175 us, 1180 TFLOP/s of fp16 products (a
// library product of 8192 x 8192 fp16 matrices reaches 1110 there), with the matrix pipe busy
// 67 % of the cycles at the 1.7 GHz that the power limit leaves; A and P take 105-115 us.
template <Product WHAT, class TILE>
__device__ __forceinline__ void tile_sum(const ProductArgs& p, uint8_t* s_lds, size_t g, int i0,
                                         int j0, int k0, int k_len,
                                         v16f (&acc)[TILE::RI][TILE::RJ]) {
  constexpr int RI = TILE::RI, RJ = TILE::RJ;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / TILE::WJ * 32 * RI, wj = wave % TILE::WJ * 32 * RJ;

  // copy q of the wave: 1 KB of an operand half's rows, a slice further each time
  const uint32_t lane_bytes = lane * 16;
  const uint8_t* from[TILE::COPIES];
  uint32_t further[TILE::COPIES];
#pragma unroll
  for (int q = 0; q < TILE::COPIES; ++q) {
    const int at = (q * TILE::WAVES + wave) * 1024, h = at / TILE::HALF;
    const Split& op = h < 2 ? p.left : p.right;
    const _Float16* half = (h & 1) ? op.lo : op.hi;
    from[q] = reinterpret_cast<const uint8_t*>(half + g * op.group +
                                               (size_t)k0 * op.rows +
                                               (size_t)(h < 2 ? i0 : j0) * kSlice) +
              at % TILE::HALF;
    further[q] = op.rows * kSlice * 2;
  }
  auto copy = [&](int q, int stage) {
    copy_to_lds(from[q], s_lds + stage * TILE::STAGE + (q * TILE::WAVES + wave) * 1024,
                lane_bytes);
    from[q] += further[q];
  };

#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < RJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // a slice of both operands' halves in registers: `left`, `right` hold [half][32 rows]
  struct Step {
    v8h left[2][RI], right[2][RJ];
  };
  const int at_l = (wi + (lane & 31)) * 32 + ((lane >> 5) ^ (lane >> 3 & 1)) * 16;
  const int at_r = 2 * TILE::HALF + (wj + (lane & 31)) * 32 +
                   ((lane >> 5) ^ (lane >> 3 & 1)) * 16;
  auto read = [&](Step& f, int n, int stage) {  // the n-th of 2 (RI + RJ) reads
    const uint8_t* base = s_lds + stage * TILE::STAGE;
    if (n < 2 * RJ)
      f.right[n / RJ][n % RJ] = *reinterpret_cast<const v8h*>(
          base + at_r + n / RJ * TILE::HALF + n % RJ * 1024);
    else
      f.left[(n - 2 * RJ) / RI][(n - 2 * RJ) % RI] = *reinterpret_cast<const v8h*>(
          base + at_l + (n - 2 * RJ) / RI * TILE::HALF + (n - 2 * RJ) % RI * 1024);
  };
  // One slice: its products, with the reads of the next one (in stage `then`) and the copies of
  // the one S - 1 further (into stage `into`) spread among them - a wave that issues copies in
  // a row waits for the copy path, and the matrix pipe with it.
  auto step = [&](const Step& f, Step& next, int then, int into, bool reads, bool copies) {
    constexpr int READS = 2 * (RI + RJ);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
#pragma unroll
      for (int j = 0; j < RJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.right[0][j], f.left[0][i], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int n = 0; n < READS; ++n)
        if (reads && n * RI / READS == i) read(next, n, then);
#pragma unroll
      for (int j = 0; j < RJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.right[1][j], f.left[0][i], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int q = 0; q < TILE::COPIES; ++q)
        if (copies && q * RI / TILE::COPIES == i) copy(q, into);
#pragma unroll
      for (int j = 0; j < RJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.right[0][j], f.left[1][i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // At the end of step s the copies of slice s + 2 have landed and everyone has read slice
  // s + 1, so step s + 1 may read the one and step s + 2 copy over the other. While copies go
  // on, those of the S - 3 slices behind s + 2 may still be under way.
  constexpr int S = TILE::S, AHEAD = S - 1;
  const int slices = k_len / kSlice;  // a multiple of four
  Step even, odd;
  for (int s = 0; s < AHEAD && s < slices; ++s)
#pragma unroll
    for (int q = 0; q < TILE::COPIES; ++q) copy(q, s);
  if (slices >= AHEAD) wait_copies<(AHEAD - 2) * TILE::COPIES>();
  else wait_copies<0>();
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 2 * (RI + RJ); ++n) read(even, n, 0);
  // N steps from stage 0 on, of which the last LEFT have no slice left to copy.
  auto steps = [&](auto count, auto left) {
    constexpr int N = count(), LEFT = left();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const bool copies = n < N - LEFT, reads = LEFT == 0 || n + 1 < N;
      if (n % 2 == 0) step(even, odd, (n + 1) % S, (n + S - 1) % S, reads, copies);
      else step(odd, even, (n + 1) % S, (n + S - 1) % S, reads, copies);
      if (copies) wait_copies<(AHEAD - 2) * TILE::COPIES>();
      else wait_copies<0>();
      __syncthreads();
    }
  };
  using std::integral_constant;
  int todo = slices;
  for (; todo > 2 * S - 2; todo -= S)
    steps(integral_constant<int, S>{}, integral_constant<int, 0>{});
  // with S = 4 four slices are left, with S = 8 four, eight or twelve
  if (S == 4 || todo == 4) {
    steps(integral_constant<int, 4>{}, integral_constant<int, AHEAD < 4 ? AHEAD : 4>{});
  } else if (todo == 8) {
    steps(integral_constant<int, 8>{}, integral_constant<int, AHEAD>{});
  } else {
    steps(integral_constant<int, 12>{}, integral_constant<int, AHEAD>{});
  }
}

// The powers of two that X and P are held larger by, and that of the next step's X.
struct Bits {
  int x, p, x_next;
};
template <Product WHAT>
__device__ __forceinline__ Bits bits_of(const ProductArgs& p, size_t g) {
  if constexpr (WHAT == kGram) return Bits{0, 0, 0};  // A's power follows from X's
  const int2* at = p.ns.bits + g * (kMaxSteps + 1) + p.step;
  return Bits{at[0].x, at[0].y, at[1].x};
}

// Writes a tile's sums, in the caller's or the next product's form.
template <Product WHAT, class TILE>
__device__ __forceinline__ void tile_write(const ProductArgs& p, uint8_t* s_lds, size_t g, int i0,
                                           int j0, v16f (&acc)[TILE::RI][TILE::RJ]) {
  constexpr bool SYM = WHAT == kGram || WHAT == kPoly;
  constexpr int RI = TILE::RI, RJ = TILE::RJ;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = wave / TILE::WJ * 32 * RI, wj = wave % TILE::WJ * 32 * RJ;
  // LDS, whose stages everyone has read, is the waves' turning space

  // lane: row 32 i + (lane & 31) of the wave's part; registers 4 q .. 4 q + 3: columns
  // 32 j + 8 q + 4 (lane >> 5) ..
  uint32_t* turn = reinterpret_cast<uint32_t*>(s_lds + wave * TILE::TURN);
  constexpr int LD = TILE::TURN_LD;
  const bool mirror = !SYM || i0 != j0;
  const Bits bits = bits_of<WHAT>(p, g);
  const float a_true = ldexpf(1.f, -2 * bits.x);  // 0 where A is too small to show
  const float cb = p.cb * a_true, cc = p.cc * a_true * a_true;
  const float held = WHAT == kGram    ? kScaleA
                     : WHAT == kPoly  ? ldexpf(kScaleP, bits.p)
                     : WHAT == kApply ? ldexpf(kScaleX, bits.x_next - bits.x - bits.p)
                                      : 0.f;
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
      const int row0 = i0 + wi + 32 * i, col0 = j0 + wj + 32 * j;
      uint32_t w[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e] * p.to_value;
        if constexpr (WHAT == kPoly) {
          const int row = row0 + (lane & 31), col = col0 + 8 * q + 4 * (lane >> 5);
          const size_t at = p.a.at(g, row, col);
          const v4h hi = *reinterpret_cast<const v4h*>(p.a.hi + at);
          const v4h lo = *reinterpret_cast<const v4h*>(p.a.lo + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float av = ((float)hi[e] + (float)lo[e]) * (1.f / kScaleA);
            v[e] = fmaf(cc, v[e], cb * av) + (row == col + e ? p.ca : 0.f);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (WHAT == kLast)
            w[4 * q + e] = __float_as_uint(
                bits.x + bits.p == 0
                    ? v[e] * p.ns.scale
                    : (float)ldexp((double)v[e] * (double)p.ns.scale, -bits.x - bits.p));
          else
            w[4 * q + e] = pack_halves(v[e] * held);
        }
      }
      // each lane group reads back what other lanes of its own wave wrote
      const bool direct = WHAT != kLast || !p.ns.tall;
      if (direct) {
        wave_order();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(turn + (lane & 31) * LD + 8 * q + 4 * (lane >> 5)) =
              make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        wave_order();
        if constexpr (WHAT == kLast) store_out(turn, LD, p.ns, g, row0, col0, lane);
        else store_split(turn, LD, p.c, g, row0, col0, lane);
      }
      if (WHAT == kLast ? p.ns.tall : mirror) {
        wave_order();
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            turn[(8 * q + 4 * (lane >> 5) + e) * LD + (lane & 31)] = w[4 * q + e];
        wave_order();
        if constexpr (WHAT == kLast) store_out(turn, LD, p.ns, g, col0, row0, lane);
        else store_split(turn, LD, p.ct, g, col0, row0, lane);
      }
    }
}

template <Product WHAT, class TILE>
__device__ __forceinline__ void tile_product(const ProductArgs& p, uint8_t* s_lds, size_t g,
                                             int i0, int j0) {
  v16f acc[TILE::RI][TILE::RJ];
  tile_sum<WHAT, TILE>(p, s_lds, g, i0, j0, 0, p.K, acc);
  tile_write<WHAT, TILE>(p, s_lds, g, i0, j0, acc);
}

// The b-th pair ti <= tj of a triangle, its rows one after another.
__device__ __forceinline__ void triangle_tile(int b, int tiles, int& ti, int& tj) {
  ti = 0;
  for (int len = tiles; b >= len; --len) {
    b -= len;
    ++ti;
  }
  tj = ti + b;
}

// A = X X^T of few tiles and a long K: each tile's sum is cut along K into `parts`, whose
// workgroups leave their accumulators in memory (a lane's next to its neighbours'), and
// ns_gram_join adds them in order: else few CUs work through many slices, 60 ns each. All five
// steps, whole sums and parts: 64 x 4099 150 and 108 us, two matrices of 256 x 4096 217 and 162,
// three of 230 x 1878 155 and 139 (now 2 us more each, for the powers of two).
template <class TILE>
__global__ __launch_bounds__(TILE::THREADS) void ns_gram_part(ProductArgs p) {
  extern __shared__ __align__(16) uint8_t s_lds[];
  const int part = blockIdx.x % p.parts, tile = blockIdx.x / p.parts;
  const int per_matrix = p.tiles_i * (p.tiles_i + 1) / 2;
  int ti, tj;
  triangle_tile(tile % per_matrix, p.tiles_i, ti, tj);
  v16f acc[TILE::RI][TILE::RJ];
  const int k0 = part * p.part_k;
  tile_sum<kGram, TILE>(p, s_lds, tile / per_matrix, ti * TILE::T, tj * TILE::T, k0,
                        min(p.part_k, p.K - k0), acc);
  float* to = p.sums + (size_t)blockIdx.x * TILE::T * TILE::T + threadIdx.x;
#pragma unroll
  for (int i = 0; i < TILE::RI * TILE::RJ; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      to[(i * 16 + r) * TILE::THREADS] = acc[i / TILE::RJ][i % TILE::RJ][r];
}

template <class TILE>
__global__ __launch_bounds__(TILE::THREADS) void ns_gram_join(ProductArgs p) {
  constexpr int N = TILE::RI * TILE::RJ;
  extern __shared__ __align__(16) uint8_t s_lds[];
  const int tile = blockIdx.x, per_matrix = p.tiles_i * (p.tiles_i + 1) / 2;
  int ti, tj;
  triangle_tile(tile % per_matrix, p.tiles_i, ti, tj);
  v16f acc[TILE::RI][TILE::RJ];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i / TILE::RJ][i % TILE::RJ][r] = 0.f;
#pragma unroll 4  // four parts' loads under way at once
  for (int part = 0; part < p.parts; ++part) {
    const float* from =
        p.sums + ((size_t)tile * p.parts + part) * TILE::T * TILE::T + threadIdx.x;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        acc[i / TILE::RJ][i % TILE::RJ][r] += from[(i * 16 + r) * TILE::THREADS];
  }
  tile_write<kGram, TILE>(p, s_lds, tile / per_matrix, ti * TILE::T, tj * TILE::T, acc);
}

// All tiles of a product: `whole` of them in the tile's own size, the rest, which would be left
// over for a round of their own on a few CUs, in quarters. The quarter below the diagonal of a
// symmetric result's diagonal tile is its mirror's.
template <Product WHAT, class TILE, class QUARTER>
__global__ __launch_bounds__(TILE::THREADS) void ns_product(ProductArgs p) {
  constexpr bool SYM = WHAT == kGram || WHAT == kPoly;
  constexpr int T = TILE::T;
  extern __shared__ __align__(16) uint8_t s_lds[];
  int b = blockIdx.x, quarter = -1;
  if (b < p.whole) {
    b = tile_of_block(b, p.whole);
  } else {
    quarter = (b - p.whole) & 3;
    b = p.whole + ((b - p.whole) >> 2);
  }
  const int per_matrix = SYM ? p.tiles_i * (p.tiles_i + 1) / 2 : p.tiles_i * p.tiles_j;
  const size_t g = b / per_matrix;
  b %= per_matrix;
  int ti, tj;
  if constexpr (SYM) {
    triangle_tile(b, p.tiles_i, ti, tj);
  } else {
    ti = b / p.tiles_j;
    tj = b % p.tiles_j;
  }
  if (quarter < 0) {
    tile_product<WHAT, TILE>(p, s_lds, g, ti * T, tj * T);
  } else if constexpr (TILE::T != QUARTER::T) {
    static_assert(TILE::T == 2 * QUARTER::T && TILE::THREADS == QUARTER::THREADS, "a quarter");
    if (SYM && ti == tj && quarter == 2) return;
    tile_product<WHAT, QUARTER>(p, s_lds, g, ti * T + (quarter >> 1) * QUARTER::T,
                                tj * T + (quarter & 1) * QUARTER::T);
  }
}

using Tile64 = TileOf<64, 2, 2, 8>;
using Tile128 = TileOf<128, 2, 2, 4>;
using Tile256 = TileOf<256, 2, 4, 4>;
using Quarter128 = TileOf<64, 2, 2, 4>;
using Quarter256 = TileOf<128, 2, 4, 4>;

// How a product is dealt to the 256 CUs, one workgroup of Tile256 or two of the others on each.
struct Deal {
  int tile, whole, blocks;  // tile size, tiles kept whole, workgroups
  double cost;
};

// Larger tiles copy fewer bytes for each product, smaller ones leave fewer CUs without work.
// Costs are relative to a full round of Tile256, from measurements with K = 2048: full rounds
// of 256 x 256, 512 x 128 and 512 x 64 tiles take 175, 98 and 41 us; what is left over takes
// 61 (128-tiles, one to a CU) or 31 us (64-tiles), or is cut into quarters when those fit one
// round (0.35 of a Tile256, 0.2 in all for Tile128).
Deal deal(int tile, long tiles) {
  const int slots = tile == 256 ? 256 : 512;
  const long full = tiles / slots, left = tiles % slots;
  const bool cut = tile > 64 && left > 0 && left <= slots / 4;
  const double round = tile == 256 ? 1.0 : tile == 128 ? 0.56 : 0.236;
  const double rest = left == 0 ? 0.0
                      : tile == 256 ? (cut ? 0.35 : 1.0)
                      : tile == 128 ? (cut ? 0.2 : left <= 256 ? 0.35 : 0.56)
                                    : (left <= 256 ? 0.175 : 0.236);
  const long whole = cut ? tiles - left : tiles;
  return Deal{tile, (int)whole, (int)(whole + (tiles - whole) * 4), full * round + rest};
}

// The cheapest deal of G matrices of rows x cols (multiples of 64 at least).
Deal best_deal(int G, int rows, int cols, bool symmetric) {
  Deal best{};
  for (int tile : {256, 128, 64}) {
    const long ti = cdiv(rows, tile), tj = cdiv(cols, tile);
    const Deal d = deal(tile, G * (symmetric ? ti * (ti + 1) / 2 : ti * tj));
    if (tile == 256 || d.cost < best.cost) best = d;
  }
  return best;
}

struct Workspace {
  int m, n, mp, np;
  Deal symmetric, apply;
  int parts, part_k;  // of the sums of A = X X^T
  size_t x, xt[2], a, p, norms, bits, sums, bytes;
  Workspace(int G, int M, int N) {
    m = std::min(M, N);
    n = std::max(M, N);
    symmetric = best_deal(G, m, m, true);
    apply = best_deal(G, m, n, false);
    // both sides in whole tiles of both
    const int pad = std::max(symmetric.tile, apply.tile);
    mp = cdiv(m, pad) * pad;
    np = cdiv(n, pad) * pad;
    // the tiles of the padded sides
    const long s = mp / symmetric.tile;
    symmetric = deal(symmetric.tile, G * (s * (s + 1) / 2));
    apply = deal(apply.tile, (long)G * (mp / apply.tile) * (np / apply.tile));
    const size_t big = (size_t)G * mp * np * 2 * sizeof(_Float16);
    const size_t small = (size_t)G * mp * mp * 2 * sizeof(_Float16);
    x = 0;
    xt[0] = x + big;
    xt[1] = xt[0] + big;
    a = xt[1] + big;
    p = a + small;
    norms = p + small;
    bits = norms + (size_t)G * kNormBlocks * sizeof(double);
    sums = round_up(bits + (size_t)G * (kMaxSteps + 1) * sizeof(int2), 256);
    // X X^T in parts of at least eight slices, no more workgroups than CUs, where that saves more
    // than the parts' way through memory takes: a sum shorter by 56 or 64 slices is no
    // faster (128 x 1024 95 us both, seven of 200 x 1500 164 and 168), by 88 it is (200 x 1500
    // 132 and 125)
    part_k = np;
    const int slices = np / kSlice, tiles = symmetric.blocks;
    if (symmetric.tile == Tile64::T && tiles <= 128) {
      const int most = std::min(256 / tiles, slices / 8);
      const int len = most > 1 ? cdiv(cdiv(slices, most), 4) * 4 : slices;
      if (slices - len >= 72) part_k = len * kSlice;
    }
    parts = cdiv(np, part_k);
    bytes = sums;
    if (parts > 1) bytes += (size_t)tiles * parts * Tile64::T * Tile64::T * sizeof(float);
  }
  Split at(void* base, size_t off, int G, int rows, int k) const {
    _Float16* hi = reinterpret_cast<_Float16*>((char*)base + off);
    return Split{hi, hi + (size_t)G * rows * k, rows, (size_t)rows * k};
  }
};

// The largest |x p(x^2)| that the steps reach from singular values in [0, 1], and of the
// polynomial P that multiplies X: a bound from the ends and the stationary points. False where
// they leave the range of the halves.
bool stays_in_range(int steps, const float* coeffs, Growth& growth) {
  double top = 1.0;
  growth.steps = steps;
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
    growth.a[s] = std::fabs(coeffs[3 * s]);
    growth.b[s] = std::fabs(coeffs[3 * s + 1]);
    growth.c[s] = std::fabs(coeffs[3 * s + 2]);
    growth.most[s] = (float)p_top;
    growth.top[s] = (float)next;
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
  Growth growth{};
  if (!stays_in_range(steps, coeffs, growth))
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
                  reinterpret_cast<double*>((char*)workspace + ws.norms),
                  (int)std::min<long>(kNormBlocks, ((long)M * N + 4095) / 4096),
                  reinterpret_cast<int2*>((char*)workspace + ws.bits)};
  ns_norm<<<dim3(ns.norm_blocks, G), kThreads, 0, stream>>>(ns);
  const int rows = M > N ? np : mp, cols = M > N ? mp : np;
  ns_split<<<dim3(cols / kSplitTile, rows / kSplitTile + 1, G), kThreads, 0, stream>>>(
      ns, growth, x, xt);
  auto run_tile = [&](auto tile, auto quarter, auto what, const Deal& deal, ProductArgs args) {
    using TILE = decltype(tile);
    args.tiles_i = mp / TILE::T;
    args.tiles_j = (what() == kGram || what() == kPoly ? mp : np) / TILE::T;
    args.whole = deal.whole;
    auto kernel = ns_product<what(), TILE, decltype(quarter)>;
    if (TILE::LDS > 64 * 1024 &&
        hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                            TILE::LDS) != hipSuccess)
      return false;
    kernel<<<deal.blocks, TILE::THREADS, TILE::LDS, stream>>>(args);
    return true;
  };
  auto run = [&](auto what, const ProductArgs& args) {
    const Deal& d = what() == kGram || what() == kPoly ? ws.symmetric : ws.apply;
    return d.tile == 64    ? run_tile(Tile64{}, Tile64{}, what, d, args)
           : d.tile == 128 ? run_tile(Tile128{}, Quarter128{}, what, d, args)
                           : run_tile(Tile256{}, Quarter256{}, what, d, args);
  };
  float* sums = reinterpret_cast<float*>((char*)workspace + ws.sums);
  auto run_gram = [&](ProductArgs args) {
    if (args.parts == 1) return run(std::integral_constant<Product, kGram>{}, args);
    args.tiles_i = mp / Tile64::T;
    const int tiles = ws.symmetric.blocks;
    ns_gram_part<Tile64><<<tiles * args.parts, Tile64::THREADS, Tile64::LDS, stream>>>(args);
    ns_gram_join<Tile64><<<tiles, Tile64::THREADS, Tile64::LDS, stream>>>(args);
    return true;
  };
  bool ok = true;
  for (int s = 0; s < steps && ok; ++s) {
    const ProductArgs gram{x, x, np, 0, 0, 0, ws.part_k, ws.parts, sums,
                           1.f / (kScaleX * kScaleX), a, a, a, 0.f, 0.f, 0.f, s, ns};
    const ProductArgs poly{a, a, mp, 0, 0, 0, mp, 1, nullptr,
                           1.f / (kScaleA * kScaleA), p, p, a,
                           coeffs[3 * s], coeffs[3 * s + 1], coeffs[3 * s + 2], s, ns};
    const ProductArgs apply{p, xt, mp, 0, 0, 0, mp, 1, nullptr,
                            1.f / (kScaleP * kScaleX), x, xt_next, a, 0.f, 0.f, 0.f, s, ns};
    using std::integral_constant;
    ok = run_gram(gram) &&
         run(integral_constant<Product, kPoly>{}, poly) &&
         (s + 1 < steps ? run(integral_constant<Product, kApply>{}, apply)
                        : run(integral_constant<Product, kLast>{}, apply));
    std::swap(xt, xt_next);
  }
  if (!ok) return fail(MGG_EHIP, "hipFuncSetAttribute failed");
  return launched();
}

}  // extern "C"
