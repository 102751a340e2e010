// Product of int8 rows with int8 weights, scales for each token and channel
// (pw_linear_i8):
//
//   out[t][n] = (sum_k x[t][k] w[n][k]) * x_scale[t] * w_scale[n] + bias[n]
//
// the sum exact in int32 (K <= 131071: 128 * 128 * K < 2^31).
//
// Few tokens, or little to do: k_few, tensor-core products fed from registers,
// the weights streamed once (for each block of tokens).  Otherwise k_thin up to 128
// tokens and k_tc above, on the 5th-generation tensor cores.  This GPU's int8 tensor
// rate is a small part of its 16-bit rate, and tcgen05 has no int8 kind here, so
// that work runs in fp16: int8 values are exact in fp16, their products (at most
// 2^14) are exact in fp32, and so are sums of up to 1024 of them (2^24).  Every 1024
// terms the fp32 accumulator moves from tensor memory into int32 registers, so the
// sum is the whole-number one at any K.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "pw_rows.cuh"
#include "pw_tc.cuh"

namespace pw {
namespace {

constexpr int kMaxDev = 64;

struct LinArgs {
  const int8_t* x;
  const int8_t* w;
  const float* xs;
  const float* ws;
  const void* bias;
  void* out;
  int64_t ldx, ldw, ldo;
  int T, N, K;
};

// Bounded waits of the tensor-core kernels that gave up (pw_linear_i8_status).
__device__ uint32_t g_linear_timeouts;
__global__ void k_count_timeout() { atomicAdd(&g_linear_timeouts, 1u); }

template <typename O>
__device__ __forceinline__ void store_out(const LinArgs& p, int t, int n, int acc, float xs, float ws, float bias) {
  const float v = fmaf(static_cast<float>(acc) * xs, ws, bias);
  static_cast<O*>(p.out)[t * p.ldo + n] = from_f32<O>(v);
}

// ---------------------------------------------------------------- few tokens

// The first n of 16 bytes at p, the others zero.
__device__ __forceinline__ uint4 load_tail(const int8_t* p, int n) {
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) v[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Weights are read once: past the L1, which keeps the tokens.
__device__ __forceinline__ uint4 load_once(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// D += A B, int8 16 x 32 by 32 x 8, int32.
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D += A B, fp16 16 x 16 by 16 x 8, fp32.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Four int8 values as two fp16 pairs: a byte b becomes the fp16 number
// 1024 + (b + 128) in the low byte of 0x6400, and 1152 is subtracted.
__device__ __forceinline__ void to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = v ^ 0x80808080u;                       // b + 128
  const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
  uint32_t a = prmt(u, 0x64646464u, 0x4140), b = prmt(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), k), y = __hsub2(*reinterpret_cast<__half2*>(&b), k);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void to_f16x16(const uint4& v, uint32_t (&h)[8]) {
  to_f16x4(v.x, h[0], h[1]);
  to_f16x4(v.y, h[2], h[3]);
  to_f16x4(v.z, h[4], h[5]);
  to_f16x4(v.w, h[6], h[7]);
}

// The sums of 16 G channels x 8 NT tokens of a warp, in the end in row c of
// sums[kRow] for channel c.  Up to 8 tokens in int8 (256 products a clock and SM,
// the weights need 190 at the memory's rate); above, where int8 would be the
// bound, in fp16, whose fp32 sums go to int32 every 1024 columns (run `n` of 16
// ends one): to registers, or to shared memory where registers are short (32
// tokens, 8192 x 4096: 15.5 us, 17.3 with registers; 16 tokens, 4096 x 4096: 6.9
// and 6.7).
template <int NT, int G>
struct FewSums {
  using D = std::conditional_t<NT == 1, int, float>;
  static constexpr int kRow = NT * 8 + 1;   // padded against bank conflicts
  static constexpr bool kShared = NT > 2 || G > 1;
  D part[G][NT][4] = {};
  int acc[G][NT][4] = {};   // where sums go to registers
  int* s = nullptr;         // of the lane's first channel and token

  __device__ __forceinline__ void place(int* sums, int lane) { s = sums + (lane >> 2) * kRow + (lane & 3) * 2; }
  __device__ __forceinline__ FewSums(int* sums, int lane) {
    if constexpr (kShared) {
      place(sums, lane);
      for (int i = lane; i < 16 * G * kRow; i += 32) sums[i] = 0;
      __syncwarp();
    }
  }
  // w: channels g and g + 8 of every 16
  __device__ __forceinline__ void add(const uint4 (&w)[2 * G], const uint4 (&x)[NT], int n) {
    if constexpr (NT == 1) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const uint4 &a = w[2 * h], &b = w[2 * h + 1];
        mma_s8(part[h][0], a.x, b.x, a.y, b.y, x[0].x, x[0].y);
        mma_s8(part[h][0], a.z, b.z, a.w, b.w, x[0].z, x[0].w);
      }
    } else {
      uint32_t hw[2 * G][8];
#pragma unroll
      for (int i = 0; i < 2 * G; ++i) to_f16x16(w[i], hw[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t hx[8];
        to_f16x16(x[j], hx);
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            mma_f16_16816(part[h][j], hw[2 * h][i], hw[2 * h + 1][i], hw[2 * h][i + 1], hw[2 * h + 1][i + 1], hx[i],
                          hx[i + 1]);
      }
      if (n % 16 == 15) flush();
    }
  }
  // part[h][j][0..3]: channels g, g, g + 8, g + 8 of 16; tokens 8 j + 2 q + 0, 1, 0, 1
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) f(h, j, i, (h * 16 + (i >> 1) * 8) * kRow + j * 8 + (i & 1));
  }
  __device__ __forceinline__ void flush() {
    each([&](int h, int j, int i, int at) {
      (kShared ? s[at] : acc[h][j][i]) += static_cast<int>(part[h][j][i]);
      part[h][j][i] = 0;
    });
  }
  __device__ __forceinline__ void finish(int* sums, int lane) {
    if constexpr (NT > 1) flush();
    if constexpr (!kShared) {
      place(sums, lane);
      each([&](int h, int j, int i, int at) { s[at] = NT > 1 ? acc[h][j][i] : static_cast<int>(part[h][j][i]); });
    }
  }
};

constexpr int kFewWarps = 8;
constexpr int few_ctas(bool ahead) { return ahead ? 2 : 3; }   // of an SM
constexpr int few_groups(int nt, bool ahead) { return nt > 1 && !ahead ? 2 : 1; }   // of 16 channels, a warp's
// k_few against k_thin, K = 4096, us: 16 tokens 6.7 and 18 at N = 4096, 28 and 36
// at 28672, 108 and 118 at 131072; 24 tokens 22 and 25 at 14336, 37 and 35 at 28672;
// 32 tokens 9 and 18 at 4096, 25 and 25 at 14336, 38 and 33 at 20000, 44 and 36 at
// 28672.
constexpr int kFewTokens = 16;
constexpr int kManyChannels = 16384;   // from which 17 to 32 tokens take k_thin

// A group of kw warps owns 16 G channels and up to 8 NT tokens (blockIdx.y) and
// shares out K in runs of 64 columns.
// Lane (g, q) = (lane / 4, lane % 4) loads the 16 bytes at column 16 q of
// channels g and g + 8 of every 16, and of token g of every 8: the operand
// registers of its products, with the columns of K in an order of their own that
// both operands share.  So the weights go from memory to the tensor cores through
// registers alone, 64 bytes of a channel at a time (128 at a time, in loads of 32
// bytes, was no faster).  NT: groups of 8 tokens.  The loads in flight come from
// three CTAs of an SM, whose other warps load while one multiplies, or from two
// that fetch their next U runs ahead (AHEAD).  One token, 28672 x 4096: 22 us,
// 79 % of the copy rate, and 25 with AHEAD; what is left there is the launch and
// the ramps, 131072 channels run at 92 %.  16 tokens, 131072 x 4096: 108 us, 74 %,
// with a token converted for 32 channels (G = 2; 116 with 16): the conversions to
// fp16 (20 instructions for each 16 bytes) and the products take half of the issue
// slots, and the warps wait for operands in the other half.
template <typename O, int NT, bool AHEAD>
__global__ void __launch_bounds__(kFewWarps * 32, few_ctas(AHEAD)) k_few(const LinArgs p, int kw) {
  constexpr int G = few_groups(NT, AHEAD), kChannels = 16 * G;
  constexpr int U = NT == 1 ? 4 : AHEAD ? 2 : 1;
  using Sums = FewSums<NT, G>;
  __shared__ int s_part[kFewWarps][kChannels * Sums::kRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int groups = kFewWarps / kw, turn = warp % kw;
  const int n0 = (blockIdx.x * groups + warp / kw) * kChannels;
  const int t0 = blockIdx.y * (NT * 8), T = min(p.T - t0, NT * 8);
  const int runs = (p.K + 63) / 64;
  const int r0 = static_cast<int>(static_cast<int64_t>(runs) * turn / kw);
  const int r1 = static_cast<int>(static_cast<int64_t>(runs) * (turn + 1) / kw);
  const int8_t* w[2 * G];
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) w[i] = p.w + min(n0 + g + 8 * i, p.N - 1) * p.ldw + q * 16;
  const int8_t* x[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) x[j] = p.x + (t0 + min(j * 8 + g, T - 1)) * p.ldx + q * 16;
  Sums sums(s_part[warp], lane);
  const int whole = min(r1, p.K / 64);
  const int last = r0 + (whole > r0 ? (whole - r0) / U * U : 0);   // turns of U whole runs end here
  uint4 a[U][2 * G];
  auto fetch = [&](int k) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2 * G; ++i) a[u][i] = load_once(w[i] + (k + u) * 64);
  };
  int k = r0;
  if (AHEAD && k < last) fetch(k);
  for (; k < last; k += U) {
    if (!AHEAD) fetch(k);
    uint4 c[U][2 * G], v[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < 2 * G; ++i) c[u][i] = a[u][i];
#pragma unroll
      for (int j = 0; j < NT; ++j) v[u][j] = __ldg(reinterpret_cast<const uint4*>(x[j] + (k + u) * 64));
    }
    if (AHEAD && k + U < last) fetch(k + U);
#pragma unroll
    for (int u = 0; u < U; ++u) sums.add(c[u], v[u], k - r0 + u);
  }
  for (; k < r1; ++k) {   // single runs, the last one perhaps not whole
    const int left = p.K - k * 64 - q * 16;
    auto part = [&](const int8_t* from) {
      return left >= 16 ? __ldg(reinterpret_cast<const uint4*>(from + k * 64)) : load_tail(from + k * 64, left);
    };
    uint4 c[2 * G], v[NT];
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) c[i] = part(w[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j) v[j] = part(x[j]);
    sums.add(c, v, k - r0);
  }
  sums.finish(s_part[warp], lane);
  __syncthreads();
  for (int i = threadIdx.x; i < groups * kChannels * T; i += kFewWarps * 32) {
    const int c = i % (groups * kChannels), t = i / (groups * kChannels), grp = c / kChannels;
    const int n = blockIdx.x * groups * kChannels + c;
    if (n >= p.N) continue;
    int sum = 0;
    for (int j = 0; j < kw; ++j) sum += s_part[grp * kw + j][c % kChannels * Sums::kRow + t];
    store_out<O>(p, t0 + t, n, sum, __ldg(p.xs + t0 + t), __ldg(p.ws + n),
                 p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n]) : 0.f);
  }
}

// How many warps share a group's K: the count that leaves the least of the last
// wave of CTAs idle, each doubling charged 6 % for its shorter loops and longer
// joins, each warp with two runs or more.  T = 1, N = 131072, K = 4096: 94.5 us
// with one warp (2.2 waves), 84.7 with four (9.0 waves); at 28672 with 1, 2, 4 and
// 8: 26.9, 21.7, 22.0 and 24.0.
template <typename O, int NT, bool AHEAD>
cudaError_t launch_few_nt(const LinArgs& p, cudaStream_t s) {
  constexpr int kChannels = 16 * few_groups(NT, AHEAD);
  const int groups = (p.N + kChannels - 1) / kChannels, runs = (p.K + 63) / 64, slots = sm_count() * few_ctas(AHEAD);
  const int token_blocks = (p.T + NT * 8 - 1) / (NT * 8);
  int kw = 1;
  float least = 0.f;
  for (int n = 1, i = 0; n <= kFewWarps && (n == 1 || runs >= 2 * n); n *= 2, ++i) {
    const float waves = static_cast<float>(groups) * token_blocks * n / (kFewWarps * slots);
    const float cost = std::ceil(waves) / waves * (1.f + 0.06f * i);
    if (n == 1 || cost < least) kw = n, least = cost;
  }
  const int per = kFewWarps / kw;
  k_few<O, NT, AHEAD><<<dim3((groups + per - 1) / per, token_blocks), kFewWarps * 32, 0, s>>>(p, kw);
  return cudaGetLastError();
}

template <typename O>
cudaError_t launch_few(const LinArgs& p, cudaStream_t s) {
  // 16 tokens, K = 4096, loading ahead against three CTAs and 32 channels to a
  // warp, us: N = 4096 6.7 and 9.7, 8192 10.7 and 11.8, 14336 17.6 and 15.4, 131072
  // 119 and 108
  if (p.T <= 16)
    return (p.N + 15) / 16 <= 4 * sm_count() ? launch_few_nt<O, 2, true>(p, s) : launch_few_nt<O, 2, false>(p, s);
  if (p.T <= 24) return launch_few_nt<O, 3, true>(p, s);
  return launch_few_nt<O, 4, true>(p, s);
}

// ---------------------------------------------------------------- tensor cores

// k_widen writes the tokens as fp16 into the workspace; then one CTA per SM
// takes tiles of 256 channels (M, the weights) x up to NT tokens (N) with another.
// Warps by role:
//  * warp 0 fetches int8 weights by TMA into a ring of S8 stages, warp 2 the
//    fp16 tokens into the operand ring of S stages;
//  * the last 8 warps, in 4 groups that take a stage in turn, convert the
//    weights to fp16 in the operand ring, in the K-major 128-byte-swizzled
//    layout the MMA reads;
//  * warp 1 issues tcgen05.mma kind::f16 (fp32 in tensor memory), up to 1024
//    columns of K into one accumulator, then as many into another;
//  * warps 4.. add each finished accumulator to their int32 registers while
//    the next one fills, and at the tile's end scale and store.
// Two CTAs of a cluster make a pair (cta_group::2), each with its own 128
// channels and half of the tokens, so a stage of 256 tokens brings 24 KB to an
// SM instead of 40 (at 40 the L2 was the bound, about 9.6 TB/s), and one issue
// serves two SMs.  The even CTA issues the MMAs for both.
// What bounds it at 256 tokens are two things alike: those 24 KB at the L2's rate
// (790 clocks a stage) and the shared-memory data pipe (128 bytes a clock), which
// the tensor cores' operand reads (48 KB) share with the conversion (24 KB) and
// the copies (24 KB): 768 of its clocks for 512 of MMA.  Converting the tokens
// here too made 1025.
// Where there are few tiles a cluster of CTAs splits K and adds the parts
// through distributed shared memory; whole numbers, so in any order.
//
// 28672 x 4096 weights: 1024, 2048, 4096 tokens in 148, 290 and 573 us (1617 to
// 1678 TFLOP/s, 86 to 89 % of the 16-bit library product in isolation, and near
// its rate in a long run: the power limit is in reach).  2048 x 4096 x 14336:
// 177 us, 1360 TFLOP/s, 128 tiles in two turns of 76 pairs.  333 x 5003 x 1411:
// 18 us, a chain of k_widen, 23 stages, the joins and the stores.  One CTA to a
// tile, converting the tokens too, took 238 us of the 177; two issuers, or two
// stages to a barrier, gained nothing; the last two turns' tiles cut into equal
// runs of K gave 171, and 160 instead of 153 at 1024 x 28672 x 4096.
constexpr int kM = 128;
constexpr int kBK = 64;         // K columns of a stage: a 128-byte row of fp16
constexpr int kConvWarps = 8;
constexpr int kGroups = 4;      // of converting warps, a stage at a time each
constexpr int kGroupWarps = kConvWarps / kGroups;
constexpr int kChunk = 1024 / kBK;   // stages that fp32 adds exactly: 2^24 / 2^14 products
constexpr int kEpiWarp0 = 4;

// Whether the converting groups, which take the stages in turn, can wait by
// parity.  A parity tells a stage's last use from the one before, not from
// earlier ones, and loads land in any order: at step s a group must know by
// itself that the load of step s - S8 has landed.  It does where that step was its
// own (S8 a multiple of the groups), or where a product that it has waited for was
// at or behind it: the one of s - groups - S, which its last step waited for, or,
// where a step waits for its operand stage first, the one of s - S.  The operand
// ring's uses end in order, as the products do.
constexpr bool parities_suffice(int groups, int S, int S8, bool operand_first) {
  return groups <= S && groups <= S8 && (S8 % groups == 0 || S8 >= S + (operand_first ? 0 : groups));
}

struct Tile {
  static constexpr int NT = 256;
  static constexpr int EW = 8;                            // accumulating warps
  static constexpr int ACC = NT / (EW / 4);               // int32 sums of one of their threads
  static constexpr int kConvWarp0 = kEpiWarp0 + EW;
  static constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
  static constexpr int kRowsB = NT / 2;                   // tokens that a CTA holds
  static constexpr int A = kM * kBK * 2, B = kRowsB * kBK * 2;   // bytes of a stage's operands
  static constexpr int A8 = kM * kBK;                     // and of its int8 weights
  static constexpr int S = 5;                             // operand stages
  static constexpr int S8 = 8;                            // int8 stages
  static constexpr int kRing8 = S * (A + B);
  static constexpr int kOffBar = kRing8 + S8 * A8;
  static constexpr int kSmem = kOffBar + 8 * (3 * S + 2 * S8 + 6) + 16 + 1024;
  static constexpr uint32_t kCols = 2 * NT;
  // D f32, A and B f16, N / 8 and M / 16
  __host__ __device__ static constexpr uint32_t idesc(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(2 * kM >> 4) << 24);
  }
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kM * NT * 4 <= kRing8, "a CTA's int32 sums fit the operand ring");
  static_assert(parities_suffice(kGroups, S, S8, false), "no group is a lap ahead of another");
};

// Registers by role; the accumulating threads hold 128 sums:
// 640 threads are launched with kRegsLaunch each; 128 * (32 + 2 * 160 + 2 * 64)
// = 640 * 96 = 61440.  Every role returns to kRegsLaunch at its end: the
// accumulating warps give theirs back before a CTA barrier, the others take
// them after it (a warp that took its share while the accumulating warps were
// still waiting for theirs would leave them waiting for good).
constexpr int kRegsLaunch = 96, kRegsIssue = 32, kRegsAcc = 160, kRegsConv = 64;
static_assert(128 * (kRegsIssue + 2 * kRegsAcc + 2 * kRegsConv) <= 640 * kRegsLaunch, "register split");

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// A converting thread's part of a stage: 16 columns at 16 (tid % 4) of the
// channels tid / 4 + 8 WARPS i.  Eight neighbouring threads read two rows of 64
// bytes (with the TMA's 64-byte swizzle) and write 16-byte pieces of two fp16
// rows, each time to different banks.
template <int ROWS, int WARPS>
struct Weights {
  static constexpr int kN = ROWS / (WARPS * 8);
  uint4 v[kN];

  __device__ __forceinline__ void load(uint32_t src, int tid, int rows = ROWS) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (i * (WARPS * 8) >= rows) break;
      const int r = (tid >> 2) + i * (WARPS * 8);
      v[i] = lds16(src + r * 64 + (((tid & 3) ^ ((r >> 1) & 3)) << 4));
    }
  }
  __device__ __forceinline__ void store(uint32_t dst, int tid, int rows = ROWS) const {
    const int j = (tid & 3) * 2;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (i * (WARPS * 8) >= rows) break;
      const int r = (tid >> 2) + i * (WARPS * 8);
      uint32_t h[8];
      to_f16x16(v[i], h);
      sts16(dst + r * 128 + ((j ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
      sts16(dst + r * 128 + (((j + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
    }
  }
};

__device__ __forceinline__ int4 ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Polls up to kPolls times (about a second; PAUSE ns between two) for the phase
// of the given parity; false, and the abort flag, when they run out or another
// thread has raised it.
constexpr int kPolls = 1 << 23;
template <int PAUSE = 0>
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, volatile int* abort) {
  for (int n = 0; !test_wait(bar, parity); ++n) {
    if (*abort) return false;
    if (n == kPolls) {
      atomicAdd(&g_linear_timeouts, 1u);
      *abort = 1;
      return false;
    }
    if (PAUSE) __nanosleep(PAUSE);
  }
  return true;
}

// MMA of a pair of CTAs.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
template <typename O>
__global__ void __launch_bounds__(Tile::kThreads, 1)
k_tc(const LinArgs p, const __grid_constant__ CUtensorMap mapw, const __grid_constant__ CUtensorMap mapx, int nt,
     int split) {
  using C = Tile;
  constexpr int NT = C::NT;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = saddr(smem);
  const uint32_t fullw = base + C::kOffBar, fullx = fullw + 8 * C::S, empty = fullx + 8 * C::S;
  const uint32_t full8 = empty + 8 * C::S, empty8 = full8 + 8 * C::S8;
  const uint32_t dfull = empty8 + 8 * C::S8, dempty = dfull + 16, fin = dempty + 16;
  int* s_misc = reinterpret_cast<int*>(smem + C::kOffBar + 8 * (3 * C::S + 2 * C::S8 + 6));   // tmem, abort
  volatile int* abort = s_misc + 1;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the compiler then knows that it is uniform
  // the CTA's place: in its pair, and among the parts of K
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const uint32_t side = rank & 1, part = rank >> 1, leader = rank - side;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(s_misc)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::S; ++i) {
      // the weights of a stage in both CTAs, and the odd CTA's tokens
      mbar_init(fullw + 8 * i, 2 * kGroupWarps + 1);
      mbar_init(fullx + 8 * i, 1);   // the CTA's own tokens
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < C::S8; ++i) mbar_init(full8 + 8 * i, 1), mbar_init(empty8 + 8 * i, kGroupWarps);
    mbar_init(fin, 1);
    for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, 2 * C::EW);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_misc[1] = 0;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers and tensor memory
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(s_misc[0]), 0);

  // a warp waits through one thread: polls of all its lanes would keep the
  // other warps' barrier operations waiting
  auto warp_ok = [&](bool ok) {
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();
    return ok;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return warp_ok(lane != 0 || poll(bar, parity, abort)); };
  // after an abort, what this thread has in flight still ends before the CTA
  // does: the last use of every stage of a ring, the current lap's below r.stage
  auto drain = [&](uint32_t bars, uint32_t stages, const auto& r) {
    volatile int none = 0;
    for (uint32_t i = 0; i < stages; ++i) {
      if (i < r.stage)
        poll(bars + 8 * i, r.parity, &none);
      else if (!r.first)
        poll(bars + 8 * i, r.parity ^ 1, &none);
    }
  };

  const int ntn = (p.N + 2 * kM - 1) / (2 * kM), ntt = (p.T + nt - 1) / nt;
  const int tiles = ntn * ntt;
  const int steps_all = (p.K + kBK - 1) / kBK;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps_all) * part / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps_all) * (part + 1) / split);
  const int steps = s1 - s0;
  const int tile0 = blockIdx.x / (2 * split), tile_step = gridDim.x / (2 * split);
  auto channel0 = [&](int tile) { return ((tile % ntn) * 2 + static_cast<int>(side)) * kM; };

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {
      // ---- int8 weights by TMA
      Ring<C::S8> r;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        const int n0 = channel0(tile);
        for (int k = s0; k < s1; ++k, r.next()) {
          if (!r.first && !(ok = poll(empty8 + 8 * r.stage, r.parity ^ 1, abort))) break;
          mbar_expect_tx(full8 + 8 * r.stage, C::A8);
          tma_load_2d(base + C::kRing8 + r.stage * C::A8, &mapw, k * kBK, n0, full8 + 8 * r.stage);
        }
      }
      if (*abort) drain(full8, C::S8, r);
    }
    if (warp == 2 && lane == 0) {
      // ---- fp16 tokens by TMA, once k_widen has written them
      asm volatile("griddepcontrol.wait;" ::: "memory");
      Ring<C::S> r;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        const int t0 = (tile / ntn) * nt + static_cast<int>(side) * (nt / 2);
        for (int k = s0; k < s1; ++k, r.next()) {
          if (!r.first && !(ok = poll(empty + 8 * r.stage, r.parity ^ 1, abort))) break;
          mbar_expect_tx(fullx + 8 * r.stage, nt / 2 * kBK * 2);
          tma_load_2d(base + r.stage * (C::A + C::B) + C::A, &mapx, k * kBK, t0, fullx + 8 * r.stage);
        }
      }
      if (*abort) drain(fullx, C::S, r);
    }
    if (warp == 1 && side) {
      // ---- the odd CTA's tokens are reported to the even one
      if (lane == 0) {
        Ring<C::S> r;
        const int64_t all = static_cast<int64_t>(steps) * ((tiles - tile0 + tile_step - 1) / tile_step);
        for (int64_t g = 0; g < all && poll(fullx + 8 * r.stage, r.parity, abort); ++g, r.next())
          arrive_at(fullw + 8 * r.stage, leader);
      }
    } else if (warp == 1) {
      // ---- MMA issue: the whole warp in step, so that the operands stay in
      // uniform registers, and an elected thread for the instructions.  A
      // barrier takes over 100 clocks to read, so the next stage's is read
      // before this stage's MMAs are issued and looked at after
      const uint16_t both = static_cast<uint16_t>(3u << leader);
      Ring<C::S> r;
      const uint32_t idesc = C::idesc(nt);
      Ring<2> d;
      bool ok = true, ready = false;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        for (int k = 0; k < steps && ok; d.next()) {
          if (!d.first && !(ok = wait(dempty + 8 * d.stage, d.parity ^ 1))) break;
          tc_fence_after();
          const uint32_t acc = tmem + d.stage * NT;
          const int end = min(steps, k + kChunk);
          for (uint32_t more = 0; k < end; ++k) {
            if (!ready && !(ok = wait(fullx + 8 * r.stage, r.parity) && wait(fullw + 8 * r.stage, r.parity))) break;
            tc_fence_after();
            const uint32_t stage = r.stage;
            r.next();
            ready = test_wait(fullx + 8 * r.stage, r.parity) & test_wait(fullw + 8 * r.stage, r.parity);
            if (elect_one()) {
              const uint64_t da = smem_desc(base + stage * (C::A + C::B)), db = da + (C::A >> 4);
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) mma_pair(acc, da + kk * 2, db + kk * 2, idesc, more | kk);
              commit_pair(empty + 8 * stage, both);
            }
            ready = __all_sync(0xffffffffu, ready);
            more = 1;
          }
          if (ok && elect_one()) commit_pair(dfull + 8 * d.stage, both);
          __syncwarp();
        }
      }
      if (*abort) {   // the MMAs in flight end before the CTA does
        if (elect_one()) {
          volatile int none = 0;
          commit_pair(fin, static_cast<uint16_t>(1u << leader));
          poll(fin, 0, &none);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    cta_barrier();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  } else if (warp < C::kConvWarp0) {
    // ---- accumulate and store
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAcc));
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * C::ACC;
    Ring<2> d;
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
      int acc[C::ACC];
#pragma unroll
      for (int i = 0; i < C::ACC; ++i) acc[i] = 0;
      for (int k = 0; k < steps; k += kChunk, d.next()) {
        if (!(ok = warp_ok(lane != 0 || poll<100>(dfull + 8 * d.stage, d.parity, abort)))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::ACC; c += 16) {
          uint32_t r[16];
          tmem_ld16(lanes + d.stage * NT + c, r);
          tmem_wait(r);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(dempty + 8 * d.stage, leader);
      }
      if (!ok) break;
      const int n0 = channel0(tile), t0 = (tile / ntn) * nt, t1 = min(p.T, t0 + nt);
      if (split == 1) {
        // the token scales are read ahead and passed around the warp: a load
        // beside each store would wait for the store (they might be the same memory)
        const int n = n0 + q * 32 + lane, ts = t0 + half * C::ACC;
        float xs[C::ACC / 32], ws = 0.f, bias = 0.f;
#pragma unroll
        for (int i = 0; i < C::ACC / 32; ++i) xs[i] = ts + i * 32 + lane < t1 ? __ldg(p.xs + ts + i * 32 + lane) : 0.f;
        if (n < p.N) {
          ws = __ldg(p.ws + n);
          if (p.bias) bias = to_f32<O>(static_cast<const O*>(p.bias)[n]);
        }
        O* out = static_cast<O*>(p.out) + ts * p.ldo + n;
#pragma unroll
        for (int i = 0; i < C::ACC; ++i) {
          const float x = __shfl_sync(0xffffffffu, xs[i / 32], i % 32);
          if (n < p.N && ts + i < t1) *out = from_f32<O>(fmaf(static_cast<float>(acc[i]) * x, ws, bias));
          out += p.ldo;
        }
      } else {
        // every stage of the ring has been read: its space takes the sums
        int* sums = reinterpret_cast<int*>(smem);
#pragma unroll
        for (int i = 0; i < C::ACC; ++i) sums[(half * C::ACC + i) * kM + q * 32 + lane] = acc[i];
      }
    }
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    cta_barrier();
  } else {
    // ---- int8 to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    const int ctid = (tid - C::kConvWarp0 * 32) % (kGroupWarps * 32);
    const int group = (warp - C::kConvWarp0) / kGroupWarps;
    Ring<C::S> r;
    Ring<C::S8> r8;
    r.next(group);
    r8.next(group);
    const int64_t mine = static_cast<int64_t>(steps) * ((tiles - tile0 + tile_step - 1) / tile_step);
    for (int64_t g = group; g < mine; g += kGroups, r.next(kGroups), r8.next(kGroups)) {
      if (!wait(full8 + 8 * r8.stage, r8.parity)) break;
      Weights<kM, kGroupWarps> w;
      w.load(base + C::kRing8 + r8.stage * C::A8, ctid);
      if (!r.first && !wait(empty + 8 * r.stage, r.parity ^ 1)) break;
      w.store(base + r.stage * (C::A + C::B), ctid);
      proxy_fence_smem();
      __syncwarp();
      if (lane == 0) {
        arrive_at(fullw + 8 * r.stage, leader);
        mbar_arrive(empty8 + 8 * r8.stage);   // not before the stores: the loads have then arrived for sure
      }
    }
    __syncwarp();
    cta_barrier();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  }

  __syncwarp();
  if (split > 1) {
    // the parts of one tile: each CTA adds and stores its share of the tokens
    cluster_sync();
    if (!*abort) {
      const int n0 = channel0(tile0), t0 = (tile0 / ntn) * nt;
      const int j0 = nt * part / split, j1 = nt * (part + 1) / split;
      const int end = j1 * (kM / 4);
      const int n = n0 + tid % (kM / 4) * 4;   // four channels, the same for all of the thread's tokens
      float ws[4], bias[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool in = n + c < p.N;
        ws[c] = in ? __ldg(p.ws + n + c) : 0.f;
        bias[c] = in && p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n + c]) : 0.f;
      }
      constexpr int U = 4;                     // tokens whose loads are in flight together
      for (int i0 = j0 * (kM / 4) + tid; i0 < end; i0 += U * C::kThreads) {
        int4 sum[U];
        float xs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * C::kThreads, t = t0 + i / (kM / 4);
          sum[u] = make_int4(0, 0, 0, 0);
          xs[u] = i < end && t < p.T ? __ldg(p.xs + t) : 0.f;
        }
        for (int r = 0; r < split; ++r) {
          int4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) v[u] = ld_cluster(base + min(i0 + u * C::kThreads, end - 1) * 16, r * 2 + side);
#pragma unroll
          for (int u = 0; u < U; ++u)
            sum[u].x += v[u].x, sum[u].y += v[u].y, sum[u].z += v[u].z, sum[u].w += v[u].w;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * C::kThreads, t = t0 + i / (kM / 4);
          if (i >= end || t >= p.T) continue;
          const int v[4] = {sum[u].x, sum[u].y, sum[u].z, sum[u].w};
          O* out = static_cast<O*>(p.out) + t * p.ldo + n;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (n + c < p.N) out[c] = from_f32<O>(fmaf(static_cast<float>(v[c]) * xs[u], ws[c], bias[c]));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // nothing of this CTA is read or signalled any more
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
}

// ---------------------------------------------------------------- up to 128 tokens

// An MMA takes about 130 clocks however few columns it has, so with the
// channels as its rows (k_tc) few tokens leave it mostly empty.  Here they are
// its columns: one CTA, up to 128 tokens (M, rows past T hold anything) x 128 to
// 256 channels (N).  Roles and rings as in k_tc, without the pair: half the MMAs
// for the same weights.  MT: tokens that a stage has room for; the MMA reads
// 128 rows, the ones past MT from the weights behind them, into lanes that
// nobody reads.  A stage of 256 channels x 64 columns goes into shared memory by
// TMA (16 KB), out for conversion, in again as fp16 (32 KB) and out to the MMA,
// about 1000 clocks of its data pipe with the tokens, and 1100 are taken; at 192
// channels it is 1050, so the chain of barriers and conversions counts too.
// 28672 x 4096 weights: 36, 39 and 42 us for 32, 64 and 128 tokens (46 % of the
// copy rate at 64); k_tc takes 53 for 129 to 160.
constexpr int kThinN = 256;
template <int MT>
struct Thin {
  static constexpr int EW = 8, ACC = 128;
  static constexpr int kConvWarp0 = kEpiWarp0 + EW;
  static constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
  static constexpr int kGroups = 2, kGroupWarps = kConvWarps / kGroups;
  static constexpr int X = MT * kBK * 2, W = kThinN * kBK * 2;   // bytes of a stage's operands
  static constexpr int W8 = kThinN * kBK;                        // and of its int8 weights
  static constexpr int S = MT == 32 ? 4 : 3;
  static constexpr int S8 = MT == 64 ? 6 : 5;
  // whether a converting group waits for its operand stage before the weights: what
  // 4 and 5 stages need (parities_suffice).  32 x 28672 and 32 x 131072 x 4096: 36 and
  // 120 us; weights first with 3 and 6 stages 38 and 141, with 4 and 4 49 and 181.  64
  // rows, whose 6 stages are a multiple of the groups: 39 us, and 41 operand first
  static constexpr bool kOperandFirst = MT == 32;
  static constexpr int kRing8 = S * (X + W);
  static constexpr int kOffBar = kRing8 + S8 * W8;
  static constexpr int kSmem = kOffBar + 8 * (3 * S + 2 * S8 + 5) + 16 + 1024;
  static constexpr uint32_t kCols = 2 * kThinN;
  __host__ __device__ static constexpr uint32_t idesc(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kM >> 4) << 24);
  }
  static constexpr int kSumRow = MT + 1;                         // of a channel's int32 sums, padded
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  // a tile's int32 sums, and half of them once more, fit the rings
  static_assert(kThinN * kSumRow * 4 + MT * (kThinN / 2 + 1) * 4 <= kOffBar, "sums");
  static_assert(kM * kBK * 2 <= X + W, "the rows past MT are inside the stage");
  static_assert(parities_suffice(kGroups, S, S8, kOperandFirst), "no group is a lap ahead of another");
};

__device__ __forceinline__ int ld_cluster1(uint32_t addr, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

template <typename O, int MT>
__global__ void __launch_bounds__(Thin<MT>::kThreads, 1)
k_thin(const LinArgs p, const __grid_constant__ CUtensorMap mapw, const __grid_constant__ CUtensorMap mapx, int box,
       int nw, int split) {
  using C = Thin<MT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = saddr(smem);
  const uint32_t fullw = base + C::kOffBar, fullx = fullw + 8 * C::S, empty = fullx + 8 * C::S;
  const uint32_t full8 = empty + 8 * C::S, empty8 = full8 + 8 * C::S8;
  const uint32_t dfull = empty8 + 8 * C::S8, dempty = dfull + 16, fin = dempty + 16;
  int* s_misc = reinterpret_cast<int*>(smem + C::kOffBar + 8 * (3 * C::S + 2 * C::S8 + 5));   // tmem, abort
  volatile int* abort = s_misc + 1;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  uint32_t part;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(part));

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(s_misc)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::S; ++i) {
      mbar_init(fullw + 8 * i, C::kGroupWarps);
      mbar_init(fullx + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < C::S8; ++i) mbar_init(full8 + 8 * i, 1), mbar_init(empty8 + 8 * i, C::kGroupWarps);
    for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, C::EW);
    mbar_init(fin, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_misc[1] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(s_misc[0]), 0);

  auto warp_ok = [&](bool ok) {
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();
    return ok;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return warp_ok(lane != 0 || poll(bar, parity, abort)); };
  auto drain = [&](uint32_t bars, uint32_t stages, const auto& r) {   // as in k_tc
    volatile int none = 0;
    for (uint32_t i = 0; i < stages; ++i) {
      if (i < r.stage)
        poll(bars + 8 * i, r.parity, &none);
      else if (!r.first)
        poll(bars + 8 * i, r.parity ^ 1, &none);
    }
  };

  const int tiles = (p.N + nw - 1) / nw;
  const int steps_all = (p.K + kBK - 1) / kBK;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps_all) * part / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps_all) * (part + 1) / split);
  const int steps = s1 - s0;
  const int tile0 = blockIdx.x / split, tile_step = gridDim.x / split;

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {
      // ---- int8 weights by TMA
      Ring<C::S8> r;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        for (int k = s0; k < s1; ++k, r.next()) {
          if (!r.first && !(ok = poll(empty8 + 8 * r.stage, r.parity ^ 1, abort))) break;
          mbar_expect_tx(full8 + 8 * r.stage, nw * kBK);
          tma_load_2d(base + C::kRing8 + r.stage * C::W8, &mapw, k * kBK, tile * nw, full8 + 8 * r.stage);
        }
      }
      if (*abort) drain(full8, C::S8, r);
    }
    if (warp == 2 && lane == 0) {
      // ---- fp16 tokens by TMA, once k_widen has written them
      asm volatile("griddepcontrol.wait;" ::: "memory");
      Ring<C::S> r;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        for (int k = s0; k < s1; ++k, r.next()) {
          if (!r.first && !(ok = poll(empty + 8 * r.stage, r.parity ^ 1, abort))) break;
          mbar_expect_tx(fullx + 8 * r.stage, box * kBK * 2);
          tma_load_2d(base + r.stage * (C::X + C::W), &mapx, k * kBK, 0, fullx + 8 * r.stage);
        }
      }
      if (*abort) drain(fullx, C::S, r);
    }
    if (warp == 1) {
      // ---- MMA issue
      const uint32_t idesc = C::idesc(nw);
      Ring<C::S> r;
      Ring<2> d;
      bool ok = true, ready = false;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        for (int k = 0; k < steps && ok; d.next()) {
          if (!d.first && !(ok = wait(dempty + 8 * d.stage, d.parity ^ 1))) break;
          tc_fence_after();
          const uint32_t acc = tmem + d.stage * kThinN;
          const int end = min(steps, k + kChunk);
          for (uint32_t more = 0; k < end; ++k) {
            if (!ready && !(ok = wait(fullx + 8 * r.stage, r.parity) && wait(fullw + 8 * r.stage, r.parity))) break;
            tc_fence_after();
            const uint32_t stage = r.stage;
            r.next();
            ready = test_wait(fullx + 8 * r.stage, r.parity) & test_wait(fullw + 8 * r.stage, r.parity);
            if (elect_one()) {
              const uint64_t da = smem_desc(base + stage * (C::X + C::W)), db = da + (C::X >> 4);
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) mma_f16(acc, da + kk * 2, db + kk * 2, idesc, more | kk);
              mma_commit(empty + 8 * stage);
            }
            ready = __all_sync(0xffffffffu, ready);
            more = 1;
          }
          if (ok && elect_one()) mma_commit(dfull + 8 * d.stage);
          __syncwarp();
        }
      }
      if (*abort) {   // the MMAs in flight end before the CTA does
        if (elect_one()) {
          volatile int none = 0;
          mma_commit(fin);
          poll(fin, 0, &none);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    cta_barrier();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  } else if (warp < C::kConvWarp0) {
    // ---- accumulate and store: a token to a lane, 128 channels to a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAcc));
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * C::ACC;
    const int t = q * 32 + lane;
    const bool busy = q * 32 < p.T;
    Ring<2> d;
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
      int acc[C::ACC];
#pragma unroll
      for (int i = 0; i < C::ACC; ++i) acc[i] = 0;
      for (int k = 0; k < steps; k += kChunk, d.next()) {
        if (!(ok = warp_ok(lane != 0 || poll<100>(dfull + 8 * d.stage, d.parity, abort)))) break;
        tc_fence_after();
        if (busy) {
#pragma unroll
          for (int c = 0; c < C::ACC; c += 16) {
            uint32_t r[16];
            tmem_ld16(lanes + d.stage * kThinN + c, r);
            tmem_wait(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dempty + 8 * d.stage);
      }
      if (!ok) break;
      if (!busy) continue;
      if (split == 1) {
        // lane l holds the scales of channels n + 4 l .. + 3 of this half
        const int n = tile * nw + half * C::ACC, end = min(p.N, (tile + 1) * nw);
        float ws[4], bias[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool in = n + lane * 4 + c < end;
          ws[c] = in ? __ldg(p.ws + n + lane * 4 + c) : 0.f;
          bias[c] = in && p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n + lane * 4 + c]) : 0.f;
        }
        const float xs = t < p.T ? __ldg(p.xs + t) : 0.f;
        O* out = static_cast<O*>(p.out) + t * p.ldo + n;
        constexpr int E = 16 / sizeof(O);   // channels of a 16-byte store
        const bool wide = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ldo % E == 0;
#pragma unroll
        for (int i = 0; i < C::ACC; i += E) {
          alignas(16) O v[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float w = __shfl_sync(0xffffffffu, ws[(i + e) % 4], (i + e) / 4);
            const float b = __shfl_sync(0xffffffffu, bias[(i + e) % 4], (i + e) / 4);
            v[e] = from_f32<O>(fmaf(static_cast<float>(acc[i + e]) * xs, w, b));
          }
          if (t < p.T) {
            if (wide && n + i + E <= end) {
              *reinterpret_cast<uint4*>(out + i) = *reinterpret_cast<const uint4*>(v);
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e)
                if (n + i + e < end) out[i + e] = v[e];
            }
          }
        }
      } else if (t < MT) {
        // every stage has been read: the rings take the sums, [channel][token]
        int* sums = reinterpret_cast<int*>(smem);
#pragma unroll
        for (int i = 0; i < C::ACC; ++i) sums[(half * C::ACC + i) * C::kSumRow + t] = acc[i];
      }
    }
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    cta_barrier();
  } else {
    // ---- int8 to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    const int ctid = (tid - C::kConvWarp0 * 32) % (C::kGroupWarps * 32);
    const int group = (warp - C::kConvWarp0) / C::kGroupWarps;
    Ring<C::S> r;
    Ring<C::S8> r8;
    r.next(group);
    r8.next(group);
    const int64_t mine = static_cast<int64_t>(steps) * ((tiles - tile0 + tile_step - 1) / tile_step);
    for (int64_t g = group; g < mine; g += C::kGroups, r.next(C::kGroups), r8.next(C::kGroups)) {
      if (C::kOperandFirst && !r.first && !wait(empty + 8 * r.stage, r.parity ^ 1)) break;
      if (!wait(full8 + 8 * r8.stage, r8.parity)) break;
      Weights<kThinN, C::kGroupWarps> w;
      w.load(base + C::kRing8 + r8.stage * C::W8, ctid, nw);
      if (!C::kOperandFirst && !r.first && !wait(empty + 8 * r.stage, r.parity ^ 1)) break;
      w.store(base + r.stage * (C::X + C::W) + C::X, ctid, nw);
      proxy_fence_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(fullw + 8 * r.stage);
        mbar_arrive(empty8 + 8 * r8.stage);   // not before the stores: the loads have then arrived for sure
      }
    }
    __syncwarp();
    cta_barrier();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  }

  __syncwarp();
  if (split > 1) {
    // the parts of one tile: each CTA adds its share of the channels, tokens
    // side by side as they lie in the other CTAs (a warp's remote reads are then
    // one line each), into [token][channel] behind the sums, and stores those
    cluster_sync();
    if (!*abort) {
      const int share = nw / split, c0 = share * part;   // nw is a multiple of 32, split at most 8
      int* rows = reinterpret_cast<int*>(smem) + kThinN * C::kSumRow;
      constexpr int U = 4;   // with four parts each: 16 reads in flight together
      for (int i0 = tid; i0 < share * MT; i0 += U * C::kThreads) {
        int sum[U] = {};
        for (int r0 = 0; r0 < split; r0 += 4) {
          int v[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * C::kThreads, share * MT - 1);
            const uint32_t at = base + ((c0 + i / MT) * C::kSumRow + i % MT) * 4;
#pragma unroll
            for (int r = 0; r < 4; ++r) v[u][r] = r0 + r < split ? ld_cluster1(at, r0 + r) : 0;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) sum[u] += v[u][0] + v[u][1] + v[u][2] + v[u][3];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * C::kThreads;
          if (i < share * MT) rows[(i % MT) * (share + 1) + i / MT] = sum[u];
        }
      }
      __syncthreads();
      const int c = tid % share, n = tile0 * nw + c0 + c, t_step = C::kThreads / share;   // a thread keeps its channel
      if (n < p.N && tid < t_step * share) {
        const float ws = __ldg(p.ws + n), bias = p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n]) : 0.f;
#pragma unroll 4
        for (int t = tid / share; t < p.T; t += t_step)
          store_out<O>(p, t, n, rows[t * (share + 1) + c], __ldg(p.xs + t), ws, bias);
      }
    }
    cluster_sync();   // nothing of this CTA is read any more
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
}

// Tokens as fp16, [T][kp] with kp a multiple of 64, zero past K.
__global__ void __launch_bounds__(256) k_widen(const int8_t* x, int64_t ldx, int T, int K, int kp, __half* out) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int per = kp / 16;
  for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < static_cast<int64_t>(T) * per; i += gridDim.x * 256) {
    const int64_t t = i / per;
    const int k = static_cast<int>(i - t * per) * 16;
    const int8_t* from = x + t * ldx + k;
    const uint4 v = k + 16 <= K ? __ldg(reinterpret_cast<const uint4*>(from)) : load_tail(from, K - k);
    uint32_t h[8];
    to_f16x16(v, h);
    uint4* to = reinterpret_cast<uint4*>(out + t * kp + k);
    to[0] = make_uint4(h[0], h[1], h[2], h[3]);
    to[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// Boxes of kBK columns x box rows of an int8 (size 1) or fp16 (2) matrix of
// stride ld bytes; columns and rows past its ends read as zero.
cudaError_t map_tile(CUtensorMap* m, int size, const void* base, int64_t ld, int rows, int cols, int box) {
  const auto encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t boxes[2] = {kBK, static_cast<cuuint32_t>(box)};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = encode(m, size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                            const_cast<void*>(base), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            size == 1 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int padded_k(int K) { return (K + 63) & ~63; }

// What a tensor-core kernel's launches need to know about a device, asked once.
struct OnDevice {
  std::atomic<bool> ready{false};
  int clusters[4] = {};   // of 1, 2, 4 and 8 CTAs, at once
};
template <typename K>
cudaError_t prepare(OnDevice* all, K* kernel, int threads, int smem, OnDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  OnDevice& d = all[dev];
  if (!d.ready.load(std::memory_order_acquire)) {
    static std::mutex asking;
    const std::lock_guard<std::mutex> lock(asking);
    *out = &d;
    if (d.ready.load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes at{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    // the register split must be what the CTA is launched with
    if (at.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    for (int i = 0; i < 4; ++i) d.clusters[i] = max_clusters(kernel, threads, smem, 1 << i);
    d.ready.store(true, std::memory_order_release);
  }
  *out = &d;
  return cudaSuccess;
}

cudaError_t widen(const LinArgs& p, void* ws, cudaStream_t s) {
  const int kp = padded_k(p.K);
  const int64_t chunks = static_cast<int64_t>(p.T) * (kp / 16);
  k_widen<<<static_cast<unsigned>(std::min<int64_t>((chunks + 255) / 256, sm_count() * 8)), 256, 0, s>>>(
      p.x, p.ldx, p.T, p.K, kp, static_cast<__half*>(ws));
  return cudaGetLastError();
}

// A launch in clusters that may start while k_widen runs: only its token loads
// wait for k_widen, which itself started after everything before it had ended.
template <typename... P, typename... A>
cudaError_t launch_after_widen(void (*kernel)(P...), unsigned grid, int threads, int smem, int cluster, cudaStream_t s,
                               A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute a[2]{};
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  a[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Parts of K, up to 2^most: while all of them still run at once (clusters of 8
// fit a processing cluster's SMs less often than their number says, and a
// second turn costs as much as the first) and have eight stages or more each.
int parts_of_k(const OnDevice& d, int64_t tiles, int steps, int first, int most) {
  int i = 0;
  while (i < most && tiles <= d.clusters[first + i + 1] && steps >= 16 << i) ++i;
  return 1 << i;
}

template <typename O>
cudaError_t launch_tc(const LinArgs& p, void* ws, cudaStream_t s) {
  using C = Tile;
  static OnDevice all[kMaxDev];
  OnDevice* d;
  cudaError_t e = prepare(all, k_tc<O>, C::kThreads, C::kSmem, &d);
  CUtensorMap mapw, mapx;
  // tokens of a tile, about the same for all and a multiple of the 32 that a
  // pair's MMA takes: 333 are 192 and 141, not 256 and 77 (300 x 4096 x 4096: 22.0
  // and 23.6 us; 260 x 28672 x 4096: 74.4 and 77.1)
  const int ntt = (p.T + C::NT - 1) / C::NT, nt = ((p.T + ntt - 1) / ntt + 31) / 32 * 32;
  const int kp = padded_k(p.K);
  if (e == cudaSuccess) e = map_tile(&mapw, 1, p.w, p.ldw, p.N, p.K, kM);
  if (e == cudaSuccess) e = map_tile(&mapx, 2, ws, kp * int64_t{2}, p.T, kp, nt / 2);
  if (e == cudaSuccess) e = widen(p, ws, s);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.N + 2 * kM - 1) / (2 * kM)) * ntt;
  const int split = parts_of_k(*d, tiles, (p.K + kBK - 1) / kBK, 1, 2);
  const int64_t pairs = split > 1 ? tiles * split : std::min<int64_t>(tiles, sm_count() / 2);
  return launch_after_widen(k_tc<O>, static_cast<unsigned>(2 * pairs), C::kThreads, C::kSmem, 2 * split, s, p,
                            mapw, mapx, nt, split);
}

template <typename O, int MT>
cudaError_t launch_thin(const LinArgs& p, void* ws, cudaStream_t s) {
  using C = Thin<MT>;
  static OnDevice all[kMaxDev];
  OnDevice* d;
  cudaError_t e = prepare(all, k_thin<O, MT>, C::kThreads, C::kSmem, &d);
  if (e != cudaSuccess) return e;
  const int kp = padded_k(p.K), steps = (p.K + kBK - 1) / kBK, box = (p.T + 7) / 8 * 8;
  // channels of a tile: what gives the SMs the least to do in turn, a stage's
  // time being some constant and a part that grows with them.  64 x 28672 x 4096:
  // 42.1 us with 256 (112 tiles), 39.0 with 192 (150), 58 with 128 (two turns);
  // 32 x 131072 x 4096: 125, 135 and, with the 224 of the rule, 119; 128 x 4096 x
  // 14336: 43.3, 39.4 and, K split over more CTAs with 128, 34.8
  int nw = kThinN, split = 1;
  float least = 0.f;
  for (int n = kThinN; n >= kThinN / 2; n -= 32) {
    const int tiles = (p.N + n - 1) / n, parts = parts_of_k(*d, tiles, steps, 0, 3);
    const int turns = (tiles + sm_count() - 1) / sm_count();   // one where K is split
    const float cost = static_cast<float>(turns * (n + 64)) / parts;
    if (n == kThinN || cost < least) nw = n, split = parts, least = cost;
  }
  CUtensorMap mapw, mapx;
  e = map_tile(&mapw, 1, p.w, p.ldw, p.N, p.K, nw);
  if (e == cudaSuccess) e = map_tile(&mapx, 2, ws, kp * int64_t{2}, p.T, kp, box);
  if (e == cudaSuccess) e = widen(p, ws, s);
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + nw - 1) / nw;
  return launch_after_widen(k_thin<O, MT>, static_cast<unsigned>(split > 1 ? tiles * split : std::min(tiles, sm_count())),
                            C::kThreads, C::kSmem, split, s, p, mapw, mapx, box, nw, split);
}

template <typename O>
cudaError_t launch_linear(const LinArgs& p, void* ws, cudaStream_t s) {
  // Few tokens, or little to do (k_few in blocks of tokens): in blocks of 8 as long
  // as one wave of CTAs holds them, N = 60, K = 4096: 64 tokens 3.7 us and 13.6 by
  // the tensor-core kernels, 256 tokens 3.8 and 18; 16 x 3600 in two blocks 7.5 and
  // 6.6 in one.  Then in blocks of 32, K = 4096: 64 x 2048 9.4 and 16.7, 64 x 4096
  // 15.6 and 17.9, 2048 x 60 10.4 and 22.6, 64 x 8192 26.9 and 22.1; K = 14336:
  // 64 x 2048 21.7 and 24.2, 64 x 4096 41 and 33; K = 2048: 128 x 4096 16.8 and 17.0.
  const int64_t blocks = int64_t{(p.N + 15) / 16} * ((p.T + 7) / 8);
  if (p.T <= 8 || blocks <= sm_count() * (p.T <= kFewTokens ? 2 : 3)) return launch_few_nt<O, 1, false>(p, s);
  if (p.T <= kFewTokens || (p.T <= 32 && p.N < kManyChannels)) return launch_few<O>(p, s);
  if (p.T > 32 && (blocks <= sm_count() * 7 || (blocks <= 4096 && blocks * p.K <= 1 << 23)))
    return launch_few_nt<O, 4, true>(p, s);
  if (p.T <= 32) return launch_thin<O, 32>(p, ws, s);
  if (p.T <= 64) return launch_thin<O, 64>(p, ws, s);
  if (p.T <= 128) return launch_thin<O, 128>(p, ws, s);
  return launch_tc<O>(p, ws, s);
}

// By the tokens alone, so that one workspace serves a model's products of any N; the
// calls above kFewTokens that k_few takes leave it untouched.
size_t linear_ws_bytes(int T, int K) {
  return T <= kFewTokens ? 0 : static_cast<size_t>(T) * padded_k(K) * 2;
}

}  // namespace

int sm_count() {
  static std::atomic<int> n[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 1;
  int v = n[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) v = 1;
    n[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

}  // namespace pw

extern "C" {

size_t pw_linear_i8_workspace_bytes(int T, int K) {
  return T < 0 || K < 1 || K > PW_MAX_K_I8 ? 0 : pw::linear_ws_bytes(T, K);
}

int pw_linear_i8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w, int64_t ldw,
                 const float* w_scale, const void* bias, int T, int N, int K, int out_dtype, void* out, int64_t ldo,
                 void* workspace, size_t ws_bytes, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_linear_i8");
  if (T < 0 || T > PW_MAX_VOCAB || N < 1 || N > PW_MAX_VOCAB || K < 1 || K > PW_MAX_K_I8)
    return pw::failf(PW_EINVAL, "pw_linear_i8: need 0 <= T <= %d, 1 <= N <= %d, 1 <= K <= %d (T %d, N %d, K %d)",
                     PW_MAX_VOCAB, PW_MAX_VOCAB, PW_MAX_K_I8, T, N, K);
  if (!pw::dtype_ok(out_dtype)) return pw::failf(PW_EINVAL, "pw_linear_i8: unknown out_dtype %d", out_dtype);
  if (T == 0) return PW_OK;
  if (!x || !x_scale || !w || !w_scale || !out) return pw::failf(PW_EINVAL, "pw_linear_i8: null x, w, scales or out");
  if (ldx < K || ldw < K || ldo < N)
    return pw::failf(PW_EINVAL, "pw_linear_i8: a row stride is below its row (K = %d, N = %d)", K, N);
  if (!pw::aligned(x, 16) || !pw::aligned(w, 16) || ldx % 16 || ldw % 16)
    return pw::failf(PW_EINVAL, "pw_linear_i8: rows of x and w must start on 16-byte boundaries");
  const size_t es = pw::dtype_bytes(out_dtype);
  if (!pw::aligned(out, es) || !pw::aligned(bias, es) || !pw::aligned(x_scale, 4) || !pw::aligned(w_scale, 4))
    return pw::failf(PW_EINVAL, "pw_linear_i8: misaligned pointer");
  const size_t need = pw::linear_ws_bytes(T, K);
  if (ws_bytes < need || (need && !workspace))
    return pw::failf(PW_ENOMEM, "pw_linear_i8: workspace of %zu bytes, %zu are needed", workspace ? ws_bytes : 0, need);
  if (need && !pw::aligned(workspace, 256))
    return pw::failf(PW_EINVAL, "pw_linear_i8: the workspace must be 256-byte aligned");
  const pw::LinArgs a{x, w, x_scale, w_scale, bias, out, ldx, ldw, ldo, T, N, K};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = out_dtype == PW_F16    ? pw::launch_linear<__half>(a, workspace, st)
                        : out_dtype == PW_BF16 ? pw::launch_linear<__nv_bfloat16>(a, workspace, st)
                                               : pw::launch_linear<float>(a, workspace, st);
  return pw::launch_status(e, "pw_linear_i8");
}

int pw_linear_i8_status(pw_stream_t s, int* status) {
  pw::NvtxCall nvtx_range("pw_linear_i8_status");
  if (!status) return pw::failf(PW_EINVAL, "pw_linear_i8_status: null status");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  uint32_t now = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= pw::kMaxDev)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(&now, pw::g_linear_timeouts, sizeof now, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return pw::failf(PW_ECUDA, "pw_linear_i8_status: %s", cudaGetErrorString(e));
  // the count up to which an earlier call has told; another thread may tell meanwhile
  static std::atomic<uint32_t> told[pw::kMaxDev];
  uint32_t before = told[dev].load();
  bool more = false;
  while ((more = static_cast<int32_t>(now - before) > 0) && !told[dev].compare_exchange_weak(before, now)) {
  }
  *status = more ? PW_STATUS_TIMEOUT : 0;
  return PW_OK;
}

int pw_debug_linear_timeout(pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_debug_linear_timeout");
  pw::k_count_timeout<<<1, 1, 0, reinterpret_cast<cudaStream_t>(s)>>>();
  return pw::launch_status(cudaGetLastError(), "pw_debug_linear_timeout");
}

}  // extern "C"
