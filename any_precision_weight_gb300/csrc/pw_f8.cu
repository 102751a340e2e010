// Products in 8-bit floating point (e4m3) with a scale for each block of 128
// (pw_linear_f8), and the same for rows sorted by expert (pw_grouped_linear_f8):
//
//   out[t][n] = sum_b xs[t][b] ws[n / 128][b] sum_{k in b} x[t][k] w[n][k] + bias[n]
//
// with b the blocks of 128 columns of K.  Products of two e4m3 numbers are exact in
// fp32; the sums of a block and the sum over blocks are fp32.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "pw_rows.cuh"
#include "pw_tc.cuh"

namespace pw {
namespace {

constexpr int kMaxDev = 64;
constexpr int kB = 128;   // columns of K, and channels, that share a scale

struct F8Args {
  const uint8_t* x;
  const uint8_t* w;
  const float* xs;
  const float* ws;
  const void* bias;
  const int32_t* offsets;   // rows of group e: [offsets[e], offsets[e + 1]); NULL: one group of all rows
  void* out;
  int64_t ldx, ldxs, ldw, ldws, ldo;
  int64_t gw, gws;          // from a group's weights and scales to the next one's
  int T, N, K, E;
};

// Offsets come from the device: one outside [0, T] is cut to it.  Where they descend the
// rows between are some group's, or several groups' after another; k_tc_f8, whose tiles are
// counted, takes the largest so far.  (To look for that in k_few_f8 too takes 2 us.)
__device__ __forceinline__ int offset_in(const F8Args& p, int i) { return min(max(__ldg(p.offsets + i), 0), p.T); }

// Rows of a group.
struct Rows {
  int begin, end;
};
__device__ __forceinline__ Rows rows_of(const F8Args& p, int e) {
  if (!p.offsets) return {0, p.T};
  const int begin = offset_in(p, e);
  return {begin, max(begin, offset_in(p, e + 1))};
}

// ---------------------------------------------------------------- few rows

// The first n of 16 bytes at p, the others zero.
__device__ __forceinline__ uint4 load_tail(const uint8_t* p, int n) {
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) v[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Weights are read once: past the L1, which keeps the rows.
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// D += A B, fp16 16 x 16 by 16 x 8, fp32.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sixteen e4m3 numbers as fp16 pairs (exact).
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
__device__ __forceinline__ void widen16(const uint4& v, uint32_t (&h)[8]) {
  widen4(v.x, h[0], h[1]);
  widen4(v.y, h[2], h[3]);
  widen4(v.z, h[4], h[5]);
  widen4(v.w, h[6], h[7]);
}

constexpr int kFewWarps = 8;
constexpr int kFewCtas = 2;   // of an SM

// A group of kw warps owns 16 channels and shares out the blocks of K; blockIdx.y is an
// expert and one of `turns` that share its rows, 8 NT at a time.  Lane (g, q) =
// (lane / 4, lane % 4) loads the 16 bytes at column 16 q of channels g and g + 8, and of
// row g of every 8: the operand registers of its products, with the columns of K in an
// order of their own that both operands share.  So the weights go from memory to the
// tensor cores through registers alone.  Each block's sums are scaled into fp32 sums.
// The weights' bytes bound it: 1 x 28672 x 4096 takes 22.7 us, 5.2 TB/s or 76 % of a copy's
// rate (registers hold no more loads in flight than four blocks of two CTAs; 2 us and more are
// the launch, the first loads and the sums over the warps).  The products, at most 16 rows,
// take a fifth of the tensor cores' time.
template <typename O, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, kFewCtas) k_few_f8(const F8Args p, int kw, int turns) {
  constexpr int kRow = NT * 8 + 1;   // padded against bank conflicts
  __shared__ float s_part[kFewWarps][16 * kRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int groups = kFewWarps / kw, turn = warp % kw;
  const int e = blockIdx.y / turns;
  after_those_before();
  const Rows rows = rows_of(p, e);
  const int n0 = (blockIdx.x * groups + warp / kw) * 16;
  const int blocks = (p.K + kB - 1) / kB, whole = p.K / kB;
  const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * turn / kw);
  const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (turn + 1) / kw);
  const uint8_t* w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = p.w + e * p.gw + min(n0 + g + 8 * i, p.N - 1) * p.ldw + q * 16;
  const float* ws = p.ws + e * p.gws + min(n0, p.N - 1) / kB * p.ldws;
  const O* bias = p.bias ? static_cast<const O*>(p.bias) + static_cast<int64_t>(e) * p.N : nullptr;

  for (int t0 = rows.begin + blockIdx.y % turns * (NT * 8); t0 < rows.end; t0 += turns * (NT * 8)) {
    const int T = min(rows.end - t0, NT * 8);
    const uint8_t* x[NT];
    const float* xs[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      x[j] = p.x + (t0 + min(j * 8 + g, T - 1)) * p.ldx + q * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) xs[j][i] = p.xs + (t0 + min(j * 8 + q * 2 + i, T - 1)) * p.ldxs;
    }
    float acc[NT][4] = {};
    // the block b: two runs of 64 columns, 16 of them to a lane
    struct Part {
      uint4 a[2][2], v[2][NT];
      float s, f[NT][2];
    };
    auto scales = [&](Part& m, int b) {
      m.s = __ldg(ws + b);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) m.f[j][i] = __ldg(xs[j][i] + b);
    };
    auto add = [&](const Part& m) {
      float part[NT][4] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t ha[2][8];
        widen16(m.a[u][0], ha[0]);
        widen16(m.a[u][1], ha[1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t hx[8];
          widen16(m.v[u][j], hx);
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            mma_16816(part[j], ha[0][i], ha[1][i], ha[0][i + 1], ha[1][i + 1], hx[i], hx[i + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float s0 = m.f[j][0] * m.s, s1 = m.f[j][1] * m.s;
        acc[j][0] = fmaf(part[j][0], s0, acc[j][0]);
        acc[j][1] = fmaf(part[j][1], s1, acc[j][1]);
        acc[j][2] = fmaf(part[j][2], s0, acc[j][2]);
        acc[j][3] = fmaf(part[j][3], s1, acc[j][3]);
      }
    };
    auto fetch = [&](Part& m, int b) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) m.a[u][i] = load_once(w[i] + b * kB + u * 64);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < NT; ++j) m.v[u][j] = __ldg(reinterpret_cast<const uint4*>(x[j] + b * kB + u * 64));
      scales(m, b);
    };
    const int end = min(b1, whole);
    int b = b0;
    // blocks whose loads are in flight together
    auto together = [&](auto n) {
      for (; b + n.value <= end; b += n.value) {
        Part m[n.value];
#pragma unroll
        for (int u = 0; u < n.value; ++u) fetch(m[u], b + u);
#pragma unroll
        for (int u = 0; u < n.value; ++u) add(m[u]);
      }
    };
    if constexpr (NT == 1) {
      together(std::integral_constant<int, 4>());
      together(std::integral_constant<int, 2>());
    }
    together(std::integral_constant<int, 1>());
    if (end < b1) {   // the last block, not whole
      Part m;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = end * kB + u * 64, left = p.K - at - q * 16;
        auto part = [&](const uint8_t* from) {
          return left >= 16 ? __ldg(reinterpret_cast<const uint4*>(from + at)) : load_tail(from + at, left);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) m.a[u][i] = part(w[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) m.v[u][j] = part(x[j]);
      }
      scales(m, end);
      add(m);
    }
    // acc[j][0..3]: channels g, g, g + 8, g + 8; rows 8 j + 2 q + 0, 1, 0, 1
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_part[warp][(g + (i >> 1) * 8) * kRow + j * 8 + q * 2 + (i & 1)] = acc[j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < groups * 16 * T; i += kFewWarps * 32) {
      const int c = i % (groups * 16), t = i / (groups * 16);
      const int n = blockIdx.x * groups * 16 + c;
      if (n >= p.N) continue;
      float sum = 0.f;
      for (int j = 0; j < kw; ++j) sum += s_part[c / 16 * kw + j][c % 16 * kRow + t];
      if (bias) sum += to_f32<O>(bias[n]);
      static_cast<O*>(p.out)[(t0 + t) * p.ldo + n] = from_f32<O>(sum);
    }
    __syncthreads();   // s_part has been read
  }
}

// The launch: blocks of 8 rows as long as about one wave of CTAs holds them, then of 16, which
// read the weights half as often (64 x 1024 x 4096 7.4 and 6.2 us, 256 x 60 x 4096 3.9 and
// 4.5); `turns`, from the average group's rows, and kw as in the kernel.  A larger group's rows go
// through its `turns` CTAs one pass after another, and each pass reads the weights again: 256 rows by
// 128 experts of 2048 x 1408 take 50 us in groups that differ as a router's do, 104 with half of
// the rows in one group, 198 with all in one (k_tc_f8 60, 58 and 12; twice or four times the turns
// cost the even ones a tenth).
// `cost`, to compare with k_tc_f8, in ns: 1000, and for each wave of CTAs 2000 (half more where a
// row ends inside 16 bytes) and 500 for a block of K, 1.4 times both for 16 rows at a time.
// How many groups have rows is not known here.  kw takes 0.6 T up to T = E and 0.6 E + 0.1 T (at
// most E) above; `cost` takes max(min(E, T), T / M + E / 2) passes, and with more rows than groups
// 1.75 waves at least; plan_of takes T / M + E / 2 tiles.  256 rows by 60 groups: 60, 60 and 38,
// where 49 have rows if the shares are uniform over the simplex.  Each was fitted where it is
// used, over sizes drawn at random, and none is an estimate for the others.
struct Few {
  int nt, turns, kw;
  double cost;
};
Few few_of(const F8Args& p) {
  Few f{};
  const int groups = (p.N + 15) / 16, blocks = (p.K + kB - 1) / kB, slots = sm_count() * kFewCtas;
  const int64_t rows = p.offsets ? (p.T + p.E - 1) / p.E : p.T;   // of a group, about
  f.nt = rows <= 8 || groups * ((rows + 7) / 8) <= slots ? 1 : 2;
  const int M = f.nt * 8;
  f.turns = static_cast<int>(std::min<int64_t>((rows + M - 1) / M, 65535 / p.E));
  double least = 0.;
  for (int n = 1, i = 0; n <= kFewWarps && (n == 1 || blocks >= n); n *= 2, ++i) {
    double cost;
    if (p.offsets) {
      // some experts have no rows: their CTAs end at once, and the others may be less than a
      // wave, or end with half of one.  2 rows by 8 experts of 4096 x 14336 with kw 1, 2, 4, 8:
      // 40.4, 24.7, 16.5, 14.4 us; of 28672 x 4096 24.9, 26.9, 33.2, 46.5; 16 rows by 60 of 2048 x
      // 1408 11.7, 13.1, 16.7, 24.1; 64 by 128 of 1024 x 4096 40.4, 35.0, 37.0, 47.6
      const double wave = static_cast<double>((groups * n + kFewWarps - 1) / kFewWarps) / slots;
      const double in = p.T <= p.E ? 0.6 * p.T : std::min<double>(p.E, 0.6 * p.E + 0.1 * p.T);
      const double busy = wave * in, idle = std::max(0., wave * p.E * f.turns - busy);
      cost = (busy > 1 ? busy + 0.5 : 1.) * (1000 + 400 * ((blocks + n - 1) / n)) + 650 * idle;
    } else {   // how full the waves are, and what the sums over the warps add
      const double waves = static_cast<double>(groups) * f.turns * n / (kFewWarps * slots);
      cost = std::ceil(waves) / waves * (1. + 0.06 * i);
    }
    if (n == 1 || cost < least) f.kw = n, least = cost;
  }
  const double in = p.offsets ? std::max<double>(std::min(p.E, p.T), p.T / M + p.E / 2) : (p.T + M - 1) / M;
  const double waves = std::max((groups * f.kw + kFewWarps - 1) / kFewWarps * in / slots, p.T > p.E && p.offsets ? 1.75 : 1.);
  f.cost = 1000 + waves * (f.nt == 2 ? 1.4 : 1.) * (2000 * (p.K % 16 ? 1.5 : 1.) + 500 * ((blocks + f.kw - 1) / f.kw));
  return f;
}
template <typename O, int NT>
cudaError_t launch_few(const F8Args& p, const Few& f, cudaStream_t s) {
  const int groups = (p.N + 15) / 16, per = kFewWarps / f.kw;
  return launch_close(k_few_f8<O, NT>, dim3((groups + per - 1) / per, static_cast<unsigned>(p.E * f.turns)), kFewWarps * 32, 0,
                      1, s, p, f.kw, f.turns);
}

// ---------------------------------------------------------------- tensor cores

// One CTA to an SM takes tiles of 128 rows (M) x up to 256 channels (N), a pair of CTAs
// (cta_group::2) tiles of 256 rows, with tcgen05.mma kind::f8f6f4.  Each block of 128
// columns of K goes into an accumulator of its own in tensor memory, of two or four that
// take turns, and from there scaled into fp32 registers.  A lane of tensor memory is a row,
// so 64 channels (half a block of the weights' scales) take one factor to a thread.
// Warps by role:
//  * warp 0 fetches rows and weights by TMA into a ring of stages (128 columns each);
//  * warp 1 issues the MMAs (of a pair in the even CTA, for both; in the odd one it
//    reports its loads to the even one);
//  * warps 2 and 3 write a block's scales into a ring of SS and report them with the loads
//    of the block: an MMA that has ended says that its block's scales are there, and one
//    that starts, that those of the block that had its accumulator before have been read;
//  * warps 4.. scale each finished accumulator into their sums while the next ones fill,
//    and at the tile's end store.
// Where there are few tiles a cluster splits K and adds the parts through distributed
// shared memory, in the order of the parts.
// 2048 x 28672 x 4096 takes 194 us, 2475 TFLOP/s (206 to 212 a call among others).  A pair's MMAs of
// a block take 512 clocks, and its accumulators' way from tensor memory through two warps of each
// scheduler (read, wait, 256 x 128 multiply-adds of a CTA) some 1150, the tensor cores busy for half
// of them.  (The power cap, 1385 of 1400 W, takes 4 % of the clock.)  To sum over K in tensor memory
// alone has no place for the blocks' scales.  64 x 28672 x 4096 takes 25.9 us, 4.5 TB/s of weights;
// small products 9 us, of which 5 are the tensor memory, the barriers, the first tiles and the sums'
// way out.
constexpr int kM = 128;          // rows of a CTA
constexpr int kEpiWarp0 = 4;

struct Tc {
  static constexpr int NT = 256;                          // most channels of a tile
  static constexpr int EW = 8;                            // accumulating warps
  static constexpr int ACC = NT / (EW / 4);               // sums of one of their threads
  static constexpr int kThreads = 32 * (kEpiWarp0 + EW);
  static constexpr int kRing = 184 * 1024;                // bytes of the stages
  static constexpr int S = 8;                             // most of them
  static constexpr int D = 4;                             // most accumulators
  static constexpr int kPiece = 32 * 128;                 // what a warp stores at a time: 32 rows x 32 channels
  static constexpr int SS = 12;
  static constexpr int kScale = kM + 4;                   // floats: the rows', and one for each 64 channels
  static constexpr int kOffOut = kRing;
  static constexpr int kOffScale = kOffOut + EW * kPiece;
  static constexpr int kOffBar = kOffScale + SS * kScale * 4;
  static constexpr int kBars = 2 * S + 2 * D + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;    // tmem, abort, first tile and row of each group
  static constexpr int kSmem = kOffMisc + 16 + 2 * 4 * (PW_MAX_GROUPS + 1);
  static constexpr uint32_t kCols = 512;                  // of tensor memory
  static constexpr int kSumPad = 4;                       // floats behind a row's sums in the ring
  static_assert(kOffBar % 8 == 0 && kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(SS >= S + D, "the scales of a block that may be fetched have been read");
  static_assert(kM * (NT + kSumPad) * 4 <= kRing, "a CTA's sums fit the ring");
};

// What a launch chose: CTAs to a tile, rows of it (of a CTA's part: 128, or fewer in a CTA alone),
// channels of it (a multiple of 64) and parts of K; and what follows: bytes of a stage's
// rows and of the stage, stages, accumulators.
struct Plan {
  int ctas, rows, nw, split, x_bytes, stage, stages, accs;
  float cost;   // ns of the tiles, about
};

// Registers by role: 384 threads are launched with kRegsLaunch each, and the
// accumulating ones hold 128 sums.  Every role returns to kRegsLaunch at its end, the
// accumulating warps before a CTA barrier and the others after it.
constexpr int kRegsLaunch = 168, kRegsIssue = 72, kRegsAcc = 216;
static_assert(128 * (kRegsIssue + 2 * kRegsAcc) <= Tc::kThreads * kRegsLaunch, "register split");

// Bounded waits of the kernel that gave up (pw_linear_f8_status).
__device__ uint32_t g_f8_timeouts;
__global__ void k_count_timeout() { atomicAdd(&g_f8_timeouts, 1u); }

// Waits for the phase of the given parity, up to a second; false, and the abort flag, when
// that has passed or another thread has raised it.  (With test_wait in the place of try_wait,
// whose threads sleep, the polls of the warps keep one another and the arrivals waiting: 2048
// x 28672 x 4096 203 and 193 us.)
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (try_wait(bar, parity)) return true;
  const uint64_t start = now_ns();
  while (!try_wait(bar, parity)) {
    if (*abort) return false;
    if (now_ns() - start > 1000000000ull) {
      atomicAdd(&g_f8_timeouts, 1u);
      *abort = 1;
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// What a CTA alone and a pair do differently.
template <int CTAS> struct Cta;
template <> struct Cta<1> {
  static __device__ __forceinline__ void alloc(uint32_t to) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(Tc::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  static __device__ __forceinline__ void dealloc(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Tc::kCols));
  }
  // 32 columns of K
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  }
  static __device__ __forceinline__ void commit(uint32_t bar, uint32_t) { mma_commit(bar); }
};
template <> struct Cta<2> {
  static __device__ __forceinline__ void alloc(uint32_t to) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(Tc::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  static __device__ __forceinline__ void dealloc(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Tc::kCols));
  }
  static __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  }
  static __device__ __forceinline__ void commit(uint32_t bar, uint32_t leader) {
    commit_pair(bar, static_cast<uint16_t>(3u << leader));
  }
};
// D f32, A and B e4m3, N / 8 and M / 16.
__host__ __device__ constexpr uint32_t idesc_of(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// 32 consecutive fp32 columns of this thread's TMEM lane (after tmem_wait32).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ float lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Tensor maps: rows in boxes of 128, 64, 32 and 16, weights in boxes of a CTA's channels,
// outputs in boxes of 32 rows x 32 channels.
struct Maps {
  CUtensorMap x[4], w, out;
};

// A position in a ring of a size known at run time.
struct Turn {
  uint32_t stage = 0, parity = 0;
  bool first = true;   // no stage has been used before
  __device__ __forceinline__ void next(uint32_t n) {
    if (++stage == n) stage = 0, parity ^= 1, first = false;
  }
};

// A tile: its group, rows [t0, t1) and first channel.
struct Tile {
  int e, t0, t1, n0;
  // Of a pair whose tile is of 256 channels: at most 128 rows, 64 to a CTA.
  __device__ __forceinline__ bool half() const { return t1 - t0 <= kM; }
};

// The tiles in order of the groups, `start` the first of each and `off` its rows' first;
// within a group bands of kBand row tiles, so that CTAs at work share operands in the L2.  A
// CTA takes every `step`th; from one to its next a band's row tiles go round by one, so that
// the last of a group, which may have fewer rows, falls to all CTAs alike.
constexpr int kBand = 8;
struct Tiles {
  const int *start, *off;
  int ntn, M, nw, step, e = 0;
  template <bool HALF>
  __device__ __forceinline__ Tile at(int tile) {
    while (tile >= start[e + 1]) ++e;
    const int begin = off[e], end = off[e + 1];
    const int local = tile - start[e], band = local / (kBand * ntn), rest = local - band * kBand * ntn;
    const int width = min(kBand, (end - begin + M - 1) / M - band * kBand);
    const int column = rest / width, row = rest - column * width;
    const int less = (end - begin) % M;   // rows of the group's last tile, or none
    const int round = HALF && less && less <= M / 2 ? column * width / step * ((width + 1 - step % width) % width) : 0;
    const int t0 = begin + (band * kBand + (row + round) % width) * M;
    return {e, t0, min(end, t0 + M), column * nw};
  }
};

// The first row and the first tile of each group, and behind them the ends, by one warp.
__device__ __forceinline__ void first_tiles(const F8Args& p, int ntn, int M, int* start, int* off) {
  const int lane = threadIdx.x & 31;
  int before = 0, begin = p.offsets ? offset_in(p, 0) : 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const bool in = e0 + lane < p.E;
    int end = !in ? 0 : p.offsets ? offset_in(p, e0 + lane + 1) : p.T;   // then the largest up to here
    end = max(end, begin);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end = max(end, v);
    }
    const int last = __shfl_up_sync(0xffffffffu, end, 1), mine = lane ? last : begin;
    const int n = in ? (end - mine + M - 1) / M * ntn : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (in) start[e0 + lane] = before + sum - n, off[e0 + lane] = mine;
    before += __shfl_sync(0xffffffffu, sum, 31);
    begin = __shfl_sync(0xffffffffu, end, 31);
  }
  if (lane == 0) start[p.E] = before, off[p.E] = begin;
}

// FULL: tiles of 256 channels, where a thread's 128 are one block of the weights' scales, and
// K whole.  HALF: the same, but that of a pair's tile of at most 128 rows each CTA takes 64,
// in 0.75 of the time: 4096 rows by 8 experts of 28672 x 4096 take 495 us, without 512, 2048
// rows 288 and 311 (by single CTAs); 300 x 28672 x 4096 51.5 and 55.  (Its choice in every pair
// costs 2048 x 28672 x 4096 5 us, so it is a kernel of its own.)
template <typename O, int CTAS, bool FULL, bool HALF>
__global__ void __launch_bounds__(Tc::kThreads, 1)
k_tc_f8(const F8Args p, const __grid_constant__ Maps maps, const Plan plan, int bulk) {
  using C = Tc;
  using G = Cta<CTAS>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t base = saddr(smem);
  if (base % 1024) {   // the swizzled tiles would lie wrong (the array is aligned, so it never is)
    if (threadIdx.x == 0) atomicAdd(&g_f8_timeouts, 1u);
    return;
  }
  const uint32_t full = base + C::kOffBar, empty = full + 8 * C::S;
  const uint32_t dfull = empty + 8 * C::S, dempty = dfull + 8 * C::D, fin = dempty + 8 * C::D;
  int* s_misc = reinterpret_cast<int*>(smem + C::kOffMisc);   // tmem, abort
  int *s_start = s_misc + 4, *s_off = s_start + PW_MAX_GROUPS + 1;
  volatile int* abort = s_misc + 1;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // the compiler then knows that it is uniform
  // the CTA's place: in its pair, and among the parts of K
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int side = static_cast<int>(rank % CTAS), part = static_cast<int>(rank / CTAS);
  const uint32_t leader = rank - side;
  const int nw = FULL ? C::NT : plan.nw, split = FULL ? 1 : plan.split, ntn = (p.N + nw - 1) / nw;
  const uint32_t accs = FULL ? C::kCols / C::NT : plan.accs, acc_cols = C::kCols / accs;

  if (tid == 96) {   // a map's first use otherwise waits for it
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.w)) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.x[i])) : "memory");
  }
  if (warp == 1) G::alloc(saddr(s_misc));
  if (tid == 0) {
    for (int i = 0; i < C::S; ++i) {
      // the CTA's loads, its scales by two warps, and the odd CTA's report
      mbar_init(full + 8 * i, CTAS == 2 && side == 0 ? 4 : 3);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < C::D; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, CTAS * C::EW);
    mbar_init(fin, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_misc[1] = 0;
  }
  after_those_before();
  if (warp == 2) first_tiles(p, ntn, CTAS * plan.rows, s_start, s_off);
  tc_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();   // the other CTA's barriers and tensor memory
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(s_misc[0]), 0);

  // (a look at a barrier takes 41 clocks by the whole warp, and 96 by one thread that
  // tells the others)
  auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, poll(bar, parity, abort)); };

  const int tiles = s_start[p.E], blocks = (p.K + kB - 1) / kB;
  const int s0 = static_cast<int>(static_cast<int64_t>(blocks) * part / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(blocks) * (part + 1) / split);
  const int tile0 = blockIdx.x / (CTAS * split), tile_step = gridDim.x / (CTAS * split);
  Tiles order{s_start, s_off, ntn, CTAS * plan.rows, nw, tile_step};

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {
      // ---- operands by TMA
      Turn r;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        const Tile t = order.template at<HALF>(tile);
        const bool half = HALF && t.half();
        const int t0 = t.t0 + side * (half ? kM / 2 : kM), rows = half ? min(t.t1 - t0, kM / 2) : t.t1 - t0, wn = nw / CTAS;
        const int box = rows > 64 ? 0 : rows > 32 ? 1 : rows > 16 ? 2 : 3;   // the least that holds the rows
        for (int k = s0; k < s1; ++k, r.next(plan.stages)) {
          if (!r.first && !(ok = poll(empty + 8 * r.stage, r.parity ^ 1, abort))) break;
          const uint32_t bar = full + 8 * r.stage, to = base + r.stage * plan.stage;
          mbar_expect_tx(bar, ((128 >> box) + wn) * kB);
          tma_load_2d(to, &maps.x[box], k * kB, t0, bar);
          tma_load_3d(to + plan.x_bytes, &maps.w, k * kB, t.n0 + side * wn, p.gw ? t.e : 0, bar);
        }
      }
      if (*abort) {   // what is in flight still ends before the CTA does
        volatile int none = 0;
        for (uint32_t i = 0; i < static_cast<uint32_t>(plan.stages); ++i) {
          if (i < r.stage)
            poll(full + 8 * i, r.parity, &none);
          else if (!r.first)
            poll(full + 8 * i, r.parity ^ 1, &none);
        }
      }
    }
    if (warp >= 2) {
      // ---- scales: two rows to a lane, four blocks at a time, and those of the weights
      const int row = (warp - 2) * 64 + lane * 2;
      Turn r;
      uint32_t slot = 0;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        const Tile t = order.template at<HALF>(tile);
        const int t0 = t.t0 + side * (HALF && t.half() ? kM / 2 : kM);
        const float* xs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) xs[i] = p.xs + min(t0 + row + i, t.t1 - 1) * p.ldxs;
        const float* ws = p.ws + t.e * p.gws + min(t.n0 + (lane & 3) * 64, p.N - 1) / kB * p.ldws;
        for (int k0 = s0; k0 < s1 && ok; k0 += 4) {
          float v[2][4], w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = min(k0 + j, s1 - 1);
            w[j] = __ldg(ws + k);
#pragma unroll
            for (int i = 0; i < 2; ++i) v[i][j] = __ldg(xs[i] + k);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (k0 + j >= s1) break;
            if (!r.first && !(ok = wait(empty + 8 * r.stage, r.parity ^ 1))) break;
            float* to = reinterpret_cast<float*>(smem + C::kOffScale) + slot * C::kScale;
            *reinterpret_cast<float2*>(to + row) = make_float2(v[0][j], v[1][j]);
            if (warp == 2 && lane < 4) to[kM + lane] = w[j];
            __syncwarp();
            if (lane == 0) mbar_arrive(full + 8 * r.stage);
            r.next(plan.stages);
            if (++slot == C::SS) slot = 0;
          }
        }
      }
    }
    if (warp == 1 && side) {
      // ---- the odd CTA's loads are reported to the even one
      if (lane == 0) {
        Turn r;
        const int64_t all = static_cast<int64_t>(s1 - s0) * (tiles > tile0 ? (tiles - tile0 + tile_step - 1) / tile_step : 0);
        for (int64_t g = 0; g < all && poll(full + 8 * r.stage, r.parity, abort); ++g, r.next(plan.stages))
          arrive_at(full + 8 * r.stage, leader);
      }
    } else if (warp == 1) {
      // ---- MMA issue: the whole warp in step, so that the operands stay in uniform
      // registers, and an elected thread for the instructions
      Turn r, d;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        const uint32_t idesc = idesc_of(HALF && order.template at<HALF>(tile).half() ? kM : CTAS * kM, nw);
        for (int k = s0; k < s1; ++k) {
          if (!(ok = wait(full + 8 * r.stage, r.parity))) break;
          const uint32_t at = base + r.stage * plan.stage;
          const uint64_t da = smem_desc(at), db = smem_desc(at + plan.x_bytes);
          if (!d.first && !(ok = wait(dempty + 8 * d.stage, d.parity ^ 1))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kB / 32; ++kk) G::mma(tmem + d.stage * acc_cols, da + kk * 2, db + kk * 2, idesc, kk);
            G::commit(dfull + 8 * d.stage, leader);
            G::commit(empty + 8 * r.stage, leader);
          }
          __syncwarp();
          r.next(plan.stages), d.next(accs);
        }
      }
      if (*abort) {   // the MMAs in flight end before the CTA does
        if (elect_one()) {
          volatile int none = 0;
          if (CTAS == 2) commit_pair(fin, static_cast<uint16_t>(1u << leader));
          else mma_commit(fin);
          poll(fin, 0, &none);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    cta_barrier();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
  } else {
    // ---- scale, accumulate and store: a row to a lane, half of the channels to a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAcc));
    const int q = warp & 3, h = (warp - kEpiWarp0) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t scales = base + C::kOffScale;
    unsigned char* const piece = smem + C::kOffOut + (warp - kEpiWarp0) * C::kPiece;
    uint32_t slot = 0;
    int turn = 0;
    Turn d;
    bool ok = true;
    for (int tile = tile0; tile < tiles; tile += tile_step) {
      const Tile t = order.template at<HALF>(tile);
      // the warp's channels [c0, c0 + mine) and rows.  Half a pair's rows lie in the lanes 0 to
      // 63, with the first half of the channels, and in 64 to 127 with the second
      const bool half = HALF && t.half();
      const int mine = half ? C::ACC / 2 : FULL ? C::ACC : nw / 2;
      const int r0 = half ? q % 2 * 32 : q * 32, c0 = half ? q / 2 * C::ACC + h * mine : h * mine;
      const uint32_t row_at = (r0 + lane) * 4, w_at = (kM + c0 / 64) * 4;
      const int odd = c0 % 64;   // where they start in their 64
      const int row0 = t.t0 + side * (half ? kM / 2 : kM) + r0;
      const bool busy = row0 < t.t1;
      float acc[C::ACC];
#pragma unroll
      for (int i = 0; i < C::ACC; ++i) acc[i] = 0.f;
      for (int k = s0; k < s1; ++k) {
        if (!(ok = wait(dfull + 8 * d.stage, d.parity))) break;
        tc_fence_after();
        const uint32_t from = lanes + h * mine + d.stage * acc_cols, free = dempty + 8 * d.stage;
        const uint32_t at = scales + slot * (C::kScale * 4);
        auto release = [&]() {   // all of it is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (side) arrive_at(free, leader);
            else mbar_arrive(free);
          }
        };
        // (two warps share the FMA pipe, so that one's loads are behind the other's sums)
        auto add = [&](int c, float f, bool last) {
          uint32_t v[32];
          tmem_ld32(from + c, v);
          tmem_wait32(v);
          if (last) release();
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c + i] = fmaf(__uint_as_float(v[i]), f, acc[c + i]);
        };
        if (!busy) {
          release();
        } else if (FULL) {
          const float f = lds4(at + row_at) * lds4(at + w_at);
#pragma unroll
          for (int c = 0; c < C::ACC; c += 32) {
            if (HALF && c == C::ACC / 2 && half) break;
            add(c, f, c + 32 == (HALF ? mine : C::ACC));
          }
        } else {
          const float xs = lds4(at + row_at);
#pragma unroll
          for (int c = 0; c < C::ACC; c += 32) {
            if (c >= mine) break;
            add(c, xs * lds4(at + w_at + (odd + c) / 64 * 4), c + 32 >= mine);
          }
        }
        d.next(accs);
        if (++slot == C::SS) slot = 0;
      }
      if (!ok) break;
      if (!busy) continue;
      const int n0 = t.n0 + c0;
      if (split > 1) {
        // every stage of the ring has been read: its space takes the sums
        float* sums = reinterpret_cast<float*>(smem) + (q * 32 + lane) * (nw + C::kSumPad) + h * mine;
#pragma unroll
        for (int i = 0; i < C::ACC; i += 4)
          if (i < mine) *reinterpret_cast<float4*>(sums + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        continue;
      }
      if (p.bias) {   // a channel to a lane, read together (each by all lanes: 3 us more)
        const O* bias = static_cast<const O*>(p.bias) + static_cast<int64_t>(t.e) * p.N;
        float b[C::ACC / 32];
#pragma unroll
        for (int c = 0; c < C::ACC; c += 32) b[c / 32] = to_f32<O>(__ldg(bias + min(n0 + c + lane, p.N - 1)));
#pragma unroll
        for (int i = 0; i < C::ACC; ++i) acc[i] += __shfl_sync(~0u, b[i / 32], i % 32);
      }
      // 32 channels of each of the warp's rows at a time, through shared memory: by TMA where
      // all of the rows are the group's and the tensor map does not end inside 16 bytes (all
      // 16 would be written), else row by row
      constexpr int V = 16 / sizeof(O), P = 32 / V;   // channels of 16 bytes; such pieces of a row
      constexpr int kTurns = C::kPiece / (32 * 32 * sizeof(O));   // that fit beside one another
      const bool whole = bulk && row0 + 32 <= t.t1;
      // the TMA's swizzle: 128 bytes (8 pieces) or 64 (4)
      auto place = [](int r, int i) { return r * (P * 16) + ((i ^ (P == 8 ? r & 7 : (r >> 1) & 3)) << 4); };
#pragma unroll
      for (int c = 0; c < C::ACC; c += 32) {
        if (c >= mine) break;
        unsigned char* stage = piece + turn * (32 * 32 * sizeof(O));
        turn = (turn + 1) % kTurns;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kTurns - 1) : "memory");   // its last use
        __syncwarp();
#pragma unroll
        for (int i = 0; i < P; ++i) {
          alignas(16) O o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = from_f32<O>(acc[c + i * V + e]);
          *reinterpret_cast<uint4*>(stage + place(lane, i)) = *reinterpret_cast<const uint4*>(o);
        }
        if (whole && (p.N % V == 0 || n0 + c + 32 <= p.N)) {
          proxy_fence_smem();
          __syncwarp();
          if (lane == 0 && n0 + c < p.N) tma_store_2d(&maps.out, n0 + c, row0, saddr(stage));
        } else if (!bulk) {   // rows that start anywhere: a channel to a lane
          __syncwarp();
          const int n = n0 + c + lane, r1 = n < p.N ? min(32, t.t1 - row0) : 0;
          O* out = static_cast<O*>(p.out) + row0 * p.ldo + n;
          constexpr int U = 16;   // rows read before any is written (one by one: 3171 x 27509 x 1851 216 us, so 194)
#pragma unroll 1
          for (int r = 0; r < r1; r += U) {
            O v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = reinterpret_cast<const O*>(stage + place(r + u, lane / V))[lane % V];
#pragma unroll
            for (int u = 0; u < U; ++u, out += p.ldo)
              if (r + u < r1) *out = v[u];
          }
        } else {
          __syncwarp();
          const int n = n0 + c + lane % P * V;
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int r = i * (32 / P) + lane / P, row = row0 + r;
            const uint4 raw = *reinterpret_cast<const uint4*>(stage + place(r, lane % P));
            if (row >= t.t1) continue;
            O* out = static_cast<O*>(p.out) + row * p.ldo + n;
            if (n + V <= p.N) {
              *reinterpret_cast<uint4*>(out) = raw;
            } else {
              const O* v = reinterpret_cast<const O*>(&raw);
#pragma unroll
              for (int e = 0; e < V; ++e)
                if (n + e < p.N) out[e] = v[e];
            }
          }
        }
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");   // one for every turn
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    cta_barrier();
  }

  __syncwarp();
  if (split > 1) {
    // the parts of one tile: each CTA adds and stores its share of the rows
    cluster_sync();
    if (!*abort && tile0 < tiles) {
      const Tile t = order.template at<HALF>(tile0);
      const int t0 = t.t0 + side * kM, rows = min(kM, t.t1 - t0), cols = min(nw, p.N - t.n0);
      const int r0 = rows > 0 ? rows * part / split : 0, r1 = rows > 0 ? rows * (part + 1) / split : 0;
      // four channels of a row to a thread, U such at a time with all of their reads on the way
      constexpr int U = 2;
      const int per = nw / 4, units = (r1 - r0) * per;
      for (int i0 = tid; i0 < units; i0 += U * C::kThreads) {
        float4 v[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * C::kThreads, units - 1);
          const uint32_t at = base + ((r0 + i / per) * (nw + C::kSumPad) + i % per * 4) * 4;
#pragma unroll
          for (int s = 0; s < 4; ++s) v[u][s] = s < split ? ld_cluster(at, s * CTAS + side) : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * C::kThreads, c = i % per * 4;
          if (i >= units) break;
          float sum[4] = {((v[u][0].x + v[u][1].x) + v[u][2].x) + v[u][3].x, ((v[u][0].y + v[u][1].y) + v[u][2].y) + v[u][3].y,
                          ((v[u][0].z + v[u][1].z) + v[u][2].z) + v[u][3].z, ((v[u][0].w + v[u][1].w) + v[u][2].w) + v[u][3].w};
          O* out = static_cast<O*>(p.out) + (t0 + r0 + i / per) * p.ldo + t.n0 + c;
          const O* bias = p.bias ? static_cast<const O*>(p.bias) + static_cast<int64_t>(t.e) * p.N + t.n0 + c : nullptr;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < cols) out[e] = from_f32<O>(sum[e] + (bias ? to_f32<O>(__ldg(bias + e)) : 0.f));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CTAS * split > 1) cluster_sync();   // nothing of this CTA is read or signalled any more
  tc_fence_after();
  if (warp == 1) G::dealloc(tmem);
}

// Boxes of `cols_box` columns x `box` rows of a tensor [groups][rows][cols] (groups 0: a
// matrix) with strides in bytes; columns and rows past the ends read as zero, and are not
// written.
cudaError_t map_tile(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int64_t ld,
                     int64_t group, int groups, int rows, int cols, int box, int cols_box) {
  const auto encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(groups)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld), static_cast<cuuint64_t>(group)};
  const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(cols_box), static_cast<cuuint32_t>(box), 1}, es[3] = {1, 1, 1};
  const CUresult r = encode(m, type, groups ? 3 : 2, const_cast<void*>(base), dims, strides, boxes, es,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// e4m3 rows in boxes of 128 columns, [groups][rows][cols].
cudaError_t map_rows(CUtensorMap* m, const void* base, int64_t ld, int64_t group, int groups, int rows, int cols, int box) {
  return map_tile(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, base, ld, group, groups, rows, cols, box, kB);
}

// What the kernel's launches need to know about a device, asked once.
struct OnDevice {
  std::atomic<bool> ready{false};
  int clusters[4] = {};   // of 1, 2, 4 and 8 CTAs, at once
};
template <typename K>
cudaError_t prepare(OnDevice* all, K* kernel, OnDevice** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  OnDevice& d = all[dev];
  *out = &d;
  if (d.ready.load(std::memory_order_acquire)) return cudaSuccess;
  static std::mutex asking;
  const std::lock_guard<std::mutex> lock(asking);
  if (d.ready.load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc::kSmem);
  cudaFuncAttributes at{};
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, kernel);
  if (e != cudaSuccess) return e;
  // the register split must be what the CTA is launched with
  if (at.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  for (int i = 0; i < 4; ++i) d.clusters[i] = max_clusters(kernel, Tc::kThreads, Tc::kSmem, 1 << i);
  d.ready.store(true, std::memory_order_release);
  return cudaSuccess;
}

// Of a pair's row tiles, those of at most half of its rows: of rows in groups every other
// group's last one.
double halves(const F8Args& p) {
  const int less = p.T % (2 * kM);
  return p.offsets ? p.E / 2. : less > 0 && less <= kM;
}

// What follows from a plan's tile.
void lay_out(Plan& p) {
  p.x_bytes = p.rows * kB;
  p.stage = p.x_bytes + p.nw / p.ctas * kB;
  p.stages = std::min(Tc::S, Tc::kRing / p.stage);
  p.accs = p.nw > 128 ? 2 : 4;
}

// CTAs to a tile, its channels and parts of K: what takes the least by this model.  A block
// takes 2.2 ns for each channel and 64 more (a pair of CTAs 1.9, for twice the rows), and
// 350 (400) at least.  Pairs, us, against CTAs alone: 2048 x 28672 x 4096 194 and 225, 512 x
// 28672 x 4096 54 and 62, 201 x 2891 x 1411 11.7 and 9.8; 4096 rows by 8 experts of 28672 x
// 4096 495 and 525, of 4096 x 14336 349 and 248 (five turns of 76 pairs, or four of 152 CTAs);
// 4096 rows by 60 of 2048 x 1408 49 and 44.  Channels: 64 x 28672 x 4096 25.9 with 192, 26.7
// with 256, two turns, 35.6 with 128.  K is split (in 2 or 4) where all parts run at once and
// have two blocks or more; to join them takes 2.5 us, and more with their sums: 64 x 4096 x
// 4096 12.3 in 4 parts of 128 channels, 17.0 whole with 64; 201 x 2891 x 1411 11.4 in 2 of
// 128, 9.8 whole with 64.
Plan plan_of(const F8Args& p, const OnDevice* one, const OnDevice* two) {
  const auto clusters = [&](int ctas, int size) { return (ctas == 1 ? one : two)->clusters[size == 2 ? 1 : size == 4 ? 2 : 3]; };
  const int blocks = (p.K + kB - 1) / kB;
  Plan best{};
  double least = 0;
  for (int ctas = 1; ctas <= 2; ++ctas) {
    const int units = sm_count() / ctas;
    // rows of a tile: no more than there are, and for small groups 32, so that more stages fit
    const int most = p.offsets && p.T / p.E < 16 ? 32 : kM;
    const int rows = p.T > 64 ? most : p.T > 32 ? std::min(most, 64) : p.T > 16 ? 32 : 16;
    if (ctas == 2 && (rows < kM || p.T <= kM)) break;
    // row tiles: of rows in groups about half a tile more for each, which holds where groups are
    // longer than a tile and is low where they are shorter (and of a pair's, which more seldom has
    // several, one at least)
    const int M = rows * ctas;
    const int64_t more = std::max<int64_t>(p.T / M + (p.E + 1) / 2, ctas == 2 ? p.E : 1);
    const int64_t ntt = p.offsets ? std::min<int64_t>(p.T, more) : (p.T + M - 1) / M;
    for (int nw = Tc::NT; nw >= 64; nw -= 64) {
      const int64_t tiles = ntt * ((p.N + nw - 1) / nw);
      double turns = static_cast<double>((tiles + units - 1) / units);
      if (ctas == 2 && nw == Tc::NT) turns *= 1. - 0.15 * halves(p) / ntt;
      for (int split = 1; split <= 4; split *= 2) {
        if (split > 1 && (p.offsets || blocks < 2 * split || tiles > clusters(ctas, split * ctas))) break;
        const double join = split > 1 ? 2500. + 0.085 * std::min(p.T, kM) * nw : 0.;
        const double block = ctas == 1 ? std::max(350., 2.2 * (nw + 64)) : std::max(400., 1.9 * (nw + 64));
        const double cost = turns * blocks / split * block + join;
        if (best.ctas == 0 || cost < least) best = {ctas, rows, nw, split, 0, 0, 0, 0, static_cast<float>(cost)}, least = cost;
      }
    }
  }
  lay_out(best);
  return best;
}

template <typename O, int CTAS, bool FULL, bool HALF>
cudaError_t launch_plan(const F8Args& p, const Plan& plan, cudaStream_t s) {
  Maps maps{};
  // stores by TMA, and of 16 bytes
  const bool bulk = aligned(p.out, 16) && p.ldo * sizeof(O) % 16 == 0;
  cudaError_t e = map_rows(&maps.w, p.w, p.ldw, p.gw ? p.gw : p.ldw, p.gw ? p.E : 1, p.N, p.K, plan.nw / CTAS);
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) e = map_rows(&maps.x[i], p.x, p.ldx, 0, 0, p.T, p.K, 128 >> i);
  if (e == cudaSuccess && bulk)
    e = std::is_same_v<O, float>
            ? map_tile(&maps.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, CU_TENSOR_MAP_SWIZZLE_128B, p.out, p.ldo * 4, 0, 0, p.T,
                       p.N, 32, 32)
            : map_tile(&maps.out, CU_TENSOR_MAP_DATA_TYPE_UINT16, CU_TENSOR_MAP_SWIZZLE_64B, p.out, p.ldo * 2, 0, 0, p.T,
                       p.N, 32, 32);
  if (e != cudaSuccess) return e;
  const int M = plan.rows * CTAS;
  // every tile that there is; of rows in groups there may be as many more as groups
  const int64_t ntt = (p.T + M - 1) / M, ntn = (p.N + plan.nw - 1) / plan.nw;
  const int64_t tiles = ntn * (p.offsets ? std::min<int64_t>(p.T, ntt + p.E) : ntt);
  const int64_t grid = plan.split > 1 ? tiles * plan.split : std::min<int64_t>(tiles, sm_count() / CTAS);
  return launch_close(k_tc_f8<O, CTAS, FULL, HALF>, dim3(static_cast<unsigned>(grid * CTAS)), Tc::kThreads, Tc::kSmem,
                      CTAS * plan.split, s, p, maps, plan, static_cast<int>(bulk));
}

// A given plan (pw_debug_linear_f8): ctas 1 or 2: k_tc_f8's tile and parts of K; 0: k_few_f8's
// rows at a time, CTAs that share a group's rows (`channels`) and warps that share out K (`parts`).
struct Given {
  int ctas, rows, channels, parts;
};
// Whether the kernels take it: the plans that few_of and plan_of can make, for any size.
bool given_ok(const Given& g, const F8Args& p) {
  const int blocks = (p.K + kB - 1) / kB;
  const bool power = g.parts == 1 || g.parts == 2 || g.parts == 4 || (g.ctas == 0 && g.parts == 8);
  if (!power) return false;
  if (g.ctas == 0)
    return (g.rows == 8 || g.rows == 16) && g.channels >= 1 && g.channels <= 65535 / p.E && g.parts <= blocks;
  if (g.ctas != 1 && g.ctas != 2) return false;
  if (g.rows != kM && (g.ctas == 2 || (g.rows != 64 && g.rows != 32 && g.rows != 16))) return false;
  if (g.channels < 64 || g.channels > Tc::NT || g.channels % 64) return false;
  // (every tile has a cluster of its own where K is split, and a grid its limit)
  const int M = g.rows * g.ctas;
  const int64_t tiles = (static_cast<int64_t>(p.T) + M - 1) / M * ((p.N + g.channels - 1) / g.channels);
  return g.parts == 1 || (!p.offsets && blocks >= 2 * g.parts && tiles <= 65535);
}

template <typename O>
cudaError_t launch_few(const F8Args& p, const Few& f, cudaStream_t s) {
  return f.nt == 1 ? launch_few<O, 1>(p, f, s) : launch_few<O, 2>(p, f, s);
}
template <typename O>
cudaError_t launch_tc(const F8Args& p, const Plan& plan, cudaStream_t s) {
  if (plan.ctas == 1) return launch_plan<O, 1, false, false>(p, plan, s);
  if (plan.nw < Tc::NT || plan.split > 1) return launch_plan<O, 2, false, false>(p, plan, s);
  return halves(p) > 0. ? launch_plan<O, 2, true, true>(p, plan, s) : launch_plan<O, 2, true, false>(p, plan, s);
}

template <typename O>
cudaError_t launch_f8(const F8Args& p, const Given* given, cudaStream_t s) {
  static OnDevice all[4][kMaxDev];
  OnDevice *one, *two, *full, *half;
  cudaError_t e = prepare(all[0], k_tc_f8<O, 1, false, false>, &one);
  if (e == cudaSuccess) e = prepare(all[1], k_tc_f8<O, 2, false, false>, &two);
  if (e == cudaSuccess) e = prepare(all[2], k_tc_f8<O, 2, true, false>, &full);
  if (e == cudaSuccess) e = prepare(all[3], k_tc_f8<O, 2, true, true>, &half);
  if (e != cudaSuccess) return e;
  if (given) {
    if (given->ctas == 0) return launch_few<O>(p, Few{given->rows / 8, given->channels, given->parts, 0.}, s);
    Plan plan{given->ctas, given->rows, given->channels, given->parts, 0, 0, 0, 0, 0.f};
    lay_out(plan);
    return launch_tc<O>(p, plan, s);
  }
  // Few rows, where memory bounds both, us against k_tc_f8: 8 x 28672 x 4096 24.9 and 25.7, 16 x
  // 4096 x 14336 15.8 and 19.1, 16 x 28672 x 4096 28.8 and 25.5.  Rows in groups, about two to each
  // or less: 16 rows by 8 experts of 28672 x 4096 76 and 80, of 4096 x 14336 43 and 55, 120 rows by
  // 60 of 2048 x 1408 27.8 and 31.4; 32 rows by 8 136 and 120, 256 rows by 60 39.8 and 34.3.
  const int64_t least = p.offsets ? 2 * static_cast<int64_t>(p.E) : 8;
  const double work = static_cast<double>(p.T) * p.N * p.K;
  const bool little = work <= (p.T <= 16 && !p.offsets ? 1e9 : 7e8);
  if (p.T <= least || little) {
    // Little to do: what takes less (k_tc_f8 5 us beside its tiles).  64 x 60 x 4096 3.9 and 9.6, 32
    // x 1024 x 4096 4.8 and 9.1, 128 x 2048 x 2048 9.8 and 10.1; 67 x 8384 x 890 21.7 and 7.8, 1990
    // x 576 x 512 18.0 and 6.7, 1833 rows by 26 of 192 x 1408 20.5 and 9.9.
    const Few few = few_of(p);
    if (p.T <= least || few.cost < 5000 + plan_of(p, one, two).cost) return launch_few<O>(p, few, s);
  }
  return launch_tc<O>(p, plan_of(p, one, two), s);
}

int linear_f8(const char* what, F8Args p, int out_dtype, pw_stream_t s, const Given* given = nullptr) {
  if (p.E == 1) p.gw = p.gws = 0;   // no other group
  if (p.T < 0 || p.T > PW_MAX_VOCAB || p.N < 1 || p.N > PW_MAX_VOCAB || p.K < 1 || p.K > PW_MAX_VOCAB || p.E < 1 ||
      p.E > PW_MAX_GROUPS)
    return failf(PW_EINVAL, "%s: need 0 <= T, 1 <= N, K up to %d and 1 <= E <= %d (T %d, N %d, K %d, E %d)", what,
                 PW_MAX_VOCAB, PW_MAX_GROUPS, p.T, p.N, p.K, p.E);
  if (!dtype_ok(out_dtype)) return failf(PW_EINVAL, "%s: unknown out_dtype %d", what, out_dtype);
  if (p.T == 0) return PW_OK;
  if (!p.x || !p.xs || !p.w || !p.ws || !p.out) return failf(PW_EINVAL, "%s: null x, w, scales or out", what);
  const int64_t kb = (p.K + kB - 1) / kB;
  if (p.ldx < p.K || p.ldw < p.K || p.ldo < p.N || p.ldxs < kb || p.ldws < kb)
    return failf(PW_EINVAL, "%s: a row stride is below its row (K = %d, N = %d)", what, p.K, p.N);
  if (!aligned(p.x, 16) || !aligned(p.w, 16) || p.ldx % 16 || p.ldw % 16 || p.gw % 16)
    return failf(PW_EINVAL, "%s: rows of x and w must start on 16-byte boundaries", what);
  if (p.E > 1 && (p.gw < 0 || p.gws < 0)) return failf(PW_EINVAL, "%s: a group stride is negative", what);
  if ((p.T / 16 + 1 + static_cast<int64_t>(p.E)) * (p.N / 64 + 1) > PW_MAX_VOCAB)   // tiles
    return failf(PW_EINVAL, "%s: an output of %d x %d is too large", what, p.T, p.N);
  const size_t es = dtype_bytes(out_dtype);
  if (!aligned(p.out, es) || !aligned(p.bias, es) || !aligned(p.xs, 4) || !aligned(p.ws, 4) || !aligned(p.offsets, 4))
    return failf(PW_EINVAL, "%s: misaligned pointer", what);
  if (given && !given_ok(*given, p))
    return failf(PW_EINVAL, "%s: no plan of %d CTAs, %d rows, %d channels and %d parts", what, given->ctas, given->rows,
                 given->channels, given->parts);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = out_dtype == PW_F16    ? launch_f8<__half>(p, given, st)
                        : out_dtype == PW_BF16 ? launch_f8<__nv_bfloat16>(p, given, st)
                                               : launch_f8<float>(p, given, st);
  return launch_status(e, what);
}

}  // namespace
}  // namespace pw

extern "C" {

int pw_linear_f8(const uint8_t* x, int64_t ldx, const float* x_scale, int64_t ldxs, const uint8_t* w, int64_t ldw,
                 const float* w_scale, int64_t ldws, const void* bias, int T, int N, int K, int out_dtype, void* out,
                 int64_t ldo, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_linear_f8");
  return pw::linear_f8("pw_linear_f8",
                       pw::F8Args{x, w, x_scale, w_scale, bias, nullptr, out, ldx, ldxs, ldw, ldws, ldo, 0, 0, T, N, K, 1},
                       out_dtype, s);
}

int pw_grouped_linear_f8(const uint8_t* x, int64_t ldx, const float* x_scale, int64_t ldxs, const uint8_t* w,
                         int64_t ldw, int64_t group_w, const float* w_scale, int64_t ldws, int64_t group_ws,
                         const int32_t* offsets, const void* bias, int T, int E, int N, int K, int out_dtype, void* out,
                         int64_t ldo, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_grouped_linear_f8");
  if (T > 0 && !offsets) return pw::failf(PW_EINVAL, "pw_grouped_linear_f8: null offsets");
  return pw::linear_f8("pw_grouped_linear_f8",
                       pw::F8Args{x, w, x_scale, w_scale, bias, offsets, out, ldx, ldxs, ldw, ldws, ldo, group_w,
                                  group_ws, T, N, K, E},
                       out_dtype, s);
}

int pw_linear_f8_status(pw_stream_t s, int* status) {
  pw::NvtxCall nvtx_range("pw_linear_f8_status");
  if (!status) return pw::failf(PW_EINVAL, "pw_linear_f8_status: null status");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  uint32_t now = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= pw::kMaxDev)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(&now, pw::g_f8_timeouts, sizeof now, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return pw::failf(PW_ECUDA, "pw_linear_f8_status: %s", cudaGetErrorString(e));
  // the count up to which an earlier call has told; another thread may tell meanwhile
  static std::atomic<uint32_t> told[pw::kMaxDev];
  uint32_t before = told[dev].load();
  bool more = false;
  while ((more = static_cast<int32_t>(now - before) > 0) && !told[dev].compare_exchange_weak(before, now)) {
  }
  *status = more ? PW_STATUS_TIMEOUT : 0;
  return PW_OK;
}

int pw_debug_linear_f8(int ctas, int rows, int channels, int parts, const uint8_t* x, int64_t ldx, const float* x_scale,
                       int64_t ldxs, const uint8_t* w, int64_t ldw, int64_t group_w, const float* w_scale, int64_t ldws,
                       int64_t group_ws, const int32_t* offsets, const void* bias, int T, int E, int N, int K, int out_dtype,
                       void* out, int64_t ldo, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_debug_linear_f8");
  if (!offsets && E != 1) return pw::failf(PW_EINVAL, "pw_debug_linear_f8: null offsets with E = %d", E);
  const pw::Given given{ctas, rows, channels, parts};
  return pw::linear_f8("pw_debug_linear_f8",
                       pw::F8Args{x, w, x_scale, w_scale, bias, offsets, out, ldx, ldxs, ldw, ldws, ldo, group_w,
                                  group_ws, T, N, K, E},
                       out_dtype, s, &given);
}

int pw_debug_linear_f8_timeout(pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_debug_linear_f8_timeout");
  pw::k_count_timeout<<<1, 1, 0, reinterpret_cast<cudaStream_t>(s)>>>();
  return pw::launch_status(cudaGetLastError(), "pw_debug_linear_f8_timeout");
}

}  // extern "C"
