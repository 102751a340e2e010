// Product of int8 rows with int8 weights, scales for each token and channel
// (pw_linear_i8):
//
//   out[t][n] = (sum_k x[t][k] w[n][k]) * x_scale[t] * w_scale[n] + bias[n]
//
// the sum exact in int32 (K <= 131071: 128 * 128 * K < 2^31).
//
// Up to 8 tokens: k_gemv, byte dot products on CUDA cores, the weights
// streamed once.  More tokens: k_tc on the tensor cores.  This GPU's int8
// tensor rate is a small part of its 16-bit rate, so the tensor work runs in
// fp16: int8 values are exact in fp16, their products (at most 2^14) are exact
// in fp32, and so are sums of up to 1024 of them (2^24).  Every 1024 terms the
// fp32 accumulator moves from tensor memory into int32 registers, so the sum
// is the whole-number one at any K.

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "pw_rows.cuh"
#include "pw_tc.cuh"

namespace pw {
namespace {

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

// PW_STATUS_* bits of the tensor-core kernel's bounded waits (pw_linear_i8_status).
__device__ int g_linear_status;

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

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

constexpr int kGemvWarps = 8;
constexpr int kGemvTokens = 8;

// A group of KW warps owns R channels and TT tokens and takes K in turns of
// 512 bytes (16 a lane); KW warps of one group join in shared memory.
template <typename O, int TT, int R>
__global__ void __launch_bounds__(kGemvWarps * 32) k_gemv(const LinArgs p, int kw) {
  __shared__ int s_part[kGemvWarps][R * TT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x * (kGemvWarps / kw) + warp / kw, turn = warp % kw;
  const int n0 = group * R;
  const int8_t* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = p.w + min(n0 + r, p.N - 1) * p.ldw;
  int acc[R][TT] = {};
  const int whole = p.K & ~15;
  const int step = kw * 512;
  int k = turn * 512 + lane * 16;
#pragma unroll 2
  for (; k < whole; k += step) {
    uint4 wv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = load_once(w[r] + k);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t < p.T) {
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.x + t * p.ldx + k));
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][t] = dot16(wv[r], xv, acc[r][t]);
      }
    }
  }
  if (k == whole && whole < p.K) {   // the lane whose turn the last, partial 16 bytes are
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t < p.T) {
        const uint4 xv = load_tail(p.x + t * p.ldx + k, p.K - whole);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][t] = dot16(load_tail(w[r] + k, p.K - whole), xv, acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int v = __reduce_add_sync(0xffffffffu, acc[r][t]);
      if (lane == 0) s_part[warp][r * TT + t] = v;
    }
  __syncthreads();
  // thread i: value i % (R * TT) of the CTA's group i / (R * TT)
  const int i = threadIdx.x, g = i / (R * TT), v = i % (R * TT);
  if (g >= kGemvWarps / kw) return;
  const int n = (blockIdx.x * (kGemvWarps / kw) + g) * R + v / TT, t = v % TT;
  if (n >= p.N || t >= p.T) return;
  int sum = 0;
  for (int j = 0; j < kw; ++j) sum += s_part[g * kw + j][v];
  store_out<O>(p, t, n, sum, p.xs[t], p.ws[n], p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n]) : 0.f);
}

template <typename O, int TT>
void launch_gemv_t(const LinArgs& p, cudaStream_t s) {
  // enough warps to fill the GPU: four channels to a warp where there are many
  // (one read of the tokens serves four), one where there are few, and as many
  // warps to a channel as it takes, each with at least one turn
  const int turns = (p.K + 511) / 512;
  const int want = sm_count() * 16;
  const int R = p.N >= 4 * sm_count() ? 4 : 1;
  const int groups = (p.N + R - 1) / R;
  int kw = 1;
  while (kw < kGemvWarps && kw < turns && groups * kw < want) kw *= 2;
  const int grid = (groups + kGemvWarps / kw - 1) / (kGemvWarps / kw);
  if (R == 4)
    k_gemv<O, TT, 4><<<grid, kGemvWarps * 32, 0, s>>>(p, kw);
  else
    k_gemv<O, TT, 1><<<grid, kGemvWarps * 32, 0, s>>>(p, kw);
}

template <typename O>
cudaError_t launch_gemv(const LinArgs& p, cudaStream_t s) {
  if (p.T == 1)
    launch_gemv_t<O, 1>(p, s);
  else if (p.T == 2)
    launch_gemv_t<O, 2>(p, s);
  else if (p.T <= 4)
    launch_gemv_t<O, 4>(p, s);
  else
    launch_gemv_t<O, 8>(p, s);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- tensor cores

// One CTA per SM; a tile is 128 channels (M, the weights) x NT tokens (N).
// Warps by role:
//  * warp 0 fetches int8 tiles of BK columns by TMA into a ring of S8 stages;
//  * the last 8 warps convert a stage to fp16, both operands, into the K-major
//    128-byte-swizzled layout the MMA reads: a ring of S16 stages.  A byte b
//    becomes the fp16 number 1024 + (b + 128) by placing it in the low byte of
//    0x6400, and 1152 is subtracted: five operations for four values;
//  * warp 1 issues tcgen05.mma kind::f16 (fp32 in tensor memory, two
//    accumulators of NT columns), 1024 columns of K into one accumulator,
//    then the next 1024 into the other;
//  * warps 4.. add each finished accumulator to their int32 registers while
//    the next one fills, and at the tile's end scale and store.
// Where there are few tiles a cluster of CTAs splits K and adds the parts
// through distributed shared memory; whole numbers, so in any order.
constexpr int kM = 128;
constexpr int kConvWarps = 8;
constexpr int kExactK = 1024;   // 2^24 / 2^14 products that fp32 adds exactly
constexpr int kEpiWarp0 = 4;

template <int NT>
struct Tile {
  static constexpr int BK = NT <= 64 ? 128 : 64;          // K columns of a stage
  static constexpr int EW = NT <= 64 ? 4 : 8;             // accumulating warps
  static constexpr int ACC = NT / (EW / 4);               // int32 sums of one of their threads
  static constexpr int kConvWarp0 = kEpiWarp0 + EW;
  static constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
  static constexpr int A8 = kM * BK, B8 = NT * BK;        // bytes of an int8 stage
  static constexpr int A16 = 2 * A8, B16 = 2 * B8;        // and of an fp16 stage
  static constexpr int S8 = NT <= 64 ? 4 : NT == 128 ? 5 : 3;
  static constexpr int S16 = NT <= 64 ? 2 : NT == 128 ? 4 : 3;
  static constexpr int kRing16 = S16 * (A16 + B16);
  static constexpr int kOffBar = kRing16 + S8 * (A8 + B8);
  static constexpr int kSmem = kOffBar + 8 * (2 * S8 + 2 * S16 + 4) + 16 + 1024;
  static constexpr uint32_t kCols = NT < 16 ? 32 : 2 * NT;
  static constexpr int kSubs = BK / 64;                   // 64-column halves of a stage
  static constexpr int kChunk = kExactK / BK;             // stages of one exact sum
  // D f32, A and B f16, N / 8 and M / 16
  static constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(NT >> 3) << 17) |
                                     (static_cast<uint32_t>(kM >> 4) << 24);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kM * NT * 4 <= kRing16, "a tile's int32 sums fit the fp16 ring");
};

// Registers by role for NT = 256, whose accumulating threads hold 128 sums:
// 640 threads are launched with kRegsLaunch each; 128 * (32 + 2 * 160 + 2 * 64)
// = 640 * 96 = 61440.  Every role returns to kRegsLaunch at its end: the
// accumulating warps give theirs back before a CTA barrier, the others take
// them after it (a warp that took its share while the accumulating warps were
// still waiting for theirs would leave them waiting for good).
constexpr int kRegsLaunch = 96, kRegsIssue = 32, kRegsAcc = 160, kRegsConv = 64;
static_assert(128 * (kRegsIssue + 2 * kRegsAcc + 2 * kRegsConv) <= 640 * kRegsLaunch, "register split");

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Four int8 values as two fp16 pairs.
__device__ __forceinline__ void to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = v ^ 0x80808080u;                       // b + 128
  const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
  uint32_t a = prmt(u, 0x64646464u, 0x4140), b = prmt(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), k), y = __hsub2(*reinterpret_cast<__half2*>(&b), k);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Address of 16-byte chunk c of row r in an int8 tile as the TMA writes it:
// rows of 128 bytes with the 128-byte swizzle, or of 64 with the 64-byte one.
template <int BK>
__device__ __forceinline__ uint32_t at8(uint32_t base, int r, int c) {
  return BK == 128 ? base + r * 128 + ((c ^ (r & 7)) << 4) : base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// This thread's chunks of an int8 tile of ROWS rows, converted to fp16: 64
// columns are a 128-byte row of an fp16 half tile, 16 bytes become two chunks.
template <int BK, int ROWS>
struct Convert {
  static constexpr int kTotal = ROWS * BK / 16, kThreads = kConvWarps * 32;
  static constexpr int kN = (kTotal + kThreads - 1) / kThreads;
  uint4 v[kN];

  __device__ __forceinline__ void load(uint32_t src, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = tid + i * kThreads;
      if (kTotal % kThreads == 0 || at < kTotal) v[i] = lds16(at8<BK>(src, at % ROWS, at / ROWS));
    }
  }
  __device__ __forceinline__ void store(uint32_t dst, int tid) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = tid + i * kThreads;
      if (kTotal % kThreads == 0 || at < kTotal) {
        const int r = at % ROWS, c = at / ROWS;
        const uint32_t row = dst + (c >> 2) * (ROWS * 128) + r * 128;
        const int j = (c & 3) * 2;
        uint32_t h[8];
        to_f16x4(v[i].x, h[0], h[1]);
        to_f16x4(v[i].y, h[2], h[3]);
        to_f16x4(v[i].z, h[4], h[5]);
        to_f16x4(v[i].w, h[6], h[7]);
        sts16(row + ((j ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
        sts16(row + (((j + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
      }
    }
  }
};

// 16 consecutive fp32 columns of this thread's TMEM lane (after tmem_wait).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void cta_barrier() { asm volatile("bar.sync 0;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Waits up to kWaitClocks for the phase of the given parity; false when the
// time runs out or another thread has raised the abort flag.
constexpr long long kWaitClocks = 1ll << 31;   // about a second
__device__ __forceinline__ bool wait_clocks(uint32_t bar, uint32_t parity, const volatile int* abort) {
  const long long t0 = clock64();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if (*abort || clock64() - t0 > kWaitClocks) return false;
  }
}

// Ring position of the i-th use: stage, and the parity of that use.
struct Use {
  uint32_t stage, parity;
};
template <int S>
__device__ __forceinline__ Use use(uint32_t i) {
  return Use{i % S, (i / S) & 1};
}

template <typename O, int NT>
__global__ void __launch_bounds__(Tile<NT>::kThreads, 1)
k_tc(const LinArgs p, const __grid_constant__ CUtensorMap mapw, const __grid_constant__ CUtensorMap mapx, int split) {
  using C = Tile<NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = saddr(smem);
  const uint32_t full8 = base + C::kOffBar, empty8 = full8 + 8 * C::S8;
  const uint32_t full16 = empty8 + 8 * C::S8, empty16 = full16 + 8 * C::S16;
  const uint32_t dfull = empty16 + 8 * C::S16, dempty = dfull + 16;
  int* s_misc = reinterpret_cast<int*>(smem + C::kOffBar + 8 * (2 * C::S8 + 2 * C::S16 + 4));   // tmem, abort
  volatile int* abort = s_misc + 1;
  const uint32_t ring8 = base + C::kRing16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t rank = 0;
  if (split > 1) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(s_misc)),
                 "r"(C::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < C::S8; ++i) mbar_init(full8 + 8 * i, 1), mbar_init(empty8 + 8 * i, kConvWarps);
    for (int i = 0; i < C::S16; ++i) mbar_init(full16 + 8 * i, kConvWarps), mbar_init(empty16 + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, C::EW);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_misc[1] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_misc[0]);

  // a bounded wait; false (and the abort flag) when it runs out
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (wait_clocks(bar, parity, abort)) return true;
    atomicOr(&g_linear_status, PW_STATUS_TIMEOUT);
    *abort = 1;
    return false;
  };

  const int ntn = (p.N + kM - 1) / kM, ntt = (p.T + NT - 1) / NT;
  const int tiles = ntn * ntt;
  const int steps_all = (p.K + C::BK - 1) / C::BK;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps_all) * rank / split);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps_all) * (rank + 1) / split);
  const int steps = s1 - s0;
  const int tile0 = blockIdx.x / split, tile_step = gridDim.x / split;

  constexpr bool kSplitRegs = NT == 256;
  if (warp < kEpiWarp0) {
    if constexpr (kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {
      // ---- int8 tiles by TMA
      uint32_t g = 0;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        const int n0 = (tile % ntn) * kM, t0 = (tile / ntn) * NT;
        for (int k = s0; k < s1; ++k, ++g) {
          const Use u = use<C::S8>(g);
          if (g >= C::S8 && !wait(empty8 + 8 * u.stage, u.parity ^ 1)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring8 + u.stage * (C::A8 + C::B8);
          mbar_expect_tx(full8 + 8 * u.stage, C::A8 + C::B8);
          tma_load_2d(dst, &mapw, k * C::BK, n0, full8 + 8 * u.stage);
          tma_load_2d(dst + C::A8, &mapx, k * C::BK, t0, full8 + 8 * u.stage);
        }
      }
      // after an abort the copies in flight still land before the CTA ends
      if (*abort) {
        const int none = 0;
        for (uint32_t i = g > C::S8 ? g - C::S8 : 0; i < g; ++i)
          wait_clocks(full8 + 8 * use<C::S8>(i).stage, use<C::S8>(i).parity, &none);
      }
    }
    if (warp == 1 && lane == 0) {
      // ---- MMA issue
      uint32_t g = 0, d = 0;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
        for (int k = 0; k < steps && ok; ++d) {
          const Use ud = use<2>(d);
          if (d >= 2 && !(ok = wait(dempty + 8 * ud.stage, ud.parity ^ 1))) break;
          tc_fence_after();
          const uint32_t acc = tmem + ud.stage * NT;
          const int end = min(steps, k + C::kChunk);
          for (bool first = true; k < end; ++k, ++g) {
            const Use u = use<C::S16>(g);
            if (!(ok = wait(full16 + 8 * u.stage, u.parity))) break;
            tc_fence_after();
            const uint32_t a = base + u.stage * (C::A16 + C::B16), b = a + C::A16;
#pragma unroll
            for (int s = 0; s < C::kSubs; ++s)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                mma_f16(acc, smem_desc(a + s * kM * 128 + kk * 32), smem_desc(b + s * NT * 128 + kk * 32), C::kIdesc,
                        !first || s || kk);
              }
            first = false;
            mma_commit(empty16 + 8 * u.stage);
          }
          if (ok) mma_commit(dfull + 8 * ud.stage);
        }
      }
      if (*abort && g) {   // the MMAs in flight end before the CTA does
        const int none = 0;
        const Use u = use<C::S16>(g - 1);
        wait_clocks(empty16 + 8 * u.stage, u.parity, &none);
      }
    }
    __syncwarp();
    if constexpr (kSplitRegs) {
      cta_barrier();
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    }
  } else if (warp < C::kConvWarp0) {
    // ---- accumulate and store
    if constexpr (kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAcc));
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * C::ACC;
    uint32_t d = 0;
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
      int acc[C::ACC];
#pragma unroll
      for (int i = 0; i < C::ACC; ++i) acc[i] = 0;
      for (int k = 0; k < steps; k += C::kChunk, ++d) {
        const Use ud = use<2>(d);
        ok = __all_sync(0xffffffffu, wait(dfull + 8 * ud.stage, ud.parity));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::ACC; c += 16) {
          uint32_t r[16];
          tmem_ld16(lanes + ud.stage * NT + c, r);
          tmem_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[c + i] += __float2int_rn(__uint_as_float(r[i]));
        }
        tc_fence_before();
        if (lane == 0) mbar_arrive(dempty + 8 * ud.stage);
      }
      if (!ok) break;
      const int n0 = (tile % ntn) * kM, t0 = (tile / ntn) * NT;
      if (split == 1) {
        const int n = n0 + q * 32 + lane;
        if (n < p.N) {
          const float ws = p.ws[n], bias = p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n]) : 0.f;
#pragma unroll
          for (int i = 0; i < C::ACC; ++i) {
            const int t = t0 + half * C::ACC + i;
            if (t < p.T) store_out<O>(p, t, n, acc[i], p.xs[t], ws, bias);
          }
        }
      } else {
        // every stage of the rings has been read: their space takes the sums
        int* part = reinterpret_cast<int*>(smem);
#pragma unroll
        for (int i = 0; i < C::ACC; ++i) part[(half * C::ACC + i) * kM + q * 32 + lane] = acc[i];
      }
    }
    __syncwarp();
    if constexpr (kSplitRegs) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
      cta_barrier();
    }
  } else {
    // ---- int8 to fp16
    if constexpr (kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    const int ctid = tid - C::kConvWarp0 * 32;
    uint32_t g = 0;
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += tile_step) {
      for (int k = 0; k < steps; ++k, ++g) {
        const Use u8 = use<C::S8>(g), u16 = use<C::S16>(g);
        ok = __all_sync(0xffffffffu, wait(full8 + 8 * u8.stage, u8.parity));
        if (!ok) break;
        const uint32_t src = ring8 + u8.stage * (C::A8 + C::B8);
        Convert<C::BK, kM> ca;
        Convert<C::BK, NT> cb;
        ca.load(src, ctid);
        cb.load(src + C::A8, ctid);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty8 + 8 * u8.stage);
        if (g >= C::S16) ok = __all_sync(0xffffffffu, wait(empty16 + 8 * u16.stage, u16.parity ^ 1));
        if (!ok) break;
        const uint32_t dst = base + u16.stage * (C::A16 + C::B16);
        ca.store(dst, ctid);
        cb.store(dst + C::A16, ctid);
        proxy_fence_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full16 + 8 * u16.stage);
      }
    }
    __syncwarp();
    if constexpr (kSplitRegs) {
      cta_barrier();
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsLaunch));
    }
  }

  __syncwarp();
  if (split > 1) {
    // the cluster's parts of one tile: CTA r adds and stores its share of the tokens
    cluster_sync();
    if (!*abort) {
      const int n0 = (tile0 % ntn) * kM, t0 = (tile0 / ntn) * NT;
      const int j0 = NT * rank / split, j1 = NT * (rank + 1) / split;
      for (int i = j0 * kM + tid; i < j1 * kM; i += C::kThreads) {
        const int t = t0 + i / kM, n = n0 + i % kM;
        if (t >= p.T || n >= p.N) continue;
        int sum = 0;
        for (int r = 0; r < split; ++r) sum += ld_cluster(base + i * 4, r);
        store_out<O>(p, t, n, sum, p.xs[t], p.ws[n], p.bias ? to_f32<O>(static_cast<const O*>(p.bias)[n]) : 0.f);
      }
    }
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols));
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// Boxes of bk columns x box rows of an int8 matrix; columns and rows past its
// ends read as zero.
cudaError_t map_i8(CUtensorMap* m, const int8_t* base, int64_t ld, int rows, int cols, int bk, int box) {
  const auto encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(bk), static_cast<cuuint32_t>(box)};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r =
      encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, boxes, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, bk == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int kMaxDev = 64;

template <typename O, int NT>
cudaError_t launch_tc_nt(const LinArgs& p, cudaStream_t s) {
  using C = Tile<NT>;
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(k_tc<O, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    cudaFuncAttributes at{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, k_tc<O, NT>);
    if (e != cudaSuccess) return e;
    // the register split must fit what the CTA is launched with
    if (NT == 256 && at.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    ready[dev].store(true, std::memory_order_release);
  }
  CUtensorMap mapw, mapx;
  e = map_i8(&mapw, p.w, p.ldw, p.N, p.K, C::BK, kM);
  if (e == cudaSuccess) e = map_i8(&mapx, p.x, p.ldx, p.T, p.K, C::BK, NT);
  if (e != cudaSuccess) return e;
  const int sms = sm_count();
  const int64_t tiles = static_cast<int64_t>((p.N + kM - 1) / kM) * ((p.T + NT - 1) / NT);
  const int steps = (p.K + C::BK - 1) / C::BK;
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sms && steps >= 4 * split) split *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(split > 1 ? tiles * split : std::min<int64_t>(tiles, sms)));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tc<O, NT>, p, mapw, mapx, split);
}

template <typename O>
cudaError_t launch_linear(const LinArgs& p, cudaStream_t s) {
  if (p.T <= kGemvTokens) return launch_gemv<O>(p, s);
  if (p.T <= 16) return launch_tc_nt<O, 16>(p, s);
  if (p.T <= 32) return launch_tc_nt<O, 32>(p, s);
  if (p.T <= 64) return launch_tc_nt<O, 64>(p, s);
  if (p.T <= 128) return launch_tc_nt<O, 128>(p, s);
  return launch_tc_nt<O, 256>(p, s);
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

int pw_linear_i8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w, int64_t ldw,
                 const float* w_scale, const void* bias, int T, int N, int K, int out_dtype, void* out, int64_t ldo,
                 pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_linear_i8");
  if (T < 0 || N < 1 || K < 1 || K > PW_MAX_K_I8)
    return pw::failf(PW_EINVAL, "pw_linear_i8: need T >= 0, N >= 1, 1 <= K <= %d (T %d, N %d, K %d)", PW_MAX_K_I8, T,
                     N, K);
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
  const pw::LinArgs a{x, w, x_scale, w_scale, bias, out, ldx, ldw, ldo, T, N, K};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = out_dtype == PW_F16    ? pw::launch_linear<__half>(a, st)
                        : out_dtype == PW_BF16 ? pw::launch_linear<__nv_bfloat16>(a, st)
                                               : pw::launch_linear<float>(a, st);
  return pw::launch_status(e, "pw_linear_i8");
}

int pw_linear_i8_status(pw_stream_t s, int* status) {
  pw::NvtxCall nvtx_range("pw_linear_i8_status");
  if (!status) return pw::failf(PW_EINVAL, "pw_linear_i8_status: null status");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, pw::g_linear_status, sizeof v, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return pw::failf(PW_ECUDA, "pw_linear_i8_status: %s", cudaGetErrorString(e));
  *status = v;
  return PW_OK;
}

}  // extern "C"
