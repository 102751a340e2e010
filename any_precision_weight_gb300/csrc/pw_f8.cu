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
#include <cmath>
#include <mutex>

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

// Rows of a group.  Offsets come from the device: what is out of order or range is cut,
// so that no row outside [0, T) is touched.
struct Rows {
  int begin, end;
};
__device__ __forceinline__ Rows rows_of(const F8Args& p, int e) {
  if (!p.offsets) return {0, p.T};
  const int a = min(max(__ldg(p.offsets + e), 0), p.T), z = min(max(__ldg(p.offsets + e + 1), 0), p.T);
  return {a, max(a, z)};
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
template <typename O, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, kFewCtas) k_few_f8(const F8Args p, int kw, int turns) {
  constexpr int kRow = NT * 8 + 1;   // padded against bank conflicts
  __shared__ float s_part[kFewWarps][16 * kRow];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int groups = kFewWarps / kw, turn = warp % kw;
  const int e = blockIdx.y / turns;
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
    // a block: two runs of 64 columns, 16 of them to a lane
    auto add = [&](const uint4 (&a)[2][2], const uint4 (&v)[2][NT], int b) {
      float part[NT][4] = {};
      const float s = __ldg(ws + b);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t ha[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) widen16(a[u][i], ha[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t hx[8];
          widen16(v[u][j], hx);
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            mma_16816(part[j], ha[0][i], ha[1][i], ha[0][i + 1], ha[1][i + 1], hx[i], hx[i + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float s0 = __ldg(xs[j][0] + b) * s, s1 = __ldg(xs[j][1] + b) * s;
        acc[j][0] = fmaf(part[j][0], s0, acc[j][0]);
        acc[j][1] = fmaf(part[j][1], s1, acc[j][1]);
        acc[j][2] = fmaf(part[j][2], s0, acc[j][2]);
        acc[j][3] = fmaf(part[j][3], s1, acc[j][3]);
      }
    };
    int b = b0;
    for (; b < min(b1, whole); ++b) {
      uint4 a[2][2], v[2][NT];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) a[u][i] = load_once(w[i] + b * kB + u * 64);
#pragma unroll
        for (int j = 0; j < NT; ++j) v[u][j] = __ldg(reinterpret_cast<const uint4*>(x[j] + b * kB + u * 64));
      }
      add(a, v, b);
    }
    if (b < b1) {   // the last block, not whole
      uint4 a[2][2], v[2][NT];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = b * kB + u * 64, left = p.K - at - q * 16;
        auto part = [&](const uint8_t* from) {
          return left >= 16 ? __ldg(reinterpret_cast<const uint4*>(from + at)) : load_tail(from + at, left);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) a[u][i] = part(w[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) v[u][j] = part(x[j]);
      }
      add(a, v, b);
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

template <typename O, int NT>
cudaError_t launch_few(const F8Args& p, int turns, cudaStream_t s) {
  const int groups = (p.N + 15) / 16, blocks = (p.K + kB - 1) / kB, slots = sm_count() * kFewCtas;
  const int64_t rows = static_cast<int64_t>(p.E) * turns;
  int kw = 1;
  float least = 0.f;
  for (int n = 1, i = 0; n <= kFewWarps && (n == 1 || blocks >= n); n *= 2, ++i) {
    const float waves = static_cast<float>(groups) * rows * n / (kFewWarps * slots);
    const float cost = std::ceil(waves) / waves * (1.f + 0.06f * i);
    if (n == 1 || cost < least) kw = n, least = cost;
  }
  const int per = kFewWarps / kw;
  k_few_f8<O, NT><<<dim3((groups + per - 1) / per, static_cast<unsigned>(rows)), kFewWarps * 32, 0, s>>>(p, kw, turns);
  return cudaGetLastError();
}

template <typename O>
cudaError_t launch_f8(const F8Args& p, cudaStream_t s) {
  const int64_t rows = p.offsets ? (p.T + p.E - 1) / p.E : p.T;   // of a group, about
  const int nt = rows <= 8 ? 1 : 2;
  const int turns = static_cast<int>(std::min<int64_t>((rows + nt * 8 - 1) / (nt * 8), 65535 / p.E));
  return nt == 1 ? launch_few<O, 1>(p, turns, s) : launch_few<O, 2>(p, turns, s);
}

int linear_f8(const char* what, const F8Args& p, int out_dtype, pw_stream_t s) {
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
  const size_t es = dtype_bytes(out_dtype);
  if (!aligned(p.out, es) || !aligned(p.bias, es) || !aligned(p.xs, 4) || !aligned(p.ws, 4) || !aligned(p.offsets, 4))
    return failf(PW_EINVAL, "%s: misaligned pointer", what);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = out_dtype == PW_F16    ? launch_f8<__half>(p, st)
                        : out_dtype == PW_BF16 ? launch_f8<__nv_bfloat16>(p, st)
                                               : launch_f8<float>(p, st);
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

}  // extern "C"
