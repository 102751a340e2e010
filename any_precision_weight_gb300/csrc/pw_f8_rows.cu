// Rows of the expert layer in 8-bit floating point (e4m3, largest number 448):
//
//   pw_quant_f8, pw_silu_quant_f8:  for every row t and 128 columns b
//     scale[t][b] = max|x| / 448,  q = x * 448 / max|x| rounded to e4m3
//     (x: a row that `rows` names, or silu(gate) * up)
//   pw_quant_f8_blocks: the same with one scale for 128 rows x 128 columns
//   pw_combine:  out[t] = residual[t] + sum_j weight[t][j] * y[inv[t][j]]
//
// All are bound by HBM for many rows and by their latency for few.

#include <cuda_fp8.h>

#include <algorithm>

#include "pw_rows.cuh"

namespace pw {
namespace {

constexpr float kTop = 448.f;   // largest e4m3 number
constexpr int kBlock = 128;     // columns (and rows of weights) that share a scale

// x * 448 / max for the elements of one block.  The factor is held as two fp32
// numbers, so that the quotient is off by less than a rounding: quotients of 16-bit
// inputs that are halfway between two e4m3 numbers come out exactly there, and go to
// the even one.  Blocks whose largest element is below 2^-60 are taken times 2^64
// first, where 448 / max stays in range.
struct ToF8 {
  float hi, lo, unit, scale;
  __device__ __forceinline__ explicit ToF8(float amax) {
    unit = amax < 0x1p-60f ? 0x1p64f : 1.f;
    scale = amax / kTop;
    const float m = amax * unit;
    // zeros, and sizes whose scale is below fp32's numbers: scale 0; a NaN or an
    // infinity: that scale; q is 0 in all of them
    const bool ok = scale > 0.f && amax < INFINITY;
    hi = ok ? kTop / m : 0.f;
    lo = ok ? fmaf(-hi, m, kTop) / m : 0.f;
  }
  __device__ __forceinline__ float operator()(float x) const {
    x *= unit;
    return fmaf(x, hi, x * lo);
  }
  // two numbers, the first in the low byte; 0 for a block without numbers
  __device__ __forceinline__ uint32_t pair(float a, float b) const {
    if (hi == 0.f) return 0;
    return __nv_cvt_float2_to_fp8x2(make_float2((*this)(a), (*this)(b)), __NV_SATFINITE, __NV_E4M3);
  }
};

// The largest of a group of N neighbouring lanes.
template <int N>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

struct QuantArgs {
  const void* x;
  const int32_t* rows;
  uint8_t* q;
  float* scale;
  int64_t ldx, ldq, lds, n_x;
  int T, K, per;
};

// Eight consecutive elements of a row from column k (those past K: 0).
template <typename T, bool WIDE>
__device__ __forceinline__ void load8(const T* row, int k, int K, float (&v)[8]) {
  if (WIDE && k + 8 <= K) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      const uint4 raw = __ldg(reinterpret_cast<const uint4*>(row + k + i));
      float f[E];
      unpack16<T>(raw, f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[i + e] = f[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? to_f32<T>(row[k + i]) : 0.f;
  }
}

__device__ __forceinline__ void store8(uint8_t* row, int k, int K, const float (&v)[8], const ToF8& f, bool wide) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = f.pair(v[2 * i], v[2 * i + 1]);
  if (wide && k + 8 <= K) {
    *reinterpret_cast<uint2*>(row + k) = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) row[k + i] = static_cast<uint8_t>(p[i / 2] >> (i % 2 * 8));
  }
}

__device__ __forceinline__ float silu_up(float g, float u) { return g / (1.f + expf(-g)) * u; }

// 16 lanes take a block of 128 columns, 8 columns each.
template <typename T, bool ACT, bool WIDE>
__global__ void __launch_bounds__(256) k_quant(const QuantArgs p) {
  const int lane = threadIdx.x & 15, blocks = (p.K + kBlock - 1) / kBlock;
  const int64_t all = static_cast<int64_t>(p.T) * blocks, step = static_cast<int64_t>(gridDim.x) * 16;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 16; i0 < all; i0 += step) {
    const int64_t i = i0 + (threadIdx.x >> 4), at = i < all ? i : all - 1;   // the last ones again: every lane takes part
    const int64_t t = at / blocks;
    const int b = static_cast<int>(at - t * blocks), k = b * kBlock + lane * 8;
    float v[8] = {};
    int64_t from = t;
    if (!ACT && p.rows) {
      const int r = __ldg(p.rows + t);
      from = r < 0 ? -1 : r / p.per;
    }
    if (from >= 0 && from < p.n_x) {
      const T* row = static_cast<const T*>(p.x) + from * p.ldx;
      load8<T, WIDE>(row, k, p.K, v);
      if constexpr (ACT) {
        float u[8];
        load8<T, WIDE>(row + p.K, k, p.K, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = silu_up(v[e], u[e]);
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[e]));
    const ToF8 f(group_max<16>(amax));
    if (i < all) {
      store8(p.q + t * p.ldq, k, p.K, v, f, WIDE);
      if (lane == 0) p.scale[t * p.lds + b] = f.scale;
    }
  }
}

// A CTA to a block of 128 rows x 128 columns.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) k_quant_blocks(const QuantArgs p) {
  __shared__ float s_max[8];
  const int k = blockIdx.x * kBlock + (threadIdx.x & 15) * 8, r0 = threadIdx.x >> 4;
  for (int64_t b = blockIdx.y; b * kBlock < p.T; b += gridDim.y) {
    const int64_t t0 = b * kBlock;
    float v[8][8], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = t0 + r0 + i * 16;
      if (t < p.T) {
        load8<T, WIDE>(static_cast<const T*>(p.x) + t * p.ldx, k, p.K, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[i][e]));
    amax = group_max<32>(amax);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) amax = max_nan(amax, s_max[w]);
    const ToF8 f(amax);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t t = t0 + r0 + i * 16;
      if (t < p.T) store8(p.q + t * p.ldq, k, p.K, v[i], f, WIDE);
    }
    if (threadIdx.x == 0) p.scale[b * p.lds + blockIdx.x] = f.scale;
    __syncthreads();   // s_max has been read
  }
}

template <typename T>
cudaError_t launch_quant(const QuantArgs& p, bool act, bool by_block, cudaStream_t s) {
  const int E = 16 / sizeof(T);
  // 16-byte loads and 8-byte stores
  const bool wide = aligned(p.x, 16) && p.ldx % E == 0 && (!act || p.K % E == 0) && aligned(p.q, 8) && p.ldq % 8 == 0;
  const int blocks = (p.K + kBlock - 1) / kBlock;
  if (by_block) {
    const dim3 grid(blocks, std::min<int64_t>((static_cast<int64_t>(p.T) + kBlock - 1) / kBlock, 65535));
    if (wide) k_quant_blocks<T, true><<<grid, 256, 0, s>>>(p);
    else k_quant_blocks<T, false><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  const int64_t turns = (static_cast<int64_t>(p.T) * blocks + 15) / 16;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(turns, sm_count() * 8));
  if (act) {
    if (wide) k_quant<T, true, true><<<grid, 256, 0, s>>>(p);
    else k_quant<T, true, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (wide) k_quant<T, false, true><<<grid, 256, 0, s>>>(p);
    else k_quant<T, false, false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

int quant(const char* what, QuantArgs p, int dtype, bool act, bool by_block, pw_stream_t s) {
  if (p.T < 0 || p.T > PW_MAX_VOCAB || p.K < 1 || p.K > PW_MAX_VOCAB)
    return failf(PW_EINVAL, "%s: need 0 <= rows <= %d and 1 <= K <= %d (rows %d, K %d)", what, PW_MAX_VOCAB,
                 PW_MAX_VOCAB, p.T, p.K);
  if (!dtype_ok(dtype)) return failf(PW_EINVAL, "%s: unknown dtype %d", what, dtype);
  if (p.per < 1) return failf(PW_EINVAL, "%s: per must be 1 or more, not %d", what, p.per);
  if (p.n_x < 0 || (p.rows == nullptr && p.n_x < p.T))
    return failf(PW_EINVAL, "%s: x has %lld rows", what, static_cast<long long>(p.n_x));
  if (p.T == 0) return PW_OK;
  if ((!p.x && p.n_x > 0) || !p.q || !p.scale) return failf(PW_EINVAL, "%s: null x, q or scale", what);
  const int blocks = (p.K + kBlock - 1) / kBlock;
  if (p.ldx < (act ? 2 * static_cast<int64_t>(p.K) : p.K) || p.ldq < p.K || p.lds < blocks)
    return failf(PW_EINVAL, "%s: a row stride is below its row (K = %d)", what, p.K);
  if (!aligned(p.x, dtype_bytes(dtype)) || !aligned(p.scale, 4) || !aligned(p.rows, 4))
    return failf(PW_EINVAL, "%s: misaligned pointer", what);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = dtype == PW_F16    ? launch_quant<__half>(p, act, by_block, st)
                        : dtype == PW_BF16 ? launch_quant<__nv_bfloat16>(p, act, by_block, st)
                                           : launch_quant<float>(p, act, by_block, st);
  return launch_status(e, what);
}

// ---------------------------------------------------------------- the experts' sum

struct CombineArgs {
  const void* y;
  const float* w;
  const int32_t* inv;
  const void* res;
  void* out;
  int64_t ldy, ldr, ldo, R;
  int T, H, k;
};

// Eight elements as type O to row + h (those past H: not).
template <typename O, bool WIDE>
__device__ __forceinline__ void put8(O* row, int h, int H, const float (&v)[8]) {
  if (WIDE && h + 8 <= H) {
    constexpr int E = 16 / sizeof(O);
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      alignas(16) O o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = from_f32<O>(v[i + e]);
      *reinterpret_cast<uint4*>(row + h + i) = *reinterpret_cast<const uint4*>(o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h + i < H) row[h + i] = from_f32<O>(v[i]);
  }
}

// A thread takes 8 columns of a token.  Places outside [0, R) and weights of 0 add
// nothing, and nothing is read for them.  The sum goes in the order of the slots.
template <typename Y, typename O, bool WIDE>
__global__ void __launch_bounds__(256) k_combine_rows(const CombineArgs p) {
  const int per = (p.H + 7) / 8;
  const int64_t all = static_cast<int64_t>(p.T) * per, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += step) {
    const int64_t t = i / per;
    const int h = static_cast<int>(i - t * per) * 8;
    float sum[8] = {};
    for (int j = 0; j < p.k; ++j) {
      const int at = __ldg(p.inv + t * p.k + j);
      const float w = __ldg(p.w + t * p.k + j);
      if (at < 0 || at >= p.R || w == 0.f) continue;
      float v[8];
      load8<Y, WIDE>(static_cast<const Y*>(p.y) + at * p.ldy, h, p.H, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, v[e], sum[e]);
    }
    if (p.res) {
      float r[8];
      load8<O, WIDE>(static_cast<const O*>(p.res) + t * p.ldr, h, p.H, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += r[e];
    }
    put8<O, WIDE>(static_cast<O*>(p.out) + t * p.ldo, h, p.H, sum);
  }
}

template <typename Y, typename O>
cudaError_t launch_combine(const CombineArgs& p, cudaStream_t s) {
  constexpr int EY = 16 / sizeof(Y), EO = 16 / sizeof(O);
  const bool wide = aligned(p.y, 16) && p.ldy % EY == 0 && aligned(p.out, 16) && p.ldo % EO == 0 &&
                    (!p.res || (aligned(p.res, 16) && p.ldr % EO == 0));
  const int64_t all = static_cast<int64_t>(p.T) * ((p.H + 7) / 8);
  const int threads = all < sm_count() * 256 ? 64 : 256;   // few columns: over more SMs
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((all + threads - 1) / threads, sm_count() * 32));
  if (wide) k_combine_rows<Y, O, true><<<grid, threads, 0, s>>>(p);
  else k_combine_rows<Y, O, false><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename Y>
cudaError_t launch_combine_y(const CombineArgs& p, int out_dtype, cudaStream_t s) {
  if (out_dtype == PW_F16) return launch_combine<Y, __half>(p, s);
  if (out_dtype == PW_BF16) return launch_combine<Y, __nv_bfloat16>(p, s);
  return launch_combine<Y, float>(p, s);
}

}  // namespace
}  // namespace pw

extern "C" {

int pw_quant_f8(const void* x, int64_t ldx, int64_t x_rows, const int32_t* rows, int per, int T, int K, int dtype,
                uint8_t* q, int64_t ldq, float* scale, int64_t lds, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_quant_f8");
  return pw::quant("pw_quant_f8", pw::QuantArgs{x, rows, q, scale, ldx, ldq, lds, x_rows, T, K, per}, dtype, false,
                   false, s);
}

int pw_silu_quant_f8(const void* x, int64_t ldx, int T, int K, int dtype, uint8_t* q, int64_t ldq, float* scale,
                     int64_t lds, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_silu_quant_f8");
  return pw::quant("pw_silu_quant_f8", pw::QuantArgs{x, nullptr, q, scale, ldx, ldq, lds, T, T, K, 1}, dtype, true,
                   false, s);
}

int pw_quant_f8_blocks(const void* w, int64_t ldw, int N, int K, int dtype, uint8_t* q, int64_t ldq, float* scale,
                       int64_t lds, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_quant_f8_blocks");
  return pw::quant("pw_quant_f8_blocks", pw::QuantArgs{w, nullptr, q, scale, ldw, ldq, lds, N, N, K, 1}, dtype, false,
                   true, s);
}

int pw_combine(const void* y, int64_t ldy, int64_t y_rows, int dtype, const float* weight, const int32_t* inv,
               const void* residual, int64_t ldr, int T, int k, int H, int out_dtype, void* out, int64_t ldo,
               pw_stream_t s) {
  using namespace pw;
  NvtxCall nvtx_range("pw_combine");
  if (T < 0 || T > PW_MAX_VOCAB || H < 1 || H > PW_MAX_VOCAB || k < 1 || k > PW_MAX_GROUPS || y_rows < 0)
    return failf(PW_EINVAL, "pw_combine: need 0 <= T <= %d, 1 <= H <= %d, 1 <= k <= %d, y_rows >= 0 (T %d, H %d, k %d)",
                 PW_MAX_VOCAB, PW_MAX_VOCAB, PW_MAX_GROUPS, T, H, k);
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype))
    return failf(PW_EINVAL, "pw_combine: unknown dtype %d or out_dtype %d", dtype, out_dtype);
  if (T == 0) return PW_OK;
  if ((!y && y_rows > 0) || !weight || !inv || !out) return failf(PW_EINVAL, "pw_combine: null y, weight, inv or out");
  if (ldy < H || ldo < H || (residual && ldr < H)) return failf(PW_EINVAL, "pw_combine: a row stride is below H = %d", H);
  const size_t eo = dtype_bytes(out_dtype);
  if (!aligned(y, dtype_bytes(dtype)) || !aligned(weight, 4) || !aligned(inv, 4) || !aligned(residual, eo) ||
      !aligned(out, eo))
    return failf(PW_EINVAL, "pw_combine: misaligned pointer");
  const CombineArgs a{y, weight, inv, residual, out, ldy, ldr, ldo, y_rows, T, H, k};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = dtype == PW_F16    ? launch_combine_y<__half>(a, out_dtype, st)
                        : dtype == PW_BF16 ? launch_combine_y<__nv_bfloat16>(a, out_dtype, st)
                                           : launch_combine_y<float>(a, out_dtype, st);
  return launch_status(e, "pw_combine");
}

}  // extern "C"
