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
// the even one.  Where 448 / max would leave fp32's range the elements are taken times
// 2^64 first.
struct ToF8 {
  float hi, lo, scale;
  bool tiny;
  __device__ __forceinline__ explicit ToF8(float amax) {
    scale = amax / kTop;
    tiny = amax < 0x1p-100f;
    const float m = tiny ? amax * 0x1p64f : amax;
    // zeros, and sizes whose scale is below fp32's numbers: scale 0; a NaN or an
    // infinity: that scale; q is 0 in all of them
    const bool ok = scale > 0.f && amax < INFINITY;
    hi = ok ? kTop / m : 0.f;
    lo = fmaf(-hi, m, ok ? kTop : 0.f) * (hi / kTop);
    if (!ok) lo = 0.f;
  }
  __device__ __forceinline__ float operator()(float x) const { return fmaf(x, hi, x * lo); }
  // eight numbers as bytes, in order; 0 for a block without numbers
  __device__ __forceinline__ uint2 pack(float* v) const {
    if (hi == 0.f) return make_uint2(0, 0);
    if (tiny) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= 0x1p64f;
    }
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __nv_cvt_float2_to_fp8x2(make_float2((*this)(v[2 * i]), (*this)(v[2 * i + 1])), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
  }
};

// The largest of N neighbouring lanes.
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

// How rows lie: whole blocks on 16-byte boundaries; on such boundaries with a short last
// block; anywhere.  (The code for short ends costs registers, and those loads in flight.)
enum Lie { kWhole, kWide, kAny };

// N elements of a block of 128 columns by lane l of L = 128 / N, as they were loaded: columns
// 8 l + i and so on 8 L further, in 16-byte loads; kAny: columns L i + l, in loads that lie
// side by side.
template <typename T, Lie LIE, int N> struct Part {
  static constexpr int E = 16 / sizeof(T), L = kBlock / N;
  uint4 raw[N / E];
  __device__ __forceinline__ void load(const T* row, int k0, int l, int K) {
#pragma unroll
    for (int j = 0; j < N / 8; ++j) {
      const int k = k0 + l * 8 + j * 8 * L;
      if (LIE == kWhole || k + 8 <= K) {
#pragma unroll
        for (int i = 0; i < 8 / E; ++i) raw[j * (8 / E) + i] = __ldg(reinterpret_cast<const uint4*>(row + k + i * E));
      } else {
        alignas(16) T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < K ? row[k + i] : from_f32<T>(0.f);
#pragma unroll
        for (int i = 0; i < 8 / E; ++i) raw[j * (8 / E) + i] = reinterpret_cast<const uint4*>(v)[i];
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N / E; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N / E; ++i) {
      float f[E];
      unpack16<T>(raw[i], f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[i * E + e] = f[e];
    }
  }
};
template <typename T, int N> struct Part<T, kAny, N> {
  static constexpr int L = kBlock / N;
  T v[N];
  __device__ __forceinline__ void load(const T* row, int k0, int l, int K) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = k0 + i * L + l < K ? row[k0 + i * L + l] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f32<T>(v[i]);
  }
};

// Such elements as bytes, to where they lie in the row.
template <Lie LIE, int N>
__device__ __forceinline__ void store_part(uint8_t* row, int k0, int l, int K, float (&v)[N], const ToF8& f) {
  constexpr int L = kBlock / N;
#pragma unroll
  for (int j = 0; j < N / 8; ++j) {
    const uint2 p = f.pack(v + j * 8);
    const int k = k0 + l * 8 + j * 8 * L;
    if (LIE == kWhole || (LIE == kWide && k + 8 <= K)) {
      *reinterpret_cast<uint2*>(row + k) = p;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = LIE == kWide ? k + i : k0 + (j * 8 + i) * L + l;
        if (c < K) row[c] = static_cast<uint8_t>((i < 4 ? p.x : p.y) >> (i % 4 * 8));
      }
    }
  }
}

// silu(g) * u.  The exponential's argument is rounded, and so is the constant in it (by 0.23 of
// a rounding), so the result is off by (4 + 1.23 |g|) (1 - sigmoid(g)) 2^-24 and 5 x 2^-24 more:
// nothing beside the 2^-4 of the quantiser, and nine tenths of the time that expf takes.  The
// reciprocal is off by 2^-23 and takes a seventh of a division's instructions.  Below -87.3 it
// is one of fp32's subnormals (steps of 2^-149); below -88.7 the exponential is infinite, and
// the result 0 (exactly it would be above -2^-121.5 |u|).
__device__ __forceinline__ float silu_up(float g, float u) {
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));   // -log2 e
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r * u;
}
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N], float m = 0.f) {
#pragma unroll
  for (int e = 0; e < N; ++e) m = max_nan(m, fabsf(v[e]));
  return m;
}

// A warp takes four blocks of a row, eight lanes to a block (16 lanes took a seventh longer: each
// lane works out the block's factor), and fetches its next row while it quantises this one;
// blockIdx.y takes the rest of a row.  28672 x 4096 fp16: 59.5 us, 5.9 TB/s, 87 % of the copy
// rate; silu 4096 x 14336 fp16: 51.5 us, 84 %, bound by the issue slots and HBM alike.
template <typename T, bool ACT, Lie LIE>
__global__ void __launch_bounds__(256, LIE != kWhole ? 2 : ACT ? 3 : 4) k_quant(const QuantArgs p) {
  constexpr int N = 16, kStep = 4 * kBlock;
  using P = Part<T, LIE, N>;
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 7;
  after_those_before();
  let_next_begin();
  for (int64_t c = blockIdx.y * kStep; c < p.K; c += static_cast<int64_t>(gridDim.y) * kStep) {
    const int k0 = static_cast<int>(c) + (threadIdx.x >> 3 & 3) * kBlock;
    const bool in = k0 < p.K;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    // the row that row t is made of; -1: of nothing
    auto source = [&](int64_t t) -> int64_t {
      if (ACT || !p.rows) return t;
      const int r = __ldg(p.rows + t);
      return r < 0 || r / p.per >= p.n_x ? -1 : r / p.per;
    };
    P a, b;
    auto fetch = [&](int64_t from) {
      const T* row = static_cast<const T*>(p.x) + from * p.ldx;
      if (in) {
        a.load(row, k0, l, p.K);
        if constexpr (ACT) b.load(row + p.K, k0, l, p.K);
      }
    };
    int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp, from = t < p.T ? source(t) : -1;
    if (from >= 0) fetch(from);
    for (; t < p.T; t += step) {
      uint8_t* q = p.q + t * p.ldq;
      float* scale = p.scale + t * p.lds;
      const bool any = from >= 0;
      P x = a, y;
      if constexpr (ACT) y = b;
      from = t + step < p.T ? source(t + step) : -1;
      if (from >= 0) fetch(from);
      float v[N] = {};
      if (any && in) {
        x.get(v);
        if constexpr (ACT) {
          float w[N];
          y.get(w);
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = silu_up(v[e], w[e]);
        }
      }
      const ToF8 f(group_max<P::L>(largest(v)));
      if (in) {
        store_part<LIE>(q, k0, l, p.K, v, f);
        if (l == 0) scale[k0 / kBlock] = f.scale;
      }
    }
  }
}

// A CTA to a block of 128 rows x 128 columns, held as it was loaded (as fp32 it would take
// twice the registers, and half of the loads would be in flight).  28672 x 4096 bf16:
// 66.5 us, 5.3 TB/s, 78 % of the copy rate.
template <typename T, Lie LIE>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : LIE == kWhole ? 3 : 2) k_quant_blocks(const QuantArgs p) {
  __shared__ float s_max[8];
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4, k0 = blockIdx.x * kBlock;
  after_those_before();
  for (int64_t b = blockIdx.y; b * kBlock < p.T; b += gridDim.y) {
    const int64_t t0 = b * kBlock + r0;
    const T* x0 = static_cast<const T*>(p.x) + t0 * p.ldx;
    Part<T, LIE, 8> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t0 + i * 16 < p.T) x[i].load(x0 + i * 16 * p.ldx, k0, l, p.K);
      else x[i].zero();
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      x[i].get(v);
      amax = largest(v, amax);
    }
    amax = group_max<32>(amax);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) amax = max_nan(amax, s_max[w]);
    const ToF8 f(amax);
    uint8_t* q = p.q + t0 * p.ldq;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      x[i].get(v);
      if (t0 + i * 16 < p.T) store_part<LIE>(q + i * 16 * p.ldq, k0, l, p.K, v, f);
    }
    if (threadIdx.x == 0) p.scale[b * p.lds + blockIdx.x] = f.scale;
    __syncthreads();   // s_max has been read
  }
}

template <typename T, bool ACT>
cudaError_t launch_rows(const QuantArgs& p, Lie lie, cudaStream_t s) {
  const int64_t segments = (static_cast<int64_t>(p.K) + 4 * kBlock - 1) / (4 * kBlock);
  const unsigned gy = static_cast<unsigned>(std::min<int64_t>(segments, 65535));
  const int64_t rows = (static_cast<int64_t>(p.T) + 7) / 8;
  const unsigned gx = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(rows, sm_count() * int64_t{8} / gy)));
  if (lie == kWhole) return launch_close(k_quant<T, ACT, kWhole>, dim3(gx, gy), 256, 0, 1, s, p);
  if (lie == kWide) return launch_close(k_quant<T, ACT, kWide>, dim3(gx, gy), 256, 0, 1, s, p);
  return launch_close(k_quant<T, ACT, kAny>, dim3(gx, gy), 256, 0, 1, s, p);
}

template <typename T>
cudaError_t launch_quant(const QuantArgs& p, bool act, bool by_block, cudaStream_t s) {
  const int E = 16 / sizeof(T);
  // 16-byte loads and 8-byte stores
  const bool wide = aligned(p.x, 16) && p.ldx % E == 0 && (!act || p.K % E == 0) && aligned(p.q, 8) && p.ldq % 8 == 0;
  const Lie lie = !wide ? kAny : p.K % kBlock ? kWide : kWhole;
  const int blocks = (p.K + kBlock - 1) / kBlock;
  if (by_block) {
    const dim3 grid(blocks, std::min<int64_t>((static_cast<int64_t>(p.T) + kBlock - 1) / kBlock, 65535));
    if (lie == kWhole) return launch_close(k_quant_blocks<T, kWhole>, grid, 256, 0, 1, s, p);
    if (lie == kWide) return launch_close(k_quant_blocks<T, kWide>, grid, 256, 0, 1, s, p);
    return launch_close(k_quant_blocks<T, kAny>, grid, 256, 0, 1, s, p);
  }
  return act ? launch_rows<T, true>(p, lie, s) : launch_rows<T, false>(p, lie, s);
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

// Eight columns of a row, as they were loaded: those past H are 0.  OUT: of a row that may be
// the output itself, so by ordinary loads; the read-only path wants memory that the kernel
// does not write.
template <typename T, bool WIDE, bool OUT>
__device__ __forceinline__ void load_cols(const T* row, int h, int H, T (&v)[8]) {
  if (WIDE && h + 8 <= H) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      const uint4* from = reinterpret_cast<const uint4*>(row + h + i);
      *reinterpret_cast<uint4*>(v + i) = OUT ? *from : __ldg(from);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h + i < H ? row[h + i] : from_f32<T>(0.f);
  }
}
template <typename T, bool WIDE>
__device__ __forceinline__ void put_cols(T* row, int h, int H, const float (&v)[8]) {
  if (WIDE && h + 8 <= H) {
    constexpr int E = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      alignas(16) T o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = from_f32<T>(v[i + e]);
      *reinterpret_cast<uint4*>(row + h + i) = *reinterpret_cast<const uint4*>(o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h + i < H) row[h + i] = from_f32<T>(v[i]);
  }
}

// A CTA takes 8 columns a thread of N tokens, blockIdx.y the rest of them.  The rows of J
// slots of each are on their way together (two of two tokens, or four).  Places outside [0, R)
// and weights of 0 add nothing, and nothing is read for them.  The sum goes in the order of
// the slots.  8192 x 4096 fp16, two slots, residual: 50.6 us, 5.3 TB/s, 78 % of the copy rate
// (CTAs that stay, three to an SM; 65 with one to a token).
template <typename Y, typename O, bool WIDE, int N, int J>
__global__ void __launch_bounds__(256, WIDE ? 3 : 2) k_combine_rows(const CombineArgs p) {
  after_those_before();
  for (int64_t h0 = static_cast<int64_t>(blockIdx.y) * blockDim.x * 8; h0 < p.H; h0 += static_cast<int64_t>(gridDim.y) * blockDim.x * 8) {
    const int64_t hl = h0 + threadIdx.x * 8;
    if (hl >= p.H) continue;
    const int h = static_cast<int>(hl);
    // places and weights of J slots: the next tokens' are on their way with this one's rows
    int next_at[N][J];
    float next_w[N][J];
    auto slots = [&](int64_t t0, int j0) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool in = j0 + j < p.k && t0 + n < p.T;
          next_at[n][j] = in ? __ldg(p.inv + (t0 + n) * p.k + j0 + j) : -1;
          next_w[n][j] = in ? __ldg(p.w + (t0 + n) * p.k + j0 + j) : 0.f;
        }
    };
    slots(blockIdx.x * N, 0);
    for (int64_t t0 = blockIdx.x * N; t0 < p.T; t0 += gridDim.x * N) {
      float sum[N][8] = {};
      alignas(16) O r[N][8];
      if (p.res) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (t0 + n < p.T) load_cols<O, WIDE, true>(static_cast<const O*>(p.res) + (t0 + n) * p.ldr, h, p.H, r[n]);
      }
      for (int j0 = 0; j0 < p.k; j0 += J) {
        if (j0) slots(t0, j0);
        int at[N][J];
        float w[N][J];
        alignas(16) Y v[N][J][8];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            at[n][j] = next_at[n][j] >= p.R || next_w[n][j] == 0.f ? -1 : next_at[n][j];
            w[n][j] = next_w[n][j];
            if (at[n][j] >= 0) load_cols<Y, WIDE, false>(static_cast<const Y*>(p.y) + at[n][j] * p.ldy, h, p.H, v[n][j]);
          }
        if (j0 + J >= p.k) slots(t0 + gridDim.x * N, 0);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (at[n][j] >= 0) {
#pragma unroll
              for (int e = 0; e < 8; ++e) sum[n][e] = fmaf(w[n][j], to_f32<Y>(v[n][j][e]), sum[n][e]);
            }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (t0 + n >= p.T) break;
        if (p.res) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[n][e] += to_f32<O>(r[n][e]);
        }
        put_cols<O, WIDE>(static_cast<O*>(p.out) + (t0 + n) * p.ldo, h, p.H, sum[n]);
      }
    }
  }
}

template <typename Y, typename O>
cudaError_t launch_combine(const CombineArgs& p, cudaStream_t s) {
  constexpr int EY = 16 / sizeof(Y), EO = 16 / sizeof(O);
  const bool wide = aligned(p.y, 16) && p.ldy % EY == 0 && aligned(p.out, 16) && p.ldo % EO == 0 &&
                    (!p.res || (aligned(p.res, 16) && p.ldr % EO == 0));
  const int64_t chunks = (static_cast<int64_t>(p.H) + 7) / 8;
  // a token's columns over CTAs of 256 threads, or of 64 where that fills more SMs
  const int threads = p.T * ((chunks + 255) / 256) < sm_count() * 2 ? 64 : 256;
  const unsigned gy = static_cast<unsigned>(std::min<int64_t>((chunks + threads - 1) / threads, 65535));
  const unsigned gx = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(p.T, sm_count() * int64_t{3} / gy)));
  if (!wide) return launch_close(k_combine_rows<Y, O, false, 1, 2>, dim3(gx, gy), threads, 0, 1, s, p);
  if (p.k <= 2 && p.T > sm_count() * 8) return launch_close(k_combine_rows<Y, O, true, 2, 2>, dim3(gx, gy), threads, 0, 1, s, p);
  return launch_close(k_combine_rows<Y, O, true, 1, 4>, dim3(gx, gy), threads, 0, 1, s, p);
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
