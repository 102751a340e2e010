// Root-mean-square norm with the residual's addition, and int8 rows with a
// scale per row (pw_rms_norm, pw_quant_i8).
//
//   s = x + residual (fp32);  y = s * w / sqrt(mean(s^2) + eps)
//   scale = max|y| / 127;     q = rint(y / scale)
//
// One CTA per row; the row stays in registers as fp32, so every input is read
// once.  Both row reductions, sum s^2 and max|s * w|, are taken in one pass and
// joined behind one barrier: max|y| = max|s * w| * rstd, and
// y / scale = s * w * 127 / max|s * w| does not need rstd at all.
// Bound by HBM for many rows, by latency for few.

#include "pw_rows.cuh"

namespace pw {
namespace {

struct RowArgs {
  const void* x;
  const void* r;        // residual or null
  const void* w;        // weight [H] (norm only)
  void* sum;            // x + residual or null
  void* y;              // 16/32-bit output or null
  int8_t* q;            // int8 output or null
  float* scale;         // with q
  int64_t ldx, ldr, lds, ldy, ldq;
  int H;
  float eps;
};

// VE elements at element e0 of a row of H, as fp32 (0 past the end).
template <typename T, int VE>
__device__ __forceinline__ void load_chunk(const T* row, int e0, int H, float (&v)[VE]) {
  if constexpr (VE == 1) {
    v[0] = e0 < H ? to_f32<T>(row[e0]) : 0.f;
  } else {
    if (e0 + VE <= H) {
      unpack16<T>(*reinterpret_cast<const uint4*>(row + e0), v);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i) v[i] = e0 + i < H ? to_f32<T>(row[e0 + i]) : 0.f;
    }
  }
}

template <typename T, int VE>
__device__ __forceinline__ void store_chunk(T* row, int e0, int H, const float (&v)[VE]) {
  if (VE > 1 && e0 + VE <= H) {
    alignas(16) T e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = from_f32<T>(v[i]);
    if constexpr (VE > 1) *reinterpret_cast<uint4*>(row + e0) = *reinterpret_cast<const uint4*>(e);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (e0 + i < H) row[e0 + i] = from_f32<T>(v[i]);
  }
}

template <int VE>
__device__ __forceinline__ void store_q(int8_t* row, int e0, int H, const int (&v)[VE]) {
  if (VE > 1 && e0 + VE <= H) {
    alignas(8) int8_t e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = static_cast<int8_t>(v[i]);
    if constexpr (VE == 8) *reinterpret_cast<uint2*>(row + e0) = *reinterpret_cast<const uint2*>(e);
    if constexpr (VE == 4) *reinterpret_cast<uint32_t*>(row + e0) = *reinterpret_cast<const uint32_t*>(e);
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (e0 + i < H) row[e0 + i] = static_cast<int8_t>(v[i]);
  }
}

// Sum of `a` and largest `b` over the CTA, in every thread.
__device__ __forceinline__ void block_reduce(float& a, float& b, float2* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = (threadIdx.x & 31) < nw ? sh[threadIdx.x & 31] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
}

// Factors of a row's outputs: y = s * w * rstd; q = rint(s * w * up * inv).
// Rows whose largest value is so small that 127 / max overflows are first
// scaled up by 2^100.
struct RowScale {
  float rstd, up, inv, scale;
};
template <bool NORM>
__device__ __forceinline__ RowScale row_scale(float ss, float amax, int H, float eps) {
  RowScale f;
  f.rstd = NORM ? 1.f / sqrtf(ss / static_cast<float>(H) + eps) : 1.f;
  f.up = amax < 0x1p-100f ? 0x1p100f : 1.f;
  f.inv = amax > 0.f ? 127.f / (amax * f.up) : 0.f;   // NaN: the comparison fails, q = 0
  f.scale = amax * f.rstd / 127.f;
  return f;
}

template <typename T, int VE, int VPT, bool NORM>
__global__ void __launch_bounds__(1024, 1) k_rows(const RowArgs p) {
  __shared__ float2 sh[32];
  const int64_t row = blockIdx.x;
  const int H = p.H;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.ldr : nullptr;
  const T* w = static_cast<const T*>(p.w);
  float s[VPT][VE], g[VPT][VE];
  float ss = 0.f, amax = 0.f;
#pragma unroll
  for (int c = 0; c < VPT; ++c) {
    const int e0 = (threadIdx.x + c * blockDim.x) * VE;
    load_chunk<T, VE>(x, e0, H, s[c]);
    if (NORM) load_chunk<T, VE>(w, e0, H, g[c]);
    if (r) {
      float rv[VE];
      load_chunk<T, VE>(r, e0, H, rv);
#pragma unroll
      for (int i = 0; i < VE; ++i) s[c][i] += rv[i];
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      ss = fmaf(s[c][i], s[c][i], ss);
      amax = max_nan(amax, fabsf(NORM ? s[c][i] * g[c][i] : s[c][i]));
    }
  }
  if (p.sum) {
    T* d = static_cast<T*>(p.sum) + row * p.lds;
#pragma unroll
    for (int c = 0; c < VPT; ++c) store_chunk<T, VE>(d, (threadIdx.x + c * blockDim.x) * VE, H, s[c]);
  }
  block_reduce(ss, amax, sh);
  const RowScale f = row_scale<NORM>(ss, amax, H, p.eps);
#pragma unroll
  for (int c = 0; c < VPT; ++c) {
    const int e0 = (threadIdx.x + c * blockDim.x) * VE;
    if (p.y) {
      float v[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) v[i] = NORM ? s[c][i] * f.rstd * g[c][i] : s[c][i];
      store_chunk<T, VE>(static_cast<T*>(p.y) + row * p.ldy, e0, H, v);
    }
    if (p.q) {
      int v[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i)
        v[i] = __float2int_rn((NORM ? s[c][i] * g[c][i] : s[c][i]) * f.up * f.inv);
      store_q<VE>(p.q + row * p.ldq, e0, H, v);
    }
  }
  if (p.q && threadIdx.x == 0) p.scale[row] = f.scale;
}

// Rows too long for the registers of one CTA: the row is read twice.
template <typename T, int VE, bool NORM>
__global__ void __launch_bounds__(1024, 1) k_rows_long(const RowArgs p) {
  __shared__ float2 sh[32];
  const int64_t row = blockIdx.x;
  const int H = p.H, step = blockDim.x * VE;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.ldr : nullptr;
  const T* w = static_cast<const T*>(p.w);
  auto load = [&](int e0, float (&s)[VE], float (&g)[VE]) {
    load_chunk<T, VE>(x, e0, H, s);
    if (r) {
      float rv[VE];
      load_chunk<T, VE>(r, e0, H, rv);
#pragma unroll
      for (int i = 0; i < VE; ++i) s[i] += rv[i];
    }
    if (NORM) load_chunk<T, VE>(w, e0, H, g);
  };
  float ss = 0.f, amax = 0.f;
  for (int64_t e = static_cast<int64_t>(threadIdx.x) * VE; e < H; e += step) {
    float s[VE], g[VE];
    load(static_cast<int>(e), s, g);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      ss = fmaf(s[i], s[i], ss);
      amax = max_nan(amax, fabsf(NORM ? s[i] * g[i] : s[i]));
    }
  }
  block_reduce(ss, amax, sh);
  const RowScale f = row_scale<NORM>(ss, amax, H, p.eps);
  for (int64_t e = static_cast<int64_t>(threadIdx.x) * VE; e < H; e += step) {
    const int e0 = static_cast<int>(e);
    float s[VE], g[VE], v[VE];
    load(e0, s, g);
    if (p.sum) store_chunk<T, VE>(static_cast<T*>(p.sum) + row * p.lds, e0, H, s);
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = NORM ? s[i] * f.rstd * g[i] : s[i];
    if (p.y) store_chunk<T, VE>(static_cast<T*>(p.y) + row * p.ldy, e0, H, v);
    if (p.q) {
      int qv[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) qv[i] = __float2int_rn((NORM ? s[i] * g[i] : s[i]) * f.up * f.inv);
      store_q<VE>(p.q + row * p.ldq, e0, H, qv);
    }
  }
  if (p.q && threadIdx.x == 0) p.scale[row] = f.scale;
}

template <typename T, int VE, bool NORM>
cudaError_t launch_ve(const RowArgs& p, int T_, cudaStream_t s) {
  const int chunks = (p.H + VE - 1) / VE;
  auto threads = [&](int vpt) { return ((chunks + vpt - 1) / vpt + 31) / 32 * 32; };
  if (chunks <= 512) {
    k_rows<T, VE, 1, NORM><<<T_, threads(1), 0, s>>>(p);
  } else if (chunks <= 1024) {
    k_rows<T, VE, 2, NORM><<<T_, threads(2), 0, s>>>(p);
  } else if (chunks <= 4096) {
    k_rows<T, VE, 4, NORM><<<T_, threads(4), 0, s>>>(p);
  } else {
    k_rows_long<T, VE, NORM><<<T_, 1024, 0, s>>>(p);
  }
  return cudaGetLastError();
}

// 16-byte chunks where every row of every operand starts on 16 bytes (8 or 4
// for q), single elements otherwise.
template <typename T, bool NORM>
cudaError_t launch_t(const RowArgs& p, int T_, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(T);
  auto ok = [](const void* b, int64_t ld, size_t size, size_t to) {
    return !b || (aligned(b, to) && (ld * static_cast<int64_t>(size)) % static_cast<int64_t>(to) == 0);
  };
  const bool vec = ok(p.x, p.ldx, sizeof(T), 16) && ok(p.r, p.ldr, sizeof(T), 16) && ok(p.w, 0, sizeof(T), 16) &&
                   ok(p.sum, p.lds, sizeof(T), 16) && ok(p.y, p.ldy, sizeof(T), 16) && ok(p.q, p.ldq, 1, VE);
  return vec ? launch_ve<T, VE, NORM>(p, T_, s) : launch_ve<T, 1, NORM>(p, T_, s);
}

template <bool NORM>
cudaError_t launch_rows(const RowArgs& p, int T_, int dtype, cudaStream_t s) {
  if (dtype == PW_F16) return launch_t<__half, NORM>(p, T_, s);
  if (dtype == PW_BF16) return launch_t<__nv_bfloat16, NORM>(p, T_, s);
  return launch_t<float, NORM>(p, T_, s);
}

}  // namespace
}  // namespace pw

extern "C" {

int pw_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, float eps,
                int T, int H, int dtype, void* sum_out, int64_t lds, void* y, int64_t ldy, int8_t* q, int64_t ldq,
                float* scale, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_rms_norm");
  if (T < 0 || H < 1) return pw::failf(PW_EINVAL, "pw_rms_norm: need T >= 0 and H >= 1 (T %d, H %d)", T, H);
  if (!pw::dtype_ok(dtype)) return pw::failf(PW_EINVAL, "pw_rms_norm: unknown dtype %d", dtype);
  if (!(eps >= 0.f)) return pw::failf(PW_EINVAL, "pw_rms_norm: eps must not be negative or NaN");
  if (T == 0) return PW_OK;
  if (!x || !weight) return pw::failf(PW_EINVAL, "pw_rms_norm: null x or weight");
  if (!y && !q) return pw::failf(PW_EINVAL, "pw_rms_norm: neither y nor q is given");
  if (q && !scale) return pw::failf(PW_EINVAL, "pw_rms_norm: q without scale");
  if (ldx < H || (residual && ldr < H) || (sum_out && lds < H) || (y && ldy < H) || (q && ldq < H))
    return pw::failf(PW_EINVAL, "pw_rms_norm: a row stride is below H = %d", H);
  const size_t es = pw::dtype_bytes(dtype);
  if (!pw::aligned(x, es) || !pw::aligned(weight, es) || !pw::aligned(residual, es) || !pw::aligned(sum_out, es) ||
      !pw::aligned(y, es) || !pw::aligned(scale, 4))
    return pw::failf(PW_EINVAL, "pw_rms_norm: misaligned pointer");
  const pw::RowArgs a{x, residual, weight, sum_out, y, q, scale, ldx, ldr, lds, ldy, ldq, H, eps};
  return pw::launch_status(pw::launch_rows<true>(a, T, dtype, reinterpret_cast<cudaStream_t>(s)), "pw_rms_norm");
}

int pw_quant_i8(const void* x, int64_t ldx, int T, int K, int dtype, int8_t* q, int64_t ldq, float* scale,
                pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_quant_i8");
  if (T < 0 || K < 1) return pw::failf(PW_EINVAL, "pw_quant_i8: need T >= 0 and K >= 1 (T %d, K %d)", T, K);
  if (!pw::dtype_ok(dtype)) return pw::failf(PW_EINVAL, "pw_quant_i8: unknown dtype %d", dtype);
  if (T == 0) return PW_OK;
  if (!x || !q || !scale) return pw::failf(PW_EINVAL, "pw_quant_i8: null x, q or scale");
  if (ldx < K || ldq < K) return pw::failf(PW_EINVAL, "pw_quant_i8: a row stride is below K = %d", K);
  if (!pw::aligned(x, pw::dtype_bytes(dtype)) || !pw::aligned(scale, 4))
    return pw::failf(PW_EINVAL, "pw_quant_i8: misaligned pointer");
  const pw::RowArgs a{x, nullptr, nullptr, nullptr, nullptr, q, scale, ldx, 0, 0, 0, ldq, K, 0.f};
  return pw::launch_status(pw::launch_rows<false>(a, T, dtype, reinterpret_cast<cudaStream_t>(s)), "pw_quant_i8");
}

}  // extern "C"
