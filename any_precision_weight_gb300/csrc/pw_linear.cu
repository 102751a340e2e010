// Product of int8 rows with int8 weights, scales for each token and channel
// (pw_linear_i8):
//
//   out[t][n] = (sum_k x[t][k] w[n][k]) * x_scale[t] * w_scale[n] + bias[n]
//
// the sum exact in int32 (K <= 131071: 128 * 128 * K < 2^31).

#include "pw_rows.cuh"

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

// 16 bytes at k of a row of K (zero past the end).
__device__ __forceinline__ uint4 load16(const int8_t* row, int k, int K) {
  if (k + 16 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (k + i < K) v[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), c);
  c = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), c);
  c = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), c);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), c);
}

template <typename O>
__device__ __forceinline__ void store_out(const LinArgs& p, int t, int n, int acc) {
  float v = static_cast<float>(acc) * p.xs[t] * p.ws[n];
  if (p.bias) v += to_f32<O>(static_cast<const O*>(p.bias)[n]);
  static_cast<O*>(p.out)[t * p.ldo + n] = from_f32<O>(v);
}

constexpr int kTT = 8;   // tokens of one pass

// One warp per channel and group of kTT tokens.
template <typename O>
__global__ void __launch_bounds__(256) k_linear_simple(const LinArgs p) {
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int t0 = blockIdx.y * kTT;
  if (n >= p.N) return;
  const int8_t* w = p.w + n * p.ldw;
  int acc[kTT] = {};
  for (int k = lane * 16; k < p.K; k += 512) {
    const uint4 wv = load16(w, k, p.K);
#pragma unroll
    for (int t = 0; t < kTT; ++t)
      if (t0 + t < p.T) acc[t] = dot16(wv, load16(p.x + (t0 + t) * p.ldx, k, p.K), acc[t]);
  }
#pragma unroll
  for (int t = 0; t < kTT; ++t) {
    const int v = __reduce_add_sync(0xffffffffu, acc[t]);
    if (lane == 0 && t0 + t < p.T) store_out<O>(p, t0 + t, n, v);
  }
}

template <typename O>
cudaError_t launch_linear(const LinArgs& p, cudaStream_t s) {
  k_linear_simple<O><<<dim3((p.N + 7) / 8, (p.T + kTT - 1) / kTT), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace pw

extern "C" int pw_linear_i8(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w, int64_t ldw,
                            const float* w_scale, const void* bias, int T, int N, int K, int out_dtype, void* out,
                            int64_t ldo, pw_stream_t s) {
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
