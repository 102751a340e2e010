// Routing on its own (pw_route): for every token the top-k experts by logit (ties to
// the lower index) with their softmax weights, and the routed pairs t * k + j in
// (expert, token) order with every expert's first place among them.
//
//   weight[t][j] = exp(logit_j - max) / sum, the sum over all experts, or over the k
//   chosen ones (renorm)
//
// A warp takes a token; a CTA takes a run of tokens and counts its pairs by expert.
// The sort is a counting sort: an expert's pairs start behind those of the experts and
// the CTAs before.  Up to kSmallTokens tokens one CTA does all of it (one launch, bound
// by its latencies); above, a second launch places them once every CTA has counted.
// Each of its CTAs adds up the counts of those before it by itself, which costs less
// than a launch between the two.

#include <algorithm>
#include <cmath>

#include "pw_rows.cuh"

namespace pw {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSmallTokens = 32;
constexpr int kMaxCtas = 128;

struct RouteArgs {
  const float* logits;
  int64_t ld;
  int32_t* idx;
  float* weight;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv;
  int32_t* counts;   // [CTA][E]
  int T, E, k, renorm, tokens;   // tokens: of one CTA
};

// A float as an unsigned number of the same order; both zeros are one.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}

// One token by a warp, NPER logits to a lane.  A NaN counts as -inf.  Rows without a
// number above -inf have weights 0; where +inf is among the logits, those share the
// weight.
template <int NPER>
__device__ __forceinline__ void load_token(const RouteArgs& p, int64_t t, float (&v)[NPER]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < NPER; ++i) v[i] = lane + 32 * i < p.E ? __ldg(p.logits + t * p.ld + lane + 32 * i) : -INFINITY;
}
template <int NPER>
__device__ __forceinline__ void route_token(const RouteArgs& p, int64_t t, float (&v)[NPER]) {
  const int lane = threadIdx.x & 31;
  uint32_t key[NPER];   // 0: taken, or past E
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 32 * i;
    if (isnan(v[i])) v[i] = -INFINITY;
    key[i] = e < p.E ? order_of(v[i]) : 0;
  }
  float m = v[0];
#pragma unroll
  for (int i = 1; i < NPER; ++i) m = fmaxf(m, v[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool none = m == -INFINITY;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    v[i] = none ? 0.f : v[i] == m ? 1.f : expf(v[i] - m);
    sum += v[i];
  }
  if (!p.renorm) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  float chosen = 0.f, mine = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += 32) {   // lane j keeps the slot j0 + j
    int e_mine = 0;
    for (int j = j0; j < min(p.k, j0 + 32); ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int i = 1; i < NPER; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(0xffffffffu, best);
      unsigned at = 0xffffffffu;
#pragma unroll
      for (int i = NPER - 1; i >= 0; --i)
        if (key[i] == best) at = lane + 32 * i;
      at = __reduce_min_sync(0xffffffffu, at);
      float w = 0.f;
#pragma unroll
      for (int i = 0; i < NPER; ++i)
        if (at == lane + 32u * i) w = v[i], key[i] = 0;
      w = __shfl_sync(0xffffffffu, w, at & 31);
      chosen += w;
      if (lane == j - j0) mine = w, e_mine = static_cast<int>(at);
    }
    const int j = j0 + lane;
    if (j < p.k) {
      p.idx[t * p.k + j] = e_mine;
      // renorm with more than 32 slots: divided below, once all of them are known
      if (!p.renorm || p.k <= 32) p.weight[t * p.k + j] = none ? 0.f : mine / (p.renorm ? chosen : sum);
      else p.weight[t * p.k + j] = mine;
    }
  }
  if (p.renorm && p.k > 32 && !none)
    for (int j = lane; j < p.k; j += 32) p.weight[t * p.k + j] /= chosen;
}

// Places the pairs [q0, q1) of this CTA, whose first place for expert e is base[e]:
// warps count runs of them, the counts are scanned into each warp's first places, and
// each warp places its run 32 at a time.  s_c: [kWarps][E].
__device__ __forceinline__ void place_pairs(const RouteArgs& p, int q0, int q1, const int* base, int* s_c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E;
  const int run = (q1 - q0 + kWarps - 1) / kWarps;
  const int a = min(q1, q0 + warp * run), z = min(q1, a + run);
  int* mine = s_c + warp * E;
  for (int e = lane; e < E; e += 32) mine[e] = 0;
  __syncwarp();
  for (int q = a + lane; q < z; q += 32) atomicAdd(&mine[p.idx[q]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    int at = base[e];
    for (int w = 0; w < kWarps; ++w) {
      const int c = s_c[w * E + e];
      s_c[w * E + e] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int b = a; b < z; b += 32) {
    const int q = b + lane;
    const unsigned act = __ballot_sync(0xffffffffu, q < z);
    if (q < z) {
      const int e = p.idx[q];
      const unsigned same = __match_any_sync(act, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int pos = mine[e] + rank;
      p.perm[pos] = q;
      p.inv[q] = pos;
      __syncwarp(act);   // every lane has read its expert's place
      if (rank == 0) mine[e] += __popc(same);
    }
    __syncwarp();
  }
}

// Exclusive sums of s[0..E) in place by one warp; s[E] = their total.
__device__ __forceinline__ void scan_counts(int* s, int E) {
  const int lane = threadIdx.x;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane, c = e < E ? s[e] : 0;
    int sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (e < E) s[e] = before + sum - c;
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) s[E] = before;
}

// A CTA's run of tokens; where it is the only CTA, their places too.
template <int NPER>
__global__ void __launch_bounds__(kThreads) k_route_count(const RouteArgs p) {
  extern __shared__ int s_mem[];   // counts [E + 1], then [kWarps][E]
  int* s_n = s_mem;
  const int warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * p.tokens, t1 = min(p.T, t0 + p.tokens);
  for (int e = threadIdx.x; e < p.E; e += kThreads) s_n[e] = 0;
  float v[NPER], next[NPER];   // the next token's logits are on their way while this one is routed
  if (t0 + warp < t1) load_token<NPER>(p, t0 + warp, next);
  for (int t = t0 + warp; t < t1; t += kWarps) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) v[i] = next[i];
    if (t + kWarps < t1) load_token<NPER>(p, t + kWarps, next);
    route_token<NPER>(p, t, v);
  }
  __syncthreads();
  for (int q = t0 * p.k + threadIdx.x; q < t1 * p.k; q += kThreads) atomicAdd(&s_n[p.idx[q]], 1);
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += kThreads) p.counts[blockIdx.x * p.E + e] = s_n[e];
    return;
  }
  if (threadIdx.x < 32) scan_counts(s_n, p.E);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = s_n[e];
  place_pairs(p, 0, p.T * p.k, s_n, s_mem + p.E + 1);
}

__global__ void __launch_bounds__(kThreads) k_route_place(const RouteArgs p) {
  extern __shared__ int s_mem[];
  int *s_base = s_mem, *s_off = s_mem + p.E, *s_c = s_off + p.E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kThreads) s_base[e] = s_off[e] = 0;
  __syncthreads();
  for (int e = lane; e < p.E; e += 32) {   // a warp adds the counts of every 16th CTA
    int before = 0, all = 0;
#pragma unroll 8
    for (int c = warp; c < static_cast<int>(gridDim.x); c += kWarps) {
      const int n = p.counts[c * p.E + e];
      if (c < static_cast<int>(blockIdx.x)) before += n;
      all += n;
    }
    atomicAdd(&s_base[e], before);
    atomicAdd(&s_off[e], all);
  }
  __syncthreads();
  if (threadIdx.x < 32) scan_counts(s_off, p.E);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) s_base[e] += s_off[e];
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = s_off[e];
  __syncthreads();
  const int t0 = blockIdx.x * p.tokens, t1 = min(p.T, t0 + p.tokens);
  place_pairs(p, t0 * p.k, t1 * p.k, s_base, s_c);
}

// CTAs of a batch.
int ctas_of(int T) {
  if (T <= kSmallTokens) return 1;
  return std::min((T + kWarps - 1) / kWarps, kMaxCtas);
}

template <int NPER>
cudaError_t launch_route(RouteArgs p, cudaStream_t s) {
  const int n = ctas_of(p.T);
  p.tokens = (p.T + n - 1) / n;
  const unsigned grid = static_cast<unsigned>((p.T + p.tokens - 1) / p.tokens);
  const size_t smem = sizeof(int) * (2 * p.E + 1 + static_cast<size_t>(kWarps) * p.E);
  k_route_count<NPER><<<grid, kThreads, smem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || grid == 1) return e;
  k_route_place<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

bool route_shape_ok(int T, int E, int k) {
  return T >= 0 && E >= 1 && E <= PW_MAX_GROUPS && k >= 1 && k <= E && static_cast<int64_t>(T) * k <= PW_MAX_VOCAB;
}

}  // namespace
}  // namespace pw

extern "C" {

size_t pw_route_workspace_bytes(int T, int E, int k) {
  if (!pw::route_shape_ok(T, E, k)) return 0;
  const int n = pw::ctas_of(T);
  return n > 1 ? static_cast<size_t>(n) * E * sizeof(int32_t) : 0;
}

int pw_route(const float* logits, int64_t ld, int T, int E, int k, int renorm, int32_t* idx, float* weight,
             int32_t* offsets, int32_t* perm, int32_t* inv, void* workspace, size_t ws_bytes, pw_stream_t s) {
  using namespace pw;
  NvtxCall nvtx_range("pw_route");
  if (!route_shape_ok(T, E, k))
    return failf(PW_EINVAL, "pw_route: need T >= 0, 1 <= E <= %d, 1 <= k <= E, T * k <= %d (T %d, E %d, k %d)",
                 PW_MAX_GROUPS, PW_MAX_VOCAB, T, E, k);
  if (!offsets || !aligned(offsets, 4)) return failf(PW_EINVAL, "pw_route: null or misaligned offsets");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  if (T == 0) return launch_status(cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (E + 1), st), "pw_route");
  if (!logits || !idx || !weight || !perm || !inv) return failf(PW_EINVAL, "pw_route: null logits or output");
  if (ld < E) return failf(PW_EINVAL, "pw_route: the row stride is below E = %d", E);
  if (!aligned(logits, 4) || !aligned(idx, 4) || !aligned(weight, 4) || !aligned(perm, 4) || !aligned(inv, 4))
    return failf(PW_EINVAL, "pw_route: misaligned pointer");
  const size_t need = pw_route_workspace_bytes(T, E, k);
  if (ws_bytes < need || (need && !workspace))
    return failf(PW_ENOMEM, "pw_route: workspace of %zu bytes, %zu are needed", workspace ? ws_bytes : 0, need);
  if (need && !aligned(workspace, 4)) return failf(PW_EINVAL, "pw_route: the workspace must be 4-byte aligned");
  const RouteArgs a{logits, ld, idx, weight, offsets, perm, inv, static_cast<int32_t*>(workspace), T, E, k, renorm, 0};
  const cudaError_t e = E <= 32    ? launch_route<1>(a, st)
                        : E <= 64  ? launch_route<2>(a, st)
                        : E <= 128 ? launch_route<4>(a, st)
                        : E <= 256 ? launch_route<8>(a, st)
                                   : launch_route<16>(a, st);
  return launch_status(e, "pw_route");
}

}  // extern "C"
