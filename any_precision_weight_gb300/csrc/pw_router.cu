// Routing on its own (pw_route): for every token the top-k experts by logit (ties to
// the lower index) with their softmax weights, and the routed pairs t * k + j in
// (expert, token) order with every expert's first place among them.
//
//   weight[t][j] = exp(logit_j - max) / sum, the sum over all experts, or over the k
//   chosen ones (renorm)
//
// A warp takes a token.  Up to kSmallTokens tokens one CTA does everything (one launch,
// bound by its latencies): it counts its pairs by expert and places them by a counting sort.
// Above, a second launch has CTAs for one, two or four experts each: a CTA reads the experts
// of all pairs twice, first counting those before its own experts and its own, then placing
// its own in their order.  So no CTA needs another's results, and there is no workspace; 8192
// x 60, 4 each, reads 8 MB from the L2 for it.  4 x 60, 4 each, 3.5 us, 256 x 60 3.8, 2048 x 60
// 5.6, 8192 x 60 10 to 11: launches, latencies and, in the largest, the issue slots of the choice.

#include <algorithm>
#include <cmath>

#include "pw_rows.cuh"

namespace pw {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSmallTokens = 32;
constexpr int kMaxCtas = 128;   // of the second launch

struct RouteArgs {
  const float* logits;
  int64_t ld;
  int32_t* idx;
  float* weight;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv;
  int T, E, k, renorm;
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
__device__ __forceinline__ void route_token(const RouteArgs& p, int64_t t) {
  const int lane = threadIdx.x & 31;
  float v[NPER];
  uint32_t key[NPER];   // 0: taken, or past E
#pragma unroll
  for (int i = 0; i < NPER; ++i) v[i] = lane + 32 * i < p.E ? __ldg(p.logits + t * p.ld + lane + 32 * i) : -INFINITY;
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

// Places all pairs by one CTA: warps count runs of them, the counts are scanned into each
// warp's first places behind base[e], and each warp places its run 32 at a time.
// s_c: [kWarps][E].
__device__ __forceinline__ void place_pairs(const RouteArgs& p, const int* base, int* s_c) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = p.E, P = p.T * p.k;
  const int run = (P + kWarps - 1) / kWarps;
  const int a = min(P, warp * run), z = min(P, a + run);
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

// A small batch by one CTA.
template <int NPER>
__global__ void __launch_bounds__(kThreads) k_route_small(const RouteArgs p) {
  extern __shared__ int s_mem[];   // counts [E + 1], then [kWarps][E]
  after_those_before();
  let_next_begin();
  for (int e = threadIdx.x; e < p.E; e += kThreads) s_mem[e] = 0;
  for (int t = threadIdx.x >> 5; t < p.T; t += kWarps) route_token<NPER>(p, t);
  __syncthreads();
  for (int q = threadIdx.x; q < p.T * p.k; q += kThreads) atomicAdd(&s_mem[p.idx[q]], 1);
  __syncthreads();
  if (threadIdx.x < 32) scan_counts(s_mem, p.E);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += kThreads) p.offsets[e] = s_mem[e];
  place_pairs(p, s_mem, s_mem + p.E + 1);
}

template <int NPER>
__global__ void __launch_bounds__(256) k_route_tokens(const RouteArgs p) {
  after_those_before();
  let_next_begin();
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t < p.T) route_token<NPER>(p, t);
}

// The pairs of the experts G blockIdx.x + 0 .. G - 1, by warps that take a run of all pairs
// each.
template <int G, int W>
__global__ void __launch_bounds__(W * 32) k_route_place(const RouteArgs p) {
  constexpr int U = W / 2;   // reads on their way together
  __shared__ int s_n[W][G + 1];
  after_those_before();
  let_next_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = blockIdx.x * G;
  const int64_t P = static_cast<int64_t>(p.T) * p.k;
  const int64_t run = (P + W * 32 - 1) / (W * 32) * 32, a = min(P, warp * run), z = min(P, a + run);
  // f(expert of this lane's pair, or -1, and the pair) for the warp's pairs in order
  auto each = [&](auto&& f) {
    for (int64_t b = a; b < z; b += 32 * U) {
      int v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = b + u * 32 + lane < z ? p.idx[b + u * 32 + lane] : -1;
#pragma unroll
      for (int u = 0; u < U; ++u) f(v[u], static_cast<int>(b + u * 32 + lane));
    }
  };
  int n[G + 1] = {};   // of the experts before, and of each of its own
  each([&](int e, int) {
    n[0] += e >= 0 && e < e0;
#pragma unroll
    for (int g = 0; g < G; ++g) n[g + 1] += e == e0 + g;
  });
#pragma unroll
  for (int g = 0; g <= G; ++g) {
    const int sum = __reduce_add_sync(0xffffffffu, n[g]);
    if (lane == 0) s_n[warp][g] = sum;
  }
  __syncthreads();
  // a lane has a warp's counts
  auto sum_of = [&](int g, int warps) { return __reduce_add_sync(0xffffffffu, lane < warps ? s_n[lane][g] : 0); };
  int at[G], first = sum_of(0, W);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (threadIdx.x == 0 && e0 + g <= p.E) p.offsets[e0 + g] = first;
    at[g] = first + sum_of(g + 1, warp);
    first += sum_of(g + 1, W);
  }
  if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) p.offsets[p.E] = first;
  each([&](int e, int q) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const unsigned same = __ballot_sync(0xffffffffu, e == e0 + g);
      if (e == e0 + g) {
        const int pos = at[g] + __popc(same & ((1u << lane) - 1u));
        p.perm[pos] = q;
        p.inv[q] = pos;
      }
      at[g] += __popc(same);
    }
  });
}

// 16 warps to a CTA, or 32: 256 x 60, 4 each, 4.5 us and 6.2; 8192 x 60 13.1 and 10.4.
template <int G>
cudaError_t launch_place(const RouteArgs& p, bool many, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((p.E + G - 1) / G);
  if (many) return launch_close(k_route_place<G, 32>, grid, 1024, 0, 1, s, p);
  return launch_close(k_route_place<G, 16>, grid, 512, 0, 1, s, p);
}

template <int NPER>
cudaError_t launch_route(const RouteArgs& p, cudaStream_t s) {
  if (p.T <= kSmallTokens)
    return launch_close(k_route_small<NPER>, 1, kThreads, sizeof(int) * (p.E + 1 + static_cast<size_t>(kWarps) * p.E), 1, s, p);
  const cudaError_t e = launch_close(k_route_tokens<NPER>, (p.T + 7) / 8, 256, 0, 1, s, p);
  if (e != cudaSuccess) return e;
  const bool many = static_cast<int64_t>(p.T) * p.k > 8192;
  if (p.E <= kMaxCtas) return launch_place<1>(p, many, s);
  if (p.E <= 2 * kMaxCtas) return launch_place<2>(p, many, s);
  return launch_place<4>(p, many, s);
}

bool route_shape_ok(int T, int E, int k) {
  return T >= 0 && E >= 1 && E <= PW_MAX_GROUPS && k >= 1 && k <= E && static_cast<int64_t>(T) * k <= PW_MAX_VOCAB;
}

}  // namespace
}  // namespace pw

extern "C" {

int pw_route(const float* logits, int64_t ld, int T, int E, int k, int renorm, int32_t* idx, float* weight,
             int32_t* offsets, int32_t* perm, int32_t* inv, pw_stream_t s) {
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
  const RouteArgs a{logits, ld, idx, weight, offsets, perm, inv, T, E, k, renorm};
  const cudaError_t e = E <= 32    ? launch_route<1>(a, st)
                        : E <= 64  ? launch_route<2>(a, st)
                        : E <= 128 ? launch_route<4>(a, st)
                        : E <= 256 ? launch_route<8>(a, st)
                                   : launch_route<16>(a, st);
  return launch_status(e, "pw_route");
}

}  // extern "C"
