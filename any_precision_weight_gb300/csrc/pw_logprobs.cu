// Log probabilities of given tokens with entropy, rank and top alternatives
// (pw_logprobs).
//
// In base 2, with L = log2 e and b a whole number at or just above max x * L:
//   s = sum 2^(x L - b),  u = sum (x L - b) 2^(x L - b)
//   logprob = (x[id] L - b - log2 s) / L;  entropy = (log2 s - u / s) / L
//   rank = #{x > x[id]} + #{x = x[id] at a lower index}
//   alternatives: the largest x by (value descending, index ascending)
// A whole b costs no rounding, and a thread that finds a larger b scales its
// sums by a power of two.
//
// One pass over the row for the sums, the rank and the largest element of each
// thread's batch (16 elements), kept in 16 bits.  The k-th largest of groups of
// the threads' largest elements is a bound that at least k elements reach, so
// only the batches that reach it, about k of them, are read again for the
// alternatives.  A row
// that few rows leave SMs for is split over a cluster of CTAs, whose results
// CTA 0 joins through distributed shared memory.
//
// Bound by HBM for many rows of 32-bit logits; 16-bit logits are near the
// issue rate, hence the paired arithmetic (f32x2, and 16-bit pairs for maxima
// and comparisons).  2048 x 131072: fp16 without alternatives 88 us, 6.1 TB/s,
// 90 % of the copy rate; bf16 with 20 of them 112 us, 4.8 TB/s, 70 %.  One row of
// 131072 fp32, 5 alternatives: 6.6 us of latencies.

#include <cmath>

#include "pw_rows.cuh"

namespace pw {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 16;
constexpr int kKept = 48;                           // batches of a thread whose largest elements are kept
constexpr int kCand = kWarps * 32;                  // batches or elements that reach the bound, before another way is taken
constexpr float kL = 1.44269504088896340736f;       // log2 e
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLeast = -1e30f;                    // least distance of two bases that is told apart

struct LogArgs {
  const void* x;
  const void* ids;       // int32 or int64, or null
  float* logprob;        // with ids
  int32_t* rank;         // with ids, or null
  float* entropy;        // or null
  int32_t* top_ids;      // [T][top]
  float* top_logprobs;   // [T][top]
  int64_t ld;
  int V, top, ids64;
};

using u64 = unsigned long long;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ u64 pair(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What differs by element type.  Elements are cut below at kLow before they
// meet the sums, so that masked ones (-inf) stay finite and the rounding of
// x L stays small; rows whose largest element is not above kSlowBelow, or is
// above kSlowAbove (where whole bases lose their last bit), go through slow_row.
template <typename T> struct Type;
template <> struct Type<float> {
  static constexpr float kLow = -0x1p29f, kSlowBelow = -0x1p22f, kSlowAbove = 0x1p22f;
  using B = __nv_bfloat16;   // a batch's largest element, not rounded down
  static __device__ __forceinline__ B above(float v) { return __float2bfloat16_ru(v); }
};
template <> struct Type<__nv_bfloat16> {
  using P = __nv_bfloat162;
  using B = __nv_bfloat16;
  static __device__ __forceinline__ B above(float v) { return __float2bfloat16_rn(v); }
  static constexpr float kLow = -0x1p29f, kSlowBelow = -0x1p22f, kSlowAbove = 0x1p22f;
  static __device__ __forceinline__ float2 wide(P v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ P both(float v) { return __float2bfloat162_rn(v); }
};
template <> struct Type<__half> {
  using P = __half2;
  using B = __half;
  static __device__ __forceinline__ B above(float v) { return __float2half_rn(v); }
  static constexpr float kLow = -65504.f, kSlowBelow = -65504.f, kSlowAbove = 65504.f;
  static __device__ __forceinline__ float2 wide(P v) { return __half22float2(v); }
  static __device__ __forceinline__ P both(float v) { return __float2half2_rn(v); }
};

// Sums over some elements, relative to the base b (a whole number).
struct Stat {
  float m, b, s, u;   // largest element (no NaN); base; sums
  int before;         // elements that come before the given token
};

// The sums' factor and shift for a larger base.
__device__ __forceinline__ float raise(float b, float to, float& d) {
  d = fmaxf(b - to, kLeast);
  return exp2_approx(b - to);
}

// The joined sums of a warp's lanes, in every lane.
__device__ __forceinline__ Stat join_lanes(Stat st) {
  const float b = static_cast<float>(__reduce_max_sync(0xffffffffu, __float2int_rn(st.b)));   // whole
  float d;
  const float f = raise(st.b, b, d);
  st.u = (st.u + d * st.s) * f;
  st.s *= f;
  st.b = b;
  st.before = __reduce_add_sync(0xffffffffu, st.before);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
    st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
    st.u += __shfl_xor_sync(0xffffffffu, st.u, o);
  }
  return st;
}

constexpr float kNoBase = -1e10f;   // below every base
__device__ __forceinline__ Stat no_stat() { return Stat{-INFINITY, kNoBase, 0.f, 0.f, 0}; }

// The least number of type T above x (+inf becomes NaN: nothing is above it).
template <typename T>
__device__ __forceinline__ float next_up(float x) {
  if (sizeof(T) == 4) {
    if (x == 0.f) return __uint_as_float(1u);
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float(b & 0x80000000u ? b - 1 : b + 1);
  }
  const T t = from_f32<T>(x);
  uint16_t b = *reinterpret_cast<const uint16_t*>(&t);
  b = x == 0.f ? 1 : b & 0x8000u ? b - 1 : b + 1;
  return to_f32<T>(*reinterpret_cast<const T*>(&b));
}

// The sums of one thread.  The given token's logit is met with >= by the
// vectors of lower index and with > by the others; its own vector's share of
// equal elements before it is added apart.
template <typename T>
struct Sums {
  static constexpr int VE = 16 / sizeof(T);
  float m = -INFINITY, b = kNoBase;
  u64 s2 = 0, u2 = 0;
  int before = 0;

  // NV vectors; t[i]: the least value in vector i that comes before the token.
  // Returns the largest element.
  template <int NV>
  __device__ __forceinline__ float add(const uint4 (&raw)[NV], const float (&t)[NV]) {
    constexpr int NP = NV * VE / 2;
    u64 x2[NP];
    float bm;
    if constexpr (sizeof(T) == 4) {
      bm = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float e[4] = {__uint_as_float(raw[i].x), __uint_as_float(raw[i].y), __uint_as_float(raw[i].z),
                            __uint_as_float(raw[i].w)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bm = fmaxf(bm, e[j]);
          before += e[j] >= t[i] ? 1 : 0;
        }
        x2[2 * i] = pair(max_nan(e[0], Type<T>::kLow), max_nan(e[1], Type<T>::kLow));
        x2[2 * i + 1] = pair(max_nan(e[2], Type<T>::kLow), max_nan(e[3], Type<T>::kLow));
      }
    } else {
      using P = typename Type<T>::P;
      const P low = Type<T>::both(Type<T>::kLow);
      P mx = *reinterpret_cast<const P*>(&raw[0].x);
      uint32_t cnt = 0;   // two 16-bit counts
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const P tt = Type<T>::both(t[i]);
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const P e = *reinterpret_cast<const P*>(&w[j]);
          mx = __hmax2(mx, e);
          cnt += __hge2_mask(e, tt) & 0x00010001u;
          const float2 f = Type<T>::wide(__hmax2_nan(e, low));
          x2[i * 4 + j] = pair(f.x, f.y);
        }
      }
      const float2 f = Type<T>::wide(mx);
      bm = fmaxf(f.x, f.y);
      before += (cnt & 0xffff) + (cnt >> 16);
    }
    m = fmaxf(m, bm);
    base(bm);
    const u64 nb2 = pair(-b, -b), l2 = pair(kL, kL);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const u64 y2 = fma2(x2[i], l2, nb2);
      const float2 y = unpair(y2);
      const u64 e2 = pair(exp2_approx(y.x), exp2_approx(y.y));
      s2 = add2(s2, e2);
      u2 = fma2(y2, e2, u2);
    }
    return bm;
  }
  __device__ __forceinline__ void base(float x) {
    const float nb = ceilf(fmaxf(x, Type<T>::kLow) * kL);
    if (nb > b) {
      float d;
      const float f = raise(b, nb, d);
      u2 = fma2(pair(d, d), s2, u2);
      s2 = fma2(s2, pair(f, f), 0);
      u2 = fma2(u2, pair(f, f), 0);
      b = nb;
    }
  }
  __device__ __forceinline__ void single(float x, float t) {
    before += x >= t ? 1 : 0;
    m = fmaxf(m, x);
    base(x);
    const float y = fmaf(max_nan(x, Type<T>::kLow), kL, -b), e = exp2_approx(y);
    s2 = add2(s2, pair(e, 0.f));
    u2 = add2(u2, pair(y * e, 0.f));
  }
  __device__ __forceinline__ Stat stat() const {
    const float2 s = unpair(s2), u = unpair(u2);
    return Stat{m, b, s.x + s.y, u.x + u.y, before};
  }
};

// ---------------------------------------------------------------- alternatives

// A key is the value's bits in ascending order above the complement of the
// index: no two are equal, and 0 is none.
__device__ __forceinline__ u64 key_of(float x, int idx) {
  const uint32_t b = __float_as_uint(x + 0.f);   // -0 and +0 are equal
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return static_cast<u64>(o) << 32 | static_cast<uint32_t>(~idx);
}
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// The larger half of two descending lists of 32 (one value a lane), descending.
template <typename K>
__device__ __forceinline__ K merge32(K a, K other, int lane) {
  const K o = __shfl_sync(0xffffffffu, other, 31 - lane);
  if (o > a) a = o;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const K v = __shfl_xor_sync(0xffffffffu, a, d);
    if (((lane & d) == 0) == (v > a)) a = v;
  }
  return a;
}

// A warp's values, one a lane, in descending order.
template <typename K>
__device__ __forceinline__ K sort32(K a, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int d = k >> 1; d; d >>= 1) {
      const K v = __shfl_xor_sync(0xffffffffu, a, d);
      const bool larger = ((lane & d) == 0) == ((lane & k) == 0 || k == 32);
      if (larger == (v > a)) a = v;
    }
  return a;
}

// Joins the warps' lists (descending, one value a lane) into warp 0's.
__device__ __forceinline__ u64 merge_warps(u64 a, u64 (*sh)[32], int warp, int lane) {
#pragma unroll
  for (int n = kWarps / 2; n; n >>= 1) {
    if (warp >= n && warp < 2 * n) sh[warp][lane] = a;
    __syncthreads();
    if (warp < n) a = merge32(a, sh[warp + n][lane], lane);
  }
  return a;
}

// A warp's 32 largest keys so far, descending over the lanes.
struct TopList {
  u64 key = 0, last = 0;   // last: the key at place `top`
  __device__ __forceinline__ void offer(u64 k, bool valid, int top, int lane) {
    unsigned mask = __ballot_sync(0xffffffffu, valid && k > last);
    while (mask) {
      const u64 c = __shfl_sync(0xffffffffu, k, __ffs(mask) - 1);
      mask &= mask - 1;
      if (c <= last) continue;
      const int pos = __popc(__ballot_sync(0xffffffffu, key > c));
      const u64 up = __shfl_up_sync(0xffffffffu, key, 1);
      if (lane >= pos) key = lane == pos ? c : up;
      last = __shfl_sync(0xffffffffu, key, top - 1);
    }
  }
};

// ---------------------------------------------------------------- kernel

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared variable of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return a;
}
__device__ __forceinline__ float ld_cluster_f(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ u64 ld_cluster_k(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}

// Rows whose largest element is at an end of the number range (masks of the
// type's lowest value that leave nothing, rows of -inf, infinities): sums of
// e^(x - m), in natural units, by one CTA.  Returned as a Stat with b = 0:
// s and u scaled to base 2.
template <typename T>
__device__ __noinline__ Stat slow_row(const T* x, int V, float m, Stat* sh) {
  Stat st{m, 0.f, 0.f, 0.f, 0};
  for (int i = threadIdx.x; i < V; i += kThreads) {
    const float xi = to_f32<T>(x[i]);
    if (xi == -INFINITY) continue;
    const float y = fmaxf(xi - m, kLeast) * kL, e = xi != xi || m == INFINITY ? NAN : exp2_approx(y);
    st.s += e;
    st.u += y * e;
  }
  st = join_lanes(st);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = st;
  __syncthreads();
  st = sh[0];
  for (int w = 1; w < kWarps; ++w) st.s += sh[w].s, st.u += sh[w].u;
  st.m = m;
  return st;
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) k_logprobs(const LogArgs p, int split) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int NV = 2 * (sizeof(T) / 2);        // vectors of a batch: 16 elements a thread
  __shared__ Stat s_stat[kWarps], s_cta;
  __shared__ u64 s_cand[kCand], s_top[32];
  __shared__ float s_group[64];
  __shared__ typename Type<T>::B s_batch[TOP ? kKept : 1][kThreads];
  __shared__ int s_at[TOP ? kCand : 1];
  __shared__ int s_count, s_found;
  u64(*s_list)[32] = reinterpret_cast<u64(*)[32]>(s_cand);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x / split;
  const int rank = blockIdx.x % split;
  const T* x = static_cast<const T*>(p.x) + row * p.ld;

  long long id64 = -1;
  if (p.ids) id64 = p.ids64 ? static_cast<const long long*>(p.ids)[row] : static_cast<const int32_t*>(p.ids)[row];
  const bool has = id64 >= 0 && id64 < p.V;
  const int id = has ? static_cast<int>(id64) : -1;
  const float xt = has ? to_f32<T>(x[id]) : NAN;
  const float xt_up = next_up<T>(xt);

  // elements before the first 16-byte boundary, whole vectors, the rest; this
  // CTA's share of the vectors
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % VE);
  const int head = min(p.V, (VE - off) % VE);
  const int nvec = (p.V - head) / VE;
  const int done = head + nvec * VE;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  const int va = static_cast<int>(static_cast<int64_t>(nvec) * rank / split);
  const int vb = static_cast<int>(static_cast<int64_t>(nvec) * (rank + 1) / split);
  const int vid = id >= head && id < done ? (id - head) / VE : id < head ? -1 : nvec;   // the token's vector
  const int vlow = min(vid, vb);   // this CTA's vectors below it are met with >=
  const bool do_head = rank == 0 && warp == 0, do_tail = rank == split - 1 && warp == kWarps - 1;

  Sums<T> sums;
  if (do_head && lane < head) sums.single(to_f32<T>(x[lane]), lane < id ? xt : xt_up);
  const uint32_t ninf = sizeof(T) == 4 ? 0xff800000u : Type<T>::kLow == -65504.f ? 0xfc00fc00u : 0xff80ff80u;
  const uint4 none = make_uint4(ninf, ninf, ninf, ninf);
  constexpr int kStep = kThreads * NV;
  const int first = va + warp * NV * 32 + lane;
  uint4 next[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) next[i] = first + i * 32 < vb ? __ldg(xv + first + i * 32) : none;
  // 2^ws batches of a thread share a place among those kept
  int ws = 0;
  while (TOP && (vb - va + kStep - 1) / kStep > kKept << ws) ++ws;
  float wm = -INFINITY;
  int batch = 0;
  for (int v = first; v - lane < vb; v += kStep) {
    uint4 raw[NV];
    float t[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      raw[i] = next[i];
      t[i] = v + i * 32 < vlow ? xt : xt_up;
      const int n = v + kStep + i * 32;
      next[i] = n < vb ? __ldg(xv + n) : none;
    }
    const float bm = sums.template add<NV>(raw, t);
    if (TOP) {
      wm = fmaxf(batch & ((1 << ws) - 1) ? wm : -INFINITY, bm);
      s_batch[batch >> ws][threadIdx.x] = Type<T>::above(wm);
      ++batch;
    }
  }
  if (do_tail && done + lane < p.V) sums.single(to_f32<T>(x[done + lane]), done + lane < id ? xt : xt_up);
  // the token's own vector was met with > throughout: its equal elements before the token
  if (rank == 0 && warp == 0 && vid >= 0 && vid < nvec) {
    const int i = head + vid * VE + lane;
    if (lane < VE && i < id && to_f32<T>(x[i]) == xt) ++sums.before;
  }

  {
    const Stat st = join_lanes(sums.stat());
    if (lane == 0) s_stat[warp] = st;
  }
  u64 best = 0;
  if constexpr (TOP) {
    // the bound: the top-th largest of 64 groups' largest elements (4 threads
    // each), so that some 64 ln(64 / (64 - top)) elements reach it: 24 for 20
    float gm = fmaxf(sums.m, __shfl_xor_sync(0xffffffffu, sums.m, 1));
    gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
    if ((lane & 3) == 0) s_group[threadIdx.x >> 2] = gm;
    if (threadIdx.x == 0) s_count = s_found = 0;
    __syncthreads();
    const float thr = __shfl_sync(
        0xffffffffu, merge32(sort32(s_group[lane], lane), sort32(s_group[lane + 32], lane), lane), p.top - 1);
    // the kept batches that reach it, and then their elements
    if (sums.m >= thr) {
      const int kept = (batch + (1 << ws) - 1) >> ws;
#pragma unroll 8
      for (int k = 0; k < kept; ++k) {
        if (static_cast<float>(s_batch[k][threadIdx.x]) >= thr) {
          const int pos = atomicAdd(&s_found, 1);
          if (pos < kCand) s_at[pos] = k * kThreads + threadIdx.x;
        }
      }
    }
    __syncthreads();
    const int found = s_found;
    auto keep = [&](float e, int i) {
      if (e >= thr) {
        const int pos = atomicAdd(&s_count, 1);
        if (pos < kCand) s_cand[pos] = key_of(e, i);
      }
    };
    if (found <= kCand) {
      if (do_head && lane < head) keep(to_f32<T>(x[lane]), lane);
      if (do_tail && done + lane < p.V) keep(to_f32<T>(x[done + lane]), done + lane);
      const int per = NV << ws;   // vectors of a kept place
      for (int i = threadIdx.x; i < found * per; i += kThreads) {
        const int at = s_at[i / per], n = i % per, k = at / kThreads, owner = at % kThreads;
        const int v = va + (owner >> 5) * NV * 32 + (owner & 31) + ((k << ws) + n / NV) * kStep + n % NV * 32;
        if (v >= vb) continue;
        float e[VE];
        unpack16<T>(__ldg(xv + v), e);
#pragma unroll
        for (int j = 0; j < VE; ++j) keep(e[j], head + v * VE + j);
      }
    }
    __syncthreads();
    const int n = s_count;
    if (found <= kCand && n <= kCand) {
      if (warp == 0) {
        for (int i = 0; i < n; i += 32) {
          const u64 k = sort32(i + lane < n ? s_cand[i + lane] : u64(0), lane);
          best = i ? merge32(best, k, lane) : k;
        }
      }
    } else {   // many equal elements: every element once more, into a list in each warp
      TopList list;
      auto offer = [&](float e, int i, bool exists) { list.offer(key_of(e, i), exists && e >= thr, p.top, lane); };
      if (do_head) offer(lane < head ? to_f32<T>(x[lane]) : 0.f, lane, lane < head);
      if (do_tail) offer(done + lane < p.V ? to_f32<T>(x[done + lane]) : 0.f, done + lane, done + lane < p.V);
      for (int k = 0; k < batch; ++k) {
        if (!__any_sync(0xffffffffu, static_cast<float>(s_batch[k >> ws][threadIdx.x]) >= thr)) continue;
#pragma unroll 1
        for (int i = 0; i < NV; ++i) {
          const int v = first + k * kStep + i * 32;
          float e[VE];
          unpack16<T>(v < vb ? __ldg(xv + v) : none, e);
#pragma unroll
          for (int j = 0; j < VE; ++j) offer(e[j], head + v * VE + j, v < vb);
        }
      }
      __syncthreads();
      best = merge_warps(list.key, s_list, warp, lane);
    }
  } else {
    __syncthreads();
  }

  // this CTA's results, and the cluster's in CTA 0
  if (warp == 0) {
    Stat st = lane < kWarps ? s_stat[lane] : no_stat();
    st = join_lanes(st);
    if (lane == 0) s_cta = st;
    if (TOP) s_top[lane] = best;
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    if (rank == 0) {
      if (warp == 0) {
        Stat st = no_stat();
        if (lane < split) {
          const uint32_t a = in_cta(&s_cta, lane);
          st = Stat{ld_cluster_f(a), ld_cluster_f(a + 4), ld_cluster_f(a + 8), ld_cluster_f(a + 12),
                    __float_as_int(ld_cluster_f(a + 16))};
        }
        st = join_lanes(st);
        if (lane == 0) s_cta = st;
      }
      if (TOP) {
        u64 a = warp < split ? ld_cluster_k(in_cta(&s_top[lane], warp)) : 0;
        if (warp + kWarps < split) a = merge32(a, ld_cluster_k(in_cta(&s_top[lane], warp + kWarps)), lane);
        __syncthreads();
        best = merge_warps(a, s_list, warp, lane);
      }
    }
    __syncwarp();
    cluster_sync();
    if (rank) return;
  }
  __syncthreads();
  Stat st = s_cta;
  const bool slow = !(st.m > Type<T>::kSlowBelow) || st.m > Type<T>::kSlowAbove;
  if (slow && (st.m != -INFINITY || st.s == st.s)) {
    const int before = st.before;
    st = slow_row<T>(x, p.V, st.m, s_stat);
    st.before = before;
  }
  if (warp) return;
  // log2 of an element's probability; -inf where nothing has any
  const bool empty = st.m == -INFINITY && st.s == 0.f;
  const float ls = log2f(st.s);
  auto logp = [&](float v) {
    if (empty) return -INFINITY;
    if (!slow && v < -1e30f) return v - (st.b + ls) * kLn2;   // v L would overflow
    return ((slow ? (v - st.m) * kL : fmaf(v, kL, -st.b)) - ls) * kLn2;
  };
  if (lane == 0) {
    if (p.ids) {
      if (p.logprob) p.logprob[row] = has ? logp(xt) : 0.f;
      if (p.rank) p.rank[row] = !has || xt != xt ? -1 : st.before;
    }
    if (p.entropy) p.entropy[row] = empty ? 0.f : (ls - st.u / st.s) * kLn2;
  }
  if (TOP && lane < p.top) {
    p.top_ids[row * p.top + lane] = best ? static_cast<int32_t>(~static_cast<uint32_t>(best)) : -1;
    p.top_logprobs[row * p.top + lane] = best ? logp(key_value(best)) : NAN;
  }
}

template <typename T, bool TOP>
cudaError_t launch_top(const LogArgs& p, int T_, cudaStream_t s) {
  // a row is split until every SM has a CTA, each with 2048 elements or more;
  // until every SM has two was slower (33 x 50001 fp16, 32 alternatives: 7.8 and
  // 9.6 us; 256 x 32000: 10.7 and 12.9)
  const int sms = sm_count();
  int split = 1;
  while (split < kMaxCluster && static_cast<int64_t>(T_) * split < sms && p.V >= 4096 * split) split *= 2;
  if (static_cast<int64_t>(T_) * split > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (split > 8) {
    const cudaError_t e = cudaFuncSetAttribute(k_logprobs<T, TOP>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(T_) * split);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cfg.attrs = &a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_logprobs<T, TOP>, p, split);
}

template <typename T>
cudaError_t launch_logprobs(const LogArgs& p, int T_, cudaStream_t s) {
  return p.top ? launch_top<T, true>(p, T_, s) : launch_top<T, false>(p, T_, s);
}

}  // namespace
}  // namespace pw

extern "C" int pw_logprobs(const void* logits, int64_t ld, int dtype, int T, int V, const void* ids, int ids64,
                           int top, float* logprob, int32_t* rank, float* entropy, int32_t* top_ids,
                           float* top_logprobs, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_logprobs");
  if (T < 0 || V < 1 || V > PW_MAX_VOCAB)
    return pw::failf(PW_EINVAL, "pw_logprobs: need T >= 0 and 1 <= V <= %d (T %d, V %d)", PW_MAX_VOCAB, T, V);
  if (!pw::dtype_ok(dtype)) return pw::failf(PW_EINVAL, "pw_logprobs: unknown dtype %d", dtype);
  if (top < 0 || top > PW_MAX_TOP || top > V)
    return pw::failf(PW_EINVAL, "pw_logprobs: top %d outside [0, min(V, %d)]", top, PW_MAX_TOP);
  if (T == 0) return PW_OK;
  if (!logits) return pw::failf(PW_EINVAL, "pw_logprobs: null logits");
  if (ld < V) return pw::failf(PW_EINVAL, "pw_logprobs: the row stride is below V = %d", V);
  if ((logprob || rank) && !ids) return pw::failf(PW_EINVAL, "pw_logprobs: logprob or rank without ids");
  if (top && (!top_ids || !top_logprobs)) return pw::failf(PW_EINVAL, "pw_logprobs: top without its outputs");
  if (!pw::aligned(logits, pw::dtype_bytes(dtype)) || !pw::aligned(ids, ids64 ? 8 : 4) || !pw::aligned(logprob, 4) ||
      !pw::aligned(rank, 4) || !pw::aligned(entropy, 4) || !pw::aligned(top_ids, 4) || !pw::aligned(top_logprobs, 4))
    return pw::failf(PW_EINVAL, "pw_logprobs: misaligned pointer");
  const pw::LogArgs a{logits, ids, logprob, rank, entropy, top_ids, top_logprobs, ld, V, top, ids64 ? 1 : 0};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(s);
  const cudaError_t e = dtype == PW_F16    ? pw::launch_logprobs<__half>(a, T, st)
                        : dtype == PW_BF16 ? pw::launch_logprobs<__nv_bfloat16>(a, T, st)
                                           : pw::launch_logprobs<float>(a, T, st);
  return pw::launch_status(e, "pw_logprobs");
}
