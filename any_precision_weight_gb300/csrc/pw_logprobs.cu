// Log probabilities of given tokens with entropy, rank and top alternatives
// (pw_logprobs).
//
//   m = max x,  s = sum e^(x - m),  u = sum (x - m) e^(x - m)
//   logprob = (x[id] - m) - ln s;  entropy = ln s - u / s
//   rank = #{x > x[id]} + #{x = x[id] at a lower index}
//   alternatives: the largest x by (value descending, index ascending)
//
// One pass over the row.  Every thread keeps its own running (m, s, u); every
// warp keeps a sorted list of its 32 largest keys, one per lane, and looks at
// single elements only when the largest of its batch reaches the list's k-th
// value.  A key is the value's bits in ascending order above the complement of
// the index, so no two keys are equal and the lists' joins need no tie rule.

#include <cmath>

#include "pw_rows.cuh"

namespace pw {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLeast = -1e30f;   // x - m of masked elements: finite, and so are its sums

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

struct Stat {
  float m, s, u;   // max, sum e^(x-m), sum (x-m) e^(x-m)
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Moves st to the larger maximum m.
__device__ __forceinline__ void raise_max(Stat& st, float m) {
  if (m > st.m) {
    if (st.m > -INFINITY) {   // nothing is in the sums before the first finite maximum
      const float d = st.m - m, c = exp2_approx(d * kLog2e);
      st.u = (st.u + fmaxf(d, kLeast) * st.s) * c;
      st.s *= c;
    }
    st.m = m;
  }
}

__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  raise_max(a, m);
  raise_max(b, m);
  return Stat{m, a.s + b.s, a.u + b.u};
}

// One element into st, whose maximum is at least x.  The base of a row that so
// far holds only -inf is 0, so that -inf - base stays -inf (e = 0); a masked
// element's (x - m) is cut to a finite value before it meets its e = 0.
__device__ __forceinline__ void add(Stat& st, float base, float x) {
  const float d = x - base, e = exp2_approx(d * kLog2e);
  st.s += e;
  st.u = fmaf(fmaxf(d, kLeast), e, st.u);
}

__device__ __forceinline__ unsigned long long key_of(float x, int idx) {
  const uint32_t b = __float_as_uint(x + 0.f);   // -0 and +0 are equal
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return static_cast<unsigned long long>(o) << 32 | static_cast<uint32_t>(~idx);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// The least float above x.
__device__ __forceinline__ float next_up(float x) {
  if (x == 0.f) return __uint_as_float(1u);
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float(b & 0x80000000u ? b - 1 : b + 1);   // +inf becomes NaN: no x is above it
}

// A warp's 32 largest keys, descending over the lanes (0: no key).
struct TopList {
  unsigned long long key;
  float thr;   // no x below it can enter the first `top` places

  __device__ __forceinline__ void insert(unsigned long long k, int lane) {
    const int pos = __popc(__ballot_sync(0xffffffffu, key > k));
    const unsigned long long up = __shfl_up_sync(0xffffffffu, key, 1);
    if (lane >= pos) key = lane == pos ? k : up;
  }
  // Elements come in ascending order of their index (batch by batch), so a
  // later one that equals the last kept value does not enter.
  __device__ __forceinline__ void refresh(int top) {
    const unsigned long long k = __shfl_sync(0xffffffffu, key, top - 1);
    thr = k ? next_up(key_value(k)) : -INFINITY;
  }
  // The 32 largest of this list and another one.
  __device__ __forceinline__ void merge(unsigned long long other, int lane) {
    const unsigned long long o = __shfl_sync(0xffffffffu, other, 31 - lane);
    if (o > key) key = o;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      const unsigned long long v = __shfl_xor_sync(0xffffffffu, key, d);
      const bool upper = (lane & d) == 0;
      if (upper == (v > key)) key = v;
    }
  }
};

// What one warp has seen of the row.
template <bool TOP>
struct Pass {
  Stat st{-INFINITY, 0.f, 0.f};
  TopList list{0, -INFINITY};
  int before = 0;     // elements that come before the given token
  float xt;           // the given token's logit (NaN: none)
  float xt_up;        // the least float above it
  int id, top, lane, V;

  // N elements of this lane, element j at index i0[j]; the warp's elements
  // come in ascending order from call to call.  Places past the row (index V
  // and above) hold -inf: they add nothing and are kept out of the list.
  template <int N>
  __device__ __forceinline__ void batch(const float (&x)[N], const int (&i0)[N]) {
    float bm = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) bm = fmaxf(bm, x[j]);
    raise_max(st, bm);
    const float base = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      add(st, base, x[j]);
      before += x[j] >= (i0[j] < id ? xt : xt_up) ? 1 : 0;
    }
    if (TOP && __any_sync(0xffffffffu, bm >= list.thr)) {
#pragma unroll 1
      for (int j = 0; j < N; ++j) {
        float v = x[0];
        int i = i0[0];
#pragma unroll
        for (int l = 1; l < N; ++l)
          if (l == j) v = x[l], i = i0[l];
        unsigned mask = __ballot_sync(0xffffffffu, v >= list.thr && i < V);
        if (!mask) continue;
        const unsigned long long k = key_of(v, i);
        while (mask) {
          list.insert(__shfl_sync(0xffffffffu, k, __ffs(mask) - 1), lane);
          mask &= mask - 1;
        }
      }
      list.refresh(top);
    }
  }
  // One element that only lanes with `valid` have.
  __device__ __forceinline__ void single(float x, int i, bool valid) {
    if (valid) {
      raise_max(st, x);
      add(st, st.m == -INFINITY ? 0.f : st.m, x);
      before += x >= (i < id ? xt : xt_up) ? 1 : 0;
    }
    if (TOP) {
      unsigned mask = __ballot_sync(0xffffffffu, valid && x >= list.thr);
      const unsigned long long k = key_of(x, i);
      while (mask) {
        list.insert(__shfl_sync(0xffffffffu, k, __ffs(mask) - 1), lane);
        mask &= mask - 1;
      }
      list.refresh(top);
    }
  }
};

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads) k_logprobs(const LogArgs p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int NV = 16 / VE;              // vectors of a batch: 16 elements a lane
  __shared__ Stat s_stat[kWarps];
  __shared__ int s_before[kWarps];
  __shared__ unsigned long long s_list[kWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ld;

  Pass<TOP> w;
  w.lane = lane;
  w.top = p.top;
  w.V = p.V;
  long long id = -1;
  if (p.ids) id = p.ids64 ? static_cast<const long long*>(p.ids)[row] : static_cast<const int32_t*>(p.ids)[row];
  const bool has = id >= 0 && id < p.V;
  w.id = has ? static_cast<int>(id) : -1;
  w.xt = has ? to_f32<T>(x[w.id]) : NAN;
  w.xt_up = next_up(w.xt);

  // elements before the first 16-byte boundary, whole vectors, the rest
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) / sizeof(T) % VE);
  const int head = min(p.V, (VE - off) % VE);
  const int nvec = (p.V - head) / VE;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  if (warp == 0 && head) w.single(lane < head ? to_f32<T>(x[lane]) : 0.f, lane, lane < head);
  for (int v0 = warp * NV * 32; v0 < nvec; v0 += kThreads * NV) {
    float e[16];
    int at[16];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = v0 + j * 32 + lane;
      float t[VE];
      if (v < nvec) {
        unpack16<T>(xv[v], t);
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) t[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < VE; ++i) e[j * VE + i] = t[i], at[j * VE + i] = v < nvec ? head + v * VE + i : p.V;
    }
    w.batch(e, at);
  }
  const int done = head + nvec * VE;
  if (warp == kWarps - 1 && done < p.V) {
    const bool ok = done + lane < p.V;
    w.single(ok ? to_f32<T>(x[done + lane]) : 0.f, done + lane, ok);
  }

  // join: lanes, then warps
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(0xffffffffu, w.st.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, w.st.s, o);
    b.u = __shfl_xor_sync(0xffffffffu, w.st.u, o);
    w.st = join(w.st, b);
  }
  w.before = __reduce_add_sync(0xffffffffu, w.before);
  if (lane == 0) {
    s_stat[warp] = w.st;
    s_before[warp] = w.before;
  }
  if (TOP) s_list[warp][lane] = w.list.key;
  __syncthreads();
  if (warp) return;
  Stat st = s_stat[0];
  int before = s_before[0];
  for (int i = 1; i < kWarps; ++i) {
    st = join(st, s_stat[i]);
    before += s_before[i];
    if (TOP) w.list.merge(s_list[i][lane], lane);
  }
  const float ls = logf(st.s);   // -inf for a row of -inf alone
  const bool empty = st.m == -INFINITY && st.s == 0.f;
  if (lane == 0) {
    if (p.ids) {
      if (p.logprob) p.logprob[row] = !has ? 0.f : empty ? -INFINITY : (w.xt - st.m) - ls;
      if (p.rank) p.rank[row] = !has || w.xt != w.xt ? -1 : before;
    }
    if (p.entropy) p.entropy[row] = empty ? 0.f : ls - st.u / st.s;
  }
  if (TOP && lane < p.top) {
    const unsigned long long k = w.list.key;
    p.top_ids[row * p.top + lane] = k ? static_cast<int32_t>(~static_cast<uint32_t>(k)) : -1;
    p.top_logprobs[row * p.top + lane] = !k ? NAN : empty ? -INFINITY : (key_value(k) - st.m) - ls;
  }
}

template <typename T>
cudaError_t launch_logprobs(const LogArgs& p, int T_, cudaStream_t s) {
  if (p.top)
    k_logprobs<T, true><<<T_, kThreads, 0, s>>>(p);
  else
    k_logprobs<T, false><<<T_, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace pw

extern "C" int pw_logprobs(const void* logits, int64_t ld, int dtype, int T, int V, const void* ids, int ids64,
                           int top, float* logprob, int32_t* rank, float* entropy, int32_t* top_ids,
                           float* top_logprobs, pw_stream_t s) {
  pw::NvtxCall nvtx_range("pw_logprobs");
  if (T < 0 || V < 1) return pw::failf(PW_EINVAL, "pw_logprobs: need T >= 0 and V >= 1 (T %d, V %d)", T, V);
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
