// Root-mean-square norm with the residual's addition, and int8 rows with a
// scale per row (pw_rms_norm, pw_quant_i8).
//
//   s = x + residual (fp32);  y = s * w / sqrt(mean(s^2) + eps)
//   scale = max|y| / 127;     q = rint(y / scale)
//
// A row stays in registers as fp32, so every input is read once.  Both row
// reductions, sum s^2 and max|s * w|, are taken in one pass and joined behind
// one barrier: max|y| = max|s * w| * rstd, and y / scale = s * w * 127 /
// max|s * w| does not need rstd at all.
//
// Bound by latency for few rows, by HBM for many: there one CTA per row leaves
// the memory idle while it reduces and stores (8192 x 4096 fp16 with residual
// and int8 output: 50 to 85 us), so persistent CTAs keep the next row's loads
// in flight (38 us, 6.1 TB/s, 90 % of the copy peak; 28672 x 4096 fp16 to int8:
// 63 us, 5.6 TB/s, 83 %; with one rounded factor, which sends halves of 16-bit
// inputs either way, 60).  One row of 4096: 2.1 us.

#include <algorithm>
#include <type_traits>

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

// One 16-byte load (a plain reference to it would be read element by element).
template <typename T>
__device__ __forceinline__ uint4 load16(const T* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// VE elements at element e0 of a row of H, as fp32 (0 past the end).
template <typename T, int VE>
__device__ __forceinline__ void load_chunk(const T* row, int e0, int H, float (&v)[VE]) {
  if constexpr (VE == 1) {
    v[0] = e0 < H ? to_f32<T>(row[e0]) : 0.f;
  } else {
    if (e0 + VE <= H) {
      unpack16<T>(load16(row + e0), v);
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

// Sum of `a` (where SUM) and largest `b` >= 0 over the CTA, in every thread.  The
// bits of numbers that are not negative are in their order, and NaN's are above
// them all.
template <bool SUM>
__device__ __forceinline__ void block_reduce(float& a, float& b, float2* sh) {
  auto warp_max = [](float v) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v))); };
  if (SUM) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  }
  b = warp_max(b);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = (threadIdx.x & 31) < nw ? sh[threadIdx.x & 31] : make_float2(0.f, 0.f);
  a = v.x;
  if (SUM) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  }
  b = warp_max(v.y);
}

// Squares of bf16 and fp32 rows leave fp32's range from 2^64 up, and below 2^-75
// where eps does not cover them.  Such rows take s times a power of two: y, q and
// y / max|y| do not change with it, and the sum of squares and eps take its square.
// fp16 rows (below 2^18 with a residual, no square under 2^-48) have no need of it.
constexpr float kLargeSum = 0x1p100f, kSmallSum = 0x1p-90f;   // of squares
constexpr float kDown = 0x1p-80f, kUp = 0x1p70f;
template <typename T, bool NORM> constexpr bool kRange = NORM && !std::is_same_v<T, __half>;
__device__ __forceinline__ bool too_large(float ss) { return !(ss <= kLargeSum); }   // and NaN
__device__ __forceinline__ bool too_small(float ss, float eps) { return ss < kSmallSum && eps < kSmallSum; }

// Factors of a row's outputs, v = s * w: y = v * rstd; q = 127 v / max, rounded,
// with v and max first times `up` where max is so small or large that a factor
// or product would leave fp32's range.  Rows without a step (zeros, NaN,
// infinities) have q 0.
struct RowScale {
  float rstd, scale;
  float steps, fine;   // 127 / max is steps + fine (fine where NORM does not hold)
  float up;
  bool far, none;
};
template <bool NORM>
__device__ __forceinline__ RowScale row_scale(float ss, float amax, int H, float eps) {
  RowScale f;
  const float whole = amax;
  const float ms = ss / static_cast<float>(H) + eps;
  f.rstd = !NORM ? 1.f : ms == 0.f ? 0.f : 1.f / sqrtf(ms);   // zeros without eps stay zeros
  f.none = !(amax > 0.f && amax < INFINITY);
  f.up = amax < 0x1p-100f ? 0x1p100f : amax > 0x1p100f ? 0x1p-100f : 1.f;
  f.far = f.up != 1.f;
  amax *= f.up;
  f.steps = 127.f / amax;
  if (!NORM) f.fine = fmaf(-f.steps, amax, 127.f) * f.steps * (1.f / 127.f);
  f.scale = whole * f.rstd;   // times 1 / 127, by the thread that stores it
  return f;
}

// Two fp32 numbers in one operation.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The steps of two values rounded to the nearest whole number (ties to even), in
// the low bytes: 1.5 * 2^23 is added, above which fp32 holds whole numbers only.
// Where v is an input itself (not NORM), ties are common (16-bit inputs have few
// digits), so the factor 127 / max is taken as two numbers: v times both, rounded
// once, makes a quotient that is a half come out as a half.
template <bool NORM>
__device__ __forceinline__ void to_steps(const RowScale& f, float va, float vb, uint32_t& a, uint32_t& b) {
  const uint64_t magic = pair2(12582912.f, 12582912.f), v = pair2(va, vb), steps = pair2(f.steps, f.steps);
  const uint64_t r = NORM ? fma2(v, steps, magic) : add2(fma2(v, steps, mul2(v, pair2(f.fine, f.fine))), magic);
  a = static_cast<uint32_t>(r);
  b = static_cast<uint32_t>(r >> 32);
}

template <int VE, bool NORM>
__device__ __forceinline__ void store_q(int8_t* row, int e0, int H, const float (&v)[VE], const RowScale& f) {
  uint32_t b[VE];
  auto at = [&](int i) { return f.far ? v[i] * f.up : v[i]; };
  if constexpr (VE == 1) {
    const float v0 = at(0);
    b[0] = __float_as_uint(NORM ? fmaf(v0, f.steps, 12582912.f) : fmaf(v0, f.steps, v0 * f.fine) + 12582912.f);
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 2) to_steps<NORM>(f, at(i), at(i + 1), b[i], b[i + 1]);
  }
  if (f.none) {
#pragma unroll
    for (int i = 0; i < VE; ++i) b[i] = 0;
  }
  if (VE > 1 && e0 + VE <= H) {
    uint32_t w[(VE + 3) / 4];
#pragma unroll
    for (int i = 0; i + 3 < VE; i += 4)
      w[i / 4] = __byte_perm(__byte_perm(b[i], b[i + 1], 0x0040), __byte_perm(b[i + 2], b[i + 3], 0x0040), 0x5410);
    if constexpr (VE == 8) *reinterpret_cast<uint2*>(row + e0) = make_uint2(w[0], w[1]);
    if constexpr (VE == 4) *reinterpret_cast<uint32_t*>(row + e0) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (e0 + i < H) row[e0 + i] = static_cast<int8_t>(b[i]);
  }
}

// Rows and two steps of a grid stay below 2^32.  A row's number is held in what
// takes fewer registers: with chunks of one element the compiler keeps 64-bit sums.
template <int VE> using RowIndex = std::conditional_t<VE == 1, int64_t, uint32_t>;

// A thread's chunks of a row, chunk c at element at(c): from v = x + residual
// to the row's outputs.  weight(c, g) gives the weights of chunk c; `own` is a slot of
// shared memory of the thread's own (where kRange).
template <typename T, int VE, int VPT, bool NORM, typename At, typename Weight>
__device__ __forceinline__ void finish_row(const RowArgs& p, RowIndex<VE> row, float (&v)[VPT][VE], float2* sh, float* own,
                                           At&& at, Weight&& weight) {
  const int H = p.H;
  float ss = 0.f, amax = 0.f, eps = p.eps;
  if (p.sum) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) store_chunk<T, VE>(static_cast<T*>(p.sum) + row * p.lds, at(c), H, v[c]);
  }
  // f(v) for all of the thread's values
  auto each = [&](auto&& f) {
#pragma unroll
    for (int c = 0; c < VPT; ++c)
#pragma unroll
      for (int i = 0; i < VE; ++i) f(v[c][i]);
  };
  // A thread whose own squares leave the range keeps v and their sum in another unit;
  // a large one adds nothing to the CTA's sum and makes the largest element infinite.
  bool down = false, up = false;
  if constexpr (kRange<T, NORM>) {
    each([&](float x) { ss = fmaf(x, x, ss); });
    down = too_large(ss), up = too_small(ss, eps);
    if (down || up) {
      const float u = up ? kUp : kDown;
      float sum = 0.f;
      each([&](float& x) { x *= u, sum = fmaf(x, x, sum); });
      *own = sum;   // no register for what hardly any row needs
      if (down) ss = 0.f;
    }
  }
#pragma unroll
  for (int c = 0; c < VPT; ++c) {
    float g[VE];
    if (NORM) weight(c, g);
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (NORM && !kRange<T, NORM>) ss = fmaf(v[c][i], v[c][i], ss);
      if (NORM) v[c][i] *= g[i];
      amax = max_nan(amax, fabsf(v[c][i]));
    }
  }
  if (down) amax = INFINITY;
  if (up) amax /= kUp;
  block_reduce<NORM>(ss, amax, sh);
  if constexpr (kRange<T, NORM>) {
    // (an infinite weight does not make a row large)
    const bool large = !(amax < INFINITY) && __syncthreads_or(down), small = !large && too_small(ss, eps);
    if (up && !small) each([&](float& x) { x /= kUp; });
    if (large || small) {   // the row in one unit; where it is small, kUp is every thread's
      const float u = large ? kDown : kUp;
      if (large && !down) each([&](float& x) { x *= kDown; });
      float sum = down || small ? *own : 0.f;
      amax = 0.f, eps *= u, eps *= u;
      each([&](float x) { amax = max_nan(amax, fabsf(x)); });
      __syncthreads();   // sh has been read
      block_reduce<NORM>(sum, amax, sh);
      ss = large ? fmaf(ss * kDown, kDown, sum) : sum;
    }
  }
  const RowScale f = row_scale<NORM>(ss, amax, H, eps);
  if (p.y) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float y[VE];
#pragma unroll
      for (int i = 0; i < VE; ++i) y[i] = v[c][i] * f.rstd;
      store_chunk<T, VE>(static_cast<T*>(p.y) + row * p.ldy, at(c), H, y);
    }
  }
  if (p.q) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) store_q<VE, NORM>(p.q + row * p.ldq, at(c), H, v[c], f);
    if (threadIdx.x == 0) p.scale[row] = f.scale / 127.f;
  }
}

// One CTA per row: few rows, and rows that are not 16-byte aligned.
template <typename T, int VE, int VPT, bool NORM>
__global__ void __launch_bounds__(1024, 1) k_rows(const RowArgs p) {
  __shared__ float2 sh[32];
  __shared__ float own[kRange<T, NORM> ? 1024 : 1];
  const RowIndex<VE> row = blockIdx.x;
  const int H = p.H;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.ldr : nullptr;
  auto at = [&](int c) { return static_cast<int>(threadIdx.x + c * blockDim.x) * VE; };
  float v[VPT][VE];
#pragma unroll
  for (int c = 0; c < VPT; ++c) load_chunk<T, VE>(x, at(c), H, v[c]);
  if (r) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float rv[VE];
      load_chunk<T, VE>(r, at(c), H, rv);
#pragma unroll
      for (int i = 0; i < VE; ++i) v[c][i] += rv[i];
    }
  }
  finish_row<T, VE, VPT, NORM>(p, row, v, sh, own + (kRange<T, NORM> ? threadIdx.x : 0), at, [&](int c, float(&g)[VE]) {
    load_chunk<T, VE>(static_cast<const T*>(p.w), at(c), H, g);
  });
}

// A chunk as it was loaded.
template <typename T, int VE> struct Raw {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = load16(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(float (&f)[VE]) const { unpack16<T>(v, f); }
};
template <typename T> struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = from_f32<T>(0.f); }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = to_f32<T>(v); }
};

// Many rows: persistent CTAs.  The weight stays in registers, and the loads of
// the next row (RES: with its residual) or of the next two are in flight while
// this one is reduced and stored.  Whole chunks only.
// Where rows may leave the range a thread's weights stay in shared memory: what such
// rows need would spill registers of loads in flight, and a spill waits for its load (8192 x 4096 bf16, residual and int8 out: 39.8 and
// 50 us; no residual: 25.3 and 36).
template <typename T, int VE, int VPT, bool NORM, bool RES>
__global__ void __launch_bounds__(1024, 1) k_rows_many(const RowArgs p, int T_) {
  using R = Raw<T, VE>;
  using Row = RowIndex<VE>;
  constexpr bool kShared = kRange<T, NORM>;
  __shared__ float2 sh[2][32];
  extern __shared__ __align__(16) unsigned char of_thread[];   // kRange: a float for each thread, and its chunks
  const int H = p.H;
  auto at = [&](int c) { return static_cast<int>(threadIdx.x + c * blockDim.x) * VE; };
  R x[VPT], r[VPT];   // r: the residual, or the row after next
  R w[VPT];
  float* const own = reinterpret_cast<float*>(of_thread) + threadIdx.x;
  R* const ws = reinterpret_cast<R*>(of_thread + blockDim.x * sizeof(float)) + threadIdx.x;
  auto fetch = [&](R(&to)[VPT], const void* from, int64_t ld, Row row) {
#pragma unroll
    for (int c = 0; c < VPT; ++c)
      if (at(c) < H) to[c].load(static_cast<const T*>(from) + row * ld + at(c));
  };
#pragma unroll
  for (int c = 0; c < VPT; ++c) x[c].zero(), r[c].zero(), w[c].zero();
  const Row step = gridDim.x, rows = T_;
  Row row = blockIdx.x;
  fetch(x, p.x, p.ldx, row);
  if (RES)
    fetch(r, p.r, p.ldr, row);
  else if (row + step < rows)
    fetch(r, p.x, p.ldx, row + step);
  if (NORM) fetch(w, p.w, 0, 0);
  if (kShared) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) ws[c * blockDim.x] = w[c];
  }
  for (int turn = 0; row < rows; row += step, turn ^= 1) {
    float v[VPT][VE];
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      x[c].unpack(v[c]);
      if (RES) {
        float rv[VE];
        r[c].unpack(rv);
#pragma unroll
        for (int i = 0; i < VE; ++i) v[c][i] += rv[i];
      } else {
        x[c] = r[c];
      }
    }
    if (RES) {
      if (row + step < rows) {
        fetch(x, p.x, p.ldx, row + step);
        fetch(r, p.r, p.ldr, row + step);
      }
    } else if (row + 2 * step < rows) {
      fetch(r, p.x, p.ldx, row + 2 * step);
    }
    finish_row<T, VE, VPT, NORM>(p, row, v, sh[turn], own, at, [&](int c, float(&g)[VE]) {
      const R k = kShared ? ws[c * blockDim.x] : w[c];
      k.unpack(g);
    });
  }
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
  float ss, amax, unit = 1.f, eps = p.eps;
  auto pass = [&](auto scaled) {
    ss = 0.f, amax = 0.f;
    for (int64_t e = static_cast<int64_t>(threadIdx.x) * VE; e < H; e += step) {
      float s[VE], g[VE];
      load(static_cast<int>(e), s, g);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (scaled) s[i] *= unit;
        ss = fmaf(s[i], s[i], ss);
        amax = max_nan(amax, fabsf(NORM ? s[i] * g[i] : s[i]));
      }
    }
    block_reduce<NORM>(ss, amax, sh);
  };
  pass(std::false_type{});
  if (kRange<T, NORM> && (too_large(ss) || too_small(ss, eps))) {
    unit = too_large(ss) ? kDown : kUp;
    eps *= unit, eps *= unit;
    __syncthreads();   // sh has been read
    pass(std::true_type{});
  }
  const RowScale f = row_scale<NORM>(ss, amax, H, eps);
  auto finish = [&](auto scaled) {
    for (int64_t e = static_cast<int64_t>(threadIdx.x) * VE; e < H; e += step) {
      const int e0 = static_cast<int>(e);
      float s[VE], g[VE], v[VE];
      load(e0, s, g);
      if (p.sum) store_chunk<T, VE>(static_cast<T*>(p.sum) + row * p.lds, e0, H, s);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        if (scaled) s[i] *= unit;
        if (NORM) s[i] *= g[i];
        v[i] = s[i] * f.rstd;
      }
      if (p.y) store_chunk<T, VE>(static_cast<T*>(p.y) + row * p.ldy, e0, H, v);
      if (p.q) store_q<VE, NORM>(p.q + row * p.ldq, e0, H, s, f);
    }
  };
  if (unit == 1.f)
    finish(std::false_type{});
  else
    finish(std::true_type{});
  if (p.q && threadIdx.x == 0) p.scale[row] = f.scale / 127.f;
}

template <typename T, int VE, int VPT, bool NORM>
void launch_many(const RowArgs& p, int T_, int threads, cudaStream_t s) {
  const int grid = std::min(T_, sm_count() * std::min(32, 1024 / threads));
  constexpr size_t kThread = !kRange<T, NORM> ? 0 : sizeof(float) + VPT * sizeof(Raw<T, VE>);
  static_assert(1024 * kThread + sizeof(float2) * 64 <= 48 * 1024, "shared memory");
  const size_t smem = threads * kThread;
  if (p.r)
    k_rows_many<T, VE, VPT, NORM, true><<<grid, threads, smem, s>>>(p, T_);
  else
    k_rows_many<T, VE, VPT, NORM, false><<<grid, threads, smem, s>>>(p, T_);
}

// Few rows take the shortest way through a row, one chunk a thread; many are
// streamed by persistent CTAs, 1024 threads to an SM (64 registers a thread).
template <typename T, int VE, bool NORM>
cudaError_t launch_ve(const RowArgs& p, int T_, cudaStream_t s) {
  // chunks of a persistent thread: as many as its registers hold, fp32 rows being twice as long
  constexpr int kMany = VE == 1 ? 8 : VE == 4 && !NORM ? 4 : 2;
  const int chunks = (p.H + VE - 1) / VE;
  auto threads = [&](int vpt) { return ((chunks + vpt - 1) / vpt + 31) / 32 * 32; };
  if (T_ >= 2 * sm_count() && p.H % VE == 0 && chunks <= 1024 * kMany) {
    if (chunks <= 32)
      launch_many<T, VE, 1, NORM>(p, T_, 32, s);
    else
      launch_many<T, VE, kMany, NORM>(p, T_, threads(kMany), s);
  } else if (chunks <= 1024) {
    k_rows<T, VE, 1, NORM><<<T_, threads(1), 0, s>>>(p);
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
  if (T < 0 || H < 1 || H > PW_MAX_VOCAB)
    return pw::failf(PW_EINVAL, "pw_rms_norm: need T >= 0 and 1 <= H <= %d (T %d, H %d)", PW_MAX_VOCAB, T, H);
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
  if (T < 0 || K < 1 || K > PW_MAX_VOCAB)
    return pw::failf(PW_EINVAL, "pw_quant_i8: need T >= 0 and 1 <= K <= %d (T %d, K %d)", PW_MAX_VOCAB, T, K);
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
