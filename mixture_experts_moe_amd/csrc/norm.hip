// Root-mean-square norm of the residual stream and its gradient, and rows in
// 8-bit integers with one scale each.
//
//   h = x + residual (rounded to the act dtype: what the caller keeps as the
//   stream is what is normalised), y = h r w with r = 1 / sqrt(mean(h^2) + eps),
//   scale = max |y| / 127, codes = y / scale to the nearest integer
//
// Every element is read once and every result written once; six operations an
// element are nothing beside that, so all of it is bound by memory (a few
// rows: by the latency of one read, the row sums and one write).  A row stays
// in the registers of its lanes between the steps.

#include "common.h"
#include "kernels.h"

namespace moe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------ rows in registers

// 16 bytes of a row at any alignment: 8 bf16 or 4 fp32.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
struct __attribute__((packed, aligned(1))) NormUnit {
  u32x4 v;
};
template <int N>
struct NormBytes;
template <>
struct __attribute__((packed, aligned(1))) NormBytes<8> {
  u32x2 v;
};
template <>
struct __attribute__((packed, aligned(1))) NormBytes<4> {
  uint32_t v;
};

template <typename AT>
struct NormRow {
  static constexpr int kN = 16 / (int)sizeof(AT);  // elements of a unit

  // elements c .. c + kN - 1 of a row of d, zero past its end.  Rows that stay in
  // registers are read once: nontemporal (8192 x 4096 bf16 to y and codes 51.7 ->
  // 49.6 us; stores with the hint took 5% more in fp32).  Longer rows, which are
  // read again, take the hint too; plain loads there, fp32: codes of 64 / 2048 x 32768
  // 12.2 / 99 -> 8.0 / 93 us, but y of 256 x 131072 71 -> 79, and the gradient's first
  // pass 4096 x 7168 without dsum 106 -> 111, bf16 2048 x 16384 with it 90 -> 87.
  static __device__ __forceinline__ u32x4 raw(const AT* row, int c, int d) {
    if (c + kN <= d)
      return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + c));
    union {
      u32x4 v;
      AT e[kN];
    } u;
    u.v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c + i < d) u.e[i] = row[c + i];
    return u.v;
  }
  static __device__ __forceinline__ void values(u32x4 q, float (&f)[kN]) {
    if constexpr (sizeof(AT) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(q[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(q[i] << 16);
        f[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
      }
    }
  }
  // to nearest even, NaN kept
  static __device__ __forceinline__ u32x4 rounded(const float (&f)[kN]) {
    if constexpr (sizeof(AT) == 4) {
      return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3])};
    } else {
      bf16x8 h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = static_cast<__bf16>(f[i]);
      return __builtin_bit_cast(u32x4, h);
    }
  }
  static __device__ __forceinline__ void store(AT* row, int c, int d, u32x4 q) {
    if (c + kN <= d) {
      reinterpret_cast<NormUnit*>(row + c)->v = q;
      return;
    }
    union {
      u32x4 v;
      AT e[kN];
    } u;
    u.v = q;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c + i < d) row[c + i] = u.e[i];
  }
  // weights of the unit's columns (none: ones)
  static __device__ __forceinline__ void weights(const float* w, int c, int d, float (&f)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = 1.0f;
    if (!w) return;
    if (c + kN <= d) {  // (16-byte aligned: w is, c a multiple of four)
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(w + c + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i + j] = q[j];
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c + i < d) f[i] = w[c + i];
  }
  // The unit's codes: y / scale to the nearest integer.  1.5 * 2^23 + v holds
  // v's nearest integer in its low bits (|v| <= 127, one rounding, of the exact
  // product by the fused multiply-add); the product with 1 / scale in place of
  // the quotient is off by less than 2^-16 of a step.
  static __device__ __forceinline__ void store_codes(int8_t* row, int c, int d,
                                                     const float (&y)[kN], float inv) {
    uint32_t q[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) q[i] = __float_as_uint(__builtin_fmaf(y[i], inv, 12582912.0f));
    if (c + kN <= d) {
      uint32_t p[kN / 4];
#pragma unroll
      for (int i = 0; i < kN / 4; ++i)
        p[i] = __builtin_amdgcn_perm(
            __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x0c0c0400u),
            __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0c0c0400u), 0x05040100u);
      NormBytes<kN> b;
      if constexpr (kN == 8)
        b.v = u32x2{p[0], p[1]};
      else
        b.v = p[0];
      *reinterpret_cast<NormBytes<kN>*>(row + c) = b;
      return;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (c + i < d) row[c + i] = static_cast<int8_t>(q[i]);
  }
};

// The sum, or the largest, of one value per lane over the kLanes lanes of a
// row, in every one of them.  `red` holds one value per wave.
template <int kLanes, typename T, typename F>
__device__ __forceinline__ T norm_over_row(T v, T* red, const F& f) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = f(v, __shfl_xor(v, off, kWave));
  if constexpr (kLanes > kWave) {
    __syncthreads();  // red has been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < kLanes / kWave; ++i) v = f(v, red[i]);
  }
  return v;
}

// Two sums at once: one meeting in LDS (2 values per wave).
template <int kLanes>
__device__ __forceinline__ void norm_over_row2(float& v, float& w, float (*red)[2]) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    v += __shfl_xor(v, off, kWave);
    w += __shfl_xor(w, off, kWave);
  }
  if constexpr (kLanes > kWave) {
    __syncthreads();  // red has been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][0] = v, red[threadIdx.x >> 6][1] = w;
    __syncthreads();
    v = red[0][0], w = red[0][1];
#pragma unroll
    for (int i = 1; i < kLanes / kWave; ++i) v += red[i][0], w += red[i][1];
  }
}

struct NormAdd {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// Magnitudes as bit patterns: a NaN is above infinity, which is above every
// number, so one comparison finds the largest and what is not finite.
struct NormMax {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
    return a > b ? a : b;
  }
};

// Scale and 1 / scale of a row whose largest magnitude has the bits `amax`.
// Zeros: 1.  A value that is not finite: NaN, and codes of zero.  The scale
// stays a normal number, so that 1 / scale is one.
__device__ __forceinline__ float norm_scale(uint32_t amax, float* inv) {
  if (amax >= 0x7f800000u) {
    *inv = 0.0f;
    return __uint_as_float(0x7fc00000u);
  }
  float s = __uint_as_float(amax) / 127.0f;
  if (amax == 0) s = 1.0f;
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;
  *inv = 1.0f / s;
  return s;
}

// A launch holds fewer than 2^32 threads per grid dimension: workgroups beyond
// kNormGridX go on in y.
constexpr int64_t kNormGridX = 1 << 20;
static dim3 norm_grid(int64_t workgroups) {
  const int64_t x = workgroups < kNormGridX ? workgroups : kNormGridX;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((workgroups + x - 1) / x));
}
__device__ __forceinline__ int64_t norm_workgroup() {
  return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

// kLanes lanes (64: a wave, and four rows per workgroup) x kUnits units hold a
// row.
template <int kLanes>
struct NormGeom {
  static constexpr int kThreads = kLanes < 256 ? 256 : kLanes;
  static constexpr int kRows = kThreads / kLanes;
};

template <typename AT, bool kNorm, int kLanes, int kUnits>
__global__ __launch_bounds__(NormGeom<kLanes>::kThreads) void norm_kernel(NormArgs a) {
  using R = NormRow<AT>;
  using G = NormGeom<kLanes>;
  constexpr int N = R::kN;
  __shared__ float red[G::kThreads / kWave];
  __shared__ uint32_t redm[G::kThreads / kWave];
  const int lane = threadIdx.x % kLanes;
  const int64_t m = norm_workgroup() * G::kRows + threadIdx.x / kLanes;
  if (m >= a.rows) return;  // whole waves; a row of several waves is the workgroup's only one
  const AT* x = static_cast<const AT*>(a.x) + m * a.ldx;
  const AT* res = static_cast<const AT*>(a.res) + m * a.ldr;
  u32x4 q[kUnits], p[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) q[u] = R::raw(x, (u * kLanes + lane) * N, a.cols);
  if (kNorm && a.res)
#pragma unroll
    for (int u = 0; u < kUnits; ++u) p[u] = R::raw(res, (u * kLanes + lane) * N, a.cols);
  float h[kUnits][N];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) R::values(q[u], h[u]);
  if constexpr (kNorm) {
    if (a.res) {
      AT* sum = static_cast<AT*>(a.sum) + m * a.ldsum;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        float f[N];
        R::values(p[u], f);
#pragma unroll
        for (int i = 0; i < N; ++i) h[u][i] += f[i];
        const u32x4 r = R::rounded(h[u]);
        if (a.sum) R::store(sum, (u * kLanes + lane) * N, a.cols, r);
        R::values(r, h[u]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) s += h[u][i] * h[u][i];
    s = norm_over_row<kLanes>(s, red, NormAdd{});
    const float r = 1.0f / sqrtf(s / a.cols + a.eps);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float w[N];
      R::weights(a.weight, (u * kLanes + lane) * N, a.cols, w);
#pragma unroll
      for (int i = 0; i < N; ++i) h[u][i] = h[u][i] * r * w[i];
      if ((u * kLanes + lane) * N + N > a.cols)  // 0 * r past the end may be NaN
#pragma unroll
        for (int i = 0; i < N; ++i)
          if ((u * kLanes + lane) * N + i >= a.cols) h[u][i] = 0.0f;
    }
    if (a.y) {
      AT* y = static_cast<AT*>(a.y) + m * a.ldy;
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        R::store(y, (u * kLanes + lane) * N, a.cols, R::rounded(h[u]));
    }
    if (!a.codes) return;
  }
  uint32_t amax = 0;
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i)
      amax = NormMax{}(amax, __float_as_uint(h[u][i]) & 0x7fffffffu);
  amax = norm_over_row<kLanes>(amax, redm, NormMax{});
  float inv;
  const float scale = norm_scale(amax, &inv);
  // (a value that is not finite times 0 is NaN: its low bits are not a code)
  const bool finite = amax < 0x7f800000u;
  int8_t* codes = a.codes + m * a.ldc;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (!finite)
#pragma unroll
      for (int i = 0; i < N; ++i) h[u][i] = 0.0f;
    R::store_codes(codes, (u * kLanes + lane) * N, a.cols, h[u], inv);
  }
  if (lane == 0) a.scale[m] = scale;
}

// Rows that the registers of a workgroup do not hold: a workgroup per row
// reads it again for every step (fp32 to codes, 2048 x 32768: 99 us, one read and
// the codes 67 at the rate of a copy; to y 127, 107).
constexpr int kNormLong = 1024;
template <typename AT, bool kNorm>
__global__ __launch_bounds__(kNormLong) void norm_long_kernel(NormArgs a) {
  using R = NormRow<AT>;
  constexpr int N = R::kN;
  __shared__ float red[kNormLong / kWave];
  __shared__ uint32_t redm[kNormLong / kWave];
  const int64_t m = norm_workgroup();
  if (m >= a.rows) return;
  const int first = threadIdx.x * N, step = kNormLong * N;
  const AT* x = static_cast<const AT*>(a.x) + m * a.ldx;
  const AT* res = a.res ? static_cast<const AT*>(a.res) + m * a.ldr : nullptr;
  AT* sum = a.sum ? static_cast<AT*>(a.sum) + m * a.ldsum : nullptr;
  auto load = [&](int c, float (&h)[N]) {
    R::values(R::raw(x, c, a.cols), h);
    if (!res) return;
    float f[N];
    R::values(R::raw(res, c, a.cols), f);
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] += f[i];
    R::values(R::rounded(h), h);
  };
  float r = 1.0f;
  if constexpr (kNorm) {
    float s = 0.0f;
    for (int c = first; c < a.cols; c += step) {
      float h[N];
      load(c, h);
      if (sum) R::store(sum, c, a.cols, R::rounded(h));
#pragma unroll
      for (int i = 0; i < N; ++i) s += h[i] * h[i];
    }
    s = norm_over_row<kNormLong>(s, red, NormAdd{});
    r = 1.0f / sqrtf(s / a.cols + a.eps);
    // the sum may have been written over x or the residual
    if (sum) x = sum, res = nullptr;
  }
  auto value = [&](int c, float (&h)[N]) {
    load(c, h);
    if constexpr (kNorm) {
      float w[N];
      R::weights(a.weight, c, a.cols, w);
#pragma unroll
      for (int i = 0; i < N; ++i) h[i] = c + i < a.cols ? h[i] * r * w[i] : 0.0f;
    }
  };
  float inv = 0.0f;
  bool finite = true;
  if (a.codes) {
    uint32_t amax = 0;
    for (int c = first; c < a.cols; c += step) {
      float h[N];
      value(c, h);
#pragma unroll
      for (int i = 0; i < N; ++i) amax = NormMax{}(amax, __float_as_uint(h[i]) & 0x7fffffffu);
    }
    amax = norm_over_row<kNormLong>(amax, redm, NormMax{});
    const float scale = norm_scale(amax, &inv);
    finite = amax < 0x7f800000u;
    if (threadIdx.x == 0) a.scale[m] = scale;
  }
  for (int c = first; c < a.cols; c += step) {
    float h[N];
    value(c, h);
    if (kNorm && a.y) R::store(static_cast<AT*>(a.y) + m * a.ldy, c, a.cols, R::rounded(h));
    if (a.codes) {
      if (!finite)
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = 0.0f;
      R::store_codes(a.codes + m * a.ldc, c, a.cols, h, inv);
    }
  }
}

// ------------------------------------------------------------ gradient
//
// With g = w dy:  dh = (g - h r^2 mean(g h)) r (+ dsum),  dw = sum of dy h r.
// r and mean(g h) come from the rows themselves, which have to be read anyway.
// The second term is (h r)(r mean(g h)): |h r| is at most sqrt(cols), while r^2
// leaves fp32 where mean(h^2) + eps is below 3e-39 and dh is far from its limits.
// A workgroup walks every gridDim.x-th row with its columns' share of dw in
// registers; the workgroups' shares are added by a second launch, in order, so
// dw does not depend on the run.  The next row is loaded while one is worked on.

// A unit's share of dweight (rows of shares start at any multiple of four bytes).
template <int N>
__device__ __forceinline__ void norm_store_share(float* part, int c, int d, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    if (c + i + 4 <= d) {
      reinterpret_cast<NormUnit*>(part + c + i)->v =
          u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                __float_as_uint(v[i + 3])};
    } else {
#pragma unroll
      for (int j = i; j < i + 4; ++j)
        if (c + j < d) part[c + j] = v[j];
    }
}

template <typename AT, int kLanes, int kUnits>
__global__ __launch_bounds__(NormGeom<kLanes>::kThreads, 4) void norm_backward_kernel(
    NormBackwardArgs a) {
  using R = NormRow<AT>;
  using G = NormGeom<kLanes>;
  constexpr int N = R::kN;
  __shared__ float red[G::kThreads / kWave][2];
  __shared__ float shares[G::kRows > 1 ? G::kRows : 1][G::kRows > 1 ? kLanes * kUnits * N : 1];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  float w[kUnits][N], dw[kUnits][N];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    R::weights(a.weight, (u * kLanes + lane) * N, a.cols, w[u]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[u][i] = 0.0f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * G::kRows;
  int64_t m = static_cast<int64_t>(blockIdx.x) * G::kRows + sub;
  u32x4 qh[kUnits], qg[kUnits];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      qh[u] = R::raw(static_cast<const AT*>(a.h) + row * a.ldh, (u * kLanes + lane) * N, a.cols);
      qg[u] = R::raw(static_cast<const AT*>(a.dy) + row * a.ldy, (u * kLanes + lane) * N, a.cols);
    }
  };
  if (m < a.rows) fetch(m);
  for (; m < a.rows; m += step) {  // uniform over the row's lanes
    u32x4 ch[kUnits], cg[kUnits], qs[kUnits];
    float hh = 0.0f, gh = 0.0f;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      ch[u] = qh[u], cg[u] = qg[u];
      if (a.dsum)
        qs[u] = R::raw(static_cast<const AT*>(a.dsum) + m * a.ldsum, (u * kLanes + lane) * N, a.cols);
    }
    if (m + step < a.rows) fetch(m + step);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float h[N], g[N];
      R::values(ch[u], h);
      R::values(cg[u], g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        hh += h[i] * h[i];
        gh += g[i] * w[u][i] * h[i];
      }
      // (bf16: the row stays packed between the sums and the results; the
      // compiler would keep the values, twice the registers)
      if constexpr (sizeof(AT) == 2) asm volatile("" : "+v"(ch[u]), "+v"(cg[u]));
    }
    norm_over_row2<kLanes>(hh, gh, red);
    const float r = 1.0f / sqrtf(hh / a.cols + a.eps);
    const float k = r * (gh / a.cols);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float h[N], g[N], s[N];
      R::values(ch[u], h);
      R::values(cg[u], g);
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = 0.0f;
      if (a.dsum) R::values(qs[u], s);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = h[i] * r;
        dw[u][i] += g[i] * n;
        s[i] += (g[i] * w[u][i] - n * k) * r;
      }
      R::store(static_cast<AT*>(a.dx) + m * a.ldx, (u * kLanes + lane) * N, a.cols, R::rounded(s));
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
  if constexpr (G::kRows > 1) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) shares[sub][(u * kLanes + lane) * N + i] = dw[u][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += G::kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < G::kRows; ++i) s += shares[i][c];
      part[c] = s;
    }
  } else {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) norm_store_share<N>(part, (u * kLanes + lane) * N, a.cols, dw[u]);
  }
}

// Rows that registers do not hold: r and r mean(g h) of every row first ...
template <typename AT>
__global__ __launch_bounds__(kNormLong) void norm_backward_stats_kernel(NormBackwardArgs a) {
  using R = NormRow<AT>;
  constexpr int N = R::kN;
  __shared__ float red[kNormLong / kWave][2];
  const int64_t m = norm_workgroup();
  if (m >= a.rows) return;
  float hh = 0.0f, gh = 0.0f;
  for (int c = threadIdx.x * N; c < a.cols; c += kNormLong * N) {
    float h[N], g[N], w[N];
    R::values(R::raw(static_cast<const AT*>(a.h) + m * a.ldh, c, a.cols), h);
    R::values(R::raw(static_cast<const AT*>(a.dy) + m * a.ldy, c, a.cols), g);
    R::weights(a.weight, c, a.cols, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      hh += h[i] * h[i];
      gh += c + i < a.cols ? g[i] * w[i] * h[i] : 0.0f;
    }
  }
  norm_over_row2<kNormLong>(hh, gh, red);
  const float r = 1.0f / sqrtf(hh / a.cols + a.eps);
  if (threadIdx.x == 0) {
    a.stats[2 * m] = r;
    a.stats[2 * m + 1] = r * (gh / a.cols);
  }
}
// ... then a workgroup takes 256 units of columns (blockIdx.y) of every
// gridDim.x-th row.
constexpr int kNormCols = 256;
template <typename AT>
__global__ __launch_bounds__(kNormCols) void norm_backward_long_kernel(NormBackwardArgs a) {
  using R = NormRow<AT>;
  constexpr int N = R::kN;
  const int c = (blockIdx.y * kNormCols + threadIdx.x) * N;
  if (c >= a.cols) return;
  float w[N], dw[N];
  R::weights(a.weight, c, a.cols, w);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = 0.0f;
  for (int64_t m = blockIdx.x; m < a.rows; m += gridDim.x) {
    const float r = a.stats[2 * m], k = a.stats[2 * m + 1];
    float h[N], g[N], s[N];
    R::values(R::raw(static_cast<const AT*>(a.h) + m * a.ldh, c, a.cols), h);
    R::values(R::raw(static_cast<const AT*>(a.dy) + m * a.ldy, c, a.cols), g);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.0f;
    if (a.dsum) R::values(R::raw(static_cast<const AT*>(a.dsum) + m * a.ldsum, c, a.cols), s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float n = h[i] * r;
      dw[i] += g[i] * n;
      s[i] += (g[i] * w[i] - n * k) * r;
    }
    R::store(static_cast<AT*>(a.dx) + m * a.ldx, c, a.cols, R::rounded(s));
  }
  if (!a.part) return;
  norm_store_share<N>(a.part + static_cast<int64_t>(blockIdx.x) * a.cols, c, a.cols, dw);
}

// dweight[c] = the workgroups' shares of column c, added in a fixed order: a
// workgroup takes 32 columns, 32 slices of eight threads (four columns each)
// every 32nd share; the slices' sums meet in LDS.
constexpr int kNormSum = 256, kNormSumCols = 32, kNormSlices = kNormSum / (kNormSumCols / 4);
__global__ __launch_bounds__(kNormSum) void norm_backward_sum_kernel(const float* part, int shares,
                                                                     int cols, float* dweight) {
  __shared__ f32x4 s[kNormSlices][kNormSumCols / 4];
  const int quad = threadIdx.x % (kNormSumCols / 4), slice = threadIdx.x / (kNormSumCols / 4);
  const int c = blockIdx.x * kNormSumCols + 4 * quad;
  f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
  if (c + 4 <= cols) {
#pragma unroll 8
    for (int i = slice; i < shares; i += kNormSlices)
      v += __builtin_bit_cast(
          f32x4, reinterpret_cast<const NormUnit*>(part + static_cast<int64_t>(i) * cols + c)->v);
  } else {
    for (int i = slice; i < shares; i += kNormSlices)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < cols) v[j] += part[static_cast<int64_t>(i) * cols + c + j];
  }
  s[slice][quad] = v;
  __syncthreads();
  if (threadIdx.x < kNormSumCols && blockIdx.x * kNormSumCols + threadIdx.x < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormSlices; ++i) t += s[i][threadIdx.x / 4][threadIdx.x % 4];
    dweight[blockIdx.x * kNormSumCols + threadIdx.x] = t;
  }
}

// ------------------------------------------------------------ launchers

// f(lanes, units) of the smallest geometry that holds a row, or none.
template <typename F, typename L>
static hipError_t norm_geometry(int cols, int size, const F& f, const L& longer) {
  const int units = static_cast<int>((static_cast<int64_t>(cols) * size + 15) / 16);
  if (units <= 64) return f(LinInt<64>{}, LinInt<1>{});
  if (units <= 128) return f(LinInt<64>{}, LinInt<2>{});
  if (units <= 256) return f(LinInt<256>{}, LinInt<1>{});
  if (units <= 512) return f(LinInt<256>{}, LinInt<2>{});
  // (4096 x 7168 bf16 to codes: 256 x 4 40.3 us, 512 x 2 39.4, 1024 x 1 46.6; one
  // row 6.3, 5.4, 5.0)
  if (units <= 1024) return f(LinInt<512>{}, LinInt<2>{});
  if (units <= 2048) return f(LinInt<512>{}, LinInt<4>{});
  if (units <= 4096) return f(LinInt<1024>{}, LinInt<4>{});
  return longer();
}

template <typename AT, bool kNorm>
static hipError_t launch_norm_type(const NormArgs& a, hipStream_t s) {
  return norm_geometry(
      a.cols, sizeof(AT),
      [&](auto lanes, auto units) {
        using G = NormGeom<lanes.value>;
        norm_kernel<AT, kNorm, lanes.value, units.value>
            <<<norm_grid((a.rows + G::kRows - 1) / G::kRows), G::kThreads, 0, s>>>(a);
        return hipGetLastError();
      },
      [&]() {
        norm_long_kernel<AT, kNorm><<<norm_grid(a.rows), kNormLong, 0, s>>>(a);
        return hipGetLastError();
      });
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.act_dtype == kDtypeF32)
    return a.norm ? launch_norm_type<float, true>(a, s) : launch_norm_type<float, false>(a, s);
  return a.norm ? launch_norm_type<bf16_t, true>(a, s) : launch_norm_type<bf16_t, false>(a, s);
}

// The gradient's geometries: its weights, shares of dweight and the next row
// leave room for 16 bf16 or 8 fp32 of a row per lane.  The widest has 512 lanes:
// rows over 16 KiB are read twice (fp32 4096 x 7168 with dsum 128 us, 94 at the rate
// of a copy; 4096 x 4096, held, 48 and 54).  1024 lanes with as much each, for rows
// to 32 KiB, have not been built.
template <typename F, typename L>
static auto norm_backward_geometry(int cols, int act_dtype, const F& f, const L& longer) {
  const int size = act_dtype == kDtypeF32 ? 4 : 2;
  const int units = static_cast<int>((static_cast<int64_t>(cols) * size + 15) / 16);
  if (units <= 64) return f(LinInt<64>{}, LinInt<1>{});
  if (units <= 128) return f(LinInt<64>{}, LinInt<2>{});
  if (units <= 256) return f(LinInt<256>{}, LinInt<1>{});
  if (units <= 512) return f(LinInt<256>{}, LinInt<2>{});
  if (units <= 1024) return f(LinInt<512>{}, LinInt<2>{});
  return longer();
}

// Workgroups that share the rows: three of 256 threads or two of 512 for a
// compute unit, no more, since each leaves a row of dweight's sums (8192 x 4096
// bf16, 256 threads: 512 workgroups 56.3 us, 768 54.4; 4096 x 4096 fp32, 512
// threads: 512 49.1, 768 54.6).
constexpr int kNormShares = 768;
int norm_backward_shares(int64_t rows, int cols, int act_dtype) {
  return norm_backward_geometry(
      cols, act_dtype,
      [&](auto lanes, auto) {
        using G = NormGeom<lanes.value>;
        constexpr int kMost = G::kThreads == 256 ? kNormShares : kNormShares * 2 / 3;
        const int64_t most = (rows + G::kRows - 1) / G::kRows;
        return static_cast<int>(most < kMost ? most : kMost);
      },
      [&]() { return static_cast<int>(rows < kNormShares ? rows : kNormShares); });
}
bool norm_backward_in_registers(int cols, int act_dtype) {
  return norm_backward_geometry(cols, act_dtype, [](auto, auto) { return true; },
                                []() { return false; });
}

template <typename AT>
static hipError_t launch_norm_backward_type(const NormBackwardArgs& a, hipStream_t s) {
  hipError_t e = norm_backward_geometry(
      a.cols, a.act_dtype,
      [&](auto lanes, auto units) {
        norm_backward_kernel<AT, lanes.value, units.value>
            <<<a.shares, NormGeom<lanes.value>::kThreads, 0, s>>>(a);
        return hipGetLastError();
      },
      [&]() {
        norm_backward_stats_kernel<AT><<<norm_grid(a.rows), kNormLong, 0, s>>>(a);
        const int units = (a.cols + NormRow<AT>::kN - 1) / NormRow<AT>::kN;
        norm_backward_long_kernel<AT>
            <<<dim3(a.shares, (units + kNormCols - 1) / kNormCols), kNormCols, 0, s>>>(a);
        return hipGetLastError();
      });
  if (e == hipSuccess && a.shares > 1 && a.dweight) {
    norm_backward_sum_kernel<<<(a.cols + kNormSumCols - 1) / kNormSumCols, kNormSum, 0, s>>>(
        a.part, a.shares, a.cols, a.dweight);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, hipStream_t s) {
  if (a.act_dtype == kDtypeF32) return launch_norm_backward_type<float>(a, s);
  return launch_norm_backward_type<bf16_t>(a, s);
}

}  // namespace moe
