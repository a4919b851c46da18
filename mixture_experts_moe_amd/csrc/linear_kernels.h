// Kernels of the dense product with its epilogue: out = act((x . W^T) * scale +
// bias) + residual, or act(gate half) * (up half) + residual when gated.  The
// kind of product the routed experts run, without routing: shared experts,
// dense feed-forward layers and projections beside a fused MoE layer.
// WT: the weights' type (the tokens' goes with it), OT: the results'.
//
// The product is computed transposed, as in the expert kernels: weight rows
// (output channels) on the 16-row side of the MFMA and tokens on its columns,
// so a lane ends with consecutive channels of one token.
//
// int8 weights go with int8 tokens, int32 sums and a scale per token, applied
// when the sums become values; their rows may be sorted by expert, each expert's
// with weights of its own.
#pragma once

#include "kernels.h"
#include "stream.h"

namespace moe {

// ------------------------------------------------------------ epilogue
//
// Sums are fp32 throughout; the one rounding to the output type is the store
// (to nearest even).  gelu through erfc and both sigmoids through
// z / (1 + e^-u): no cancellation for large negative z, exp overflow gives a
// quotient of zero.

// With bf16 results the sigmoids use the hardware's exp2 and reciprocal: the
// quotient's relative error is at most |u| 2^-23 + 2^-21 of e^-u's argument as
// given, while that and its reciprocal are normal numbers (|u| <= 87; beyond,
// z / (1 + e^-u) is below |z| 2^-125 and may come out as zero).  gelu_tanh's u
// grows with z^3 and carries roundings of its own, |u| 2^-21 in all: 2^-15 at
// z = -10, where the tail ends, against the result's half step of 2^-8 at most.
template <bool kFast>
__device__ __forceinline__ float lin_sigmoid_times(float z, float u) {  // z / (1 + e^-u)
  if constexpr (kFast) return z * __builtin_amdgcn_rcpf(1.0f + __expf(-u));
  return z / (1.0f + expf(-u));
}

// z Phi(z), Phi(z) = erfc(-z / sqrt 2) / 2.  For bf16 results Phi's tail is
// e^(-z^2/2) P(t), t = 1 / (1 + 0.38 |z| / sqrt 2), P of degree 7: a minimax fit
// of e^(x^2) erfc(x) / 2 over 0 <= x <= 12 whose relative error is 1.1e-6, so the
// tail keeps its relative accuracy down to where it leaves the type's range.  It
// is short enough to stand in the epilogue once per value (802 x 13400 x 2888 bf16:
// erfcf, one copy in a loop, 98 us; this 79).
template <bool kFast>
__device__ __forceinline__ float lin_gelu(float z) {
  if constexpr (!kFast) return 0.5f * z * erfcf(z * -0.70710678118654752f);
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.26870057685088805f * fabsf(z));
  float p = -0.0627079869797211f;
  p = p * t + 0.16801539047659845f;
  p = p * t - 0.03495267354882652f;
  p = p * t + 0.12391424436400950f;
  p = p * t + 0.09029839441786437f;
  p = p * t + 0.10828843519853950f;
  p = p * t + 0.10714368014064054f;
  const float q = p * t * __expf(-0.5f * z * z);
  return z * (z < 0.f ? q : 1.0f - q);
}

template <bool kFast>
__device__ __forceinline__ float lin_act(int fn, float z) {
  switch (fn) {
    case kFnRelu: return z < 0.f ? 0.f : z;  // NaN stays
    case kFnSilu: return lin_sigmoid_times<kFast>(z, z);
    case kFnGelu: return lin_gelu<kFast>(z);
    case kFnGeluTanh:  // tanh(u) = 2 / (1 + e^-2u) - 1, u = sqrt(2/pi) (z + 0.044715 z^3)
      return lin_sigmoid_times<kFast>(z, 1.5957691216057308f * (z + 0.044715f * z * z * z));
  }
  return z;
}

template <typename AT>
__device__ __forceinline__ float lin_load(const AT* p) {
  if constexpr (sizeof(AT) == 4)
    return *reinterpret_cast<const float*>(p);
  else
    return bf16_to_f32(*reinterpret_cast<const bf16_t*>(p));
}

template <typename AT>
__device__ __forceinline__ void lin_store(AT* p, float v) {
  if constexpr (sizeof(AT) == 4)
    *p = v;
  else
    *p = f32_to_bf16(v);
}

// Finish and store out[m, n] from its channel sums (zu: the up half's, when
// gated).  The residual is read and the result written by one thread, so out
// may be the residual itself.
template <typename AT>
__device__ __forceinline__ void lin_finish(const LinearArgs& a, float zg, float zu, int64_t m,
                                           int n) {
  if (a.scale) {
    zg *= a.scale_channel ? a.scale[n] : a.scale[0];
    if (a.gated) zu *= a.scale_channel ? a.scale[a.N + n] : a.scale[0];
  }
  if (a.bias) {
    zg += a.bias[n];
    if (a.gated) zu += a.bias[a.N + n];
  }
  float v = lin_act<sizeof(AT) == 2>(a.fn, zg);
  if (a.gated) v *= zu;
  if (a.res) v += lin_load(static_cast<const AT*>(a.res) + m * a.ldr + n);
  lin_store(static_cast<AT*>(a.out) + m * a.ldo + n, v);
}

// Four consecutive channels n .. n+3 (those below N) for several tokens: the
// scales and biases are read once.
template <typename AT, bool kGated>
struct LinQuad {
  f32x4 sg, su, bg, bu;
  int n, valid;  // channels that exist

  __device__ __forceinline__ void init(const LinearArgs& a, int n_) {
    n = n_;
    valid = min(a.N - n, 4);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int c = min(n + v, a.N - 1);
      sg[v] = !a.scale ? 1.f : a.scale[a.scale_channel ? c : 0];
      bg[v] = a.bias ? a.bias[c] : 0.f;
      if (kGated) {
        su[v] = !a.scale ? 1.f : a.scale[a.scale_channel ? a.N + c : 0];
        bu[v] = a.bias ? a.bias[a.N + c] : 0.f;
      }
    }
  }

  // kRows tokens' sums zg (and zu) -> values, with the function chosen once
  template <int kRows>
  __device__ __forceinline__ void values(const LinearArgs& a, f32x4 (&zg)[kRows],
                                         f32x4 (&zu)[kRows]) const {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      zg[i] = zg[i] * sg + bg;
      if (kGated) zu[i] = zu[i] * su + bu;
    }
    auto apply = [&](int fn) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) zg[i][v] = lin_act<sizeof(AT) == 2>(fn, zg[i][v]);
    };
    switch (a.fn) {
      case kFnRelu: apply(kFnRelu); break;
      case kFnSilu: apply(kFnSilu); break;
      case kFnGeluTanh: apply(kFnGeluTanh); break;
      case kFnGelu:
        if constexpr (sizeof(AT) == 2) {
          apply(kFnGelu);
          break;
        }
        // a long function in fp32: one copy
#pragma unroll 1
        for (int i = 0; i < 4 * kRows; ++i) {
          float z = zg[0][0];
#pragma unroll
          for (int j = 1; j < 4 * kRows; ++j) z = i == j ? zg[j / 4][j % 4] : z;
          z = lin_act<sizeof(AT) == 2>(kFnGelu, z);
#pragma unroll
          for (int j = 0; j < 4 * kRows; ++j) zg[j / 4][j % 4] = i == j ? z : zg[j / 4][j % 4];
        }
        break;
    }
    if (kGated) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) zg[i] *= zu[i];
    }
  }

  // + residual, rounded, stored
  __device__ __forceinline__ void store(const LinearArgs& a, f32x4 z, int64_t m) const {
    AT* o = static_cast<AT*>(a.out) + m * a.ldo + n;
    const AT* r = static_cast<const AT*>(a.res) + m * a.ldr + n;
    if (a.vec4 && valid == 4) {
      if constexpr (sizeof(AT) == 4) {
        if (a.res) z += *reinterpret_cast<const f32x4*>(r);
        *reinterpret_cast<f32x4*>(o) = z;
      } else {
        if (a.res) {
          const uint2 q = *reinterpret_cast<const uint2*>(r);
          z += f32x4{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u),
                     __uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u)};
        }
        // the hardware's conversion: to nearest even, NaN kept
        typedef __bf16 bf16x4v __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4v*>(o) = __builtin_convertvector(z, bf16x4v);
      }
      return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < valid) lin_store(o + v, a.res ? z[v] + lin_load(r + v) : z[v]);
  }

  // the sums of this K range instead, where K is split
  __device__ __forceinline__ void store_part(const LinearArgs& a, f32x4 zg, f32x4 zu,
                                             int64_t m) const {
    float* p = a.part + (static_cast<size_t>(blockIdx.z) * a.part_rows + m) * a.R + n;
    if (a.N % 4 == 0) {
      *reinterpret_cast<f32x4*>(p) = zg;
      if (kGated) *reinterpret_cast<f32x4*>(p + a.N) = zu;
      return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < valid) {
        p[v] = zg[v];
        if (kGated) p[a.N + v] = zu[v];
      }
  }
};

// Eight consecutive channels n .. n+7 (those below N): scales and biases read
// once, then any number of tokens.
template <typename AT, bool kGated>
struct LinOct {
  float sg[8], su[8], bg[8], bu[8];
  int n, valid;  // channels that exist

  __device__ __forceinline__ void init(const LinearArgs& a, int n_) {
    n = n_;
    valid = min(a.N - n, 8);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      const int c = min(n + v, a.N - 1);
      sg[v] = !a.scale ? 1.f : a.scale[a.scale_channel ? c : 0];
      bg[v] = a.bias ? a.bias[c] : 0.f;
      if (kGated) {
        su[v] = !a.scale ? 1.f : a.scale[a.scale_channel ? a.N + c : 0];
        bu[v] = a.bias ? a.bias[a.N + c] : 0.f;
      }
    }
  }

  // The same from a tile's copies: scales and biases of its rows, of which
  // these channels are c .. c+7 (up half: u .. u+7).
  __device__ __forceinline__ void init(const LinearArgs& a, int n_, const float* scale,
                                       const float* bias, int c, int u) {
    n = n_;
    valid = min(a.N - n, 8);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      sg[v] = scale[c + v], bg[v] = bias[c + v];
      if (kGated) su[v] = scale[u + v], bu[v] = bias[u + v];
    }
  }

  // One token's channel sums zg (zu: the up half's) -> out[m, n ..].
  __device__ __forceinline__ void finish(const LinearArgs& a, float (&zg)[8], float (&zu)[8],
                                         int64_t m) const {
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      zg[v] = zg[v] * sg[v] + bg[v];
      if (kGated) zu[v] = zu[v] * su[v] + bu[v];
    }
    auto apply = [&](int fn) {
#pragma unroll
      for (int v = 0; v < 8; ++v) zg[v] = lin_act<sizeof(AT) == 2>(fn, zg[v]);
    };
    switch (a.fn) {
      case kFnRelu: apply(kFnRelu); break;
      case kFnSilu: apply(kFnSilu); break;
      case kFnGeluTanh: apply(kFnGeluTanh); break;
      case kFnGelu:
        if constexpr (sizeof(AT) == 2) {
          apply(kFnGelu);
          break;
        }
        // a long function in fp32: one copy
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          float z = zg[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) z = i == j ? zg[j] : z;
          z = lin_act<sizeof(AT) == 2>(kFnGelu, z);
#pragma unroll
          for (int j = 0; j < 8; ++j) zg[j] = i == j ? z : zg[j];
        }
        break;
    }
    if (kGated) {
#pragma unroll
      for (int v = 0; v < 8; ++v) zg[v] *= zu[v];
    }
    AT* o = static_cast<AT*>(a.out) + m * a.ldo + n;
    const AT* r = static_cast<const AT*>(a.res) + m * a.ldr + n;
    // (two 16-byte pieces of four fp32, or one of eight bf16)
    if ((sizeof(AT) == 4 ? a.vec4 : a.vec8) && valid == 8) {
      constexpr int kParts = sizeof(AT) == 4 ? 2 : 1;  // 16-byte pieces
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        if constexpr (sizeof(AT) == 4) {
          f32x4 z{zg[4 * p], zg[4 * p + 1], zg[4 * p + 2], zg[4 * p + 3]};
          if (a.res) z += reinterpret_cast<const f32x4*>(r)[p];
          reinterpret_cast<f32x4*>(o)[p] = z;
        } else {
          if (a.res) {
            const uint4 q = *reinterpret_cast<const uint4*>(r);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              zg[2 * i] += __uint_as_float(w[i] << 16);
              zg[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
            }
          }
          // the hardware's conversion: to nearest even, NaN kept
          bf16x8 h;
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = static_cast<__bf16>(zg[i]);
          *reinterpret_cast<bf16x8*>(o) = h;
        }
      }
      return;
    }
#pragma unroll
    for (int v = 0; v < 8; ++v)
      if (v < valid) lin_store(o + v, a.res ? zg[v] + lin_load(r + v) : zg[v]);
  }

  // the sums of this K range instead, where K is split
  __device__ __forceinline__ void store_part(const LinearArgs& a, const float (&zg)[8],
                                             const float (&zu)[8], int64_t m) const {
    float* p = a.part + (static_cast<size_t>(blockIdx.z) * a.part_rows + m) * a.R + n;
#pragma unroll
    for (int h = 0; h < (kGated ? 2 : 1); ++h) {
      const float* z = h ? zu : zg;
      float* q = p + (h ? a.N : 0);
      if (a.N % 4 == 0) {
#pragma unroll
        for (int v = 0; v < 8; v += 4)
          if (v < valid) *reinterpret_cast<f32x4*>(q + v) = f32x4{z[v], z[v + 1], z[v + 2], z[v + 3]};
      } else {
#pragma unroll
        for (int v = 0; v < 8; ++v)
          if (v < valid) q[v] = z[v];
      }
    }
  }
};

// A wave's tile on its way out: its sums go through LDS of its own (2 KB per
// 64 rows), eight tokens at a time, so that a lane finishes eight consecutive
// channels of one token and the wave stores whole lines; the epilogue is one
// short loop whatever the tile.  kRW: weight rows of the wave (gated: gate
// rows, then up rows).
template <typename AT, bool kGated, int kRW>
struct LinOut {
  static constexpr int kC = kGated ? kRW / 2 : kRW;  // channels
  static constexpr int kLanes = kC / 8;              // of a token
  static constexpr int kBytes = 8 * kRW * 4;
  LinOct<AT, kGated> oct;
  f32x4* lds;  // [8 tokens][kRW / 4], units swizzled by the token

  // The channel of the lane's first output among the wave's kC.
  static __device__ __forceinline__ int lane_channel() {
    return (threadIdx.x & 63) % kLanes * 8;
  }
  // four sums of rows 4q .. 4q+3 for token t
  __device__ __forceinline__ void put(int t, int q, f32x4 v) const {
    lds[t * (kRW / 4) + (q ^ (t & 7))] = v;
  }
  // tokens m0 .. m0+7
  __device__ __forceinline__ void flush(const LinearArgs& a, int64_t m0) const {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int lane = threadIdx.x & 63, q = lane % kLanes * 2;
#pragma unroll
    for (int it = 0; it < (8 * kLanes + 63) / 64; ++it) {
      const int t = it * (64 / kLanes) + lane / kLanes;
      if (t >= 8 || m0 + t >= a.M || oct.valid <= 0) continue;
      float zg[8], zu[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 g = lds[t * (kRW / 4) + ((q + h) ^ (t & 7))];
        const f32x4 u = kGated ? lds[t * (kRW / 4) + ((kC / 4 + q + h) ^ (t & 7))] : g;
#pragma unroll
        for (int v = 0; v < 4; ++v) zg[4 * h + v] = g[v], zu[4 * h + v] = u[v];
      }
      if (a.part)
        oct.store_part(a, zg, zu, m0 + t);
      else
        oct.finish(a, zg, zu, m0 + t);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
};

// ------------------------------------------------------------ tiled product
//
// A workgroup computes TN weight rows x TM tokens, its waves in a WN x WM
// grid of TA x TB 16x16 MFMA tiles each.  K moves through LDS in stages of
// 128-byte rows (64 bf16 / 32 fp32 / 128 int8; e4m3fn weights 64 bytes for the
// 64 K of their tokens) split into 16-byte units; unit s of row r sits in slot s ^ swz(r), so
// that the 16 rows a 16-lane group reads for one s fall in 16 different
// 16-byte bank groups.  Gated tiles hold TN/2 gate rows and the matching up
// rows; a wave owns both of a channel.

template <typename WT> struct LinTypes {
  using AT = bf16_t;
  using Acc = f32x4;
  static constexpr int kKC = 64;
};
template <> struct LinTypes<float> {
  using AT = float;
  using Acc = f32x4;
  static constexpr int kKC = 32;
};
template <> struct LinTypes<int8_t> {
  using AT = int8_t;
  using Acc = i32x4;
  static constexpr int kKC = 128;
};
template <typename WT>
inline constexpr bool kLinInt8 = std::is_same_v<WT, int8_t>;
// weights of half the bytes of their tokens: one 16-byte unit against two
template <typename WT>
inline constexpr bool kLinHalf = sizeof(WT) == 1 && !kLinInt8<WT>;

// Four sums of a token as values: int8 products times the token's scale, or
// as they are while K is split (a.part).
__device__ __forceinline__ f32x4 lin_sums(const LinearArgs&, f32x4 acc, float) { return acc; }
__device__ __forceinline__ f32x4 lin_sums(const LinearArgs& a, i32x4 acc, float xs) {
  if (a.part) return __builtin_bit_cast(f32x4, acc);
  f32x4 z;
#pragma unroll
  for (int v = 0; v < 4; ++v) z[v] = static_cast<float>(acc[v]) * xs;  // |sum| < 2^31: 2^-24 off
  return z;
}
// The scale of token m (int8 tokens; a token past the last has none).
template <typename WT>
__device__ __forceinline__ float lin_token_scale(const LinearArgs& a, int64_t m) {
  if constexpr (kLinInt8<WT>) return m < a.M ? a.x_scale[m] : 0.0f;
  return 1.0f;
}

template <typename WT, int WN_, int WM_, int TA_, int TB_>
struct LinGeom {
  using AT = typename LinTypes<WT>::AT;
  using Acc = typename LinTypes<WT>::Acc;
  static constexpr int WN = WN_, WM = WM_, TA = TA_, TB = TB_;
  static constexpr int kThreads = 64 * WN * WM;
  static constexpr int TN = 16 * TA * WN, TM = 16 * TB * WM;
  static constexpr int kKC = LinTypes<WT>::kKC;            // K per stage
  static constexpr int kWRow = kKC * (int)sizeof(WT);      // bytes of a weight row
  static constexpr int kXRow = 128;                        // bytes of a token row
  static constexpr int kWUnits = TN * kWRow / 16 / kThreads;  // 16-byte units per thread
  static constexpr int kXUnits = TM * kXRow / 16 / kThreads;
  static constexpr int kWBytes = TN * kWRow;
  static constexpr int kStage = kWBytes + TM * kXRow;
  static constexpr int kWRowsPerQ = kThreads / (kWRow / 16);
  static constexpr int kXRowsPerQ = kThreads / (kXRow / 16);
  static_assert(kWUnits >= 1 && kXUnits >= 1, "every thread loads");
  static_assert(kWRowsPerQ % 16 == 0 && kXRowsPerQ % 16 == 0, "one swizzle per thread");
};

template <int kRowBytes>
__device__ __forceinline__ int lin_swz(int row) {
  return kRowBytes == 128 ? (row >> 1) & 7 : (row >> 2) & 3;
}

// A 16-byte unit of a row at any byte alignment of its element type.
typedef StreamUnit LinUnit;

// Elements k .. k + 16/sizeof(T) - 1 of a row of K, zero past its end.
template <typename T>
__device__ __forceinline__ u32x4 lin_unit(const T* row, int k, int K) {
  constexpr int n = 16 / (int)sizeof(T);
  if (k + n <= K) return reinterpret_cast<const LinUnit*>(row + k)->v;
  union {
    u32x4 v;
    T e[n];
  } u;
  u.v = u32x4{0, 0, 0, 0};
  if (std::is_same_v<T, int8_t> && K >= n)
    return k < K ? stream_last16(reinterpret_cast<const uint8_t*>(row + k), K - k) : u.v;
#pragma unroll
  for (int i = 0; i < n; ++i)
    if (k + i < K) u.e[i] = row[k + i];
  return u.v;
}

template <class G>
using LinAcc = typename G::Acc[G::TA][G::TB];

// acc += W_rows . X_rows^T over one stage.  wrow(t), xrow(u): LDS rows of
// this lane's 16-row tiles.
template <typename WT, class G>
struct LinFrags {
  static constexpr int kW = kLinHalf<WT> ? 1 : 2;  // 16-byte units per lane and weight tile
  uint4 w[kW][G::TA], x[2][G::TB];
};

template <typename WT, class G>
__device__ __forceinline__ void lin_read(LinFrags<WT, G>& f, const uint8_t* stage,
                                         const int (&wrow)[G::TA], const int (&xrow)[G::TB]) {
  const uint8_t* ws = stage;
  const uint8_t* xs = stage + G::kWBytes;
  const int g = (threadIdx.x & 63) >> 4;
  auto wunit = [&](int t, int s) {
    return *reinterpret_cast<const uint4*>(ws + wrow[t] * G::kWRow +
                                           ((s ^ lin_swz<G::kWRow>(wrow[t])) << 4));
  };
  auto xunit = [&](int u, int s) {
    return *reinterpret_cast<const uint4*>(xs + xrow[u] * G::kXRow +
                                           ((s ^ lin_swz<G::kXRow>(xrow[u])) << 4));
  };
  constexpr int kW = LinFrags<WT, G>::kW;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h < kW)
#pragma unroll
      for (int t = 0; t < G::TA; ++t) f.w[h][t] = wunit(t, 4 * h + g);
    // e4m3fn: a lane's 16 codes are k = 16g .. 16g+15, so its token units are
    // those of the same k
#pragma unroll
    for (int u = 0; u < G::TB; ++u) f.x[h][u] = xunit(u, kW == 1 ? 2 * g + h : 4 * h + g);
  }
}

template <typename WT, class G>
__device__ __forceinline__ void lin_mma(const LinFrags<WT, G>& f, LinAcc<G>& acc) {
  if constexpr (kLinInt8<WT>) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < G::TA; ++t)
#pragma unroll
        for (int u = 0; u < G::TB; ++u)
          acc[t][u] = mfma16x16x64i8(__builtin_bit_cast(u32x4, f.w[h][t]),
                                     __builtin_bit_cast(u32x4, f.x[h][u]), acc[t][u]);
  } else if constexpr (sizeof(WT) == 1) {
    // the first eight codes in one MFMA, the last eight in the next
#pragma unroll
    for (int t = 0; t < G::TA; ++t) {
      const uint4 q = f.w[0][t];
      const bf16x8 lo = as_frag(e4m3x8_to_frag_bits(q.x, q.y));
      const bf16x8 hi = as_frag(e4m3x8_to_frag_bits(q.z, q.w));
#pragma unroll
      for (int u = 0; u < G::TB; ++u) acc[t][u] = mfma16x16x32(lo, as_frag(f.x[0][u]), acc[t][u]);
#pragma unroll
      for (int u = 0; u < G::TB; ++u) acc[t][u] = mfma16x16x32(hi, as_frag(f.x[1][u]), acc[t][u]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (sizeof(WT) == 2) {
#pragma unroll
        for (int t = 0; t < G::TA; ++t)
#pragma unroll
          for (int u = 0; u < G::TB; ++u)
            acc[t][u] = mfma16x16x32(as_frag(f.w[h][t]), as_frag(f.x[h][u]), acc[t][u]);
      } else {
        // MFMA i takes element i of every lane group's four k
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < G::TA; ++t)
#pragma unroll
            for (int u = 0; u < G::TB; ++u)
              acc[t][u] = mfma16x16x4f32(__builtin_bit_cast(f32x4, f.w[h][t])[i],
                                         __builtin_bit_cast(f32x4, f.x[h][u])[i], acc[t][u]);
      }
    }
  }
}

// The channel, of its half of the tile, whose weights go to LDS row `row` of
// the half: the H tiles of a wave take four rows each in turn, so that a lane's
// sums (rows 4g .. 4g+3 of every tile) are 4H consecutive channels and leave in
// 16-byte stores of whole lines (2770 x 2000 x 80 bf16: in row order 14.3 us,
// so 13.0).
template <class G, bool kGated>
__device__ __forceinline__ int lin_channel(int row) {
  constexpr int H = kGated ? G::TA / 2 : G::TA;
  return row / (16 * H) * (16 * H) + row % 16 / 4 * (4 * H) + row / 16 % H * 4 + row % 4;
}

// Tile row of wave row-index wn, tile t: gated waves hold gate tiles, then
// the matching up tiles.
template <class G, bool kGated>
__device__ __forceinline__ int lin_tile_row(int wn, int t) {
  if (!kGated) return 16 * (G::TA * wn + t);
  constexpr int H = G::TA / 2;
  return t < H ? 16 * (H * wn + t) : G::TN / 2 + 16 * (H * wn + t - H);
}

// Store the wave's tiles: finished outputs, or this K range's sums.
template <typename WT, typename OT, class G, bool kGated>
__device__ __forceinline__ void lin_epilogue(const LinearArgs& a, LinAcc<G>& acc, int64_t m0,
                                             int n0, int wn, int wm) {
  const int lane = threadIdx.x & 63;
  const int r16 = lane & 15, g = lane >> 4;
  constexpr int H = kGated ? G::TA / 2 : G::TA;
  const int n1 = n0 + 16 * H * wn + 4 * H * g;  // the lane's channels, 4H of them
  float xs[G::TB];
#pragma unroll
  for (int u = 0; u < G::TB; ++u)
    xs[u] = lin_token_scale<WT>(a, m0 + 16 * (G::TB * wm + u) + r16);
  if constexpr (H % 2 == 0) {
#pragma unroll
    for (int p = 0; p < H / 2; ++p) {
      LinOct<OT, kGated> oct;
      oct.init(a, n1 + 8 * p);
      if (oct.valid <= 0) break;
#pragma unroll
      for (int u = 0; u < G::TB; ++u) {
        const int64_t m = m0 + 16 * (G::TB * wm + u) + r16;
        float zg[8], zu[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 g4 = lin_sums(a, acc[2 * p + h][u], xs[u]);
          const f32x4 u4 = kGated ? lin_sums(a, acc[(2 * p + h + H) % G::TA][u], xs[u]) : g4;
#pragma unroll
          for (int v = 0; v < 4; ++v) zg[4 * h + v] = g4[v], zu[4 * h + v] = u4[v];
        }
        if (m < a.M) {
          if (a.part)
            oct.store_part(a, zg, zu, m);
          else
            oct.finish(a, zg, zu, m);
        }
      }
    }
  } else {
    static_assert(H == 1, "one quad");
    LinQuad<OT, kGated> quad;
    quad.init(a, n1);
    if (quad.valid <= 0) return;
    f32x4 zg[G::TB], zu[G::TB];
#pragma unroll
    for (int u = 0; u < G::TB; ++u) {
      zg[u] = lin_sums(a, acc[0][u], xs[u]);
      zu[u] = kGated ? lin_sums(a, acc[H % G::TA][u], xs[u]) : zg[u];
    }
    if (!a.part) quad.template values<G::TB>(a, zg, zu);
#pragma unroll
    for (int u = 0; u < G::TB; ++u) {
      const int64_t m = m0 + 16 * (G::TB * wm + u) + r16;
      if (m < a.M) {
        if (a.part)
          quad.store_part(a, zg[u], zu[u], m);
        else
          quad.store(a, zg[u], m);
      }
    }
  }
}

// ------------------------------------------------------------ groups of rows
//
// Rows sorted by expert (LinearArgs::grouped): rows offsets[e] ..
// offsets[e + 1] - 1 meet the e-th R x K weights.  A tile never spans two
// experts, so the number of row tiles is only known on the device: every
// workgroup of a grid for the most there can be counts the experts' tiles
// from the offsets and takes its tile of the realised ones.  Every wave does so
// by itself (a lane has every 64th part of the experts; a scan in registers),
// which takes no LDS and no barrier.  Offsets are held to [0, M], whatever they
// are.
struct LinGroups {
  int per;    // experts of a lane
  int at, n;  // row tiles before this lane's experts, and theirs
  int total;  // row tiles in all

  static __device__ __forceinline__ void bounds(const LinearArgs& a, int e, int* begin, int* end) {
    const int M = static_cast<int>(a.M);
    *begin = *end = 0;
    if (e < a.groups) {
      *begin = min(max(a.offsets[e], 0), M);
      *end = min(max(a.offsets[e + 1], *begin), M);
    }
  }
  __device__ __forceinline__ void count(const LinearArgs& a, int tm) {
    const int lane = threadIdx.x & 63;
    per = (a.groups + kWave - 1) / kWave;
    n = 0;
    for (int i = 0; i < per; ++i) {
      int begin, end;
      bounds(a, lane * per + i, &begin, &end);
      n += (end - begin + tm - 1) / tm;
    }
    int incl = n;  // over the rows of 16 lanes, then over the rows
#define LIN_SCAN(ctrl, mask) incl += __builtin_amdgcn_update_dpp(0, incl, ctrl, mask, 0xf, false)
    LIN_SCAN(0x111, 0xf);  // row_shr:1, 2, 4, 8
    LIN_SCAN(0x112, 0xf);
    LIN_SCAN(0x114, 0xf);
    LIN_SCAN(0x118, 0xf);
    LIN_SCAN(0x142, 0xa);  // row_bcast:15 into rows 1, 3
    LIN_SCAN(0x143, 0xc);  // row_bcast:31 into rows 2, 3
#undef LIN_SCAN
    at = incl - n;
    total = __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  // Row tile tx (< total): its first row, and in *a its expert's weights,
  // scales and bias and the end of its rows.
  __device__ __forceinline__ int64_t take(LinearArgs* a, int tx, int tm) const {
    const int lane = threadIdx.x & 63;
    const uint64_t has = __ballot(tx >= at && tx < at + n);
    const int src = __builtin_amdgcn_readfirstlane(__ffsll(static_cast<unsigned long long>(has)) - 1);
    int t = tx - at, ge = 0, gm = 0, gend = 0;
    for (int i = 0; i < per; ++i) {
      int begin, end;
      bounds(*a, lane * per + i, &begin, &end);
      const int k = (end - begin + tm - 1) / tm;
      if (t >= 0 && t < k) ge = lane * per + i, gm = begin + t * tm, gend = end;
      t -= k;
    }
    const int e = __builtin_amdgcn_readlane(ge, src);
    const int m0 = __builtin_amdgcn_readlane(gm, src);
    a->M = __builtin_amdgcn_readlane(gend, src);
    const int64_t r = static_cast<int64_t>(e) * a->R;
    a->w = static_cast<const int8_t*>(a->w) + r * a->ldw;
    if (a->scale) a->scale += a->scale_channel ? r : e;
    if (a->bias) a->bias += r;
    return m0;
  }
};

// The expert of row m among groups, or -1.
__device__ __forceinline__ int lin_group_of(const LinearArgs& a, int64_t m) {
  if (m < a.offsets[0] || m >= a.offsets[a.groups]) return -1;
  int lo = 0, hi = a.groups;  // offsets[lo] <= m < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.offsets[mid] <= m)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Operands staged through registers: rows of any length and alignment.
template <typename WT, typename OT, class G, bool kGated>
__global__ __launch_bounds__(G::kThreads) void linear_staged_kernel(LinearArgs a) {
  using AT = typename G::AT;
  __shared__ __attribute__((aligned(1024))) uint8_t stage[G::kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int gy = (a.N + (kGated ? G::TN / 2 : G::TN) - 1) / (kGated ? G::TN / 2 : G::TN);
  const int n0 = (blockIdx.x % gy) * (kGated ? G::TN / 2 : G::TN);
  int64_t m0 = static_cast<int64_t>(blockIdx.x / gy) * G::TM;
  if constexpr (kLinInt8<WT>)
    if (a.grouped) {
      LinGroups groups;
      groups.count(a, G::TM);
      if (static_cast<int>(blockIdx.x) / gy >= groups.total) return;  // uniform
      m0 = groups.take(&a, blockIdx.x / gy, G::TM);
    }
  const int k_begin = blockIdx.z * a.ksplit;
  const int k_end = min(a.K, k_begin + a.ksplit);
  const int wn = wave % G::WN, wm = wave / G::WN;

  int wrow[G::TA], xrow[G::TB];
#pragma unroll
  for (int t = 0; t < G::TA; ++t) wrow[t] = lin_tile_row<G, kGated>(wn, t) + (lane & 15);
#pragma unroll
  for (int u = 0; u < G::TB; ++u) xrow[u] = 16 * (G::TB * wm + u) + (lane & 15);

  LinAcc<G> acc;
#pragma unroll
  for (int t = 0; t < G::TA; ++t)
#pragma unroll
    for (int u = 0; u < G::TB; ++u) acc[t][u] = typename G::Acc{0, 0, 0, 0};

  const WT* w = static_cast<const WT*>(a.w);
  const AT* x = static_cast<const AT*>(a.x);
  u32x4 wv[G::kWUnits], xv[G::kXUnits];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int q = 0; q < G::kWUnits; ++q) {
      const int tr = q * G::kWRowsPerQ + tid / (G::kWRow / 16);
      const int k = k0 + ((tid % (G::kWRow / 16)) ^ lin_swz<G::kWRow>(tr)) * (16 / (int)sizeof(WT));
      const int half = kGated && tr >= G::TN / 2;
      const int n = n0 + lin_channel<G, kGated>(tr - (half ? G::TN / 2 : 0));
      wv[q] = n < a.N ? lin_unit<WT>(w + (static_cast<int64_t>(half) * a.N + n) * a.ldw, k, k_end)
                      : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int q = 0; q < G::kXUnits; ++q) {
      const int tr = q * G::kXRowsPerQ + tid / 8;
      const int k = k0 + ((tid % 8) ^ lin_swz<G::kXRow>(tr)) * (16 / (int)sizeof(AT));
      xv[q] = m0 + tr < a.M ? lin_unit<AT>(x + (m0 + tr) * a.ldx, k, k_end) : u32x4{0, 0, 0, 0};
    }
  };
  fetch(k_begin);
  for (int k0 = k_begin; k0 < k_end; k0 += G::kKC) {
    __syncthreads();  // the previous stage has been read
#pragma unroll
    for (int q = 0; q < G::kWUnits; ++q)
      *reinterpret_cast<u32x4*>(stage + 16 * (q * G::kThreads + tid)) = wv[q];
#pragma unroll
    for (int q = 0; q < G::kXUnits; ++q)
      *reinterpret_cast<u32x4*>(stage + G::kWBytes + 16 * (q * G::kThreads + tid)) = xv[q];
    __syncthreads();
    if (k0 + G::kKC < k_end) fetch(k0 + G::kKC);  // in flight during the MFMAs
    LinFrags<WT, G> f;
    lin_read<WT, G>(f, stage, wrow, xrow);
    lin_mma<WT, G>(f, acc);
  }
  lin_epilogue<WT, OT, G, kGated>(a, acc, m0, n0, wn, wm);
}

// ------------------------------------------------------------ large products
//
// 256 weight rows x 256 tokens per workgroup, eight waves of 128 x 64 (two
// per SIMD), each wave's tile in four quadrants of 64 x 32.  A K stage of
// 128-byte rows is four pieces of 128 rows (weight rows w0, w1 of the quadrant
// rows; gated: gate rows and up rows; tokens x0, x1 of the quadrant columns),
// each in an LDS array of its own, two buffers.  A stage runs in four phases,
// one per quadrant:
//   load part:    fragments LDS -> registers (eight or four 16-byte reads); the
//                 direct-to-LDS loads of one piece; a wait for the piece that
//                 the next phase reads
//   matrix part:  the quadrant's MFMAs
// with a workgroup barrier after each part.  The waves of one half of the
// workgroup run one barrier behind the others: on every SIMD one wave's
// MFMAs run while the other loads, with the matrix wave's priority raised.
// The quadrants go (0,f) (0,o) (1,o) (1,f) with f the stage's first token
// column, 0 in even stages and 1 in odd ones, so that the last phase can read
// the next stage's first tokens into the registers that have just become
// free, and every phase reads at most eight fragments.  A piece of the stage
// after the next is loaded as soon as both halves have read the piece it
// replaces, six phases (over a microsecond) before it is read.  Rows past M
// or N and K past the end read from past the end of their buffer resource:
// zeros, without a memory access.

constexpr int kPpThreads = 512;
constexpr int kPpCols = 4;  // channel tiles of a super-row of the raster
constexpr int kPpPiece = 128;  // rows of a piece
constexpr uint32_t kPpDead = 0x80000000u;  // an offset past every resource

__device__ __forceinline__ void pp_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
template <int N>
__device__ __forceinline__ void pp_wait_loads() {
  static_assert(N >= 0 && N <= 63, "six-bit count");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// 16 bytes per lane from a resource straight into LDS (64 lanes: 1 KB from
// `lds`).
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off,
                                           int base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off,
                                           base, 0, 0);
}

// One operand's direct-to-LDS loads: piece p holds rows 128p .. 128p+127 of
// the tile.
template <typename T, int kRowBytes>
struct PpLoader {
  static constexpr int kUnits = kRowBytes / 16;                       // per row
  static constexpr int kLoads = kPpPiece * kUnits / kPpThreads;       // per piece and thread
  static constexpr int kStep = kPpThreads / kUnits;                   // rows between loads
  static_assert(kLoads >= 1, "every thread loads");
  __amdgpu_buffer_rsrc_t r[2];
  uint32_t off[kLoads];
  int ke;  // this lane's K within a stage

  // base*: the pieces' first rows; rows*: their rows that exist (others lie
  // past the resource's end); K in elements
  __device__ __forceinline__ void init(const uint8_t* base0, const uint8_t* base1, int64_t rows0,
                                       int64_t rows1, int64_t ld, int K) {
    const int tid = threadIdx.x;
    const int row = tid / kUnits;
    ke = ((tid % kUnits) ^ lin_swz<kRowBytes>(row)) * (16 / (int)sizeof(T));
    r[0] = resource(base0, rows0, ld, K);
    r[1] = resource(base1, rows1, ld, K);
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      off[q] = static_cast<uint32_t>((row + q * kStep) * ld + ke) * (uint32_t)sizeof(T);
  }
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t* base,
                                                                    int64_t rows, int64_t ld,
                                                                    int K) {
    const int64_t n = rows < kPpPiece ? rows : kPpPiece;
    const int64_t bytes = n > 0 ? ((n - 1) * ld + K) * (int)sizeof(T) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0,
                                             static_cast<int>(bytes), 0x00020000);
  }
  // K k0 .. of piece p into lds
  __device__ __forceinline__ void issue(int p, uint8_t* lds, int k0, int k_end) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      lds_load16(r[p], lds + (q * kPpThreads + 64 * wave) * 16,
                 k0 + ke < k_end ? off[q] : kPpDead, k0 * (int)sizeof(T));
  }
};

template <typename WT>
struct PpTypes {
  using AT = typename LinTypes<WT>::AT;
  static constexpr int kKC = LinTypes<WT>::kKC;
  static constexpr int kWRow = kKC * (int)sizeof(WT);
  static constexpr int kWFrags = kWRow / 64;  // 16-byte reads per row and stage
  static constexpr int kW = 4, kX = 2;        // 16-row tiles of a quadrant
};

template <typename WT>
struct PpFrags {
  using P = PpTypes<WT>;
  u32x4 w[P::kW][P::kWFrags];
  u32x4 x[2][P::kX][2];  // both quadrant columns
};

template <typename WT>
__device__ __forceinline__ void pp_read_w(PpFrags<WT>& f, const uint8_t* piece, int row0) {
  using P = PpTypes<WT>;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int t = 0; t < P::kW; ++t) {
    const int row = row0 + 16 * t + (lane & 15);
#pragma unroll
    for (int h = 0; h < P::kWFrags; ++h)
      f.w[t][h] = *reinterpret_cast<const u32x4*>(
          piece + row * P::kWRow + (((4 * h + (lane >> 4)) ^ lin_swz<P::kWRow>(row)) << 4));
  }
}
template <typename WT>
__device__ __forceinline__ void pp_read_x(PpFrags<WT>& f, int j, const uint8_t* piece, int row0) {
  using P = PpTypes<WT>;
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int u = 0; u < P::kX; ++u) {
    const int row = row0 + 16 * u + (lane & 15);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = kLinHalf<WT> ? 2 * g + h : 4 * h + g;
      f.x[j][u][h] = *reinterpret_cast<const u32x4*>(piece + row * 128 +
                                                     ((slot ^ lin_swz<128>(row)) << 4));
    }
  }
}

template <typename WT>
using PpAcc = typename LinTypes<WT>::Acc[PpTypes<WT>::kW][PpTypes<WT>::kX];

template <typename WT>
__device__ __forceinline__ void pp_mma(const PpFrags<WT>& f, int j, PpAcc<WT>& acc) {
  using P = PpTypes<WT>;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int t = 0; t < P::kW; ++t) {
      if constexpr (kLinInt8<WT>) {
#pragma unroll
        for (int u = 0; u < P::kX; ++u)
          acc[t][u] = mfma16x16x64i8(f.w[t][h], f.x[j][u][h], acc[t][u]);
      } else {
        bf16x8 w;
        if constexpr (sizeof(WT) == 2)
          w = __builtin_bit_cast(bf16x8, f.w[t][h]);
        else
          w = as_frag(e4m3x8_to_frag_bits(f.w[t][0][2 * h], f.w[t][0][2 * h + 1]));
#pragma unroll
        for (int u = 0; u < P::kX; ++u)
          acc[t][u] = mfma16x16x32(w, __builtin_bit_cast(bf16x8, f.x[j][u][h]), acc[t][u]);
      }
    }
  }
}

template <typename WT, bool kGated>
struct PpTile {
  using P = PpTypes<WT>;
  using AT = typename P::AT;
  using LW = PpLoader<WT, P::kWRow>;
  using LX = PpLoader<AT, 128>;
  const LW& lw;
  const LX& lx;
  int wrow, xrow;  // this wave's first row in a piece
  int k_begin, k_end;

  // One stage from the pieces w0, w1, x0, x1; its first tokens are already in
  // registers, those of the next stage (piece nx of the other buffer) are
  // read.  kTail: 0 loads the stage after the next (K from kn) into the
  // pieces just read; 1, 2: the last stage but one, the last.
  template <int kFirst, int kTail>
  __device__ __forceinline__ void stage(uint8_t* w0, uint8_t* w1, uint8_t* x0, uint8_t* x1,
                                        const uint8_t* nx, int kn, PpFrags<WT>& f,
                                        PpAcc<WT> (&acc)[2][2]) const {
    constexpr int W = LW::kLoads, X = LX::kLoads, O = 1 - kFirst;
    uint8_t* const xf = kFirst ? x1 : x0;
    uint8_t* const xo = kFirst ? x0 : x1;
    // the loads issued after the piece that must have landed may be in flight
    pp_read_w<WT>(f, w0, wrow);
    if (kTail == 0) lx.issue(kFirst, xf, kn, k_end);
    pp_wait_loads<kTail == 0 ? 3 * W + 3 * X : kTail == 1 ? 3 * W + 2 * X : W>();  // xo
    matrix(f, kFirst, acc[0][kFirst]);
    pp_read_x<WT>(f, O, xo, xrow);
    if (kTail == 0) lw.issue(0, w0, kn, k_end);
    pp_wait_loads<kTail == 0 ? 3 * W + 3 * X : kTail == 1 ? 2 * W + 2 * X : 0>();  // w1
    matrix(f, O, acc[0][O]);
    pp_read_w<WT>(f, w1, wrow);
    if (kTail == 0) lx.issue(O, xo, kn, k_end);
    if (kTail < 2) pp_wait_loads<kTail == 0 ? 3 * W + 3 * X : 2 * W + X>();  // nx
    matrix(f, O, acc[1][O]);
    if (kTail < 2) pp_read_x<WT>(f, O, nx, xrow);
    if (kTail == 0) lw.issue(1, w1, kn, k_end);
    if (kTail < 2) pp_wait_loads<kTail == 0 ? 3 * W + 3 * X : W + X>();  // the next w0
    matrix(f, kFirst, acc[1][kFirst]);
  }

  __device__ __forceinline__ void matrix(const PpFrags<WT>& f, int j, PpAcc<WT>& acc) const {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    pp_barrier();
    __builtin_amdgcn_s_setprio(1);
    pp_mma<WT>(f, j, acc);
    __builtin_amdgcn_s_setprio(0);
    pp_barrier();
  }
};

// Workgroup p's tile: contiguous runs of the logical order per XCD
// (workgroup p runs on XCD p mod 8), in super-rows of kCols channel tiles
// with the token tiles inside, so that the tiles an XCD runs together share
// weight rows and token rows in its L2.
__device__ __forceinline__ bool lin_raster(int p, int gx, int gy, int cols, int* tx, int* ty) {
  const int total = gx * gy, per = (total + 7) / 8;
  const int l = p % 8 * per + p / 8;
  if (p / 8 >= per || l >= total) return false;
  const int band = cols * gx, sr = l / band, rem = l - sr * band;
  const int c = min(cols, gy - sr * cols);
  *tx = rem / c;
  *ty = sr * cols + rem % c;
  return true;
}

template <typename WT, typename OT, bool kGated>
__global__ __launch_bounds__(kPpThreads, 2) void linear_pp_kernel(LinearArgs a, int gx, int gy) {
  using P = PpTypes<WT>;
  using AT = typename P::AT;
  using T = PpTile<WT, kGated>;
  constexpr int kWP = kPpPiece * P::kWRow, kXP = kPpPiece * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t w00[kWP], w01[kWP], x00[kXP], x01[kXP];
  __shared__ __attribute__((aligned(1024))) uint8_t w10[kWP], w11[kWP], x10[kXP], x11[kXP];
  __shared__ __attribute__((aligned(1024))) uint8_t sums[8][4096];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kCh = kGated ? kPpPiece : 2 * kPpPiece;  // channels of a tile
  LinGroups groups;
  if constexpr (kLinInt8<WT>)
    if (a.grouped) {
      groups.count(a, 256);
      gx = min(gx, groups.total);  // (wrong offsets can make more)
    }
  int tx, ty;
  if (!lin_raster(blockIdx.x, gx, gy, kPpCols, &tx, &ty)) return;  // uniform
  const int n0 = ty * kCh;
  int64_t m0 = static_cast<int64_t>(tx) * 256;
  if constexpr (kLinInt8<WT>)
    if (a.grouped) m0 = groups.take(&a, tx, 256);
  const int k_begin = blockIdx.z * a.ksplit;
  const int k_end = min(a.K, k_begin + a.ksplit);

  typename T::LW lw;
  const uint8_t* wb = static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * a.ldw * sizeof(WT);
  const size_t second = static_cast<size_t>(kGated ? a.N : kPpPiece) * a.ldw * sizeof(WT);
  lw.init(wb, wb + second, a.N - n0, a.N - n0 - (kGated ? 0 : kPpPiece), a.ldw, a.K);
  typename T::LX lx;
  const uint8_t* xb = static_cast<const uint8_t*>(a.x) + m0 * a.ldx * sizeof(AT);
  lx.init(xb, xb + kPpPiece * a.ldx * sizeof(AT), a.M - m0, a.M - m0 - kPpPiece, a.ldx, a.K);

  const int wm = wave & 1, wn = wave >> 1;  // weight rows, tokens
  const T tile{lw, lx, 64 * wm, 32 * wn, k_begin, k_end};
  PpAcc<WT> acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < P::kW; ++t)
#pragma unroll
        for (int u = 0; u < P::kX; ++u)
          acc[i][j][t][u] = typename LinTypes<WT>::Acc{0, 0, 0, 0};
  PpFrags<WT> f;

  // int8: the tile's scales and biases, loaded ahead of the stages and kept in
  // the epilogue's LDS, so that no load is waited for behind the last stage
  float scale = 0.f, bias = 0.f;
  if constexpr (kLinInt8<WT>) {
    const int r = threadIdx.x % 256;  // a row of W (gated: gate rows, then up), or a token
    const int c = min(n0 + (kGated ? r % kPpPiece : r), a.N - 1) + (kGated && r >= kPpPiece ? a.N : 0);
    if (threadIdx.x < 256) {
      scale = a.scale[a.scale_channel ? c : 0];
      bias = a.bias ? a.bias[c] : 0.f;
    } else {
      scale = m0 + r < a.M ? a.x_scale[m0 + r] : 0.f;
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  constexpr int KC = P::kKC;
  lx.issue(0, x00, k_begin, k_end);
  lw.issue(0, w00, k_begin, k_end);
  lx.issue(1, x01, k_begin, k_end);
  lw.issue(1, w01, k_begin, k_end);
  lx.issue(1, x11, k_begin + KC, k_end);
  lw.issue(0, w10, k_begin + KC, k_end);
  lx.issue(0, x10, k_begin + KC, k_end);
  lw.issue(1, w11, k_begin + KC, k_end);
  pp_wait_loads<3 * (T::LW::kLoads + T::LX::kLoads)>();  // stage 0's x0 and w0
  float* const rows = reinterpret_cast<float*>(sums);    // scales, biases, tokens' scales
  if constexpr (kLinInt8<WT>) {
    rows[threadIdx.x < 256 ? threadIdx.x : 256 + threadIdx.x] = scale;
    if (threadIdx.x < 256) rows[256 + threadIdx.x] = bias;
  }
  pp_barrier();
  pp_read_x<WT>(f, 0, x00, tile.xrow);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  pp_barrier();  // x00 may be overwritten
  const bool late = wave >= 4;  // one barrier behind
  if (late) pp_barrier();
  // two stages at a time (an odd count's last one reads zeros), the last two
  // outside the loop
  int k = k_begin;
  for (; k + 2 * KC < k_end; k += 2 * KC) {
    tile.template stage<0, 0>(w00, w01, x00, x01, x11, k + 2 * KC, f, acc);
    tile.template stage<1, 0>(w10, w11, x10, x11, x00, k + 3 * KC, f, acc);
  }
  tile.template stage<0, 1>(w00, w01, x00, x01, x11, 0, f, acc);
  tile.template stage<1, 2>(w10, w11, x10, x11, nullptr, 0, f, acc);
  if (!late) pp_barrier();

  // 128 weight rows of the wave: 64 of each piece (gated: 64 gate, 64 up)
  using Out = LinOut<OT, kGated, 128>;
  Out out;
  out.lds = reinterpret_cast<f32x4*>(sums[wave]);
  const int c = Out::lane_channel();
  const int ch = 64 * wm + c + (!kGated && c >= 64 ? 64 : 0);  // of the tile
  if constexpr (kLinInt8<WT>)
    out.oct.init(a, n0 + ch, rows, rows + 256, ch, kGated ? kPpPiece + ch : 0);
  else
    out.oct.init(a, n0 + ch);
  const int r16 = lane & 15, g = lane >> 4;
  // int8: all sums become values first (in the loop below the choice of four
  // would take a conversion each: 4096 x 14336 gated x 4096 452 us)
  f32x4 z[2][2][P::kW][P::kX];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int u = 0; u < P::kX; ++u) {
      const float xs = kLinInt8<WT> ? rows[512 + 128 * j + 32 * wn + 16 * u + r16] : 1.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < P::kW; ++t) z[i][j][t][u] = lin_sums(a, acc[i][j][t][u], xs);
    }
  if constexpr (kLinInt8<WT>) __syncthreads();  // every wave has read the scales
#pragma unroll 1
  for (int h = 0; h < 8; ++h) {  // eight tokens of token tile u = h / 2 % 2, column j = h / 4
    if (r16 / 8 == h % 2) {
#pragma unroll
      for (int ju = 0; ju < 4; ++ju)
        if (h / 2 == ju) {
#pragma unroll
          for (int t = 0; t < P::kW; ++t) {
            out.put(r16 & 7, 4 * t + g, z[0][ju / 2][t][ju % 2]);
            out.put(r16 & 7, 16 + 4 * t + g, z[1][ju / 2][t][ju % 2]);
          }
        }
    }
    out.flush(a, m0 + 128 * (h / 4) + 32 * wn + 8 * (h % 4));
  }
}

// ------------------------------------------------------------ middle sizes
//
// LinGeom's tile with both operands by direct-to-LDS loads, through a ring of
// S stages in LDS arrays of their own (reads of one stage then wait for no
// load into another): S - 1 stages are in flight while one is multiplied, so
// a workgroup alone on its compute unit covers the memory latency.  What is
// left is a fixed part of every stage (barrier, waits, fragment reads: 0.25 us)
// and what a compute unit takes in, about 60 GB/s of 128-byte row pieces: 0.54 us
// for the 16 KB of a 64 x 64 stage, alike with four stages and with eight.

// One operand of a tile: kRows rows, of which [0, kSplit) start at one base
// and the rest at another (gated weights; else kSplit = kRows).
template <typename T, int kRowBytes, int kThreads, int kRows, int kSplit>
struct TileLoader {
  static constexpr int kUnits = kRowBytes / 16;
  static constexpr int kStep = kThreads / kUnits;             // rows per load
  static constexpr int kLoads = kRows / kStep;                // per stage and thread
  static_assert(kRows % kStep == 0 && kSplit % (64 / kUnits) == 0, "whole loads");
  static_assert(kStep % 16 == 0, "one swizzle per thread");
  __amdgpu_buffer_rsrc_t r[2];
  uint32_t off[kLoads];
  int ke;

  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t* base,
                                                                    int64_t rows, int64_t ld,
                                                                    int K) {
    const int64_t n = rows < kRows ? rows : kRows;
    const int64_t bytes = n > 0 ? ((n - 1) * ld + K) * (int)sizeof(T) : 0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0,
                                             static_cast<int>(bytes), 0x00020000);
  }
  // source(row): the matrix's row for LDS row `row` of a half
  template <typename F>
  __device__ __forceinline__ void init(const uint8_t* base0, const uint8_t* base1, int64_t rows,
                                       int64_t ld, int K, F source) {
    const int row = threadIdx.x / kUnits;
    ke = ((threadIdx.x % kUnits) ^ lin_swz<kRowBytes>(row)) * (16 / (int)sizeof(T));
    r[0] = resource(base0, kSplit < kRows && rows > kSplit ? kSplit : rows, ld, K);
    r[1] = resource(base1, rows > kSplit ? kSplit : rows, ld, K);
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      off[q] = static_cast<uint32_t>(source((row + q * kStep) % kSplit) * ld + ke) *
               (uint32_t)sizeof(T);
  }
  __device__ __forceinline__ void issue(uint8_t* lds, int k0, int k_end) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      lds_load16(q * kStep + wave * (64 / kUnits) >= kSplit ? r[1] : r[0],
                 lds + (q * kThreads + 64 * wave) * 16,
                 k0 + ke < k_end ? off[q] : kPpDead, k0 * (int)sizeof(T));
  }
};

// f(LinInt<A>), ..., f(LinInt<B - 1>)
template <int A, int B, class F>
__device__ __forceinline__ void lin_for(const F& f) {
  if constexpr (A < B) {
    f(LinInt<A>{});
    lin_for<A + 1, B>(f);
  }
}

template <typename WT, typename OT, class G, int S, bool kGated>
__global__ __launch_bounds__(G::kThreads) void linear_tile_kernel(LinearArgs a, int gx, int gy) {
  using AT = typename G::AT;
  // A workgroup that is alone on its compute unit reads a stage's fragments
  // while it multiplies the one before (512 x 7168 x 4096 bf16, 128 x 128:
  // 59.6 -> 51.3 us); two that take turns need not, and their 128 registers
  // hold no second set.  64 x 64 tiles gain 2% and, short as their products
  // are, lose as much to the longer start.
  constexpr bool kAhead = S > 3 && G::TN > 64;
  static_assert(S >= 2 && S <= 6 && (S % 2 == 0 || !kAhead), "ring depth");
  constexpr int kCh = kGated ? G::TN / 2 : G::TN;
  // arrays of their own: reads of one stage wait for no load into another
  __shared__ __attribute__((aligned(1024))) uint8_t s0[G::kStage], s1[G::kStage],
      s2[S > 2 ? G::kStage : 16], s3[S > 3 ? G::kStage : 16], s4[S > 4 ? G::kStage : 16],
      s5[S > 5 ? G::kStage : 16];
  auto ring = [&](auto i) -> uint8_t* {
    constexpr int k = decltype(i)::value % S;
    if constexpr (k == 0) return s0;
    if constexpr (k == 1) return s1;
    if constexpr (k == 2) return s2;
    if constexpr (k == 3) return s3;
    if constexpr (k == 4) return s4;
    if constexpr (k == 5) return s5;
  };
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  LinGroups groups;
  if constexpr (kLinInt8<WT>)
    if (a.grouped) {
      groups.count(a, G::TM);
      gx = min(gx, groups.total);  // (wrong offsets can make more)
    }
  int tx, ty;
  if (!lin_raster(blockIdx.x, gx, gy, kPpCols, &tx, &ty)) return;  // uniform
  const int n0 = ty * kCh;
  int64_t m0 = static_cast<int64_t>(tx) * G::TM;
  if constexpr (kLinInt8<WT>)
    if (a.grouped) m0 = groups.take(&a, tx, G::TM);
  const int k_begin = blockIdx.z * a.ksplit;
  const int k_end = min(a.K, k_begin + a.ksplit);
  const int nst = (k_end - k_begin + G::kKC - 1) / G::kKC;

  TileLoader<WT, G::kWRow, G::kThreads, G::TN, kCh> lw;
  const uint8_t* wb = static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * a.ldw * sizeof(WT);
  lw.init(wb, wb + static_cast<size_t>(a.N) * a.ldw * sizeof(WT), a.N - n0, a.ldw, a.K,
          lin_channel<G, kGated>);
  TileLoader<AT, G::kXRow, G::kThreads, G::TM, G::TM> lx;
  const uint8_t* xb = static_cast<const uint8_t*>(a.x) + m0 * a.ldx * sizeof(AT);
  lx.init(xb, xb, a.M - m0, a.ldx, a.K, [](int row) { return row; });
  constexpr int L = decltype(lw)::kLoads + decltype(lx)::kLoads;

  const int wn = wave % G::WN, wm = wave / G::WN;
  int wrow[G::TA], xrow[G::TB];
#pragma unroll
  for (int t = 0; t < G::TA; ++t) wrow[t] = lin_tile_row<G, kGated>(wn, t) + (lane & 15);
#pragma unroll
  for (int u = 0; u < G::TB; ++u) xrow[u] = 16 * (G::TB * wm + u) + (lane & 15);
  LinAcc<G> acc;
#pragma unroll
  for (int t = 0; t < G::TA; ++t)
#pragma unroll
    for (int u = 0; u < G::TB; ++u) acc[t][u] = typename G::Acc{0, 0, 0, 0};

  auto issue = [&](uint8_t* st, int i) {
    lw.issue(st, k_begin + i * G::kKC, k_end);
    lx.issue(st + G::kWBytes, k_begin + i * G::kKC, k_end);
  };
  // Stage i is in buffer (i + first) % S: the last one is in the ring's last
  // buffer, so that whole turns follow the first, shortened one.
  const int first = (S - nst % S) % S;
  constexpr int kFirst = kAhead ? S : S - 1;  // stages issued before the first is used
  lin_for<0, 2 * S - 1>([&](auto j) {         // in order
    const int i = j.value - first;
    if (i >= 0 && i < kFirst && i < nst) issue(ring(j), i);
  });
  LinFrags<WT, G> f[kAhead ? 2 : 1];
  if constexpr (kAhead) {
    if (nst >= S)
      pp_wait_loads<L * (S - 1)>();
    else
      pp_wait_loads<0>();
    asm volatile("s_barrier" ::: "memory");
    lin_for<0, S>([&](auto j) {
      if (j.value == first) lin_read<WT, G>(f[j.value % 2], ring(j), wrow, xrow);
    });
  }
  for (int turn = -first; turn < nst; turn += S)
    lin_for<0, S>([&](auto j) {
      constexpr int J = decltype(j)::value;
      const int i = turn + J;
      if (i < 0) return;  // uniform
      if constexpr (kAhead) {
        if (i + S < nst) {
          pp_wait_loads<L * (S - 2)>();  // stage i + 1 has landed
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          issue(ring(j), i + S);  // every wave has read stage i
        } else if (J + 1 < S) {
          pp_wait_loads<L * (J + 2 < S ? S - 2 - J : 0)>();
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        __builtin_amdgcn_sched_barrier(0);
        // (after the last stage, of a buffer whose contents mean nothing)
        lin_read<WT, G>(f[(J + 1) % 2], ring(LinInt<J + 1>{}), wrow, xrow);
        __builtin_amdgcn_sched_barrier(0);
        lin_mma<WT, G>(f[J % 2], acc);
      } else {
        if (i + S - 1 < nst) {
          pp_wait_loads<L * (S - 2)>();  // stage i has landed
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          issue(ring(LinInt<J + S - 1>{}), i + S - 1);  // every wave has read stage i - 1
        } else {
          pp_wait_loads<0>();
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        __builtin_amdgcn_sched_barrier(0);
        lin_read<WT, G>(f[0], ring(j), wrow, xrow);
        lin_mma<WT, G>(f[0], acc);
      }
    });
  lin_epilogue<WT, OT, G, kGated>(a, acc, m0, n0, wn, wm);
}

// The K ranges' sums of four channels of a token, added in order and finished.
constexpr int kReduceThreads = 256;
template <typename WT, typename OT, bool kGated>
__global__ __launch_bounds__(kReduceThreads) void linear_reduce_kernel(LinearArgs a) {
  using Acc = typename LinTypes<WT>::Acc;
  const int quads = (a.N + 3) / 4;
  const int64_t o = static_cast<int64_t>(blockIdx.x) * kReduceThreads + threadIdx.x;
  const int64_t m = o / quads;
  if (m >= a.M) return;
  if constexpr (kLinInt8<WT>)
    if (a.grouped) {
      const int e = lin_group_of(a, m);
      if (e < 0) return;
      const int64_t r = static_cast<int64_t>(e) * a.R;
      if (a.scale) a.scale += a.scale_channel ? r : e;
      if (a.bias) a.bias += r;
    }
  LinQuad<OT, kGated> quad;
  quad.init(a, static_cast<int>(o % quads) * 4);
  Acc sg{0, 0, 0, 0}, su{0, 0, 0, 0};
  // four ranges' loads at a time (ranges past the last repeat it, not added; one
  // at a time 51 x 136 x 5704 fp32 took 18.5 us, so 15.0, eight the same)
  for (int z0 = 0; z0 < a.splits; z0 += 4) {
    f32x4 g[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int z = min(z0 + i, a.splits - 1);
      const float* p = a.part + (static_cast<size_t>(z) * a.part_rows + m) * a.R + quad.n;
      if (a.N % 4 == 0) {
        g[i] = *reinterpret_cast<const f32x4*>(p);
        if (kGated) u[i] = *reinterpret_cast<const f32x4*>(p + a.N);
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int c = min(v, quad.valid - 1);  // (never stored past valid)
          g[i][v] = p[c];
          if (kGated) u[i][v] = p[a.N + c];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (z0 + i < a.splits) {
        sg += __builtin_bit_cast(Acc, g[i]);
        if (kGated) su += __builtin_bit_cast(Acc, u[i]);
      }
  }
  a.part = nullptr;
  const float xs = lin_token_scale<WT>(a, m);
  f32x4 zg[1] = {lin_sums(a, sg, xs)}, zu[1] = {kGated ? lin_sums(a, su, xs) : zg[0]};
  quad.template values<1>(a, zg, zu);
  quad.store(a, zg[0], m);
}

// ------------------------------------------------------------ few tokens
//
// At most 16 tokens (int8: 64): the product is a read of W (stream.h).  A workgroup
// takes 16 * RT weight rows (gated: half of them gate rows, half the matching
// up rows), its eight waves every eighth K chunk each, so that together they
// read 2 KB of a row at a time; the waves' sums meet in LDS in a fixed order.
//
// int8: four waves.  A wave's share of a row is half that of bf16, so the sum
// over the waves weighs twice as much, and more and smaller workgroups keep
// streaming beside one that adds (16 x 14336 gated x 4096 27.1 us with eight, 23.3
// with four, 23.5 with two; 16 x 4096 x 14336 13.3, 13.2, 14.8).
//
// 17 to 64 tokens: a workgroup alone on its compute unit takes in about 45 GB/s
// with these loads in flight (a measured rate of this kernel, no limit of the chip),
// and two thirds of that or more are tokens, which pass through LDS with the weights;
// 144 KB of it hold six waves (32 x 4096 x 14336: four 17.5 us, six
// 16.5; up to 48 tokens 160 KB hold five, up to 64 four), or four with two row
// tiles each, which halves the tokens where there are more tiles than units
// (32 x 7168 x 7168: 17.4 us with one tile, 13.9 with two).

template <typename WT>
inline constexpr int kLinStreamThreads = kLinInt8<WT> ? 256 : 512;

// kQuads: at most four tokens, 4x4 MFMAs, else 16x16 (RT tiles of 16 rows;
// gated: eight gate rows, then eight up rows), XT tiles of 16 tokens.
template <typename WT, typename OT, int RT, bool kQuads, bool kGated, bool kAligned, int XT,
          int kThreads>
__global__ __launch_bounds__(kThreads, XT > 1 ? 1 : RT > 1 ? 2 : 4) void linear_stream_kernel(
    LinearArgs a) {
  using G = StreamGeom<WT>;
  using AT = typename G::AT;
  using Acc = typename StreamTypes<WT>::Acc;
  using S16 = Stream16<WT, RT, kAligned, false, XT>;
  constexpr int kWaves = kThreads / kWave;
  constexpr int kRows = 16 * RT, kCh = kGated ? kRows / 2 : kRows;
  constexpr int kTok = kQuads ? 4 : 16 * XT, kParts = kQuads ? 4 * kWaves : kWaves;
  // partial sums of four rows of a token; before them, the waves' weights
  union Lds {
    Acc red[kParts][kRows / 4][kTok];
    uint8_t w[!kQuads && kAligned ? kWaves : 1][!kQuads && kAligned ? S16::kLds : 16];
  };
  __shared__ __attribute__((aligned(1024))) Lds lds;
  __shared__ __attribute__((aligned(1024))) uint8_t w1[!kQuads && kAligned ? kWaves : 1]
                                                      [!kQuads && kAligned ? S16::kLds : 16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * kCh;
  const size_t ldb = a.ldw * sizeof(WT);
  const int full = a.K / G::kChunk, left = a.K % G::kChunk;
  const int mine = full > wave ? (full - wave + kWaves - 1) / kWaves : 0;
  const bool last = left && full % kWaves == wave;
  const int M = static_cast<int>(a.M);
  // The workgroup's channel c as a weight row, in its half of W; channels
  // past the last repeat it (never stored).
  auto first = [&](int c, bool up) {
    return static_cast<const uint8_t*>(a.w) +
           ((up ? static_cast<size_t>(a.N) : 0) + min(n0 + c, a.N - 1)) * ldb;
  };
  auto offset = [&](int c, int r) {  // from first(c) to row r after it
    return static_cast<uint32_t>((min(n0 + c + r, a.N - 1) - min(n0 + c, a.N - 1)) * ldb);
  };

  if constexpr (kQuads) {
    Stream<WT, 4 * RT, 1, kAligned> st;
#pragma unroll
    for (int q = 0; q < 4 * RT; ++q) {
      const int r = 4 * q % (kRows / 2);  // its first row in its half
      st.place(q, [&](int i) { return offset(q < 2 * RT || kGated ? 0 : kRows / 2, r + i); });
    }
    st.wq[0] = first(0, false);
    st.wq[1] = first(kGated ? 0 : kRows / 2, kGated);
    st.xb = static_cast<const uint8_t*>(a.x);
    st.xo[0] = static_cast<uint32_t>(min(lane & 3, M - 1) * a.ldx * sizeof(AT)) +
               (lane >> 2) * (G::kLaneK * sizeof(AT));
    Acc acc[4 * RT][1];
#pragma unroll
    for (int q = 0; q < 4 * RT; ++q) acc[q][0] = Acc{0, 0, 0, 0};
    st.template run<4 / RT>(wave, mine, kWaves, acc);
    if (last) st.tail(full, left, acc);
#pragma unroll
    for (int q = 0; q < 4 * RT; ++q) {
      Acc v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = stream_row_sum(acc[q][0][i]);
      if ((lane & 12) == 0) lds.red[4 * wave + (lane >> 4)][q][lane & 3] = v;
    }
  } else {
    S16 st;
    auto row_off = [&](int t, int r) {
      return kGated ? offset(8 * t, r & 7) : offset(16 * t + (r & 8), r & 7);
    };
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      st.wq[t][0] = first(kGated ? 8 * t : 16 * t, false);
      st.wq[t][1] = first(kGated ? 8 * t : 16 * t + 8, kGated);
      st.place(t, [&](int r) { return row_off(t, r); });
    }
    st.lds[0] = lds.w[!kQuads && kAligned ? wave : 0];
    st.lds[1] = w1[!kQuads && kAligned ? wave : 0];
    st.xb = static_cast<const uint8_t*>(a.x);
    st.place_tokens(M, static_cast<uint32_t>(a.ldx * sizeof(AT)));
    Acc acc[RT * XT];
#pragma unroll
    for (int t = 0; t < RT * XT; ++t) acc[t] = Acc{0, 0, 0, 0};
    st.run(wave, mine, kWaves, acc);
    if (last) st.tail(full, left, row_off, acc);
    __syncthreads();  // the weights have been read
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int y = 0; y < XT; ++y)
        lds.red[wave][4 * t + (lane >> 4)][16 * y + (lane & 15)] = acc[t * XT + y];
  }
  __syncthreads();
  for (int o = tid; o < kCh * kTok; o += kThreads) {
    const int c = o % kCh, m = o / kCh;
    if (m >= M || n0 + c >= a.N) continue;
    // the LDS rows of channel c (gate) and of its up row
    const int rg = kGated && !kQuads ? c / 8 * 16 + c % 8 : c;
    const int ru = kQuads ? (kCh + c) % kRows : (rg + 8) % kRows;
    std::remove_reference_t<decltype(lds.red[0][0][0][0])> zg = 0, zu = 0;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      zg += lds.red[p][rg / 4][m][rg % 4];
      if (kGated) zu += lds.red[p][ru / 4][m][ru % 4];
    }
    if constexpr (kLinInt8<WT>) {
      const float xs = a.x_scale[m];
      lin_finish<OT>(a, static_cast<float>(zg) * xs, static_cast<float>(zu) * xs, m, n0 + c);
    } else {
      lin_finish<OT>(a, zg, zu, m, n0 + c);
    }
  }
}

// ------------------------------------------------------------ packing
//
// Rows that do not start at multiples of 16 bytes cannot go through the
// direct-to-LDS loads; where the product is large enough to pay for it they
// are copied into the workspace first, each row to a multiple of 16 bytes and
// zero past its end.  A thread makes one 16-byte unit of x or of W.

constexpr int kPackThreads = 256;
template <typename WT>
__global__ __launch_bounds__(kPackThreads) void linear_pack_kernel(LinearArgs a) {
  using AT = typename StreamTypes<WT>::AT;
  constexpr int xn = 16 / (int)sizeof(AT), wn = 16 / (int)sizeof(WT);
  const int64_t xu = a.pack_x ? a.kpack / xn : 0, wu = a.pack_w ? a.kpack / wn : 0;
  int64_t o = static_cast<int64_t>(blockIdx.x) * kPackThreads + threadIdx.x;
  if (o < a.M * xu) {
    const AT* row = static_cast<const AT*>(a.x) + o / xu * a.ldx;
    static_cast<u32x4*>(a.xpack)[o] = lin_unit<AT>(row, static_cast<int>(o % xu) * xn, a.K);
    return;
  }
  o -= a.M * xu;
  if (o < a.groups * static_cast<int64_t>(a.R) * wu) {
    const WT* row = static_cast<const WT*>(a.w) + o / wu * a.ldw;
    static_cast<u32x4*>(a.wpack)[o] = lin_unit<WT>(row, static_cast<int>(o % wu) * wn, a.K);
  }
}

template <typename WT>
static hipError_t launch_pack(LinearArgs* a, hipStream_t s) {
  constexpr int xn = 16 / (int)sizeof(typename StreamTypes<WT>::AT), wn = 16 / (int)sizeof(WT);
  const int64_t units = (a->pack_x ? a->M * (a->kpack / xn) : 0) +
                        (a->pack_w ? a->groups * static_cast<int64_t>(a->R) * (a->kpack / wn) : 0);
  linear_pack_kernel<WT><<<static_cast<unsigned>((units + kPackThreads - 1) / kPackThreads),
                           kPackThreads, 0, s>>>(*a);
  if (a->pack_x) a->x = a->xpack, a->ldx = a->kpack;
  if (a->pack_w) a->w = a->wpack, a->ldw = a->kpack;
  return hipGetLastError();
}

// ------------------------------------------------------------ launchers

template <typename WT, typename OT, int RT, bool kQuads, bool kGated, int XT = 1,
          int kThreads = kLinStreamThreads<WT>>
static hipError_t launch_stream(const LinearArgs& a, hipStream_t s) {
  const int ch = kGated ? 8 * RT : 16 * RT;
  const unsigned grid = static_cast<unsigned>((a.N + ch - 1) / ch);
  // (int8: aligned rows on the 16x16 MFMAs, others on the 4x4 ones)
  if (a.aligned) {
    if constexpr (!kLinInt8<WT> || !kQuads) {
      linear_stream_kernel<WT, OT, RT, kQuads, kGated, true, XT, kThreads><<<grid, kThreads, 0, s>>>(a);
      return hipGetLastError();
    }
  } else if constexpr (!kLinInt8<WT> || kQuads) {
    linear_stream_kernel<WT, OT, RT, kQuads, kGated, false, XT, kThreads><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  return hipErrorInvalidValue;
}

template <typename WT, typename OT, bool kGated>
static hipError_t launch_stream(const LinearArgs& a, hipStream_t s) {
  if (a.tile == kTileStream4) return launch_stream<WT, OT, 1, true, kGated>(a, s);
  if constexpr (kLinHalf<WT>)
    if (a.tile == kTileStream16Pair) return launch_stream<WT, OT, 2, false, kGated>(a, s);
  if constexpr (kLinInt8<WT>) {
    // (eight waves: one workgroup per compute unit; 16 x 4704 x 6576 four 14.0 us, eight 12.8)
    if (a.tile == kTileStream16Pair) return launch_stream<WT, OT, 2, false, kGated, 1, 512>(a, s);
    if (a.tile == kTileStream32) return launch_stream<WT, OT, 1, false, kGated, 2, 384>(a, s);
    if (a.tile == kTileStream32Pair) return launch_stream<WT, OT, 2, false, kGated, 2>(a, s);
    if (a.tile == kTileStream48) return launch_stream<WT, OT, 1, false, kGated, 3, 320>(a, s);
    if (a.tile == kTileStream64) return launch_stream<WT, OT, 1, false, kGated, 4>(a, s);
  }
  return launch_stream<WT, OT, 1, false, kGated>(a, s);
}

template <typename WT, typename OT>
static hipError_t launch_stream(const LinearArgs& a, hipStream_t s) {
  return a.gated ? launch_stream<WT, OT, true>(a, s) : launch_stream<WT, OT, false>(a, s);
}

template <typename WT, typename OT>
static hipError_t launch_pp(const LinearArgs& a, hipStream_t s) {
  const int ch = a.gated ? kPpPiece : 2 * kPpPiece;
  const int gx = static_cast<int>(linear_row_tiles(a, 256)), gy = (a.N + ch - 1) / ch;
  const dim3 grid((gx * gy + 7) / 8 * 8, 1, a.splits);
  if (a.gated)
    linear_pp_kernel<WT, OT, true><<<grid, kPpThreads, 0, s>>>(a, gx, gy);
  else
    linear_pp_kernel<WT, OT, false><<<grid, kPpThreads, 0, s>>>(a, gx, gy);
  return hipGetLastError();
}

template <typename WT, typename OT, class G, int S>
static hipError_t launch_tile(const LinearArgs& a, hipStream_t s) {
  const int ch = a.gated ? G::TN / 2 : G::TN;
  const int gx = static_cast<int>(linear_row_tiles(a, G::TM)), gy = (a.N + ch - 1) / ch;
  const dim3 grid((gx * gy + 7) / 8 * 8, 1, a.splits);
  if (a.gated)
    linear_tile_kernel<WT, OT, G, S, true><<<grid, G::kThreads, 0, s>>>(a, gx, gy);
  else
    linear_tile_kernel<WT, OT, G, S, false><<<grid, G::kThreads, 0, s>>>(a, gx, gy);
  return hipGetLastError();
}

template <typename WT, typename OT>
static hipError_t launch_reduce(const LinearArgs& a, hipStream_t s) {
  const int64_t n = a.M * ((a.N + 3) / 4);
  const unsigned grid = static_cast<unsigned>((n + kReduceThreads - 1) / kReduceThreads);
  if (a.gated)
    linear_reduce_kernel<WT, OT, true><<<grid, kReduceThreads, 0, s>>>(a);
  else
    linear_reduce_kernel<WT, OT, false><<<grid, kReduceThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename WT, typename OT, class G>
static hipError_t launch_staged(const LinearArgs& a, hipStream_t s) {
  const int tn = a.gated ? G::TN / 2 : G::TN;
  const dim3 grid(static_cast<unsigned>(((a.N + tn - 1) / tn) * linear_row_tiles(a, G::TM)), 1,
                  a.splits);
  if (a.gated)
    linear_staged_kernel<WT, OT, G, true><<<grid, G::kThreads, 0, s>>>(a);
  else
    linear_staged_kernel<WT, OT, G, false><<<grid, G::kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename WT, typename OT>
static hipError_t launch_type(LinearArgs a, hipStream_t s) {
  hipError_t e = hipErrorInvalidValue;
  if (a.pack_x || a.pack_w) {
    e = launch_pack<WT>(&a, s);
    if (e != hipSuccess) return e;
    if (a.pack_w) a.K = a.kpack;  // zeros in both operands past the row
  }
  switch (a.tile) {
    case kTileStream4:
    case kTileStream16:
    case kTileStream16Pair:
    case kTileStream32:
    case kTileStream32Pair:
    case kTileStream48:
    case kTileStream64: return launch_stream<WT, OT>(a, s);
    case kTile256:
      if constexpr (sizeof(WT) != 4) e = launch_pp<WT, OT>(a, s);
      break;
    // a ring of four stages alone on its compute unit, or less LDS and two
    // workgroups side by side
    case kTile128:
      if constexpr (sizeof(WT) == 2 || kLinInt8<WT>) e = launch_tile<WT, OT, LinGeom<WT, 2, 4, 4, 2>, 4>(a, s);
      break;
    case kTile128Pair: e = launch_tile<WT, OT, LinGeom<WT, 2, 4, 4, 2>, 2>(a, s); break;
    case kTile128x64:
      if constexpr (sizeof(WT) != 4)
        e = launch_tile<WT, OT, LinGeom<WT, 4, 2, 2, 2>, kLinHalf<WT> ? 4 : 6>(a, s);
      break;
    case kTile128x64Pair:
      if constexpr (!kLinHalf<WT>) e = launch_tile<WT, OT, LinGeom<WT, 4, 2, 2, 2>, 3>(a, s);
      break;
    case kTile64: e = launch_tile<WT, OT, LinGeom<WT, 2, 2, 2, 2>, 4>(a, s); break;
    case kTileStaged128: e = launch_staged<WT, OT, LinGeom<WT, 2, 4, 4, 2>>(a, s); break;
    case kTileStaged64: e = launch_staged<WT, OT, LinGeom<WT, 2, 2, 2, 2>>(a, s); break;
  }
  if (e == hipSuccess && a.part) e = launch_reduce<WT, OT>(a, s);
  return e;
}

}  // namespace moe
