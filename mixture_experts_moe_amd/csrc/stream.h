// Weight streaming for a few tokens (at most 16): the matrix-vector end of a
// product, bound by how fast the weight rows arrive.
//
// One load instruction takes four weight rows x 256 contiguous bytes: lane l
// holds 16 bytes of row l % 4 at K unit l / 4.  The 4x4 MFMAs (16 independent
// blocks of four lanes) take exactly that: block l / 4 multiplies its four
// rows with four tokens over its own K unit, and the 16 blocks' sums are
// added once at the end.  Against the 16x16 MFMA, whose operand layout makes
// a load cover 16 rows x 64 bytes (half of each row's 128-byte line), this
// reads whole lines with no LDS in between, for every weight type: 16 bytes
// are 8 bf16 (two 4x4x4 MFMAs), 16 e4m3fn (widened to bf16 exactly, four) or
// 4 fp32 (four 4x4x1).
#pragma once

#include "common.h"

namespace moe {

typedef short bf16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename WT> struct StreamTypes {
  using AT = bf16_t;
};
template <> struct StreamTypes<float> {
  using AT = float;
};

template <typename WT>
struct StreamGeom {
  using AT = typename StreamTypes<WT>::AT;
  static constexpr int kLaneK = 16 / (int)sizeof(WT);         // K per lane and load
  static constexpr int kChunk = 16 * kLaneK;                  // K per load instruction
  static constexpr int kTokLoads = kLaneK * (int)sizeof(AT) / 16;  // 16-byte loads per token
};

// D(4x4, f32) += A(4x4) . B(4x4) in each of 16 blocks: lane l supplies A row
// and B column l % 4 of block l / 4 and receives D column l % 4, rows 0..3.
__device__ __forceinline__ f32x4 mfma4x4x4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1,
                                           f32x4 c) {
  const uint2 a{a0, a1}, b{b0, b1};
  return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(bf16x4, a),
                                                __builtin_bit_cast(bf16x4, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma4x4x1(uint32_t a, uint32_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_4x4x1f32(__uint_as_float(a), __uint_as_float(b), c, 0, 0, 0);
}

// 16 bytes at any byte alignment.
struct __attribute__((packed, aligned(1))) StreamUnit {
  u32x4 v;
};

template <typename WT, int TQ>
using StreamTok = u32x4[TQ][StreamGeom<WT>::kTokLoads];

// acc[q][t] += rows of quad q . tokens of quad t over one chunk.
template <typename WT, int RQ, int TQ>
__device__ __forceinline__ void stream_mma(const u32x4 (&w)[RQ], const StreamTok<WT, TQ>& x,
                                           f32x4 (&acc)[RQ][TQ]) {
  if constexpr (sizeof(WT) == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < TQ; ++t)
#pragma unroll
        for (int q = 0; q < RQ; ++q)
          acc[q][t] = mfma4x4x4(w[q][2 * i], w[q][2 * i + 1], x[t][0][2 * i], x[t][0][2 * i + 1],
                                acc[q][t]);
  } else if constexpr (sizeof(WT) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < TQ; ++t)
#pragma unroll
        for (int q = 0; q < RQ; ++q) acc[q][t] = mfma4x4x1(w[q][i], x[t][0][i], acc[q][t]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // four codes of word i: K 4i .. 4i+3 of the lane's 16
#pragma unroll
      for (int q = 0; q < RQ; ++q) {
        const uint32_t lo = e4m3x2_to_bf16x2(w[q][i], false), hi = e4m3x2_to_bf16x2(w[q][i], true);
#pragma unroll
        for (int t = 0; t < TQ; ++t)
          acc[q][t] = mfma4x4x4(lo, hi, x[t][i / 2][2 * (i % 2)], x[t][i / 2][2 * (i % 2) + 1],
                                acc[q][t]);
      }
    }
  }
}

// The operand rows.  Weight quad q: wq[0] for the first half of the quads,
// wq[1] for the second (wave-uniform) + wo[q] (this lane's row and K unit,
// bytes); token quad t: xb (wave-uniform) + xo[t] (this
// lane's token row and K unit; columns past the last token repeat it and are
// dropped).
//
// kAligned: every row starts at a multiple of 16 bytes.  The weights are read
// once: nontemporal.
template <typename WT, int RQ, int TQ, bool kAligned>
struct Stream {
  using G = StreamGeom<WT>;
  using AT = typename G::AT;
  const uint8_t* wq[2];
  uint32_t wo[RQ];
  const uint8_t* xb;
  uint32_t xo[TQ];

  // quad q's rows: row_off(r) = bytes from its half's base to row r of the quad
  template <class F>
  __device__ __forceinline__ void place(int q, F row_off) {
    const int lane = threadIdx.x & 63;
    wo[q] = row_off(lane & 3) + 16 * (lane >> 2);
  }
  __device__ __forceinline__ const uint8_t* base(int q) const { return wq[RQ > 1 && q >= RQ / 2]; }

  static constexpr int kWStep = 256;                            // bytes per chunk
  static constexpr int kXStep = G::kChunk * (int)sizeof(AT);
  static constexpr int kNonTemporal = 2;

  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0x7fffffff, 0x00020000);
  }

  __device__ __forceinline__ void load(u32x4 (&w)[RQ], StreamTok<WT, TQ>& x, int chunk) const {
    if constexpr (kAligned) {
#pragma unroll
      for (int q = 0; q < RQ; ++q)
        w[q] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc(base(q)), wo[q], chunk * kWStep,
                                                         kNonTemporal));
#pragma unroll
      for (int t = 0; t < TQ; ++t)
#pragma unroll
        for (int i = 0; i < G::kTokLoads; ++i)
          x[t][i] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc(xb), xo[t] + 16 * i,
                                                           chunk * kXStep, 0));
    } else {
#pragma unroll
      for (int q = 0; q < RQ; ++q)
        w[q] = reinterpret_cast<const StreamUnit*>(base(q) + static_cast<size_t>(chunk) * kWStep +
                                                   wo[q])
                   ->v;
#pragma unroll
      for (int t = 0; t < TQ; ++t)
#pragma unroll
        for (int i = 0; i < G::kTokLoads; ++i)
          x[t][i] = reinterpret_cast<const StreamUnit*>(
                        xb + static_cast<size_t>(chunk) * kXStep + xo[t] + 16 * i)
                        ->v;
    }
  }

  // N chunks from i on: all their loads, then their MFMAs.
  template <int N>
  __device__ __forceinline__ void batch(int c0, int step, f32x4 (&acc)[RQ][TQ]) const {
    u32x4 w[N][RQ];
    StreamTok<WT, TQ> x[N];
#pragma unroll
    for (int p = 0; p < N; ++p) load(w[p], x[p], c0 + p * step);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < N; ++p) stream_mma<WT, RQ, TQ>(w[p], x[p], acc);
    __builtin_amdgcn_sched_barrier(0);
  }

  // acc += over chunks c0, c0 + step, ... (n of them), P at a time.  A wave
  // waits for a whole batch; the other waves of its SIMD keep the loads
  // coming (a ring that refills each chunk's registers as soon as they are
  // used needs copies of the whole ring at its ends, which spill).
  template <int P>
  __device__ __forceinline__ void run(int c0, int n, int step, f32x4 (&acc)[RQ][TQ]) const {
    for (; n >= P; n -= P, c0 += P * step) batch<P>(c0, step, acc);
    if constexpr (P > 4) {
      if (n >= 4) {
        batch<4>(c0, step, acc);
        n -= 4, c0 += 4 * step;
      }
    }
    if constexpr (P > 2) {
      if (n >= 2) {
        batch<2>(c0, step, acc);
        n -= 2, c0 += 2 * step;
      }
    }
    if (n >= 1) batch<1>(c0, step, acc);
  }

  // The last, partial chunk: `left` (< kChunk) elements of K.
  __device__ __forceinline__ void tail(int chunk, int left, f32x4 (&acc)[RQ][TQ]) const {
    const int k = (threadIdx.x & 63) / 4 * G::kLaneK;  // this lane's K unit
    u32x4 w[RQ];
    StreamTok<WT, TQ> x;
#pragma unroll
    for (int q = 0; q < RQ; ++q)
      w[q] = part<WT>(base(q) + static_cast<size_t>(chunk) * kWStep + wo[q], left - k);
#pragma unroll
    for (int t = 0; t < TQ; ++t)
#pragma unroll
      for (int i = 0; i < G::kTokLoads; ++i)
        x[t][i] = part<AT>(xb + static_cast<size_t>(chunk) * kXStep + xo[t] + 16 * i,
                           left - k - i * (16 / (int)sizeof(AT)));
    stream_mma<WT, RQ, TQ>(w, x, acc);
  }

  // 16 bytes of which the first n elements exist; zeros for the others.  With
  // aligned rows whose length is a multiple of 16 bytes n is never in
  // between.
  template <typename T>
  static __device__ __forceinline__ u32x4 part(const uint8_t* p, int n) {
    constexpr int per = 16 / (int)sizeof(T);
    union {
      u32x4 v;
      T e[per];
    } u;
    u.v = u32x4{0, 0, 0, 0};
    if (n >= per) {
      u.v = reinterpret_cast<const StreamUnit*>(p)->v;
    } else if (!kAligned) {
#pragma unroll
      for (int i = 0; i < per; ++i)
        if (i < n) u.e[i] = reinterpret_cast<const T*>(p)[i];
    }
    return u.v;
  }
};

// The same for 5 to 16 tokens on the 16x16 MFMAs: one token fragment serves
// every tile of weight rows, where the 4x4 MFMAs need one per four tokens.
// Their operand (lane l: row l % 16, K unit l / 16) would make a load cover 16
// rows x 64 bytes, half lines, so aligned rows go through LDS: direct-to-LDS
// loads of four rows x 256 bytes into the wave's own two regions (in arrays of
// their own: reads of one then wait for no load into the other), unit u of row
// r in slot u ^ (r & 15) (the 16 rows read for one unit fall in 16 bank
// groups).  acc[t]: D column (token) l % 16, rows 4 (l / 16) .. +3 of tile t,
// already summed over K.
// kHalf: the tiles have eight rows (the other eight sums mean nothing).
template <typename WT, int RT, bool kAligned, bool kHalf = false>
struct Stream16 {
  using G = StreamGeom<WT>;
  using AT = typename G::AT;
  const uint8_t* wq[RT][2];  // wave-uniform: rows 0 and 8 of tile t
  // this lane's byte offsets from those: aligned, of rows 4i + l / 16 for
  // i = 0..3 with the unit that its LDS slot takes; else of row l % 16 at
  // unit l / 16
  uint32_t wo[RT][kAligned ? 4 : 1];
  const uint8_t* xb;      // wave-uniform
  uint32_t xo;            // this lane's token row and K unit, bytes
  uint8_t* lds[2];        // the wave's two regions of kLds bytes (aligned)

  static constexpr int kLds = RT * 4096;              // one chunk
  static constexpr int kWStep = 256;
  static constexpr int kXStep = G::kChunk * (int)sizeof(AT);
  static constexpr int kUnits = 4;                    // MFMA operand units per row and chunk
  static constexpr int kXUnit = kXStep / kUnits;      // token bytes a unit spans

  using Toks = u32x4[kUnits][G::kTokLoads];

  // The offsets of tile t: row_off(r) = bytes to row r from its half's base
  // (rows 0 and 8).
  template <class F>
  __device__ __forceinline__ void place(int t, F row_off) {
    const int lane = threadIdx.x & 63;
    if constexpr (kAligned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + (lane >> 4);
        wo[t][i] = kHalf && i >= 2 ? 0 : row_off(r) + 16 * ((lane & 15) ^ r);
      }
    } else {
      wo[t][0] = row_off(lane & (kHalf ? 7 : 15)) + 16 * (lane >> 4);
    }
  }

  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0x7fffffff, 0x00020000);
  }
  // the base of this lane's row (l % 16) of tile t
  __device__ __forceinline__ const uint8_t* lane_row(int t) const {
    return !kHalf && (threadIdx.x & 8) ? wq[t][1] : wq[t][0];
  }

  __device__ __forceinline__ void load_x(Toks& x, int chunk) const {
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < G::kTokLoads; ++i)
        if constexpr (kAligned)
          x[u][i] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc(xb), xo + kXUnit * u + 16 * i,
                                                           chunk * kXStep, 0));
        else
          x[u][i] = reinterpret_cast<const StreamUnit*>(xb + static_cast<size_t>(chunk) * kXStep +
                                                        xo + kXUnit * u + 16 * i)
                        ->v;
  }

  static __device__ __forceinline__ f32x4 mma(u32x4 w, const u32x4 (&x)[G::kTokLoads], f32x4 acc) {
    if constexpr (sizeof(WT) == 2) {
      return mfma16x16x32(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x[0]), acc);
    } else if constexpr (sizeof(WT) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc = mfma16x16x4f32(__uint_as_float(w[i]), __uint_as_float(x[0][i]), acc);
      return acc;
    } else {
      acc = mfma16x16x32(as_frag(e4m3x8_to_frag_bits(w[0], w[1])),
                         __builtin_bit_cast(bf16x8, x[0]), acc);
      return mfma16x16x32(as_frag(e4m3x8_to_frag_bits(w[2], w[3])),
                          __builtin_bit_cast(bf16x8, x[G::kTokLoads - 1]), acc);
    }
  }

  // Chunk c into region `slot` and its tokens into registers; kLoadCount
  // vector-memory instructions.
  static constexpr int kLoadCount = RT * (kHalf ? 2 : 4) + kUnits * G::kTokLoads;
  __device__ __forceinline__ void fetch(int slot, Toks& x, int c) const {
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int i = 0; i < (kHalf ? 2 : 4); ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc(wq[t][i / 2]),
            (__attribute__((address_space(3))) void*)(lds[slot] + 4096 * t + 1024 * i), 16, wo[t][i],
            c * kWStep, 0, 2);
    load_x(x, c);
    __builtin_amdgcn_sched_barrier(0);
  }
  // kLater: loads issued after the chunk's
  template <int kLater>
  __device__ __forceinline__ void use(int slot, const Toks& x, f32x4 (&acc)[RT]) const {
    // the chunk's loads have landed; the compiler does not see that the LDS
    // reads below depend on them
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLater) : "memory");
    const int r16 = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
        acc[t] = mma(*reinterpret_cast<const u32x4*>(lds[slot] + 4096 * t + 256 * r16 +
                                                     16 * ((4 * u + g) ^ r16)),
                     x[u], acc[t]);
    // every read has returned before later loads overwrite the region
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // N chunks straight to registers: all their loads, then their MFMAs.
  template <int N>
  __device__ __forceinline__ void direct(int c0, int step, f32x4 (&acc)[RT]) const {
    Toks x[N];
    u32x4 w[N][kUnits][RT];
#pragma unroll
    for (int p = 0; p < N; ++p) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          w[p][u][t] = reinterpret_cast<const StreamUnit*>(
                           lane_row(t) + static_cast<size_t>(c0 + p * step) * kWStep + wo[t][0] +
                           64 * u)
                           ->v;
      load_x(x[p], c0 + p * step);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int p = 0; p < N; ++p)
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = mma(w[p][u][t], x[p][u], acc[t]);
    __builtin_amdgcn_sched_barrier(0);
  }

  // acc += over chunks c0, c0 + step, ... (n of them), the next one loading
  // while one is multiplied.
  __device__ __forceinline__ void run(int c0, int n, int step, f32x4 (&acc)[RT]) const {
    if constexpr (kAligned) {
      static_assert(kLoadCount <= 63, "six-bit count");
      if (n <= 0) return;
      Toks x0, x1;
      fetch(0, x0, c0);
      for (;; n -= 2, c0 += 2 * step) {
        if (n == 1) {
          use<0>(0, x0, acc);
          return;
        }
        fetch(1, x1, c0 + step);
        use<kLoadCount>(0, x0, acc);
        if (n == 2) {
          use<0>(1, x1, acc);
          return;
        }
        fetch(0, x0, c0 + 2 * step);
        use<kLoadCount>(1, x1, acc);
      }
    } else {
      for (; n >= 2; n -= 2, c0 += 2 * step) direct<2>(c0, step, acc);
      if (n >= 1) direct<1>(c0, step, acc);
    }
  }

  // The last, partial chunk: `left` (< kChunk) elements of K; row_off as for
  // place().
  template <class F>
  __device__ __forceinline__ void tail(int c, int left, F row_off, f32x4 (&acc)[RT]) const {
    using S = Stream<WT, 1, 1, kAligned>;
    constexpr int per = 16 / (int)sizeof(AT);
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int k = (4 * u + (lane >> 4)) * G::kLaneK;
      u32x4 x[G::kTokLoads];
#pragma unroll
      for (int i = 0; i < G::kTokLoads; ++i)
        x[i] = S::template part<AT>(
            xb + static_cast<size_t>(c) * kXStep + xo + kXUnit * u + 16 * i, left - k - i * per);
#pragma unroll
      for (int t = 0; t < RT; ++t)
        acc[t] = mma(S::template part<WT>(lane_row(t) + static_cast<size_t>(c) * kWStep +
                                              row_off(t, lane & (kHalf ? 7 : 15)) +
                                              16 * (lane >> 4) + 64 * u,
                                          left - k),
                     x, acc[t]);
    }
  }
};

// The largest value of a wave, in every lane.
__device__ __forceinline__ uint32_t stream_wave_max(uint32_t v) {
#define STREAM_MAX(ctrl) \
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), ctrl, 0xf, 0xf, false)))
  STREAM_MAX(0x121);  // row_ror:1, 2, 4, 8
  STREAM_MAX(0x122);
  STREAM_MAX(0x124);
  STREAM_MAX(0x128);
#undef STREAM_MAX
  auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(static_cast<uint32_t>(a[0]), static_cast<uint32_t>(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(static_cast<uint32_t>(b[0]), static_cast<uint32_t>(b[1]));
}

// Sum over the 16 blocks of a wave, four rows of 16 lanes first: afterwards
// lane l holds its row of 16 lanes' sum for token l % 4.
__device__ __forceinline__ float stream_row_sum(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x124, 0xf,
                                                          0xf, false));  // row_ror:4
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x128, 0xf,
                                                          0xf, false));  // row_ror:8
  return v;
}
__device__ __forceinline__ float stream_wave_sum(float v) {
  v = stream_row_sum(v);
  // rows of 16 lanes 0 <-> 1, 2 <-> 3, then the halves: each swap leaves both
  // sides' values in the pair of results
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

}  // namespace moe
