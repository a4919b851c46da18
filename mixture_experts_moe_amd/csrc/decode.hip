// The whole MoE layer for at most 16 tokens in two launches.
//
//   1. decode_route_kernel: logits = x . W_gate^T (fp32), a workgroup per
//      expert and four tokens; it also clears the words that the next
//      launch's workgroups meet through.
//   2. decode_layer_kernel: every workgroup selects the experts from the
//      logits by itself (a few hundred values, cheaper than another launch),
//      computes its share of h = SiLU(W1 x) * (W3 x), publishes it, and then
//      its share of the output channels: out = residual + sum_j gate_j W2 h_j,
//      all experts of a channel in one workgroup, so nothing is added up
//      through memory (but where there are fewer than two channel quads per
//      workgroup several share one, see w2_share).
//
// With so few tokens the layer is a read of the selected experts' weights:
// each is read exactly once (stream.h), whatever the number of its tokens.
//
// Between the two halves every workgroup needs every other's h.  Each
// workgroup has a flag of its own, written once its h rows are out at device
// scope; workgroup 0 reads them all and tells the others, a word for 32 of
// them.  No workgroup depends on another one being resident: one that finds a
// share missing for longer than the limit computes that share itself (the
// same bits, to the same place), so every wait ends whatever else the GPU runs.

#include "kernels.h"
#include "stream.h"

namespace moe {

// Waves of a workgroup, one workgroup per compute unit: eight, whose 256
// registers hold eight chunks in flight each (two such workgroups per unit
// with four chunks each took 89 us for 4 tokens of d = 2048, E = 64, top-8,
// I = 1024 in bf16 against 78); sixteen with e4m3fn weights, which the waves
// widen as they go, and few tokens.
template <typename WT, bool kMany>
constexpr int dec_waves() { return sizeof(WT) == 1 && !kMany ? 16 : 8; }
constexpr int kDecMaxRows = kDecodeMaxTokens * kMaxTopK;  // slots
constexpr int kDecMaxWgs = 256;
constexpr int kDecGroup = 32;  // workgroups that share a go word
constexpr int kDecGroups = kDecMaxWgs / kDecGroup;
// Words that workgroups meet through, each in a cache line of its own (hundreds
// of workgroups polling, adding to or storing to one line take tens of
// microseconds): a flag per workgroup, a go word per group, a counter per row
// quad whose sum is split over workgroups.
constexpr int kDecLine = 64;
constexpr int kDecFlag = 0, kDecGo = kDecMaxWgs, kDecCount = kDecGo + kDecGroups;
constexpr int kDecLines = kDecCount + kDecMaxWgs / 2;
constexpr int kDecMeetBytes = kDecLines * kDecLine;
// and the split sums: [workgroup][token][4 rows] fp32
constexpr int kDecSumBytes = kDecMaxWgs * kDecodeMaxTokens * 4 * 4;

// A value that every lane holds alike, as a scalar: addresses built from it
// stay in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int32_t* dec_word(const DecodeArgs& a, int i) {
  return reinterpret_cast<int32_t*>(a.meet + i * kDecLine);
}
__device__ __forceinline__ int dec_read(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void dec_write(int32_t* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ------------------------------------------------------------ router logits

constexpr int kRouteThreads = 512;

// One expert and up to kRouteTokens tokens per workgroup; a thread takes every
// 512th unit of four K.
constexpr int kRouteTokens = 4;
template <typename AT>
__global__ __launch_bounds__(kRouteThreads) void decode_route_kernel(
    const AT* __restrict__ x, const float* __restrict__ w_gate, float* __restrict__ logits,
    uint8_t* __restrict__ meet, int T, int E, int d) {
  __shared__ float part[kRouteThreads / 64][kRouteTokens];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x, t0 = blockIdx.y * kRouteTokens;
  const int n = min(T - t0, kRouteTokens);
  // this launch clears the meeting words of the next, a slice per workgroup
  for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * kRouteThreads + tid; i < kDecMeetBytes / 16;
       i += gridDim.x * gridDim.y * kRouteThreads)
    reinterpret_cast<uint4*>(meet)[i] = uint4{0, 0, 0, 0};
  x += static_cast<size_t>(t0) * d;
  w_gate += static_cast<size_t>(e) * d;
  float acc[kRouteTokens] = {};
#pragma unroll 2
  for (int u = tid; u < d / 4; u += kRouteThreads) {
    const float4 w = *reinterpret_cast<const float4*>(w_gate + 4 * u);
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
      // tokens past the last repeat it
      const AT* row = x + static_cast<size_t>(min(t, n - 1)) * d + 4 * u;
      float v[4];
      if constexpr (sizeof(AT) == 4) {
        const float4 q = *reinterpret_cast<const float4*>(row);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(row);
        v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
        v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
      }
      acc[t] = fmaf(w.x, v[0], acc[t]);
      acc[t] = fmaf(w.y, v[1], acc[t]);
      acc[t] = fmaf(w.z, v[2], acc[t]);
      acc[t] = fmaf(w.w, v[3], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kRouteTokens; ++t) {
    const float v = wave_sum(acc[t]);
    if (lane == 0) part[wave][t] = v;
  }
  __syncthreads();
  if (tid < n) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteThreads / 64; ++w) v += part[w][tid];
    logits[static_cast<size_t>(t0 + tid) * E + e] = v;
  }
}

// ------------------------------------------------------------ selection

// What the workgroup knows of the routing: the selected experts in index
// order, each with its tokens in order.  A row is one (expert, token) pair;
// expert i's rows are base[i] .. base[i+1]-1, and h has one row each.
struct DecSel {
  uint16_t expert[kMaxExperts];
  uint16_t base[kMaxExperts + 1];
  uint8_t token[kDecMaxRows];
  float gate[kDecMaxRows];
  int n;  // experts selected
};

// Used while selecting only.
struct DecScratch {
  float slot_gate[kDecMaxRows];
  uint32_t mask[kMaxExperts];  // bit t: token t selected this expert
  uint16_t slot_e[kDecMaxRows];
  uint16_t first[kMaxExperts];  // an expert's first row
};

// Order-preserving key: greater logit, greater key; NaN as -inf; both zeros
// alike; 0 below every logit's key.
__device__ __forceinline__ uint32_t dec_key(float v) {
  if (v != v) v = -INFINITY;
  if (v == 0.f) v = 0.f;
  const uint32_t b = __float_as_uint(v);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float dec_logit(uint32_t key) {
  return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key);
}

// One wave selects the top k of a token's E logits: lane l holds experts
// l*per .. l*per+per-1, so the first lane holding the maximum has the lowest
// index; gates = softmax over the selection.
template <int kPer>  // E <= 64 * kPer
__device__ __forceinline__ void dec_topk(const float* row, int E, int k, uint16_t* slot_e,
                                         float* slot_gate) {
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < per) {  // uniform
      const int e = lane * per + i;
      const float v = row[min(e, E - 1)];
      key[i] = e < E ? dec_key(v) : 0u;
    } else {
      key[i] = 0u;
    }
  uint32_t my_key = 0;
  int my_e = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per && key[i] > best) {
        best = key[i];
        bi = i;
      }
    const uint32_t m = uniform(static_cast<int>(stream_wave_max(best)));
    const int src = __ffsll(static_cast<unsigned long long>(__ballot(best == m))) - 1;
    const int e = __builtin_amdgcn_readlane(lane * per + bi, src);
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i == bi) key[i] = 0;
    }
    if (lane == j) {
      my_key = m;
      my_e = e;
    }
  }
  const float v = dec_logit(my_key);
  const float l0 = __shfl(v, 0, 64);
  const float p = lane < k ? expf(v - l0) : 0.f;
  const float s = wave_sum(p);
  if (lane < k) {
    slot_e[lane] = static_cast<uint16_t>(my_e);
    slot_gate[lane] = p / s;
  }
}

template <int kWaves>
__device__ __forceinline__ void dec_select(const float* logits, int T, int E, int k, DecSel& s,
                                           DecScratch& w) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kThreads = 64 * kWaves;
  for (int e = tid; e < E; e += kThreads) w.mask[e] = 0;
  for (int t = wave; t < T; t += kWaves) {
    const float* row = logits + static_cast<size_t>(t) * E;
    if (E <= 256)
      dec_topk<4>(row, E, k, w.slot_e + t * k, w.slot_gate + t * k);
    else
      dec_topk<kMaxExperts / 64>(row, E, k, w.slot_e + t * k, w.slot_gate + t * k);
  }
  __syncthreads();
  for (int f = tid; f < T * k; f += kThreads) atomicOr(&w.mask[w.slot_e[f]], 1u << (f / k));
  __syncthreads();
  if (wave == 0) {  // compact the used experts; rows in expert order
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t m = e < E ? w.mask[e] : 0u;
      const uint64_t used = __ballot(m != 0);
      const int before = __popcll(used & ((1ull << lane) - 1));
      const int cnt = __popc(m);
      // rows before this lane's expert (cnt <= 16: five bits)
      const uint64_t below = (1ull << lane) - 1;
      int first = rows, all = 0;
#pragma unroll
      for (int bit = 0; bit < 5; ++bit) {
        const uint64_t set = __ballot((cnt >> bit) & 1);
        first += __popcll(set & below) << bit;
        all += __popcll(set) << bit;
      }
      if (m) {
        s.expert[n + before] = static_cast<uint16_t>(e);
        s.base[n + before] = static_cast<uint16_t>(first);
        w.first[e] = static_cast<uint16_t>(first);
      }
      n += __popcll(used);
      rows += all;
    }
    if (lane == 0) {
      s.base[n] = static_cast<uint16_t>(rows);
      s.n = n;
    }
  }
  __syncthreads();
  for (int f = tid; f < T * k; f += kThreads) {
    const int e = w.slot_e[f], t = f / k;
    const int r = w.first[e] + __popc(w.mask[e] & ((1u << t) - 1));
    s.token[r] = static_cast<uint8_t>(t);
    s.gate[r] = w.slot_gate[f];
  }
  __syncthreads();
}

// ------------------------------------------------------------ the layer

// kMany: more than four tokens in the call; experts with up to four of them
// take the 4x4 MFMAs, the others the 16x16 (stream.h).
template <typename WT, bool kMany>
struct DecLayer {
  using G = StreamGeom<WT>;
  using AT = typename G::AT;
  template <bool kHalf>
  using S16 = Stream16<WT, 1, true, kHalf>;
  static constexpr int kTok = kMany ? 16 : 4;  // token columns of an expert
  static constexpr int kWaves = dec_waves<WT, kMany>(), kThreads = 64 * kWaves;
  // chunks of 16 rows in flight per wave
  static constexpr int kBatch = sizeof(WT) > 1 ? 8 : kMany ? 4 : 2;
  const DecodeArgs& a;
  DecSel& sel;
  // Work inside the workgroup goes in units that the waves take from a counter
  // in LDS (the memory serves older waves first: with equal shares some
  // finished in two thirds of the others' time).  A unit's sums have a slot of
  // their own, so they are the same whichever wave takes it.
  static constexpr int kSlots = kMany ? 32 : 8 * kWaves;
  float (*red)[kTok][16];  // [kSlots]: a unit's sums of 16 rows per token
  int* ticket;
  uint8_t* lds0;           // this wave's weights (kMany)
  uint8_t* lds1;

  int lane, wave;

  __device__ __forceinline__ int take() const {
    int u = 0;
    if (lane == 0) u = atomicAdd(ticket, 1);
    return uniform(u);
  }

  // The lane's token row (of n rows from `base`; columns past the last repeat
  // it, never stored): wave-uniform base and byte offset.
  __device__ __forceinline__ void token(const AT* m, int ld, int base, int n, int col, bool h_rows,
                                        const uint8_t** xb, uint32_t* xo) const {
    *xb = reinterpret_cast<const uint8_t*>(m + (h_rows ? static_cast<size_t>(base) * ld : 0));
    const int j = min(col, n - 1);
    *xo = static_cast<uint32_t>(h_rows ? j : sel.token[base + j]) * ld * sizeof(AT);
  }

  // ---- W13: 8 channels (gate rows, the matching up rows) from c0 of selected
  // expert i, K split `sub` of `S`; sums to red[slot]: 8 gate, 8 up.
  __device__ __forceinline__ void w13_group(int i, int c0, int sub, int S, int slot) const {
    const int e = uniform(sel.expert[i]), base = uniform(sel.base[i]);
    const int n = uniform(sel.base[i + 1]) - base;
    const size_t ldb = static_cast<size_t>(a.d) * sizeof(WT);
    const uint8_t* gate = static_cast<const uint8_t*>(a.w13) +
                          (static_cast<size_t>(e) * 2 * a.I + c0) * ldb;
    const uint8_t* up = gate + a.I * ldb;
    const int full = a.d / G::kChunk, left = a.d % G::kChunk;
    const int mine = full > sub ? (full - sub + S - 1) / S : 0;
    const bool last = left && full % S == sub;
    if (kMany && n > 4) {
      S16<false> st;
      st.wq[0][0] = gate;
      st.wq[0][1] = up;
      auto row_off = [&](int, int r) { return static_cast<uint32_t>((r & 7) * ldb); };
      st.place(0, [&](int r) { return row_off(0, r); });
      st.lds[0] = lds0;
      st.lds[1] = lds1;
      token(static_cast<const AT*>(a.x), a.d, base, n, lane & 15, false, &st.xb, &st.xo);
      st.xo += (lane >> 4) * (G::kLaneK * sizeof(AT));
      f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
      st.run(sub, mine, S, acc);
      if (last) st.tail(full, left, row_off, acc);
      *reinterpret_cast<f32x4*>(&red[slot][(lane & 15) % kTok][4 * (lane >> 4)]) = acc[0];
      return;
    }
    Stream<WT, 4, 1, true> st;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st.place(q, [&](int r) { return static_cast<uint32_t>((4 * (q & 1) + r) * ldb); });
    st.wq[0] = gate;
    st.wq[1] = up;
    token(static_cast<const AT*>(a.x), a.d, base, n, lane & 3, false, &st.xb, &st.xo[0]);
    st.xo[0] += (lane >> 2) * (G::kLaneK * sizeof(AT));
    f32x4 acc[4][1];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    st.template run<kBatch>(sub, mine, S, acc);
    if (last) st.tail(full, left, acc);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[q][0][v] = stream_wave_sum(acc[q][0][v]);
      if (lane < 4) *reinterpret_cast<f32x4*>(&red[slot][lane][4 * q]) = acc[q][0];
    }
  }

  // K ranges per group so that the workgroup's waves finish together: the
  // least time in chunks over S = 1, 2, 4, 8, counting about two chunks for
  // a pass's start and end.
  __device__ __forceinline__ int pick_split(int groups) const {
    const int chunks = (a.d + G::kChunk - 1) / G::kChunk;
    int best = 1 << 30, s = 1;
    for (int S = 1; S <= 8; S *= 2) {
      const int passes = (groups * S + kWaves - 1) / kWaves;
      const int cost = passes * ((chunks + S - 1) / S + 2);
      if (cost < best) {
        best = cost;
        s = S;
      }
    }
    return s;
  }

  // Share b of h.
  __device__ void w13_share(int b) const {
    const int per = a.I / 8;  // groups per expert
    const int64_t total = static_cast<int64_t>(uniform(sel.n)) * per;
    const int g0 = static_cast<int>(total * b / a.wgs);
    const int g1 = static_cast<int>(total * (b + 1) / a.wgs);
    const int S = pick_split(g1 - g0);
    const int rounds = ((g1 - g0) * S + kSlots - 1) / kSlots;
    const int step = rounds ? (g1 - g0 + rounds - 1) / rounds : 1;  // groups of a round
    for (int g = g0; g < g1; g += step) {
      const int n = min(step, g1 - g);
      for (int u = take(); u < n * S; u = take())
        w13_group((g + u / S) / per, 8 * ((g + u / S) % per), u % S, S, u);
      __syncthreads();
      if (threadIdx.x == 0) *ticket = 0;
      // channel pair cp of token column j of the gs-th of these groups, whose
      // sums are in the S slots from gs * S on
      for (int o = threadIdx.x; o < n * kTok * 4; o += kThreads) {
        const int cp = o & 3, j = (o >> 2) % kTok, gs = (o >> 2) / kTok;
        const int i = (g + gs) / per, c = 8 * ((g + gs) % per) + 2 * cp;
        const int base = sel.base[i];
        if (j >= sel.base[i + 1] - base) continue;
        float hv[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          float zg = 0.f, zu = 0.f;
          for (int s = 0; s < S; ++s) {
            zg += red[gs * S + s][j][2 * cp + v];
            zu += red[gs * S + s][j][8 + 2 * cp + v];
          }
          if (sizeof(WT) == 1) {
            const size_t e = sel.expert[i];
            const bool ch = a.scale_mode == kScaleChannel;
            zg *= a.s13[ch ? e * 2 * a.I + c + v : e];
            zu *= a.s13[ch ? e * 2 * a.I + a.I + c + v : e];
          }
          hv[v] = silu(zg) * zu;
        }
        // h is rounded to the activation type (the MFMA operand of W2), as
        // the layer's other paths do; written at device scope for readers on
        // other XCDs
        AT* h = static_cast<AT*>(a.h) + static_cast<size_t>(base + j) * a.I + c;
        if constexpr (sizeof(AT) == 2) {
          const uint32_t v = f32_to_bf16(hv[0]) | (static_cast<uint32_t>(f32_to_bf16(hv[1])) << 16);
          __hip_atomic_store(reinterpret_cast<uint32_t*>(h), v, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
        } else {
          __hip_atomic_store(h, hv[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(h + 1, hv[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
      __syncthreads();  // the sums have been read
    }
  }

  // ---- W2: output rows r0 .. r0+4*RQ-1.

  // four rows' sums v of one expert for token column j, into the unit's out sums
  __device__ __forceinline__ void add(int slot, int e, int base, int j, int r0, int r,
                                      f32x4 v) const {
    const float gate = sel.gate[base + j];
    float* o = &red[slot][sel.token[base + j]][r];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(WT) == 1)
        v[i] *= a.s2[a.scale_mode == kScaleChannel ? static_cast<size_t>(e) * a.d + r0 + r + i : e];
      o[i] += gate * v[i];
    }
  }

  // chunks [c0, c1) of selected expert i (the last may be partial); adds the
  // expert's gated, scaled sums to the unit's out sums
  template <int RQ>
  __device__ __forceinline__ void w2_part(int slot, int i, int r0, int c0, int c1) const {
    const int e = uniform(sel.expert[i]), base = uniform(sel.base[i]);
    const int n = uniform(sel.base[i + 1]) - base;
    const size_t ldb = static_cast<size_t>(a.I) * sizeof(WT);
    const uint8_t* w = static_cast<const uint8_t*>(a.w2) + (static_cast<size_t>(e) * a.d + r0) * ldb;
    const int full = a.I / G::kChunk, left = a.I % G::kChunk;
    if (kMany && n > 4) {
      S16<(RQ <= 2)> st;
      st.wq[0][0] = w;
      st.wq[0][1] = w + 8 * ldb;
      // rows past the last repeat it
      auto row_off = [&](int, int r) {
        return static_cast<uint32_t>((min(r, 4 * RQ - 1) - (r & 8)) * ldb);
      };
      st.place(0, [&](int r) { return row_off(0, r); });
      st.lds[0] = lds0;
      st.lds[1] = lds1;
      token(static_cast<const AT*>(a.h), a.I, base, n, lane & 15, true, &st.xb, &st.xo);
      st.xo += (lane >> 4) * (G::kLaneK * sizeof(AT));
      f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
      st.run(c0, min(c1, full) - c0, 1, acc);
      if (c1 > full) st.tail(full, left, row_off, acc);
      const int j = lane & 15, r = 4 * (lane >> 4);
      if (j < n && r < 4 * RQ) add(slot, e, base, j, r0, r, acc[0]);
      return;
    }
    Stream<WT, RQ, 1, true> st;
#pragma unroll
    for (int q = 0; q < RQ; ++q)
      st.place(q, [&](int r) { return static_cast<uint32_t>((4 * q + r) * ldb); });
    st.wq[0] = st.wq[1] = w;
    token(static_cast<const AT*>(a.h), a.I, base, n, lane & 3, true, &st.xb, &st.xo[0]);
    st.xo[0] += (lane >> 2) * (G::kLaneK * sizeof(AT));
    f32x4 acc[RQ][1];
#pragma unroll
    for (int q = 0; q < RQ; ++q) acc[q][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    st.template run<kBatch>(c0, min(c1, full) - c0, 1, acc);
    if (c1 > full) st.tail(full, left, acc);
#pragma unroll
    for (int q = 0; q < RQ; ++q) {
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[q][0][v] = stream_wave_sum(acc[q][0][v]);
      if (lane < n) add(slot, e, base, lane, r0, 4 * q, acc[q][0]);
    }
  }

  // Rows r0 .. r0+4*RQ-1, summed over part `part` of `parts` of the (expert,
  // chunk) list.  Where there are several parts their sums meet in memory and
  // the workgroup that comes last adds them, in order.
  template <int RQ>
  __device__ __forceinline__ void w2_rows(int r0, int part, int parts) const {
    const int tid = threadIdx.x;
    // the (expert, chunk) list in equal units, as many for each wave, of at
    // least 16 chunks where there are enough
    const int C = (a.I + G::kChunk - 1) / G::kChunk;
    const int all = uniform(sel.n) * C;
    const int first = static_cast<int>(static_cast<int64_t>(all) * part / parts);
    const int items = static_cast<int>(static_cast<int64_t>(all) * (part + 1) / parts) - first;
    const int units = kWaves * min(max(items / (16 * kWaves), 1), kMany ? kSlots / kWaves : 4);
    for (int o = tid; o < units * kTok * 16; o += kThreads) (&red[0][0][0])[o] = 0.f;
    if (tid == 0) *ticket = 0;
    __syncthreads();
    for (int u = take(); u < units; u = take()) {
      const int i1 = first + static_cast<int>(static_cast<int64_t>(items) * (u + 1) / units);
      for (int it = first + static_cast<int>(static_cast<int64_t>(items) * u / units); it < i1;) {
        const int i = it / C, c0 = it % C;
        const int c1 = min(C, c0 + i1 - it);
        w2_part<RQ>(u, i, r0, c0, c1);
        it += c1 - c0;
      }
    }
    __syncthreads();
    for (int o = tid; o < a.T * 4 * RQ; o += kThreads) {
      const int t = o / (4 * RQ), r = o % (4 * RQ);
      float v = 0.f;
      for (int u = 0; u < units; ++u) v += red[u][t][r];
      if (parts == 1)
        finish(v, t, r0 + r);
      else
        __hip_atomic_store(sums(r0 / 4, part) + o, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (parts > 1) {  // RQ == 1
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0)
        *ticket = __hip_atomic_fetch_add(dec_word(a, kDecCount + r0 / 4), 1, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      if (*ticket == parts - 1)
        for (int o = tid; o < a.T * 4; o += kThreads) {
          float v = 0.f;
          for (int p = 0; p < parts; ++p)
            v += __hip_atomic_load(sums(r0 / 4, p) + o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          finish(v, o / 4, r0 + o % 4);
        }
    }
    __syncthreads();  // the sums have been read
  }

  __device__ __forceinline__ float* sums(int quad, int part) const {
    const int w = part * (a.d / 4) + quad;  // the workgroup that holds them
    return reinterpret_cast<float*>(a.meet + kDecMeetBytes) + w * (kDecodeMaxTokens * 4);
  }

  __device__ __forceinline__ void finish(float v, int t, int row) const {
    const size_t at = static_cast<size_t>(t) * a.d + row;
    if constexpr (sizeof(AT) == 2) {
      if (a.res) v += bf16_to_f32(static_cast<const bf16_t*>(a.res)[at]);
      static_cast<bf16_t*>(a.out)[at] = f32_to_bf16(v);
    } else {
      if (a.res) v += static_cast<const float*>(a.res)[at];
      static_cast<float*>(a.out)[at] = v;
    }
  }

  __device__ void w2_share(int b) const {
    const int quads = a.d / 4;
    if (2 * quads <= a.wgs) {
      // fewer row quads than workgroups: several workgroups share one, each
      // with at least eight chunks per wave
      const int C = (a.I + G::kChunk - 1) / G::kChunk;
      const int parts = max(min(a.wgs / quads, uniform(sel.n) * C / (8 * kWaves)), 1);
      if (b < quads * parts) w2_rows<1>(4 * (b % quads), b / quads, parts);
      return;
    }
    const int q1 = static_cast<int>(static_cast<int64_t>(quads) * (b + 1) / a.wgs);
    int q = static_cast<int>(static_cast<int64_t>(quads) * b / a.wgs);
    for (; q + 4 <= q1; q += 4) w2_rows<4>(4 * q, 0, 1);
    switch (q1 - q) {
      case 3: w2_rows<3>(4 * q, 0, 1); break;
      case 2: w2_rows<2>(4 * q, 0, 1); break;
      case 1: w2_rows<1>(4 * q, 0, 1); break;
    }
  }
};

// The meeting between the halves.  A workgroup that has written its share sets
// its flag.  Workgroup 0 polls the flags, a thread each, and writes the groups'
// go words once all are set; the others poll their group's.  A workgroup that
// has waited too long reads the flags itself.

// Share b is out (every thread's stores of it are complete before the barrier).
__device__ __forceinline__ void dec_publish(const DecodeArgs& a, int b) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) dec_write(dec_word(a, kDecFlag + b), 1);
}

// Waits until every share is out (-1), or until `limit` ticks of the 100 MHz
// clock have passed: then one whose flag is missing, the first from the
// caller's own index on (-1 if none is by now).
__device__ __forceinline__ int dec_wait(const DecodeArgs& a, int64_t limit, int* lds) {
  constexpr int kNone = 1 << 30;
  const int tid = threadIdx.x, me = blockIdx.x;
  const int64_t start = wall_clock64();
  bool done;
  if (me == 0) {
    bool late;
    do {
      done = __syncthreads_and(tid >= a.wgs || dec_read(dec_word(a, kDecFlag + tid)));
      late = __syncthreads_or(tid == 0 && wall_clock64() - start >= limit);
    } while (!done && !late);
  } else {
    if (tid < 64) {
      const int32_t* go = dec_word(a, kDecGo + me / kDecGroup);
      int set;
      while (!(set = uniform(dec_read(go))) && wall_clock64() - start < limit)
        __builtin_amdgcn_s_sleep(1);
      if (tid == 0) *lds = set;
    }
    __syncthreads();
    done = *lds != 0;
    __syncthreads();
  }
  int found = -1;
  if (!done) {
    if (tid == 0) *lds = kNone;
    __syncthreads();
    if (tid < a.wgs && !dec_read(dec_word(a, kDecFlag + tid)))
      atomicMin(lds, (tid - me + a.wgs) % a.wgs);
    __syncthreads();
    const int missing = uniform(*lds);
    __syncthreads();
    if (missing != kNone) found = (missing + me) % a.wgs;
  }
  if (found < 0 && me == 0 && tid < kDecGroups) dec_write(dec_word(a, kDecGo + tid), 1);
  return found;
}

template <typename WT, bool kMany>
__global__ __launch_bounds__((64 * dec_waves<WT, kMany>()), (dec_waves<WT, kMany>() / 4)) void
decode_layer_kernel(DecodeArgs a, int phases) {
  using Layer = DecLayer<WT, kMany>;
  __shared__ DecSel sel;
  // the units' sums; before them, the selection's scratch
  __shared__ __attribute__((aligned(16))) union {
    float red[Layer::kSlots][Layer::kTok][16];
    DecScratch scratch;
  } lds;
  __shared__ __attribute__((aligned(1024))) uint8_t w0[kMany ? 8 : 1][kMany ? 4096 : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t w1[kMany ? 8 : 1][kMany ? 4096 : 16];
  __shared__ int next, ticket;
  if (threadIdx.x == 0) ticket = 0;
  dec_select<Layer::kWaves>(a.logits, a.T, a.E, a.k, sel, lds.scratch);
  const int wave = static_cast<int>(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  const Layer layer{a, sel, lds.red, &ticket, w0[kMany ? wave : 0], w1[kMany ? wave : 0],
                    static_cast<int>(threadIdx.x & 63), wave};
  if (phases & 1) {
    int64_t limit = a.wait_limit;
    for (int b = blockIdx.x; b >= 0;) {  // b is wave-uniform
      layer.w13_share(b);
      if (!(phases & 2)) return;
      dec_publish(a, b);
      b = dec_wait(a, limit, &next);
      limit = 0;
    }
    // h as the others wrote it: one wave discards what this compute unit and
    // its XCD hold, the barrier extends that to the other waves (a fence in
    // every wave, 4096 in all, cost 25 us, this one 3)
    if (threadIdx.x < 64) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    __syncthreads();
  }
  layer.w2_share(blockIdx.x);
}

// ------------------------------------------------------------ launchers

int decode_workgroups(int cus) { return cus < kDecMaxWgs ? cus : kDecMaxWgs; }

size_t decode_meet_bytes() { return kDecMeetBytes + kDecSumBytes; }

template <typename AT>
static hipError_t route(const DecodeArgs& a, hipStream_t s) {
  const dim3 grid(a.E, (a.T + kRouteTokens - 1) / kRouteTokens);
  decode_route_kernel<AT><<<grid, kRouteThreads, 0, s>>>(static_cast<const AT*>(a.x), a.w_gate,
                                                         a.logits, a.meet, a.T, a.E, a.d);
  return hipGetLastError();
}

hipError_t launch_decode_route(const DecodeArgs& a, hipStream_t s) {
  return a.w_dtype == kDtypeF32 ? route<float>(a, s) : route<bf16_t>(a, s);
}

template <typename WT>
static hipError_t layer(const DecodeArgs& a, int phases, hipStream_t s) {
  if (a.T <= 4)
    decode_layer_kernel<WT, false><<<a.wgs, 64 * dec_waves<WT, false>(), 0, s>>>(a, phases);
  else
    decode_layer_kernel<WT, true><<<a.wgs, 64 * dec_waves<WT, true>(), 0, s>>>(a, phases);
  return hipGetLastError();
}

hipError_t launch_decode_layer(const DecodeArgs& a, int phases, hipStream_t s) {
  if (a.T < 1 || a.T > kDecodeMaxTokens || a.wgs < 1 || a.wgs > kDecMaxWgs)
    return hipErrorInvalidValue;
  switch (a.w_dtype) {
    case kDtypeF32: return layer<float>(a, phases, s);
    case kDtypeBF16: return layer<bf16_t>(a, phases, s);
    case kDtypeE4M3FN: return layer<fp8_t>(a, phases, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
