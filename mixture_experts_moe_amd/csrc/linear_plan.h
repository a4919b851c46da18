// The dense product's arguments and the choice of its kernel (host code that
// needs no HIP).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace moe {

// Mirrors of the ABI dtype / scale codes (moe.h), for device code.
constexpr int kDtypeF32 = 0;
constexpr int kDtypeBF16 = 1;
constexpr int kDtypeE4M3FN = 2;
constexpr int kScaleNone = 0;
constexpr int kScaleTensor = 1;
constexpr int kScaleChannel = 2;

// Mirrors of MOE_FN_* (moe.h).
constexpr int kFnNone = 0;
constexpr int kFnRelu = 1;
constexpr int kFnSilu = 2;
constexpr int kFnGelu = 3;
constexpr int kFnGeluTanh = 4;

struct LinearArgs {
  const void* x;       // [M, K] act dtype
  const void* w;       // [R, K] weight dtype
  const float* scale;  // [R] or [1], or nullptr
  const float* bias;   // [R] or nullptr
  const void* res;     // [M, N] act dtype or nullptr
  void* out;           // [M, N] act dtype
  float* part;         // [splits, M, R] fp32 (workspace) when K is split, else nullptr
  int64_t M;
  int N, R, K;         // R = N, or 2N when gated
  int64_t ldx, ldw, ldr, ldo;  // elements
  int act_dtype, w_dtype, fn;
  bool gated, scale_channel;
  bool vec4, vec8;     // out (and residual) rows hold aligned vectors of four, eight
  int tile;            // the kernel that runs (linear_plan)
  bool aligned;        // every row that it reads holds whole 16-byte units
  int splits;          // K ranges, each ksplit long (the last may be shorter)
  int ksplit;
  bool pack_x, pack_w; // rows copied to the workspace first, kpack elements each
  int kpack;
  void* xpack;
  void* wpack;
};

// At most this many tokens stream W (stream.h).
constexpr int kLinStreamTokens = 16;

// ------------------------------------------------------------ choice of kernel
//
// Up to four tokens take the 4x4 MFMAs, up to 16 the 16x16 ones (4 x 4096 x
// 4096 bf16: 4x4 8.6 us, 16x16 10.2; 4 x 28672 x 4096 e4m3fn 28.7, 36.6), one
// 16-row tile of W per workgroup.  More tiles than compute units but fewer than
// two each leave some with twice the work of others; e4m3fn weights are half
// the bytes of their tokens, so two tiles per workgroup, sharing each token
// load, are faster there (16 x 4500 x 7168: 20.5 us with one, 15.9 with two;
// 8 x 7168 x 4096 12.7, 12.4) and slower elsewhere (8 x 4096 x 4096: 8.6, 10.1;
// 8 x 28672 x 4096: 33.8, 38.2).
//
// More than 16 tokens: the tile and the number of K ranges with the least
// estimated time.  A workgroup's K stage takes what its loads take (a part
// that does not depend on the size and about 60 GB/s per compute unit,
// shared by the workgroups on it) or what its MFMAs take; in fp32 the MFMAs are
// nearly all of a stage and it takes a multiple of theirs that was measured for
// each tile.  Workgroups run in rounds of as many as a compute unit's LDS holds;
// the raster gives each XCD whole tiles, so that with few of them some XCDs have
// one more than others, or none (333 x 1696 x 8752 bf16, 42 tiles of 128 x 128:
// six K ranges 44 us, four 35).  Split sums are written and read once more.
// The constants were fitted to the tiles' times alone and side by side (bf16,
// one workgroup per unit: 128 x 128 0.81 us a stage, 64 x 64 0.54; the 256 x 256
// tile 1.08).  Against every tile with every number of K ranges the choice is
// on average 4% slower than the best in bf16 (83 sizes of 17..4096 tokens x
// 64..14336 rows and K; at worst 21%), 3% in e4m3fn (74; 14%) and 2% in fp32
// (141; 16%).

enum LinearTile { kTileStream4, kTileStream16, kTileStream16Pair, kTile256, kTile128, kTile128Pair,
                  kTile128x64, kTile128x64Pair, kTile64, kTileStaged128, kTileStaged64 };

struct TileCost {
  int tile, rows, tokens;
  int types;      // weight bytes that it is built for, or'ed
  int lds_kb[2];  // stages in LDS: with weights of two or four bytes, of one
  float fixed;    // us per stage apart from the bytes
  float start;    // us per workgroup: first loads and epilogue
  // fp32: a stage in times of its MFMAs, of one workgroup and of each of several
  // on a compute unit, and `start`
  float alone, shared, start32;
};
// the aligned tiles, then the staged ones (a tile is not built for types whose
// every size has a cheaper one: fp32 is bound by its MFMAs in any tile, and
// e4m3fn's stages are small enough to hold two workgroups or four stages)
constexpr TileCost kTileCosts[] = {
    {kTile256, 256, 256, 1 | 2, {160, 128}, 0.27f, 11.f, 0.f, 0.f, 0.f},
    {kTile128, 128, 128, 2, {128, 96}, 0.27f, 1.f, 0.f, 0.f, 0.f},
    {kTile128Pair, 128, 128, 1 | 2 | 4, {64, 48}, 0.27f, 1.f, 1.2f, 0.97f, 1.7f},
    {kTile128x64, 128, 64, 1 | 2, {144, 64}, 0.27f, 1.f, 0.f, 0.f, 0.f},
    {kTile128x64Pair, 128, 64, 2 | 4, {72, 48}, 0.27f, 1.f, 1.2f, 1.01f, 0.1f},
    {kTile64, 64, 64, 1 | 2 | 4, {64, 48}, 0.25f, 0.5f, 1.4f, 1.16f, 0.f},
    {kTileStaged128, 128, 128, 1 | 2 | 4, {32, 24}, 1.2f, 1.f, 1.2f, 1.04f, 5.5f},
    {kTileStaged64, 64, 64, 1 | 2 | 4, {16, 12}, 0.7f, 1.f, 1.48f, 1.25f, 0.f},
};
constexpr int kComputeUnits = 256;
constexpr int kRasterXcds = 8;
constexpr float kUsPerKb = 0.017f;

// The tile and K ranges of the least estimated time among the aligned tiles
// or the staged ones: that time, and the choice in *a.
inline float linear_choose(LinearArgs* a, bool aligned) {
  const int wb = a->w_dtype == kDtypeE4M3FN ? 1 : a->w_dtype == kDtypeBF16 ? 2 : 4;
  const int kc = wb == 4 ? 32 : 64;
  const float bytes = static_cast<float>(a->R) * a->K * wb +
                      static_cast<float>(a->M) * (a->K + a->N) * (wb == 4 ? 4 : 2);
  float best = 1e30f;
  for (const TileCost& t : kTileCosts) {
    if (!(t.types & wb) || aligned != (t.tile < kTileStaged128)) continue;
    const int64_t tiles = ((a->M + t.tokens - 1) / t.tokens) * ((a->R + t.rows - 1) / t.rows);
    const float kb = (t.rows * kc * wb + t.tokens * 128) / 1024.f;
    // a compute unit's MFMAs: 4096 flops a clock in bf16, 256 in fp32, 2.1 GHz
    const float mfma = 2.f * t.rows * t.tokens * kc / (wb == 4 ? 256.f : 4096.f) / 2100.f;
    const int waves = t.rows == 64 ? 4 : 8;
    int held = 160 / t.lds_kb[wb == 1];
    if (held > 16 / waves) held = 16 / waves;
    for (int want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      // ranges of whole stage pairs, of at least four stages
      const int per = ((a->K + want - 1) / want + 2 * kc - 1) / (2 * kc) * (2 * kc);
      if (want > 1 && per < 4 * kc) break;
      const int splits = (a->K + per - 1) / per;
      const float stages = static_cast<float>((per + kc - 1) / kc);
      // workgroups of the compute unit that has most (the aligned tiles' raster
      // is per XCD, the staged ones' workgroups go to the units in turn)
      constexpr int kUnits = kComputeUnits / kRasterXcds;
      const int64_t here =
          aligned ? ((tiles + kRasterXcds - 1) / kRasterXcds * splits + kUnits - 1) / kUnits
                  : (tiles * splits + kComputeUnits - 1) / kComputeUnits;
      auto round_us = [&](int n) {
        if (wb == 4) return stages * mfma * (n == 1 ? t.alone : n * t.shared) + t.start32;
        // (staged tiles overlap their MFMAs with little else)
        const float products = n * mfma * (aligned ? 1.1f : 1.6f);
        float stage = t.fixed + kUsPerKb * kb;
        if (n * kUsPerKb * kb > stage) stage = n * kUsPerKb * kb;
        if (products > stage) stage = products;
        return stages * stage + t.start;
      };
      float us = (here / held) * round_us(held);
      if (here % held) us += round_us(static_cast<int>(here % held));
      if (us < bytes / 4.7e6f) us = bytes / 4.7e6f;
      if (splits > 1)
        us += 2.5f + static_cast<float>(splits) * a->M * a->R * 8.f / (wb == 4 ? 5e6f : 3e6f);
      if (us < best) {
        best = us;
        a->tile = t.tile;
        a->splits = splits;
        a->ksplit = splits > 1 ? per : a->K;
      }
    }
  }
  return best;
}

// Chooses the kernel and the K split (the other fields set, pointers not yet
// needed).
inline void linear_plan(LinearArgs* a) {
  const int wsz = a->w_dtype == kDtypeE4M3FN ? 1 : a->w_dtype == kDtypeBF16 ? 2 : 4;
  const int xsz = a->act_dtype == kDtypeF32 ? 4 : 2;
  const bool w_ok = a->ldw * wsz % 16 == 0 && a->K * wsz % 16 == 0;
  const bool x_ok = a->ldx * xsz % 16 == 0 && a->K * xsz % 16 == 0;
  a->splits = 1;
  a->ksplit = a->K;
  a->pack_x = a->pack_w = false;
  a->kpack = (a->K * wsz + 15) / 16 * 16 / wsz;
  if (a->M <= kLinStreamTokens) {
    const int tiles = (a->R + 15) / 16;
    const bool pair = wsz == 1 && tiles > kComputeUnits && tiles < 2 * kComputeUnits;
    a->tile = a->M <= 4 ? kTileStream4 : pair ? kTileStream16Pair : kTileStream16;
    // a few unaligned tokens cost less to copy than W costs to read unaligned
    a->pack_x = a->M > 4 && w_ok && !x_ok;
    a->aligned = w_ok && (x_ok || a->pack_x);
    return;
  }
  a->aligned = w_ok && x_ok;
  if (a->aligned) {
    linear_choose(a, true);
    return;
  }
  LinearArgs packed = *a;
  packed.pack_x = !x_ok || !w_ok;  // K must be padded in both
  packed.pack_w = !w_ok;
  packed.aligned = true;
  float us = linear_choose(&packed, true) + 2.5f;
  us += 2.f * static_cast<float>(a->M) * a->K * xsz / 4e6f;
  if (packed.pack_w) us += 2.f * static_cast<float>(a->R) * a->K * wsz / 4e6f;
  // (a launch of at most 2^32 threads)
  const bool fits = (static_cast<int64_t>(a->R) * wsz + a->M * xsz) * a->kpack < int64_t{1} << 35;
  if (us < linear_choose(a, false) && fits) *a = packed;
}

// Workspace: the K ranges' sums, packed x, packed W.
inline size_t linear_part_bytes(const LinearArgs& a) {
  return a.splits > 1 ? static_cast<size_t>(a.splits) * a.M * a.R * 4 : 0;
}
// The bytes a plan needs; sets its pointers into `ws` unless that is null.
inline size_t linear_workspace(LinearArgs* a, void* ws) {
  size_t at = 0;
  auto take = [&](size_t n) {
    void* p = ws && n ? static_cast<char*>(ws) + at : nullptr;
    at += (n + 255) / 256 * 256;
    return p;
  };
  const int wsz = a->w_dtype == kDtypeE4M3FN ? 1 : a->w_dtype == kDtypeBF16 ? 2 : 4;
  a->part = static_cast<float*>(take(linear_part_bytes(*a)));
  const int xsz = a->act_dtype == kDtypeF32 ? 4 : 2;
  a->xpack = take(a->pack_x ? static_cast<size_t>(a->M) * a->kpack * xsz : 0);
  a->wpack = take(a->pack_w ? static_cast<size_t>(a->R) * a->kpack * wsz : 0);
  return at;
}

}  // namespace moe
