// How the GEMMs divide tiles and K slabs among CTAs: the part of the W8A16
// schedule that the kernel and the host must agree on, and the rules by which the
// host chooses a form from the sizes. Nothing here touches the GPU, so all of it
// is checked on the host (tests/native/schedule_check.cu).
#pragma once

#include <stdint.h>

#include "internal.cuh"

namespace fp8blk {

// The slabs one CTA runs, as a run of segments (tile, [kb0, kb1)). Tiles
// [0, dp_tiles) run whole, round robin (CTA c takes c, c + G, ...; G the grid);
// the U = (tiles - dp_tiles) x KB slabs of the other tiles, in
// tile-major order, run stream-K: CTA c takes the contiguous range
// [c U / S, (c + 1) U / S) with S = min(G, U), so every CTA gets the same share
// within one slab, and with fewer slabs than CTAs the first U take one each
// (a CTA in the middle of a split tile must not be without a slab: the
// fix-up reads a partial from every CTA between the tile's first and last).
// A stream-K tile may be split across consecutive CTAs; only a CTA's first
// and last stream-K segments can be partial. dp_tiles = 0 is pure stream-K,
// dp_tiles = tiles pure round robin.
// (Slab counts fit in 32 bits: the host checks tiles x KB.)
// FEW: U may be smaller than G (with one sub-tile the host launches at most U CTAs).
template <bool FEW>
struct Schedule {
  int u, end, first;
  int tile, KB, dp_tiles, grid;
  __host__ __device__ Schedule(int kb_per_tile, int tiles, int dp, unsigned cta, unsigned ctas)
      : tile(static_cast<int>(cta)), KB(kb_per_tile), dp_tiles(dp), grid(static_cast<int>(ctas)) {
    const int64_t U = static_cast<int64_t>(tiles - dp) * kb_per_tile;
    if constexpr (FEW) {
      const int64_t S = U < ctas ? U : ctas;
      const bool some = cta < S;
      first = u = some ? static_cast<int>(U * cta / S) : 0;
      end = some ? static_cast<int>(U * (cta + 1) / S) : 0;
    } else {
      first = u = static_cast<int>(U * cta / ctas);
      end = static_cast<int>(U * (cta + 1) / ctas);
    }
  }
  __host__ __device__ int slabs() const {
    const int dp = tile < dp_tiles ? ((dp_tiles - 1 - tile) / grid + 1) * KB : 0;
    return dp + (end - first);
  }
  __host__ __device__ bool next(int& t, int& kb0, int& kb1) {
    if (tile < dp_tiles) {
      t = tile;
      kb0 = 0;
      kb1 = KB;
      tile += grid;
      return true;
    }
    if (u >= end) return false;
    const int lt = u / KB;
    t = dp_tiles + lt;
    kb0 = u - lt * KB;
    kb1 = KB < kb0 + (end - u) ? KB : kb0 + (end - u);
    u += kb1 - kb0;
    return true;
  }
};

// CTAs a stream-K launch may use (the workspace is sized for this many).
constexpr int kStreamKMaxCtas = 160;

// The tiles a stream-K launch splits across CTAs, worked out on the host:
// CTA c holds slabs [c U / G, (c + 1) U / G) of the U = tiles x KB slabs (G the
// CTAs that have any: at most U), so
// a tile is split when a range boundary falls inside it. Each split tile
// lists its first contributor c0 (whose last segment it is), the number of
// contributors, and the workspace slot c0 wrote (0 if the tile was also
// c0's first segment, else 1); later contributors wrote slot 0.
struct SplitTiles {
  int count;
  int tile[kStreamKMaxCtas];
  short c0[kStreamKMaxCtas];
  unsigned char ncontrib[kStreamKMaxCtas];
  unsigned char slot0[kStreamKMaxCtas];
};

inline SplitTiles split_tiles(int64_t ntiles, int64_t KB, int64_t G) {
  SplitTiles st{};
  const int64_t U = ntiles * KB;
  for (int64_t c0 = 0; c0 + 1 < G; ++c0) {
    const int64_t x = U * (c0 + 1) / G;  // first slab of CTA c0 + 1
    const int64_t t = x / KB, s0 = t * KB;
    const int64_t c0_start = U * c0 / G;
    if (x == s0 || c0_start > s0) continue;  // no split here, or not the tile's first boundary
    const int64_t c1 = ((s0 + KB) * G - 1) / U;  // holds the tile's last slab
    st.tile[st.count] = static_cast<int>(t);
    st.c0[st.count] = static_cast<short>(c0);
    st.ncontrib[st.count] = static_cast<unsigned char>(c1 - c0 + 1);
    st.slot0[st.count] = static_cast<unsigned char>(c0_start == s0 ? 0 : 1);
    ++st.count;
  }
  return st;
}

// Tokens of a W8A16 sub-tile (above 128 tokens a tile is two of them).
inline int token_tile(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

// Workspace bytes of a stream-K launch with grid CTAs and tok-token tiles:
// two FP32 partial slots of [tok][128] per CTA.
inline size_t streamk_bytes(int64_t grid, int tok) {
  return static_cast<size_t>(grid) * 2 * tok * 128 * sizeof(float);
}

// What the stream-K fix-up costs a call, in slabs of one CTA's time (a slab takes
// about twice as long with 128 tokens). Measured, whole minus split in us (device time,
// clean L2), range and median over 20, 40, 74, 110, 200 and 400 tiles of 4 to 68 slabs,
// by the slabs that the split saves:
//                1, 24, 64 tokens   8 saved           11                14                20
//   with residual             -6.8 .. -1.6 (-3.6)  -4.1 .. 0.1 (-1.9)  -3.2 .. 1.6 (-0.7)  -2.7 .. 3.9 (1.2)
//   gated                     -3.7 .. -0.1 (-1.8)  -1.3 .. 1.3 (-0.4)  -0.6 .. 2.8 (1.2)    0.6 .. 5.1 (2.8)
//                128 tokens         3 saved           5                 7                 10
//   with residual             -5.7 .. -0.6 (-4.7)  -4.6 .. -0.5 (-3.4)  -3.0 .. 0.8 (-2.4)  -2.1 .. 3.8 (-0.3)
//   gated                     -2.9 .. 0.8 (-1.7)   -1.7 .. 1.2 (-1.0)  -0.4 .. 2.4 (0.6)    0.3 .. 9.5 (2.4)
// The medians cross near 12 and 6 with the gate and near 15 and 10 with a residual; one
// number for both forms, just below the lower of the two.
constexpr int64_t fixup_slabs(int token_tile) { return token_tile >= 128 ? 5 : 11; }

// The launch of a W8A16 GEMM: the first dp_tiles tiles whole, the others split.
struct SlabPlan {
  int64_t dp_tiles, grid;
};

// One token tile (M <= 128): stream-K over all the slabs, so every SM
// streams the same share of the weights however few tiles there are. With an
// epilogue, whole tiles where the even split would save less than its fix-up costs.
// (The plain linear keeps its order of sums.)
inline SlabPlan one_token_tile_plan(int64_t tiles, int64_t KB, int num_sms, int token_tile,
                                    bool epilogue) {
  const int64_t G = num_sms < kStreamKMaxCtas ? num_sms : kStreamKMaxCtas;
  if (epilogue && cdiv(tiles, G) * KB <= cdiv(tiles * KB, G) + fixup_slabs(token_tile))
    return {tiles, tiles < G ? tiles : G};
  return {0, tiles * KB < G ? tiles * KB : G};
}

// More tokens: whole tiles round robin. When the last wave of tiles would leave at
// least 15% of the SM time idle, and the workspace (bytes of it usable) allows, the
// tiles of that wave run stream-K over all CTAs instead. (Below that the partial
// round trip and the fix-up cost what the even split saves: at 10% idle
// -- 400 tiles on 148 SMs -- both ran in the same time.)
inline SlabPlan many_token_tiles_plan(int64_t tiles, int64_t KB, int num_sms, size_t ws_bytes) {
  const int64_t G = num_sms < kStreamKMaxCtas ? num_sms : kStreamKMaxCtas;
  const int64_t waves = tiles / G, rem = tiles - waves * G;
  const int64_t tail_grid = waves > 0 ? G : (rem * KB < G ? rem * KB : G);
  const bool tail_sk = rem > 0 && (G - rem) * 100 >= 15 * (waves + 1) * G && tail_grid >= 2 &&
                       ws_bytes >= streamk_bytes(tail_grid, 256);
  if (tail_sk) return {waves * G, tail_grid};
  return {tiles, tiles < num_sms ? tiles : num_sms};
}

// CTAs per tile of a W8A8 GEMM with an epilogue: the least of rounds x (slabs per
// CTA + what a round costs besides), in slabs (0.5 us each here): a start and an end
// of about kRoundSlabs, and for the trade kTradeSlabs, more with two CTAs, where each
// finishes half of a tile. At least kMinSplitSlabs slabs each. Measured (one CTA per
// tile -> this rule, 16 tokens, residual): 25600 -> 5120 119 -> 48 us, 8192 -> 5120
// 44 -> 23, 4096 -> 2560 25 -> 13, 1024 -> 5120 12.5 -> 12.3; two CTAs: 8192 -> 16384
// 50 -> 43, 5120 -> 16384 35 -> 32, and at the border 4224 -> 16384 30.1 -> 29.8.
// resident(s): clusters of s CTAs that can be resident at once (0: none).
constexpr int64_t kRoundSlabs = 8, kTradeSlabs = 4, kTradeSlabs2 = 16, kMinSplitSlabs = 2;
template <class F>
int ctas_per_tile(int64_t tiles, int64_t KB, int num_sms, F resident) {
  int best = 1;
  int64_t cost = cdiv(tiles, num_sms) * (KB + kRoundSlabs);
  if (tiles * 2 > num_sms || KB < 2 * kMinSplitSlabs) return 1;  // not few, or nothing to share
  for (int s = 2; s <= 8; s *= 2) {
    const int64_t clusters = resident(s);
    if (clusters <= 0 || KB < s * kMinSplitSlabs) continue;
    const int64_t c =
        cdiv(tiles, clusters) * (cdiv(KB, s) + kRoundSlabs + (s == 2 ? kTradeSlabs2 : kTradeSlabs));
    if (c < cost) cost = c, best = s;
  }
  return best;
}

}  // namespace fp8blk
