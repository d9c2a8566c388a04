// Host-side check of the GEMMs' schedule (test code, csrc/schedule.cuh).
//
// Without arguments: for many tile, slab and CTA counts, what the CTAs' Schedules
// run covers every slab of every tile exactly once; a CTA writes at most two
// partials, to different slots; and split_tiles lists exactly the split tiles,
// each with the CTAs and slots that hold its slabs, in order, none of them without
// a slab. Prints "ok <cases>" or the first failure.
//
// With arguments, the form that the host rules choose for a size on 148 SMs:
//   w8a16 <0 plain | 1 fused | 2 gated> M N K   -> tiles run whole, tiles split
//   w8a8  <1 fused | 2 gated> M N K R2 R4 R8    -> CTAs per tile, when R2, R4 and R8
//                                                 clusters can be resident
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "schedule.cuh"

using namespace fp8blk;

struct Piece {
  int kb0, kb1, cta, slot;
};

// Walks the CTAs of a launch as the kernels do.
template <bool FEW>
static int check(int tiles, int KB, int dp, int grid) {
  std::vector<std::vector<Piece>> got(tiles);
  for (int c = 0; c < grid; ++c) {
    Schedule<FEW> sc(KB, tiles, dp, c, grid);
    const int total = sc.slabs();
    int t, kb0, kb1, slabs = 0;
    bool first_split = true, used[2] = {false, false};
    while (sc.next(t, kb0, kb1)) {
      if (t < 0 || t >= tiles || kb0 < 0 || kb1 > KB || kb0 >= kb1) return 1;
      slabs += kb1 - kb0;
      const int slot = first_split ? 0 : 1;
      if (t >= dp) first_split = false;
      const bool whole = kb0 == 0 && kb1 == KB;
      if (!whole) {
        if (t < dp || used[slot]) return 2;
        used[slot] = true;
      }
      got[t].push_back({kb0, kb1, c, whole ? -1 : slot});
    }
    if (slabs != total) return 3;
  }
  // What the host tells the fix-up.
  const int64_t U = static_cast<int64_t>(tiles - dp) * KB;
  SplitTiles st{};
  if (dp < tiles && grid >= 2) st = split_tiles(tiles - dp, KB, U < grid ? U : grid);
  if (st.count > kStreamKMaxCtas) return 4;
  std::vector<int> listed(tiles, -1);
  for (int i = 0; i < st.count; ++i) {
    const int t = st.tile[i] + dp;
    if (t < dp || t >= tiles || listed[t] >= 0) return 5;
    listed[t] = i;
  }
  for (int t = 0; t < tiles; ++t) {
    int at = 0;
    for (const Piece& p : got[t]) {  // CTAs in order hold the slabs in order
      if (p.kb0 != at) return 6;
      at = p.kb1;
    }
    if (at != KB) return 7;
    if ((got[t].size() > 1) != (listed[t] >= 0)) return 8;
    if (listed[t] < 0) continue;
    const int i = listed[t];
    if (st.ncontrib[i] != got[t].size()) return 9;
    for (size_t c = 0; c < got[t].size(); ++c)
      if (got[t][c].cta != st.c0[i] + static_cast<int>(c) || got[t][c].slot != (c == 0 ? st.slot0[i] : 0))
        return 10;
  }
  return 0;
}

static int check_all() {
  int cases = 0, r = 0;
  auto fail = [&](const char* what, int64_t tiles, int64_t KB, const SlabPlan& p) {
    printf("fail %d: %s, tiles %lld, slabs %lld, whole %lld, CTAs %lld\n", r, what, (long long)tiles,
           (long long)KB, (long long)p.dp_tiles, (long long)p.grid);
    return 1;
  };
  for (int sms : {1, 2, 7, 132, 148, 160, 200})
    for (int tiles = 1; tiles <= 420; tiles += tiles < 40 ? 1 : 13)
      for (int KB : {1, 2, 3, 4, 5, 7, 8, 16, 33, 40, 64, 200}) {
        for (int bt : {16, 32, 64, 128})
          for (bool epilogue : {false, true}) {
            const SlabPlan p = one_token_tile_plan(tiles, KB, sms, bt, epilogue);
            if (p.grid < 1 || p.grid > sms || p.grid > kStreamKMaxCtas) return fail("grid", tiles, KB, p);
            ++cases;
            if ((r = check<false>(tiles, KB, static_cast<int>(p.dp_tiles), static_cast<int>(p.grid))))
              return fail("one token tile", tiles, KB, p);
          }
        for (size_t ws : {size_t(0), streamk_bytes(kStreamKMaxCtas, 256)}) {
          const SlabPlan p = many_token_tiles_plan(tiles, KB, sms, ws);
          if (p.grid < 1 || p.grid > sms) return fail("grid", tiles, KB, p);
          ++cases;
          if ((r = check<true>(tiles, KB, static_cast<int>(p.dp_tiles), static_cast<int>(p.grid))))
            return fail("many token tiles", tiles, KB, p);
        }
      }
  printf("ok %d\n", cases);
  return 0;
}

int main(int argc, char** argv) {
  if (argc == 1) return check_all();
  auto arg = [&](int i) { return static_cast<int64_t>(atoll(argv[i])); };
  const int64_t epi = arg(2), M = arg(3), N = arg(4), KB = cdiv(arg(5), 128);
  if (!strcmp(argv[1], "w8a16")) {
    const bool one = M <= 128;
    const int64_t tiles = cdiv(M, one ? 128 : 256) * cdiv(N, epi == 2 ? 64 : 128);
    const SlabPlan p = one ? one_token_tile_plan(tiles, KB, 148, token_tile(M), epi != 0)
                           : many_token_tiles_plan(tiles, KB, 148, streamk_bytes(kStreamKMaxCtas, 256));
    const int64_t U = (tiles - p.dp_tiles) * KB;
    const int split = U > 0 && p.grid >= 2 ? split_tiles(tiles - p.dp_tiles, KB, U < p.grid ? U : p.grid).count : 0;
    printf("%lld %d\n", (long long)p.dp_tiles, split);
  } else {
    const int64_t tiles = cdiv(M, 128) * cdiv(N, epi == 2 ? 128 : 256);
    printf("%d\n", ctas_per_tile(tiles, KB, 148, [&](int s) { return arg(s == 2 ? 6 : s == 4 ? 7 : 8); }));
  }
  return 0;
}
