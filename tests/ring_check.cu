// The page ring of the mma.sync decode kernel, replayed on the host.
//
// Teams of warps walk a stream of 16-key blocks (block j goes to team j mod
// teams), pages of `bpp` blocks lie in a ring of S stages, and a stage's last
// reader issues the page S ahead into it. A wait for a page looks at the
// parity of its stage's phase only. For the ring that geometry() gives every
// shape the replay stalls a team or a page's copy for as long as anything else
// can move, over and over, and checks that no wait passes before its page has
// landed and that none waits for ever.
//
//   ring_check            every shape; prints "rings <n> bad <n>"
//   ring_check S teams bpp gated   one ring
#include <cstdio>
#include <cstdlib>
#include <set>
#include <tuple>
#include <vector>

#include "nk_decode_mma.cuh"

static unsigned long long seed = 1;
static unsigned rnd(unsigned n) {
  seed = seed * 6364136223846793005ull + 1442695040888963407ull;
  return (unsigned)(seed >> 33) % n;
}

// false: a wait passed early, or nothing moves any more
static bool replay(int S, int teams, int bpp, bool gated, int trials) {
  const int pages = 6 * S + 4 * teams + 5, blocks = pages * bpp;
  for (int trial = 0; trial < trials; ++trial) {
    std::vector<int> issued(S), landed(S), done(pages), next(teams);
    for (int s = 0; s < S && s < pages; ++s) issued[s] = 1;
    for (int t = 0; t < teams; ++t) next[t] = t;
    auto can = [&](int a) {  // actors: teams, then the stages' copies
      if (a >= teams) return landed[a - teams] < issued[a - teams];
      if (next[a] >= blocks) return false;
      const int q = next[a] / bpp, s = q % S, k = q / S;
      if (gated && issued[s] <= k) return false;
      return (landed[s] & 1) != (k & 1);  // try_wait.parity
    };
    const int actors = teams + S;
    int victim = (int)rnd(actors), moves = 0;
    for (;;) {
      int a = -1;
      const int from = (int)rnd(actors);
      for (int i = 0; i < actors && a < 0; ++i) {
        const int c = (from + i) % actors;
        if (c != victim && can(c)) a = c;
      }
      if (a < 0) {  // only the stalled one is left: one step, then another is stalled
        if (!can(victim)) break;
        a = victim;
        victim = (int)rnd(actors);
      } else if (++moves % 64 == 0 && rnd(8) == 0) {
        victim = (int)rnd(actors);
      }
      if (a >= teams) {
        ++landed[a - teams];
        continue;
      }
      const int q = next[a] / bpp, s = q % S, k = q / S;
      if (landed[s] != k + 1) return false;
      next[a] += teams;
      if (++done[q] == bpp && q + S < pages) ++issued[s];
    }
    for (int t = 0; t < teams; ++t)
      if (next[t] < blocks) return false;
  }
  return true;
}

int main(int argc, char** argv) {
  if (argc == 5) {
    const bool ok = replay(atoi(argv[1]), atoi(argv[2]), atoi(argv[3]), atoi(argv[4]) != 0, 200);
    printf("%s\n", ok ? "good" : "bad");
    return 0;
  }
  using namespace nk;
  std::set<std::tuple<int, int, int, bool>> rings;
  const int fmts[4] = {kFmtI8F32, kFmtI8F16, kFmtRk8v4, kFmtBf16};
  int wrong = 0;
  for (int f = 0; f < 4; ++f)
    for (int win = 0; win < 2; ++win)
      for (int D = 64; D <= 256; D *= 2)
        for (int NT = 1; NT <= 6; ++NT)
          for (int P = 16; P <= 256; P += 16)
            for (int B = 1; B <= 1024; B += B < 64 ? 9 : 64) {
              if (win && fmts[f] != kFmtI8F32) continue;
              const int CS = fmts[f] == kFmtRk8v4 ? mma::channel_split_rk(D, NT) : mma::channel_split(D, NT);
              const mma::Geometry g = mma::geometry(fmts[f], D, NT, CS, P, B, win != 0);
              if (g.stages < 2) continue;
              if (g.total > mma::kSmemLimit || g.stages > g.max_stages) ++wrong;
              rings.insert(std::make_tuple(g.stages, mma::kConsumerWarps / CS, P / 16, g.gated));
            }
  for (const auto& r : rings)
    if (!replay(std::get<0>(r), std::get<1>(r), std::get<2>(r), std::get<3>(r), 40)) {
      printf("%d stages, %d teams, %d blocks a page, gated %d\n", std::get<0>(r), std::get<1>(r), std::get<2>(r),
             (int)std::get<3>(r));
      ++wrong;
    }
  printf("rings %d bad %d\n", (int)rings.size(), wrong);
  return 0;
}
