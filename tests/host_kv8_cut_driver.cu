// How a ragged step is cut (kv8_step.cuh), over random steps on the host:
// the pieces of a block cover its tiles once and in order, fit the fields that
// hold them, and never exceed what the plan and the workspace are sized for.
// Usage: host_kv8_cut_driver steps seed; prints the first step that fails.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "kv8_step.cuh"

using namespace bm::kv8;

static std::mt19937_64 rng;
static long long pick(long long lo, long long hi) {   // even over the logarithm, often an end
  if (lo >= hi || rng() % 16 == 0) return lo;
  if (rng() % 16 == 0) return hi;
  const double u = (double)(rng() >> 11) / 9007199254740992.0;
  const long long v = (long long)((double)lo * std::pow((double)hi / (double)lo, u));
  return v < lo ? lo : v > hi ? hi : v;
}

struct Step {
  int B, T, G, kvh, cap, n, len, tree;
};
static int fail(const Step& s, const char* what) {
  std::printf("%s: B %d T %d group %d kv heads %d capacity %d, stream of %d rows and %d positions, tree %d\n", what, s.B, s.T, s.G, s.kvh, s.cap,
              s.n, s.len, s.tree);
  return 1;
}

int main(int argc, char** argv) {
  const int steps = std::atoi(argv[1]);
  rng.seed(std::atoi(argv[2]));
  long long uncut_many = 0, evenly = 0, line = 0, wide = 0;
  for (int i = 0; i < steps; ++i) {
    Step s{};
    s.G = 1 + rng() % kMaxStepGroup;
    s.kvh = (int)pick(1, 1024 / s.G);
    s.cap = (int)pick(1, 2147483647);
    s.B = (int)pick(1, 20);
    int64_t items = 0, records = 0, rows = 0;
    struct One {
      int n, len, tree;
    };
    One of[20];
    for (int b = 0; b < s.B; ++b) {
      of[b].tree = rng() % 4 == 0;
      const long long left = kMaxRows - rows - (s.B - 1 - b);   // a row for each stream that follows
      of[b].n = (int)pick(1, std::min<long long>(s.cap, of[b].tree ? std::min<long long>(left, kDrafts) : left));
      of[b].len = of[b].n + (int)(s.cap == of[b].n ? 0 : pick(1, s.cap - of[b].n) - (rng() % 3 == 0));
      rows += of[b].n;
    }
    s.T = (int)rows;
    if (rows > kMaxRows || !step_shapes_ok(s.B, s.T, s.G * s.kvh, s.kvh)) return fail(s, "a step out of range");
    for (int b = 0; b < s.B; ++b) {
      s.n = of[b].n;
      s.len = of[b].len;
      s.tree = of[b].tree;
      const int blocks = blocks_of(s.n, s.G);
      const int64_t P = (int64_t)blocks * s.kvh;
      const Cut cut = cut_of(s.n, s.len, s.G, s.kvh);
      const int most = most_pieces(tiles_of(s.len), cut);
      if (blocks > 65536 || most >= (int)kWhole) return fail(s, "a field of an item");
      if (most > 1) records += ((int64_t)s.n * s.G + 15) / 16 * s.kvh * most;
      (cut.cut == 0 ? uncut_many : P <= kSms / 2 ? evenly : line) += 1;
      // all blocks of small streams; of large ones the ends and some between, and as many pieces as they could have
      const bool all = P <= 2000;
      int64_t seen = 0;
      for (int64_t k = 0; k < (all ? P : 64); ++k) {
        const int64_t at = all ? k : k < 16 ? k : k < 32 ? P - 1 - (k - 16) : (int64_t)(rng() % P);
        const int ext = extent_of((int)(at / s.kvh), s.n, s.len, s.G, s.tree);
        if (ext < 1 || ext > s.len) return fail(s, "an extent");
        const Pieces p((int)at, cut, ext);
        wide += p.from + p.ext >= 0x7FFFFFFF;
        if (p.count < 1 || p.count > most) return fail(s, "pieces of a block");
        int tile = 0;
        for (int c = 0; c < p.count; ++c) {
          if (p.begin(c) != tile || p.end(c) <= tile) return fail(s, "a piece's tiles");
          tile = p.end(c);
        }
        if (tile != tiles_of(ext)) return fail(s, "a block's tiles");
        seen += p.count;
      }
      items += all ? seen : cut.cut == 0 ? P : P <= kSms / 2 ? P * most : kSms + 2 * P;
    }
    if (items > most_items(s.B, s.T, s.G * s.kvh, s.kvh)) return fail(s, "more items than the plan holds");
    if (16 * records > most_records(s.B, s.T, s.G * s.kvh, s.kvh, s.cap)) return fail(s, "more records than the workspace holds");
  }
  std::printf("steps %d: blocks whole in %lld streams, cut evenly %lld, on the line %lld, places past 31 bits %lld\n", steps, uncut_many, evenly, line, wide);
  return uncut_many && evenly && line && wide ? 0 : 1;
}
