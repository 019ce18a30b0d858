// The plan of a ragged step over the 8-bit cache: what kv8_plan writes and the
// step's other calls read.
//
// A step has B streams; stream b brings n consecutive rows (a prompt, a part
// of one, a token) or a tree of at most 64 drafted rows.  For the attention, a
// stream's n rows x G heads of a kv head's group are n * G query rows (row r
// is head r % G of row r / G), 256 to a block, and the blocks of all its kv
// heads stand one behind the other with `tiles` tiles of 128 positions each:
// cut every `cut` tiles, that line falls into the pieces which the GPU works
// on.  The cut depends on the stream's own n and length only, so a stream's
// bytes do not depend on its batch.
#pragma once

#include <algorithm>

#include "kv8.cuh"

namespace bm {
namespace kv8 {

constexpr int kMaxStreams = 1024, kMaxRows = 1 << 20, kMaxStepGroup = 8, kDrafts = 64;
constexpr int kBlockRows = 256, kTile = 128;
constexpr int kPlanMagic = 0x6b763870;

struct PlanHead {
  int magic, B, T, qh, kvh, slots, cap, items;
  int units, pad[7];      // slabs of 16 query rows of cut streams
};
struct PlanStream {
  int start, n, slot, len;    // first row, rows (0: none, or refused), slot, positions with the step's own
  int tree;                   // 1: the rows attend to each other by their masks
  int cut, pitch, most;       // tiles to a piece (0: uncut), to a block on the line; the most pieces a block has
  int unit;                   // of the cut streams' slabs of 16 query rows, the first of this one's
  long long rec;              // its first record: a slab has `most` of them
  int base, refused;          // positions before the step; 1: a stream that does not fit
  int pad[2];
};
// One piece of one block: tiles t0 .. t1 - 1.
struct PlanItem {
  unsigned who;               // stream, kv head << 10
  unsigned what;              // block, piece << 16 (65535: the block's only one)
  int t0, t1;
};
static_assert(sizeof(PlanHead) == 64 && sizeof(PlanStream) == 64 && sizeof(PlanItem) == 16, "layout");
constexpr unsigned kWhole = 65535;

// Addresses inside a plan: head, streams, masks, items.
struct Plan {
  PlanHead* head;
  PlanStream* streams;
  unsigned long long* masks;
  PlanItem* items;
  __host__ __device__ Plan(void* p, int B, int T) {
    head = static_cast<PlanHead*>(p);
    streams = reinterpret_cast<PlanStream*>(head + 1);
    masks = reinterpret_cast<unsigned long long*>(streams + B);
    items = reinterpret_cast<PlanItem*>(masks + (T + 1) / 2 * 2);
  }
};

__host__ __device__ inline int blocks_of(int n, int G) { return (n * G + kBlockRows - 1) / kBlockRows; }
__host__ __device__ inline int tiles_of(int len) { return (int)(((long long)len + kTile - 1) / kTile); }

// Tiles to a piece (0: blocks stay whole), and tiles from one block's begin to the next's on the line.
// A piece has a fixed cost (its query rows, its records to write and to merge), so cuts are at least 4 tiles
// apart, twice that for each fourfold length beyond 2048; what is left behind a block's last cut is a piece of its
// own, shorter than that (33 tiles are cut 8 8 8 8 1), and so are pieces at both ends of a block on the line.  A stream
// alone should fill the GPU: up to half as many blocks as SMs are each cut evenly; more of them, up to four for each SM, where the line of
// all blocks passes a multiple of an SM's share, so that the SMs end together (rows that
// mostly attend to each other have blocks of many sizes, which do without).
struct Cut {
  int cut, pitch;
};
__host__ __device__ inline Cut cut_of(int n, int len, int G, int kvh) {
  const long long P = (long long)blocks_of(n, G) * kvh;
  const int tiles = tiles_of(len);
  int least = 4;
  for (long long border = 2048; len > border; border *= 4) least *= 2;
  if (P <= kSms / 2) {
    const int pieces = kSms / (int)P, even = (tiles + pieces - 1) / pieces, cut = even > least ? even : least;
    return cut < tiles ? Cut{cut, (tiles + cut - 1) / cut * cut} : Cut{0, tiles};
  }
  if (P >= 4 * kSms || tiles < 32 || len / 2 < n) return Cut{0, tiles};
  const int even = (int)((P * tiles + kSms - 1) / kSms);
  return Cut{even > least ? even : least, tiles};
}
// The most pieces a block falls into.
__host__ __device__ inline int most_pieces(int tiles, Cut c) { return !c.cut ? 1 : c.pitch % c.cut == 0 ? c.pitch / c.cut : (tiles - 1) / c.cut + 2; }

// Block i (= block * kvh + kv head) of a stream: its pieces, of the tiles that its rows attend to.
struct Pieces {
  long long from, first;   // where the block begins on the line, and the piece of the line that holds it
  int count, cut, ext;
  __host__ __device__ Pieces(int i, Cut c, int ext_positions) {
    cut = c.cut;
    ext = tiles_of(ext_positions);
    from = (long long)i * c.pitch;
    if (!cut || ext <= 0) {
      first = 0;
      count = 1;
    } else if (from + ext < 0x7FFFFFFF) {           // as a rule: a 64-bit quotient takes far longer
      first = (int)from / cut;
      count = ((int)from + ext - 1) / cut - (int)first + 1;
    } else {
      first = from / cut;
      count = (int)((from + ext - 1) / cut - first) + 1;
    }
  }
  __host__ __device__ int begin(int c) const { return c == 0 || !cut ? 0 : (int)((first + c) * cut - from); }
  __host__ __device__ int end(int c) const { return c == count - 1 || !cut ? ext : (int)((first + c + 1) * cut - from); }
};
// Positions that a block's last row attends to.
__host__ __device__ inline int extent_of(int block, int n, int len, int G, int tree) {
  if (tree) return len;
  const long long last = (long long)block * kBlockRows + kBlockRows - 1, rows = (long long)n * G;
  return len - n + (int)((last < rows ? last : rows - 1) / G) + 1;
}

// Bounds on what a step needs, from its sizes alone; none falls where B, T or the cache's capacity grows.
// Blocks: 256 P query rows are at most the stream's own and a block more for each kv head.  Pieces: at most kSms
// where blocks are cut evenly, kSms + 2 P on a line.
inline int64_t most_items(int B, int T, int qh, int kvh) {
  return (int64_t)B * (kSms + 2 * kvh + 2) + 2 * (((int64_t)T * qh + kBlockRows - 1) / kBlockRows);
}
inline size_t plan_bytes(int B, int T, int qh, int kvh) {
  return sizeof(PlanHead) + B * sizeof(PlanStream) + (size_t)(T + 1) / 2 * 16 + most_items(B, T, qh, kvh) * sizeof(PlanItem);
}
// Records, in query rows times pieces: a stream's rows of a kv head are rounded up to 16.  At most kSms blocks' worth of a
// stream whose blocks are cut evenly, 9 kSms (kSms and twice 4 kSms) on a line.
inline int64_t most_records(int B, int T, int qh, int kvh, int cap) {
  const int tiles = tiles_of(cap);
  int64_t most = 0, least = 4;
  for (long long border = 2048; cap > border; border *= 4, least *= 2) most = border / kTile / least;
  most = std::max<int64_t>(most, (tiles + least - 1) / least);
  most = std::min<int64_t>(most, kSms / kvh);
  if (tiles >= 32) most = std::max<int64_t>(most, 4);
  if (most < 2) return 0;
  const bool line = (int64_t)blocks_of(T, qh / kvh) * kvh > kSms / 2;
  return std::min<int64_t>(((int64_t)T * qh + (int64_t)B * 16 * kvh) / 16 * 16 * most, (int64_t)B * kBlockRows * kSms * (line ? 9 : 1));
}

inline bool step_shapes_ok(int B, int T, int qh, int kvh) {
  return B >= 1 && B <= kMaxStreams && T >= 1 && T <= kMaxRows && kvh >= 1 && kvh <= 1024 && qh >= 1 && qh <= 1024 && qh % kvh == 0 &&
         qh / kvh <= kMaxStepGroup;
}

}  // namespace kv8
}  // namespace bm
