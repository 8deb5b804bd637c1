// How the tensor-core key-weight kernel divides its work, over every row count and split
// count that a call may have: prints the first thing that does not hold, exit code 1.
#include <cstdio>
#include <initializer_list>

#include "va_kweights_plan.cuh"

using namespace va::kwplan;

#define HOLDS(c, ...)                                \
  do {                                               \
    if (!(c)) {                                      \
      std::printf("not %s: ", #c);                   \
      std::printf(__VA_ARGS__);                      \
      std::printf("\n");                             \
      return 1;                                      \
    }                                                \
  } while (0)

// Every part of every tile has a row block, and a tile's parts are its blocks in order.
template <int M>
static int parts_have_blocks(int rows, int splits) {
  Shape<M> sh;
  sh.set(rows);
  int stay, pass;
  block_rows(M, &stay, &pass);
  HOLDS(sh.blocks == row_blocks(rows, stay, pass), "mode %d rows %d", M, rows);
  HOLDS(sh.blocks * sh.cols >= rows && sh.cols % 64 == 0, "mode %d rows %d", M, rows);
  const int parts = tile_parts(splits, sh.blocks), kv_len = 600;
  HOLDS(parts >= 1 && parts <= splits, "mode %d rows %d splits %d", M, rows, splits);
  const int n = part_count(kv_len, parts);
  HOLDS(n == 3 * parts, "mode %d rows %d splits %d", M, rows, splits);
  HOLDS(part_cost(sh, parts) >= 1, "mode %d rows %d splits %d", M, rows, splits);
  int next = 0;
  for (int t = 0; t < n; ++t) {
    const Part o = part_at(t, parts, sh.blocks);
    HOLDS(o.at == t / parts && o.part == t % parts, "mode %d rows %d splits %d", M, rows, splits);
    HOLDS(o.rb0 == (o.part ? next : 0), "mode %d rows %d splits %d", M, rows, splits);
    HOLDS(o.rb0 < o.rb1, "mode %d rows %d splits %d part %d of %d", M, rows, splits, o.part, parts);
    next = o.rb1;
    HOLDS(o.part + 1 < parts || next == sh.blocks, "mode %d rows %d splits %d", M, rows, splits);
  }
  return 0;
}

// Keys and rows of a block fit beside each other in shared memory, each ring with a slot.
template <int M>
static int rings_fit(int rows) {
  using Ch = Chunks<M>;
  Shape<M> sh;
  sh.set(rows);
  HOLDS(sh.k_slots() >= 1 && sh.k_slots() <= kMaxK, "mode %d rows %d", M, rows);
  const int keys_end = sh.k_at() + sh.k_slots() * Ch::k_slot;
  HOLDS(keys_end <= kRegion, "mode %d rows %d", M, rows);
  if (sh.stay) {
    HOLDS(sh.q_at() + Ch::n * sh.q_slot() >= sh.rows_stay() && sh.rows_stay() <= sh.k_at(),
          "mode %d rows %d", M, rows);
  } else {
    HOLDS(sh.q_slots() >= 1 && sh.q_slots() <= kMaxQ, "mode %d rows %d", M, rows);
    HOLDS(sh.q_at() >= keys_end && sh.q_at() + sh.q_slots() * sh.q_slot() <= kRegion,
          "mode %d rows %d", M, rows);
  }
  return 0;
}

template <int M>
static int mode() {
  for (int rows = 0; rows <= VA_MAX_QLEN * 128; ++rows) {
    if (rings_fit<M>(rows)) return 1;
    for (int splits = 1; splits <= VA_MAX_SPLITS; ++splits)
      if (parts_have_blocks<M>(rows, splits)) return 1;
  }
  for (int rows : {1 << 16, (1 << 22) - 1, 1 << 22})
    if (rings_fit<M>(rows) || parts_have_blocks<M>(rows, 1) || parts_have_blocks<M>(rows, VA_MAX_SPLITS))
      return 1;
  // what a call plans for is within the limits of its workspace and status
  for (long long nodes : {1, 5, 16, 65})
    for (long long heads : {1, 16, 64, 128})
      for (long long tiles = 1; tiles < 5000; tiles = tiles * 3 / 2 + 1) {
        const int s = plan_splits(M, nodes * heads, tiles, 74);
        HOLDS(s >= 1 && s <= VA_MAX_SPLITS, "mode %d rows %lld tiles %lld", M, nodes * heads, tiles);
      }
  return 0;
}

int main() { return mode<kBf16>() || mode<kFp8>() || mode<kF32>(); }
