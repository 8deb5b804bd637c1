// How the tensor-core key-weight kernel divides its work: the row blocks of a request,
// the parts of a key tile, the shared memory of a block and what a tile costs.
// Plain arithmetic for the host and the device; no CUDA header is needed.
#pragma once

#include "verifyattn.h"

#ifdef __CUDACC__
#define VA_PLAN_FN __host__ __device__ __forceinline__
#else
#define VA_PLAN_FN inline
#endif

namespace va {
namespace kwplan {

constexpr int kKwDc = VA_D_LATENT, kKwDr = VA_D_ROPE;
constexpr int kTileKeys = 256;        // of the pair
constexpr int kKSlot = 128 * 128;     // bytes of a key chunk: 128 keys x 128 bytes
constexpr int kMaxK = 12, kMaxQ = 8;  // ring slots, at most
constexpr int kRegion = 9 * kKSlot + 9 * 64 * 128;  // keys and rows: 216 KB

VA_PLAN_FN constexpr int plan_min(int a, int b) { return a < b ? a : b; }
VA_PLAN_FN constexpr int plan_max(int a, int b) { return a > b ? a : b; }

enum Mode { kBf16, kFp8, kF32 };

// A row's dims in chunks of 128 bytes: 8 of c_kv and one of k_pe in bf16, 4 of
// c_kv and half a one of k_pe in FP8; planes: numbers that an element is the sum of.
template <int M>
struct Chunks {
  static constexpr int n = M == kFp8 ? 5 : 9;
  static constexpr int planes = M == kBf16 ? 1 : 3, k_planes = M == kF32 ? 3 : 1;
  static constexpr int row_bytes = planes * (M == kFp8 ? 1 : 2) * (kKwDc + kKwDr);  // of a query row
  static constexpr int k_slot = k_planes * kKSlot;
  static VA_PLAN_FN int width(int kc) { return M == kFp8 && kc == n - 1 ? 64 : 128; }
};

// Row blocks of a request of R counted rows, at least one: a single one for up to `stay`
// rows, else blocks of at most `pass`.
VA_PLAN_FN int row_blocks(int R, int stay, int pass) {
  return R <= stay ? 1 : plan_max(1, (R + pass - 1) / pass);
}
// Parts of each of its key tiles where the call plans `splits` for more rows: no more than
// there are blocks, so that every part has one.  The kernel needs that: its loads and
// products are what keeps the barrier between a pair's requests one phase at a time.
VA_PLAN_FN int tile_parts(int splits, int blocks) { return plan_min(splits, blocks); }

struct Part {
  int at, part, rb0, rb1;  // key tile, its part, and that one's row blocks
};
// The t-th of a request's parts, tile by tile.
VA_PLAN_FN Part part_at(int t, int parts, int blocks) {
  const int at = t / parts, part = t - at * parts;
  return Part{at, part, blocks * part / parts, blocks * (part + 1) / parts};
}

// How the rows of a request are multiplied: `blocks` passes of `cols` columns.
// Up to kStay rows stay in shared memory.  Columns go in steps of 64: beside 192 of them 6
// key chunks are in flight, beside 256 only 4, too few for HBM's latency (8000 clocks
// a tile, rows through the ring 5000).  129 to 160 rows take 192 columns; 161 to 192
// would too, but pass by, which has not been measured against it.
template <int M>
struct Shape {
  using Ch = Chunks<M>;
  static constexpr int kStay = M == kFp8 ? 128 : M == kF32 ? -1 : 160, kPass = M == kBf16 ? 256 : 128;
  static constexpr int kKeySlots = M == kF32 ? 3 : Ch::n;  // when rows pass by
  int blocks, cols;
  bool stay;
  VA_PLAN_FN void set(int R) {
    stay = R <= kStay;
    blocks = row_blocks(R, kStay, kPass);
    cols = plan_max(64, ((R + blocks - 1) / blocks + 63) & ~63);
  }
  // ring slots, and where keys and rows lie in the region
  VA_PLAN_FN int rows_stay() const { return cols / 2 * Ch::row_bytes; }
  VA_PLAN_FN int k_slots() const {
    return stay ? plan_min(kMaxK, (kRegion - rows_stay()) / Ch::k_slot) : kKeySlots;
  }
  VA_PLAN_FN int k_at() const { return stay ? rows_stay() : 0; }
  VA_PLAN_FN int q_slot() const { return cols / 2 * 128 * Ch::planes; }
  VA_PLAN_FN int q_slots() const {
    return plan_min(kMaxQ, (kRegion - kKeySlots * Ch::k_slot) / q_slot());
  }
  VA_PLAN_FN int q_at() const { return stay ? 0 : kKeySlots * Ch::k_slot; }
  // Clocks of a tile, for dividing the work: a fit to single tiles, few rows waiting for
  // the keys' share of HBM and rows through the ring for its latency (5400 a pass of
  // 192 columns, 6500 of 256).  A call takes longer than their sum over a pair (78 of
  // 110 us, 217 of 243, 28 of 68 for the first three batches that the kernel's file
  // names): set-up, the first loads and what a change of request drains are not in it.
  VA_PLAN_FN int cost() const {
    const int column = M == kFp8 ? 27 : M == kF32 ? 108 : 18;
    return stay ? plan_max(M == kFp8 ? 3400 : 5400, column * cols + 1000)
                : blocks * (2200 + column * cols) + 300;
  }
};

// Parts of a request's tiles in all, and what one costs.
VA_PLAN_FN int part_count(int kv_len, int parts) {
  return (kv_len + kTileKeys - 1) / kTileKeys * parts;
}
template <int M>
VA_PLAN_FN int part_cost(const Shape<M>& sh, int parts) {
  return plan_max(1, sh.cost() / parts);
}

// Rows that stay and rows of a pass, by mode.
inline void block_rows(int m, int* stay, int* pass) {
  *stay = m == kFp8 ? Shape<kFp8>::kStay : m == kF32 ? Shape<kF32>::kStay : Shape<kBf16>::kStay;
  *pass = m == kFp8 ? Shape<kFp8>::kPass : m == kF32 ? Shape<kF32>::kPass : Shape<kBf16>::kPass;
}

// Parts of a tile that a call plans for: two of them a pair where there are fewer tiles than pairs, while
// there are row blocks for it.  33 against 21 us for 9 tiles of 9 blocks, 53 against
// 27 for 5 of 17, 94 against 69 for 32 of 33; with a tile a pair and more the keys'
// second loads cost more than the even shares give (238 against 260 for 272 of 17).
// fp32 loads the keys for every block anyway.
inline int plan_splits(int m, long long rows, long long tiles, long long pairs) {
  int stay, pass;
  block_rows(m, &stay, &pass);
  if (rows <= stay) return 1;
  const long long blocks = (rows + pass - 1) / pass;
  if (tiles >= (m == kF32 ? 8 : 1) * pairs) return 1;
  long long s = ((m == kF32 ? 8 : 2) * pairs + tiles - 1) / tiles;
  if (s > blocks) s = blocks;
  if (s > VA_MAX_SPLITS) s = VA_MAX_SPLITS;
  return s < 1 ? 1 : (int)s;
}

}  // namespace kwplan
}  // namespace va
