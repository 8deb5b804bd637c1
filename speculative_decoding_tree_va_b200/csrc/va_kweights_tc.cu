// Key weights on tensor cores, sm_100a: bf16 queries over a bf16 or FP8 cache, fp32
// queries over an fp32 or FP8 cache.
//
//   w_j = sum over counted rows r, j visible to r, of
//         exp(scale q_r . k_j - lse_r)
// The keys are the M side of the product and the rows the N side: a CTA pair
// (tcgen05.mma.cta_group::2, M = 256) takes a tile of 256 keys, 128 a CTA,
// and up to 256 rows at a time.  In tensor memory a key is then a lane and a
// row a column, so a thread adds its key's exponentials over the columns in
// a register, and nothing is exchanged between threads but the two halves
// of a tile's columns.  Where tiles are fewer than pairs, several pairs share
// a tile's row blocks, and a small kernel joins their sums in order.
//
// A request's tiles are walked in one of two layouts of shared memory.  Few rows
// (at most 160) are loaded once per pair and request and stay, and the tiles'
// keys come through a ring of 16 KB chunks (128 keys x 64 dims).  More rows: a
// tile's 9 key chunks stay while the rows pass by through a ring, in equal
// blocks.  Either way each key is read from HBM once.  The tiles of
// all requests, in order and weighted by what they cost, are divided into
// equal contiguous ranges, one per pair.
//
// FP8 cache: the codes are the product's operand as they are (kind::f8f6f4), in
// chunks of 128 dims; a first kernel multiplies each query row by a power of two
// and writes it as the sum of three E5M2 numbers.  Three of 3 significant bits
// hold the 8 of a bf16, down to 2^-31 of the row's largest element, so three
// products add up to the exact one; the epilogue undoes the power in fp32.
//
// fp32: a number is the sum of three bf16 (8 + 8 + 8 bits).  Two kernels lay queries
// and cached keys out as such planes; of the nine products those of plane 0 with
// plane 0 go to one accumulator and the five next larger ones to another, which the
// epilogue adds in fp32 (the three left out are below 2^-24 of the first).  A chunk's
// planes of both sides pass through rings, keys again for every row block.
//
// Bound by HBM for few rows (1152 or 576 bytes a key) and by the tensor cores
// for many (128 clocks per 256 x 256 x 16; the tensor pipe is 86 % active for 4160
// rows), in between by the latency of the rings' loads (2900 to 3600 clocks from a
// slot's release to its refill); the exponentials take 16 a clock and SM.
// Measured at 1965 MHz: 64 requests of 512 to 8192 keys and 64 to 576 rows 110 us (930
// TFLOP/s, 3.1 TB/s), 16 of 4161 keys and 4160 rows 243 us (1310 TFLOP/s), 16 of 16449
// FP8 keys and 16 to 112 rows 68 us (2.3 TB/s), 2081 fp32 keys and 2112 rows 49 us.
// The first two draw so much power that the clock falls to 1580 and 1395 MHz within half
// a second of calls: 129 and 283 us then.
#include "va_kweights.cuh"
#include "va_kweights_plan.cuh"
#include "va_tc_ops.cuh"

namespace va {

__device__ unsigned int g_kw_timeouts = 0;  // count of barrier waits that expired

namespace {

using namespace tc;
using namespace kwplan;

constexpr int kWarpK = 0, kWarpMma = 1, kWarpEpi = 2, kWarpQ = 10, kWarpInfo = 11;
constexpr int kThreads = 13 * 32;     // two warps of column data

struct TcParams {
  KwParams k;
  int dense;             // rows of request b start at b * T * H of the q maps
  int run;               // rows that lie in order from a multiple of it on
  const float* q_scale;  // FP8 cache: [B, T H] power of two that undoes the row's
  float scale;           // k.scale, raised against the tensor cores' rounding
  int stall;             // test hook: issue no products (the waits expire)
};

// The tensor cores' fp32 sums round toward zero at each addition, so that scores come
// out short.  By this share of the score on average over the weights, measured against
// 64 bits for mean scores of 3 to 18: bf16 and fp32 4.8e-7 to 5.4e-7, bf16 over FP8
// 1.3e-7 to 2.0e-7, fp32 over FP8 1.0e-7 to 1.5e-7 (a code has one plane, so the
// accumulator of the large products rounds less away).  Left in, it is a common
// error of all rows and does not average out: 1.4e-6 of the weights at a mean score of 3,
// 1e-5 at 18; raised by it 2e-7 and 1.5e-6.  Sums that happen to be exact come out
// long by as much.  A bf16 verify call's own lse is short in the same way, which the
// raise does not undo: relative to the lse it is given the weights are right, and a row's
// add up to 1 + 1.7e-6 at a mean score of 3.
constexpr double kShortBf16 = 5.2e-7, kShortFp8 = 1.8e-7, kShortF32Fp8 = 1.3e-7;

constexpr int kBoxes = 4;  // query boxes of 8, 16, 32 or 64 rows
struct QMaps {
  CUtensorMap nope[kBoxes], pe[kBoxes];
};

struct __align__(16) Ctl {
  uint64_t k_full[kMaxK], k_empty[kMaxK];
  uint64_t q_full[kMaxQ], q_empty[kMaxQ];
  uint64_t r_full;                 // rows that stay
  // A request's last tile of this pair is multiplied.  Every part of a tile has a row
  // block, so its products need loads that all four producers (keys and rows of both
  // CTAs) issue only once they have seen the request before it end here: no phase
  // completes before the one before it has been seen everywhere.
  uint64_t seg_done;
  uint64_t s_full[2], s_empty[2];  // scores in tensor memory
  uint64_t i_full[2], i_empty[2];  // column data of a pass
  uint64_t drain;
  long long start_off, lo, hi;
  int start_b, start_tile;
  uint32_t tmem;
  int abort;
  // of each column of a pass: its node, its row's log-sum-exp and factor; one bit
  // where the column adds nothing (no row, absent node, empty row); and the
  // node of all that a group of 32 columns adds (-1: several)
  uint32_t none[2][8];
  int one[2][8];
  float xsum[2][128];
  uint8_t node[2][256];
  __align__(16) float lse[2][256];
  __align__(16) float factor[2][256];  // FP8 cache
};
constexpr int kScanAt = offsetof(Ctl, xsum);  // the start-up scan uses xsum ..
static_assert(kScanAt % 8 == 0, "scan alignment");
constexpr size_t kSmemBytes = 1024 + kRegion + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The pair's tiles (parts of tiles), in order.  Every warp role walks them by itself.
template <int M>
struct Walk {
  const KwParams* p;
  long long off, end;
  int b, tile, tiles, parts, R, kv_len, cost;
  KwRequest rq;
  Shape<M> sh;
  int at, part, rb0, rb1;  // key tile, its part, and that one's row blocks
  __device__ __forceinline__ void place() {
    const Part o = part_at(tile, parts, sh.blocks);
    at = o.at;
    part = o.part;
    rb0 = o.rb0;
    rb1 = o.rb1;
  }
  __device__ __forceinline__ void load() {
    for (; b < p->B; ++b) {
      rq = kw_request(*p, b);
      if (rq.ok) break;
    }
    if (b < p->B) {
      kv_len = rq.kv_len;
      R = rq.nodes * p->H;
      sh.set(R);
      parts = tile_parts(p->splits, sh.blocks);
      tiles = part_count(kv_len, parts);
      cost = part_cost(sh, parts);
      place();
    }
  }
  __device__ __forceinline__ void start(const KwParams& kp, const Ctl& c) {
    p = &kp;
    b = c.start_b;
    tile = c.start_tile;
    off = c.start_off;
    end = c.hi;
    load();
  }
  __device__ __forceinline__ bool alive() const { return b < p->B && off < end; }
  __device__ __forceinline__ void next() {
    off += cost;
    if (++tile == tiles) {
      ++b;
      tile = 0;
      load();
    } else {
      place();
    }
  }
  // no later tile of this pair belongs to this request
  __device__ __forceinline__ bool last_of_request() const {
    return tile + 1 == tiles || off + cost >= end;
  }
};

// Position in a ring whose length changes from request to request; bit s of
// `used` is the phase of slot s.
struct Ring {
  int slot = 0, n = 1;
  uint32_t used = 0;
  __device__ __forceinline__ void restart(int slots) { slot = 0; n = slots; }
  __device__ __forceinline__ uint32_t phase() const { return (used >> slot) & 1u; }
  __device__ __forceinline__ void advance() {
    used ^= 1u << slot;
    if (++slot == n) slot = 0;
  }
};

template <int M>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kweights_tc_kernel(const __grid_constant__ QMaps tm_q, const __grid_constant__ CUtensorMap tm_ckv,
                   const __grid_constant__ CUtensorMap tm_kpe, const __grid_constant__ TcParams tp) {
  using Ch = Chunks<M>;
  constexpr bool F8 = M == kFp8, F32 = M == kF32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Ctl& c = *reinterpret_cast<Ctl*>(sm + kRegion);
  const KwParams& p = tp.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort = &c.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return warp_wait(bar, parity, abort, &g_kw_timeouts);
  };

  if (tid == 0) {
    for (int i = 0; i < kMaxK; ++i) {
      mbar_init(&c.k_full[i], 1);
      mbar_init(&c.k_empty[i], 1);
    }
    for (int i = 0; i < kMaxQ; ++i) {
      mbar_init(&c.q_full[i], 1);
      mbar_init(&c.q_empty[i], 1);
    }
    mbar_init(&c.r_full, 1);
    mbar_init(&c.seg_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.s_empty[i], 16);  // 8 epilogue warps x 2 CTAs
      mbar_init(&c.i_full[i], 1);
      mbar_init(&c.i_empty[i], 8);
    }
    mbar_init(&c.drain, 1);
    c.abort = 0;
    c.start_b = p.B;
    c.start_tile = 0;
    c.start_off = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                 ::"r"(smem_u32(&c.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }

  // This pair's range: thread t adds up requests [t q, (t + 1) q), a warp scans
  // the threads' sums, and the thread whose part holds the range's start finds it.
  {
    long long* scan = reinterpret_cast<long long*>(reinterpret_cast<uint8_t*>(&c) + kScanAt);
    static_assert(sizeof(Ctl) - kScanAt >= kThreads * sizeof(long long), "scan space");
    const int q = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * q), b1 = min(p.B, b0 + q);
    auto tiles_cost = [&](const KwRequest& rq, int* tiles) {
      Shape<M> sh;
      sh.set(rq.nodes * p.H);
      const int parts = tile_parts(p.splits, sh.blocks);
      *tiles = part_count(rq.kv_len, parts);
      return part_cost(sh, parts);
    };
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const KwRequest rq = kw_request(p, b);
      int tiles;
      if (rq.ok) {
        const int cost = tiles_cost(rq, &tiles);
        sum += (long long)tiles * cost;
      }
      if ((!rq.ok || rq.bad_accept) && blockIdx.x == 0 && p.req_status)
        p.req_status[b] = VA_ERR_INVALID_ARG;
    }
    scan[tid] = sum;
    __syncthreads();
    if (warp == 0) {
      constexpr int kPer = (kThreads + 31) / 32;
      long long mine = 0;
      for (int i = lane * kPer; i < min(kThreads, (lane + 1) * kPer); ++i) mine += scan[i];
      long long x = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      const long long total = __shfl_sync(0xffffffffu, x, 31);
      long long at = x - mine;
      for (int i = lane * kPer; i < min(kThreads, (lane + 1) * kPer); ++i) {
        const long long s = scan[i];
        scan[i] = at;
        at += s;
      }
      if (lane == 0) {
        c.lo = total * pair / pairs;
        c.hi = total * (pair + 1) / pairs;
      }
    }
    __syncthreads();
    const long long lo = c.lo;
    long long off = scan[tid];
    if (lo >= off && lo < off + sum) {
      for (int b = b0; b < b1; ++b) {
        const KwRequest rq = kw_request(p, b);
        if (!rq.ok) continue;
        int tiles;
        const int cost = tiles_cost(rq, &tiles);
        if (lo >= off + (long long)tiles * cost) {
          off += (long long)tiles * cost;
          continue;
        }
        const int t = (int)((lo - off + cost - 1) / cost);  // first tile from lo on
        c.start_b = t < tiles ? b : b + 1;
        c.start_tile = t < tiles ? t : 0;
        c.start_off = off + (long long)t * cost;
        break;
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  cluster_sync_all();
  fence_after();
  const uint32_t tmem = c.tmem;
  Walk<M> w;
  w.start(p, c);
  // Every role that touches the region begins a request's tiles alike: it waits
  // until the pair's last request there is multiplied, for its layout goes.
  int held = -1;
  uint32_t seg_parity = 1;
  auto new_request = [&](bool& go) {
    if (held == w.b) return false;
    held = w.b;
    go = wait(&c.seg_done, seg_parity);
    seg_parity ^= 1;
    return true;
  };

  if (warp == kWarpK) {
    // ------------------------------------------------------------- key chunks by TMA
    bool go = true;
    Ring ring;
    const int oob = (F32 ? p.B * p.max_pages : p.num_pages) * kPage;  // past the pool: zeros
    for (; w.alive() && go; w.next()) {
      if (new_request(go)) ring.restart(w.sh.k_slots());
      const int key = w.at * kTileKeys + (int)rank * 128;
      int r0, r1;
      if (F32) {  // laid out by request and slot
        const long long at = ((long long)w.b * p.max_pages) * kPage + key;
        r0 = key < w.kv_len ? (int)at : oob;
        r1 = key + kPage < w.kv_len ? (int)at + kPage : oob;
      } else {
        r0 = kw_pool_row(p, w.b, w.kv_len, key);
        r1 = kw_pool_row(p, w.b, w.kv_len, key + kPage);
        r0 = r0 < 0 ? oob : r0;
        r1 = r1 < 0 ? oob : r1;
      }
      for (int rb = F32 ? w.rb0 : w.rb1 - 1; rb < w.rb1 && go; ++rb) {
        for (int kc = 0; kc < Ch::n && go; ++kc) {
          const int s = ring.slot;
          go = wait(&c.k_empty[s], ring.phase() ^ 1);
          if (!go) break;
          if (elect_one()) {
            const bool pe = kc == Ch::n - 1;
            const CUtensorMap* map = pe ? &tm_kpe : &tm_ckv;
            const int bytes = 128 * Ch::width(kc);
            const uint32_t bar = map_to_rank(smem_u32(&c.k_full[s]), 0);
            if (rank == 0) arrive_expect_tx(&c.k_full[s], 2 * bytes * Ch::k_planes);
            uint32_t dst = smem_u32(sm + w.sh.k_at() + s * Ch::k_slot);
            int x = pe ? 0 : kc * (F8 ? 128 : 64);
            for (int pl = 0; pl < Ch::k_planes; ++pl) {
              tma_2d(dst, map, bar, x, r0);
              tma_2d(dst + bytes / 2, map, bar, x, r1);
              dst += kKSlot;
              x += pe ? kDr : kDc;
            }
          }
          __syncwarp();
          ring.advance();
        }
      }
    }
    // the last use of every slot must be over before the CTA may exit
    for (int s = 0; s < kMaxK && go; ++s) go = wait(&c.k_empty[s], ((ring.used >> s) & 1u) ^ 1);
    if (go) wait(&c.seg_done, seg_parity);
    if (*abort) settle();
  } else if (warp == kWarpQ) {
    // ------------------------------------------------------------ query rows by TMA
    bool go = true;
    Ring ring;
    const long long rows_total = (long long)p.B * p.T * p.H;
    // first map row of a box from row r of the request on
    auto map_row = [&](int r) -> int {
      if (tp.dense) return (int)((long long)w.b * p.T * p.H + r);
      if (r >= w.R) return (int)rows_total;
      const int i = r / p.H;
      const int n = p.path ? p.path[(size_t)w.b * p.T + i] : i;
      if (n < 0 || n >= p.T) return (int)rows_total;
      return (int)(((long long)w.b * p.T + n) * p.H + (r - i * p.H));
    };
    for (; w.alive() && go; w.next()) {
      const bool fresh = new_request(go);
      if (!go || (!fresh && w.sh.stay)) continue;
      if (fresh) ring.restart(!w.sh.stay ? w.sh.q_slots() : 1);
      const int half = w.sh.cols / 2;
      int box = kBoxes - 1;  // the tallest box that fits the half and the run
      while (box > 0 && ((half | tp.run) & ((8 << box) - 1))) --box;
      const int box_rows = 8 << box;
      const bool mine = lane < half / box_rows;
      // this lane's boxes of a chunk, one a plane
      auto boxes = [&](int kc, uint8_t* at, uint32_t bar, int y) {
        const bool pe = kc == Ch::n - 1;
        const int wide = Ch::width(kc), e = F8 ? 1 : 2;
        for (int pl = 0; pl < Ch::planes; ++pl)
          tma_2d(smem_u32(at + (pl * half + lane * box_rows) * wide),
                 pe ? &tm_q.pe[box] : &tm_q.nope[box], bar,
                 pl * (pe ? kDr : kDc) + (pe ? 0 : kc * (128 / e)), y);
      };
      if (w.sh.stay) {  // all chunks at once
        if (lane == 0 && rank == 0) arrive_expect_tx(&c.r_full, 2 * w.sh.rows_stay());
        __syncwarp();
        const uint32_t bar = map_to_rank(smem_u32(&c.r_full), 0);
        if (mine) {
          const int y = map_row((int)rank * half + lane * box_rows);
          for (int kc = 0; kc < Ch::n; ++kc) boxes(kc, sm + w.sh.q_at() + kc * w.sh.q_slot(), bar, y);
        }
        __syncwarp();
        continue;
      }
      for (int rb = w.rb0; rb < w.rb1 && go; ++rb) {
        const int y = mine ? map_row(rb * w.sh.cols + (int)rank * half + lane * box_rows) : 0;
        for (int kc = 0; kc < Ch::n && go; ++kc) {
          const int s = ring.slot;
          go = wait(&c.q_empty[s], ring.phase() ^ 1);
          if (!go) break;
          if (lane == 0 && rank == 0)
            arrive_expect_tx(&c.q_full[s], w.sh.cols * Ch::planes * Ch::width(kc));
          __syncwarp();
          if (mine)
            boxes(kc, sm + w.sh.q_at() + s * w.sh.q_slot(), map_to_rank(smem_u32(&c.q_full[s]), 0), y);
          __syncwarp();
          ring.advance();
        }
      }
    }
    for (int s = 0; s < kMaxQ && go; ++s) go = wait(&c.q_empty[s], ((ring.used >> s) & 1u) ^ 1);
    if (go) wait(&c.seg_done, seg_parity);
    if (*abort) settle();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ MMA issue
    if (rank == 0) {
      bool ok = !tp.stall;
      Ring kring, qring;
      uint32_t rphase = 0, pass = 0;
      for (; w.alive() && ok; w.next()) {
        const bool stream = !w.sh.stay;
        if (held != w.b) {
          held = w.b;
          kring.restart(w.sh.k_slots());
          qring.restart(stream ? w.sh.q_slots() : 1);
          if (!stream) {
            ok = wait(&c.r_full, rphase);
            rphase ^= 1;
          }
        }
        // fp32 sums; K-major A and B: bf16 (1, 1) of kind::f16, or E4M3 (0) and E5M2 (1)
        // of kind::f8f6f4; M = 256
        const uint32_t idesc = (1u << 4) | (F8 ? 0u : 1u << 7) | (1u << 10) |
                               ((uint32_t)(w.sh.cols >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
        const uint32_t k0 = smem_u32(sm + w.sh.k_at()), q0 = smem_u32(sm + w.sh.q_at());
        const int q_slot = w.sh.q_slot(), half = w.sh.cols / 2;
        const bool seg_end = w.last_of_request();
        const Ring first = kring;  // the tile's first chunk: every block begins there
        for (int rb = w.rb0; rb < w.rb1 && ok; ++rb, ++pass) {
          const uint32_t d = tmem + (pass & 1) * 256;
          const bool last = rb == w.rb1 - 1;
          if (rb > w.rb0 && !F32) kring = first;
          ok = wait(&c.s_empty[pass & 1], ((pass >> 1) & 1) ^ 1);
          for (int kc = 0; kc < Ch::n && ok; ++kc) {
            const int ks = kring.slot, qs = qring.slot;
            if (rb == w.rb0 || F32) ok = wait(&c.k_full[ks], kring.phase());
            if (ok && stream) ok = wait(&c.q_full[qs], qring.phase());
            if (!ok) break;
            if (elect_one()) {
              fence_after();
              const uint32_t ka = k0 + ks * Ch::k_slot, qa = q0 + (stream ? qs : kc) * q_slot;
              if (F32) {
                // planes (0, 0) to d; (0, 1), (1, 0), (0, 2), (1, 1), (2, 0) beside it
#pragma unroll 1
                for (int i = 0; i < 6; ++i) {
                  const int pa = (0x210100 >> (4 * i)) & 3, pb = (0x012010 >> (4 * i)) & 3;
                  const uint64_t a = sw128_desc(ka + pa * kKSlot), b = sw128_desc(qa + pb * half * 128);
                  const uint32_t to = i ? d + 128 : d;
                  mma_pair(to, a, b, idesc, kc != 0 || i > 1);
                  mma_pair(to, a + 2, b + 2, idesc, 1u);
                  mma_pair(to, a + 4, b + 4, idesc, 1u);
                  mma_pair(to, a + 6, b + 6, idesc, 1u);
                }
              } else if (!F8) {
                const uint64_t a = sw128_desc(ka), b = sw128_desc(qa);
                mma_pair(d, a, b, idesc, kc != 0);
                mma_pair(d, a + 2, b + 2, idesc, 1u);
                mma_pair(d, a + 4, b + 4, idesc, 1u);
                mma_pair(d, a + 6, b + 6, idesc, 1u);
              } else {
                const bool pe = kc == Ch::n - 1;
                const uint64_t a = pe ? sw64_desc(ka) : sw128_desc(ka);
#pragma unroll 1
                for (int pl = 0; pl < Ch::planes; ++pl) {
                  const uint32_t at = qa + pl * half * (pe ? 64 : 128);
                  const uint64_t b = pe ? sw64_desc(at) : sw128_desc(at);
                  mma_pair_f8(d, a, b, idesc, kc + pl != 0);
                  mma_pair_f8(d, a + 2, b + 2, idesc, 1u);
                  if (!pe) {
                    mma_pair_f8(d, a + 4, b + 4, idesc, 1u);
                    mma_pair_f8(d, a + 6, b + 6, idesc, 1u);
                  }
                }
              }
              if (stream) commit_pair(&c.q_empty[qs]);
              if (last || F32) commit_pair(&c.k_empty[ks]);
              if (kc == Ch::n - 1) {
                commit_pair(&c.s_full[pass & 1]);
                if (last && seg_end) commit_pair(&c.seg_done);
              }
            }
            __syncwarp();
            kring.advance();
            if (stream) qring.advance();
          }
        }
      }
      if (!ok) {  // let every MMA already issued finish before tensor memory is freed
        if (elect_one()) commit_pair(&c.drain);
        __syncwarp();
        final_wait(&c.drain, 0);
      }
    }
  } else if (warp >= kWarpInfo) {
    // ------------------------------------------------------- column data of each pass
    // Ahead of the epilogue, so that their loads are off its path; two warps take
    // turns.
    const int W = (p.T + 63) >> 6;
    uint32_t pass = 0;
    bool go = true;
    for (; w.alive() && go; w.next()) {
      for (int rb = w.rb0; rb < w.rb1 && go; ++rb, ++pass) {
        const int buf = pass & 1;
        if (buf != warp - kWarpInfo) continue;
        bool free = false;
#pragma unroll 1
        for (int k0 = 0; k0 * 32 < w.sh.cols && go; k0 += 4) {
          float l[4], f[4];
          uint64_t word[4];
          int node[4];
          bool ok[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = (k0 + k) * 32 + lane, r = rb * w.sh.cols + e;
            const bool in = r < w.R && e < w.sh.cols;
            const int i = in ? r / p.H : 0;
            const int n = in && p.path ? p.path[(size_t)w.b * p.T + i] : i;
            ok[k] = in && n >= 0 && n < p.T;
            if (in && !ok[k] && p.req_status) p.req_status[w.b] = VA_ERR_INVALID_ARG;
            node[k] = ok[k] ? n : 0;
            const size_t row = (size_t)w.b * p.T + node[k];
            word[k] = p.tree_mask[row * W + (node[k] >> 6)];
            l[k] = p.lse[ok[k] ? row * p.H + (r - i * p.H) : 0];
            f[k] = F8 && ok[k] ? tp.q_scale[(size_t)w.b * p.T * p.H + r] : 0.f;
          }
          if (!free) go = wait(&c.i_empty[buf], ((pass >> 1) & 1) ^ 1);
          free = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool adds = ok[k] && ((word[k] >> (node[k] & 63)) & 1ull) && l[k] != -INFINITY;
            const int e = (k0 + k) * 32 + lane;
            c.node[buf][e] = (uint8_t)node[k];
            c.lse[buf][e] = l[k];
            if (F8) c.factor[buf][e] = adds ? f[k] * tp.scale : 0.f;
            const uint32_t on = __ballot_sync(0xffffffffu, adds);
            const int first = __shfl_sync(0xffffffffu, node[k], on ? __ffs(on) - 1 : 0);
            const bool same = __all_sync(0xffffffffu, !adds || node[k] == first);
            if (lane == 0) {
              c.none[buf][k0 + k] = ~on;
              c.one[buf][k0 + k] = same ? first : -1;
            }
          }
        }
        __syncwarp();
        if (lane == 0) arrive(&c.i_full[buf]);
      }
    }
  } else if (warp >= kWarpEpi && warp < kWarpQ) {
    // ----------------------------------------------------------- exponentials, sums
    // Warp w reads lane quadrant w & 3 (keys 32 (w & 3) .. of this CTA); the two
    // warps of a quadrant take the two halves of a pass's columns.
    const int q = warp & 3, half = (warp - kWarpEpi) >> 2, m = 32 * q + lane;
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    const uint32_t free0 = map_to_rank(smem_u32(&c.s_empty[0]), 0);
    const float factor = tp.scale;
    const int W = (p.T + 63) >> 6;
    uint32_t pass = 0, tile_no = 0;
    for (; w.alive(); w.next(), ++tile_no) {
      const int key = w.at * kTileKeys + (int)rank * 128 + m;
      const int krow = half == 0 ? kw_pool_row(p, w.b, w.kv_len, key) : 0;
      const size_t slot = (size_t)w.b * p.max_pages * kPage + key;
      const float old =
          half == 0 && p.splits == 1 && p.weights_in && key < w.kv_len ? p.weights_in[slot] : 0.f;
      const int P = w.kv_len - p.T;
      // a tail key is seen by some nodes only: bit n of (seen0, seen1) for node n
      const bool tail =  // of the warp
          w.at * kTileKeys + (int)rank * 128 + 32 * q + 32 > P;
      const int nd = key - P;
      uint64_t seen0 = ~0ull, seen1 = ~0ull;
      if (tail && nd >= 0) {
        const uint64_t* mask = p.tree_mask + (size_t)w.b * p.T * W + (nd < p.T ? nd >> 6 : 0);
        seen0 = seen1 = 0;
#pragma unroll 8
        for (int n = 0; n < p.T; ++n) {
          const uint64_t bit = nd < p.T ? (mask[n * W] >> (nd & 63)) & 1ull : 0ull;
          if (n < 64) seen0 |= bit << n; else seen1 |= bit << (n - 64);
        }
      }
      auto sees = [&](int n) -> uint32_t {
        return (uint32_t)((n < 64 ? seen0 >> n : seen1 >> (n - 64)) & 1ull);
      };
      const int cols = w.sh.cols / 2, c0 = half * cols;  // this half's: a multiple of 32
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int rb = w.rb0; rb < w.rb1; ++rb, ++pass) {
        const int buf = pass & 1;
        const uint32_t parity = (pass >> 1) & 1;
        wait(&c.i_full[buf], parity);
        wait(&c.s_full[buf], parity);
        fence_after();
        const uint32_t scores = tmem + lane_base + buf * 256 + c0;
        // One body for all groups, and small: the roles' loops share the instruction
        // cache, and with three unrolled copies of this one a quarter of all stalls
        // were waits for instructions.
#pragma unroll 1
        for (int g = 0; g < cols; g += 32) {
          float x[32];
          ld32(scores + g, x);
          if (F32) {
            float y[32];
            ld32(scores + 128 + g, y);
            wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] += y[i];
          } else {
            wait_ld();
          }
          if (g + 32 == cols) {  // all scores are in registers: the buffer may be written again
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(free0 + buf * 8);
          }
          const int at = c0 + g;
          uint32_t off = c.none[buf][at >> 5];  // columns that add nothing to this key
          if (tail) {
            const int n = c.one[buf][at >> 5];
            if (n >= 0) {  // as with 32 heads and more
              if (!sees(n)) off = ~0u;
            } else {
#pragma unroll 1
              for (int i = 0; i < 32; ++i) off |= (sees(c.node[buf][at + i]) ^ 1u) << i;
            }
          }
          const float* ls = &c.lse[buf][at];
          const float* fc = &c.factor[buf][at];
          // scale s - lse first: small where the weight is large, and so its rounding
          auto prob = [&](float s, int i) {
            return ex2f(fmaf(s, F8 ? fc[i] : factor, -ls[i]) * kLog2e);
          };
          if (__any_sync(0xffffffffu, off != 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float v = prob(x[i], i);
              sum[i & 3] += (off >> i) & 1u ? 0.f : v;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sum[i & 3] += prob(x[i], i);
          }
        }
        __syncwarp();
        if (lane == 0) arrive(&c.i_empty[buf]);
      }
      // the two halves of a key meet in shared memory (the quadrant's 64 threads)
      const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (half == 1) c.xsum[tile_no & 1][m] = s;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
      if (half == 0 && key < w.kv_len) {
        const float all = krow >= 0 ? s + c.xsum[tile_no & 1][m] : 0.f;
        if (p.splits == 1) p.weights[slot] = p.decay * old + all;
        else p.part[(size_t)w.part * p.B * p.max_pages * kPage + slot] = all;
        if (krow < 0 && p.req_status) p.req_status[w.b] = VA_ERR_INVALID_ARG;
        if (*abort && p.req_status) p.req_status[w.b] = VA_ERR_CUDA;
      }
    }
  }

  __syncwarp();
  fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == kWarpMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// x as the sum of three bf16 (what is left of it after two has 8 bits); the first is
// rounded toward zero where the nearest would be an infinity that x is not.
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&o)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    o[i] = __float2bfloat16_rn(x);
    if (i == 0 && __hisinf(o[0])) o[0] = __float2bfloat16_rz(x);
    x -= __bfloat162float(o[i]);
  }
}
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_fp8_e4m3* p, float (&x)[4]) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(__half2(
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v >> (16 * i)), __NV_E4M3)));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
// One warp writes a row's planes: [3][512] at row `to` of n, [3][64] of pe.
template <typename T>
__device__ __forceinline__ void split_row(const T* nope, const T* rope, size_t to, void* n, void* pe) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 5; ++i) {  // four elements a lane
    if (i == 4 && lane >= 16) break;
    float x[4];
    load4(i < 4 ? nope + (i * 32 + lane) * 4 : rope + lane * 4, x);
    __nv_bfloat16 o[4][3];
#pragma unroll
    for (int k = 0; k < 4; ++k) split3(x[k], o[k]);
    uint2* dst = i < 4 ? reinterpret_cast<uint2*>(n) + to * (3 * kDc / 4) + i * 32 + lane
                       : reinterpret_cast<uint2*>(pe) + to * (3 * kDr / 4) + lane;
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) {
      __nv_bfloat162 lo(o[0][pl], o[1][pl]), hi(o[2][pl], o[3][pl]);
      dst[pl * (i < 4 ? kDc / 4 : kDr / 4)] =
          make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    }
  }
}

// The requests' cached keys as planes of three bf16: slot j of request b is row
// (b max_pages) 64 + j.  One warp per key; keys of pages outside the pool are left out.
template <typename T>
__global__ void __launch_bounds__(256)
kweights_keys_kernel(const KwParams p, void* __restrict__ n, void* __restrict__ pe) {
  const int b = blockIdx.y, key = blockIdx.x * 8 + (threadIdx.x >> 5);
  const KwRequest rq = kw_request(p, b);
  const int row = rq.ok ? kw_pool_row(p, b, rq.kv_len, key) : -1;
  if (row < 0) return;
  split_row(reinterpret_cast<const T*>(p.c_kv) + (size_t)row * kDc,
            reinterpret_cast<const T*>(p.k_pe) + (size_t)row * kDr,
            (size_t)b * p.max_pages * kPage + key, n, pe);
}

// Counted rows of every request, dense from b * T * H on.  For an FP8 cache each
// row is multiplied by the power of two that brings its largest element to [2^14,
// 2^15), and an element x is written as the E5M2 numbers nearest to x, to what is
// left of it, and to what is left then: planes [3][512] and [3][64] of a row;
// `scale` gets the inverse power.  One warp per row.
template <int M>
__global__ void __launch_bounds__(256)
kweights_rows_kernel(const KwParams p, uint4* __restrict__ qn, uint4* __restrict__ qp,
                     float* __restrict__ scale) {
  constexpr bool F8 = M == kFp8;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  const KwRequest rq = kw_request(p, b);
  if (!rq.ok || r >= rq.nodes * p.H) return;
  int node;
  const int g = kw_query_row(p, b, rq, r, &node);
  if (g < 0) return;
  const size_t to = (size_t)b * p.T * p.H + r;
  if (M == kF32) {
    split_row(reinterpret_cast<const float*>(p.q_nope) + (size_t)g * kDc,
              reinterpret_cast<const float*>(p.q_pe) + (size_t)g * kDr, to, qn, qp);
    return;
  }
  const uint4* sn = reinterpret_cast<const uint4*>(p.q_nope) + (size_t)g * (kDc / 8);
  const uint4* sp = reinterpret_cast<const uint4*>(p.q_pe) + (size_t)g * (kDr / 8);
  uint4 v[3];  // 8 elements each: of q_nope from 8 lane and 256 + 8 lane on, of q_pe from 8 lane
  v[0] = sn[lane];
  v[1] = sn[lane + 32];
  v[2] = lane < 8 ? sp[lane] : make_uint4(0, 0, 0, 0);
  if (!F8) {
    qn[to * (kDc / 8) + lane] = v[0];
    qn[to * (kDc / 8) + lane + 32] = v[1];
    if (lane < 8) qp[to * (kDr / 8) + lane] = v[2];
    return;
  }
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      big = fmaxf(big, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u))));
  }
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
  // exponent of 2 to multiply by; zero and non-finite rows stay as they are
  int ex = 0;
  if (big > 0.f && big < INFINITY) ex = min(14 - ilogbf(big), 120);
  const float up = ldexpf(1.f, ex);
  uint2* n8 = reinterpret_cast<uint2*>(qn) + to * (3 * kDc / 8);
  uint2* p8 = reinterpret_cast<uint2*>(qp) + to * (3 * kDr / 8);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i == 2 && lane >= 8) break;
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint64_t plane[3] = {0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float x = __uint_as_float(k & 1 ? u[k >> 1] & 0xffff0000u : u[k >> 1] << 16) * up;
      const bool finite = fabsf(x) < INFINITY;
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        __nv_fp8_storage_t q = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E5M2);
        x -= __half2float(__half(__nv_cvt_fp8_to_halfraw(q, __NV_E5M2)));
        if (!finite) q = pl == 0 ? 0x7f : 0;  // NaN: the row's scores come out as NaN
        plane[pl] |= (uint64_t)q << (8 * k);
      }
    }
#pragma unroll
    for (int pl = 0; pl < 3; ++pl) {
      const uint2 o = make_uint2((uint32_t)plane[pl], (uint32_t)(plane[pl] >> 32));
      if (i < 2) n8[pl * (kDc / 8) + i * 32 + lane] = o;
      else p8[pl * (kDr / 8) + lane] = o;
    }
  }
  if (lane == 0) scale[to] = ldexpf(1.f, -ex);
}

int mode_of(const va_key_weight_args& a) {
  return a.dtype == VA_F32 ? kF32 : (a.flags & VA_FLAG_KV_FP8_E4M3) ? kFp8 : kBf16;
}
struct Layout {
  size_t qn, qp, scale, kn, kp, total;
};
// Counted rows are laid out densely first when they need converting, or when the
// accepted nodes' runs of H rows are no whole number of 8-row swizzle groups; fp32
// keys too, for the pages that the page table can hold.
bool needs_rows(const va_key_weight_args& a) {
  return mode_of(a) != kBf16 || (a.path && a.H % 8 != 0);
}
Layout layout(const va_key_weight_args& a) {
  const int m = mode_of(a);
  const size_t rows = needs_rows(a) ? (size_t)a.B * a.T * a.H : 0;
  const size_t keys = m == kF32 ? (size_t)a.B * a.max_pages * kPage : 0;
  const int bytes = m == kFp8 ? 3 : m == kF32 ? 6 : 2;
  Layout l;
  l.qn = 0;
  l.qp = align256(rows * kDc * bytes);
  l.scale = l.qp + align256(rows * kDr * bytes);
  l.kn = l.scale + (m == kFp8 ? align256(rows * sizeof(float)) : 0);
  l.kp = l.kn + align256(keys * kDc * 6);
  l.total = l.kp + align256(keys * kDr * 6);
  return l;
}
// Rows of a request as the host sees them: an accepted path of the deepest tree at most.
long long rows_seen(const va_key_weight_args& a) {
  const long long nodes = a.path && a.T > VA_MAX_DEPTH + 1 ? VA_MAX_DEPTH + 1 : a.T;
  return nodes * a.H;
}
long long tiles_of(const va_key_weight_args& a) {
  return (long long)a.B * (((long long)a.max_pages * kPage + kTileKeys - 1) / kTileKeys);
}

template <int M>
cudaError_t launch(const QMaps& tq, const CUtensorMap& tckv, const CUtensorMap& tkpe,
                   const TcParams& tp, int pairs, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = raise_smem_once(kweights_tc_kernel<M>, (int)kSmemBytes, done);
  if (e != cudaSuccess) return e;
  kweights_tc_kernel<M><<<2 * pairs, kThreads, kSmemBytes, st>>>(tq, tckv, tkpe, tp);
  return cudaGetLastError();
}

}  // namespace

// Calls run here unless the caller asks for CUDA cores, or fp32 keys' planes (3456
// bytes each) would take over 1 GB of workspace.  One tile of 128 x 128 takes the
// CUDA cores about 65 us; a small fp32 call here takes 19 to 27 with its launches.
bool kweights_on_tc(const va_key_weight_args& a) {
  if (a.flags & VA_FLAG_BF16_CUDA_CORES) return false;
  const long long keys = (long long)a.B * a.max_pages * kPage;
  return a.dtype == VA_BF16 || keys * 6 * kDqk <= (1LL << 30);
}

int kweights_tc_splits(const va_key_weight_args& a, int sms) {
  return plan_splits(mode_of(a), rows_seen(a), tiles_of(a), sms / 2);
}
void kweights_tc_blocks(const va_key_weight_args& a, int* stay, int* pass) {
  block_rows(mode_of(a), stay, pass);
}

size_t kweights_tc_workspace(const va_key_weight_args& a) { return layout(a).total; }

cudaError_t launch_kweights_tc(const va_key_weight_args& a, const KwParams& p, int sms,
                               cudaStream_t st) {
  const int m = mode_of(a);
  const bool f8 = m == kFp8;
  const uint64_t rows = (uint64_t)a.B * a.T * a.H;
  TcParams tp;
  tp.k = p;
  tp.dense = needs_rows(a);
  tp.run = tp.dense || !a.path ? 64 : a.H;
  tp.q_scale = nullptr;
  const bool codes = a.flags & VA_FLAG_KV_FP8_E4M3;
  tp.scale = (float)((double)p.scale *
                     (1.0 + (!codes ? kShortBf16 : m == kF32 ? kShortF32Fp8 : kShortFp8)));
  tp.stall = (a.flags & VA_FLAG_TEST_STALL_KEY_WEIGHTS) ? 1 : 0;
  const Layout l = layout(a);
  char* ws = static_cast<char*>(a.workspace);
  const void* qn = a.q_nope;
  const void* qp = a.q_pe;
  if (tp.dense) {
    qn = ws + l.qn;
    qp = ws + l.qp;
    float* scale = f8 ? reinterpret_cast<float*>(ws + l.scale) : nullptr;
    tp.q_scale = scale;
    const dim3 grid((unsigned)((a.T * a.H + 7) / 8), (unsigned)a.B);
    auto* k = f8 ? kweights_rows_kernel<kFp8>
                 : m == kF32 ? kweights_rows_kernel<kF32> : kweights_rows_kernel<kBf16>;
    k<<<grid, 256, 0, st>>>(p, (uint4*)qn, (uint4*)qp, scale);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const void* ckv = a.c_kv;
  const void* kpe = a.k_pe;
  uint64_t pool = (uint64_t)a.num_pages * kPage;
  if (m == kF32) {
    ckv = ws + l.kn;
    kpe = ws + l.kp;
    pool = (uint64_t)a.B * a.max_pages * kPage;
    const dim3 grid((unsigned)(a.max_pages * (kPage / 8)), (unsigned)a.B);
    auto* k = (a.flags & VA_FLAG_KV_FP8_E4M3) ? kweights_keys_kernel<__nv_fp8_e4m3>
                                              : kweights_keys_kernel<float>;
    k<<<grid, 256, 0, st>>>(p, ws + l.kn, ws + l.kp);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  QMaps tq = {};
  CUtensorMap tckv, tkpe;
  const int qe = f8 ? 3 : m == kF32 ? 6 : 2, ke = f8 ? 1 : m == kF32 ? 6 : 2;
  // the boxes that halves (multiples of 32 rows) take in these runs: the run's own
  // power of two, and 32 beside 64
  int tallest = kBoxes - 1;
  while (tallest > 0 && tp.run % (8 << tallest)) --tallest;
  for (int i = tallest == kBoxes - 1 ? tallest - 1 : tallest; i <= tallest; ++i)
    if (!encode_rows(&tq.nope[i], qn, rows, kDc * qe, 8 << i, 128, f8) ||
        !encode_rows(&tq.pe[i], qp, rows, kDr * qe, 8 << i, f8 ? 64 : 128, f8))
      return cudaErrorInvalidValue;
  if (!encode_rows(&tckv, ckv, pool, kDc * ke, kPage, 128, f8) ||
      !encode_rows(&tkpe, kpe, pool, kDr * ke, kPage, f8 ? 64 : 128, f8))
    return cudaErrorInvalidValue;
  const long long parts = tiles_of(a) * p.splits;
  const int pairs = (int)(parts < sms / 2 ? parts : sms / 2);
  return f8          ? launch<kFp8>(tq, tckv, tkpe, tp, pairs, st)
         : m == kF32 ? launch<kF32>(tq, tckv, tkpe, tp, pairs, st)
                     : launch<kBf16>(tq, tckv, tkpe, tp, pairs, st);
}

unsigned int kw_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kw_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

}  // namespace va
