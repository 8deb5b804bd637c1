// Key weights on tensor cores (bf16 queries; bf16 or FP8 cache), sm_100a.
//
//   w_j = sum over counted rows r, j visible to r, of
//         exp(scale q_r . k_j - lse_r)
// The keys are the M side of the product and the rows the N side: a CTA pair
// (tcgen05.mma.cta_group::2, M = 256) takes a tile of 256 keys, 128 a CTA,
// and up to 256 rows at a time.  In tensor memory a key is then a lane and a
// row a column, so a thread adds its key's exponentials over the columns in
// a register, and nothing is exchanged between threads but the two halves
// of a tile's columns.  No partial sums leave the SM.
//
// A request's tiles are walked in one of two layouts of shared memory.  Few rows
// (at most 160) are loaded once per pair and request and stay, and the tiles'
// keys come through a ring of 16 KB chunks (128 keys x 64 dims).  More rows: a
// tile's 9 key chunks stay while the rows pass by through a ring, in equal
// blocks.  Either way each key is read from HBM once.  The tiles of
// all requests, in order and weighted by what they cost, are divided into
// equal contiguous ranges, one per pair.
//
// FP8 cache: the codes come through a ring of their own, and converter warps
// write them as fp16, which holds every E4M3 value; the queries are multiplied
// by a power of two per row and stored as fp16 by a first kernel (exact down
// to 2^-39 of the row's largest element), and the epilogue undoes it in fp32.
//
// Bound by HBM for few rows (1152 or 576 bytes a key) and by the tensor cores
// for many (128 clocks per 256 x 256 x 16), with the latency of the rings'
// loads close behind (about 2200 clocks from a slot's release to its refill);
// the exponentials take 16 a clock and SM.
#include "va_kweights.cuh"
#include "va_tc_ops.cuh"

namespace va {

__device__ unsigned int g_kw_timeouts = 0;  // count of barrier waits that expired

namespace {

using namespace tc;

constexpr int kTileKeys = 256;       // of the pair
constexpr int kChunks = 9;           // 64-dim chunks of a row: 8 of c_kv, 1 of k_pe
constexpr int kKChunk = 128 * 128;   // bytes: 128 keys x 64 dims
constexpr int kMaxK = 12, kMaxQ = 8; // ring slots, at most (codes: kMaxRaw = kMaxK)
constexpr int kRegion = kChunks * kKChunk + kChunks * 64 * 128;  // keys and rows: 216 KB
constexpr int kMaxRaw = 12, kRawSlot = 128 * 64;  // FP8 codes: 128 keys x 64 dims
constexpr int kWarpK = 0, kWarpMma = 1, kWarpEpi = 2, kWarpQ = 10, kWarpInfo = 11;
constexpr int kConvWarps = 8, kConvTeams = 4;  // a team converts every 4th chunk
// Warps of column data: two for a bf16 cache, whose passes may be short; with an
// FP8 cache one, which leaves 96 registers a thread beside the converters.
template <bool F8> constexpr int kInfoWarps = F8 ? 1 : 2;
template <bool F8> constexpr int kWarpConv = kWarpInfo + kInfoWarps<F8>;
template <bool F8> constexpr int kWarps = kWarpConv<F8> + (F8 ? kConvWarps : 0);

struct TcParams {
  KwParams k;
  int dense;             // rows of request b start at b * T * H of the q maps
  int run;               // rows that lie in order from a multiple of it on
  const float* q_scale;  // FP8 cache: [B, T H] power of two that undoes the row's
};

constexpr int kBoxes = 4;  // query boxes of 8, 16, 32 or 64 rows
struct QMaps {
  CUtensorMap nope[kBoxes], pe[kBoxes];
};

struct __align__(16) Ctl {
  uint64_t k_full[kMaxK], k_empty[kMaxK];
  uint64_t q_full[kMaxQ], q_empty[kMaxQ];
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t r_full;                 // rows that stay
  uint64_t seg_done;               // a request's last tile of this pair is multiplied
  uint64_t s_full[2], s_empty[2];  // scores in tensor memory
  uint64_t i_full[2], i_empty[2];  // column data of a pass
  uint64_t drain;
  long long start_off, lo, hi;
  int start_b, start_tile;
  uint32_t tmem;
  int abort;
  // of each column of a pass: its node, its row's log2-sum and factor; one bit
  // where the column adds nothing (no row, absent node, empty row); and the
  // node of all that a group of 32 columns adds (-1: several)
  uint32_t none[2][8];
  int one[2][8];
  float xsum[2][128];
  uint8_t node[2][256];
  __align__(16) float l2[2][256];
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

// How the rows of a request are multiplied: `blocks` passes of `cols` columns.
// Up to kStay rows stay in shared memory: with more, fewer than 7 key chunks
// would be in flight beside them, which HBM's latency needs (4 slots beside 256
// rows took 8000 clocks a tile, rows through the ring 5000).  With an FP8 cache
// it is the codes that HBM's latency holds up: their ring gets the room, and 4
// slots do for the key chunks on their way from the converters.
template <bool F8>
struct Shape {
  static constexpr int kStay = F8 ? 192 : 160, kPass = F8 ? 128 : 256;
  static constexpr int kConvRing = 4 * kKChunk, kRawBeside = 5;
  int blocks, cols;
  bool stay;
  __device__ __forceinline__ void set(int R) {
    stay = R <= kStay;
    blocks = stay ? 1 : (R + kPass - 1) / kPass;
    cols = max(64, ((R + blocks - 1) / blocks + 63) & ~63);
  }
  // ring slots, and where keys, rows and codes lie in the region
  __device__ __forceinline__ int rows_stay() const { return kChunks * cols * 64; }
  __device__ __forceinline__ int k_slots() const {
    return !stay ? kChunks : F8 ? 4 : min(kMaxK, (kRegion - rows_stay()) / kKChunk);
  }
  __device__ __forceinline__ int k_at() const { return stay ? rows_stay() : 0; }
  __device__ __forceinline__ int q_slots() const {
    return min(kMaxQ, (kRegion - kChunks * kKChunk - (F8 ? kRawBeside * kRawSlot : 0)) / (cols * 64));
  }
  __device__ __forceinline__ int q_at() const { return stay ? 0 : kChunks * kKChunk; }
  __device__ __forceinline__ int raw_slots() const {
    return stay ? min(kMaxRaw, (kRegion - rows_stay() - kConvRing) / kRawSlot) : kRawBeside;
  }
  __device__ __forceinline__ int raw_at() const {
    return stay ? rows_stay() + kConvRing : kRegion - kRawBeside * kRawSlot;
  }
  // Clocks of a tile, as measured: few rows wait for the keys' share of HBM, rows
  // through the ring for its latency (5400 a pass of 192 columns, 6500 of 256).
  __device__ __forceinline__ int cost() const {
    return stay ? max(F8 ? 3400 : 5400, 18 * cols + 1000) : blocks * (2200 + 17 * cols) + 300;
  }
};

// The pair's tiles, in order.  Every warp role walks them by itself.
template <bool F8>
struct Walk {
  const KwParams* p;
  long long off, end;
  int b, tile, tiles, R, kv_len, cost;
  KwRequest rq;
  Shape<F8> sh;
  __device__ __forceinline__ void load() {
    for (; b < p->B; ++b) {
      rq = kw_request(*p, b);
      if (rq.ok) break;
    }
    if (b < p->B) {
      kv_len = rq.kv_len;
      tiles = (kv_len + kTileKeys - 1) / kTileKeys;
      R = rq.nodes * p->H;
      sh.set(R);
      cost = sh.cost();
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

template <bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWarps<F8> * 32, 1)
kweights_tc_kernel(const __grid_constant__ QMaps tm_q, const __grid_constant__ CUtensorMap tm_ckv,
                   const __grid_constant__ CUtensorMap tm_kpe, const __grid_constant__ TcParams tp) {
  constexpr int kThreads = kWarps<F8> * 32;
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
      mbar_init(&c.k_full[i], F8 ? 2 * (kConvWarps / kConvTeams) : 1);
      mbar_init(&c.k_empty[i], 1);
    }
    for (int i = 0; i < kMaxQ; ++i) {
      mbar_init(&c.q_full[i], 1);
      mbar_init(&c.q_empty[i], 1);
    }
    for (int i = 0; i < kMaxRaw; ++i) {
      mbar_init(&c.raw_full[i], 1);
      mbar_init(&c.raw_empty[i], kConvWarps / kConvTeams);
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
      Shape<F8> sh;
      sh.set(rq.nodes * p.H);
      *tiles = (rq.kv_len + kTileKeys - 1) / kTileKeys;
      return sh.cost();
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
  Walk<F8> w;
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
    // -------------------------------------------------- key chunks (or codes) by TMA
    bool go = true;
    Ring ring;
    const int oob = p.num_pages * kPage;  // past the pool: zeros
    for (; w.alive() && go; w.next()) {
      if (new_request(go)) ring.restart(F8 ? w.sh.raw_slots() : w.sh.k_slots());
      const int key = w.tile * kTileKeys + (int)rank * 128;
      int r0 = kw_pool_row(p, w.b, w.kv_len, key);
      int r1 = kw_pool_row(p, w.b, w.kv_len, key + kPage);
      r0 = r0 < 0 ? oob : r0;
      r1 = r1 < 0 ? oob : r1;
      uint8_t* ring_at = sm + (F8 ? w.sh.raw_at() : w.sh.k_at());
      for (int kc = 0; kc < kChunks && go; ++kc) {
        const int s = ring.slot;
        go = wait(F8 ? &c.raw_empty[s] : &c.k_empty[s], ring.phase() ^ 1);
        if (!go) break;
        if (elect_one()) {
          const CUtensorMap* map = kc < 8 ? &tm_ckv : &tm_kpe;
          const int x = kc < 8 ? kc * 64 : 0;
          if (F8) {
            arrive_expect_tx(&c.raw_full[s], kRawSlot);
            const uint32_t dst = smem_u32(ring_at + s * kRawSlot);
            tma_2d_local(dst, map, &c.raw_full[s], x, r0);
            tma_2d_local(dst + kRawSlot / 2, map, &c.raw_full[s], x, r1);
          } else {
            const uint32_t bar = map_to_rank(smem_u32(&c.k_full[s]), 0);
            if (rank == 0) arrive_expect_tx(&c.k_full[s], 2 * kKChunk);
            const uint32_t dst = smem_u32(ring_at + s * kKChunk);
            tma_2d(dst, map, bar, x, r0);
            tma_2d(dst + kKChunk / 2, map, bar, x, r1);
          }
        }
        __syncwarp();
        ring.advance();
      }
    }
    // the last use of every slot must be over before the CTA may exit
    for (int s = 0; s < kMaxK && go; ++s)
      go = wait(F8 ? &c.raw_empty[s] : &c.k_empty[s], ((ring.used >> s) & 1u) ^ 1);
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
      const int half = w.sh.cols / 2, bytes = half * 128;
      int box = kBoxes - 1;  // the tallest box that fits the half and the run
      while (box > 0 && ((half | tp.run) & ((8 << box) - 1))) --box;
      const int box_rows = 8 << box;
      const CUtensorMap* tm_qn = &tm_q.nope[box];
      const CUtensorMap* tm_qp = &tm_q.pe[box];
      const bool mine = lane < half / box_rows;
      uint8_t* at = sm + w.sh.q_at() + lane * box_rows * 128;
      for (int rb = 0; rb < w.sh.blocks && go; ++rb) {
        const int y = mine ? map_row(rb * w.sh.cols + (int)rank * half + lane * box_rows) : 0;
        if (w.sh.stay) {  // all nine chunks at once, to stay
          if (lane == 0 && rank == 0) arrive_expect_tx(&c.r_full, 2 * bytes * kChunks);
          __syncwarp();
          const uint32_t bar = map_to_rank(smem_u32(&c.r_full), 0);
          if (mine)
            for (int kc = 0; kc < kChunks; ++kc)
              tma_2d(smem_u32(at + kc * bytes), kc < 8 ? tm_qn : tm_qp, bar, kc < 8 ? kc * 64 : 0, y);
          __syncwarp();
          continue;
        }
        for (int kc = 0; kc < kChunks && go; ++kc) {
          const int s = ring.slot;
          go = wait(&c.q_empty[s], ring.phase() ^ 1);
          if (!go) break;
          if (lane == 0 && rank == 0) arrive_expect_tx(&c.q_full[s], 2 * bytes);
          __syncwarp();
          if (mine)
            tma_2d(smem_u32(at + s * bytes), kc < 8 ? tm_qn : tm_qp,
                   map_to_rank(smem_u32(&c.q_full[s]), 0), kc < 8 ? kc * 64 : 0, y);
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
      bool ok = true;
      Ring kring, qring;
      uint32_t rphase = 0, pass = 0;
      const uint64_t desc = sw128_desc(smem_u32(sm));
      for (; w.alive() && ok; w.next()) {
        const bool stream = !w.sh.stay;
        const int bytes = w.sh.cols * 64;  // of a chunk of this CTA's rows
        if (held != w.b) {
          held = w.b;
          kring.restart(w.sh.k_slots());
          qring.restart(stream ? w.sh.q_slots() : 1);
          if (!stream) {
            ok = wait(&c.r_full, rphase);
            rphase ^= 1;
          }
        }
        // kind::f16: fp32 sums; A, B bf16 (1) or fp16 (0), K-major; M = 256
        const uint32_t idesc = (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) |
                               ((uint32_t)(w.sh.cols >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
        const uint64_t dk = desc + (uint64_t)(w.sh.k_at() >> 4);
        const uint64_t dq = desc + (uint64_t)(w.sh.q_at() >> 4);
        const bool seg_end = w.last_of_request();
        const Ring first = kring;  // the tile's first chunk: every block begins there
        for (int rb = 0; rb < w.sh.blocks && ok; ++rb, ++pass) {
          const uint32_t d = tmem + (pass & 1) * 256;
          const bool last = rb == w.sh.blocks - 1;
          if (rb > 0) kring = first;
          ok = wait(&c.s_empty[pass & 1], ((pass >> 1) & 1) ^ 1);
          for (int kc = 0; kc < kChunks && ok; ++kc) {
            const int ks = kring.slot, qs = qring.slot;
            if (rb == 0) ok = wait(&c.k_full[ks], kring.phase());
            if (ok && stream) ok = wait(&c.q_full[qs], qring.phase());
            if (!ok) break;
            if (elect_one()) {
              fence_after();
              const uint64_t a = dk + (uint64_t)((ks * kKChunk) >> 4);
              const uint64_t b = dq + (uint64_t)(((stream ? qs : kc) * bytes) >> 4);
              mma_pair(d, a, b, idesc, kc != 0);
              mma_pair(d, a + 2, b + 2, idesc, 1u);
              mma_pair(d, a + 4, b + 4, idesc, 1u);
              mma_pair(d, a + 6, b + 6, idesc, 1u);
              if (stream) commit_pair(&c.q_empty[qs]);
              if (last) commit_pair(&c.k_empty[ks]);
              if (kc == kChunks - 1) {
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
  } else if (F8 && warp >= kWarpConv<F8>) {
    // ------------------------------------------------------- FP8 codes to fp16 chunks
    // The teams work on different chunks at once, because a chunk's path (code wait,
    // loads, conversion, stores, proxy fence, arrival) takes over 1000 clocks.  Two
    // warps a team, 64 keys each: lane l has codes 16 (l & 3) .. of keys l / 4 + 8 i.
    // A phase bit cannot tell a slot's last use from the one two before, so a team
    // must not ask for a slot whose last use another team is still at: with 4 slots
    // that was its own, and with 9 it is 9 chunks back, while codes arrive only when
    // the chunks kRawBeside = 5 and more before them are converted.
    constexpr int kKeysPerWarp = 128 * kConvTeams / kConvWarps;
    const int cw = warp - kWarpConv<F8>, team = cw % kConvTeams;
    const int m0 = cw / kConvTeams * kKeysPerWarp, sub = lane >> 2, u0 = lane & 3;
    const uint32_t full0 = map_to_rank(smem_u32(&c.k_full[0]), 0);
    bool go = true;
    Ring raw, ring;
    int turn = 0;
    for (; w.alive() && go; w.next()) {
      if (new_request(go)) {
        ring.restart(w.sh.k_slots());
        raw.restart(w.sh.raw_slots());
      }
      const uint8_t* codes = sm + w.sh.raw_at() + (m0 + sub) * 64 + u0 * 16;
      uint8_t* k_at = sm + w.sh.k_at() + (m0 + sub) * 128;
      for (int kc = 0; kc < kChunks && go; ++kc) {
        if (turn == team) {
          go = wait(&c.raw_full[raw.slot], raw.phase());
          if (go) go = wait(&c.k_empty[ring.slot], ring.phase() ^ 1);
          if (!go) break;
#pragma unroll 2
          for (int i = 0; i < kKeysPerWarp / 8; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(codes + raw.slot * kRawSlot + i * 512);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2(
                  (__nv_fp8x2_storage_t)(x[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
              o[j] = (uint32_t)f.x | (uint32_t)f.y << 16;
            }
            uint8_t* to = k_at + ring.slot * kKChunk + i * 1024;  // key m0 + sub + 8 i
            *reinterpret_cast<uint4*>(to + (((2 * u0) ^ sub) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(to + (((2 * u0 + 1) ^ sub) << 4)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            arrive(&c.raw_empty[raw.slot]);
            arrive_cluster(full0 + ring.slot * 8);
          }
        }
        turn = turn + 1 == kConvTeams ? 0 : turn + 1;
        raw.advance();
        ring.advance();
      }
    }
    for (int s = 0; s < kMaxK && go; ++s) go = wait(&c.k_empty[s], ((ring.used >> s) & 1u) ^ 1);
    if (go) wait(&c.seg_done, seg_parity);
  } else if (warp >= kWarpInfo && warp < kWarpConv<F8>) {
    // ------------------------------------------------------- column data of each pass
    // Ahead of the epilogue, so that their loads are off its path; two warps take
    // turns.
    const int W = (p.T + 63) >> 6;
    uint32_t pass = 0;
    bool go = true;
    for (; w.alive() && go; w.next()) {
      for (int rb = 0; rb < w.sh.blocks && go; ++rb, ++pass) {
        const int buf = pass & 1;
        if (kInfoWarps<F8> == 2 && buf != warp - kWarpInfo) continue;
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
            c.l2[buf][e] = l[k] * kLog2e;
            if (F8) c.factor[buf][e] = adds ? f[k] * (p.scale * kLog2e) : 0.f;
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
    const float factor = p.scale * kLog2e;
    const int W = (p.T + 63) >> 6;
    uint32_t pass = 0, tile_no = 0;
    for (; w.alive(); w.next(), ++tile_no) {
      const int key = w.tile * kTileKeys + (int)rank * 128 + m;
      const int krow = half == 0 ? kw_pool_row(p, w.b, w.kv_len, key) : 0;
      const size_t slot = (size_t)w.b * p.max_pages * kPage + key;
      const float old = half == 0 && p.weights_in && key < w.kv_len ? p.weights_in[slot] : 0.f;
      const int P = w.kv_len - p.T;
      // a tail key is seen by some nodes only: bit n of (seen0, seen1) for node n
      const bool tail = w.tile * kTileKeys + (int)rank * 128 + 32 * q + 32 > P;  // of the warp
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
      for (int rb = 0; rb < w.sh.blocks; ++rb, ++pass) {
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
          wait_ld();
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
          const float* l2 = &c.l2[buf][at];
          const float* fc = &c.factor[buf][at];
          if (__any_sync(0xffffffffu, off != 0)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float v = ex2f(fmaf(x[i], F8 ? fc[i] : factor, -l2[i]));
              sum[i & 3] += (off >> i) & 1u ? 0.f : v;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sum[i & 3] += ex2f(fmaf(x[i], F8 ? fc[i] : factor, -l2[i]));
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
        p.weights[slot] = p.decay * old + (krow >= 0 ? s + c.xsum[tile_no & 1][m] : 0.f);
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

// Counted rows of every request, dense from b * T * H on; for an FP8 cache as
// fp16, multiplied by the power of two that brings the row's largest element
// to [2^14, 2^15), and its inverse.  One warp per row.
template <bool F8>
__global__ void __launch_bounds__(256)
kweights_rows_kernel(const KwParams p, uint4* __restrict__ qn, uint4* __restrict__ qp,
                     float* __restrict__ scale) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  const KwRequest rq = kw_request(p, b);
  if (!rq.ok || r >= rq.nodes * p.H) return;
  int node;
  const int g = kw_query_row(p, b, rq, r, &node);
  if (g < 0) return;
  const size_t to = (size_t)b * p.T * p.H + r;
  const uint4* sn = reinterpret_cast<const uint4*>(p.q_nope) + (size_t)g * (kDc / 8);
  const uint4* sp = reinterpret_cast<const uint4*>(p.q_pe) + (size_t)g * (kDr / 8);
  uint4 v[3];
  v[0] = sn[lane];
  v[1] = sn[lane + 32];
  v[2] = lane < 8 ? sp[lane] : make_uint4(0, 0, 0, 0);
  if (F8) {
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
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 h = __floats2half2_rn(__uint_as_float(u[k] << 16) * up,
                                            __uint_as_float(u[k] & 0xffff0000u) * up);
        u[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
      v[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    if (lane == 0) scale[to] = ldexpf(1.f, -ex);
  }
  qn[to * (kDc / 8) + lane] = v[0];
  qn[to * (kDc / 8) + lane + 32] = v[1];
  if (lane < 8) qp[to * (kDr / 8) + lane] = v[2];
}

struct RowsLayout {
  size_t qn, qp, scale, total;
};
RowsLayout rows_layout(const va_key_weight_args& a, bool f8) {
  const size_t rows = (size_t)a.B * a.T * a.H;
  RowsLayout l;
  l.qn = 0;
  l.qp = align256(rows * kDc * 2);
  l.scale = l.qp + align256(rows * kDr * 2);
  l.total = l.scale + (f8 ? align256(rows * sizeof(float)) : 0);
  return l;
}
// The rows are laid out densely first when they need converting, or when the
// accepted nodes' runs of H rows are no whole number of 8-row swizzle groups.
bool needs_rows(const va_key_weight_args& a) {
  return (a.flags & VA_FLAG_KV_FP8_E4M3) || (a.path && a.H % 8 != 0);
}

}  // namespace

size_t kweights_tc_workspace(const va_key_weight_args& a) {
  return needs_rows(a) ? rows_layout(a, a.flags & VA_FLAG_KV_FP8_E4M3).total : 0;
}

cudaError_t launch_kweights_tc(const va_key_weight_args& a, const KwParams& p, int sms,
                               cudaStream_t st) {
  const bool f8 = a.flags & VA_FLAG_KV_FP8_E4M3;
  const uint64_t rows = (uint64_t)a.B * a.T * a.H;
  TcParams tp;
  tp.k = p;
  tp.dense = needs_rows(a);
  tp.run = tp.dense || !a.path ? 64 : a.H;
  tp.q_scale = nullptr;
  const void* qn = a.q_nope;
  const void* qp = a.q_pe;
  if (tp.dense) {
    const RowsLayout l = rows_layout(a, f8);
    char* ws = static_cast<char*>(a.workspace);
    qn = ws + l.qn;
    qp = ws + l.qp;
    float* scale = f8 ? reinterpret_cast<float*>(ws + l.scale) : nullptr;
    tp.q_scale = scale;
    const dim3 grid((unsigned)((a.T * a.H + 7) / 8), (unsigned)a.B);
    auto* k = f8 ? kweights_rows_kernel<true> : kweights_rows_kernel<false>;
    k<<<grid, 256, 0, st>>>(p, (uint4*)qn, (uint4*)qp, scale);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  QMaps tq = {};
  CUtensorMap tckv, tkpe;
  const uint64_t pool = (uint64_t)a.num_pages * kPage;
  // the boxes that halves (multiples of 32 rows) take in these runs: the run's own
  // power of two, and 32 beside 64
  int tallest = kBoxes - 1;
  while (tallest > 0 && tp.run % (8 << tallest)) --tallest;
  for (int i = tallest == kBoxes - 1 ? tallest - 1 : tallest; i <= tallest; ++i)
    if (!encode_rows(&tq.nope[i], qn, rows, kDc, 8 << i, f8 ? Elem::f16 : Elem::bf16) ||
        !encode_rows(&tq.pe[i], qp, rows, kDr, 8 << i, f8 ? Elem::f16 : Elem::bf16))
      return cudaErrorInvalidValue;
  if (!encode_rows(&tckv, a.c_kv, pool, kDc, kPage, f8 ? Elem::u8 : Elem::bf16) ||
      !encode_rows(&tkpe, a.k_pe, pool, kDr, kPage, f8 ? Elem::u8 : Elem::bf16))
    return cudaErrorInvalidValue;
  const long long tiles = (long long)a.B * (((long long)a.max_pages * kPage + kTileKeys - 1) / kTileKeys);
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  auto* k = f8 ? kweights_tc_kernel<true> : kweights_tc_kernel<false>;
  static std::atomic<bool> done[2][kMaxDevices];
  cudaError_t e = raise_smem_once(k, (int)kSmemBytes, done[f8]);
  if (e != cudaSuccess) return e;
  const int threads = (f8 ? kWarps<true> : kWarps<false>) * 32;
  k<<<2 * pairs, threads, kSmemBytes, st>>>(tq, tckv, tkpe, tp);
  return cudaGetLastError();
}

unsigned int kw_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kw_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

}  // namespace va
