// Key weights on tensor cores (bf16 queries; bf16 or FP8 cache), sm_100a.
//
//   w_j = sum over counted rows r, j visible to r, of
//         exp(scale q_r . k_j - lse_r)
// The keys are the M side of the product and the rows the N side: a CTA pair
// (tcgen05.mma.cta_group::2, M = 256) takes a tile of 256 keys, 128 a CTA,
// and up to 256 rows at a time.  In tensor memory a key is then a lane and a
// row a column, so a thread adds its key's exponentials over the columns in
// a register, and nothing is exchanged between threads but the two halves
// of a tile's columns.
//
// A tile's keys (9 chunks of 64 dims, 144 KB a CTA) stay in shared memory
// while all rows of the request pass by, so each key is read from HBM once
// and no partial sums leave the SM.  Rows come through a ring of 16 KB slots;
// a request of at most 128 rows has them resident instead, loaded once for
// all of the pair's tiles.  The tiles of all requests, in order and weighted
// by what their load and rows cost, are divided into equal contiguous
// ranges, one per pair.
//
// FP8 cache: converter warps read the codes and write them as fp16, which
// holds every E4M3 value; the queries are multiplied by a power of two per
// row and stored as fp16 by a first kernel (exact down to 2^-39 of the row's
// largest element), and the epilogue undoes it in fp32.
//
// Bound by HBM for few rows (1152 or 576 bytes a key), by the operand traffic
// from L2 into shared memory for many (64 bytes a clock and SM at the full
// MMA rate), with the exponentials (16 a clock and SM) close behind.
#include "va_kweights.cuh"
#include "va_tc_ops.cuh"

namespace va {

__device__ unsigned int g_kw_timeouts = 0;  // count of barrier waits that expired

namespace {

using namespace tc;

constexpr int kTileKeys = 256;          // of the pair
constexpr int kChunks = 9;              // 64-dim chunks: 8 of c_kv, 1 of k_pe
constexpr int kKChunk = 128 * 128;      // bytes: 128 keys x 64 dims
constexpr int kQSlots = 4;
constexpr int kQSlot = 128 * 128;       // bytes: up to 128 rows x 64 dims
constexpr int kQBytes = kChunks * 64 * 128;  // resident rows: 64 a CTA (>= the ring)
constexpr int kRowsResident = 128;      // of the pair
constexpr int kWarpK = 0, kWarpMma = 1, kWarpEpi = 2, kWarpQ = 10, kWarpInfo = 11, kWarpConv = 12;
constexpr int kConvWarps = 8;          // 16 keys of the CTA's tile each
constexpr int kConvAhead = 4;           // chunks whose codes are in flight
static_assert(kQBytes >= kQSlots * kQSlot, "the ring shares the resident rows' space");

struct TcParams {
  KwParams k;
  int dense;             // rows of request b start at b * T * H of the q maps
  int box_rows;          // rows of a query box
  const float* q_scale;  // FP8 cache: [B, T H] power of two that undoes the row's
};

struct __align__(16) Ctl {
  uint64_t k_full[kChunks], k_empty[kChunks];
  uint64_t q_full[kQSlots], q_empty[kQSlots];
  uint64_t r_full, r_empty;   // resident rows
  uint64_t s_full[2], s_empty[2];
  uint64_t i_full[2], i_empty[2];  // column data of a pass
  uint64_t drain;
  long long start_off, lo, hi;
  int start_b, start_tile;
  uint32_t tmem;
  int abort;
  // of each column of a pass: its node, its row's log2-sum and factor; and one
  // bit where the column adds nothing (no row, absent node, empty row)
  uint32_t none[2][8];
  int one[2][8];         // the node of all that a 32-column group adds, or -1
  float xsum[2][128];
  uint8_t node[2][256];
  float l2[2][256];
  float factor[2][256];  // FP8 cache
};
constexpr int kScanAt = offsetof(Ctl, xsum);  // the start-up scan uses xsum ..
static_assert(kScanAt % 8 == 0, "scan alignment");
constexpr size_t kSmemBytes = 1024 + (size_t)kChunks * kKChunk + kQBytes + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__host__ __device__ __forceinline__ int pad64(int n) { return n < 64 ? 64 : (n + 63) & ~63; }
// Columns of row block rb of a request of R rows.
__device__ __forceinline__ int block_cols(int R, int rb) { return pad64(min(256, R - rb * 256)); }
__device__ __forceinline__ int row_blocks(int R) { return R <= 256 ? 1 : (R + 255) >> 8; }
// What a tile costs: its keys' load (256) and its rows'.
__device__ __forceinline__ int tile_cost(int R) {
  return 256 + ((R <= 256 ? 0 : (R - 1) & ~255) + block_cols(R, row_blocks(R) - 1));
}

// The pair's tiles, in order.  Every warp role walks them by itself.
struct Walk {
  const KwParams* p;
  long long off, end;
  int b, tile, tiles, R, kv_len, cost;
  KwRequest rq;
  __device__ __forceinline__ void load() {
    for (; b < p->B; ++b) {
      rq = kw_request(*p, b);
      if (rq.ok) break;
    }
    if (b < p->B) {
      kv_len = rq.kv_len;
      tiles = (kv_len + kTileKeys - 1) / kTileKeys;
      R = rq.nodes * p->H;
      cost = tile_cost(R);
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

template <bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__((kWarpConv + (F8 ? kConvWarps : 0)) * 32, 1)
kweights_tc_kernel(const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qp,
                   const __grid_constant__ CUtensorMap tm_ckv,
                   const __grid_constant__ CUtensorMap tm_kpe, const __grid_constant__ TcParams tp) {
  constexpr int kThreads = (kWarpConv + (F8 ? kConvWarps : 0)) * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sK = base;
  uint8_t* sQ = sK + (size_t)kChunks * kKChunk;
  Ctl& c = *reinterpret_cast<Ctl*>(sQ + kQBytes);
  const KwParams& p = tp.k;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  unsigned int* expired = &g_kw_timeouts;
  volatile int* abort = &c.abort;

  if (tid == 0) {
    for (int i = 0; i < kChunks; ++i) {
      mbar_init(&c.k_full[i], F8 ? 2 * kConvWarps : 1);
      mbar_init(&c.k_empty[i], 1);
    }
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(&c.q_full[i], 1);
      mbar_init(&c.q_empty[i], 1);
    }
    mbar_init(&c.r_full, 1);
    mbar_init(&c.r_empty, 1);
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
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
      const KwRequest rq = kw_request(p, b);
      if (rq.ok) sum += (long long)((rq.kv_len + kTileKeys - 1) / kTileKeys) * tile_cost(rq.nodes * p.H);
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
        const int tiles = (rq.kv_len + kTileKeys - 1) / kTileKeys;
        const int cost = tile_cost(rq.nodes * p.H);
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
  Walk w;
  w.start(p, c);

  if (warp == kWarpK) {
    // ------------------------------------------------- key chunks by TMA (bf16 cache)
    if (!F8) {
      bool go = true;
      uint32_t phase = 0;
      const int oob = p.num_pages * kPage;  // past the pool: zeros
      for (; w.alive() && go; w.next(), phase ^= 1) {
        const int key = w.tile * kTileKeys + (int)rank * 128;
        const int r0 = kw_pool_row(p, w.b, w.kv_len, key);
        const int r1 = kw_pool_row(p, w.b, w.kv_len, key + kPage);
        for (int kc = 0; kc < kChunks && go; ++kc) {
          go = warp_wait(&c.k_empty[kc], phase ^ 1, abort, expired);
          if (!go) break;
          if (elect_one()) {
            const uint32_t bar = map_to_rank(smem_u32(&c.k_full[kc]), 0);
            if (rank == 0) arrive_expect_tx(&c.k_full[kc], 2 * kKChunk);
            const uint32_t dst = smem_u32(sK + (size_t)kc * kKChunk);
            const CUtensorMap* map = kc < 8 ? &tm_ckv : &tm_kpe;
            const int x = kc < 8 ? kc * 64 : 0;
            tma_2d(dst, map, bar, x, r0 < 0 ? oob : r0);
            tma_2d(dst + kKChunk / 2, map, bar, x, r1 < 0 ? oob : r1);
          }
          __syncwarp();
        }
      }
      // the last use of every chunk must be over before the CTA may exit
      for (int kc = 0; kc < kChunks && go; ++kc)
        go = warp_wait(&c.k_empty[kc], phase ^ 1, abort, expired);
      if (*abort) settle();
    }
  } else if (warp == kWarpQ) {
    // ------------------------------------------------------------ query rows by TMA
    bool go = true;
    int slot = 0;
    uint32_t phase = 0, rphase = 0;
    int held = -1;           // request whose rows are resident
    bool streaming = false;  // the space's last use was the ring
    const long long rows_total = (long long)p.B * p.T * p.H;
    // first map row of rows [r, r + box_rows) of the request (one node's, or dense)
    auto map_row = [&](int r) -> int {
      if (tp.dense) return (int)((long long)w.b * p.T * p.H + r);
      if (r >= w.R) return (int)rows_total;
      const int i = r / p.H;
      const int n = p.path ? p.path[(size_t)w.b * p.T + i] : i;
      if (n < 0 || n >= p.T) return (int)rows_total;
      return (int)(((long long)w.b * p.T + n) * p.H + (r - i * p.H));
    };
    auto ring_empty = [&]() {  // every slot's last rows have been used
      for (int i = 0; i < kQSlots && go; ++i) {
        const int s = (slot + i) % kQSlots;
        go = warp_wait(&c.q_empty[s], (s < slot ? phase : phase ^ 1), abort, expired);
      }
    };
    for (; w.alive() && go; w.next()) {
      if (w.R <= kRowsResident) {
        if (held == w.b) continue;
        if (streaming) ring_empty();
        streaming = false;
        if (go) go = warp_wait(&c.r_empty, rphase ^ 1, abort, expired);
        if (!go) break;
        const int half = block_cols(w.R, 0) / 2;
        if (lane == 0 && rank == 0) arrive_expect_tx(&c.r_full, 2 * half * 128 * kChunks);
        __syncwarp();
        const uint32_t bar = map_to_rank(smem_u32(&c.r_full), 0);
        if (lane < half / tp.box_rows) {
          const int y = map_row((int)rank * half + lane * tp.box_rows);
          for (int kc = 0; kc < kChunks; ++kc)
            tma_2d(smem_u32(sQ + kc * half * 128 + lane * tp.box_rows * 128),
                   kc < 8 ? &tm_qn : &tm_qp, bar, kc < 8 ? kc * 64 : 0, y);
        }
        __syncwarp();
        rphase ^= 1;
        held = w.b;
      } else {
        if (held >= 0) {  // resident rows of the last request: wait for their last use
          go = warp_wait(&c.r_empty, rphase ^ 1, abort, expired);
          held = -1;
        }
        streaming = true;
        const int blocks = row_blocks(w.R);
        for (int rb = 0; rb < blocks && go; ++rb) {
          const int half = block_cols(w.R, rb) / 2;
          const bool mine = lane < half / tp.box_rows;
          const int y = mine ? map_row(rb * 256 + (int)rank * half + lane * tp.box_rows) : 0;
          for (int kc = 0; kc < kChunks && go; ++kc) {
            go = warp_wait(&c.q_empty[slot], phase ^ 1, abort, expired);
            if (!go) break;
            if (lane == 0 && rank == 0) arrive_expect_tx(&c.q_full[slot], 2 * half * 128);
            __syncwarp();
            if (mine)
              tma_2d(smem_u32(sQ + slot * kQSlot + lane * tp.box_rows * 128),
                     kc < 8 ? &tm_qn : &tm_qp, map_to_rank(smem_u32(&c.q_full[slot]), 0),
                     kc < 8 ? kc * 64 : 0, y);
            __syncwarp();
            if (++slot == kQSlots) { slot = 0; phase ^= 1; }
          }
        }
      }
    }
    if (go) ring_empty();
    if (go) warp_wait(&c.r_empty, rphase ^ 1, abort, expired);
    if (*abort) settle();
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ MMA issue
    if (rank == 0) {
      bool ok = true;
      int slot = 0, held = -1;
      uint32_t qphase = 0, kphase = 0, rphase = 0, pass = 0;
      const uint64_t dk = sw128_desc(smem_u32(sK)), dq = sw128_desc(smem_u32(sQ));
      for (; w.alive() && ok; w.next(), kphase ^= 1) {
        const bool resident = w.R <= kRowsResident;
        if (resident && held != w.b) {
          ok = warp_wait(&c.r_full, rphase, abort, expired);
          rphase ^= 1;
          held = w.b;
        }
        if (!resident) held = -1;
        const int blocks = row_blocks(w.R);
        for (int rb = 0; rb < blocks && ok; ++rb, ++pass) {
          const int cols = block_cols(w.R, rb);
          // kind::f16: fp32 sums; A, B bf16 (1) or fp16 (0), K-major; M = 256
          const uint32_t idesc = (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) |
                                 ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
          const uint32_t d = tmem + (pass & 1) * 256;
          ok = warp_wait(&c.s_empty[pass & 1], ((pass >> 1) & 1) ^ 1, abort, expired);
          for (int kc = 0; kc < kChunks && ok; ++kc) {
            if (rb == 0) ok = warp_wait(&c.k_full[kc], kphase, abort, expired);
            if (ok && !resident) ok = warp_wait(&c.q_full[slot], qphase, abort, expired);
            if (!ok) break;
            if (elect_one()) {
              fence_after();
              const uint64_t a = dk + (uint64_t)((kc * kKChunk) >> 4);
              const uint64_t b = dq + (uint64_t)((resident ? kc * cols * 64 : slot * kQSlot) >> 4);
              mma_pair(d, a, b, idesc, kc != 0);
              mma_pair(d, a + 2, b + 2, idesc, 1u);
              mma_pair(d, a + 4, b + 4, idesc, 1u);
              mma_pair(d, a + 6, b + 6, idesc, 1u);
              if (!resident) commit_pair(&c.q_empty[slot]);
              if (rb == blocks - 1) commit_pair(&c.k_empty[kc]);
              if (kc == kChunks - 1) {
                commit_pair(&c.s_full[pass & 1]);
                if (resident && w.last_of_request()) commit_pair(&c.r_empty);
              }
            }
            __syncwarp();
            if (!resident && ++slot == kQSlots) { slot = 0; qphase ^= 1; }
          }
        }
      }
      if (!ok) {  // let every MMA already issued finish before tensor memory is freed
        if (elect_one()) commit_pair(&c.drain);
        __syncwarp();
        final_wait(&c.drain, 0);
      }
    }
  } else if (F8 && warp >= kWarpConv) {
    // ------------------------------------------- key chunks from FP8 codes, as fp16
    // A warp converts 16 keys of one page.  Of a chunk, lane l reads 16 codes (l & 3)
    // of keys l / 4 + 8 i, so that 4 lanes read a key's 64 bytes; the codes of the
    // next kConvAhead chunks are in flight in registers (volatile: loads stay there).
    const int m0 = (warp - kWarpConv) * 16, sub = lane >> 2, u0 = lane & 3;
    const uint8_t* ckv = reinterpret_cast<const uint8_t*>(p.c_kv) + u0 * 16;
    const uint8_t* kpe = reinterpret_cast<const uint8_t*>(p.k_pe) + u0 * 16;
    uint4 code[kChunks][2];
    // pool row of the warp's first key, and how many of its keys exist
    struct Keys { int row, n; };
    auto keys_of = [&](const Walk& v) {
      Keys k{0, 0};
      if (!v.alive()) return k;
      const int key = v.tile * kTileKeys + (int)rank * 128 + m0;
      const int row = kw_pool_row(p, v.b, v.kv_len, key);
      if (row >= 0) { k.row = row; k.n = v.kv_len - key; }
      return k;
    };
    auto fetch = [&](int kc, const Keys& k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4& v = code[kc][i];
        v = make_uint4(0, 0, 0, 0);
        const int r = sub + 8 * i;
        const uint8_t* src = kc < 8 ? ckv + (size_t)(k.row + r) * kDc + kc * 64
                                    : kpe + (size_t)(k.row + r) * kDr;
        if (r < k.n)
          asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src));
      }
    };
    const uint32_t full0 = map_to_rank(smem_u32(&c.k_full[0]), 0);
    Keys keys = keys_of(w);
#pragma unroll
    for (int kc = 0; kc < kConvAhead; ++kc) fetch(kc, keys);
    uint32_t phase = 0;
    bool go = true;
    while (w.alive() && go) {
      w.next();
      const Keys next = keys_of(w);
#pragma unroll
      for (int kc = 0; kc < kChunks; ++kc) {
        if (kc + kConvAhead < kChunks) fetch(kc + kConvAhead, keys);
        else fetch(kc + kConvAhead - kChunks, next);
        if (go) go = warp_wait(&c.k_empty[kc], phase ^ 1, abort, expired);
        uint8_t* dst = sK + (size_t)kc * kKChunk + m0 * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = sub + 8 * i;
          const uint32_t cw[4] = {code[kc][i].x, code[kc][i].y, code[kc][i].z, code[kc][i].w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)(cw[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
            o[j] = (uint32_t)f.x | (uint32_t)f.y << 16;
          }
          uint8_t* row = dst + r * 128;
          *reinterpret_cast<uint4*>(row + (((2 * u0) ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(row + (((2 * u0 + 1) ^ (r & 7)) << 4)) =
              make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_cluster(full0 + kc * 8);
      }
      keys = next;
      phase ^= 1;
    }
    for (int kc = 0; kc < kChunks && go; ++kc)
      go = warp_wait(&c.k_empty[kc], phase ^ 1, abort, expired);
  } else if (warp == kWarpInfo) {
    // ------------------------------------------------------- column data of each pass
    // One pass ahead of the epilogue, so that its loads are off the epilogue's path.
    const int W = (p.T + 63) >> 6;
    uint32_t pass = 0;
    bool go = true;
    for (; w.alive() && go; w.next()) {
      const int blocks = row_blocks(w.R);
      for (int rb = 0; rb < blocks && go; ++rb, ++pass) {
        const int buf = pass & 1;
        float l[8], f[8];
        uint64_t word[8];
        int node[8];
        bool ok[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = rb * 256 + k * 32 + lane;
          const bool in = r < w.R;
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
        go = warp_wait(&c.i_empty[buf], ((pass >> 1) & 1) ^ 1, abort, expired);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool adds = ok[k] && ((word[k] >> (node[k] & 63)) & 1ull) && l[k] != -INFINITY;
          const int e = k * 32 + lane;
          c.node[buf][e] = (uint8_t)node[k];
          c.l2[buf][e] = l[k] * kLog2e;
          if (F8) c.factor[buf][e] = adds ? f[k] * (p.scale * kLog2e) : 0.f;
          const uint32_t none = __ballot_sync(0xffffffffu, !adds);
          const int first = __shfl_sync(0xffffffffu, node[k], none == ~0u ? 0 : __ffs(~none) - 1);
          const bool same = __all_sync(0xffffffffu, !adds || node[k] == first);
          if (lane == 0) {
            c.none[buf][k] = none;
            c.one[buf][k] = same ? first : -1;
          }
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&c.i_full[buf]))
                       : "memory");
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
      const int blocks = row_blocks(w.R);
      const int key = w.tile * kTileKeys + (int)rank * 128 + m;
      const int krow = half == 0 ? kw_pool_row(p, w.b, w.kv_len, key) : 0;
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
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int rb = 0; rb < blocks; ++rb, ++pass) {
        const int buf = pass & 1;
        const int cols = block_cols(w.R, rb) / 2;  // this half's
        const int c0 = half * cols;
        const uint32_t parity = (pass >> 1) & 1;
        warp_wait(&c.i_full[buf], parity, abort, expired);
        warp_wait(&c.s_full[buf], parity, abort, expired);
        fence_after();
        const uint32_t scores = tmem + lane_base + buf * 256 + c0;
        // one group of 32 columns: x holds its scores
        auto group = [&](const float (&x)[32], int g) {
          const float* l2 = &c.l2[buf][c0 + g];
          const float* fc = &c.factor[buf][c0 + g];
          uint32_t off = c.none[buf][(c0 + g) >> 5];  // columns that add nothing to this key
          if (tail) {
            const uint8_t* nodes = &c.node[buf][c0 + g];
            const int n = c.one[buf][(c0 + g) >> 5];
            uint32_t on = 0;
            if (n >= 0) {  // as with 32 heads and more
              on = ((n < 64 ? seen0 >> n : seen1 >> (n - 64)) & 1ull) ? ~0u : 0u;
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int n = nodes[i];
                on |= (uint32_t)((n < 64 ? seen0 >> n : seen1 >> (n - 64)) & 1ull) << i;
              }
            }
            off |= ~on;
          }
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
        };
        // all scores are in registers: the buffer may be written again
        auto drained = [&]() {
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(free0 + buf * 8);
        };
        float xa[32];
        if (F8) {  // 96 registers a thread, and bound by memory: one group at a time
#pragma unroll 1
          for (int g = 0; g < cols; g += 32) {
            ld32(scores + g, xa);
            wait_ld();
            if (g + 32 == cols) drained();
            group(xa, g);
          }
        } else {   // the next group's scores are on their way while one is worked on
          float xb[32];
          ld32(scores, xa);
#pragma unroll 1
          for (int g = 0; g < cols; g += 64) {
            wait_ld();
            const bool more = g + 32 < cols;
            if (more) ld32(scores + g + 32, xb);
            else drained();
            group(xa, g);
            if (more) {
              wait_ld();
              if (g + 64 < cols) ld32(scores + g + 64, xa);
              else drained();
              group(xb, g + 32);
            }
          }
        }
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&c.i_empty[buf]))
                       : "memory");
      }
      // the two halves of a key meet in shared memory (the quadrant's 64 threads)
      const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (half == 1) c.xsum[tile_no & 1][m] = s;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
      if (half == 0 && key < w.kv_len) {
        kw_store(p, w.b, 0, key, krow >= 0 ? s + c.xsum[tile_no & 1][m] : 0.f);
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
  tp.box_rows = tp.dense || !a.path || a.H % 32 == 0 ? 32 : a.H % 16 == 0 ? 16 : 8;
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
  CUtensorMap tqn, tqp, tckv, tkpe;
  if (!encode_rows(&tqn, qn, rows, kDc, tp.box_rows, f8) ||
      !encode_rows(&tqp, qp, rows, kDr, tp.box_rows, f8))
    return cudaErrorInvalidValue;
  if (f8) {  // the converters read the cache: no maps over it
    tckv = tqn;
    tkpe = tqp;
  } else if (!encode_rows(&tckv, a.c_kv, (uint64_t)a.num_pages * kPage, kDc, kPage, false) ||
             !encode_rows(&tkpe, a.k_pe, (uint64_t)a.num_pages * kPage, kDr, kPage, false)) {
    return cudaErrorInvalidValue;
  }
  const long long tiles = (long long)a.B * (((long long)a.max_pages * kPage + kTileKeys - 1) / kTileKeys);
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  auto* k = f8 ? kweights_tc_kernel<true> : kweights_tc_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  const int threads = (kWarpConv + (f8 ? kConvWarps : 0)) * 32;
  k<<<2 * pairs, threads, kSmemBytes, st>>>(tqn, tqp, tckv, tkpe, tp);
  return cudaGetLastError();
}

unsigned int kw_timeouts() {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kw_timeouts, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

}  // namespace va
