// Eviction from the paged latent cache by accumulated attention weight: the
// plan (which keys stay, in which slots) and the move of one cache's keys.
//
// Plan.  One cluster per request; CTA r of C owns a contiguous part of the
// slots.  A slot's key is 0 for a dropped slot, all ones for a protected one, else
// order-preserving bits of the weight (those lie strictly between).  The k heaviest
// unprotected candidates are found by a radix select on the keys (digits of 11, 11
// and 10 bits; one shared-memory histogram per CTA, joined over distributed shared
// memory), ties by lower slot through each CTA's count of the last digit.  Kept
// slots at or above the new length ("movers") fill the free slots below it
// ("holes"), both in ascending order: the holes are listed in the still unused end
// of from_slot, and each mover looks its hole up.  Order-preserving compaction would
// move every key behind the first hole; this moves only those past the new length.
//
// Parts of up to 32768 slots hold their keys in shared memory (Held): a thread takes a
// run of up to 32 slots, one block scan of both counts gives the indices, and holes
// and movers are listed in shared memory, in the keys' place, before they are written
// or looked up.  Longer parts read weights and positions again for every digit and scan
// tile by tile of four slots a thread, whose keep bits are held as a byte: batches of
// long requests, as 64 of 131072 slots with positions (225 us; 64 of 32832, whose keys
// are held, take 39).
//
// Move.  A CTA per 64 destination slots lists the slots that change and
// copies their rows with 16-byte accesses.  No slot is both source and
// destination, so the copy is in place and in any order.
//
// Both are bound by memory: 8 bytes a slot and an array for the plan, two
// row accesses per moved key for the move.
#include <climits>

#include "va_common.cuh"

namespace va {
namespace {

constexpr int kNT = 1024;
constexpr int kVec = 4;               // consecutive slots of a thread in a tile
constexpr int kTile = kNT * kVec;
constexpr int kBins = 2048;
constexpr int kBatch = 8, kFew = 4;   // loads of a thread in flight
constexpr int kMaxKeepBytes = 128 * 1024;  // keep bits of a CTA's slots in shared memory
constexpr int kMaxRun = 32;                // slots of a thread whose keys are held, at most
constexpr uint32_t kDropped = 0u, kProtected = ~0u;
constexpr int kMaxCluster = 8;
constexpr unsigned kFull = 0xffffffffu;

struct PlanParams {
  const float* weights;
  const int32_t* kv_len;
  const int32_t* budget;
  const int32_t* path;
  const int32_t* accept_len;
  const int32_t* pos;
  int cap, T, n_sink, n_recent;
  int32_t* new_len;
  int32_t* from_slot;
  float* weights_out;
  int32_t* pos_out;
  int32_t* req_status;
};

// Slots of each CTA of a cluster of C, a whole number of threads' quads.
__host__ __device__ __forceinline__ int slots_per_cta(int cap, int C) {
  return (int)(((long long)cap + C - 1) / C + kVec - 1) / kVec * kVec;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 remote_u32x2(const void* p, uint32_t rank) {
  uint32_t a;
  uint2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
// Sum of *p over CTAs [0, n) of the cluster; the loads are independent.
__device__ __forceinline__ uint32_t remote_sum(const uint32_t* p, int n) {
  uint32_t v[kMaxCluster], sum = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) v[r] = r < n ? remote_u32(p, r) : 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) sum += v[r];
  return sum;
}
// Bits that order like the weight: -0 like +0, NaN like -inf.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (!(x == x)) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Shared {
  __align__(8) uint32_t hist[2][kBins];
  __align__(8) uint32_t sum[kBins];  // this CTA's share of the bins, over the cluster
  uint32_t warp_sum[32];
  uint32_t total;
  int32_t newest;                 // of this CTA
  uint32_t cnt[4];                // protected | ties | kept below new_len | kept from it on
  uint32_t pick[3];               // digit, keys above it, keys in it
  uint32_t acc[3];                // accepted nodes, one bit each
  int bad;
};

// Exclusive prefix sum over the CTA's threads; the total goes to *total.
__device__ uint32_t block_scan(uint32_t v, Shared& s, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s.warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = s.warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, w, d);
      if (lane >= d) w += y;
    }
    s.warp_sum[lane] = w;  // inclusive over warps
  }
  __syncthreads();
  const uint32_t before = (warp ? s.warp_sum[warp - 1] : 0) + x - v;
  *total = s.warp_sum[31];
  __syncthreads();
  return before;
}

template <bool Held>
__global__ void __launch_bounds__(kNT) evict_plan_kernel(const PlanParams p, int C) {
  static_assert(sizeof(Shared) <= 28 * 1024, "beside 20 KB of dynamic shared memory");
  __shared__ Shared s;
  extern __shared__ uint32_t dyn[];  // keys of this CTA's slots (Held) and their keep bits
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  const int b = blockIdx.x / C;
  const size_t row = (size_t)b * p.cap;
  const float* w = p.weights + row;
  const int32_t* pos = p.pos ? p.pos + row : nullptr;
  const int T = p.T, cap = p.cap;
  const int len = p.kv_len[b];
  auto sync = [&]() {
    if (C > 1)
      asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;"
                   ::: "memory");
    else
      __syncthreads();
  };

  // request checks: kv_len, then the accepted path (ascending nodes)
  const bool len_ok = len >= T && len <= cap;
  const int n_acc_in = T > 0 ? p.accept_len[b] : 0;
  if (tid == 0) { s.bad = 0; s.newest = -1; }
  if (tid < 3) s.acc[tid] = 0;
  if (tid < 4) s.cnt[tid] = 0;
  for (int i = tid; i < 2 * kBins; i += kNT) (&s.hist[0][0])[i] = 0;
  __syncthreads();
  bool path_ok = n_acc_in >= 0 && n_acc_in <= T;
  if (path_ok && tid < n_acc_in) {
    const int n = p.path[(size_t)b * T + tid];
    const int prev = tid ? p.path[(size_t)b * T + tid - 1] : -1;
    if (n <= prev || n >= T || prev < -1) s.bad = 1;
    else atomicOr(&s.acc[n >> 5], 1u << (n & 31));
  }
  __syncthreads();
  path_ok = path_ok && !s.bad;
  if ((!len_ok || !path_ok) && rank == 0 && tid == 0 && p.req_status)
    p.req_status[b] = VA_ERR_INVALID_ARG;
  const int N = len_ok ? len : 0;       // slots in use
  const int P = len_ok ? len - T : 0;   // prefix
  const bool asis = len_ok && !path_ok;
  const uint32_t a0 = s.acc[0], a1 = s.acc[1], a2 = s.acc[2];
  const int n_acc = N > 0 && !asis ? n_acc_in : 0;

  // this CTA's slots, in whole quads
  const int per = slots_per_cta(cap, C);
  const int lo = min(cap, (int)rank * per), hi = min(cap, lo + per);
  const int hiN = min(hi, max(lo, N));
  const int run = (per + kNT - 1) / kNT;  // Held: consecutive slots of a thread, at most 32
  uint32_t* held = dyn;
  uint32_t* kept = dyn + kNT * run;       // Held: then one bit per slot
  uint8_t* keep4 = reinterpret_cast<uint8_t*>(dyn);  // else: one quad a byte

  auto accepted = [&](int j) {
    const int n = j - P;
    return n >= 0 && n < T && (((n < 32 ? a0 : n < 64 ? a1 : a2) >> (n & 31)) & 1u);
  };

  // newest position of a candidate
  int newest = 0;
  if (p.n_recent > 0) {
    if (!pos) {
      int last = P - 1;
      for (int n = 0; n < T; ++n)
        if (accepted(P + n)) last = P + n;
      newest = last;
    } else {
      int mine = INT_MIN;
      for (int j0 = lo + tid; j0 < hiN; j0 += kNT * kBatch) {
        int q[kBatch];
        float x[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = j0 + u * kNT;
          q[u] = j < hiN ? pos[j] : INT_MIN;
          if (Held) x[u] = j < hiN ? w[j] : 0.f;  // in the same wait
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int j = j0 + u * kNT;
          if (j >= hiN) break;
          if (j < P || accepted(j)) mine = max(mine, q[u]);
          if (Held) held[j - lo] = order_bits(x[u]);
        }
      }
      if (tid == 0) s.newest = INT_MIN;
      __syncthreads();
      mine = __reduce_max_sync(kFull, mine);
      if (lane == 0) atomicMax(&s.newest, mine);
      sync();
      newest = s.newest;
      if (C > 1) {
        int v[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) v[r] = r < C ? (int)remote_u32(&s.newest, r) : INT_MIN;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) newest = max(newest, v[r]);
      }
    }
  }
  // positions from here on are recent
  const int recent = p.n_recent > 0
                         ? (int)max((long long)newest - p.n_recent + 1, (long long)INT_MIN)
                         : INT_MAX;
  auto key_from = [&](int j, uint32_t bits, int q) -> uint32_t {
    if (j >= P) return accepted(j) ? kProtected : kDropped;
    return q < p.n_sink || (q >= recent && p.n_recent > 0) ? kProtected : bits;
  };
  auto key_of = [&](int j) {
    return Held ? held[j - lo] : key_from(j, order_bits(w[j]), pos ? pos[j] : j);
  };
  auto ranked = [](uint32_t k) { return k != kDropped && k != kProtected; };

  // the keys, how many are protected, and the first digit's histogram
  {
    uint32_t prot = 0;
    const bool have_bits = Held && pos && p.n_recent > 0;  // with the positions, above
    for (int j0 = lo + tid; j0 < hiN; j0 += kNT * kBatch) {
      int q[kBatch];
      uint32_t bits[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = j0 + u * kNT;
        q[u] = pos && j < hiN ? pos[j] : j;
        bits[u] = j >= hiN ? 0u : have_bits ? held[j - lo] : order_bits(w[j]);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int j = j0 + u * kNT;
        if (j >= hiN) break;
        const uint32_t k = key_from(j, bits[u], q[u]);
        if (Held) held[j - lo] = k;
        prot += k == kProtected;
        if (ranked(k)) atomicAdd(&s.hist[0][k >> 21], 1u);
      }
    }
    if (Held)  // slots behind the last key, to the end of the threads' runs
      for (int j = max(hiN, lo) + tid; j < lo + kNT * run; j += kNT) held[j - lo] = kDropped;
    prot = __reduce_add_sync(kFull, prot);
    if (lane == 0 && prot) atomicAdd(&s.cnt[0], prot);
  }
  sync();
  uint32_t n_prot = s.cnt[0];
  if (C > 1) n_prot = remote_sum(&s.cnt[0], C);
  const int n_cand = P + n_acc;
  const int n_other = n_cand - (int)n_prot;
  const int n_new = asis ? N : max(min(max(p.budget[b], 0), n_cand), (int)n_prot);
  const int k = n_new - (int)n_prot;  // how many of the others stay
  const bool select = !asis && k > 0 && k < n_other;

  // radix select: the k-th largest key of the others, and how many equal to
  // it stay.  Keys above `key_lo` stay; `ties` of those equal to it.
  uint32_t prefix = 0, need = (uint32_t)max(k, 0), ties_before = 0;
  if (select) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      uint32_t* h = s.hist[pass & 1];
      if (pass > 0) {
        const int above = pass == 1 ? 21 : 10;
#pragma unroll 4
        for (int j = lo + tid; j < hiN; j += kNT) {
          const uint32_t k = key_of(j);
          if (ranked(k) && (k >> above) == (prefix >> above))
            atomicAdd(&h[(k >> shift) & (bins - 1)], 1u);
        }
        sync();
      }
      // The bins over the cluster: of more than two, each CTA adds up its share of
      // them, so that a bin is read C times and not C * C.  Thread t then holds bins d0 and d0 - 1, the
      // highest left in descending order.
      uint32_t c0 = 0, c1 = 0;
      const int d0 = bins - 1 - 2 * tid;
      if (C == 2) {
        if (d0 > 0) {
          const uint2 v = remote_u32x2(&h[d0 - 1], 0), u = remote_u32x2(&h[d0 - 1], 1);
          c0 = v.y + u.y;
          c1 = v.x + u.x;
        }
      } else if (C > 1) {
        const int share = bins / C;
        for (int i = tid; i < share; i += kNT) s.sum[i] = remote_sum(&h[(int)rank * share + i], C);
        sync();
        if (d0 > 0) {
          const uint2 v = remote_u32x2(&s.sum[(d0 - 1) % share], (uint32_t)((d0 - 1) / share));
          c0 = v.y;
          c1 = v.x;
        }
      } else if (d0 > 0) {
        c0 = h[d0];
        c1 = h[d0 - 1];
      }
      uint32_t total;
      const uint32_t before = block_scan(c0 + c1, s, &total);
      if (d0 > 0 && before < need && need <= before + c0 + c1) {
        const bool second = need > before + c0;
        s.pick[0] = (uint32_t)(second ? d0 - 1 : d0);
        s.pick[1] = before + (second ? c0 : 0);
      }
      // the other buffer is read by no one any more: clear it for the next pass
      if (pass > 0)
        for (int i = tid; i < kBins; i += kNT) s.hist[(pass + 1) & 1][i] = 0;
      __syncthreads();
      prefix |= s.pick[0] << shift;
      need -= s.pick[1];
      if (pass == 2) {
        const uint32_t digit = prefix & 1023u;
        ties_before = remote_sum(&h[digit], (int)rank);
      }
      __syncthreads();
    }
  }
  const uint32_t key_lo = prefix;

  if constexpr (Held) {
    // Each thread takes the run of slots [j0, j0 + run): which of them stay, ...
    const int j0 = lo + tid * run;
    uint32_t keep = 0, eq = 0, total;
    for (int i = 0; i < run; ++i) {
      const uint32_t o = held[tid * run + i];
      const bool in = asis ? j0 + i < hiN
                           : o == kProtected || (ranked(o) && k > 0 && (!select || o > key_lo));
      if (in) keep |= 1u << i;
      else if (select && o == key_lo) eq |= 1u << i;
    }
    if (select) {  // ... ties by lower slot
      uint32_t at = ties_before + block_scan(__popc(eq), s, &total);
      for (; eq && at < need; ++at) {
        keep |= eq & (0u - eq);
        eq &= eq - 1;
      }
    }
    const int in_run = min(max(hi - j0, 0), run), below_n = min(max(n_new - j0, 0), in_run);
    const uint32_t below = below_n >= 32 ? ~0u : (1u << below_n) - 1u;
    uint32_t hole = ~keep & below, mover = keep & ~below;
    // Indices of its holes and movers: the CTA's (at most 32768 each) in one scan,
    // then the cluster's.  The outputs may overwrite the inputs from here on.
    const uint32_t both = block_scan(__popc(hole) | __popc(mover) << 16, s, &total);
    const int holes = (int)(total & 0xffffu), movers = (int)(total >> 16);
    if (tid == 0) { s.cnt[2] = holes; s.cnt[3] = movers; }
    for (int i = tid; i < (kNT * run + 31) / 32; i += kNT) kept[i] = 0;
    // their slots in order, in the keys' place: the copies below are then contiguous
    // on at least one side, where a run's own would touch a sector per slot
    int* hole_slot = reinterpret_cast<int*>(held);
    int* mover_slot = hole_slot + holes;
    for (uint32_t i = both & 0xffffu; hole; hole &= hole - 1) hole_slot[i++] = j0 + __ffs(hole) - 1;
    for (uint32_t i = both >> 16; mover; mover &= mover - 1) mover_slot[i++] = j0 + __ffs(mover) - 1;
    sync();
    {  // the run's bits, in one or two words
      const int bit = tid * run, sh = bit & 31;
      if (keep) atomicOr(&kept[bit >> 5], keep << sh);
      if (sh && keep >> (32 - sh)) atomicOr(&kept[(bit >> 5) + 1], keep >> (32 - sh));
    }
    const int hole_at = (int)remote_sum(&s.cnt[2], (int)rank);
    const int mover_at = (int)remote_sum(&s.cnt[3], (int)rank);
    // list the holes in from_slot[n_new ..): there are as many as movers, which
    // all lie there, so the list fits
    int* list = p.from_slot + row + n_new;
    for (int i = tid; i < holes; i += kNT) list[hole_at + i] = hole_slot[i];
    __threadfence();
    sync();
    // a mover's key goes to its hole, the other kept slots keep theirs
    for (int i0 = tid; i0 < movers; i0 += kNT * kFew) {
      int j[kFew], to[kFew], q[kFew];
      float x[kFew];
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        const int i = i0 + u * kNT;
        j[u] = i < movers ? mover_slot[i] : -1;
        if (j[u] < 0) continue;
        to[u] = __ldcg(&list[mover_at + i]);
        if (p.weights_out) x[u] = w[j[u]];
        if (p.pos_out) q[u] = pos[j[u]];
      }
#pragma unroll
      for (int u = 0; u < kFew; ++u) {
        if (j[u] < 0) continue;
        p.from_slot[row + to[u]] = j[u];
        if (p.weights_out) p.weights_out[row + to[u]] = x[u];
        if (p.pos_out) p.pos_out[row + to[u]] = q[u];
      }
    }
#pragma unroll 4
    for (int j = lo + tid; j < min(hi, n_new); j += kNT) {
      if (!((kept[(j - lo) >> 5] >> ((j - lo) & 31)) & 1u)) continue;
      p.from_slot[row + j] = j;
      if (p.weights_out) p.weights_out[row + j] = w[j];
      if (p.pos_out) p.pos_out[row + j] = pos[j];
    }
    sync();
#pragma unroll 4
    for (int j = max(lo, n_new) + tid; j < hi; j += kNT) {
      p.from_slot[row + j] = -1;
      if (p.weights_out) p.weights_out[row + j] = 0.f;
      if (p.pos_out) p.pos_out[row + j] = -1;
    }
    if (rank == 0 && tid == 0) p.new_len[b] = n_new;
    return;
  }

  // One tile: which of this thread's slots stay.  `tie` counts the ties seen
  // in earlier tiles (same value in every thread).
  auto keep_bits = [&](int t0, uint32_t& tie) {
    const int j0 = t0 + tid * kVec;
    uint32_t keep = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int j = j0 + i;
      if (j >= hiN) continue;
      if (asis) { keep |= 1u << i; continue; }
      const uint32_t o = key_of(j);
      if (o == kProtected) keep |= 1u << i;
      if (ranked(o) && k > 0) {
        if (!select || o > key_lo) keep |= 1u << i;
        else if (o == key_lo) eq |= 1u << i;
      }
    }
    if (select) {
      uint32_t total;
      uint32_t at = tie + block_scan(__popc(eq), s, &total);
      tie += total;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (eq >> i & 1u) {
          if (at < need) keep |= 1u << i;
          ++at;
        }
    }
    return keep;
  };
  // slots of this thread's quad that lie below n_new
  auto below_bits = [&](int j0) {
    const int n = min(max(n_new - j0, 0), kVec);
    return (1u << n) - 1u;
  };
  auto in_bits = [&](int j0) {
    const int n = min(max(hi - j0, 0), kVec);
    return (1u << n) - 1u;
  };

  // holes and movers of this CTA, counted, then joined over the cluster.  The
  // keep bits are held from here on: the outputs may overwrite the inputs.
  {
    uint32_t tie = ties_before, holes = 0, movers = 0;
    for (int t0 = lo; t0 < hi; t0 += kTile) {
      const uint32_t keep = keep_bits(t0, tie);
      const int j0 = t0 + tid * kVec;
      if (j0 < hi) keep4[(j0 - lo) / kVec] = (uint8_t)keep;
      holes += __popc(~keep & below_bits(j0) & in_bits(j0));
      movers += __popc(keep & ~below_bits(j0));
    }
    holes = __reduce_add_sync(kFull, holes);
    movers = __reduce_add_sync(kFull, movers);
    if (lane == 0 && holes) atomicAdd(&s.cnt[2], holes);
    if (lane == 0 && movers) atomicAdd(&s.cnt[3], movers);
  }
  sync();
  const uint32_t hole_at = remote_sum(&s.cnt[2], (int)rank);
  const uint32_t mover_at = remote_sum(&s.cnt[3], (int)rank);
  // list the holes in from_slot[n_new ..): there are as many as movers, which
  // all lie there, so the list fits
  {
    uint32_t at = hole_at;
    for (int t0 = lo; t0 < min(hi, n_new); t0 += kTile) {
      const int j0 = t0 + tid * kVec;
      const uint32_t keep = j0 < hi ? keep4[(j0 - lo) / kVec] : 0;
      const uint32_t hole = ~keep & below_bits(j0) & in_bits(j0);
      uint32_t total;
      uint32_t i = at + block_scan(__popc(hole), s, &total);
      at += total;
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        if (hole >> v & 1u) p.from_slot[row + n_new + i++] = j0 + v;
    }
  }
  __threadfence();
  sync();
  // kept slots below n_new keep their key; a mover's key goes to its hole
  {
    uint32_t at = mover_at;
    for (int t0 = lo; t0 < hiN; t0 += kTile) {
      const int j0 = t0 + tid * kVec;
      const uint32_t keep = j0 < hi ? keep4[(j0 - lo) / kVec] : 0;
      const uint32_t mover = keep & ~below_bits(j0);
      uint32_t total;
      uint32_t i = at + block_scan(__popc(mover), s, &total);
      at += total;
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        if (!(keep >> v & 1u)) continue;
        const int j = j0 + v;
        int to = j;
        if (mover >> v & 1u) to = __ldcg(&p.from_slot[row + n_new + i++]);
        p.from_slot[row + to] = j;
        if (p.weights_out) p.weights_out[row + to] = w[j];
        if (p.pos_out) p.pos_out[row + to] = pos[j];
      }
    }
  }
  sync();
  for (int j = max(lo, n_new) + tid; j < hi; j += kNT) {
    p.from_slot[row + j] = -1;
    if (p.weights_out) p.weights_out[row + j] = 0.f;
    if (p.pos_out) p.pos_out[row + j] = -1;
  }
  if (rank == 0 && tid == 0) p.new_len[b] = n_new;
}

// ------------------------------------------------------------------- the move

constexpr int kMoveThreads = 256;

__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// E: bytes of an element.
template <int E>
__global__ void __launch_bounds__(kMoveThreads)
kv_move_kernel(uint4* c_kv, uint4* k_pe, int num_pages, const int32_t* __restrict__ table,
               int max_pages, const int32_t* __restrict__ from_slot,
               const int32_t* __restrict__ new_len, int32_t* __restrict__ req_status) {
  constexpr int cw = kDc * E / 16, kw = kDr * E / 16;  // 16-byte words of a row
  __shared__ int2 move[kPage];  // pool rows: destination, source
  __shared__ int n_moves;
  const int b = blockIdx.y, page = blockIdx.x, tid = threadIdx.x;
  const int cap = max_pages * kPage;
  const int n = new_len[b];
  if (n < 0 || n > cap) {
    if (page == 0 && tid == 0 && req_status) req_status[b] = VA_ERR_INVALID_ARG;
    return;
  }
  if (page * kPage >= n) return;
  if (tid == 0) n_moves = 0;
  __syncthreads();
  if (tid < kPage) {
    const int d = page * kPage + tid;
    const int f = d < n ? from_slot[(size_t)b * cap + d] : d;
    if (f != d) {
      const int32_t* t = table + (size_t)b * max_pages;
      const int pd = t[page];
      const int ps = f >= n && f < cap ? t[f / kPage] : -1;
      if (pd < 0 || pd >= num_pages || ps < 0 || ps >= num_pages) {
        if (req_status) req_status[b] = VA_ERR_INVALID_ARG;
      } else {
        move[atomicAdd(&n_moves, 1)] =
            make_int2(pd * kPage + tid, ps * kPage + f % kPage);
      }
    }
  }
  __syncthreads();
  // kWords words of each thread are in flight
  constexpr int per = cw + kw, kWords = 4;
  const int total = n_moves * per;
  for (int i0 = tid; i0 < total; i0 += kMoveThreads * kWords) {
    uint4 v[kWords];
    uint4* to[kWords];
#pragma unroll
    for (int u = 0; u < kWords; ++u) {
      const int i = i0 + u * kMoveThreads;
      to[u] = nullptr;
      if (i < total) {
        const int2 m = move[i / per];
        const int x = i % per;
        to[u] = x < cw ? c_kv + (size_t)m.x * cw + x : k_pe + (size_t)m.x * kw + (x - cw);
        v[u] = load_once(x < cw ? c_kv + (size_t)m.y * cw + x : k_pe + (size_t)m.y * kw + (x - cw));
      }
    }
#pragma unroll
    for (int u = 0; u < kWords; ++u)
      if (to[u]) *to[u] = v[u];
  }
}

}  // namespace

cudaError_t launch_evict_plan(const va_evict_args& a, int sms, cudaStream_t st) {
  PlanParams p;
  p.weights = a.weights;
  p.kv_len = a.kv_len;
  p.budget = a.budget;
  p.path = a.path;
  p.accept_len = a.accept_len;
  p.pos = a.pos;
  p.cap = a.capacity;
  p.T = a.T;
  p.n_sink = a.n_sink;
  p.n_recent = a.n_recent;
  p.new_len = a.new_len;
  p.from_slot = a.from_slot;
  p.weights_out = a.weights_out;
  p.pos_out = a.pos ? a.pos_out : nullptr;
  p.req_status = a.req_status;
  // The cluster of a request doubles while its CTAs (one an SM) have more than a tile
  // each and twice as many still have an SM each, or while their keep bits would not fit.
  int C = 1;
  while (C < kMaxCluster &&
         ((2LL * a.B * C <= sms && (long long)a.capacity > (long long)kTile * C) ||
          slots_per_cta(a.capacity, C) / kVec > kMaxKeepBytes))
    C *= 2;
  const int slots = slots_per_cta(a.capacity, C);
  if (slots / kVec > kMaxKeepBytes) return cudaErrorNotSupported;
  const int run = (slots + kNT - 1) / kNT;
  const bool held = run <= kMaxRun;
  const int bytes = held ? kNT * run * 4 + kNT * run / 8 + 4 : slots / kVec;
  auto* kernel = held ? evict_plan_kernel<true> : evict_plan_kernel<false>;
  if (bytes > 20 * 1024) {  // past the default limit, beside the static arrays
    static std::atomic<bool> done[2][kMaxDevices];
    cudaError_t e = raise_smem_once(
        kernel, held ? kNT * kMaxRun * 4 + kNT * kMaxRun / 8 + 4 : kMaxKeepBytes, done[held]);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * C));
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p, C);
}

cudaError_t launch_kv_move(void* c_kv, void* k_pe, int elem_bytes, int num_pages,
                           const int32_t* page_table, int B, int max_pages,
                           const int32_t* from_slot, const int32_t* new_len, int32_t* req_status,
                           cudaStream_t st) {
  const dim3 grid((unsigned)max_pages, (unsigned)B);
  auto* kernel = elem_bytes == 4 ? kv_move_kernel<4> : elem_bytes == 2 ? kv_move_kernel<2> : kv_move_kernel<1>;
  kernel<<<grid, kMoveThreads, 0, st>>>(static_cast<uint4*>(c_kv), static_cast<uint4*>(k_pe), num_pages,
                                        page_table, max_pages, from_slot, new_len, req_status);
  return cudaGetLastError();
}

}  // namespace va
