// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits: the drafter's per-depth top-k and the target's greedy tokens.
//
// With m the row's maximum, c = scale log2(e) and y_v = c x_v - r, where r is
// c m rounded to fp32 and eps = c m - r (exact, a multiply-add away):
//   Z = sum 2^y_v     S = sum 2^y_v y_v     ln Z' = ln Z - eps ln2
//   lse = scale m + ln Z'     lp_v = scale (x_v - m) - ln Z'
//   entropy = ln2 (log2 Z - S / Z)
// y_v is one rounding of its value, so a common r costs no accuracy.  A thread
// holds (m, Z, S) of what it has read and rescales them once per tile of its
// loads; two elements go through each addition and multiply-add (.f32x2).
// |eps| has to stay small for 2^eps to be in range: with X the power of two for
// which 2^23 <= c X < 2^24, |eps| <= 1/2 for |m| <= X, and c X is exact.  Logits below
// -X (masks, a tile's padding) are read as -X, so a thread of nothing else has y_v = 0
// and finite sums, which its first rescaling drops, because the row's maximum is
// at least 200 / c above: less than 2^-200 is left of them.  The rare row whose
// maximum is nearer to -X, or above X, is summed again element by element with
// y_v = c (x_v - m) and eps = 0; where X is the largest power taken, 2^100 (scales
// below 2^-92), that is every row.
//
// Top K: a candidate is a 64-bit key, the logit in order-preserving bits over
// the complement of its index, so that equal logits order by lower index.
// Each warp keeps a list in shared memory.  The K-th largest of its lanes'
// maxima over its first tile is a lower bound of the row's K-th logit, so a
// lane pushes only the elements of a later tile that reach the largest bound
// any warp has found; a list that grows past kCut is cut down to its K largest,
// which raises the bound.  Warps wait for each other only at the row's end.
// (Loading a tile ahead costs registers and with them a CTA per SM: 124 us
// against 126 for 2112 rows of 131072, but 16.5 against 14.4 for 960 of 4096.)
//
// Bound by the one read of the logits from HBM; the exponentials (16 a clock
// and SM, 11.5 logits of bf16 arrive a clock) come next.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "va_common.cuh"

namespace va {
namespace {

constexpr int kNT = 256;     // threads per CTA
constexpr int kWarps = kNT / 32;
constexpr int kU = 4;        // 16-byte vectors a lane holds per tile
constexpr int kCut = 64;     // candidates of a warp before they are cut down
constexpr int kCap = 128;    // room for them
constexpr int kMaxCluster = 8;
static_assert(kMaxCluster * VA_MAX_TOPK <= kNT && kWarps * VA_MAX_TOPK <= kNT, "cut_down");
constexpr unsigned kFull = 0xffffffffu;
constexpr float kApart = 200.f;    // binary orders from -X from which a row's maximum is not near it
constexpr float kFloor = -1.0e4f;  // 2^kFloor = 0; keeps 0 * y finite

struct LpParams {
  const void* logits;
  const int32_t* tokens;
  long long ld;
  int V, G, K;
  float scale;
  float far;                         // X above, also as two bf16 of -X
  uint32_t neg_far2;
  float* lse;
  float* entropy;
  float* tok_lp;
  int32_t* top_ids;
  float* top_lp;
  double* top_lp64;
  int32_t* row_status;
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Bits that order like the value (-0 like +0); NaN never reaches the output.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t make_key(float x, int idx) {
  return ((uint64_t)order_bits(x) << 32) | (uint32_t)~idx;
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// Address of `p` (this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float remote_f32(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t remote_u64(const uint64_t* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Two fp32 values in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

template <typename T> struct Vec;  // a 16-byte vector of logits
template <> struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  template <int U> static __device__ __forceinline__ float largest(const uint4 (&v)[U]) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[4];
      unpack(v[u], x);
      m = max_nan(m, max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])));
    }
    return m;
  }
  // the same with nothing below -X
  static __device__ __forceinline__ void unpack_near(const uint4& v, const LpParams& p, float (&x)[4]) {
    unpack(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = max_nan(x[i], -p.far);
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ void split(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    split(v.x, x[0], x[1]);
    split(v.y, x[2], x[3]);
    split(v.z, x[4], x[5]);
    split(v.w, x[6], x[7]);
  }
  template <int U> static __device__ __forceinline__ float largest(const uint4 (&v)[U]) {
    uint32_t m = kNegInf;
#pragma unroll
    for (int u = 0; u < U; ++u) m = max2(m, max2(max2(v[u].x, v[u].y), max2(v[u].z, v[u].w)));
    float a, b;
    split(m, a, b);
    return max_nan(a, b);
  }
  static __device__ __forceinline__ void unpack_near(const uint4& v, const LpParams& p, float (&x)[8]) {
    const uint32_t far = p.neg_far2;
    unpack(make_uint4(max2(v.x, far), max2(v.y, far), max2(v.z, far), max2(v.w, far)), x);
  }
};

// c (x - m) - z for x <= m finite or -inf.  Where x - m is past fp32's range the
// products are not both: with c x and c m each rounded it is as near, relative to itself.
__device__ __forceinline__ float below(float x, float m, float c, float z) {
  const float d = x - m;
  return d == -INFINITY && x > -INFINITY ? fmaf(x, c, -fmaf(m, c, z)) : fmaf(d, c, -z);
}

// Online sums of one thread: maximum, Z and S relative to it (`Far`: of the
// second way above).
struct Sums {
  float m, z = 0.f, s = 0.f;
  template <bool Far>
  __device__ __forceinline__ void raise(float to, float c) {  // to >= m, or NaN
    const float way = Far ? below(m, to, c, 0.f) : __fmul_rn(m, c) - __fmul_rn(to, c);
    const float d = max_nan(way, kFloor);
    const float f = ex2f(d);
    s = f * fmaf(z, d, s);
    z *= f;
    m = to;
  }
  template <bool Far>
  __device__ __forceinline__ void join(const Sums& o, float c) {
    Sums b = o;
    const float to = max_nan(m, b.m);
    raise<Far>(to, c);
    b.raise<Far>(to, c);
    z += b.z;
    s += b.s;
  }
};

// Cuts cand[0, n), n <= kNT, to its K largest keys, descending, in cand[0, K)
// (0 where there are fewer).  Called by the whole CTA; the keys other than 0
// are distinct.
__device__ void cut_down(uint64_t* cand, int n, int K) {
  const int tid = threadIdx.x;
  const uint64_t k = tid < n ? cand[tid] : 0;
  int r = 0;
  if (k)
    for (int i = 0; i < n; ++i) r += cand[i] > k;
  __syncthreads();
  if (tid < K) cand[tid] = 0;
  __syncthreads();
  if (k && r < K) cand[r] = k;
  __syncthreads();
}

// The same by one warp, n <= kCap.
__device__ void warp_cut(uint64_t* cand, int n, int K) {
  constexpr int kPer = kCap / 32;
  const int lane = threadIdx.x & 31;
  uint64_t k[kPer];
  int r[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    k[q] = lane + 32 * q < n ? cand[lane + 32 * q] : 0;
    r[q] = 0;
  }
  for (int i = 0; i < n; ++i) {
    const uint64_t o = cand[i];
#pragma unroll
    for (int q = 0; q < kPer; ++q) r[q] += o > k[q];
  }
  __syncwarp();
  if (lane < K) cand[lane] = 0;
  __syncwarp();
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (k[q] && r[q] < K) cand[r[q]] = k[q];
  __syncwarp();
}

// One row per cluster: CTA `rank` of C reads the rank-th part of the row's
// vectors, rank 0 joins the parts over distributed shared memory.
template <typename T>
__global__ void __launch_bounds__(kNT, 4) logprobs_kernel(const LpParams p, int C) {
  using VT = Vec<T>;
  constexpr int N = VT::N;
  constexpr int kStep = kWarps * kU * 32;  // vectors of the CTA's tiles side by side
  __shared__ uint64_t lists[kWarps][kCap];
  __shared__ uint64_t kth[kWarps];         // a warp's K-th key so far
  __shared__ uint64_t cand[kNT];
  __shared__ int counts[kWarps], total;
  __shared__ uint32_t bound;               // order_bits of the largest bound
  __shared__ float wm[kWarps], wz[kWarps], ws[kWarps];
  __shared__ float part[3], whole[3];      // this CTA's sums, the row's
  __shared__ float fin[2];                 // the row's maximum and ln Z
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  const long long row = blockIdx.x / C;
  const int V = p.V, K = p.K;
  const T* x0 = reinterpret_cast<const T*>(p.logits) + row * p.ld;
  // vectors are taken at 16-byte boundaries: element v of the row is element
  // v + off of the aligned base, and only a row's first and last vector may
  // reach past it (those are read element by element)
  const int off = (int)(((uintptr_t)x0 & 15) / sizeof(T));
  const T* base = x0 - off;
  const int nv = (int)(((long long)V + off + N - 1) / N);
  const int per = (nv + C - 1) / C;
  const int v0 = min(nv, (int)rank * per), v1 = min(nv, v0 + per);
  const int w0 = v0 + warp * kU * 32;      // this warp's first tile
  const float c = fminf(p.scale * kLog2e, FLT_MAX);

  if (tid == 0) { bound = order_bits(-INFINITY); total = 0; }
  if (lane == 0) { counts[warp] = 0; kth[warp] = 0; }
  __syncthreads();

  const int whole_to = min(v1, (V + off) / N);  // vectors [off > 0, whole_to) lie in the row
  auto load = [&](int t0, uint4 (&raw)[kU]) {
    if (t0 >= (off > 0) && t0 + kU * 32 <= whole_to) {
      const uint4* at = reinterpret_cast<const uint4*>(base) + t0 + lane;
#pragma unroll
      for (int u = 0; u < kU; ++u) raw[u] = load_stream(at + u * 32);
      return;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = t0 + u * 32 + lane;
      if (j < v1 && (j > 0 || off == 0) && (j + 1) * N - off <= V) {
        raw[u] = load_stream(reinterpret_cast<const uint4*>(base) + j);
      } else {
        raw[u] = make_uint4(VT::kNegInf, VT::kNegInf, VT::kNegInf, VT::kNegInf);
        if (j < v1) {
          T e[N];
          *reinterpret_cast<uint4*>(e) = raw[u];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int v = j * N + i - off;
            if (v >= 0 && v < V) e[i] = x0[v];
          }
          raw[u] = *reinterpret_cast<uint4*>(e);
        }
      }
    }
  };
  // calls f(x, index) for this lane's elements of a tile that are in the row; read
  // again from memory, element by element: for the rare paths, in little code
  auto each_again = [&](int t0, auto f) {
#pragma unroll 1
    for (int u = 0; u < kU; ++u) {
      const int j = t0 + u * 32 + lane;
#pragma unroll 1
      for (int i = 0; i < N; ++i) {
        const int v = j * N + i - off;
        if (j < v1 && v >= 0 && v < V) f(to_f32(x0[v]), v);
      }
    }
  };

  Sums acc;
  acc.m = -p.far;
  const uint64_t c2 = pack2(c, c);
  for (int t0 = w0; t0 < v1; t0 += kStep) {
    uint4 raw[kU];
    load(t0, raw);
    const float mt = VT::largest(raw);
    if (!(mt <= acc.m)) acc.raise<false>(mt, c);
    {
      const float r = __fmul_rn(acc.m, c);
      const uint64_t nr2 = pack2(-r, -r);
      uint64_t z2 = pack2(acc.z, 0.f), s2 = pack2(acc.s, 0.f);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float x[N];
        VT::unpack_near(raw[u], p, x);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const uint64_t y2 = fma2(pack2(x[i], x[i + 1]), c2, nr2);
          float ya, yb;
          unpack2(y2, ya, yb);
          const uint64_t e2 = pack2(ex2f(ya), ex2f(yb));
          z2 = add2(z2, e2);
          s2 = fma2(e2, y2, s2);
        }
      }
      float za, zb, sa, sb;
      unpack2(z2, za, zb);
      unpack2(s2, sa, sb);
      acc.z = za + zb;
      acc.s = sa + sb;
    }
    if (K > 0) {
      const float top = mt == mt ? mt : -INFINITY;
      if (t0 == w0) {  // the K-th largest of the lanes' maxima, or a smaller one
        uint32_t left = order_bits(top), kth_top = 0;
        for (int r = 0; r < K; ++r) {
          kth_top = __reduce_max_sync(kFull, left);
          if (left == kth_top) left = 0;
        }
        if (lane == 0) atomicMax(&bound, kth_top);
        __syncwarp();
      }
      const float b = order_value(*(volatile uint32_t*)&bound);
      if (__any_sync(kFull, top >= b)) {
        const uint64_t floor = kth[warp];
        if (top >= b) {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int j = t0 + u * 32 + lane;
            const int at = j * N - off;
            float x[N];
            VT::unpack(raw[u], x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              if (x[i] >= b && j < v1 && at + i >= 0 && at + i < V) {
                const uint64_t k = make_key(x[i], at + i);
                if (k > floor) {
                  const int n = atomicAdd(&counts[warp], 1);
                  if (n < kCap) lists[warp][n] = k;
                }
              }
            }
          }
        }
        if (K == 1 && top > b) atomicMax(&bound, order_bits(top));
        __syncwarp();
        const int n = *(volatile int*)&counts[warp];
        if (n > kCut) {
          if (n <= kCap) {
            warp_cut(lists[warp], n, K);
          } else {
            // More than fit (equal logits, or rows that rise): K rounds of the
            // largest key below the last one, of the list's and of the tile's,
            // which may hold the same key twice.
            uint64_t below = ~0ull, mine_at = 0;
            for (int r = 0; r < K; ++r) {
              uint64_t mine = 0;
              for (int i = lane; i < kCap; i += 32)
                if (lists[warp][i] < below && lists[warp][i] > mine) mine = lists[warp][i];
              each_again(t0, [&](float x, int v) {
                if (x >= b) {
                  const uint64_t k = make_key(x, v);
                  if (k < below && k > mine) mine = k;
                }
              });
              const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(mine >> 32));
              const uint32_t lo = __reduce_max_sync(
                  kFull, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0u);
              below = (uint64_t)hi << 32 | lo;
              if (lane == r) mine_at = below;
            }
            __syncwarp();
            if (lane < K) lists[warp][lane] = mine_at;
            __syncwarp();
          }
          if (lane == 0) {
            const uint64_t k = lists[warp][K - 1];
            counts[warp] = K;
            kth[warp] = k;
            atomicMax(&bound, (uint32_t)(k >> 32));
          }
          __syncwarp();
        }
      }
    }
  }
  if (K > 0) {
    // what reaches the final bound; where that is more than fits (equal logits),
    // each warp's K largest
    __syncthreads();
    const int n = counts[warp];
    for (int i = lane; i < n; i += 32) {
      const uint64_t k = lists[warp][i];
      if ((uint32_t)(k >> 32) >= bound) {
        const int at = atomicAdd(&total, 1);
        if (at < kNT) cand[at] = k;
      }
    }
    __syncthreads();
    int m = total;
    if (m > kNT) {
      warp_cut(lists[warp], n, K);
      if (lane < K) cand[warp * K + lane] = lists[warp][lane];
      m = kWarps * K;
      __syncthreads();
    }
    cut_down(cand, m, K);
  }

  // join the threads' sums in part[]: lanes, then warps
  auto join_cta = [&](auto far) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      Sums o;
      o.m = __shfl_xor_sync(kFull, acc.m, d);
      o.z = __shfl_xor_sync(kFull, acc.z, d);
      o.s = __shfl_xor_sync(kFull, acc.s, d);
      acc.join<far.value>(o, c);
    }
    if (lane == 0) { wm[warp] = acc.m; wz[warp] = acc.z; ws[warp] = acc.s; }
    __syncthreads();
    if (warp == 0) {
      Sums a;
      a.m = wm[lane % kWarps]; a.z = wz[lane % kWarps]; a.s = ws[lane % kWarps];
#pragma unroll
      for (int d = kWarps / 2; d > 0; d >>= 1) {
        Sums o;
        o.m = __shfl_xor_sync(kFull, a.m, d);
        o.z = __shfl_xor_sync(kFull, a.z, d);
        o.s = __shfl_xor_sync(kFull, a.s, d);
        a.join<far.value>(o, c);
      }
      if (lane == 0) { part[0] = a.m; part[1] = a.z; part[2] = a.s; }
    }
    if (C > 1) cluster_sync_all();  // part[] (and cand[0, K)) of every CTA are in place
    else __syncthreads();
  };
  join_cta(std::false_type{});
  float row_max = part[0];
  if (C > 1)
    for (int r = 0; r < C; ++r) row_max = max_nan(row_max, remote_f32(&part[0], r));
  const bool far =
      (row_max + p.far) * c < kApart || (row_max > p.far && row_max < INFINITY);
  if (far) {  // the same for all CTAs of the row: sum again, element by element
    acc.m = -FLT_MAX;
    acc.z = acc.s = 0.f;
    for (int t0 = w0; t0 < v1; t0 += kStep)
      each_again(t0, [&](float x, int) {
        if (x > acc.m) acc.raise<true>(x, c);
        const float y = max_nan(below(x, acc.m, c, 0.f), kFloor);
        const float e = ex2f(y);
        acc.z += e;
        acc.s = fmaf(e, y, acc.s);
      });
    if (C > 1) cluster_sync_all();  // the first sums have been read everywhere
    else __syncthreads();
    join_cta(std::true_type{});
  }
  if (C > 1) {
    if (rank == 0) {
      if (tid == 0) {
        Sums a;
        a.m = part[0]; a.z = part[1]; a.s = part[2];
        for (int r = 1; r < C; ++r) {
          Sums o;
          o.m = remote_f32(&part[0], r);
          o.z = remote_f32(&part[1], r);
          o.s = remote_f32(&part[2], r);
          if (far) a.join<true>(o, c);
          else a.join<false>(o, c);
        }
        whole[0] = a.m; whole[1] = a.z; whole[2] = a.s;
      }
      if (tid >= K && tid < C * K) cand[tid] = remote_u64(&cand[tid % K], tid / K);
    }
    cluster_sync_all();  // remote reads are done: the other CTAs may exit
    if (rank != 0) return;
    if (K > 0) cut_down(cand, C * K, K);
  } else if (tid == 0) {
    whole[0] = part[0]; whole[1] = part[1]; whole[2] = part[2];
  }
  __syncthreads();
  if (tid == 0) {
    const float m = whole[0], z = whole[1];
    const bool bad = !(z == z) || !(m == m) || m == INFINITY;
    const float eps = far ? 0.f : fmaf(m, c, -__fmul_rn(m, c));
    const float lnz = logf(z) - eps * kLn2;  // z = 0 (no finite logit): -inf
    fin[0] = m;
    fin[1] = bad ? NAN : lnz;
    if (p.lse) p.lse[row] = bad ? NAN : (z > 0.f ? fmaf(m, p.scale, lnz) : -INFINITY);
    if (p.entropy)
      p.entropy[row] = bad ? NAN : (z > 0.f ? fmaxf(logf(z) - kLn2 * (whole[2] / z), 0.f) : 0.f);
    if (bad && p.row_status) p.row_status[row] = VA_ERR_INVALID_ARG;
  }
  __syncthreads();
  const float m = fin[0], lnz = fin[1];
  const bool bad = !(lnz == lnz);
  const bool none = lnz == -INFINITY;
  for (int g = tid; g < p.G; g += kNT) {
    const int t = p.tokens[row * p.G + g];
    float lp = -INFINITY;
    if (t >= V) {
      lp = NAN;
      if (p.row_status) p.row_status[row] = VA_ERR_INVALID_ARG;
    } else if (t >= 0 && !none) {
      lp = below(to_f32(x0[t]), m, p.scale, lnz);
    }
    p.tok_lp[row * p.G + g] = bad ? NAN : lp;
  }
  if (tid < K) {
    const uint64_t k = cand[tid];
    const float x = order_value((uint32_t)(k >> 32));
    float lp = none ? -INFINITY : below(x, m, p.scale, lnz);
    if (bad) lp = NAN;
    p.top_ids[row * K + tid] = bad || k == 0 ? -1 : key_index(k);
    if (p.top_lp) p.top_lp[row * K + tid] = lp;
    if (p.top_lp64) p.top_lp64[row * K + tid] = (double)lp;
  }
}

template <typename T>
cudaError_t launch(const LpParams& p, int R, int C, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)R * C));
  cfg.blockDim = dim3(kNT);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p, C);
}

}  // namespace

cudaError_t launch_logprobs(const va_logprob_args& a, int sms, cudaStream_t st) {
  LpParams p;
  p.logits = a.logits;
  p.tokens = a.tokens;
  p.ld = a.ld;
  p.V = a.V;
  p.G = a.G;
  p.K = a.K;
  p.scale = a.scale;
  // at most 2^100, where c X may be less (a scale below 2^-77)
  int e;  // c = f 2^e, 1/2 <= f < 1
  frexpf(std::min(a.scale * kLog2e, FLT_MAX), &e);
  const int far_exp = std::min(24 - e, 100);
  p.far = ldexpf(1.f, far_exp);
  const uint32_t far_bits = (uint32_t)(127 + far_exp) << 7 | 0x8000u;
  p.neg_far2 = far_bits << 16 | far_bits;
  p.lse = a.lse;
  p.entropy = a.entropy;
  p.tok_lp = a.tok_lp;
  p.top_ids = a.top_ids;
  p.top_lp = a.top_lp;
  p.top_lp64 = a.top_lp64;
  p.row_status = a.row_status;
  // Few rows: the cluster of a row doubles while its CTAs have more than a tile each
  // and there are fewer than two CTAs for an SM.  So a CTA keeps at least half a tile,
  // and an SM gets fewer than four.
  const long long tile = (long long)kNT * kU * (a.dtype == VA_F32 ? 4 : 8);
  int C = 1;
  while (C < kMaxCluster && (long long)a.R * C < 2 * sms && (long long)a.V > tile * C) C *= 2;
  return a.dtype == VA_F32 ? launch<float>(p, a.R, C, st) : launch<__nv_bfloat16>(p, a.R, C, st);
}

}  // namespace va
