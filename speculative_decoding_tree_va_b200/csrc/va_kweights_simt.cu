// Key weights on CUDA cores (on request, and for the largest fp32 caches), and the
// join of row splits that the tensor-core kernel shares.
//
//   w_j = sum over counted rows r, j visible to r, of
//         exp(scale q_r . k_j - lse_r)
// With the log-sum-exp known the softmax needs no second statistic: one
// product tile [128 keys x 128 rows] over the 576 dims, then the exponentials,
// then a sum over the tile's rows that stays in the registers that hold its
// keys.  The rows of a request are counted rows only: row r is head r % H of
// the (r / H)-th accepted node.
//
// A CTA owns 128 keys and, when few key tiles would leave SMs idle, a share
// of the row blocks (split); splits write partial sums that the join adds in
// split order.  Bound by the FFMA rate: 576 multiply-adds per row and key.
#include "va_common.cuh"
#include "va_kweights.cuh"

namespace va {
namespace {

constexpr int kThreads = 256;
constexpr int kBK = 16;              // dims per step
constexpr int kPitch = kKwKeys + 4;  // shared row of one dim

// Two buffers of a step; the keys' sums at the end share the space.
struct Stage {
  float k[2][kBK][kPitch];
  float q[2][kBK][kPitch];
};
static_assert(sizeof(Stage) >= kThreads / 16 * kKwKeys * sizeof(float), "sums fit");

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 consecutive elements at p (16-byte aligned for fp32, else to 8 elements).
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_fp8_e4m3* p, float (&x)[8]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t c = (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1)));
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <typename TQ, typename TK>
__global__ void __launch_bounds__(kThreads, 2) kweights_simt_kernel(const KwParams p) {
  __shared__ __align__(16) Stage st;
  __shared__ float sLse[kKwRows];
  __shared__ uint64_t sMask[kKwRows][2];
  float (*sSum)[kKwKeys] = reinterpret_cast<float(*)[kKwKeys]>(&st);
  const int tid = threadIdx.x;
  const int b = blockIdx.y, split = blockIdx.z, j0 = blockIdx.x * kKwKeys;
  const KwRequest rq = kw_request(p, b);
  if (!rq.ok || j0 >= rq.kv_len) {
    if (!rq.ok && blockIdx.x == 0 && split == 0 && tid == 0 && p.req_status)
      p.req_status[b] = VA_ERR_INVALID_ARG;
    return;
  }
  const int P = rq.kv_len - p.T;
  if (rq.bad_accept && blockIdx.x == 0 && split == 0 && tid == 0 && p.req_status)
    p.req_status[b] = VA_ERR_INVALID_ARG;
  const int R = rq.nodes * p.H;
  const int blocks = (R + kKwRows - 1) / kKwRows;
  const int blk0 = (int)((long long)blocks * split / p.splits);
  const int blk1 = (int)((long long)blocks * (split + 1) / p.splits);

  // this thread stages key (and row) tid & 127, dims 8 (tid >> 7) .. +7 of a step
  const int sr = tid & 127, sd = (tid >> 7) * 8;
  const int key = j0 + sr;
  const int krow = kw_pool_row(p, b, rq.kv_len, key);
  if (krow < 0 && key < rq.kv_len && split == 0 && p.req_status)
    p.req_status[b] = VA_ERR_INVALID_ARG;  // page index out of range
  const TK* kc = reinterpret_cast<const TK*>(p.c_kv) + (size_t)max(krow, 0) * kDc;
  const TK* kp = reinterpret_cast<const TK*>(p.k_pe) + (size_t)max(krow, 0) * kDr;
  const int tx = tid & 15, ty = tid >> 4;
  float ksum[8] = {};

  for (int blk = blk0; blk < blk1; ++blk) {
    const int row = blk * kKwRows + sr;
    int node;
    const int g = kw_query_row(p, b, rq, row, &node);  // -1: adds nothing
    const TQ* qn = reinterpret_cast<const TQ*>(p.q_nope) + (size_t)max(g, 0) * kDc;
    const TQ* qp = reinterpret_cast<const TQ*>(p.q_pe) + (size_t)max(g, 0) * kDr;
    if (tid < kKwRows) kw_row_info(p, b, g, node, &sLse[sr], sMask[sr]);

    float x[8];
    auto fetch_k = [&](int d0) {
      const int d = d0 + sd;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (krow >= 0) {
        if (d < kDc) load8(kc + d, x); else load8(kp + d - kDc, x);
      }
    };
    auto fetch_q = [&](int d0) {
      const int d = d0 + sd;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (g >= 0) {
        if (d < kDc) load8(qn + d, x); else load8(qp + d - kDc, x);
      }
    };
    auto put = [&](float (&to)[kBK][kPitch]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) to[sd + i][sr] = x[i];
    };
    // A step's keys are loaded while its first half is multiplied and its rows while
    // the second is, so that 8 registers hold them; the operands of a dim are read
    // from shared memory one dim ahead, because 4 warps a scheduler do not hide it.
    float acc[8][8] = {};  // [row][key]
    fetch_k(0);
    put(st.k[0]);
    fetch_q(0);
    put(st.q[0]);
    __syncthreads();
    for (int s = 0; s < kDqk / kBK; ++s) {
      const int cur = s & 1;
      const bool more = s + 1 < kDqk / kBK;
      float k[2][8], q[2][8];
      auto operands = [&](int d) {
        float* kd = k[d & 1];
        float* qd = q[d & 1];
        *reinterpret_cast<float4*>(kd) = *reinterpret_cast<const float4*>(&st.k[cur][d][tx * 4]);
        *reinterpret_cast<float4*>(kd + 4) = *reinterpret_cast<const float4*>(&st.k[cur][d][64 + tx * 4]);
        *reinterpret_cast<float4*>(qd) = *reinterpret_cast<const float4*>(&st.q[cur][d][ty * 4]);
        *reinterpret_cast<float4*>(qd + 4) = *reinterpret_cast<const float4*>(&st.q[cur][d][64 + ty * 4]);
      };
      if (more) fetch_k((s + 1) * kBK);
      operands(0);
#pragma unroll
      for (int d = 0; d < kBK; ++d) {
        if (d + 1 < kBK) operands(d + 1);
        if (d == kBK / 2 && more) {
          put(st.k[cur ^ 1]);
          fetch_q((s + 1) * kBK);
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[r][c] = fmaf(q[d & 1][r], k[d & 1][c], acc[r][c]);
      }
      if (more) put(st.q[cur ^ 1]);
      __syncthreads();
    }
    const bool tail = j0 + kKwKeys > P;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int rr = (r < 4 ? 0 : 60) + ty * 4 + r;
      const float l = sLse[rr];
      if (l == INFINITY) continue;  // adds nothing, not to a key of NaN either
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int kk = (c < 4 ? 0 : 60) + tx * 4 + c;
        float w = ex2f(fmaf(acc[r][c], p.scale, -l) * kLog2e);
        if (tail) {
          const int nd = j0 + kk - P;
          if (nd >= 0 && !(nd < p.T && ((sMask[rr][nd >> 6] >> (nd & 63)) & 1ull))) w = 0.f;
        }
        ksum[c] += w;
      }
    }
    __syncthreads();  // sLse and sMask are rewritten by the next block
  }

#pragma unroll
  for (int c = 0; c < 8; ++c) sSum[ty][(c < 4 ? 0 : 60) + tx * 4 + c] = ksum[c];
  __syncthreads();
  if (tid < kKwKeys && key < rq.kv_len) {
    float w = 0.f;
#pragma unroll
    for (int y = 0; y < kThreads / 16; ++y) w += sSum[y][tid];
    kw_store(p, b, split, key, krow >= 0 ? w : 0.f);
  }
}

// Adds the splits' (or parts') partial sums, in their order, to the decayed weights.
__global__ void __launch_bounds__(64) kweights_join_kernel(const KwParams p) {
  const int b = blockIdx.y;
  const int j = blockIdx.x * 64 + threadIdx.x;
  const KwRequest rq = kw_request(p, b);
  if (!rq.ok || j >= rq.kv_len) return;
  const size_t cap = (size_t)p.max_pages * kPage;
  const size_t at = (size_t)b * cap + j, step = (size_t)p.B * cap;
  const float old = p.weights_in ? p.decay * p.weights_in[at] : 0.f;
  float w = 0.f;
  const int parts = kw_parts(p, rq);
  for (int s0 = 0; s0 < parts; s0 += 8) {  // 8 loads in flight, added in order
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = s0 + u < parts ? p.part[(s0 + u) * step + at] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) w += v[u];
  }
  p.weights[at] = old + w;
}

}  // namespace

cudaError_t launch_kweights_join(const KwParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.max_pages * kPage + 63) / 64), (unsigned)p.B);
  kweights_join_kernel<<<grid, 64, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kweights_simt(const va_key_weight_args& a, const KwParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.max_pages * kPage + kKwKeys - 1) / kKwKeys), (unsigned)p.B,
                  (unsigned)p.splits);
  const bool fp8 = a.flags & VA_FLAG_KV_FP8_E4M3;
  const bool f32 = a.dtype == VA_F32;
  auto* k = f32 ? (fp8 ? kweights_simt_kernel<float, __nv_fp8_e4m3> : kweights_simt_kernel<float, float>)
                : (fp8 ? kweights_simt_kernel<__nv_bfloat16, __nv_fp8_e4m3>
                       : kweights_simt_kernel<__nv_bfloat16, __nv_bfloat16>);
  k<<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace va
