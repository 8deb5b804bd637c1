// What the key-weight kernels share: the counted rows of a request, their
// log-sum-exp and masks, the page lookup and the store of a key's sum.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "va_common.cuh"
#include "va_kweights_plan.cuh"

namespace va {

constexpr int kKwKeys = 128;  // keys of a CTA's tile
constexpr int kKwRows = 128;  // rows of a block on CUDA cores

struct KwParams {
  const void* q_nope;
  const void* q_pe;
  const void* c_kv;
  const void* k_pe;
  const int32_t* page_table;
  const int32_t* kv_len;
  const uint64_t* tree_mask;
  const float* lse;
  const int32_t* path;
  const int32_t* accept_len;
  const float* weights_in;
  float* weights;
  float* part;  // [splits, B, 64 max_pages] when splits > 1; kw_parts of them in use
  int32_t* req_status;
  int B, H, T, max_pages, num_pages, splits;
  int stay, pass;  // tensor cores: rows that make one block, rows of a block (CUDA cores: 0)
  float scale;  // an FP8 cache's scale included
  float decay;
};

#ifdef __CUDACC__

struct KwRequest {
  int kv_len, nodes;
  bool ok;          // kv_len in range
  bool bad_accept;  // accept_len out of range: no row counts
};

__device__ __forceinline__ KwRequest kw_request(const KwParams& p, int b) {
  KwRequest r;
  r.kv_len = p.kv_len[b];
  r.ok = r.kv_len >= p.T && r.kv_len <= p.max_pages * kPage;
  r.nodes = p.path ? p.accept_len[b] : p.T;
  r.bad_accept = r.nodes < 0 || r.nodes > p.T;
  if (r.bad_accept) r.nodes = 0;
  return r;
}

// Partial sums that a request's keys have: on CUDA cores one from every split, on tensor
// cores one from each part of a tile.
__device__ __forceinline__ int kw_parts(const KwParams& p, const KwRequest& rq) {
  if (p.pass == 0) return p.splits;
  return kwplan::tile_parts(p.splits, kwplan::row_blocks(rq.nodes * p.H, p.stay, p.pass));
}

// Pool row of logical key `key`, -1 past kv_len or for a page outside the pool.
__device__ __forceinline__ int kw_pool_row(const KwParams& p, int b, int kv_len, int key) {
  if (key >= kv_len) return -1;
  const int pg = p.page_table[(size_t)b * p.max_pages + key / kPage];
  return pg < 0 || pg >= p.num_pages ? -1 : pg * kPage + key % kPage;
}

// Query row of the request's counted row r (its node in *node), or -1 where
// it adds nothing: past the end, an entry outside the tree (the request is
// flagged), an absent node, an empty row.
__device__ __forceinline__ int kw_query_row(const KwParams& p, int b, const KwRequest& rq, int r,
                                            int* node) {
  *node = 0;
  if (r >= rq.nodes * p.H) return -1;
  const int i = r / p.H;
  const int n = p.path ? p.path[(size_t)b * p.T + i] : i;
  if (n < 0 || n >= p.T) {
    if (p.req_status) p.req_status[b] = VA_ERR_INVALID_ARG;
    return -1;
  }
  *node = n;
  const uint64_t* m = p.tree_mask + ((size_t)b * p.T + n) * ((p.T + 63) >> 6);
  if (!mask_bit(m, n)) return -1;
  const int g = (int)(((long long)b * p.T + n) * p.H + (r - i * p.H));
  return p.lse[g] == -INFINITY ? -1 : g;
}

// Log-sum-exp (+inf where the row adds nothing) and mask words of a row.
__device__ __forceinline__ void kw_row_info(const KwParams& p, int b, int g, int node, float* lse,
                                            uint64_t* mask) {
  *lse = INFINITY;
  mask[0] = mask[1] = 0;
  if (g < 0) return;
  const int W = (p.T + 63) >> 6;
  const uint64_t* m = p.tree_mask + ((size_t)b * p.T + node) * W;
  *lse = p.lse[g];
  mask[0] = m[0];
  if (W > 1) mask[1] = m[1];
}

__device__ __forceinline__ void kw_store(const KwParams& p, int b, int split, int key, float w) {
  const size_t cap = (size_t)p.max_pages * kPage;
  const size_t at = (size_t)b * cap + key;
  if (p.splits > 1) p.part[((size_t)split * p.B + b) * cap + key] = w;
  else p.weights[at] = (p.weights_in ? p.decay * p.weights_in[at] : 0.f) + w;
}

#endif  // __CUDACC__

cudaError_t launch_kweights_simt(const va_key_weight_args& a, const KwParams& p, cudaStream_t st);
cudaError_t launch_kweights_join(const KwParams& p, cudaStream_t st);
// The tensor-core kernel.  Its workspace holds the counted rows where they must be
// laid out or converted first; the partial sums follow.
bool kweights_on_tc(const va_key_weight_args& a);
int kweights_tc_splits(const va_key_weight_args& a, int sms);
void kweights_tc_blocks(const va_key_weight_args& a, int* stay, int* pass);
size_t kweights_tc_workspace(const va_key_weight_args& a);
cudaError_t launch_kweights_tc(const va_key_weight_args& a, const KwParams& p, int sms,
                               cudaStream_t st);

}  // namespace va
