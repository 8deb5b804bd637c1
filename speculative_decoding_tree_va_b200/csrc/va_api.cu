// C ABI of libverifyattn: argument checks, split planning, dispatch.
// Every entry point validates on the host and returns a va_status before
// launching anything; the caller owns all device memory.
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdio>

#include "va_common.cuh"
#include "va_kweights.cuh"

namespace {

constexpr int kDefaultSms = 148;  // B200; used when no device can be queried
using va::kMaxDevices;
std::atomic<int> g_sm_count[kMaxDevices];  // 0 = not looked up yet

// SM count of the current device (the split planner's wave size), looked up
// once per device.  Without a usable device (host-only use of the planner)
// it is the B200's 148; the runtime error that lookup leaves is cleared.
int sm_count() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)cudaGetLastError();
    return kDefaultSms;
  }
  int n = g_sm_count[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2) {
    (void)cudaGetLastError();
    return kDefaultSms;
  }
  g_sm_count[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }


// Host-side checks shared by va_verify_attn / va_workspace_bytes.  A
// partials-only call (va_verify_attn_partials) writes neither out nor lse.
int check_args(const va_attn_args* a, bool needs_out = true) {
  if (!a) return VA_ERR_INVALID_ARG;
  if (a->dtype != VA_F32 && a->dtype != VA_BF16) return VA_ERR_INVALID_ARG;
  if (a->B < 0 || a->H < 1 || a->T < 1 || a->T > VA_MAX_QLEN) return VA_ERR_INVALID_ARG;
  if (a->page_size != VA_PAGE_SIZE) return VA_ERR_UNSUPPORTED;
  if (a->B > VA_MAX_BATCH) return VA_ERR_UNSUPPORTED;  // the launches' request axis (grid y)
  if (a->num_splits < 0 || a->num_splits > VA_MAX_SPLITS) return VA_ERR_INVALID_ARG;
  if (a->flags & ~(VA_FLAG_BF16_CUDA_CORES | VA_FLAG_TEST_STALL_MMA | VA_FLAG_KV_FP8_E4M3 |
                   VA_FLAG_TEST_STALL_COPIES))
    return VA_ERR_INVALID_ARG;
  if ((a->flags & VA_FLAG_TEST_STALL_COPIES) &&
      (a->dtype != VA_F32 || (a->flags & (VA_FLAG_KV_FP8_E4M3 | VA_FLAG_TEST_STALL_MMA))))
    return VA_ERR_INVALID_ARG;  // only the bulk-staged fp32 cache has the hook
  if ((a->flags & VA_FLAG_TEST_STALL_MMA) &&
      (!va::uses_tensor_cores(*a) || (a->flags & VA_FLAG_KV_FP8_E4M3)))
    return VA_ERR_INVALID_ARG;  // only the tensor-core kernel on a bf16 cache has the hook
  if ((a->flags & VA_FLAG_KV_FP8_E4M3) && !(a->kv_scale > 0.f && a->kv_scale <= FLT_MAX))
    return VA_ERR_INVALID_ARG;  // NaN, zero, negative or infinite cache scale
  if (!(a->scale == a->scale)) return VA_ERR_INVALID_ARG;  // NaN scale
  if (a->B == 0) return VA_OK;
  if (a->num_pages < 1 || a->max_pages < 1) return VA_ERR_INVALID_ARG;
  if ((long long)a->num_pages * VA_PAGE_SIZE > 0x7fffffffLL) return VA_ERR_UNSUPPORTED;
  if (va::widens_fp8_cache(*a) && (long long)a->B * a->max_pages * VA_PAGE_SIZE > 0x7fffffffLL)
    return VA_ERR_UNSUPPORTED;  // the widened pages are indexed like a pool
  const void* need16[] = {a->q_nope, a->q_pe, a->c_kv, a->k_pe};
  for (const void* p : need16)
    if (!p || !aligned(p, 16)) return VA_ERR_INVALID_ARG;
  if (needs_out && (!a->out || !aligned(a->out, 16))) return VA_ERR_INVALID_ARG;
  if (!a->page_table || !aligned(a->page_table, 4)) return VA_ERR_INVALID_ARG;
  if (!a->kv_len || !aligned(a->kv_len, 4)) return VA_ERR_INVALID_ARG;
  if (!a->tree_mask || !aligned(a->tree_mask, 8)) return VA_ERR_INVALID_ARG;
  if (needs_out && (!a->lse || !aligned(a->lse, 4))) return VA_ERR_INVALID_ARG;
  if (a->req_status && !aligned(a->req_status, 4)) return VA_ERR_INVALID_ARG;
  return VA_OK;
}

// Split count: the caller's, or (num_splits == 0) the smallest power of two
// that fills >= 90% of the last wave, keeping >= 1024 keys per split.  The
// host does not see kv_len, so the planner uses the page-table capacity as
// the key count.  A CUDA-core call with fewer segments than SMs uses the
// balanced plan instead (va_common.cuh), and its count is the plan's slots.
int plan_splits(const va_attn_args* a) {
  if (a->num_splits > 0) return a->num_splits;
  if (a->B == 0) return 1;
  const va::Balance bal = va::plan_balance(*a, sm_count());
  if (bal.G) return bal.slots;
  const long long rows = (long long)a->T * a->H;
  long long units_per_split, slots;
  const int sms = sm_count();
  if (va::uses_tensor_cores(*a)) {
    units_per_split = (long long)a->B * ((rows + 127) / 128);  // CTA pairs
    slots = sms / 2;
  } else {
    units_per_split = (long long)a->B * ((rows + 31) / 32);
    slots = sms;
  }
  const long long keys = (long long)a->max_pages * VA_PAGE_SIZE;
  for (int S = 1; S <= VA_MAX_SPLITS; S *= 2) {
    if (S > 1 && keys / S < 1024) return S / 2;
    const long long units = units_per_split * S;
    const long long waves = (units + slots - 1) / slots;
    if (units * 10 >= waves * slots * 9) return S;
  }
  return VA_MAX_SPLITS;
}

int check_key_weights(const va_key_weight_args* a) {
  if (!a) return VA_ERR_INVALID_ARG;
  if (a->dtype != VA_F32 && a->dtype != VA_BF16) return VA_ERR_INVALID_ARG;
  if (a->B < 0 || a->H < 1 || a->T < 1 || a->T > VA_MAX_QLEN) return VA_ERR_INVALID_ARG;
  if (a->page_size != VA_PAGE_SIZE || a->B > VA_MAX_BATCH) return VA_ERR_UNSUPPORTED;
  if (a->flags &
      ~(VA_FLAG_BF16_CUDA_CORES | VA_FLAG_KV_FP8_E4M3 | VA_FLAG_TEST_STALL_KEY_WEIGHTS))
    return VA_ERR_INVALID_ARG;
  if ((a->flags & VA_FLAG_TEST_STALL_KEY_WEIGHTS) && !va::kweights_on_tc(*a))
    return VA_ERR_INVALID_ARG;  // only the tensor-core kernel has the hook
  if ((a->flags & VA_FLAG_KV_FP8_E4M3) && !(a->kv_scale > 0.f && a->kv_scale <= FLT_MAX))
    return VA_ERR_INVALID_ARG;
  if (!(fabsf(a->scale) <= FLT_MAX) || !(fabsf(a->decay) <= FLT_MAX)) return VA_ERR_INVALID_ARG;
  if (a->B == 0) return VA_OK;
  if (a->num_pages < 1 || a->max_pages < 1) return VA_ERR_INVALID_ARG;
  if ((long long)a->num_pages * VA_PAGE_SIZE > 0x7fffffffLL ||
      (long long)a->max_pages * VA_PAGE_SIZE > 0x7fffffffLL - VA_SPLIT_ALIGN ||
      (long long)a->B * a->T * a->H > 0x7fffffffLL || (long long)a->T * a->H > (1 << 22))
    return VA_ERR_UNSUPPORTED;  // pool rows, slots, query rows and tile costs are 32-bit
  for (const void* p : {a->q_nope, a->q_pe, a->c_kv, a->k_pe})
    if (!p || !aligned(p, 16)) return VA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)a->page_table, (const void*)a->kv_len, (const void*)a->lse,
                        (const void*)a->weights})
    if (!p || !aligned(p, 4)) return VA_ERR_INVALID_ARG;
  if (!a->tree_mask || !aligned(a->tree_mask, 8)) return VA_ERR_INVALID_ARG;
  if ((a->path == nullptr) != (a->accept_len == nullptr)) return VA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)a->path, (const void*)a->accept_len,
                        (const void*)a->weights_in, (const void*)a->req_status})
    if (p && !aligned(p, 4)) return VA_ERR_INVALID_ARG;
  return VA_OK;
}

// Row splits of a key-weight call; on CUDA cores (grid z) a CTA's work is its key tile
// times its share of the row blocks; rows are split while the key tiles alone
// would leave SMs idle.  With an accepted path the host does not know its
// length: a path of the deepest tree is assumed, and splits without rows only
// write zeros.
int key_weight_splits(const va_key_weight_args* a) {
  if (va::kweights_on_tc(*a)) return va::kweights_tc_splits(*a, sm_count());
  const int sms = sm_count();
  const int nodes = a->path && a->T > VA_MAX_DEPTH + 1 ? VA_MAX_DEPTH + 1 : a->T;
  const long long blocks = ((long long)nodes * a->H + va::kKwRows - 1) / va::kKwRows;
  const long long tiles =
      (long long)a->B * (((long long)a->max_pages * VA_PAGE_SIZE + va::kKwKeys - 1) / va::kKwKeys);
  long long s = (2LL * sms + tiles - 1) / tiles;
  if (s > blocks) s = blocks;
  if (s > VA_MAX_SPLITS) s = VA_MAX_SPLITS;
  return s < 1 ? 1 : (int)s;
}

// Workspace of a call: the tensor-core kernel's rows, then the splits' sums.
size_t key_weight_rows(const va_key_weight_args* a) {
  return va::kweights_on_tc(*a) ? va::align256(va::kweights_tc_workspace(*a)) : 0;
}
size_t key_weight_workspace(const va_key_weight_args* a, int splits) {
  if (splits < 2) return key_weight_rows(a);
  return key_weight_rows(a) +
         va::align256((size_t)splits * a->B * a->max_pages * VA_PAGE_SIZE * sizeof(float));
}

}  // namespace

namespace va {

namespace {

// The attention launches of one call (after the FP8 widening pass and the
// request order, when they apply): splits sp of the partition, partials to
// o_part / lse_part (nullptr: a single split writing out / lse directly).
int launch_attention(const va_attn_args& a, SplitRange sp, const WorkspaceLayout& w, char* base,
                     float* o_part, float* lse_part, cudaStream_t st, const Balance& bal) {
  cudaError_t e;
  const int32_t* order = nullptr;
  if (uses_tensor_cores(a)) {
    int32_t* ord = reinterpret_cast<int32_t*>(base + w.order);
    e = launch_request_order(a.kv_len, a.B, ord, st);
    if (e != cudaSuccess) return VA_ERR_CUDA;
    order = ord;
  }
  if (widens_fp8_cache(a)) {
    // FP8 cache under bf16 queries: widen the pages the batch reads, then run
    // the tensor-core kernel on them with the cache scale folded into the
    // score scale and into the output normalisation.
    void* wc = base + w.w_ckv;
    void* wk = base + w.w_kpe;
    int32_t* wt = reinterpret_cast<int32_t*>(base + w.w_table);
    e = launch_kv_widen(a, wc, wk, wt, st);
    if (e != cudaSuccess) return VA_ERR_CUDA;
    va_attn_args b = a;
    b.c_kv = wc;
    b.k_pe = wk;
    b.page_table = wt;
    b.num_pages = a.B * a.max_pages;
    b.scale = a.scale * a.kv_scale;
    e = launch_attn_tc(b, sp, order, o_part, lse_part, st, a.kv_scale);
  } else if (uses_tensor_cores(a)) {
    e = launch_attn_tc(a, sp, order, o_part, lse_part, st, 1.f);
  } else {
    e = launch_attn_simt(a, sp, o_part, lse_part, st, bal);
  }
  if (e == cudaErrorNotSupported) return VA_ERR_UNSUPPORTED;
  if (e != cudaSuccess) return VA_ERR_CUDA;
  return VA_OK;
}

}  // namespace

int run_verify(const va_attn_args& a, int S, void* ws, cudaStream_t st) {
  const WorkspaceLayout w = workspace_layout(a, S);
  char* base = static_cast<char*>(ws);
  float* o_part = S > 1 ? reinterpret_cast<float*>(base + w.o_part) : nullptr;
  float* lse_part = S > 1 ? reinterpret_cast<float*>(base + w.lse_part) : nullptr;
  // the balanced plan is a function of the arguments and the device, so it is
  // the one the split count S came from
  const Balance bal = plan_balance(a, sm_count());
  if (bal.G && bal.slots != S) return VA_ERR_INVALID_ARG;
  if (S == 1) return launch_attention(a, SplitRange{1, 0, 1}, w, base, nullptr, nullptr, st, bal);
  // Split: a request flagged by one split (a bad page, an expired wait) must
  // come out empty although its other splits hold partials, so the splits
  // report into the call's own status array and the merge empties flagged
  // requests and passes their status on to the caller's array.
  int32_t* status = reinterpret_cast<int32_t*>(base + w.status);
  if (cudaMemsetAsync(status, 0, (size_t)a.B * sizeof(int32_t), st) != cudaSuccess)
    return VA_ERR_CUDA;
  va_attn_args as = a;
  as.req_status = status;
  const int r = launch_attention(as, SplitRange{S, 0, S}, w, base, o_part, lse_part, st, bal);
  if (r != VA_OK) return r;
  cudaError_t e = launch_merge(o_part, lse_part, S, (long long)a.B * a.T * a.H, a.dtype, a.out,
                               a.lse, st, status, a.T * a.H, a.req_status);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int run_partials(const va_attn_args& a, SplitRange sp, void* ws, float* o_part, float* lse_part,
                 cudaStream_t st) {
  const WorkspaceLayout w = workspace_layout(a, sp.S, false);
  return launch_attention(a, sp, w, static_cast<char*>(ws), o_part, lse_part, st, Balance{});
}

}  // namespace va

extern "C" {

int va_max_qlen(void) { return VA_MAX_QLEN; }

const char* va_status_string(int status) {
  switch (status) {
    case VA_OK: return "VA_OK";
    case VA_ERR_INVALID_ARG: return "VA_ERR_INVALID_ARG";
    case VA_ERR_UNSUPPORTED: return "VA_ERR_UNSUPPORTED";
    case VA_ERR_CUDA: return "VA_ERR_CUDA";
    case VA_ERR_INVALID_TREE: return "VA_ERR_INVALID_TREE";
    default: return "VA_ERR_UNKNOWN";
  }
}

int va_build_tree(const double* lp, const int32_t* tok, int B, int L, int K, int budget,
                  int32_t* parents, int32_t* tokens, int32_t* depth, int32_t* n_nodes,
                  va_stream_t stream) {
  if (B < 0 || L < 1 || L > VA_MAX_DEPTH || K < 1 || K > VA_MAX_TOPK || budget < 0 ||
      budget + 1 > VA_MAX_QLEN)
    return VA_ERR_INVALID_ARG;
  if (B == 0) return VA_OK;
  if (!lp || !tok || !parents || !tokens || !depth || !n_nodes) return VA_ERR_INVALID_ARG;
  if (!aligned(lp, 8)) return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_build_tree(lp, tok, B, L, K, budget, parents, tokens, depth,
                                        n_nodes, (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int va_build_tree_mask(const int32_t* parents, int B, int T, uint64_t* mask,
                       int32_t* tree_status, va_stream_t stream) {
  if (B < 0 || T < 1 || T > VA_MAX_QLEN) return VA_ERR_INVALID_ARG;
  if (B == 0) return VA_OK;
  if (!parents || !mask || !aligned(mask, 8)) return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_tree_mask(parents, B, T, mask, tree_status, (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int va_tree_accept(const int32_t* parents, const int32_t* tokens, const int32_t* target_next,
                   int B, int T, int32_t* path, int32_t* accept_len, int32_t* next_token,
                   va_stream_t stream) {
  if (B < 0 || T < 1 || T > VA_MAX_QLEN) return VA_ERR_INVALID_ARG;
  if (B == 0) return VA_OK;
  if (!parents || !tokens || !target_next || !path || !accept_len || !next_token)
    return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_tree_accept(parents, tokens, target_next, B, T, path, accept_len,
                                         next_token, (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int va_num_splits(const va_attn_args* args) {
  const int st = check_args(args);
  if (st != VA_OK) return -st;
  return plan_splits(args);
}

size_t va_workspace_bytes(const va_attn_args* args) {
  if (check_args(args) != VA_OK || args->B == 0) return 0;
  return va::workspace_layout(*args, plan_splits(args)).total;
}

int va_verify_attn(const va_attn_args* args, va_stream_t stream) {
  const int st = check_args(args);
  if (st != VA_OK) return st;
  if (args->B == 0) return VA_OK;
  const int S = plan_splits(args);
  const size_t need = va::workspace_layout(*args, S).total;
  if (need && (!args->workspace || !aligned(args->workspace, 256) || args->workspace_bytes < need))
    return VA_ERR_INVALID_ARG;
  return va::run_verify(*args, S, args->workspace, (cudaStream_t)stream);
}

int va_verify_attn_partials(const va_attn_args* args, int split_first, int split_count,
                            float* o_part, float* lse_part, va_stream_t stream) {
  const int st = check_args(args, false);
  if (st != VA_OK) return st;
  const int S = args->num_splits;
  if (S < 1) return VA_ERR_INVALID_ARG;  // the partition must be explicit
  if (split_first < 0 || split_count < 1 || split_first > S - split_count)
    return VA_ERR_INVALID_ARG;
  if (args->B == 0) return VA_OK;
  if (!o_part || !lse_part || !aligned(o_part, 16) || !aligned(lse_part, 4))
    return VA_ERR_INVALID_ARG;
  const size_t need = va::workspace_layout(*args, S, false).total;
  if (need && (!args->workspace || !aligned(args->workspace, 256) || args->workspace_bytes < need))
    return VA_ERR_INVALID_ARG;
  return va::run_partials(*args, va::SplitRange{S, split_first, split_count}, args->workspace,
                          o_part, lse_part, (cudaStream_t)stream);
}

int va_merge(const float* o_part, const float* lse_part, int S, int B, int T, int H,
             int out_dtype, void* out, float* lse, va_stream_t stream) {
  if (S < 1 || S > VA_MAX_SPLITS || B < 0 || T < 1 || T > VA_MAX_QLEN || H < 1)
    return VA_ERR_INVALID_ARG;
  if (out_dtype != VA_F32 && out_dtype != VA_BF16) return VA_ERR_INVALID_ARG;
  if (B == 0) return VA_OK;
  if (!o_part || !lse_part || !out || !lse) return VA_ERR_INVALID_ARG;
  if (!aligned(o_part, 16) || !aligned(out, 8) || !aligned(lse_part, 4) || !aligned(lse, 4))
    return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_merge(o_part, lse_part, S, (long long)B * T * H, out_dtype, out,
                                   lse, (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int va_token_logprobs(const va_logprob_args* a, va_stream_t stream) {
  if (!a) return VA_ERR_INVALID_ARG;
  if (a->dtype != VA_F32 && a->dtype != VA_BF16) return VA_ERR_INVALID_ARG;
  if (a->R < 0 || a->V < 1 || a->ld < a->V || a->G < 0 || a->G > 65536 || a->K < 0 ||
      a->K > VA_MAX_TOPK || a->K > a->V)
    return VA_ERR_INVALID_ARG;
  if (!(a->scale > 0.f && a->scale <= FLT_MAX)) return VA_ERR_INVALID_ARG;
  if (a->R == 0) return VA_OK;
  if (a->R > 0x7fffffff / 8 || a->V > 0x7fffffff - 65536) return VA_ERR_UNSUPPORTED;
  if (!a->logits || !aligned(a->logits, a->dtype == VA_F32 ? 4 : 2)) return VA_ERR_INVALID_ARG;
  if (a->G > 0 && (!a->tokens || !a->tok_lp)) return VA_ERR_INVALID_ARG;
  if (a->K > 0 && !a->top_ids) return VA_ERR_INVALID_ARG;
  if (a->K == 0 && (a->top_lp || a->top_lp64)) return VA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)a->tokens, (const void*)a->lse, (const void*)a->entropy,
                        (const void*)a->tok_lp, (const void*)a->top_ids, (const void*)a->top_lp,
                        (const void*)a->row_status})
    if (p && !aligned(p, 4)) return VA_ERR_INVALID_ARG;
  if (a->top_lp64 && !aligned(a->top_lp64, 8)) return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_logprobs(*a, sm_count(), (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

size_t va_key_weights_workspace_bytes(const va_key_weight_args* args) {
  if (check_key_weights(args) != VA_OK || args->B == 0) return 0;
  return key_weight_workspace(args, key_weight_splits(args));
}

int va_key_weights(const va_key_weight_args* args, va_stream_t stream) {
  const int st = check_key_weights(args);
  if (st != VA_OK) return st;
  if (args->B == 0) return VA_OK;
  const int splits = key_weight_splits(args);
  const size_t need = key_weight_workspace(args, splits);
  if (need && (!args->workspace || !aligned(args->workspace, 256) || args->workspace_bytes < need))
    return VA_ERR_INVALID_ARG;
  va::KwParams p;
  p.q_nope = args->q_nope;
  p.q_pe = args->q_pe;
  p.c_kv = args->c_kv;
  p.k_pe = args->k_pe;
  p.page_table = args->page_table;
  p.kv_len = args->kv_len;
  p.tree_mask = args->tree_mask;
  p.lse = args->lse;
  p.path = args->path;
  p.accept_len = args->accept_len;
  p.weights_in = args->weights_in;
  p.weights = args->weights;
  p.part = splits > 1 ? reinterpret_cast<float*>(static_cast<char*>(args->workspace) +
                                                  key_weight_rows(args))
                      : nullptr;
  p.req_status = args->req_status;
  p.B = args->B;
  p.H = args->H;
  p.T = args->T;
  p.max_pages = args->max_pages;
  p.num_pages = args->num_pages;
  p.splits = splits;
  p.scale = (args->flags & VA_FLAG_KV_FP8_E4M3) ? args->scale * args->kv_scale : args->scale;
  p.decay = args->decay;
  p.stay = p.pass = 0;
  if (va::kweights_on_tc(*args)) va::kweights_tc_blocks(*args, &p.stay, &p.pass);
  cudaError_t e;
  if (va::kweights_on_tc(*args)) e = va::launch_kweights_tc(*args, p, sm_count(), (cudaStream_t)stream);
  else e = va::launch_kweights_simt(*args, p, (cudaStream_t)stream);
  if (e == cudaSuccess && splits > 1) e = va::launch_kweights_join(p, (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int va_evict_plan(const va_evict_args* a, va_stream_t stream) {
  if (!a) return VA_ERR_INVALID_ARG;
  if (a->B < 0 || a->T < 0 || a->T > VA_MAX_QLEN || a->n_sink < 0 || a->n_recent < 0)
    return VA_ERR_INVALID_ARG;
  if (a->B == 0) return VA_OK;
  if (a->capacity < 1 || a->capacity < a->T) return VA_ERR_INVALID_ARG;
  if (a->B > VA_MAX_BATCH) return VA_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)a->weights, (const void*)a->kv_len, (const void*)a->budget,
                        (const void*)a->new_len, (const void*)a->from_slot})
    if (!p || !aligned(p, 4)) return VA_ERR_INVALID_ARG;
  if ((a->T > 0) != (a->path != nullptr) || (a->T > 0) != (a->accept_len != nullptr))
    return VA_ERR_INVALID_ARG;
  if (a->pos_out && !a->pos) return VA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)a->path, (const void*)a->accept_len, (const void*)a->pos,
                        (const void*)a->weights_out, (const void*)a->pos_out,
                        (const void*)a->req_status})
    if (p && !aligned(p, 4)) return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_evict_plan(*a, sm_count(), (cudaStream_t)stream);
  if (e == cudaErrorNotSupported) return VA_ERR_UNSUPPORTED;
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

int va_kv_move(void* c_kv, void* k_pe, int elem_bytes, int num_pages, int page_size,
               const int32_t* page_table, int B, int max_pages, const int32_t* from_slot,
               const int32_t* new_len, int32_t* req_status, va_stream_t stream) {
  if (B < 0 || (elem_bytes != 1 && elem_bytes != 2 && elem_bytes != 4)) return VA_ERR_INVALID_ARG;
  if (page_size != VA_PAGE_SIZE || B > VA_MAX_BATCH) return VA_ERR_UNSUPPORTED;
  if (B == 0) return VA_OK;
  if (num_pages < 1 || max_pages < 1) return VA_ERR_INVALID_ARG;
  if ((long long)num_pages * VA_PAGE_SIZE > 0x7fffffffLL ||
      (long long)max_pages * VA_PAGE_SIZE > 0x7fffffffLL)
    return VA_ERR_UNSUPPORTED;
  for (const void* p : {(const void*)c_kv, (const void*)k_pe})
    if (!p || !aligned(p, 16)) return VA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)page_table, (const void*)from_slot, (const void*)new_len})
    if (!p || !aligned(p, 4)) return VA_ERR_INVALID_ARG;
  if (req_status && !aligned(req_status, 4)) return VA_ERR_INVALID_ARG;
  cudaError_t e = va::launch_kv_move(c_kv, k_pe, elem_bytes, num_pages, page_table, B, max_pages,
                                     from_slot, new_len, req_status, (cudaStream_t)stream);
  return e == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

unsigned int va_device_timeouts(void) {
  const unsigned int a = va::tc_timeouts(), b = va::simt_timeouts(), c = va::kw_timeouts();
  if (a == 0xFFFFFFFFu || b == 0xFFFFFFFFu || c == 0xFFFFFFFFu) return 0xFFFFFFFFu;
  return a + b + c;
}

}  // extern "C"
