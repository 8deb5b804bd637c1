"""Python binding of libverifyattn (tree-verify MLA attention for DDTree, sm_100a).

Argument marshalling only: every step runs in the CUDA library's kernels.
Torch tensors cross the C ABI as raw device pointers plus the current CUDA
stream, the bridge shape the pages describe (page "The Capstone Commit:
Validating a Native CUDA DDTree Inference Engine", section "The Message
Itself": ctypes bindings accepting torch CUDA tensors via data_ptr and the
current stream).  The library must be built in-tree
(``python -m speculative_decoding_tree_va_b200.build``); importing the calls
without it raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from contextlib import ExitStack
from typing import Any, NamedTuple, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("VA_LIB", os.path.join(HERE, "libverifyattn.so"))

VA_OK, VA_ERR_INVALID_ARG, VA_ERR_UNSUPPORTED, VA_ERR_CUDA, VA_ERR_INVALID_TREE = range(5)
VA_F32, VA_BF16 = 0, 1
VA_FLAG_BF16_CUDA_CORES = 1
VA_FLAG_TEST_STALL_MMA = 2  # test hook: the tensor-core kernel's bounded waits expire
VA_FLAG_TEST_STALL_COPIES = 8  # test hook: the CUDA-core kernel's staging waits expire
VA_FLAG_TEST_STALL_KEY_WEIGHTS = 16  # test hook: the key-weight kernel's bounded waits expire
VA_FLAG_KV_FP8_E4M3 = 4     # latent cache as FP8 E4M3 codes times kv_scale
D_LATENT, D_ROPE, PAGE_SIZE, MAX_QLEN = 512, 64, 64, 65

EXPORTS = ("va_max_qlen", "va_status_string", "va_build_tree", "va_build_tree_mask",
           "va_workspace_bytes", "va_num_splits", "va_verify_attn", "va_merge",
           "va_device_timeouts", "va_verify_attn_noalloc", "va_tree_accept",
           "va_verify_attn_partials", "va_token_logprobs", "va_key_weights_workspace_bytes",
           "va_key_weights", "va_evict_plan", "va_kv_move")
NOALLOC_SCRATCH_BYTES = 32 << 20


class VaAttnArgs(ctypes.Structure):
    """Mirror of ``va_attn_args`` in include/verifyattn.h."""

    _fields_ = [
        ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int),
        ("kv_len", ctypes.c_void_p), ("tree_mask", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("req_status", ctypes.c_void_p),
        ("num_splits", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("flags", ctypes.c_int),
        ("kv_scale", ctypes.c_float),
    ]


class VaLogprobArgs(ctypes.Structure):
    """Mirror of ``va_logprob_args``."""

    _fields_ = [
        ("dtype", ctypes.c_int), ("R", ctypes.c_int), ("V", ctypes.c_int),
        ("ld", ctypes.c_longlong), ("scale", ctypes.c_float), ("logits", ctypes.c_void_p),
        ("tokens", ctypes.c_void_p), ("G", ctypes.c_int), ("K", ctypes.c_int),
        ("lse", ctypes.c_void_p), ("entropy", ctypes.c_void_p), ("tok_lp", ctypes.c_void_p),
        ("top_ids", ctypes.c_void_p), ("top_lp", ctypes.c_void_p), ("top_lp64", ctypes.c_void_p),
        ("row_status", ctypes.c_void_p),
    ]


class VaKeyWeightArgs(ctypes.Structure):
    """Mirror of ``va_key_weight_args``."""

    _fields_ = [
        ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("q_nope", ctypes.c_void_p), ("q_pe", ctypes.c_void_p),
        ("c_kv", ctypes.c_void_p), ("k_pe", ctypes.c_void_p),
        ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int),
        ("kv_len", ctypes.c_void_p), ("tree_mask", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("path", ctypes.c_void_p), ("accept_len", ctypes.c_void_p),
        ("weights_in", ctypes.c_void_p), ("decay", ctypes.c_float), ("weights", ctypes.c_void_p),
        ("req_status", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("flags", ctypes.c_int), ("kv_scale", ctypes.c_float),
    ]


class VaEvictArgs(ctypes.Structure):
    """Mirror of ``va_evict_args``."""

    _fields_ = [
        ("B", ctypes.c_int), ("capacity", ctypes.c_int), ("T", ctypes.c_int),
        ("weights", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("budget", ctypes.c_void_p),
        ("path", ctypes.c_void_p), ("accept_len", ctypes.c_void_p), ("pos", ctypes.c_void_p),
        ("n_sink", ctypes.c_int), ("n_recent", ctypes.c_int),
        ("new_len", ctypes.c_void_p), ("from_slot", ctypes.c_void_p),
        ("weights_out", ctypes.c_void_p), ("pos_out", ctypes.c_void_p),
        ("req_status", ctypes.c_void_p),
    ]


class VerifyAttnError(RuntimeError):
    pass


_lib = None


def load_library(path: Optional[str] = None):
    """Load libverifyattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise VerifyAttnError(f"libverifyattn not built: {p} missing "
                              "(run python -m speculative_decoding_tree_va_b200.build)")
    lib = ctypes.CDLL(p)
    V, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.va_max_qlen.argtypes, lib.va_max_qlen.restype = [], I
    lib.va_status_string.argtypes, lib.va_status_string.restype = [I], ctypes.c_char_p
    lib.va_build_tree.argtypes = [V, V, I, I, I, I, V, V, V, V, V]
    lib.va_build_tree.restype = I
    lib.va_build_tree_mask.argtypes = [V, I, I, V, V, V]
    lib.va_build_tree_mask.restype = I
    lib.va_workspace_bytes.argtypes, lib.va_workspace_bytes.restype = [ctypes.POINTER(VaAttnArgs)], Z
    lib.va_num_splits.argtypes, lib.va_num_splits.restype = [ctypes.POINTER(VaAttnArgs)], I
    lib.va_verify_attn.argtypes = [ctypes.POINTER(VaAttnArgs), V]
    lib.va_verify_attn.restype = I
    lib.va_merge.argtypes = [V, V, I, I, I, I, I, V, V, V]
    lib.va_merge.restype = I
    lib.va_device_timeouts.argtypes, lib.va_device_timeouts.restype = [], ctypes.c_uint
    lib.va_tree_accept.argtypes = [V, V, V, I, I, V, V, V, V]
    lib.va_tree_accept.restype = I
    lib.va_verify_attn_noalloc.argtypes = [ctypes.POINTER(VaAttnArgs), V]
    lib.va_verify_attn_noalloc.restype = I
    lib.va_verify_attn_partials.argtypes = [ctypes.POINTER(VaAttnArgs), I, I, V, V, V]
    lib.va_verify_attn_partials.restype = I
    lib.va_token_logprobs.argtypes = [ctypes.POINTER(VaLogprobArgs), V]
    lib.va_token_logprobs.restype = I
    lib.va_key_weights_workspace_bytes.argtypes = [ctypes.POINTER(VaKeyWeightArgs)]
    lib.va_key_weights_workspace_bytes.restype = Z
    lib.va_key_weights.argtypes = [ctypes.POINTER(VaKeyWeightArgs), V]
    lib.va_key_weights.restype = I
    lib.va_evict_plan.argtypes = [ctypes.POINTER(VaEvictArgs), V]
    lib.va_evict_plan.restype = I
    lib.va_kv_move.argtypes = [V, V, I, I, I, V, I, I, V, V, V, V]
    lib.va_kv_move.restype = I
    if path is None:
        _lib = lib
    return lib


def _check(status: int, what: str):
    if status != VA_OK:
        name = load_library().va_status_string(status).decode()
        raise VerifyAttnError(f"{what} failed: {name}")


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def max_qlen() -> int:
    return load_library().va_max_qlen()


def device_timeouts() -> int:
    """Expired bounded waits in the attention and key-weight kernels since load (synchronises)."""
    return int(load_library().va_device_timeouts())


def build_tree(lp, tok, budget: int, stream=None):
    """GPU best-first draft trees.  lp float64 [B, L, K], tok int32 [B, L, K] (cuda).

    Returns (parents, tokens, depth) int32 [B, budget + 1] and n_nodes int32 [B]."""
    import torch
    B, L, K = lp.shape
    T = budget + 1
    kw = dict(device=lp.device, dtype=torch.int32)
    parents, tokens, depth = (torch.empty(B, T, **kw) for _ in range(3))
    n_nodes = torch.empty(B, **kw)
    _check(load_library().va_build_tree(_ptr(lp.contiguous()), _ptr(tok.contiguous()), B, L, K,
                                        budget, _ptr(parents), _ptr(tokens), _ptr(depth),
                                        _ptr(n_nodes), _stream(stream)), "va_build_tree")
    return parents, tokens, depth, n_nodes


def tree_accept(parents, tokens, target_next, stream=None):
    """Greedy accept walk.  int32 [B, T] cuda tensors -> (path [B, T], accept_len [B],
    next_token [B])."""
    import torch
    B, T = parents.shape
    kw = dict(device=parents.device, dtype=torch.int32)
    path = torch.empty(B, T, **kw)
    alen = torch.empty(B, **kw)
    nxt = torch.empty(B, **kw)
    _check(load_library().va_tree_accept(_ptr(parents.contiguous()), _ptr(tokens.contiguous()),
                                         _ptr(target_next.contiguous()), B, T, _ptr(path),
                                         _ptr(alen), _ptr(nxt), _stream(stream)), "va_tree_accept")
    return path, alen, nxt


def build_tree_mask(parents, stream=None):
    """parents int32 [B, T] (cuda) -> (mask int64 [B, T, W] holding uint64 bits, status int32 [B])."""
    import torch
    B, T = parents.shape
    W = (T + 63) // 64
    mask = torch.empty(B, T, W, device=parents.device, dtype=torch.int64)
    status = torch.empty(B, device=parents.device, dtype=torch.int32)
    _check(load_library().va_build_tree_mask(_ptr(parents.contiguous()), B, T, _ptr(mask),
                                             _ptr(status), _stream(stream)), "va_build_tree_mask")
    return mask, status


def _fp8_cache(c_kv) -> bool:
    import torch
    return c_kv.dtype in (torch.uint8, torch.float8_e4m3fn)


def make_args(q_nope, q_pe, c_kv, k_pe, page_table, kv_len, tree_mask, out, lse, *, scale: float,
              num_splits: int = 0, workspace=None, req_status=None, flags: int = 0,
              kv_scale: float = 1.0) -> VaAttnArgs:
    """Fill a VaAttnArgs from torch tensors (no checks beyond what the library does).

    A uint8 or float8_e4m3fn cache (c_kv, k_pe) sets VA_FLAG_KV_FP8_E4M3 with
    kv_scale, the value of one cache unit."""
    import torch
    B, T, H, _ = q_nope.shape
    dt = {torch.float32: VA_F32, torch.bfloat16: VA_BF16}[q_nope.dtype]
    a = VaAttnArgs()
    a.dtype, a.B, a.H, a.T, a.scale = dt, B, H, T, float(scale)
    a.q_nope, a.q_pe, a.c_kv, a.k_pe = (t.data_ptr() for t in (q_nope, q_pe, c_kv, k_pe))
    a.num_pages, a.page_size = c_kv.shape[0], c_kv.shape[1]
    a.page_table, a.max_pages = page_table.data_ptr(), page_table.shape[1]
    a.kv_len, a.tree_mask = kv_len.data_ptr(), tree_mask.data_ptr()
    a.out, a.lse = out.data_ptr(), lse.data_ptr()
    a.req_status = None if req_status is None else req_status.data_ptr()
    a.num_splits = num_splits
    a.workspace = None if workspace is None else workspace.data_ptr()
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.flags = flags
    if _fp8_cache(c_kv):
        a.flags |= VA_FLAG_KV_FP8_E4M3
        a.kv_scale = float(kv_scale)
    return a


def workspace_bytes(args: VaAttnArgs) -> int:
    return int(load_library().va_workspace_bytes(ctypes.byref(args)))


def num_splits(args: VaAttnArgs) -> int:
    """The split count va_verify_attn uses for these arguments (for the balanced
    CUDA-core plan, the number of partials per row it merges)."""
    return int(load_library().va_num_splits(ctypes.byref(args)))


def verify_attn_args(args: VaAttnArgs, stream=None):
    _check(load_library().va_verify_attn(ctypes.byref(args), _stream(stream)), "va_verify_attn")


def verify_attn(q_nope, q_pe, c_kv, k_pe, page_table, kv_len, tree_mask, *, scale: float,
                num_splits: int = 0, out=None, lse=None, workspace=None, req_status=None,
                flags: int = 0, kv_scale: float = 1.0, stream=None):
    """Tree-verify MLA-absorb attention.  Allocates out/lse/workspace when not given.

    q_nope [B,T,H,512], q_pe [B,T,H,64] (float32 or bfloat16, cuda); c_kv
    [pages,64,512], k_pe [pages,64,64] in the query dtype, or FP8 E4M3 codes
    (uint8 / float8_e4m3fn) standing for kv_scale times their values;
    page_table int32 [B, max_pages], kv_len int32 [B], tree_mask int64 [B,T,W]
    from build_tree_mask.  Returns (out, lse) in the query dtype."""
    import torch
    B, T, H, _ = q_nope.shape
    if out is None:
        out = torch.empty(B, T, H, D_LATENT, device=q_nope.device, dtype=q_nope.dtype)
    if lse is None:
        lse = torch.empty(B, T, H, device=q_nope.device, dtype=torch.float32)
    args = make_args(q_nope, q_pe, c_kv, k_pe, page_table, kv_len, tree_mask, out, lse,
                     scale=scale, num_splits=num_splits, workspace=workspace,
                     req_status=req_status, flags=flags, kv_scale=kv_scale)
    need = workspace_bytes(args)
    if need and workspace is None:
        workspace = torch.empty(need, device=q_nope.device, dtype=torch.uint8)
        args.workspace, args.workspace_bytes = workspace.data_ptr(), need
    verify_attn_args(args, stream)
    return out, lse


def verify_attn_noalloc(args: VaAttnArgs, stream=None):
    """va_verify_attn_noalloc: split-KV partials in the library's fixed device
    array instead of a workspace (for callers that cannot allocate)."""
    _check(load_library().va_verify_attn_noalloc(ctypes.byref(args), _stream(stream)),
           "va_verify_attn_noalloc")


def partials_workspace_bytes(args: VaAttnArgs) -> int:
    """Workspace of va_verify_attn_partials: that of the same call with one split."""
    one = VaAttnArgs.from_buffer_copy(args)
    one.num_splits = 1
    return workspace_bytes(one)


def verify_attn_partials(args: VaAttnArgs, split_first: int, split_count: int, o_part, lse_part,
                         stream=None):
    """va_verify_attn_partials: splits [split_first, split_first + split_count) of the
    args.num_splits-way partition into o_part float [count, B, T, H, 512] and
    lse_part float [count, B, T, H] (cuda tensors), no merge."""
    _check(load_library().va_verify_attn_partials(ctypes.byref(args), split_first, split_count,
                                                  _ptr(o_part), _ptr(lse_part), _stream(stream)),
           "va_verify_attn_partials")


def merge(o_part, lse_part, out_dtype, stream=None):
    """o_part float [S,B,T,H,512], lse_part float [S,B,T,H] -> (out, lse)."""
    import torch
    S, B, T, H, _ = o_part.shape
    dt = {torch.float32: VA_F32, torch.bfloat16: VA_BF16}[out_dtype]
    out = torch.empty(B, T, H, D_LATENT, device=o_part.device, dtype=out_dtype)
    lse = torch.empty(B, T, H, device=o_part.device, dtype=torch.float32)
    _check(load_library().va_merge(_ptr(o_part.contiguous()), _ptr(lse_part.contiguous()), S, B, T,
                                   H, dt, _ptr(out), _ptr(lse), _stream(stream)), "va_merge")
    return out, lse


# --------------------------------------------------------------------------
# Around the verify call: logits, and the eviction of cached keys.  These
# calls check the tensors they take (device, type, shape, density); the
# library checks the rest.  What they allocate belongs to the stream that
# they run on.

def _on(t, stream):
    """Context in which t's device and the given stream are the current ones."""
    import torch
    if stream is not None and stream.device != t.device:
        raise VerifyAttnError(f"stream of {stream.device} for tensors on {t.device}")
    ctx = ExitStack()
    ctx.enter_context(torch.cuda.device(t.device))
    if stream is not None:
        ctx.enter_context(torch.cuda.stream(stream))
    return ctx


def _raw_stream(dev: int) -> int:
    """Handle of the current stream of a device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev)


def _need(t, name: str, dev: int, dtype, shape) -> int:
    """Address of one tensor argument: on cuda device `dev`, of this type and shape, dense."""
    if t.get_device() != dev or dev < 0:
        raise VerifyAttnError(f"{name} is on {t.device}: cuda tensors of one device are needed")
    if t.dtype is not dtype:
        raise VerifyAttnError(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise VerifyAttnError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise VerifyAttnError(f"{name} is not contiguous")
    return t.data_ptr()


def _axes(t, name: str, shape: str) -> None:
    """The tensor has as many axes as `shape` names (the others' sizes are read from it)."""
    if t.dim() != shape.count(",") + 1:
        raise VerifyAttnError(f"{name} has shape {tuple(t.shape)}, not [{shape}]")


class TokenLogprobs(NamedTuple):
    """What token_logprobs returns (None for what was not asked for)."""

    lse: Any       # float32 [...]
    entropy: Any   # float32 [...]
    tok_lp: Any    # float32, tokens' shape
    top_ids: Any   # int32 [..., k]
    top_lp: Any    # float32 or float64 [..., k]


def token_logprobs(logits, tokens=None, *, k: int = 0, scale: float = 1.0, wide: bool = False,
                   row_status=None, stream=None) -> TokenLogprobs:
    """Log-sum-exp, entropy, log probabilities of given tokens and top-k of rows of logits.

    logits float32 or bfloat16 [..., V] (cuda; dense or a slice [..., :V] of padded
    rows), scaled by `scale` (1 / temperature).  tokens int32 [...] or [..., G]: given
    tokens, < 0 for none.  k <= 16 alternatives, equal logits by lower index; with
    `wide` their log probabilities are float64, as build_tree reads them:
    ``build_tree(r.top_lp, r.top_ids, budget)`` for drafter logits [B, L, V], and
    ``tree_accept(parents, tokens, r.top_ids[..., 0])`` for target logits [B, T, V]
    with k = 1."""
    import torch
    dev, f32, i32 = logits.get_device(), torch.float32, torch.int32
    if dev < 0:
        raise VerifyAttnError(f"logits are on {logits.device}: cuda tensors are needed")
    if logits.dtype is not f32 and logits.dtype is not torch.bfloat16:
        raise VerifyAttnError(f"logits are {logits.dtype}, not float32 or bfloat16")
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise VerifyAttnError("logits need a vocabulary axis")
    k = int(k)
    if not 0 <= k <= 16:
        raise VerifyAttnError("k is not in 0 .. 16")
    if stream is not None or dev != torch.cuda.current_device():
        with _on(logits, stream):
            return token_logprobs(logits, tokens, k=k, scale=scale, wide=wide, row_status=row_status)
    lead, V = logits.shape[:-1], logits.shape[-1]
    R = lead.numel()
    a = VaLogprobArgs()
    a.ld = V
    if R:
        rows = logits
        if logits.dim() != 2:
            try:
                rows = logits.view(R, V)
            except RuntimeError:
                raise VerifyAttnError("logits rows are not evenly spaced") from None
        ld, step = rows.stride()
        if V > 1 and step != 1:
            raise VerifyAttnError("logits rows are not dense")
        if R > 1:
            a.ld = ld
        a.logits = logits.data_ptr()
    a.dtype = VA_F32 if logits.dtype is f32 else VA_BF16
    a.R, a.V, a.K, a.scale = R, V, k, float(scale)
    on = logits.device
    lse = torch.empty(*lead, device=on, dtype=f32) if lead else torch.empty((), device=on, dtype=f32)
    entropy = torch.empty_like(lse)
    a.lse, a.entropy = lse.data_ptr(), entropy.data_ptr()
    tok_lp = top_ids = top_lp = None
    if tokens is not None:
        G = 1 if tokens.shape == lead else tokens.shape[-1] if tokens.dim() else 0
        a.tokens = _need(tokens, "tokens", dev, i32, lead if tokens.shape == lead else lead + (G,))
        a.G = G
        tok_lp = torch.empty_like(tokens, dtype=f32)
        a.tok_lp = tok_lp.data_ptr()
    if k:
        top_ids = torch.empty(*lead, k, device=on, dtype=i32)
        top_lp = torch.empty_like(top_ids, dtype=torch.float64 if wide else f32)
        a.top_ids = top_ids.data_ptr()
        if wide:
            a.top_lp64 = top_lp.data_ptr()
        else:
            a.top_lp = top_lp.data_ptr()
    if row_status is not None:
        a.row_status = _need(row_status, "row_status", dev, i32, lead)
    _check(load_library().va_token_logprobs(ctypes.byref(a), _raw_stream(dev)), "va_token_logprobs")
    return TokenLogprobs(lse, entropy, tok_lp, top_ids, top_lp)


def key_weights(q_nope, q_pe, c_kv, k_pe, page_table, kv_len, tree_mask, lse, *, scale: float,
                path=None, accept_len=None, weights=None, decay: float = 1.0, out=None,
                workspace=None, req_status=None, flags: int = 0, kv_scale: float = 1.0,
                stream=None):
    """Attention weight that each cached key received, accumulated: what evict_plan ranks by.

    The first seven arguments and scale are verify_attn's, lse [B,T,H] is what it
    returned.  With path [B,T] and accept_len [B] (tree_accept's) only the accepted
    nodes count.  Returns out = decay * weights + the new sums, float32
    [B, 64 * max_pages]; slots from kv_len on are not touched (zeros in an array
    allocated here).  out may be weights."""
    import torch
    _axes(q_nope, "q_nope", "B, T, H, 512")
    _axes(c_kv, "c_kv", "pages, 64, 512")
    _axes(page_table, "page_table", "B, max_pages")
    B, T, H, _ = q_nope.shape
    dev, dt, i32, f32 = q_nope.get_device(), q_nope.dtype, torch.int32, torch.float32
    if dt is not f32 and dt is not torch.bfloat16:
        raise VerifyAttnError(f"q_nope is {dt}, not float32 or bfloat16")
    if dev >= 0 and (stream is not None or dev != torch.cuda.current_device()):
        with _on(q_nope, stream):
            return key_weights(q_nope, q_pe, c_kv, k_pe, page_table, kv_len, tree_mask, lse,
                               scale=scale, path=path, accept_len=accept_len, weights=weights,
                               decay=decay, out=out, workspace=workspace, req_status=req_status,
                               flags=flags, kv_scale=kv_scale)
    a = VaKeyWeightArgs()
    a.q_nope = _need(q_nope, "q_nope", dev, dt, (B, T, H, D_LATENT))
    a.q_pe = _need(q_pe, "q_pe", dev, dt, (B, T, H, D_ROPE))
    fp8 = _fp8_cache(c_kv)
    kd = c_kv.dtype if fp8 else dt
    n, m = c_kv.shape[0], page_table.shape[1]
    a.c_kv = _need(c_kv, "c_kv", dev, kd, (n, PAGE_SIZE, D_LATENT))
    a.k_pe = _need(k_pe, "k_pe", dev, kd, (n, PAGE_SIZE, D_ROPE))
    a.page_table = _need(page_table, "page_table", dev, i32, (B, m))
    a.kv_len = _need(kv_len, "kv_len", dev, i32, (B,))
    a.tree_mask = _need(tree_mask, "tree_mask", dev, torch.int64, (B, T, (T + 63) // 64))
    a.lse = _need(lse, "lse", dev, f32, (B, T, H))
    if path is not None:
        a.path = _need(path, "path", dev, i32, (B, T))
    if accept_len is not None:
        a.accept_len = _need(accept_len, "accept_len", dev, i32, (B,))
    cap = (B, m * PAGE_SIZE)
    if weights is not None:
        a.weights_in = _need(weights, "weights", dev, f32, cap)
    if req_status is not None:
        a.req_status = _need(req_status, "req_status", dev, i32, (B,))
    a.dtype = VA_F32 if dt is f32 else VA_BF16
    a.B, a.H, a.T, a.scale, a.decay = B, H, T, float(scale), float(decay)
    a.num_pages, a.page_size, a.max_pages = n, PAGE_SIZE, m
    a.flags = flags | (VA_FLAG_KV_FP8_E4M3 if fp8 else 0)
    a.kv_scale = float(kv_scale)
    if out is None:
        out = torch.zeros(cap, device=q_nope.device, dtype=f32)
    a.weights = _need(out, "out", dev, f32, cap)
    lib, ref = load_library(), ctypes.byref(a)
    need = lib.va_key_weights_workspace_bytes(ref)
    if need and workspace is None:
        workspace = torch.empty(need, device=q_nope.device, dtype=torch.uint8)
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise VerifyAttnError("the workspace is not a dense tensor of the same device")
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib.va_key_weights(ref, _raw_stream(dev)), "va_key_weights")
    return out


class EvictPlan(NamedTuple):
    """What evict_plan returns."""

    new_len: Any    # int32 [B]
    from_slot: Any  # int32 [B, capacity], -1 from new_len on
    weights: Any    # float32 [B, capacity]
    pos: Any        # int32 [B, capacity], or None without positions


def evict_plan(weights, kv_len, budget, *, path=None, accept_len=None, tree_len: int = 0, pos=None,
               n_sink: int = 0, n_recent: int = 0, weights_out=None, pos_out=None,
               req_status=None, stream=None) -> EvictPlan:
    """Which cached keys stay, and in which slots (kv_move then moves a layer's keys).

    weights float32 [B, capacity] (key_weights), kv_len and budget int32 [B].  With
    tree_len = T the last T keys are the tree's nodes: path [B,T] and accept_len [B]
    (tree_accept's) say which of them stay, and the others are dropped.  pos int32
    [B, capacity] holds each slot's token position where an earlier eviction has
    reordered them.  weights_out and pos_out may be weights and pos."""
    import torch
    if weights.dim() != 2:
        raise VerifyAttnError("weights are not [B, capacity]")
    dev, i32, f32 = weights.get_device(), torch.int32, torch.float32
    if dev >= 0 and (stream is not None or dev != torch.cuda.current_device()):
        with _on(weights, stream):
            return evict_plan(weights, kv_len, budget, path=path, accept_len=accept_len,
                              tree_len=tree_len, pos=pos, n_sink=n_sink, n_recent=n_recent,
                              weights_out=weights_out, pos_out=pos_out, req_status=req_status)
    B, cap = weights.shape
    a = VaEvictArgs()
    a.B, a.capacity, a.T, a.n_sink, a.n_recent = B, cap, tree_len, n_sink, n_recent
    a.weights = _need(weights, "weights", dev, f32, (B, cap))
    a.kv_len = _need(kv_len, "kv_len", dev, i32, (B,))
    a.budget = _need(budget, "budget", dev, i32, (B,))
    if path is not None:
        a.path = _need(path, "path", dev, i32, (B, tree_len))
    if accept_len is not None:
        a.accept_len = _need(accept_len, "accept_len", dev, i32, (B,))
    if pos is not None:
        a.pos = _need(pos, "pos", dev, i32, (B, cap))
    elif pos_out is not None:
        raise VerifyAttnError("pos_out without pos")
    if req_status is not None:
        a.req_status = _need(req_status, "req_status", dev, i32, (B,))
    new_len = torch.empty_like(kv_len)
    from_slot = torch.empty_like(weights, dtype=i32)
    a.new_len, a.from_slot = new_len.data_ptr(), from_slot.data_ptr()
    if weights_out is None:
        weights_out = torch.empty_like(weights)
        a.weights_out = weights_out.data_ptr()
    else:
        a.weights_out = _need(weights_out, "weights_out", dev, f32, (B, cap))
    if pos is not None:
        if pos_out is None:
            pos_out = torch.empty_like(pos)
        a.pos_out = _need(pos_out, "pos_out", dev, i32, (B, cap))
    _check(load_library().va_evict_plan(ctypes.byref(a), _raw_stream(dev)), "va_evict_plan")
    return EvictPlan(new_len, from_slot, weights_out, pos_out)


def kv_move(c_kv, k_pe, page_table, from_slot, new_len, *, req_status=None, stream=None) -> None:
    """Moves the keys of one cache, in place, as an evict_plan says.

    c_kv [pages,64,512] and k_pe [pages,64,64] of any cache type (float32, bfloat16 or
    8-bit codes); from_slot and new_len are the plan's.  Every page up to a request's
    old length must be that request's alone."""
    import torch
    dev, i32 = c_kv.get_device(), torch.int32
    _axes(c_kv, "c_kv", "pages, 64, 512")
    _axes(page_table, "page_table", "B, max_pages")
    n, (B, m) = c_kv.shape[0], page_table.shape
    if c_kv.dtype is not torch.float32 and c_kv.dtype is not torch.bfloat16 and not _fp8_cache(c_kv):
        raise VerifyAttnError(f"c_kv is {c_kv.dtype}: not a cache type")
    if B == 0:
        return
    if dev >= 0 and (stream is not None or dev != torch.cuda.current_device()):
        with _on(c_kv, stream):
            return kv_move(c_kv, k_pe, page_table, from_slot, new_len, req_status=req_status)
    c = _need(c_kv, "c_kv", dev, c_kv.dtype, (n, PAGE_SIZE, D_LATENT))
    k = _need(k_pe, "k_pe", dev, c_kv.dtype, (n, PAGE_SIZE, D_ROPE))
    t = _need(page_table, "page_table", dev, i32, (B, m))
    f = _need(from_slot, "from_slot", dev, i32, (B, m * PAGE_SIZE))
    l = _need(new_len, "new_len", dev, i32, (B,))
    s = None if req_status is None else _need(req_status, "req_status", dev, i32, (B,))
    _check(load_library().va_kv_move(c, k, c_kv.element_size(), n, PAGE_SIZE, t, B, m, f, l, s,
                                     _raw_stream(dev)), "va_kv_move")
