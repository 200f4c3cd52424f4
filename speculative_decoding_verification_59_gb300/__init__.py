"""GB300 (sm_103a) speculative-decoding verification.

A thin ctypes binding over the C ABI of libspecverify.so (declared in
include/spec_verify.h).  The functions named ``spec_verify_*`` take raw device
pointers and sizes exactly like the C calls; the ``verify_*`` helpers only
marshal torch CUDA tensors into those calls (pointers, current stream,
output allocation).  Every step of the verification runs in the library's
CUDA kernels: there is no CPU or PyTorch fallback, and using the package
without the built library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "SPEC_OK", "SPEC_DTYPE_F32", "SPEC_DTYPE_BF16", "SpecVerifyError", "lib_path", "load_library",
    "spec_verify_workspace_size", "spec_verify_workspace_init", "spec_verify_sample",
    "spec_verify_sample_stats", "spec_verify_sample_finish", "spec_verify_sample_noalloc",
    "spec_verify_greedy", "spec_verify_tree_greedy", "spec_verify_read_error",
    "spec_verify_status_string", "Workspace", "verify_sample", "verify_greedy", "verify_tree_greedy",
    "SPEC_DTYPE_E4M3", "KVCache", "kv_append", "kv_read", "kv_compact", "paged_attention",
    "token_logprobs", "add_norm", "gated_act", "quantize_e4m3", "matmul_e4m3",
]

SPEC_OK = 0
SPEC_ERR_INVALID_ARG = 1
SPEC_ERR_UNSUPPORTED_DTYPE = 2
SPEC_ERR_MISALIGNED = 3
SPEC_ERR_WORKSPACE_TOO_SMALL = 4
SPEC_ERR_CUDA = 5
SPEC_ERR_DEVICE_INPUT = 6
SPEC_ERR_EXCEEDS_STATIC_SCRATCH = 7
SPEC_VERIFY_NOALLOC_SCRATCH_BYTES = 8 << 20
SPEC_DTYPE_F32 = 0
SPEC_DTYPE_BF16 = 1
SPEC_DTYPE_E4M3 = 2
SPEC_ACT_SILU = 0
SPEC_ACT_GELU_TANH = 1
SPEC_MATMUL_FEW = 0
SPEC_MATMUL_WHOLE = 1
SPEC_MATMUL_CLUSTERS = 2
SPEC_MATMUL_SHARES = 3
SPEC_DEVERR_TOKEN_RANGE = 1
SPEC_DEVERR_EMPTY_ROW = 2
SPEC_DEVERR_TREE_PARENT = 4
SPEC_DEVERR_TIMEOUT = 8
SPEC_DEVERR_CACHE_RANGE = 16

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libspecverify.so")
_lib = None

# name -> (argtypes, restype); pointers travel as c_void_p, the stream as c_void_p
_P, _I, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L, _F = ctypes.c_int64, ctypes.c_float


class KVCacheStruct(ctypes.Structure):
    """spec_kv_cache_t of include/spec_verify.h."""
    _fields_ = [(n, _P) for n in ("k", "v", "k_scale", "v_scale", "block_table", "error")] + \
        [(n, _L) for n in ("page_stride", "token_stride", "head_stride", "layer_stride",
                           "scale_page_stride", "scale_token_stride", "scale_head_stride",
                           "scale_layer_stride")] + \
        [(n, ctypes.c_int32) for n in ("dtype", "layers", "num_pages", "page_size", "max_pages",
                                       "kv_heads", "head_dim")]


SIGNATURES = {
    "spec_verify_workspace_size": ([_I, _I, _I], _S),
    "spec_verify_workspace_init": ([_P, _S, _P], _I),
    "spec_verify_sample": ([_P, _P, _I, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _P, _P, _S,
                            _P], _I),
    "spec_verify_sample_lazy": ([_P, _P, _I, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _P, _P, _S,
                                 _P], _I),
    "spec_verify_lazy_groups": ([_I, _I, _I, _I, _P], _I),
    "spec_verify_sample_stats": ([_P, _P, _I, ctypes.c_float, _I, _I, _I, _P, _S, _P], _I),
    "spec_verify_sample_finish": ([_P, _P, _I, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _P, _P,
                                   _S, _P], _I),
    "spec_verify_sample_noalloc": ([_P, _P, _I, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _P,
                                    _P], _I),
    "spec_verify_greedy": ([_P, _I, _P, _I, _I, _I, _P, _P, _P, _S, _P], _I),
    "spec_verify_tree_greedy": ([_P, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P, _S, _P], _I),
    "spec_topk_workspace_size": ([_I, _I, _I], _S),
    "spec_topk_exclude": ([_P, _I, _I, _I, _I, _P, _P, _P, _P, _S, _P], _I),
    "spec_ngram_workspace_size": ([_I, _I, _I], _S),
    "spec_ngram_retrieve": ([_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _S, _P], _I),
    "spec_cosine_workspace_size": ([_I, _I], _S),
    "spec_cosine_topk": ([_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P], _I),
    "spec_kv_append": ([_P, _P, _P, _P, _L, _L, _L, _P, _P, _F, _P, _I, _I, _I, _P, _P, _P, _I, _I,
                        _I, _P, _P], _I),
    "spec_kv_read": ([_P, _P, _P, _I, _I, _I, _P, _P, _P], _I),
    "spec_kv_compact": ([_P, _P, _P, _P, _I, _I, _P], _I),
    "spec_attention_workspace_size": ([_I, _I, _I, _I, _I], _S),
    "spec_paged_attention": ([_P, _P, _L, _P, _P, _P, _F, _I, _I, _I, _P, _P, _P, _S, _P], _I),
    "spec_logprobs_workspace_size": ([_I, _I, _I], _S),
    "spec_token_logprobs": ([_P, _I, _P, _F, _I, _I, _I, _P, _P, _P, _P, _P, _S, _P], _I),
    "spec_add_norm": ([_P, _I, _L, _P, _I, _L, _P, _F, _I, _I, _P, _L, _P, _I, _P, _L, _P], _I),
    "spec_gated_act": ([_P, _P, _I, _L, _L, _I, _I, _I, _P, _I, _P, _L, _P], _I),
    "spec_quantize_e4m3": ([_P, _I, _L, _I, _I, _I, _P, _P, _L, _P], _I),
    "spec_matmul_workspace_size": ([_I, _I, _I], _S),
    "spec_matmul_plan": ([_I, _I, _I, _I, _P, _P], _I),
    "spec_matmul_e4m3": ([_P, _L, _P, _L, _P, _L, _P, _L, _I, _I, _I, _P, _I, _L, _P, _S, _P], _I),
    "spec_verify_read_error": ([_P, _P, _P], _I),
    "spec_verify_status_string": ([_I], ctypes.c_char_p),
    "spec_verify_set_wait_limit": ([ctypes.c_uint32], None),
    "spec_verify_set_lazy_split_bytes": ([ctypes.c_double], None),
    "spec_verify_default_wait_limit": ([], ctypes.c_uint32),
}


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {spec_verify_status_string(status)} (status {status})")


def lib_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libspecverify.so (built in-tree by __graft_entry__.build() or
    speculative_decoding_verification_59_gb300._build).  Raises if missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() first")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (argt, rest) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = argt
            fn.restype = rest
        _lib = lib
    return _lib


# ---- raw C-ABI calls (pointers are ints, stream is an int handle or 0) ------
def spec_verify_workspace_size(B: int, gamma_or_nodes: int, V: int) -> int:
    return load_library().spec_verify_workspace_size(B, gamma_or_nodes, V)


def spec_topk_workspace_size(rows: int, V: int, K: int) -> int:
    return load_library().spec_topk_workspace_size(rows, V, K)


def spec_topk_exclude(logits, dtype, rows, V, K, exclude, out_idx, out_val, ws, ws_bytes,
                      stream) -> int:
    return load_library().spec_topk_exclude(logits, dtype, rows, V, K, exclude, out_idx, out_val,
                                            ws, ws_bytes, stream)


def spec_ngram_workspace_size(B: int, n_max: int, max_matches: int) -> int:
    return load_library().spec_ngram_workspace_size(B, n_max, max_matches)


def spec_ngram_retrieve(tokens, lengths, B, n_max, w, L, max_matches, out_count, out_matches,
                        out_draft, ws, ws_bytes, stream) -> int:
    return load_library().spec_ngram_retrieve(tokens, lengths, B, n_max, w, L, max_matches,
                                              out_count, out_matches, out_draft, ws, ws_bytes,
                                              stream)


def spec_cosine_workspace_size(B: int, W: int) -> int:
    return load_library().spec_cosine_workspace_size(B, W)


def spec_cosine_topk(hidden, query, dtype, B, W, d, delta, positions, out_idx, out_pos, out_score,
                     ws, ws_bytes, stream) -> int:
    return load_library().spec_cosine_topk(hidden, query, dtype, B, W, d, delta, positions,
                                           out_idx, out_pos, out_score, ws, ws_bytes, stream)


def spec_verify_workspace_init(ws: int, nbytes: int, stream: int = 0) -> int:
    return load_library().spec_verify_workspace_init(ws, nbytes, stream)


def spec_verify_sample(target, draft, dtype, draft_tokens, uniforms, temperature, B, gamma, V,
                       out_tokens, out_num_accepted, out_logprobs, ws, ws_bytes, stream) -> int:
    return load_library().spec_verify_sample(target, draft, dtype, draft_tokens, uniforms,
                                             temperature, B, gamma, V, out_tokens,
                                             out_num_accepted, out_logprobs, ws, ws_bytes, stream)


def spec_verify_sample_lazy(target, draft, dtype, draft_tokens, uniforms, temperature, B, gamma,
                            V, out_tokens, out_num_accepted, out_logprobs, ws, ws_bytes,
                            stream) -> int:
    return load_library().spec_verify_sample_lazy(target, draft, dtype, draft_tokens, uniforms,
                                                  temperature, B, gamma, V, out_tokens,
                                                  out_num_accepted, out_logprobs, ws, ws_bytes,
                                                  stream)


def spec_verify_lazy_groups(B, gamma, V, dtype, ends) -> int:
    return load_library().spec_verify_lazy_groups(B, gamma, V, dtype, ends)


def lazy_groups(B: int, gamma: int, V: int, dtype: int):
    """Position groups of spec_verify_sample_lazy as [(lo, hi), ...] (host only,
    no GPU needed); raises for invalid arguments."""
    ends = (ctypes.c_int32 * 8)()
    n = spec_verify_lazy_groups(B, gamma, V, dtype, ctypes.addressof(ends))
    if n < 1:
        raise ValueError(f"spec_verify_lazy_groups: invalid arguments {(B, gamma, V, dtype)}")
    out, lo = [], 0
    for g in range(n):
        out.append((lo, int(ends[g])))
        lo = int(ends[g])
    return out


def spec_verify_sample_stats(target, draft, dtype, temperature, B, gamma, V, ws, ws_bytes,
                             stream) -> int:
    return load_library().spec_verify_sample_stats(target, draft, dtype, temperature, B, gamma, V,
                                                   ws, ws_bytes, stream)


def spec_verify_sample_finish(target, draft, dtype, draft_tokens, uniforms, temperature, B, gamma,
                              V, out_tokens, out_num_accepted, out_logprobs, ws, ws_bytes,
                              stream) -> int:
    return load_library().spec_verify_sample_finish(target, draft, dtype, draft_tokens, uniforms,
                                                    temperature, B, gamma, V, out_tokens,
                                                    out_num_accepted, out_logprobs, ws, ws_bytes,
                                                    stream)


def spec_verify_sample_noalloc(target, draft, dtype, draft_tokens, uniforms, temperature, B, gamma,
                               V, out_tokens, out_num_accepted, out_logprobs, stream) -> int:
    """spec_verify_sample without a workspace, for callers that cannot
    allocate device memory (see include/spec_verify.h)."""
    return load_library().spec_verify_sample_noalloc(target, draft, dtype, draft_tokens, uniforms,
                                                     temperature, B, gamma, V, out_tokens,
                                                     out_num_accepted, out_logprobs, stream)


def spec_verify_greedy(target, dtype, draft_tokens, B, gamma, V, out_tokens, out_num_accepted,
                       ws, ws_bytes, stream) -> int:
    return load_library().spec_verify_greedy(target, dtype, draft_tokens, B, gamma, V, out_tokens,
                                             out_num_accepted, ws, ws_bytes, stream)


def spec_verify_tree_greedy(target, dtype, node_tokens, parents, B, N, V, out_path_nodes,
                            out_tokens, out_num_accepted, ws, ws_bytes, stream) -> int:
    return load_library().spec_verify_tree_greedy(target, dtype, node_tokens, parents, B, N, V,
                                                  out_path_nodes, out_tokens, out_num_accepted,
                                                  ws, ws_bytes, stream)


def spec_verify_read_error(ws: int, stream: int = 0):
    code = ctypes.c_int32(0)
    st = load_library().spec_verify_read_error(ws, stream, ctypes.addressof(code))
    return st, code.value


def spec_verify_set_lazy_split_bytes(nbytes: float) -> None:
    load_library().spec_verify_set_lazy_split_bytes(float(nbytes))


def spec_verify_set_wait_limit(polls: int) -> None:
    load_library().spec_verify_set_wait_limit(polls)


def spec_verify_default_wait_limit() -> int:
    return load_library().spec_verify_default_wait_limit()


def spec_verify_status_string(status: int) -> str:
    try:
        return load_library().spec_verify_status_string(status).decode()
    except ImportError:
        return "status %d" % status


# ---- torch marshalling ----------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SPEC_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return SPEC_DTYPE_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check_tensor(t, name: str, shape, dtypes, device=None):
    """Raises unless t is a contiguous CUDA tensor of one of dtypes, of the
    given shape (None entries match anything) and, when given, on device: the
    C ABI reads raw device memory, so a strided, host-resident or mistyped
    tensor would be read as garbage rather than rejected."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, got device {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if len(t.shape) != len(shape) or any(w is not None and w != h for w, h in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple('*' if w is None else w for w in shape)}, "
                         f"got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _logits_dtypes():
    torch = _torch()
    return (torch.float32, torch.bfloat16)


def _stream(stream) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(status: int, what: str):
    if status != SPEC_OK:
        raise SpecVerifyError(status, what)


class Workspace:
    """Device scratch for the verification calls, zero-filled when it is
    (re)allocated so the error word starts clear.  Grows on demand."""

    def __init__(self, device=None):
        torch = _torch()
        self.device = torch.device("cuda") if device is None else torch.device(device)
        self.buf = None

    def get(self, B: int, g: int, V: int, stream=None):
        return self.get_bytes(spec_verify_workspace_size(B, g, V), stream)

    def get_bytes(self, need: int, stream=None):
        torch = _torch()
        if self.buf is None or self.buf.numel() < need:
            self.buf = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
            _check(spec_verify_workspace_init(self.buf.data_ptr(), self.buf.numel(), _stream(stream)),
                   "spec_verify_workspace_init")
        return self.buf.data_ptr(), self.buf.numel()

    def read_error(self, stream=None) -> int:
        st, code = spec_verify_read_error(self.buf.data_ptr(), _stream(stream))
        _check(st, "spec_verify_read_error")
        return code


_default_ws = {}


def _ws(workspace, device):
    if workspace is not None:
        return workspace
    key = str(device)
    if key not in _default_ws:
        _default_ws[key] = Workspace(device)
    return _default_ws[key]


def verify_sample(target, draft, draft_tokens, uniforms, temperature: float, *, logprobs=False,
                  workspace: Optional[Workspace] = None, out=None, stream=None, lazy=False):
    """Stochastic verification (see spec_verify_sample).  target [B, g+1, V],
    draft [B, g, V] (same dtype), draft_tokens [B, g] int32, uniforms
    [B, g+1] float32, all contiguous CUDA tensors.  Returns (tokens [B, g+1],
    num_accepted [B]) or, with logprobs=True, also [B, g, 2] log-probabilities.
    lazy=True: spec_verify_sample_lazy (same tokens and counts; the rows of the
    position groups after the one holding a sequence's first rejection are not
    read, and the log-probabilities of positions after the rejection are NaN)."""
    torch = _torch()
    _check_tensor(target, "target", (None, None, None), _logits_dtypes())
    B, g1, V = target.shape
    g = g1 - 1
    dev = target.device
    if g > 0:
        _check_tensor(draft, "draft", (B, g, V), (target.dtype,), dev)
        _check_tensor(draft_tokens, "draft_tokens", (B, g), (torch.int32,), dev)
    _check_tensor(uniforms, "uniforms", (B, g1), (torch.float32,), dev)
    if out is None:
        tok = torch.empty((B, g1), dtype=torch.int32, device=dev)
        acc = torch.empty((B,), dtype=torch.int32, device=dev)
        lp = torch.empty((B, g, 2), dtype=torch.float32, device=dev) if logprobs else None
    else:
        tok, acc, lp = out
        _check_tensor(tok, "out tokens", (B, g1), (torch.int32,), dev)
        _check_tensor(acc, "out num_accepted", (B,), (torch.int32,), dev)
        if lp is not None:
            _check_tensor(lp, "out logprobs", (B, g, 2), (torch.float32,), dev)
    ws = _ws(workspace, dev)
    wp, wb = ws.get(B, g, V, stream)
    fn = spec_verify_sample_lazy if lazy else spec_verify_sample
    st = fn(_ptr(target), _ptr(draft) if g > 0 else None, _dtype_code(target),
            _ptr(draft_tokens) if g > 0 else None, _ptr(uniforms), float(temperature), B, g, V,
            _ptr(tok), _ptr(acc), _ptr(lp), wp, wb, _stream(stream))
    _check(st, "spec_verify_sample_lazy" if lazy else "spec_verify_sample")
    return (tok, acc, lp) if logprobs else (tok, acc)


def topk_exclude(logits, K: int, exclude=None, *, values=False,
                 workspace: Optional[Workspace] = None, out=None, stream=None):
    """Top-K branch tokens (see spec_topk_exclude).  logits [..., V] contiguous
    CUDA tensor (bf16 or fp32), exclude int32 with one entry per row or None.
    Returns idx [..., K] int32 (and, with values=True, the logits [..., K])."""
    torch = _torch()
    _check_tensor(logits, "logits", (None,) * max(logits.dim(), 1), _logits_dtypes())
    V = logits.shape[-1]
    rows = logits.numel() // V
    dev = logits.device
    if exclude is not None:
        _check_tensor(exclude, "exclude", tuple(logits.shape[:-1]), (torch.int32,), dev)
    if out is None:
        idx = torch.empty((*logits.shape[:-1], K), dtype=torch.int32, device=dev)
        val = torch.empty((*logits.shape[:-1], K), dtype=torch.float32, device=dev) if values else None
    else:
        idx, val = out
        _check_tensor(idx, "out idx", (*logits.shape[:-1], K), (torch.int32,), dev)
        if val is not None:
            _check_tensor(val, "out values", (*logits.shape[:-1], K), (torch.float32,), dev)
    ws = _ws(workspace, dev)
    wp, wb = ws.get_bytes(spec_topk_workspace_size(rows, V, K), stream)
    st = spec_topk_exclude(_ptr(logits), _dtype_code(logits), rows, V, K, _ptr(exclude), _ptr(idx),
                           _ptr(val), wp, wb, _stream(stream))
    _check(st, "spec_topk_exclude")
    return (idx, val) if values else idx


def ngram_retrieve(tokens, lengths, w: int, L: int, max_matches: int, *,
                   workspace: Optional[Workspace] = None, stream=None):
    """Lexical retrieval (see spec_ngram_retrieve).  tokens [B, n_max] int32
    (n_max a multiple of 4), lengths [B] int32, CUDA tensors.  Returns
    (count [B], matches [B, max_matches], draft [B, L])."""
    torch = _torch()
    _check_tensor(tokens, "tokens", (None, None), (torch.int32,))
    B, n_max = tokens.shape
    dev = tokens.device
    _check_tensor(lengths, "lengths", (B,), (torch.int32,), dev)
    cnt = torch.empty((B,), dtype=torch.int32, device=dev)
    mat = torch.empty((B, max_matches), dtype=torch.int32, device=dev)
    dr = torch.empty((B, max(L, 1)), dtype=torch.int32, device=dev)
    ws = _ws(workspace, dev)
    wp, wb = ws.get_bytes(spec_ngram_workspace_size(B, n_max, max_matches), stream)
    st = spec_ngram_retrieve(_ptr(tokens), _ptr(lengths), B, n_max, w, L, max_matches, _ptr(cnt),
                             _ptr(mat), _ptr(dr), wp, wb, _stream(stream))
    _check(st, "spec_ngram_retrieve")
    return cnt, mat, dr[:, :L]


def cosine_topk(hidden, query, delta: int, positions=None, *,
                workspace: Optional[Workspace] = None, stream=None):
    """Semantic fallback (see spec_cosine_topk).  hidden [B, W, d], query
    [B, d] (same dtype, bf16 or fp32), positions [B, W] int32 or None, CUDA
    tensors.  Returns (idx [B, delta], pos [B, delta], score [B, delta])."""
    torch = _torch()
    _check_tensor(hidden, "hidden", (None, None, None), _logits_dtypes())
    B, W, d = hidden.shape
    dev = hidden.device
    _check_tensor(query, "query", (B, d), (hidden.dtype,), dev)
    if positions is not None:
        _check_tensor(positions, "positions", (B, W), (torch.int32,), dev)
    idx = torch.empty((B, delta), dtype=torch.int32, device=dev)
    pos = torch.empty((B, delta), dtype=torch.int32, device=dev)
    sc = torch.empty((B, delta), dtype=torch.float32, device=dev)
    ws = _ws(workspace, dev)
    wp, wb = ws.get_bytes(spec_cosine_workspace_size(B, W), stream)
    st = spec_cosine_topk(_ptr(hidden), _ptr(query), _dtype_code(hidden), B, W, d, delta,
                          _ptr(positions), _ptr(idx), _ptr(pos), _ptr(sc), wp, wb, _stream(stream))
    _check(st, "spec_cosine_topk")
    return idx, pos, sc


def verify_greedy(target, draft_tokens, *, workspace: Optional[Workspace] = None, out=None,
                  stream=None):
    """Greedy verification (see spec_verify_greedy).  Returns (tokens, num_accepted)."""
    torch = _torch()
    _check_tensor(target, "target", (None, None, None), _logits_dtypes())
    B, g1, V = target.shape
    g = g1 - 1
    dev = target.device
    if g > 0:
        _check_tensor(draft_tokens, "draft_tokens", (B, g), (torch.int32,), dev)
    if out is None:
        tok = torch.empty((B, g1), dtype=torch.int32, device=dev)
        acc = torch.empty((B,), dtype=torch.int32, device=dev)
    else:
        tok, acc = out
        _check_tensor(tok, "out tokens", (B, g1), (torch.int32,), dev)
        _check_tensor(acc, "out num_accepted", (B,), (torch.int32,), dev)
    ws = _ws(workspace, dev)
    wp, wb = ws.get(B, g, V, stream)
    st = spec_verify_greedy(_ptr(target), _dtype_code(target), _ptr(draft_tokens) if g > 0 else None,
                            B, g, V, _ptr(tok), _ptr(acc), wp, wb, _stream(stream))
    _check(st, "spec_verify_greedy")
    return tok, acc


def verify_tree_greedy(target, node_tokens, parents, *, workspace: Optional[Workspace] = None,
                       out=None, stream=None):
    """Greedy tree verification (see spec_verify_tree_greedy).  Returns
    (path_nodes [B, N], tokens [B, N], num_accepted [B])."""
    torch = _torch()
    _check_tensor(target, "target", (None, None, None), _logits_dtypes())
    B, N, V = target.shape
    dev = target.device
    _check_tensor(node_tokens, "node_tokens", (B, N), (torch.int32,), dev)
    _check_tensor(parents, "parents", (B, N), (torch.int32,), dev)
    if out is None:
        nodes = torch.empty((B, N), dtype=torch.int32, device=dev)
        tok = torch.empty((B, N), dtype=torch.int32, device=dev)
        acc = torch.empty((B,), dtype=torch.int32, device=dev)
    else:
        nodes, tok, acc = out
        _check_tensor(nodes, "out path_nodes", (B, N), (torch.int32,), dev)
        _check_tensor(tok, "out tokens", (B, N), (torch.int32,), dev)
        _check_tensor(acc, "out num_accepted", (B,), (torch.int32,), dev)
    ws = _ws(workspace, dev)
    wp, wb = ws.get(B, N, V, stream)
    st = spec_verify_tree_greedy(_ptr(target), _dtype_code(target), _ptr(node_tokens),
                                 _ptr(parents), B, N, V, _ptr(nodes), _ptr(tok), _ptr(acc), wp, wb,
                                 _stream(stream))
    _check(st, "spec_verify_tree_greedy")
    return nodes, tok, acc


# ---- cache, attention and log-probabilities ------------------------------------------
# These calls run on every layer of every step, where the host's share counts:
# the fixed part of their arguments is checked once (KVCache), the rest in
# _marshal (csrc/sv_torch.cpp), which also allocates the outputs and makes the
# C call.
_marshal_module = None


def _load_marshal():          # (importing the submodule binds the package's name _marshal to it)
    global _marshal_module
    if _marshal_module is None:
        torch = _torch()
        load_library()
        import importlib
        from . import _build
        try:
            # (one of another torch may load and take its classes for something else)
            if not _build.marshal_matches(os.path.dirname(torch.__file__)):
                raise ImportError("_marshal.so was built with another torch or Python")
            _marshal_module = importlib.import_module("._marshal", __name__)
        except ImportError as e:
            raise ImportError(f"{os.path.join(_HERE, '_marshal.so')} is not built for this torch; run "
                              "__graft_entry__.build() first") from e
    return _marshal_module


def _scratch(workspace: Workspace, head: int, need: int, stream):
    """The bytes of a Workspace from `head` on, grown to head + need, as _marshal takes them."""
    workspace.get_bytes(head + need, stream)
    return workspace.buf[head:]


class KVCache:
    """A paged key-value cache (see spec_kv_cache_t): views of the caller's tensors,
    checked once.

    k, v         [pages, page_size, kv_heads, head_dim], or [layers, pages, ...]: bfloat16, or
                 float8_e4m3fn with k_scale / v_scale (float32, the shape without head_dim).
                 Any strides with the last dimension contiguous, the same for k and v:
                 a head-first pool is passed transposed, keys beside values as slices.
    block_table  [B, max_pages] int32, contiguous
    A call on one layer takes cache.layer(i) (layer 0 of a cache without layers is
    the cache itself); kv_compact takes them all."""

    def __init__(self, k, v, block_table, k_scale=None, v_scale=None, _error=None):
        torch = _torch()
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
            if t.device.type != "cuda":
                raise ValueError(f"{name} must be a CUDA tensor, got device {t.device}")
            if t.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
                raise TypeError(f"{name} must have dtype bfloat16 or float8_e4m3fn, got {t.dtype}")
            if t.dim() not in (4, 5) or t.stride(-1) != 1:
                raise ValueError(f"{name} must be [layers,] pages, page_size, kv_heads, head_dim "
                                 "with head_dim contiguous")
        if v.shape != k.shape or v.stride() != k.stride() or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must agree in shape, strides, dtype and device")
        dev = k.device
        _check_tensor(block_table, "block_table", (None, None), (torch.int32,), dev)
        if dev.index is None or dev.index != block_table.get_device():
            raise ValueError(f"the cache is on {dev}, its block table on {block_table.device}")
        fp8 = k.dtype == torch.float8_e4m3fn
        if fp8 != (k_scale is not None) or fp8 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to a float8_e4m3fn cache, and to it alone")
        if fp8:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if not isinstance(t, torch.Tensor):
                    raise TypeError(f"{name} must be a torch tensor, got {type(t).__name__}")
                if t.dtype != torch.float32 or t.shape != k.shape[:-1] or t.device != dev:
                    raise ValueError(f"{name} must be float32 {tuple(k.shape[:-1])} on {dev}")
            if k_scale.stride() != v_scale.stride():
                raise ValueError("k_scale and v_scale must have the same strides")
        self.k, self.v, self.k_scale, self.v_scale, self.block_table = k, v, k_scale, v_scale, block_table
        self.error = torch.zeros(1, dtype=torch.int32, device=dev) if _error is None else _error
        self.device = dev
        L = k.dim() == 5
        pages, page, heads, dim = k.shape[-4:]
        ks, ss = k.stride(), k_scale.stride() if fp8 else (0,) * (k.dim() - 1)
        self.batch, self.max_pages = block_table.shape
        self.layers = k.shape[0] if L else 1
        self.page_size, self.kv_heads, self.head_dim, self.fp8 = page, heads, dim, fp8
        self.struct = KVCacheStruct(
            k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), block_table.data_ptr(),
            self.error.data_ptr(), ks[-4], ks[-3], ks[-2], ks[0] if L else 0,
            ss[-3], ss[-2], ss[-1], ss[0] if L else 0,
            SPEC_DTYPE_E4M3 if fp8 else SPEC_DTYPE_BF16, self.layers, pages, page, self.max_pages,
            heads, dim)
        self.addr, self.index, self.scale = ctypes.addressof(self.struct), dev.index, dim ** -0.5

    def layer(self, i: int) -> "KVCache":
        """One layer of the cache (sharing its block table and error word)."""
        if self.k.dim() == 4:
            if i != 0:
                raise IndexError(f"layer {i} of a cache of one layer")
            return self
        sc = (self.k_scale[i], self.v_scale[i]) if self.fp8 else (None, None)
        return KVCache(self.k[i], self.v[i], self.block_table, *sc, _error=self.error)

    def read_error(self, stream=None) -> int:
        """The SPEC_DEVERR_* bits that calls on this cache raised; clears them."""
        st, code = spec_verify_read_error(self.error.data_ptr(), _stream(stream))
        _check(st, "spec_verify_read_error")
        return code


def kv_append(cache: KVCache, q, k, v, context_lens, rope=None, *, q_weight=None, k_weight=None,
              eps: float = 1e-6, interleaved: bool = False, new_lens=None, positions=None, out=None,
              stream=None):
    """Normalises and rotates the new positions' queries and keys and writes keys and
    values into the cache (see spec_kv_append).  q [B, N, q_heads, head_dim] (None: keys
    and values only), k, v [B, N, kv_heads, head_dim] bfloat16; slices of one fused
    projection are fine.  context_lens [B] int32, rope [rows, rot_dim] float32 (cosines, then
    sines) or None, weights [head_dim] bfloat16 or None, positions [B, N] int32 or None,
    new_lens [B] int32 or None.  Returns the prepared queries [B, N, q_heads, head_dim]."""
    return (_marshal_module or _load_marshal()).kv_append(
        cache.addr, cache.batch, cache.index, q, k, v, context_lens, rope, q_weight, k_weight, eps,
        interleaved, new_lens, positions, out, stream)


def kv_read(cache: KVCache, T: int, *, starts=None, counts=None, dtype=None, stream=None):
    """Cached positions as dense rows (see spec_kv_read): (k, v), each [B, T, kv_heads,
    head_dim] of dtype (bfloat16 by default, or float32), row t holding position
    starts[b] + t for t < counts[b], zeros after that.  B is the length of starts or
    counts, or the cache's batch.  Small results (up to 2^20 elements) share one
    allocation."""
    f32 = False
    if dtype is not None:
        if dtype not in _logits_dtypes():
            raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
        f32 = dtype == _torch().float32
    return (_marshal_module or _load_marshal()).kv_read(
        cache.addr, cache.batch, cache.index, T, starts, counts, f32, stream)


def kv_compact(cache: KVCache, context_lens, path_nodes, num_accepted, *, stream=None) -> None:
    """Moves the accepted path of every sequence's draft tree to the front of its slots, in
    every layer (see spec_kv_compact).  path_nodes [B, N] and num_accepted [B] are
    verify_tree_greedy's."""
    (_marshal_module or _load_marshal()).kv_compact(
        cache.addr, cache.batch, cache.index, context_lens, path_nodes, num_accepted, stream)


def paged_attention(q, cache: KVCache, context_lens, *, parents=None, new_lens=None,
                    scale: Optional[float] = None, lse: bool = False, out=None, workspace=None,
                    stream=None):
    """Attention of new positions, already appended, over the cache (see
    spec_paged_attention).  q [B, N, q_heads, head_dim] bfloat16, context_lens [B] int32,
    parents [B, N] int32 for draft trees (None: chains), new_lens [B] int32 or None; scale
    defaults to head_dim ** -0.5.  Returns out [B, N, q_heads, head_dim] bfloat16, with
    lse=True also [B, N, q_heads] float32.  workspace: a Workspace (the first 256 bytes, with its
    error word, are left alone), or a uint8 tensor of spec_attention_workspace_size() bytes, of
    any contents, that no call on another stream uses at the same time.  None: one kept for
    the device and stream from the first such call to the program's end, as large as the
    largest has needed (some 38 MB for 144 rows of 128 per cached head); a captured call gets one
    of its graph's."""
    if isinstance(workspace, Workspace):
        workspace = _scratch(workspace, 256, load_library().spec_attention_workspace_size(
            q.shape[0], q.shape[1], q.shape[2], cache.kv_heads, cache.head_dim), stream)
    return (_marshal_module or _load_marshal()).paged_attention(
        cache.addr, cache.batch, cache.index, q, context_lens, parents, new_lens,
        cache.scale if scale is None else scale, lse, out, workspace, stream)


def token_logprobs(logits, tokens, K: int = 0, *, temperature: float = 1.0, workspace=None,
                   stream=None):
    """Log-probabilities of tokens with entropies and top alternatives (see
    spec_token_logprobs).  logits [..., V] contiguous bfloat16 or float32, tokens [...]
    int32.  Returns (logprob [...], entropy [...], top_idx [..., K] int32, top_logprob
    [..., K]), which share one allocation; the last two None for K = 0.  workspace: a Workspace, whose
    read_error() then tells of bad tokens and empty rows (NaN in the results either way), or a
    uint8 tensor of spec_logprobs_workspace_size() bytes, its first 256 zero.  None: one kept
    for the device and stream to the program's end, as large as the largest call has needed (a
    captured call gets one of its graph's), whose error word is not read."""
    if isinstance(workspace, Workspace):
        workspace = _scratch(workspace, 0, load_library().spec_logprobs_workspace_size(
            logits.numel() // max(logits.shape[-1], 1), logits.shape[-1], K), stream)
    return (_marshal_module or _load_marshal()).token_logprobs(logits, tokens, K, temperature, workspace, stream)


# ---- the target model's dense side -----------------------------------------------------
_ACTS = {"silu": SPEC_ACT_SILU, "gelu": SPEC_ACT_GELU_TANH}


def _f32(dtype) -> bool:
    torch = _torch()
    if dtype is torch.float32:
        return True
    if dtype is not torch.bfloat16:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return False


def add_norm(x, weight=None, residual=None, *, eps: float = 1e-6, e4m3: bool = False, dtype=None,
             sum_out=None, stream=None):
    """The residual's addition and the root-mean-square norm of its sum (see spec_add_norm).
    x [..., dim] bfloat16 or float32, weight [dim] bfloat16 or None, residual of x's shape,
    bfloat16 or float32, or None; rows may be slices (one stride apart, multiples of 16 bytes).
    Returns the normed rows [..., dim] of dtype (bfloat16 by default, or float32); with e4m3=True
    float8_e4m3fn rows and their scales [..., ceil(dim / 128)] float32 (strided as matmul_e4m3
    takes them); and with a residual, last, the sum in the residual's dtype, which sum_out
    may name a place for: the residual itself, say.  Small outputs (up to 2^20 elements) share
    one allocation."""
    if e4m3 and dtype is not None:
        raise ValueError("dtype is the output's without e4m3")
    return (_marshal_module or _load_marshal()).add_norm(
        x, weight, residual, eps, e4m3, dtype is not None and _f32(dtype), sum_out, stream)


def gated_act(gate, up=None, *, act: str = "silu", e4m3: bool = False, dtype=None, stream=None):
    """act(gate) * up (see spec_gated_act), act "silu" or "gelu" (its tanh form).  gate and up [...,
    dim] bfloat16 or float32, slices of one projection or, with up None, gate [..., 2 dim] holding
    both side by side.  Returns [..., dim] of dtype, or with e4m3=True rows and scales, as
    add_norm does."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    if e4m3 and dtype is not None:
        raise ValueError("dtype is the output's without e4m3")
    return (_marshal_module or _load_marshal()).gated_act(
        gate, up, _ACTS[act], e4m3, dtype is not None and _f32(dtype), stream)


def quantize_e4m3(x, *, block_rows: int = 1, stream=None):
    """Rounds bfloat16 or float32 rows to 8 bits (see spec_quantize_e4m3): rows x [..., dim] with a scale
    for each 128 of their elements, or, with block_rows=128, a weight x [N, dim] with one for each
    128 x 128.  Returns (float8_e4m3fn of x's shape, scales float32: [..., ceil(dim / 128)], or
    [ceil(N / 128), ceil(dim / 128)])."""
    return (_marshal_module or _load_marshal()).quantize_e4m3(x, block_rows, stream)


def matmul_e4m3(x, x_scale, w, w_scale, *, dtype=None, out=None, workspace=None, stream=None):
    """The product of 8-bit rows with an 8-bit weight (see spec_matmul_e4m3): x [..., K] and w [N, K]
    float8_e4m3fn with the scales that quantize_e4m3, add_norm and gated_act give, [...,
    ceil(K / 128)] with stride 1 from row to row, and [ceil(N / 128), ceil(K / 128)].  Rows may be a part of
    what those calls gave, q[a:b] with scale[a:b]: one row, or more than 64, any; 2 to 64 rows from a
    multiple of 4 on.  Returns [..., N] of dtype (bfloat16 by default, or float32).  workspace: a
    Workspace, whose read_error() then tells of waits that ran out (NaN in the results either way),
    or a uint8 tensor of spec_matmul_workspace_size() bytes, its first 256 zero, that no call on
    another stream uses at the same time.  None: one kept for the device and stream to the
    program's end (a captured call gets one of its graph's)."""
    if isinstance(workspace, Workspace):
        workspace = _scratch(workspace, 0, load_library().spec_matmul_workspace_size(
            x.numel() // max(x.shape[-1], 1), w.shape[0], x.shape[-1]), stream)
    return (_marshal_module or _load_marshal()).matmul_e4m3(
        x, x_scale, w, w_scale, dtype is not None and _f32(dtype), out, workspace, stream)


def matmul_plan(M: int, N: int, K: int, sms: int = 0, clusters=(0, 0, 0)):
    """How matmul_e4m3 divides a product of these sizes (see spec_matmul_plan): (way, a tile's weight rows, CTAs
    that take a tile together, CTAs or pairs in all, parts of a tile), on the current device or on
    one of `sms` SMs, of which `clusters` clusters of two, four and eight CTAs run at once."""
    given, plan = (ctypes.c_int32 * 3)(*clusters), (ctypes.c_int32 * 5)()
    _check(load_library().spec_matmul_plan(M, N, K, sms, ctypes.addressof(given), ctypes.addressof(plan)), "spec_matmul_plan")
    return tuple(plan)
