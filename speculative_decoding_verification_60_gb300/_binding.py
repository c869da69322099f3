"""ctypes binding of libspecverify (argument marshalling only).

Every step of verification runs in the library's CUDA kernels; this module
only checks tensor shapes and dtypes, allocates output tensors with PyTorch
and passes raw device pointers and the current CUDA stream.  It fails loudly
when the library has not been built: there is no fallback path.
"""

from __future__ import annotations

import array
import ctypes
import operator
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspecverify.so")

SPEC_OK = 0
SPEC_BF16, SPEC_F32, SPEC_F16 = 0, 1, 2
SPEC_OP_LINEAR, SPEC_OP_TREE = 0, 1
CHILD_WOR, CHILD_IID, CHILD_DETERMINISTIC = 0, 1, 2
DEVERR_TOKEN, DEVERR_NONFINITE, DEVERR_PARENT, DEVERR_LENGTH, DEVERR_CAPACITY = 1, 2, 4, 8, 32
TAIL_RENORM, TAIL_BUCKET = 0, 1

# Every symbol declared in include/specverify.h.
EXPORTS = ("spec_workspace_size", "spec_verify_linear", "spec_verify_linear_compact", "spec_linear_stats_decide",
           "spec_linear_draw", "spec_verify_linear_noalloc", "spec_verify_tree", "spec_verify_tree_dynamic",
           "spec_compact_accepted",
           "spec_sample_rows", "spec_token_logprobs", "spec_distill_topk", "spec_distill_topk_backward",
           "spec_advance_blocks", "spec_append_kv", "spec_tree_attention_workspace", "spec_tree_attention",
           "spec_adjust_logits", "spec_keep_path", "spec_status_string")


class SamplingParams(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float), ("seed", ctypes.c_uint64),
                ("child_mode", ctypes.c_int32)]


class CacheLayout(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_int32), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("block_stride", ctypes.c_int64), ("entry_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Adjustments(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("history_stride", ctypes.c_int64), ("history_lens", ctypes.c_void_p),
                ("prompt_lens", ctypes.c_void_p), ("history_capacity", ctypes.c_int32), ("drafted", ctypes.c_void_p),
                ("drafted_stride", ctypes.c_int64), ("parent", ctypes.c_void_p), ("parent_stride", ctypes.c_int64),
                ("n_nodes", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_count", ctypes.c_int32), ("allowed", ctypes.c_void_p), ("allowed_stride", ctypes.c_int64)]


class SpecError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} returned {status_string(status)} ({status})")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load libspecverify.so; raises when it is missing (build it with
    ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libspecverify.so not found at {LIB_PATH}: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.spec_workspace_size.argtypes = [I, I, I, I, I]
    lib.spec_workspace_size.restype = Z
    lib.spec_verify_linear.argtypes = [P, P, I, P, I, I, I, P, P, ctypes.POINTER(SamplingParams),
                                       P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_linear.restype = I
    lib.spec_verify_linear_compact.argtypes = [P, P, I, P, I, I, I, P, P, ctypes.POINTER(SamplingParams), P, I,
                                               P, P, P, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_linear_compact.restype = I
    lib.spec_linear_stats_decide.argtypes = [P, P, I, P, I, I, I, P, P, ctypes.POINTER(SamplingParams),
                                             P, P, P, P, P, P, Z, P]
    lib.spec_linear_stats_decide.restype = I
    lib.spec_linear_draw.argtypes = [P, P, I, P, I, I, I, P, P, ctypes.POINTER(SamplingParams), P, I,
                                     P, P, P, P, P, Z, P]
    lib.spec_linear_draw.restype = I
    lib.spec_verify_linear_noalloc.argtypes = [P, P, I, P, I, I, I, P, P, ctypes.POINTER(SamplingParams),
                                               P, P, P, P, P, P, P]
    lib.spec_verify_linear_noalloc.restype = I
    lib.spec_verify_tree.argtypes = [P, P, I, P, P, I, I, I, I, P, P, ctypes.POINTER(SamplingParams),
                                     P, P, P, P, P, Z, P]
    lib.spec_verify_tree.restype = I
    lib.spec_verify_tree_dynamic.argtypes = [P, P, I, P, P, P, I, I, I, I, P, P, ctypes.POINTER(SamplingParams),
                                             P, P, P, P, P, Z, P]
    lib.spec_verify_tree_dynamic.restype = I
    lib.spec_compact_accepted.argtypes = [P, I, I, I, P, P, P, I, P, P, P, P, P]
    lib.spec_compact_accepted.restype = I
    lib.spec_sample_rows.argtypes = [P, I, I, I, P, P, ctypes.POINTER(SamplingParams), P, P, P]
    lib.spec_sample_rows.restype = I
    L, F = ctypes.c_int64, ctypes.c_float
    lib.spec_token_logprobs.argtypes = [P, I, I, I, L, P, F, I, P, P, P, P, P, P, P]
    lib.spec_token_logprobs.restype = I
    lib.spec_distill_topk.argtypes = [P, I, I, I, L, P, P, I, P, F, I, P, P, P, L, P, P]
    lib.spec_distill_topk.restype = I
    lib.spec_distill_topk_backward.argtypes = [P, I, I, I, L, P, P, I, P, P, F, P, L, P]
    lib.spec_distill_topk_backward.restype = I
    lib.spec_advance_blocks.argtypes = [P, P, P, I, I, P, I, L, P, P, I, P, P, P, P, P, P, P, I, P, P]
    lib.spec_advance_blocks.restype = I
    layout = ctypes.POINTER(CacheLayout)
    lib.spec_append_kv.argtypes = [P, P, P, I, I, I, L, L, L, L, L, L, P, P, F, P, P, I, I, P, P, P, P, layout, P, P]
    lib.spec_append_kv.restype = I
    lib.spec_tree_attention_workspace.argtypes = [I, I, I, I, I]
    lib.spec_tree_attention_workspace.restype = Z
    lib.spec_tree_attention.argtypes = [P, I, I, I, I, L, L, L, P, P, layout, P, I, L, P, P, L, P, F, P, P, P, Z, P]
    lib.spec_tree_attention.restype = I
    lib.spec_adjust_logits.argtypes = [P, I, I, I, I, L, ctypes.POINTER(Adjustments), P, L, P, P]
    lib.spec_adjust_logits.restype = I
    lib.spec_keep_path.argtypes = [P, I, I, layout, I, I, P, P, P, P, I, L, P, P]
    lib.spec_keep_path.restype = I
    lib.spec_status_string.argtypes = [I]
    lib.spec_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().spec_status_string(int(status)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check(t, name, dtype=None, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def workspace_size(op: int, B: int, k_or_N: int, V: int, dtype_code: int = SPEC_BF16) -> int:
    return int(load().spec_workspace_size(op, B, k_or_N, V, dtype_code))


def verify_linear(target, draft, draft_tokens, temperature: float, top_p: float = 1.0, seed: int = 0,
                  request_ids=None, positions=None, workspace=None, out=None, stream=None) -> dict:
    """``spec_verify_linear`` on torch tensors.

    target [B, k+1, V] and draft [B, k, V] (bf16 or fp32; draft may be None
    when temperature == 0), draft_tokens [B, k] int32, request_ids and
    positions [B] int64 or None.  Returns a dict of device tensors:
    accepted_len [B], out_tokens [B, k+1], accept_prob [B, k],
    token_probs [B, k, 2], len_hist [k+1], dev_error [1]."""
    lib = load()
    B, k1, V = target.shape
    k = k1 - 1
    dt = _dtype_code(target)
    _check(target, "target")
    _check(draft, "draft", target.dtype, (B, k, V))
    _check(draft_tokens, "draft_tokens", torch.int32, (B, k))
    _check(request_ids, "request_ids", torch.int64, (B,))
    _check(positions, "positions", torch.int64, (B,))
    dev = target.device
    if out is None:
        out = dict(
            accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
            out_tokens=torch.empty(B, k + 1, dtype=torch.int32, device=dev),
            accept_prob=torch.empty(B, k, dtype=torch.float32, device=dev),
            token_probs=torch.empty(B, k, 2, dtype=torch.float32, device=dev),
            len_hist=torch.empty(k + 1, dtype=torch.int32, device=dev),
            dev_error=torch.empty(1, dtype=torch.int32, device=dev),
        )
    need = workspace_size(SPEC_OP_LINEAR, B, k, V, dt)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    sp = SamplingParams(float(temperature), float(top_p), int(seed) & (2**64 - 1), 0)
    st = lib.spec_verify_linear(_ptr(target), _ptr(draft), dt, _ptr(draft_tokens), B, k, V, _ptr(request_ids),
                                _ptr(positions), ctypes.byref(sp), _ptr(out["accepted_len"]),
                                _ptr(out["out_tokens"]), _ptr(out.get("accept_prob")),
                                _ptr(out.get("token_probs")), _ptr(out.get("len_hist")),
                                _ptr(out.get("dev_error")), _ptr(workspace), workspace.numel(), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_verify_linear", st)
    return out


def verify_linear_compact(target, draft, draft_tokens, hidden, temperature: float, top_p: float = 1.0,
                          seed: int = 0, request_ids=None, positions=None, stream=None) -> dict:
    """``spec_verify_linear_compact`` on torch tensors: verify_linear plus
    hidden [B, k+1, H] bf16; the dict adds out_hidden [B*(k+1), H],
    offsets [B+1] and next_tokens [B*(k+1)] (rows past offsets[B] are not
    written)."""
    lib = load()
    B, k1, V = target.shape
    k = k1 - 1
    H = hidden.shape[-1]
    dt = _dtype_code(target)
    _check(target, "target")
    _check(draft, "draft", target.dtype, (B, k, V))
    _check(draft_tokens, "draft_tokens", torch.int32, (B, k))
    _check(hidden, "hidden", torch.bfloat16, (B, k + 1, H))
    _check(request_ids, "request_ids", torch.int64, (B,))
    _check(positions, "positions", torch.int64, (B,))
    dev = target.device
    out = dict(
        accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
        out_tokens=torch.empty(B, k + 1, dtype=torch.int32, device=dev),
        accept_prob=torch.empty(B, k, dtype=torch.float32, device=dev),
        token_probs=torch.empty(B, k, 2, dtype=torch.float32, device=dev),
        len_hist=torch.empty(k + 1, dtype=torch.int32, device=dev),
        out_hidden=torch.zeros(B * (k + 1), H, dtype=torch.bfloat16, device=dev),
        offsets=torch.empty(B + 1, dtype=torch.int32, device=dev),
        next_tokens=torch.full((B * (k + 1),), -1, dtype=torch.int32, device=dev),
        dev_error=torch.empty(1, dtype=torch.int32, device=dev),
    )
    need = workspace_size(SPEC_OP_LINEAR, B, k, V, dt)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    sp = SamplingParams(float(temperature), float(top_p), int(seed) & (2**64 - 1), 0)
    st = lib.spec_verify_linear_compact(_ptr(target), _ptr(draft), dt, _ptr(draft_tokens), B, k, V,
                                        _ptr(request_ids), _ptr(positions), ctypes.byref(sp), _ptr(hidden), H,
                                        _ptr(out["accepted_len"]), _ptr(out["out_tokens"]), _ptr(out["accept_prob"]),
                                        _ptr(out["token_probs"]), _ptr(out["len_hist"]), _ptr(out["out_hidden"]),
                                        _ptr(out["offsets"]), _ptr(out["next_tokens"]), _ptr(out["dev_error"]),
                                        _ptr(ws), ws.numel(), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_verify_linear_compact", st)
    return out


def verify_tree(target, draft, node_tokens, parent, max_depth: int, temperature: float, top_p: float = 1.0,
                seed: int = 0, child_mode: int = CHILD_WOR, request_ids=None, positions=None, stream=None) -> dict:
    """``spec_verify_tree`` on torch tensors: target/draft [B, N, V],
    node_tokens [B, N] int32, parent [N] int32 (device).  Returns
    accepted_len [B], path_nodes [B, W], out_tokens [B, W], dev_error [1]
    with W = max_depth + 1."""
    lib = load()
    B, N, V = target.shape
    dt = _dtype_code(target)
    _check(target, "target")
    _check(draft, "draft", target.dtype, (B, N, V))
    _check(node_tokens, "node_tokens", torch.int32, (B, N))
    _check(parent, "parent", torch.int32, (N,))
    _check(request_ids, "request_ids", torch.int64, (B,))
    _check(positions, "positions", torch.int64, (B,))
    dev = target.device
    W = int(max_depth) + 1
    out = dict(
        accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
        path_nodes=torch.empty(B, W, dtype=torch.int32, device=dev),
        out_tokens=torch.empty(B, W, dtype=torch.int32, device=dev),
        dev_error=torch.empty(1, dtype=torch.int32, device=dev),
    )
    need = workspace_size(SPEC_OP_TREE, B, N, V, dt)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    sp = SamplingParams(float(temperature), float(top_p), int(seed) & (2**64 - 1), int(child_mode))
    st = lib.spec_verify_tree(_ptr(target), _ptr(draft), dt, _ptr(node_tokens), _ptr(parent), B, N, V,
                              int(max_depth), _ptr(request_ids), _ptr(positions), ctypes.byref(sp),
                              _ptr(out["accepted_len"]), _ptr(out["path_nodes"]), _ptr(out["out_tokens"]),
                              _ptr(out["dev_error"]), _ptr(ws), ws.numel(), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_verify_tree", st)
    return out


def verify_tree_dynamic(target, draft, node_tokens, parent, n_nodes, max_depth: int, temperature: float,
                        top_p: float = 1.0, seed: int = 0, child_mode: int = CHILD_WOR, request_ids=None,
                        positions=None, stream=None) -> dict:
    """``spec_verify_tree_dynamic``: as verify_tree with a tree per request,
    parent [B, N] int32 and n_nodes [B] int32 (device)."""
    lib = load()
    B, N, V = target.shape
    dt = _dtype_code(target)
    _check(target, "target")
    _check(draft, "draft", target.dtype, (B, N, V))
    _check(node_tokens, "node_tokens", torch.int32, (B, N))
    _check(parent, "parent", torch.int32, (B, N))
    _check(n_nodes, "n_nodes", torch.int32, (B,))
    _check(request_ids, "request_ids", torch.int64, (B,))
    _check(positions, "positions", torch.int64, (B,))
    if n_nodes is None:
        raise ValueError("n_nodes is required")
    dev = target.device
    W = int(max_depth) + 1
    out = dict(
        accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
        path_nodes=torch.empty(B, W, dtype=torch.int32, device=dev),
        out_tokens=torch.empty(B, W, dtype=torch.int32, device=dev),
        dev_error=torch.empty(1, dtype=torch.int32, device=dev),
    )
    need = workspace_size(SPEC_OP_TREE, B, N, V, dt)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    sp = SamplingParams(float(temperature), float(top_p), int(seed) & (2**64 - 1), int(child_mode))
    st = lib.spec_verify_tree_dynamic(_ptr(target), _ptr(draft), dt, _ptr(node_tokens), _ptr(parent), _ptr(n_nodes),
                                      B, N, V, int(max_depth), _ptr(request_ids), _ptr(positions), ctypes.byref(sp),
                                      _ptr(out["accepted_len"]), _ptr(out["path_nodes"]), _ptr(out["out_tokens"]),
                                      _ptr(out["dev_error"]), _ptr(ws), ws.numel(), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_verify_tree_dynamic", st)
    return out


def compact_accepted(hidden, accepted_len, out_tokens, path_nodes=None, stream=None) -> dict:
    """``spec_compact_accepted``: hidden [B, T, H] (2-byte elements),
    accepted_len [B], out_tokens [B, W], path_nodes [B, W] or None.
    Returns out_hidden [B*W, H] (rows past offsets[B] untouched),
    offsets [B+1], next_tokens [B*W], dev_error [1]."""
    lib = load()
    B, T, H = hidden.shape
    W = out_tokens.shape[1]
    if hidden.element_size() != 2:
        raise TypeError("hidden must have 2-byte elements (bf16)")
    _check(hidden, "hidden")
    _check(accepted_len, "accepted_len", torch.int32, (B,))
    _check(out_tokens, "out_tokens", torch.int32, (B, W))
    _check(path_nodes, "path_nodes", torch.int32, (B, W))
    dev = hidden.device
    out = dict(
        out_hidden=torch.empty(B * W, H, dtype=hidden.dtype, device=dev),
        offsets=torch.empty(B + 1, dtype=torch.int32, device=dev),
        next_tokens=torch.empty(B * W, dtype=torch.int32, device=dev),
        dev_error=torch.empty(1, dtype=torch.int32, device=dev),
    )
    st = lib.spec_compact_accepted(_ptr(hidden), B, T, H, _ptr(accepted_len), _ptr(path_nodes), _ptr(out_tokens), W,
                                   _ptr(out["out_hidden"]), _ptr(out["offsets"]), _ptr(out["next_tokens"]),
                                   _ptr(out["dev_error"]), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_compact_accepted", st)
    return out


def sample_rows(logits, temperature: float, top_p: float = 1.0, seed: int = 0, request_ids=None, positions=None,
                out=None, stream=None) -> dict:
    """``spec_sample_rows`` on torch tensors: one token per row of logits
    [R, V] (bf16 or fp32) from filter(softmax(row / temperature)).
    request_ids and positions [R] int64 or None.  Returns a dict of device
    tensors: out_tokens [R] int32, dev_error [1] int32."""
    lib = load()
    R, V = logits.shape
    dt = _dtype_code(logits)
    _check(logits, "logits")
    _check(request_ids, "request_ids", torch.int64, (R,))
    _check(positions, "positions", torch.int64, (R,))
    dev = logits.device
    if out is None:
        out = dict(out_tokens=torch.empty(R, dtype=torch.int32, device=dev),
                   dev_error=torch.empty(1, dtype=torch.int32, device=dev))
    sp = SamplingParams(float(temperature), float(top_p), int(seed) & (2**64 - 1), 0)
    st = lib.spec_sample_rows(_ptr(logits), dt, R, V, _ptr(request_ids), _ptr(positions), ctypes.byref(sp),
                              _ptr(out["out_tokens"]), _ptr(out.get("dev_error")), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_sample_rows", st)
    return out


def _rows(t, name):
    """(R, V, row stride) of a tensor [..., V] whose rows are contiguous and
    evenly spaced (a slice of a wider buffer counts)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) == 2 and stride[1] == 1 and stride[0] >= shape[1]:
        return shape[0], shape[1], stride[0]
    if len(shape) < 2:
        raise ValueError(f"{name} must have shape [..., V], got {tuple(shape)}")
    V = shape[-1]
    if V > 1 and stride[-1] != 1:
        raise ValueError(f"{name} must have contiguous rows")
    R, step = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n > 1:
            if step is None:
                step = s
            elif s != step * R:
                raise ValueError(f"{name} must have evenly spaced rows")
        R *= n
    if step is None:
        step = V
    if step < V:
        raise ValueError(f"{name} must have rows that do not overlap")
    return R, V, step


def _at(t, name, dtype, shape, device):
    """Pointer of a tensor that must be as described, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        _check(t, name, dtype, shape)
        raise ValueError(f"{name} must be on cuda:{device}")
    return t.data_ptr()


def _to(out, name, dtype, shape, device, stream):
    """Pointer of output `name`: the caller's tensor in out, checked, or a new
    one, allocated on the call's stream."""
    t = out.get(name)
    if t is None:
        with torch.cuda.stream(stream):  # no effect for None
            t = out[name] = torch.empty(shape, dtype=dtype, device=torch.device("cuda", device))
    elif t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        _check(t, name, dtype, shape)
        raise ValueError(f"{name} must be on cuda:{device}")
    return t.data_ptr()


def _handle(stream, device, *tensors):
    """The cudaStream_t of a call with a given stream, which is marked as a
    user of the tensors, so that their memory is not handed on before the
    call's work is done; or of the device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


_I32, _F32, _ONE = torch.int32, torch.float32, torch.Size((1,))


def token_logprobs(logits, tokens=None, temperature: float = 1.0, top_k: int = 0, out=None, stream=None) -> dict:
    """``spec_token_logprobs`` on torch tensors: log probability, rank and
    entropy for one token per row of logits [..., V] (bf16 or fp32; rows may
    be slices of a wider buffer), and the row's top_k alternatives.  tokens
    int32 of logits' leading shape, -1 skipping a row, or None (entropy and
    alternatives only).  With logits = target [B, k+1, V] and tokens =
    out_tokens of a verification, every emitted token is scored.  Returns a
    dict of device tensors in the leading shape: logprob, rank, entropy,
    top_ids and top_logprobs [..., top_k], dev_error [1]; tensors given in
    out are written in place."""
    lib = load()
    dt = _dtype_code(logits)
    R, V, step = _rows(logits, "logits")
    lead, device, K = logits.shape[:-1], logits.get_device(), int(top_k)
    wide = (*lead, max(K, 0))
    out = {} if out is None else out
    st = lib.spec_token_logprobs(
        logits.data_ptr(), dt, R, V, step, _at(tokens, "tokens", _I32, lead, device), temperature, K,
        _to(out, "logprob", _F32, lead, device, stream), _to(out, "rank", _I32, lead, device, stream),
        _to(out, "entropy", _F32, lead, device, stream), _to(out, "top_ids", _I32, wide, device, stream),
        _to(out, "top_logprobs", _F32, wide, device, stream), _to(out, "dev_error", _I32, _ONE, device, stream),
        _handle(stream, device, logits, tokens, *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_token_logprobs", st)
    return out


def _grad_rows(out, student, stream):
    """Pointer and row stride of the gradient: the caller's tensor (student's own counts), checked, or a new one."""
    grad = out.get("grad")
    if grad is None:
        with torch.cuda.stream(stream):
            grad = out["grad"] = torch.empty(student.shape, dtype=student.dtype, device=student.device)
    if grad.dtype is not student.dtype or grad.shape != student.shape or grad.get_device() != student.get_device():
        raise ValueError(f"grad must be {student.dtype} of shape {tuple(student.shape)} on {student.device}")
    return grad.data_ptr(), _rows(grad, "grad")[2]


def distill_topk(student, teacher_ids, teacher_logprobs, weights=None, temperature: float = 1.0,
                 tail: int = TAIL_BUCKET, with_grad: bool = True, out=None, stream=None) -> dict:
    """``spec_distill_topk`` on torch tensors: the distillation loss of every
    row of student logits [..., V] (bf16 or fp32) against a teacher's top
    log probabilities (teacher_ids int32 and teacher_logprobs float32 [...,
    K], as token_logprobs returns them; id -1 = absent), and, with with_grad,
    the gradient of sum(weights * loss) in the same pass.  weights float32 of
    the leading shape or None.  Returns a dict: loss and grad, row_stats
    [..., 8] (for distill_topk_backward), dev_error [1].  out["grad"] may be
    the student tensor itself.  The teacher's tensors are contiguous (a slice
    of token_logprobs' outputs along the drafts is not).  The loss is not part
    of an autograd graph, whether or not student requires gradients: hand grad
    to the model's backward pass, student.backward(grad)."""
    lib = load()
    dt = _dtype_code(student)
    R, V, step = _rows(student, "student")
    lead, device, K = student.shape[:-1], student.get_device(), teacher_ids.shape[-1]
    out = {} if out is None else out
    wide = (*lead, K)
    grad, grad_step = _grad_rows(out, student, stream) if with_grad else (None, V)
    st = lib.spec_distill_topk(
        student.data_ptr(), dt, R, V, step, _at(teacher_ids, "teacher_ids", _I32, wide, device),
        _at(teacher_logprobs, "teacher_logprobs", _F32, wide, device), K, _at(weights, "weights", _F32, lead, device),
        temperature, tail, _to(out, "loss", _F32, lead, device, stream),
        _to(out, "row_stats", _F32, (*lead, 8), device, stream), grad, grad_step,
        _to(out, "dev_error", _I32, _ONE, device, stream),
        _handle(stream, device, student, teacher_ids, teacher_logprobs, weights, *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_distill_topk", st)
    return out


def distill_topk_backward(student, teacher_ids, teacher_logprobs, row_stats, grad_loss=None,
                          temperature: float = 1.0, out=None, stream=None) -> dict:
    """``spec_distill_topk_backward``: the gradient of sum(grad_loss * loss)
    from the row_stats of a distill_topk call on the same student, teacher,
    temperature and tail.  grad_loss float32 of the leading shape or None (1).
    Returns a dict with grad (out["grad"] may be the student tensor)."""
    lib = load()
    dt = _dtype_code(student)
    R, V, step = _rows(student, "student")
    lead, device, K = student.shape[:-1], student.get_device(), teacher_ids.shape[-1]
    out = {} if out is None else out
    wide = (*lead, K)
    grad, grad_step = _grad_rows(out, student, stream)
    st = lib.spec_distill_topk_backward(
        student.data_ptr(), dt, R, V, step, _at(teacher_ids, "teacher_ids", _I32, wide, device),
        _at(teacher_logprobs, "teacher_logprobs", _F32, wide, device), K,
        _at(row_stats, "row_stats", _F32, (*lead, 8), device), _at(grad_loss, "grad_loss", _F32, lead, device),
        temperature, grad, grad_step,
        _handle(stream, device, student, teacher_ids, teacher_logprobs, row_stats, grad_loss, out["grad"]))
    if st != SPEC_OK:
        raise SpecError("spec_distill_topk_backward", st)
    return out


def advance_blocks(seq_lens, new_tokens, block_table, held, free_blocks, free_count, page_size: int,
                   max_tokens: int, accepted_len=None, out=None, stream=None) -> dict:
    """``spec_advance_blocks`` on torch tensors: seq_lens, new_tokens, held
    and accepted_len [B] int32 (accepted_len as verify_linear returns it, or
    None), block_table [B, max_blocks] int32 (new entries written in place),
    free_blocks [F] int32 with free_count [1] int32 entries in use.  Returns a
    dict: seq_lens, held, free_count (the state for the next call),
    cu_tokens [B+1], slots [max_tokens] int64, positions [max_tokens] int32,
    dev_error [1]."""
    lib = load()
    if block_table.dim() != 2:
        raise ValueError(f"block_table must have shape [B, max_blocks], got {tuple(block_table.shape)}")
    if block_table.dtype != torch.int32:
        raise TypeError(f"block_table must be {torch.int32}, got {block_table.dtype}")
    B, M, step = _rows(block_table, "block_table")
    device, T, F = block_table.get_device(), int(max_tokens), free_blocks.shape[0]
    out = {} if out is None else out
    each, room = (B,), (max(T, 0),)
    st = lib.spec_advance_blocks(
        _at(seq_lens, "seq_lens", _I32, each, device), _at(accepted_len, "accepted_len", _I32, each, device),
        _at(new_tokens, "new_tokens", _I32, each, device), B, page_size, block_table.data_ptr(), M, step,
        _at(held, "held", _I32, each, device), _at(free_blocks, "free_blocks", _I32, (F,), device), F,
        _at(free_count, "free_count", _I32, _ONE, device), _to(out, "seq_lens", _I32, each, device, stream),
        _to(out, "held", _I32, each, device, stream), _to(out, "free_count", _I32, _ONE, device, stream),
        _to(out, "cu_tokens", _I32, (B + 1,), device, stream), _to(out, "slots", torch.int64, room, device, stream),
        _to(out, "positions", _I32, room, device, stream), T, _to(out, "dev_error", _I32, _ONE, device, stream),
        _handle(stream, device, seq_lens, accepted_len, new_tokens, block_table, held, free_blocks, free_count,
                *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_advance_blocks", st)
    return out


def _half_code(t, name) -> int:
    if t.dtype is torch.bfloat16:
        return SPEC_BF16
    if t.dtype is torch.float16:
        return SPEC_F16
    raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def _cache(t, name, device=None):
    """Layout of a cache [blocks, page_size, heads, dim] whose dim is contiguous, as the arguments of a CacheLayout; the
    other dimensions may lie in any order and be parts of a wider buffer, but must not overlap."""
    shape, stride, on = t.shape, t.stride(), t.get_device()
    if on < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if len(shape) != 4 or 0 in shape:
        raise ValueError(f"{name} must have shape [blocks, page_size, heads, dim], got {tuple(shape)}")
    if device is not None and on != device:
        raise ValueError(f"{name} must be on cuda:{device}")
    blocks, page, heads, dim = shape
    if t.is_contiguous():
        return (blocks, page, heads, dim, page * heads * dim, heads * dim, dim)
    if dim > 1 and stride[3] != 1:
        raise ValueError(f"{name} must have contiguous heads")
    steps = [s if n > 1 else 0 for s, n in zip(stride, (blocks, page, heads))]
    room = dim
    for s, n in sorted(zip(steps, (blocks, page, heads))):
        if n > 1:
            if s < room:
                raise ValueError(f"{name} must have entries that do not overlap")
            room += s * (n - 1)
    return (blocks, page, heads, dim, *steps)


def _caches(k_cache, v_cache, device):
    """The one layout of a key and a value cache, as _cache's."""
    layout = _cache(k_cache, "k_cache", device)
    if v_cache.dtype is not k_cache.dtype or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one dtype and shape")
    if v_cache.stride() != k_cache.stride() and _cache(v_cache, "v_cache", device) != layout:
        raise ValueError("k_cache and v_cache must have the same strides")
    if v_cache.get_device() != device:
        raise ValueError(f"v_cache must be on cuda:{device}")
    return layout


def _heads(t, name, dtype, shape, device):
    """(pointer, strides but the last) of a tensor [..., heads, dim] whose heads are contiguous."""
    stride = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or (stride[-1] != 1 and shape[-1] > 1):
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}" if t.is_cuda else f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} must have contiguous heads")
    if 1 in shape:  # a stride that is not used may be any number
        stride = [s if n > 1 else 0 for s, n in zip(stride, shape)]
    return t.data_ptr(), stride[:-1]


def _table(block_table, B, device):
    """(pointer, blocks of a row, row stride) of a block table [B, max_blocks]."""
    if block_table.dtype is not _I32:
        raise TypeError(f"block_table must be {_I32}, got {block_table.dtype}")
    if block_table.dim() != 2 or block_table.shape[0] != B or block_table.get_device() != device:
        raise ValueError(f"block_table must have shape [{B}, max_blocks] on cuda:{device}")
    _, M, step = _rows(block_table, "block_table")
    return block_table.data_ptr(), M, step


def _tree(parent, B, N, device):
    """(pointer, row stride) of a parent array [N] or [B, N], or of none."""
    if parent is None:
        return None, 0
    if parent.dim() == 1:
        return _at(parent, "parent", _I32, torch.Size((N,)), device), 0
    return _at(parent, "parent", _I32, torch.Size((B, N)), device), N


def append_kv(q, k, v, positions, slots, k_cache, v_cache, inv_freq=None, q_norm=None, k_norm=None, eps: float = 1e-6,
              interleaved: bool = False, out=None, stream=None) -> dict:
    """``spec_append_kv`` on torch tensors: q [T, q_heads, dim] (or None), k and v [T, heads, dim] (bf16 or fp16;
    slices of one projection count), positions [T] int32, slots [T] int64 as advance_blocks returns them (negative:
    nothing is stored), caches [blocks, page_size, heads, dim] of one layout, written in place.  inv_freq [rot_dim / 2]
    float32 or None (no turn); q_norm and k_norm [dim] or None.  Returns a dict: q (turned; out["q"] may be q itself),
    dev_error [1]."""
    lib = load()
    dt, dtype, shape, device = _half_code(k, "k"), k.dtype, k.shape, k.get_device()
    if len(shape) != 3 or (q is not None and q.dim() != 3):
        raise ValueError("q, k and v must have shape [T, heads, dim]")
    if device < 0:
        raise ValueError("k must be a CUDA tensor")
    T, H, D = shape
    layout = _caches(k_cache, v_cache, device)
    if k_cache.dtype is not dtype or layout[2:4] != (H, D):
        raise ValueError(f"caches must be {dtype} of {H} heads of {D}")
    out = {} if out is None else out
    q_heads = 0 if q is None else q.shape[1]
    wide = torch.Size((T, q_heads, D))
    q_ptr, (q_token, q_head) = (None, (0, 0)) if q is None else _heads(q, "q", dtype, wide, device)
    k_ptr, (k_token, k_head) = _heads(k, "k", dtype, shape, device)
    v_ptr, (v_token, v_head) = _heads(v, "v", dtype, shape, device)
    one, each = torch.Size((D,)), torch.Size((T,))
    rot = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    if inv_freq is not None and positions is None:
        raise ValueError("positions are required with inv_freq")
    st = lib.spec_append_kv(
        q_ptr, k_ptr, v_ptr, dt, T, q_heads, q_token, q_head, k_token, k_head, v_token, v_head,
        _at(q_norm, "q_norm", dtype, one, device), _at(k_norm, "k_norm", dtype, one, device), eps,
        _at(positions, "positions", _I32, each, device),
        None if inv_freq is None else _at(inv_freq, "inv_freq", _F32, torch.Size((rot // 2,)), device), rot,
        bool(interleaved), _at(slots, "slots", torch.int64, each, device),
        None if q is None else _to(out, "q", dtype, wide, device, stream), k_cache.data_ptr(), v_cache.data_ptr(),
        ctypes.byref(CacheLayout(*layout)), _to(out, "dev_error", _I32, _ONE, device, stream),
        _handle(stream, device, q, k, v, positions, slots, k_cache, v_cache, inv_freq, q_norm, k_norm, *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_append_kv", st)
    return out


def tree_attention(q, k_cache, v_cache, block_table, seq_lens, parent=None, n_nodes=None, scale=None, out=None,
                   stream=None) -> dict:
    """``spec_tree_attention`` on torch tensors: q [B, N, q_heads, dim] (bf16 or fp16), caches [blocks, page_size,
    heads, dim] of one layout, block_table [B, max_blocks] and seq_lens [B] int32 (advance_blocks' state; the nodes'
    entries lie behind seq_lens), parent None (a chain), [N] or [B, N] int32, n_nodes [B] int32 or None, scale
    (default 1 / sqrt(dim)).  Returns a dict: out [B, N, q_heads, dim] (a new tensor has zeros behind a request's
    nodes; a given one keeps what it has there), dev_error [1], and workspace, used again when the dict is given as
    `out` to later calls on the same stream."""
    lib = load()
    dt = _half_code(q, "q")
    if q.dim() != 4 or q.numel() == 0:
        raise ValueError(f"q must have shape [B, N, q_heads, dim], got {tuple(q.shape)}")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    device, shape, dtype = q.get_device(), q.shape, q.dtype
    B, N, H, D = shape
    layout = _caches(k_cache, v_cache, device)
    if k_cache.dtype is not dtype or layout[3] != D or H % layout[2]:
        raise ValueError(f"caches must be {dtype} of heads that divide {H}, of {D}")
    q_ptr, (q_request, q_node, q_head) = _heads(q, "q", dtype, shape, device)
    table, M, step = _table(block_table, B, device)
    tree, tree_step = _tree(parent, B, N, device)
    out = {} if out is None else out
    each = torch.Size((B,))
    if "out" not in out and n_nodes is not None:
        with torch.cuda.stream(stream):  # no effect for None
            out["out"] = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    need = lib.spec_tree_attention_workspace(B, N, H, layout[2], D)
    space = out.get("workspace")
    if space is None or space.numel() < need or space.get_device() != device:
        with torch.cuda.stream(stream):
            space = out["workspace"] = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = lib.spec_tree_attention(
        q_ptr, dt, B, N, H, q_request, q_node, q_head, k_cache.data_ptr(), v_cache.data_ptr(),
        ctypes.byref(CacheLayout(*layout)), table, M, step, _at(seq_lens, "seq_lens", _I32, each, device), tree, tree_step,
        _at(n_nodes, "n_nodes", _I32, each, device), D ** -0.5 if scale is None else scale,
        _to(out, "out", dtype, shape, device, stream), _to(out, "dev_error", _I32, _ONE, device, stream),
        space.data_ptr(), space.numel(),
        _handle(stream, device, q, k_cache, v_cache, block_table, seq_lens, parent, n_nodes, *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_tree_attention", st)
    return out


def adjust_logits(logits, history=None, history_lens=None, prompt_lens=None, drafted=None, parent=None, n_nodes=None,
                  repetition=None, frequency=None, presence=None, bias_ids=None, bias_values=None, allowed=None,
                  out=None, stream=None) -> dict:
    """``spec_adjust_logits`` on torch tensors: logits [B, R, V] (bf16 or fp32; rows may be slices of a wider buffer);
    history [B, L] int32 with history_lens and prompt_lens [B] int32; drafted int32 [B, R - 1] (draft_tokens of a
    linear verification) or [B, R] (node_tokens of a tree's), parent None (a chain), [R] or [B, R], n_nodes [B] int32;
    repetition, frequency, presence [B] float32; bias_ids int32 and bias_values float32 [B, K]; allowed [B, R, ceil(V /
    32)] int32, a bit a token.  Returns a dict: logits (out["logits"] may be the tensor itself; by default a new one,
    in which rows behind a request's nodes are zero), dev_error [1]."""
    lib = load()
    dt = _dtype_code(logits)
    if logits.dim() != 3:
        raise ValueError(f"logits must have shape [B, R, V], got {tuple(logits.shape)}")
    _, V, step = _rows(logits, "logits")
    B, R, device = logits.shape[0], logits.shape[1], logits.get_device()
    out = {} if out is None else out
    to = out.get("logits")
    if to is None:
        make = torch.empty if n_nodes is None else torch.zeros
        with torch.cuda.stream(stream):
            to = out["logits"] = make(logits.shape, dtype=logits.dtype, device=logits.device)
    if to.dtype is not logits.dtype or to.shape != logits.shape or to.get_device() != device:
        raise ValueError(f"out logits must be {logits.dtype} of shape {tuple(logits.shape)} on {logits.device}")
    each = torch.Size((B,))
    a = Adjustments()
    if history is not None:
        if history.dtype is not _I32 or history.dim() != 2 or history.shape[0] != B or history.get_device() != device:
            raise ValueError(f"history must be {_I32} of shape [{B}, L] on cuda:{device}")
        if history_lens is None:
            raise ValueError("history_lens is required with history")
        a.history_capacity = history.shape[1]
        a.history_stride = _rows(history, "history")[2] if history.numel() else history.shape[1]
        a.history = history.data_ptr() or None
        a.history_lens = _at(history_lens, "history_lens", _I32, each, device)
        a.prompt_lens = _at(prompt_lens, "prompt_lens", _I32, each, device)
    if drafted is not None and R > 1:
        whole = drafted.dim() == 2 and drafted.shape[1] == R
        a.drafted = _at(drafted, "drafted", _I32, torch.Size((B, R if whole else R - 1)), device)
        a.drafted_stride = R if whole else R - 1
        if whole and a.drafted:
            a.drafted += 4  # node 0's token is the last of the history
        a.parent, a.parent_stride = _tree(parent, B, R, device)
    a.n_nodes = _at(n_nodes, "n_nodes", _I32, each, device)
    a.repetition = _at(repetition, "repetition", _F32, each, device)
    a.frequency = _at(frequency, "frequency", _F32, each, device)
    a.presence = _at(presence, "presence", _F32, each, device)
    if bias_ids is not None:
        wide = torch.Size((B, bias_ids.shape[-1]))
        a.bias_ids, a.bias_count = _at(bias_ids, "bias_ids", _I32, wide, device), wide[1]
        if bias_values is None:
            raise ValueError("bias_values are required with bias_ids")
        a.bias_values = _at(bias_values, "bias_values", _F32, wide, device)
    if allowed is not None:
        if allowed.dtype is not _I32 or allowed.shape != (B, R, (V + 31) // 32) or allowed.get_device() != device:
            raise ValueError(f"allowed must be {_I32} of shape {(B, R, (V + 31) // 32)} on cuda:{device}")
        a.allowed, a.allowed_stride = allowed.data_ptr(), _rows(allowed, "allowed")[2]
    st = lib.spec_adjust_logits(
        logits.data_ptr(), dt, B, R, V, step, ctypes.byref(a), to.data_ptr(), _rows(to, "out logits")[2],
        _to(out, "dev_error", _I32, _ONE, device, stream),
        _handle(stream, device, logits, history, history_lens, prompt_lens, drafted, parent, n_nodes, repetition,
                frequency, presence, bias_ids, bias_values, allowed, *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_adjust_logits", st)
    return out


_ALIKE = (operator.attrgetter("dtype"), torch.Tensor.size, torch.Tensor.stride, torch.Tensor.get_device)


def keep_path(planes, path_nodes, accepted_len, seq_lens, block_table, out=None, stream=None) -> dict:
    """``spec_keep_path`` on torch tensors: planes, a sequence of caches [blocks, page_size, heads, dim] of one layout
    and dtype (keys and values of all layers), changed in place; path_nodes [B, W] and accepted_len [B] as verify_tree
    returns them, seq_lens [B] and block_table [B, max_blocks] as the attention had them.  Returns a dict: dev_error
    [1]."""
    lib = load()
    device = path_nodes.get_device()
    if path_nodes.dim() != 2:
        raise ValueError(f"path_nodes must have shape [B, W], got {tuple(path_nodes.shape)}")
    if not path_nodes.is_cuda:
        raise ValueError("path_nodes must be a CUDA tensor")
    B, W = path_nodes.shape
    planes = tuple(planes)
    if not planes:
        raise ValueError("planes must name at least one cache")
    head = planes[0]
    layout = CacheLayout(*_cache(head, "planes[0]", device))
    for of in _ALIKE:  # a pass for each: no Python of its own for a plane, of which there are two a layer
        each = list(map(of, planes))
        if each.count(each[0]) != len(each):
            raise ValueError("planes must have one dtype, shape, device and set of strides")
    pointers = array.array("Q", map(torch.Tensor.data_ptr, planes))
    if len(set(pointers)) != len(planes):
        raise ValueError("planes must be distinct")
    each = torch.Size((B,))
    table, M, step = _table(block_table, B, device)
    out = {} if out is None else out
    st = lib.spec_keep_path(
        pointers.buffer_info()[0], len(planes), head.element_size(),
        ctypes.byref(layout), B, W, _at(path_nodes, "path_nodes", _I32, path_nodes.shape, device),
        _at(accepted_len, "accepted_len", _I32, each, device), _at(seq_lens, "seq_lens", _I32, each, device), table, M,
        step, _to(out, "dev_error", _I32, _ONE, device, stream),
        _handle(stream, device, *(planes if stream is not None else ()), path_nodes, accepted_len, seq_lens, block_table,
                *out.values()))
    if st != SPEC_OK:
        raise SpecError("spec_keep_path", st)
    return out
