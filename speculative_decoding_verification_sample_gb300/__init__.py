"""GB300 speculative-decoding verification (sm_103a).

Thin ctypes binding of the in-tree C-ABI library `libspecverify.so`: argument
marshalling only. Every step of the verification runs in the library's CUDA
kernels; PyTorch supplies device memory and the current stream. There is no
CPU fallback: without the built library (or without a GPU) these calls raise.

The entry points carry the C names:
  spec_verify_sample(...)   accept/reject with temperature softmax, residual or bonus draw
  spec_verify_greedy(...)   argmax-match verification
  spec_verify_tree_greedy(...)  argmax-match verification of a draft tree
  kv_commit_rollback(...)   commit accepted provisional KV slots, free provisional blocks
  kv_q8_append(...)         tokens into the 8-bit paged cache (e4m3, a scale per block and head)
  kv_q8_attention(...)      attention of the provisional tokens over that cache
  kv_reserve, kv_fork, kv_free   blocks for new tokens, shared prefixes, release
  qk_norm_rope(...)         norms of queries and keys for each head, rotary positions
  kv_q8_norm_rope_append(...)  the same with keys and values into the 8-bit cache
  kv_prefix_plan, kv_q8_prefix_attention   attention of rows that share a prefix's blocks
See include/specverify.h for layouts, ownership and error behaviour.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SPEC_OK, SPEC_EINVAL, SPEC_ECUDA, SPEC_ENOTSUP = 0, -1, -2, -3
SPEC_BF16, SPEC_F32 = 0, 1
SPEC_DERR_TOKEN, SPEC_DERR_LOGITS = 1, 2
SPEC_DERR_BAD_ACCEPT, SPEC_DERR_BAD_LENGTH, SPEC_DERR_NO_SPACE, SPEC_DERR_BAD_BLOCK = 4, 8, 16, 32
SPEC_DERR_TIMEOUT = 64
SPEC_DERR_BAD_SLOT = 128
SPEC_DERR_VALUE = 256
SPEC_ROW_ACCEPT_REFINED, SPEC_ROW_SAMPLE_REFINED = 1, 2
SPEC_ROW_UNCERTIFIED, SPEC_ROW_ZERO_RESIDUAL = 4, 8

EXPORTED = ("spec_verify_sample", "spec_verify_greedy", "spec_verify_workspace_bytes",
            "kv_commit_rollback", "spec_selftest_ex2", "spec_status_string", "spec_version",
            "spec_verify_greedy_noalloc", "spec_verify_greedy_noalloc_max_bytes",
            "kv_commit_inplace", "kv_evict_provisional", "spec_verify_tree_greedy",
            "spec_filter_thresholds", "kv_q8_append", "kv_q8_attention",
            "kv_q8_attention_workspace_bytes", "kv_reserve", "kv_fork", "kv_free",
            "qk_norm_rope", "kv_q8_norm_rope_append", "kv_prefix_plan", "kv_prefix_plan_bytes",
            "kv_q8_prefix_attention", "kv_q8_prefix_attention_workspace_bytes")

_lib = None


class SpecError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, fn: str, status: int):
        msg = lib().spec_status_string(status).decode() if _lib else str(status)
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libspecverify.so (built by `build.build()`); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run "
                               "speculative_decoding_verification_sample_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        Z = ctypes.c_size_t
        L.spec_verify_sample.argtypes = [P, P, P, P, F, I, I, I, P, P, P, I, P, P, P, P, P, Z, P,
                                         P, P]
        L.spec_verify_sample.restype = I
        L.spec_verify_greedy.argtypes = [P, P, I, I, I, P, P, P, I, P, P, Z, P]
        L.spec_verify_greedy.restype = I
        L.spec_verify_tree_greedy.argtypes = [P, P, P, I, I, I, P, P, P, P, I, P, P, Z]
        L.spec_verify_tree_greedy.restype = I
        L.spec_filter_thresholds.argtypes = [P, I, I, I, F, I, F, P, P, P]
        L.spec_filter_thresholds.restype = I
        L.spec_verify_greedy_noalloc.argtypes = [P, P, I, I, I, P, P, P, I, P]
        L.spec_verify_greedy_noalloc.restype = I
        L.kv_commit_inplace.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P]
        L.kv_commit_inplace.restype = I
        L.kv_evict_provisional.argtypes = [P, P, I, I, I, I, I, P, P, P, P]
        L.kv_evict_provisional.restype = I
        L.spec_verify_greedy_noalloc_max_bytes.argtypes = []
        L.spec_verify_greedy_noalloc_max_bytes.restype = Z
        L.spec_verify_workspace_bytes.argtypes = [I, I, I, I]
        L.spec_verify_workspace_bytes.restype = Z
        L.kv_commit_rollback.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, P, P, P, P,
                                         P]
        L.kv_commit_rollback.restype = I
        L.kv_q8_append.argtypes = [P, P, I, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, P]
        L.kv_q8_append.restype = I
        L.kv_q8_attention.argtypes = [P, I, P, P, P, P, P, P, P, F, I, I, I, I, I, I, I, I, I, I,
                                      I, I, P, Z, P, P]
        L.kv_q8_attention.restype = I
        L.kv_q8_attention_workspace_bytes.argtypes = [I, I, I, I]
        L.kv_q8_attention_workspace_bytes.restype = Z
        L.kv_reserve.argtypes = [P, P, P, I, I, I, I, I, P, P, P, P]
        L.kv_reserve.restype = I
        L.kv_fork.argtypes = [P, P, P, P, P, I, P, I, I, P, I, I, I, I, P, P, P, P]
        L.kv_fork.restype = I
        L.kv_free.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P]
        L.kv_free.restype = I
        S = ctypes.c_int64
        L.qk_norm_rope.argtypes = [P, S, P, S, I, P, S, P, S, P, P, F, P, I, I, F, P, P, P, I, I,
                                   I, I, I, P, P]
        L.qk_norm_rope.restype = I
        L.kv_q8_norm_rope_append.argtypes = [P, S, P, S, P, S, I, P, S, P, P, F, P, I, I, F, P, P,
                                             P, P, P, P, I, I, I, I, I, I, I, I, I, I, P, P]
        L.kv_q8_norm_rope_append.restype = I
        L.kv_prefix_plan.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, P, Z, P, P]
        L.kv_prefix_plan.restype = I
        L.kv_prefix_plan_bytes.argtypes = [I, I, I]
        L.kv_prefix_plan_bytes.restype = Z
        L.kv_q8_prefix_attention.argtypes = [P, I, P, P, P, P, P, P, P, Z, P, F, I, I, I, I, I, I,
                                             I, I, I, I, P, Z, P, P]
        L.kv_q8_prefix_attention.restype = I
        L.kv_q8_prefix_attention_workspace_bytes.argtypes = [I, I, I, I, I]
        L.kv_q8_prefix_attention_workspace_bytes.restype = Z
        L.spec_selftest_ex2.argtypes = [F, F, P, P]
        L.spec_selftest_ex2.restype = I
        L.spec_status_string.argtypes = [I]
        L.spec_status_string.restype = ctypes.c_char_p
        L.spec_version.argtypes = []
        L.spec_version.restype = I
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check(t, name, ndim=None, dtype=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


_workspaces = {}


def spec_verify_workspace_bytes(B: int, K: int, V: int, dtype_code: int) -> int:
    """Device workspace bytes the verify calls need for (B, K, V, dtype)."""
    return int(lib().spec_verify_workspace_bytes(B, K, V, dtype_code))


def workspace_for(B: int, K: int, V: int, dtype_code: int, device):
    """A cached device workspace (uint8 tensor) large enough for (B, K, V, dtype)
    on `device`. Calls sharing it must be ordered on the device."""
    import torch
    need = spec_verify_workspace_bytes(B, K, V, dtype_code)
    if need == 0:
        raise SpecError("spec_verify_workspace_bytes", SPEC_EINVAL)
    dev = torch.device(device)
    key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device())
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def _ws_args(ws, B, K, V, code, device):
    if ws is None:
        if spec_verify_workspace_bytes(B, K, V, code) == 0:
            # unsupported shape: the library call itself reports why
            return ctypes.c_void_p(0), ctypes.c_size_t(0)
        ws = workspace_for(B, K, V, code, device)
    off = (-ws.data_ptr()) % 256
    return ctypes.c_void_p(ws.data_ptr() + off), ctypes.c_size_t(ws.numel() - off)


def _counters(t, K):
    """Pointer of an optional [2K+2] 64-bit integer device tensor of counters."""
    if t is None:
        return None
    import torch
    if not t.is_cuda or t.dtype not in (torch.int64, torch.uint64) or t.numel() != 2 * K + 2 \
            or not t.is_contiguous():
        raise ValueError(f"accept_counters must be a contiguous 64-bit integer CUDA tensor "
                         f"of {2 * K + 2} elements")
    return _ptr(t)


def _thr(t, B, n):
    """Pointer of an optional [B, n] float32 CUDA tensor of row thresholds."""
    if t is None:
        return None
    import torch
    if not t.is_cuda or t.dtype != torch.float32 or t.numel() != B * n or not t.is_contiguous():
        raise ValueError(f"thresholds must be a contiguous float32 CUDA tensor of {B * n} values")
    return _ptr(t)


def spec_verify_sample(target_logits, draft_logits, draft_tokens, uniforms, temperature: float,
                       out_tokens, out_num_accepted, *, stream=None, err_flag=None,
                       row_info=None, q_at_d=None, p_at_d=None, workspace=None,
                       accept_counters=None, target_threshold=None,
                       draft_threshold=None) -> None:
    """Sampling-mode verification; shapes [B,K+1,V], [B,K,V], [B,K], [B,K+1] -> [B,K+1], [B].
    accept_counters: optional int64/uint64 [2K+2] device tensor, accumulated (see the header).
    target_threshold [B,K+1] / draft_threshold [B,K]: optional float32 logit thresholds
    (spec_filter_thresholds) for top-k / top-p filtering."""
    import torch
    _check(target_logits, "target_logits", 3)
    B, K1, V = target_logits.shape
    K = K1 - 1
    if float(temperature) != 0.0:
        _check(draft_logits, "draft_logits", 3, target_logits.dtype)
        _check(uniforms, "uniforms", 2, torch.float32)
    _check(draft_tokens, "draft_tokens", 2, torch.int32)
    _check(out_tokens, "out_tokens", 2, torch.int32)
    _check(out_num_accepted, "out_num_accepted", 1, torch.int32)
    code = _dtype_code(target_logits)
    wsp, wsn = _ws_args(workspace, B, K, V, code, target_logits.device)
    st = lib().spec_verify_sample(
        _ptr(target_logits), _ptr(draft_logits), _ptr(draft_tokens), _ptr(uniforms),
        ctypes.c_float(temperature), B, K, V, _ptr(out_tokens), _ptr(out_num_accepted),
        _stream(stream), code, _ptr(err_flag), _ptr(row_info),
        _ptr(q_at_d), _ptr(p_at_d), wsp, wsn, _counters(accept_counters, K),
        _thr(target_threshold, B, K + 1), _thr(draft_threshold, B, K))
    if st != SPEC_OK:
        raise SpecError("spec_verify_sample", st)


def spec_verify_greedy(target_logits, draft_tokens, out_tokens, out_num_accepted, *,
                       stream=None, err_flag=None, workspace=None, accept_counters=None) -> None:
    """Greedy verification; target [B,K+1,V], tokens [B,K] -> [B,K+1], [B]."""
    import torch
    _check(target_logits, "target_logits", 3)
    _check(draft_tokens, "draft_tokens", 2, torch.int32)
    _check(out_tokens, "out_tokens", 2, torch.int32)
    _check(out_num_accepted, "out_num_accepted", 1, torch.int32)
    B, K1, V = target_logits.shape
    code = _dtype_code(target_logits)
    wsp, wsn = _ws_args(workspace, B, K1 - 1, V, code, target_logits.device)
    st = lib().spec_verify_greedy(_ptr(target_logits), _ptr(draft_tokens), B, K1 - 1, V,
                                  _ptr(out_tokens), _ptr(out_num_accepted), _stream(stream),
                                  code, _ptr(err_flag), wsp, wsn,
                                  _counters(accept_counters, K1 - 1))
    if st != SPEC_OK:
        raise SpecError("spec_verify_greedy", st)


def spec_verify_tree_greedy(target_logits, tree_parents, tree_tokens, out_tokens,
                            out_num_accepted, *, out_slots=None, stream=None, err_flag=None,
                            workspace=None) -> None:
    """Greedy verification of a draft tree; target [B,N+1,V], parents and tokens [B,N]
    -> tokens [B,N+1], accepted [B], optional KV slots [B,N+1]."""
    import torch
    _check(target_logits, "target_logits", 3)
    _check(tree_parents, "tree_parents", 2, torch.int32)
    _check(tree_tokens, "tree_tokens", 2, torch.int32)
    _check(out_tokens, "out_tokens", 2, torch.int32)
    _check(out_num_accepted, "out_num_accepted", 1, torch.int32)
    if out_slots is not None:
        _check(out_slots, "out_slots", 2, torch.int32)
    B, N1, V = target_logits.shape
    code = _dtype_code(target_logits)
    wsp, wsn = _ws_args(workspace, B, N1 - 1, V, code, target_logits.device)
    st = lib().spec_verify_tree_greedy(_ptr(target_logits), _ptr(tree_parents),
                                       _ptr(tree_tokens), B, N1 - 1, V, _ptr(out_tokens),
                                       _ptr(out_num_accepted), _ptr(out_slots), _stream(stream),
                                       code, _ptr(err_flag), wsp, wsn)
    if st != SPEC_OK:
        raise SpecError("spec_verify_tree_greedy", st)


def spec_filter_thresholds(logits, temperature: float, top_k: int, top_p: float, out_threshold,
                           *, stream=None, err_flag=None) -> None:
    """Top-k / top-p logit threshold of every row of logits [..., V] -> out_threshold [...]
    (float32; keep tokens with logit >= threshold)."""
    import torch
    _check(logits, "logits")
    _check(out_threshold, "out_threshold", None, torch.float32)
    V = logits.shape[-1]
    R = logits.numel() // V
    if out_threshold.numel() != R:
        raise ValueError(f"out_threshold must hold {R} values")
    st = lib().spec_filter_thresholds(_ptr(logits), R, V, _dtype_code(logits),
                                      ctypes.c_float(temperature), int(top_k),
                                      ctypes.c_float(top_p), _ptr(out_threshold),
                                      _stream(stream), _ptr(err_flag))
    if st != SPEC_OK:
        raise SpecError("spec_filter_thresholds", st)


def spec_verify_greedy_noalloc(target_logits, draft_tokens, out_tokens, out_num_accepted, *,
                               stream=None, err_flag=None) -> None:
    """Greedy verification on the library's built-in device scratch (no workspace
    argument, nothing allocated). Calls on one device must not overlap."""
    import torch
    _check(target_logits, "target_logits", 3)
    _check(draft_tokens, "draft_tokens", 2, torch.int32)
    _check(out_tokens, "out_tokens", 2, torch.int32)
    _check(out_num_accepted, "out_num_accepted", 1, torch.int32)
    B, K1, V = target_logits.shape
    st = lib().spec_verify_greedy_noalloc(_ptr(target_logits), _ptr(draft_tokens), B, K1 - 1, V,
                                          _ptr(out_tokens), _ptr(out_num_accepted),
                                          _stream(stream), _dtype_code(target_logits),
                                          _ptr(err_flag))
    if st != SPEC_OK:
        raise SpecError("spec_verify_greedy_noalloc", st)


def spec_verify_greedy_noalloc_max_bytes() -> int:
    """Size of the built-in scratch used by spec_verify_greedy_noalloc."""
    return int(lib().spec_verify_greedy_noalloc_max_bytes())


def kv_commit_inplace(block_table, seq_lens, num_accepted, free_stack, free_top, status, *,
                      K: int, block_size: int, num_blocks: int, stream=None) -> None:
    """In-place KV commit: truncate each row to L + n + 1 and free the blocks past it."""
    import torch
    _check(block_table, "block_table", 2, torch.int32)
    for t, n in ((seq_lens, "seq_lens"), (num_accepted, "num_accepted"),
                 (free_stack, "free_stack"), (free_top, "free_top"), (status, "status")):
        _check(t, n, 1, torch.int32)
    B, MB = block_table.shape
    st = lib().kv_commit_inplace(_ptr(block_table), _ptr(seq_lens), _ptr(num_accepted),
                                 num_blocks, block_size, B, K, MB, _ptr(free_stack),
                                 _ptr(free_top), _ptr(status), _stream(stream))
    if st != SPEC_OK:
        raise SpecError("kv_commit_inplace", st)


def kv_evict_provisional(block_table, seq_lens, free_stack, free_top, status, *, K: int,
                         block_size: int, num_blocks: int, stream=None) -> None:
    """In-place layout: discard every row's K+1 provisional slots (preemption)."""
    import torch
    _check(block_table, "block_table", 2, torch.int32)
    for t, n in ((seq_lens, "seq_lens"), (free_stack, "free_stack"), (free_top, "free_top"),
                 (status, "status")):
        _check(t, n, 1, torch.int32)
    B, MB = block_table.shape
    st = lib().kv_evict_provisional(_ptr(block_table), _ptr(seq_lens), num_blocks, block_size, B,
                                    K, MB, _ptr(free_stack), _ptr(free_top), _ptr(status),
                                    _stream(stream))
    if st != SPEC_OK:
        raise SpecError("kv_evict_provisional", st)


def kv_commit_rollback(block_table, seq_lens, num_accepted, prov_blocks, kv_pool, free_stack,
                       free_top, status, *, K: int, block_size: int, stream=None,
                       slot_map=None) -> None:
    """Commit the accepted provisional slots. kv_pool: [num_blocks, layers, 2, block_size,
    heads, head_dim] (any element type); tables int32 as in include/specverify.h.
    slot_map: optional [B, K+1] int32 (a tree draft's kept slots)."""
    import torch
    if slot_map is not None:
        _check(slot_map, "slot_map", 2, torch.int32)
    for t, n in ((block_table, "block_table"), (prov_blocks, "prov_blocks")):
        _check(t, n, 2, torch.int32)
    for t, n in ((seq_lens, "seq_lens"), (num_accepted, "num_accepted"),
                 (free_stack, "free_stack"), (free_top, "free_top"), (status, "status")):
        _check(t, n, 1, torch.int32)
    _check(kv_pool, "kv_pool", 6)
    NB, NL, two, bs, H, D = kv_pool.shape
    if two != 2 or bs != block_size:
        raise ValueError("kv_pool must be [num_blocks, layers, 2, block_size, heads, head_dim]")
    B, MB = block_table.shape
    P = prov_blocks.shape[1]
    st = lib().kv_commit_rollback(
        _ptr(block_table), _ptr(seq_lens), _ptr(num_accepted), _ptr(prov_blocks), _ptr(kv_pool),
        NB, NL, H, D, kv_pool.element_size(), block_size, B, K, MB, P, _ptr(free_stack),
        _ptr(free_top), _ptr(status), _stream(stream), _ptr(slot_map))
    if st != SPEC_OK:
        raise SpecError("kv_commit_rollback", st)


# The calls below take a few microseconds on the device, so their arguments are checked with
# few Python steps: _arg covers the usual case and leaves the message to _check, and the torch
# names are looked up once.
_int32 = _float32 = _bfloat16 = _e4m3 = _uint8 = _raw_current = None
_capturing = _current_device = None


def _ready() -> ctypes.CDLL:
    """The library, with the torch names of this section set. The calls test _int32: it is set
    last, so that another thread's call meanwhile comes here too and finds nothing half set."""
    global _int32, _float32, _bfloat16, _e4m3, _uint8, _raw_current, _capturing, _current_device
    import torch
    _float32, _bfloat16, _uint8 = torch.float32, torch.bfloat16, torch.uint8
    _e4m3, _raw_current = torch.float8_e4m3fn, torch._C._cuda_getCurrentRawStream
    _capturing = torch._C._cuda_isCurrentStreamCapturing
    _current_device = torch._C._cuda_getDevice
    L = lib()
    _int32 = torch.int32
    return L


def _place(t, name):
    """The index of the device of a call's tensors, which has to be the current one: the launch
    goes there."""
    try:
        dev = t.get_device()
    except AttributeError:
        dev = -1
    if dev < 0:
        _check(t, name)
        raise ValueError(f"{name} is not a usable tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{_current_device()}")
    return dev


def _arg(t, name, ndim, dtype, dev):
    """The pointer of a contiguous tensor of `ndim` dims and `dtype` (None: any) on device `dev`."""
    try:
        if t.get_device() == dev and (t.dtype is dtype or dtype is None) and t.ndim == ndim \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check(t, name, ndim, dtype)
    raise ValueError(f"{name} must be on cuda:{dev} with the other tensors, not on {t.device}")


def _vec(t, name, n, dev):
    """The pointer of an optional int32 [n] tensor."""
    if t is None:
        return None
    p = _arg(t, name, 1, _int32, dev)
    if t.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries, got {t.shape[0]}")
    return p


def _word(t, name, dev):
    """The pointer of an optional int32 tensor of at least one entry."""
    if t is None:
        return None
    p = _arg(t, name, 1, _int32, dev)
    if t.shape[0] < 1:
        raise ValueError(f"{name} must have an entry")
    return p


def _raw_stream(stream, dev):
    """cudaStream_t of `stream`, or of the current stream of the tensors' device."""
    if stream is None:
        return _raw_current(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _q8_pool(kv_pool, kv_scales, dev):
    """Checks the 8-bit pool and its scales; returns their pointers and the pool's shape."""
    pool = _arg(kv_pool, "kv_pool", 6, None, dev)
    scales = _arg(kv_scales, "kv_scales", 4, _float32, dev)
    if kv_pool.dtype is not _e4m3 and kv_pool.dtype is not _uint8:
        raise TypeError(f"kv_pool must be float8_e4m3fn (or its uint8 bytes), got {kv_pool.dtype}")
    shape = kv_pool.shape
    if shape[2] != 2 or kv_scales.shape != shape[:4]:
        raise ValueError("kv_pool must be [num_blocks, layers, 2, kv_heads, block_size, head_dim] "
                         "and kv_scales [num_blocks, layers, 2, kv_heads]")
    return pool, scales, shape


def kv_q8_append(k, v, kv_pool, kv_scales, block_table, seq_lens, *, layer: int = 0,
                 num_new=None, stream=None, err_flag=None) -> None:
    """Writes k, v [B, T, kv_heads, head_dim] (bf16 or fp32) to positions seq_lens[b] ... of the
    8-bit cache's `layer`: kv_pool [num_blocks, layers, 2, kv_heads, block_size, head_dim]
    float8_e4m3fn, kv_scales [num_blocks, layers, 2, kv_heads]. num_new: optional int32 [B]."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(k, "k")
    pool, scales, (NB, NL, _, H, bs, D) = _q8_pool(kv_pool, kv_scales, dev)
    kp = _arg(k, "k", 4, None, dev)
    vp = _arg(v, "v", 4, k.dtype, dev)
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    B, T, kh, kd = k.shape
    rows, MB = block_table.shape
    if v.shape != k.shape or kh != H or kd != D or rows != B:
        raise ValueError(f"k and v must be [B, T, {H}, {D}] and block_table [B, max_blocks]")
    st = L.kv_q8_append(
        kp, vp, SPEC_BF16 if k.dtype is _bfloat16 else _dtype_code(k), pool, scales, bt,
        _vec(seq_lens, "seq_lens", B, dev), _vec(num_new, "num_new", B, dev), NB, NL, layer, H, D,
        bs, B, T, MB,
        _raw_stream(stream, dev), _word(err_flag, "err_flag", dev))
    if st != SPEC_OK:
        raise SpecError("kv_q8_append", st)


def _heads(t, name, dtype, dev):
    """(pointer, numbers from token to token) of a [B, T, heads, head_dim] tensor whose tokens are
    a constant number of elements apart and whose heads lie side by side."""
    try:
        if t.get_device() != dev or t.ndim != 4 or (dtype is not None and t.dtype is not dtype):
            raise AttributeError
    except AttributeError:
        _arg(t, name, 4, dtype, dev)
        raise
    B, T, H, D = t.shape
    s0, s1, s2, s3 = t.stride()
    step = s1 if T > 1 else s0 if B > 1 else H * D
    if (D > 1 and s3 != 1) or (H > 1 and s2 != D) or (T > 1 and B > 1 and s0 != T * s1) \
            or step < H * D:
        raise ValueError(f"{name} must be [B, T, heads, head_dim] with a token's heads side by "
                         f"side and tokens a constant stride apart, got strides {t.stride()}")
    return t.data_ptr(), step


def _turning(q, q_weight, k_weight, inv_freq, positions, dev):
    """Pointers of the weights, the frequencies (with their number) and the positions."""
    B, T, _, D = q.shape

    def weight(w, name):
        if w is None:
            return None
        p = _arg(w, name, 1, q.dtype, dev)
        if w.shape[0] != D:
            raise ValueError(f"{name} must have {D} entries, got {w.shape[0]}")
        return p

    freq, pairs = None, 0
    if inv_freq is not None:
        freq, pairs = _arg(inv_freq, "inv_freq", 1, _float32, dev), inv_freq.shape[0]
        if pairs == 0:
            freq = None
    pos = None
    if positions is not None:
        pos = _arg(positions, "positions", 2, _int32, dev)
        if positions.shape != (B, T):
            raise ValueError(f"positions must be [{B}, {T}], got {tuple(positions.shape)}")
    return weight(q_weight, "q_weight"), weight(k_weight, "k_weight"), freq, pairs, pos


def qk_norm_rope(q, k, seq_lens, q_out, k_out, *, inv_freq=None, rope_factor: float = 1.0,
                 interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6,
                 positions=None, num_new=None, stream=None, err_flag=None) -> None:
    """Norms (with weights [head_dim] given) and rotary positions of q [B, T, q_heads, head_dim]
    and k [B, T, kv_heads, head_dim] (or None) into q_out and k_out, which may be q and k. The
    tensors may be views of one projection's output. inv_freq: float32 [pairs], radians a
    position (rope_frequencies); token t is at seq_lens[b] + t, or at positions [B, T]."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(q, "q")
    dt = q.dtype
    qp, qs = _heads(q, "q", None, dev)
    qo, qos = _heads(q_out, "q_out", dt, dev)
    B, T, Hq, D = q.shape
    if q_out.shape != q.shape:
        raise ValueError(f"q_out must be {tuple(q.shape)}, got {tuple(q_out.shape)}")
    kp = ko = None
    ks = kos = H = 0
    if k is not None:
        kp, ks = _heads(k, "k", dt, dev)
        ko, kos = _heads(k_out, "k_out", dt, dev)
        H = k.shape[2]
        if k_out.shape != k.shape or tuple(k.shape) != (B, T, H, D):
            raise ValueError(f"k and k_out must be [{B}, {T}, kv_heads, {D}]")
    qw, kw, freq, pairs, pos = _turning(q, q_weight, k_weight, inv_freq, positions, dev)
    st = L.qk_norm_rope(
        qp, qs, kp, ks, SPEC_BF16 if dt is _bfloat16 else _dtype_code(q), qo, qos, ko, kos, qw, kw,
        eps, freq, pairs, interleaved, rope_factor, _vec(seq_lens, "seq_lens", B, dev), pos,
        _vec(num_new, "num_new", B, dev), Hq, H, D, B, T, _raw_stream(stream, dev),
        _word(err_flag, "err_flag", dev))
    if st != SPEC_OK:
        raise SpecError("qk_norm_rope", st)


def kv_q8_norm_rope_append(q, k, v, q_out, kv_pool, kv_scales, block_table, seq_lens, *,
                           layer: int = 0, inv_freq=None, rope_factor: float = 1.0,
                           interleaved: bool = False, q_weight=None, k_weight=None,
                           eps: float = 1e-6, positions=None, num_new=None, stream=None,
                           err_flag=None) -> None:
    """qk_norm_rope of q into q_out, and of k into the 8-bit cache together with v (kv_q8_append's
    layout and places), in one pass: the keys are rounded once."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(q, "q")
    dt = q.dtype
    pool, scales, (NB, NL, _, H, bs, D) = _q8_pool(kv_pool, kv_scales, dev)
    qp, qs = _heads(q, "q", None, dev)
    kp, ks = _heads(k, "k", dt, dev)
    vp, vs = _heads(v, "v", dt, dev)
    qo, qos = _heads(q_out, "q_out", dt, dev)
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    B, T, Hq, qd = q.shape
    rows, MB = block_table.shape
    if q_out.shape != q.shape or qd != D or rows != B or tuple(k.shape) != (B, T, H, D) \
            or v.shape != k.shape:
        raise ValueError(f"q and q_out must be [B, T, q_heads, {D}], k and v [B, T, {H}, {D}] and "
                         "block_table [B, max_blocks]")
    qw, kw, freq, pairs, pos = _turning(q, q_weight, k_weight, inv_freq, positions, dev)
    st = L.kv_q8_norm_rope_append(
        qp, qs, kp, ks, vp, vs, SPEC_BF16 if dt is _bfloat16 else _dtype_code(q), qo, qos, qw, kw,
        eps, freq, pairs, interleaved, rope_factor, pool, scales, bt,
        _vec(seq_lens, "seq_lens", B, dev), pos, _vec(num_new, "num_new", B, dev), NB, NL, layer,
        Hq, H, D, bs, B, T, MB, _raw_stream(stream, dev), _word(err_flag, "err_flag", dev))
    if st != SPEC_OK:
        raise SpecError("kv_q8_norm_rope_append", st)


def kv_q8_attention_workspace_bytes(T: int, num_q_heads: int, num_kv_heads: int,
                                    head_dim: int) -> int:
    """Device workspace bytes of kv_q8_attention (0: the call would be rejected)."""
    return int(lib().kv_q8_attention_workspace_bytes(T, num_q_heads, num_kv_heads, head_dim))


_attn_workspaces = {}


def _attn_workspace(shape, device, raw, stream):
    """(pointer, bytes, the tensor that holds them) of a workspace for a call on a stream.

    One is kept for each device and stream: calls on one stream are ordered, calls on two may
    overlap. It is allocated in its stream's order, so a larger one may replace it at any time.
    A capture gets a workspace of its own for each call instead, from the graph's memory: a
    replay may come long after, and on another stream than the calls that share the kept one."""
    import torch
    if stream is None or raw == _raw_current(device.index):
        if not _capturing():
            ws = _attn_workspaces.get((shape, device.index, raw))
            return _new_attn_workspace(shape, device, raw, True) if ws is None else ws
        return _new_attn_workspace(shape, device, raw, False)
    with torch.cuda.stream(stream):
        return _attn_workspace(shape, device, raw, None)


def _new_attn_workspace(shape, device, raw, keep):
    """A workspace in the order of the current stream, `raw`; `keep`: for the calls to come."""
    import torch
    need = (kv_q8_attention_workspace_bytes if len(shape) == 4
            else kv_q8_prefix_attention_workspace_bytes)(*shape)
    if need == 0:
        return None, 0, None  # an unsupported shape: the library call itself reports why
    held = _attn_workspaces.get((device.index, raw)) if keep else None
    if held is None or held.numel() < need + 256:
        held = torch.empty(need + 256, dtype=torch.uint8, device=device)
    off = (-held.data_ptr()) % 256
    ws = held.data_ptr() + off, held.numel() - off, held
    if keep:
        if _attn_workspaces.get((device.index, raw)) is not held:
            for k in [k for k in list(_attn_workspaces) if k[1:] == (device.index, raw)]:
                _attn_workspaces.pop(k, None)
            _attn_workspaces[(device.index, raw)] = held
        _attn_workspaces[(shape, device.index, raw)] = ws
    return ws


def kv_q8_attention(q, kv_pool, kv_scales, block_table, seq_lens, out, *, layer: int = 0,
                    softmax_scale: float | None = None, window: int = 0, sinks: int = 0,
                    num_new=None, tree_mask=None, workspace=None, stream=None,
                    err_flag=None) -> None:
    """Attention of q [B, T, q_heads, head_dim] (positions seq_lens[b] + t) over the 8-bit cache
    (layout as kv_q8_append) into out, same shape and dtype (bf16 or fp32). softmax_scale defaults
    to head_dim ** -0.5; window / sinks: sliding window and always-visible first positions;
    tree_mask: optional int32 [B, T], bit s of entry t lets query t see position seq_lens[b] + s.
    workspace: a uint8 tensor of kv_q8_attention_workspace_bytes + 256; None: one that the
    binding keeps for the stream, or under a capture one in the graph's memory."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(q, "q")
    pool, scales, (NB, NL, _, H, bs, D) = _q8_pool(kv_pool, kv_scales, dev)
    qp = _arg(q, "q", 4, None, dev)
    op = _arg(out, "out", 4, q.dtype, dev)
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    shape = q.shape
    B, T, Hq, qd = shape
    rows, MB = block_table.shape
    if out.shape != shape or qd != D or rows != B:
        raise ValueError(f"q and out must be [B, T, q_heads, {D}] and block_table [B, max_blocks]")
    tm = None
    if tree_mask is not None:
        tm = _arg(tree_mask, "tree_mask", 2, _int32, dev)
        if tuple(tree_mask.shape) != (B, T):
            raise ValueError(f"tree_mask must be [{B}, {T}], got {tuple(tree_mask.shape)}")
    raw = _raw_stream(stream, dev)
    if workspace is None:
        ws = _attn_workspaces.get(((T, Hq, H, D), dev, raw))
        if ws is None or stream is not None or _capturing():
            ws = _attn_workspace((T, Hq, H, D), q.device, raw, stream)
        wsp, wsn, held = ws  # `held` lives until the launch is made
    else:
        wsp = _arg(workspace, "workspace", 1, _uint8, dev)
        off = -wsp % 256
        wsp, wsn = wsp + off, max(0, workspace.numel() - off)
    st = L.kv_q8_attention(
        qp, SPEC_BF16 if q.dtype is _bfloat16 else _dtype_code(q), pool, scales, bt,
        _vec(seq_lens, "seq_lens", B, dev), _vec(num_new, "num_new", B, dev), tm, op,
        D ** -0.5 if softmax_scale is None else softmax_scale,
        window, sinks, NB, NL, layer, Hq, H, D, bs, B, T, MB, wsp, wsn, raw,
        _word(err_flag, "err_flag", dev))
    if st != SPEC_OK:
        raise SpecError("kv_q8_attention", st)


def kv_prefix_plan_bytes(B: int, num_groups: int, num_members: int) -> int:
    """Bytes of a plan of kv_prefix_plan (0: the call would be rejected)."""
    return int(lib().kv_prefix_plan_bytes(B, num_groups, num_members))


def kv_prefix_plan(block_table, seq_lens, group_starts, group_rows, *, tokens: int, q_heads: int,
                   kv_heads: int, block_size: int, num_blocks: int, num_new=None, plan=None,
                   stream=None, err_flag=None):
    """The plan of a step's kv_q8_prefix_attention calls (every layer's): which rows share the
    first blocks of their tables. group_rows int32 [members]: rows, group after group;
    group_starts int32 [groups + 1]. `tokens` is the T of the queries. Returns `plan`, a uint8
    tensor of kv_prefix_plan_bytes + 256 (None: a new one)."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(block_table, "block_table")
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    B, MB = block_table.shape
    starts = _arg(group_starts, "group_starts", 1, _int32, dev)
    rows = _arg(group_rows, "group_rows", 1, _int32, dev)
    NG, NE = group_starts.shape[0] - 1, group_rows.shape[0]
    raw = _raw_stream(stream, dev)
    if plan is None:
        import torch
        need = L.kv_prefix_plan_bytes(B, NG, NE)
        if raw == _raw_current(dev):
            plan = torch.empty(need + 256, dtype=_uint8, device=block_table.device)
        else:  # in the order of the stream that uses it
            with torch.cuda.stream(stream):
                plan = torch.empty(need + 256, dtype=_uint8, device=block_table.device)
    p, n = _aligned(plan, "plan", dev)
    st = L.kv_prefix_plan(
        bt, _vec(seq_lens, "seq_lens", B, dev), _vec(num_new, "num_new", B, dev), starts, rows, NG,
        NE, tokens, q_heads, kv_heads, num_blocks, block_size, B, MB, p, n, raw,
        _word(err_flag, "err_flag", dev))
    if st != SPEC_OK:
        raise SpecError("kv_prefix_plan", st)
    return plan


def _aligned(t, name, dev):
    """(pointer, bytes) of a uint8 tensor from its first 256-byte boundary."""
    p = _arg(t, name, 1, _uint8, dev)
    off = -p % 256
    return p + off, max(0, t.shape[0] - off)


def kv_q8_prefix_attention_workspace_bytes(B: int, T: int, num_q_heads: int, num_kv_heads: int,
                                           head_dim: int) -> int:
    """Device workspace bytes of kv_q8_prefix_attention (0: the call would be rejected)."""
    return int(lib().kv_q8_prefix_attention_workspace_bytes(B, T, num_q_heads, num_kv_heads,
                                                            head_dim))


def kv_q8_prefix_attention(q, kv_pool, kv_scales, block_table, seq_lens, plan, out, *,
                           layer: int = 0, softmax_scale: float | None = None, num_new=None,
                           tree_mask=None, workspace=None, stream=None, err_flag=None) -> None:
    """kv_q8_attention (without a window) for rows some of which share the first blocks of their
    tables: `plan` is kv_prefix_plan's for the same tables, lengths and heads. workspace as there,
    of kv_q8_prefix_attention_workspace_bytes + 256."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(q, "q")
    pool, scales, (NB, NL, _, H, bs, D) = _q8_pool(kv_pool, kv_scales, dev)
    qp = _arg(q, "q", 4, None, dev)
    op = _arg(out, "out", 4, q.dtype, dev)
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    shape = q.shape
    B, T, Hq, qd = shape
    rows, MB = block_table.shape
    if out.shape != shape or qd != D or rows != B:
        raise ValueError(f"q and out must be [B, T, q_heads, {D}] and block_table [B, max_blocks]")
    tm = None
    if tree_mask is not None:
        tm = _arg(tree_mask, "tree_mask", 2, _int32, dev)
        if tuple(tree_mask.shape) != (B, T):
            raise ValueError(f"tree_mask must be [{B}, {T}], got {tuple(tree_mask.shape)}")
    pp, pn = _aligned(plan, "plan", dev)
    raw = _raw_stream(stream, dev)
    if workspace is None:
        ws = _attn_workspaces.get(((B, T, Hq, H, D), dev, raw))
        if ws is None or stream is not None or _capturing():
            ws = _attn_workspace((B, T, Hq, H, D), q.device, raw, stream)
        wsp, wsn, held = ws  # `held` lives until the launch is made
    else:
        wsp, wsn = _aligned(workspace, "workspace", dev)
    st = L.kv_q8_prefix_attention(
        qp, SPEC_BF16 if q.dtype is _bfloat16 else _dtype_code(q), pool, scales, bt,
        _vec(seq_lens, "seq_lens", B, dev), _vec(num_new, "num_new", B, dev), tm, pp, pn, op,
        D ** -0.5 if softmax_scale is None else softmax_scale, NB, NL, layer, Hq, H, D, bs, B, T,
        MB, wsp, wsn, raw, _word(err_flag, "err_flag", dev))
    if st != SPEC_OK:
        raise SpecError("kv_q8_prefix_attention", st)


def kv_reserve(block_table, seq_lens, free_stack, free_top, status, *, n: int, block_size: int,
               num_blocks: int, num_new=None, stream=None) -> None:
    """Blocks for n (or num_new[b]) tokens past seq_lens[b]; status receives 0 or error bits."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(block_table, "block_table")
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    B, MB = block_table.shape
    st = L.kv_reserve(
        bt, _vec(seq_lens, "seq_lens", B, dev), _vec(num_new, "num_new", B, dev), n, num_blocks,
        block_size, B, MB, _vec(free_stack, "free_stack", num_blocks, dev),
        _word(free_top, "free_top", dev), _word(status, "status", dev), _raw_stream(stream, dev))
    if st != SPEC_OK:
        raise SpecError("kv_reserve", st)


def kv_fork(block_table, seq_lens, extra_refs, src_rows, dst_rows, kv_pool, free_stack, free_top,
            status, *, block_size: int, kv_scales=None, stream=None) -> None:
    """Rows dst_rows[i] become copies of rows src_rows[i]: full blocks shared, tail blocks copied.
    kv_pool: the 8-bit pool with kv_scales, or kv_commit_rollback's [num_blocks, layers, 2,
    block_size, kv_heads, head_dim] pool without."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(block_table, "block_table")
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    B, MB = block_table.shape
    if kv_scales is not None:
        pool, scales, (NB, NL, _, H, bs, D) = _q8_pool(kv_pool, kv_scales, dev)
        planes, token = NL * 2 * H, D
    else:
        pool, scales = _arg(kv_pool, "kv_pool", 6, None, dev), None
        NB, NL, two, bs, H, D = kv_pool.shape
        if two != 2:
            raise ValueError("kv_pool must be [num_blocks, layers, 2, block_size, heads, head_dim]")
        planes, token = NL * 2, H * D * kv_pool.element_size()
    if bs != block_size:
        raise ValueError(f"kv_pool holds blocks of {bs} tokens, not {block_size}")
    src = _arg(src_rows, "src_rows", 1, _int32, dev)
    n = src_rows.shape[0]
    st = L.kv_fork(
        bt, _vec(seq_lens, "seq_lens", B, dev), _vec(extra_refs, "extra_refs", NB, dev), src,
        _vec(dst_rows, "dst_rows", n, dev), n, pool, planes, token, scales, NB, block_size, B, MB,
        _vec(free_stack, "free_stack", NB, dev), _word(free_top, "free_top", dev),
        _word(status, "status", dev), _raw_stream(stream, dev))
    if st != SPEC_OK:
        raise SpecError("kv_fork", st)


def kv_free(block_table, seq_lens, extra_refs, rows, free_stack, free_top, status, *,
            num_blocks: int, stream=None) -> None:
    """Releases the listed rows; blocks that no other row holds go back on the free stack."""
    L = _lib if _int32 is not None else _ready()
    dev = _place(block_table, "block_table")
    bt = _arg(block_table, "block_table", 2, _int32, dev)
    B, MB = block_table.shape
    st = L.kv_free(
        bt, _vec(seq_lens, "seq_lens", B, dev), _vec(extra_refs, "extra_refs", num_blocks, dev),
        _arg(rows, "rows", 1, _int32, dev), rows.shape[0], num_blocks, B, MB,
        _vec(free_stack, "free_stack", num_blocks, dev), _word(free_top, "free_top", dev),
        _word(status, "status", dev), _raw_stream(stream, dev))
    if st != SPEC_OK:
        raise SpecError("kv_free", st)


def spec_selftest_ex2(lo: float, hi: float, *, stream=None) -> float:
    """Maximum relative error of the hardware exp2 over all fp32 arguments in [lo, hi]."""
    import torch
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    st = lib().spec_selftest_ex2(ctypes.c_float(lo), ctypes.c_float(hi), _ptr(out),
                                 _stream(stream))
    if st != SPEC_OK:
        raise SpecError("spec_selftest_ex2", st)
    return float(out.item())


# ------------------------------------------------------------------ conveniences
def rope_frequencies(pairs: int, base: float = 10000.0, *, scaling: str = "none",
                     factor: float = 1.0, trained_length: int = 4096, fast_turns: float = 32.0,
                     slow_turns: float = 1.0, device="cuda"):
    """(inv_freq float32 [pairs], rope_factor) for qk_norm_rope: base ** (-i / pairs), scaled for
    contexts `factor` times as long as the trained one:

      "none"    as it is
      "linear"  all frequencies / factor (positions closer together)
      "base"    a base of base * factor ** (pairs / (pairs - 1)): the slowest pair is slowed by
                `factor`, the fastest not at all
      "parts"   pairs that turn at least fast_turns times in trained_length as they are, those
                that turn at most slow_turns times / factor, those between them mixed linearly;
                rope_factor = 0.1 ln(factor) + 1
    """
    import math
    import torch
    if pairs < 1 or not base > 0 or not factor > 0:
        raise ValueError("pairs, base and factor must be positive")
    by = 1.0
    if scaling == "base":
        base = base * factor ** (pairs / max(1, pairs - 1))
    f = base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not fast_turns > slow_turns or trained_length < 1:
            raise ValueError("fast_turns must exceed slow_turns, trained_length be positive")
        turns = trained_length * f / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        by = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.float().to(device), by


def verify(target_logits, draft_logits, draft_tokens, uniforms, temperature: float, *,
           stream=None, with_info: bool = False):
    """Allocates the outputs on the logits' device and runs spec_verify_sample.
    Returns (out_tokens [B,K+1], num_accepted [B]) (+ (row_info, err) if with_info)."""
    import torch
    B, K1, _ = target_logits.shape
    dev = target_logits.device
    out = torch.empty((B, K1), dtype=torch.int32, device=dev)
    n = torch.empty((B,), dtype=torch.int32, device=dev)
    info = torch.empty((B,), dtype=torch.int32, device=dev) if with_info else None
    err = torch.zeros((1,), dtype=torch.int32, device=dev) if with_info else None
    spec_verify_sample(target_logits, draft_logits, draft_tokens, uniforms, temperature, out, n,
                       stream=stream, err_flag=err, row_info=info)
    return (out, n, info, err) if with_info else (out, n)


def verify_host(target_logits, draft_logits, draft_tokens, uniforms, temperature: float, *,
                device="cuda", stream=None):
    """End-to-end call on HOST (CPU, ideally pinned) tensors: copies the inputs to the
    device, verifies, and copies (out_tokens, num_accepted) back to the host."""
    import torch
    s = stream or torch.cuda.current_stream()
    with torch.cuda.stream(s):
        t = target_logits.to(device, non_blocking=True)
        d = draft_logits.to(device, non_blocking=True) if draft_logits is not None else None
        k = draft_tokens.to(device, non_blocking=True)
        u = uniforms.to(device, non_blocking=True)
        out, n = verify(t, d, k, u, temperature, stream=s)
        out_h = out.to("cpu", non_blocking=False)
        n_h = n.to("cpu", non_blocking=False)
    return out_h, n_h


class HostVerifier:
    """End-to-end sampling verification of batches held in HOST memory (pinned).

    The batch rows are copied to preallocated device buffers in `chunks` row
    chunks on a copy stream; chunk c is verified (spec_verify_sample on its
    rows) as soon as its copy lands, while the next chunk is still in flight,
    so the verification hides behind the transfer. Outputs stay on the device
    (`out_tokens`, `num_accepted`); `to_host` copies them into pinned host
    tensors on the same stream.
    """

    def __init__(self, B: int, K: int, V: int, *, dtype=None, chunks: int = 8, device="cuda"):
        import torch
        dtype = dtype or torch.bfloat16
        self.B, self.K, self.V = B, K, V
        self.chunks = max(1, min(chunks, B))
        d = torch.device(device)
        self.target = torch.empty((B, K + 1, V), dtype=dtype, device=d)
        self.draft = torch.empty((B, K, V), dtype=dtype, device=d)
        self.tokens = torch.empty((B, K), dtype=torch.int32, device=d)
        self.uniforms = torch.empty((B, K + 1), dtype=torch.float32, device=d)
        self.out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=d)
        self.num_accepted = torch.empty((B,), dtype=torch.int32, device=d)
        self.copy_stream = torch.cuda.Stream(device=d)
        self.events = [torch.cuda.Event() for _ in range(self.chunks)]
        step = -(-B // self.chunks)
        self.bounds = [(r0, min(B, r0 + step)) for r0 in range(0, B, step)]

    def __call__(self, target_h, draft_h, tokens_h, uniforms_h, temperature: float, *,
                 stream=None):
        import torch
        main = stream or torch.cuda.current_stream()
        start = torch.cuda.Event()
        start.record(main)                      # earlier work on the buffers is ordered first
        cs = self.copy_stream
        cs.wait_event(start)
        with torch.cuda.stream(cs):
            for (r0, r1), ev in zip(self.bounds, self.events):
                self.target[r0:r1].copy_(target_h[r0:r1], non_blocking=True)
                self.draft[r0:r1].copy_(draft_h[r0:r1], non_blocking=True)
                self.tokens[r0:r1].copy_(tokens_h[r0:r1], non_blocking=True)
                self.uniforms[r0:r1].copy_(uniforms_h[r0:r1], non_blocking=True)
                ev.record(cs)
        for (r0, r1), ev in zip(self.bounds, self.events):
            main.wait_event(ev)
            spec_verify_sample(self.target[r0:r1], self.draft[r0:r1], self.tokens[r0:r1],
                               self.uniforms[r0:r1], temperature, self.out_tokens[r0:r1],
                               self.num_accepted[r0:r1], stream=main)
        return self.out_tokens, self.num_accepted

    def to_host(self, out_h, n_h, *, stream=None):
        """Copies the outputs into host tensors (pinned for an asynchronous copy)."""
        import torch
        main = stream or torch.cuda.current_stream()
        with torch.cuda.stream(main):
            out_h.copy_(self.out_tokens, non_blocking=True)
            n_h.copy_(self.num_accepted, non_blocking=True)

