"""Thin Python binding of libspecverify.so (argument marshalling only).

Every step of the verify runs in the library's HIP kernels; this module only
turns torch tensors into device pointers, allocates outputs and the workspace
with torch on the tensors' device, and passes torch's current stream.  It
raises when the library is missing: there is no fallback path.
"""

from __future__ import annotations

import ctypes
import dataclasses
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_F32, SV_BF16 = 0, 1
ONEHOT, LOGITS, PROBS, MATCH = 0, 1, 2, 3
ROW_OK, ROW_NONFINITE, ROW_EMPTY, ROW_BAD_K, ROW_BAD_TOKEN, ROW_BAD_PARAM, ROW_INTERNAL = range(7)
ROW_NO_PAGES, ROW_BAD_PAGE = 7, 8
MAX_K = 63

_lib = None
_lock = threading.Lock()
_ws_cache: dict = {}
_kv_ws_cache: dict = {}
_kv_locks: dict = {}

_vp = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t


class SpecVerifyError(RuntimeError):
    pass


def load_library(path: str) -> ctypes.CDLL:
    """Open a build of the library at `path` with the C ABI's signatures."""
    if not os.path.exists(path):
        raise SpecVerifyError(
            f"{path} is missing; build it with `python -m lossless_rejection_sampling_spec_amd.build`")
    L = ctypes.CDLL(path)
    L.spec_verify_abi_version.restype = _i32
    L.spec_verify_abi_version.argtypes = []
    L.spec_verify_status_string.restype = ctypes.c_char_p
    L.spec_verify_status_string.argtypes = [_i32]
    L.spec_verify_workspace_bytes.restype = _sz
    L.spec_verify_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32]
    L.spec_verify_workspace_init.restype = _i32
    L.spec_verify_workspace_init.argtypes = [_vp, _sz, _vp]
    L.spec_verify_greedy.restype = _i32
    L.spec_verify_greedy.argtypes = [
        _vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
        _vp, _vp, _vp, _vp, _sz, _vp]
    L.spec_verify_sampled.restype = _i32
    L.spec_verify_sampled.argtypes = [
        _vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
        _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.spec_verify_drain.restype = _i32
    L.spec_verify_drain.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp]
    L.spec_verify_accounting.restype = _i32
    L.spec_verify_accounting.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, ctypes.c_float,
                                         ctypes.c_float, _i32, _i32, _vp, _vp, _vp]
    L.spec_verify_sampled_penalized.restype = _i32
    L.spec_verify_sampled_penalized.argtypes = [
        _vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
        _vp, _vp, _vp, _vp, _vp, _i64, _vp,
        _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    L.spec_verify_sampled_noalloc.restype = _i32
    L.spec_verify_sampled_noalloc.argtypes = [
        _vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
        _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
    L.spec_kv_page_bytes.restype = _sz
    L.spec_kv_page_bytes.argtypes = [_i32, _i32, _i32]
    L.spec_kv_append.restype = _i32
    L.spec_kv_append.argtypes = [
        _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, ctypes.c_float, _vp, _i32, _i32, _i32,
        _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp,
        _vp, _vp]
    L.spec_kv_append_at.restype = _i32
    L.spec_kv_append_at.argtypes = [
        _vp, _i64, _vp, _i64, _vp, _i64, _i32, _vp, _vp, ctypes.c_float, _vp, _i32, _i32, _i32,
        _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _i64, _vp, _i64, _vp,
        _vp, _vp, _vp]
    L.spec_kv_attention_workspace_bytes.restype = _sz
    L.spec_kv_attention_workspace_bytes.argtypes = [_i32] * 9
    L.spec_kv_attention.restype = _i32
    L.spec_kv_attention.argtypes = [
        _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _i64,
        _i32, ctypes.c_float, _i32, _i32, _vp, _i64, _vp, _vp, _sz, _vp]
    L.spec_kv_prompt_workspace_bytes.restype = _sz
    L.spec_kv_prompt_workspace_bytes.argtypes = [_i32] * 7 + [_i64, _i32, _i32]
    L.spec_kv_prompt_attention.restype = _i32
    L.spec_kv_prompt_attention.argtypes = [
        _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _i64, _i32,
        _i64, ctypes.c_float, _i32, _i32, _vp, _i64, _vp, _vp, _sz, _vp]
    L.spec_kv_weights_workspace_bytes.restype = _sz
    L.spec_kv_weights_workspace_bytes.argtypes = [_i32] * 9
    L.spec_kv_attention_weights.restype = _i32
    L.spec_kv_attention_weights.argtypes = [
        _vp, _i64, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp,
        _i64, _i32, ctypes.c_float, _i32, _i32, _vp, _vp, _i64, _vp, _vp, _sz, _vp]
    L.spec_kv_evict.restype = _i32
    L.spec_kv_evict.argtypes = [_vp, _i32, _i32, _i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _i64,
                                _vp, _i64, _vp, _i32, _i64, _vp, _vp, _vp]
    L.spec_kv_pages_workspace_bytes.restype = _sz
    L.spec_kv_pages_workspace_bytes.argtypes = [_i32, _i64]
    L.spec_kv_reserve.restype = _i32
    L.spec_kv_reserve.argtypes = [_vp, _i32, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i32,
                                  _i64, _vp, _vp, _vp, _sz, _vp]
    L.spec_kv_release.restype = _i32
    L.spec_kv_release.argtypes = [_vp, _vp, _i32, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _vp]
    L.spec_kv_fork.restype = _i32
    L.spec_kv_fork.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i64, _vp, _i64, _vp,
                               _vp]
    L.spec_kv_compact.restype = _i32
    L.spec_kv_compact.argtypes = [_i32, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64,
                                  _vp, _vp, _sz, _vp]
    return L


def lib() -> ctypes.CDLL:
    """Load libspecverify.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                _lib = load_library(LIB_PATH)
    return _lib


def abi_version() -> int:
    return int(lib().spec_verify_abi_version())


def status_string(code: int) -> str:
    return lib().spec_verify_status_string(int(code)).decode()


def workspace_bytes(batch: int, total_rows: int, vocab: int, max_k: int) -> int:
    return int(lib().spec_verify_workspace_bytes(batch, total_rows, vocab, max_k))


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise ValueError(f"unsupported logit dtype {t.dtype} (float32 or bfloat16)")


def _check_rows(t: torch.Tensor, name: str) -> None:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit stride along the vocabulary")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _check_vec(t: torch.Tensor | None, name: str, dtype, n: int | None = None) -> None:
    if t is None:
        return
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} device tensor")
    if n is not None and t.numel() < n:
        raise ValueError(f"{name} needs at least {n} elements")


def get_workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """A zero-initialised workspace cached per (device, current stream).

    The library leaves a workspace ready after every call, so it is reused
    without clearing.  Calls that may run concurrently must not share one, so
    each stream gets its own: calls on one stream are ordered by the stream."""
    device = torch.device(device)
    stream = torch.cuda.current_stream(device)
    key = (device.type, device.index, stream.cuda_stream)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def reset_workspace(workspace: torch.Tensor | None = None, device=None) -> None:
    """Zero-fill a workspace on the current stream (spec_verify_workspace_init).

    Call it after any request reports ROW_INTERNAL (a wait between the
    library's workgroups ran out): such a call can leave hand-off words in
    flight that the next call would take as fresh.  With no argument, every
    workspace cached for `device` (default: the current device) is cleared,
    each on the stream it belongs to."""
    if workspace is not None:
        targets = [(workspace, torch.cuda.current_stream(workspace.device).cuda_stream)]
    else:
        dev = torch.device(device) if device is not None else torch.device(
            "cuda", torch.cuda.current_device())
        targets = [(ws, key[2]) for key, ws in _ws_cache.items()
                   if key[0] == dev.type and key[1] == dev.index]
    for ws, stream in targets:
        _raise(lib().spec_verify_workspace_init(_ptr(ws), ws.numel(), stream))


def _raise(rc: int) -> None:
    if rc != 0:
        raise ValueError(f"spec_verify: {status_string(rc)} (code {rc})")


def verify_greedy(target: torch.Tensor, cu_seqlens: torch.Tensor, draft_tokens: torch.Tensor,
                  *, max_k: int, vocab: int | None = None, workspace: torch.Tensor | None = None,
                  out: tuple | None = None):
    """Greedy prefix-match verify.  Returns (accepted[B], out_tokens[R], status[B])."""
    _check_rows(target, "target")
    dev = target.device
    batch = cu_seqlens.numel() - 1
    total_rows = target.shape[0]
    V = target.shape[1] if vocab is None else int(vocab)
    _check_vec(cu_seqlens, "cu_seqlens", torch.int32, batch + 1)
    _check_vec(draft_tokens, "draft_tokens", torch.int32)
    if out is None:
        accepted = torch.empty(batch, dtype=torch.int32, device=dev)
        tokens = torch.empty(total_rows, dtype=torch.int32, device=dev)
        status = torch.empty(batch, dtype=torch.int32, device=dev)
    else:
        accepted, tokens, status = out
    need = workspace_bytes(batch, total_rows, V, max_k)
    if need == 0:
        raise ValueError("invalid sizes for spec_verify_greedy")
    ws = get_workspace(dev, need) if workspace is None else workspace
    rc = lib().spec_verify_greedy(
        _ptr(target), _dtype_code(target), target.stride(0), _ptr(cu_seqlens),
        _ptr(draft_tokens) if draft_tokens.numel() else None, batch, total_rows, max_k, V,
        _ptr(accepted), _ptr(tokens), _ptr(status), _ptr(ws), ws.numel(), _stream(dev))
    _raise(rc)
    return accepted, tokens, status


def verify_sampled(target: torch.Tensor, draft: torch.Tensor | None, draft_kind: torch.Tensor,
                   cu_seqlens: torch.Tensor, draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                   temperature: torch.Tensor, top_k: torch.Tensor | None = None,
                   top_p: torch.Tensor | None = None, *, max_k: int, vocab: int | None = None,
                   want_probs: bool = False, workspace: torch.Tensor | None = None,
                   out: tuple | None = None, presence: torch.Tensor | None = None,
                   frequency: torch.Tensor | None = None, history: tuple | None = None,
                   penalized: torch.Tensor | None = None):
    """Sampled verify by rejection sampling (greedy requests mixed in).

    With presence and frequency (float32 [B]) the call goes to
    spec_verify_sampled_penalized: history = (offsets int32 [B+1], tokens
    int32 [nnz], counts int32 [nnz]) or None, and `penalized` the scratch of
    the penalized rows (allocated like `target` when None).

    Returns (accepted[B], out_tokens[R], status[B], p_at_draft, q_at_draft);
    the last two are None unless want_probs."""
    _check_rows(target, "target")
    dev = target.device
    batch = cu_seqlens.numel() - 1
    total_rows = target.shape[0]
    V = target.shape[1] if vocab is None else int(vocab)
    n_draft = total_rows - batch
    if draft is not None:
        _check_rows(draft, "draft")
    _check_vec(cu_seqlens, "cu_seqlens", torch.int32, batch + 1)
    _check_vec(draft_kind, "draft_kind", torch.int32, batch)
    _check_vec(draft_tokens, "draft_tokens", torch.int32, n_draft)
    _check_vec(uniforms, "uniforms", torch.float32, total_rows)
    _check_vec(temperature, "temperature", torch.float32, batch)
    _check_vec(top_k, "top_k", torch.int32, batch)
    _check_vec(top_p, "top_p", torch.float32, batch)
    if out is None:
        accepted = torch.empty(batch, dtype=torch.int32, device=dev)
        tokens = torch.empty(total_rows, dtype=torch.int32, device=dev)
        status = torch.empty(batch, dtype=torch.int32, device=dev)
        p_at = torch.empty(max(n_draft, 1), dtype=torch.float32, device=dev) if want_probs else None
        q_at = torch.empty(max(n_draft, 1), dtype=torch.float32, device=dev) if want_probs else None
    else:
        accepted, tokens, status, p_at, q_at = out
    need = workspace_bytes(batch, total_rows, V, max_k)
    if need == 0:
        raise ValueError("invalid sizes for spec_verify_sampled")
    ws = get_workspace(dev, need) if workspace is None else workspace
    if presence is None and frequency is None:
        rc = lib().spec_verify_sampled(
            _ptr(target), _dtype_code(target), target.stride(0),
            _ptr(draft), _dtype_code(draft) if draft is not None else SV_F32,
            draft.stride(0) if draft is not None else 0,
            _ptr(draft_kind), _ptr(cu_seqlens), _ptr(draft_tokens) if n_draft else None,
            _ptr(uniforms), _ptr(temperature), _ptr(top_k), _ptr(top_p),
            batch, total_rows, max_k, V, _ptr(accepted), _ptr(tokens), _ptr(p_at), _ptr(q_at),
            _ptr(status), _ptr(ws), ws.numel(), _stream(dev))
    else:
        _check_vec(presence, "presence", torch.float32, batch)
        _check_vec(frequency, "frequency", torch.float32, batch)
        h_off = h_tok = h_cnt = None
        nnz = 0
        if history is not None:
            h_off, h_tok, h_cnt = history
            nnz = h_tok.numel()
            _check_vec(h_off, "history offsets", torch.int32, batch + 1)
            _check_vec(h_tok, "history tokens", torch.int32, nnz)
            _check_vec(h_cnt, "history counts", torch.int32, nnz)
        if penalized is None:
            penalized = torch.empty_strided(target.shape, target.stride(), dtype=target.dtype,
                                            device=dev)
        if (penalized.dtype != target.dtype or penalized.stride() != target.stride()
                or penalized.shape != target.shape or penalized.device != dev):
            raise ValueError("penalized must match target's shape, strides, dtype and device")
        rc = lib().spec_verify_sampled_penalized(
            _ptr(target), _dtype_code(target), target.stride(0),
            _ptr(draft), _dtype_code(draft) if draft is not None else SV_F32,
            draft.stride(0) if draft is not None else 0,
            _ptr(draft_kind), _ptr(cu_seqlens), _ptr(draft_tokens) if n_draft else None,
            _ptr(uniforms), _ptr(temperature), _ptr(top_k), _ptr(top_p),
            _ptr(presence), _ptr(frequency), _ptr(h_off) if nnz else None,
            _ptr(h_tok) if nnz else None, _ptr(h_cnt) if nnz else None, nnz, _ptr(penalized),
            batch, total_rows, max_k, V, _ptr(accepted), _ptr(tokens), _ptr(p_at), _ptr(q_at),
            _ptr(status), _ptr(ws), ws.numel(), _stream(dev))
    _raise(rc)
    return accepted, tokens, status, p_at, q_at


def verify_sampled_noalloc(target: torch.Tensor, draft: torch.Tensor | None,
                           draft_kind: torch.Tensor, cu_seqlens: torch.Tensor,
                           draft_tokens: torch.Tensor, uniforms: torch.Tensor,
                           temperature: torch.Tensor, top_k: torch.Tensor | None = None,
                           top_p: torch.Tensor | None = None, *, max_k: int, vocab: int,
                           out: tuple):
    """spec_verify_sampled_noalloc: the sampled verify with the library's
    static scratch array instead of a workspace.  `out` = (accepted, tokens,
    status, p_at or None, q_at or None), preallocated by the caller, so this
    call allocates nothing."""
    batch = cu_seqlens.numel() - 1
    total_rows = target.shape[0]
    accepted, tokens, status, p_at, q_at = out
    rc = lib().spec_verify_sampled_noalloc(
        _ptr(target), _dtype_code(target), target.stride(0),
        _ptr(draft), _dtype_code(draft) if draft is not None else SV_F32,
        draft.stride(0) if draft is not None else 0,
        _ptr(draft_kind), _ptr(cu_seqlens),
        _ptr(draft_tokens) if total_rows > batch else None,
        _ptr(uniforms), _ptr(temperature), _ptr(top_k), _ptr(top_p),
        batch, total_rows, max_k, int(vocab), _ptr(accepted), _ptr(tokens), _ptr(p_at),
        _ptr(q_at), _ptr(status), _stream(target.device))
    _raise(rc)
    return accepted, tokens, status, p_at, q_at


def drain(cu_seqlens: torch.Tensor, accepted: torch.Tensor, status: torch.Tensor,
          out_tokens: torch.Tensor):
    """spec_verify_drain: (committed [total_rows], commit_offsets [B+1],
    rollback [B]); only committed[:commit_offsets[B]] is written."""
    dev = out_tokens.device
    batch = cu_seqlens.numel() - 1
    total_rows = out_tokens.numel()
    for t, n in ((cu_seqlens, batch + 1), (accepted, batch), (status, batch), (out_tokens, total_rows)):
        _check_vec(t, "drain input", torch.int32, n)
    committed = torch.empty(total_rows, dtype=torch.int32, device=dev)
    offsets = torch.empty(batch + 1, dtype=torch.int32, device=dev)
    rollback = torch.empty(batch, dtype=torch.int32, device=dev)
    _raise(lib().spec_verify_drain(_ptr(cu_seqlens), _ptr(accepted), _ptr(status), _ptr(out_tokens),
                                   batch, total_rows, _ptr(committed), _ptr(offsets),
                                   _ptr(rollback), _stream(dev)))
    return committed, offsets, rollback


def accounting(cu_seqlens: torch.Tensor, accepted: torch.Tensor, status: torch.Tensor,
               ema: torch.Tensor, counters: torch.Tensor, *, beta: float = 0.1,
               threshold: float = 0.4, k_low: int = 2, k_high: int = 5):
    """spec_verify_accounting: updates `ema` (float32 [B]) and `counters`
    (int64 [4]: generated, drafted, accepted, requests) in place and returns
    k_next (int32 [B])."""
    dev = ema.device
    batch = cu_seqlens.numel() - 1
    _check_vec(cu_seqlens, "cu_seqlens", torch.int32, batch + 1)
    _check_vec(accepted, "accepted", torch.int32, batch)
    _check_vec(status, "status", torch.int32, batch)
    _check_vec(ema, "ema", torch.float32, batch)
    _check_vec(counters, "counters", torch.int64, 4)
    k_next = torch.empty(batch, dtype=torch.int32, device=dev)
    _raise(lib().spec_verify_accounting(_ptr(cu_seqlens), _ptr(accepted), _ptr(status), batch,
                                        _ptr(ema), _ptr(ema), float(beta), float(threshold),
                                        int(k_low), int(k_high), _ptr(k_next), _ptr(counters),
                                        _stream(dev)))
    return k_next


def kv_page_bytes(kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of one page of one layer (0 on invalid sizes)."""
    if not (0 < kv_heads <= 1024 and 0 < head_dim <= 256 and 0 < page_size <= 256):
        return 0                     # (ctypes would take the low 32 bits of a larger number)
    return int(lib().spec_kv_page_bytes(kv_heads, head_dim, page_size))


@dataclasses.dataclass(frozen=True, eq=False)
class KVCache:
    """The device state of a 4-bit paged KV cache (see include/specverify.h).

    pages       uint8 [layers, num_pages, kv_page_bytes]
    page_table  int32 [requests, pages per request], shared by all layers
    seq_lens    int32 [requests]
    ref_counts  int32 [num_pages], 0 = free
    """
    pages: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    ref_counts: torch.Tensor
    page_size: int
    kv_heads: int
    head_dim: int

    def __post_init__(self):
        n = kv_page_bytes(self.kv_heads, self.head_dim, self.page_size)
        if n == 0:
            raise ValueError("KVCache: head_dim is 64, 128 or 256, page_size 16, 32, 64, 128 or 256")
        p = self.pages
        if (p.dtype != torch.uint8 or not p.is_cuda or p.dim() != 3 or p.shape[2] != n
                or p.shape[0] < 1 or p.shape[1] < 1 or p.stride()[1:] != (n, 1)
                or p.stride(0) < p.shape[1] * n and p.shape[0] > 1 or p.data_ptr() % 16
                or p.stride(0) % 16 and p.shape[0] > 1):
            raise ValueError(f"pages must be a 16-byte aligned uint8 device tensor "
                             f"[layers, num_pages, {n}]")
        t = self.page_table
        # (rows further apart than they are long would lend the calls the entries between them:
        # the stride is all they know of a row's length)
        if (t.dtype != torch.int32 or t.device != p.device or t.dim() != 2 or t.shape[0] < 1
                or t.shape[1] < 1 or not t.is_contiguous()):
            raise ValueError("page_table must be a contiguous int32 device tensor [requests, pages]")
        # (past these every call, or fork and compact, would refuse: spec_kv_* take no more)
        if t.shape[0] > 1024 or p.shape[1] > 1 << 24 or p.shape[0] > 65535:
            raise ValueError("a cache holds at most 1024 requests, 2^24 pages and 65535 layers")
        _check_vec(self.seq_lens, "seq_lens", torch.int32, t.shape[0])
        _check_vec(self.ref_counts, "ref_counts", torch.int32, p.shape[1])
        if self.seq_lens.device != p.device or self.ref_counts.device != p.device:
            raise ValueError("seq_lens and ref_counts must be on the pages' device")
        # sizes the calls pass on every time
        object.__setattr__(self, "device", p.device)
        object.__setattr__(self, "layers", p.shape[0])
        object.__setattr__(self, "num_pages", p.shape[1])
        object.__setattr__(self, "page_bytes", n)
        object.__setattr__(self, "layer_bytes", p.stride(0) if p.shape[0] > 1 else p.shape[1] * n)
        object.__setattr__(self, "requests", t.shape[0])
        object.__setattr__(self, "ld_table", t.shape[1])

    @classmethod
    def create(cls, *, layers: int, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
               requests: int, max_context: int, device) -> "KVCache":
        """An empty cache: every page free, every request of length 0.
        At most 1,024 requests."""
        n = kv_page_bytes(kv_heads, head_dim, page_size)
        if n == 0:
            raise ValueError("KVCache: head_dim is 64, 128 or 256, page_size 16, 32, 64, 128 or 256")
        width = -(-int(max_context) // page_size)
        return cls(pages=torch.zeros(layers, num_pages, n, dtype=torch.uint8, device=device),
                   page_table=torch.full((requests, width), -1, dtype=torch.int32, device=device),
                   seq_lens=torch.zeros(requests, dtype=torch.int32, device=device),
                   ref_counts=torch.zeros(num_pages, dtype=torch.int32, device=device),
                   page_size=page_size, kv_heads=kv_heads, head_dim=head_dim)


def _kv_workspace(device: torch.device, nbytes: int,
                  given: torch.Tensor | None = None) -> torch.Tensor:
    """The caller's workspace, or scratch kept per (device, current stream): calls on
    one stream are ordered, so they share one.  While a graph is captured the
    call gets memory of the graph's own, so two graphs never share any.  An
    outgrown buffer goes back to torch's allocator, which reuses it on its own
    stream only, behind the work that still reads it."""
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        return given
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    key = (device.index, torch._C._cuda_getCurrentRawStream(device.index))
    ws = _kv_ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _kv_ws_cache[key] = ws
    return ws


class _on:
    """A call's launches: on the cache's device, and not between those of another
    thread's call on the same stream (a call is several launches that hand over in the
    stream's workspace)."""
    __slots__ = ("device", "guard", "lock")

    def __init__(self, device):
        self.device, self.guard = device, None

    def __enter__(self):
        index = self.device.index
        stream = torch._C._cuda_getCurrentRawStream(index)
        self.lock = _kv_locks.get((index, stream))
        if self.lock is None:
            self.lock = _kv_locks.setdefault((index, stream), threading.RLock())
        self.lock.acquire()
        if torch.cuda.current_device() != index:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        self.lock.release()


def _check_ints(t: torch.Tensor | None, name: str, device, n: int) -> None:
    if t is not None and (t.dtype != torch.int32 or t.device != device or not t.is_contiguous()
                          or t.numel() < n):
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} elements on "
                         "the cache's device")


def _kv_batch(cache: KVCache, cu_seqlens: torch.Tensor) -> int:
    batch = cu_seqlens.numel() - 1
    _check_ints(cu_seqlens, "cu_seqlens", cache.device, 2)
    if batch > cache.requests:
        raise ValueError(f"{batch} requests, but the page table has {cache.requests}")
    return batch


def _heads_of(t: torch.Tensor, name: str, cache: KVCache, dtype) -> tuple:
    """(rows, heads, elements from row to row) of a [rows, heads, head_dim] argument."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, heads, {cache.head_dim}]")
    rows, heads, dim = t.shape
    s0, s1, s2 = t.stride()
    if (dim != cache.head_dim or s2 != 1 or heads > 1 and s1 != dim or t.device != cache.device
            or t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} [rows, heads, {cache.head_dim}] on the cache's "
                         "device, heads side by side")
    # (a single row has no stride of its own)
    return rows, heads, s0 if rows > 1 else heads * dim


def _out_like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def kv_append(cache: KVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
              cu_seqlens: torch.Tensor, context_lens: torch.Tensor, *, layer: int = 0,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
              eps: float = 1e-6, cos_sin: torch.Tensor | None = None, interleaved: bool = False,
              out: torch.Tensor | None = None, want_values: bool = False,
              position_offsets: torch.Tensor | None = None):
    """spec_kv_append: head norms, rotation and the 4-bit cache write of the
    call's rows in one pass.

    q [rows, heads, D], k and v [rows, kv_heads, D] (float32 or bfloat16, views
    of one fused projection are fine); q_weight, k_weight float32 [D] or None;
    cos_sin float32 [positions, rot_dim], cos first, or None; `out` may be q.
    position_offsets (int32 [B], kv_evict's `evicted`): how far a request's positions are ahead
    of its slots, for the angles.

    Returns (q_out, status[B]), and with want_values (q_out, status, k_values,
    v_values): the values the cache now stands for.  Rows that are not processed (of no
    request, or without a position) stay as `out` holds them, undefined without `out`."""
    batch = _kv_batch(cache, cu_seqlens)
    code = _dtype_code(q)
    rows, heads, ld_q = _heads_of(q, "q", cache, q.dtype)
    k_rows, k_heads, ld_k = _heads_of(k, "k", cache, q.dtype)
    v_rows, v_heads, ld_v = _heads_of(v, "v", cache, q.dtype)
    if k_rows != rows or v_rows != rows or k_heads != cache.kv_heads or v_heads != cache.kv_heads:
        raise ValueError(f"k and v must be [{rows}, {cache.kv_heads}, {cache.head_dim}]")
    _check_ints(context_lens, "context_lens", cache.device, batch)
    _check_ints(position_offsets, "position_offsets", cache.device, batch)
    rot = positions = 0
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight"), (cos_sin, "cos_sin")):
        if t is not None and (t.dtype != torch.float32 or t.device != cache.device
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor on the cache's device")
    if (q_weight is not None and q_weight.numel() != cache.head_dim
            or k_weight is not None and k_weight.numel() != cache.head_dim):
        raise ValueError(f"the norms' weights must have {cache.head_dim} elements")
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [positions, rot_dim]")
        positions, rot = cos_sin.shape
    if not 0 <= layer < cache.layers:
        raise ValueError(f"layer {layer} of {cache.layers}")
    if out is None:
        out = _out_like(q)
        ld_out = heads * cache.head_dim
    else:
        o_rows, o_heads, ld_out = _heads_of(out, "out", cache, q.dtype)
        if o_rows != rows or o_heads != heads:
            raise ValueError("out must match q's shape")
    status = context_lens.new_empty(batch)
    k_values, v_values = (_out_like(k), _out_like(v)) if want_values else (None, None)
    with _on(cache.device) as stream:
        _raise(lib().spec_kv_append_at(
            q.data_ptr(), ld_q, k.data_ptr(), ld_k, v.data_ptr(), ld_v, code, _ptr(q_weight),
            _ptr(k_weight), eps, _ptr(cos_sin), positions, rot, interleaved, cu_seqlens.data_ptr(),
            context_lens.data_ptr(), _ptr(position_offsets), batch, rows, heads, cache.kv_heads,
            cache.head_dim, cache.pages.data_ptr() + layer * cache.layer_bytes, cache.num_pages,
            cache.page_size, cache.page_table.data_ptr(), cache.ld_table, out.data_ptr(), ld_out,
            _ptr(k_values), _ptr(v_values), status.data_ptr(), stream))
    return (out, status, k_values, v_values) if want_values else (out, status)


def kv_attention(cache: KVCache, q: torch.Tensor, cu_seqlens: torch.Tensor,
                 context_lens: torch.Tensor, *, max_k: int, max_context: int, layer: int = 0,
                 scale: float | None = None, window: int = 0, sinks: int = 0,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """spec_kv_attention: attention of the k+1 verify rows of each request over
    the cache (k = 0: decode).  scale defaults to head_dim ** -0.5.  Returns
    (out [rows, heads, D], status[B]).

    Rows of no request, and of requests with more than max_k + 1 rows, stay as `out` holds
    them (undefined without `out`).  Without `workspace` the scratch of the largest call
    so far stays with the stream; spec_kv_attention_workspace_bytes says how large."""
    batch = _kv_batch(cache, cu_seqlens)
    code = _dtype_code(q)
    rows, heads, ld_q = _heads_of(q, "q", cache, q.dtype)
    _check_ints(context_lens, "context_lens", cache.device, batch)
    if not 0 <= layer < cache.layers:
        raise ValueError(f"layer {layer} of {cache.layers}")
    if out is None:
        out = _out_like(q)
        ld_out = heads * cache.head_dim
    else:
        o_rows, o_heads, ld_out = _heads_of(out, "out", cache, q.dtype)
        if o_rows != rows or o_heads != heads:
            raise ValueError("out must match q's shape")
    # (ctypes would take the low 32 bits of a larger number)
    if not (0 <= max_k <= MAX_K and 1 <= max_context <= 1 << 30 and 0 <= window <= 1 << 30
            and 0 <= sinks <= 1 << 30):
        raise ValueError(f"max_k is at most {MAX_K}, max_context, window and sinks at most 2^30")
    status = context_lens.new_empty(batch)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    L = lib()
    need = L.spec_kv_attention_workspace_bytes(code, batch, max_k, heads, cache.kv_heads,
                                               cache.head_dim, max_context, window, sinks)
    if need == 0:
        raise ValueError("invalid sizes for spec_kv_attention")
    with _on(cache.device) as stream:
        ws = _kv_workspace(cache.device, need, workspace)
        _raise(L.spec_kv_attention(
            q.data_ptr(), ld_q, code, cu_seqlens.data_ptr(), context_lens.data_ptr(), batch, rows,
            max_k, heads, cache.kv_heads, cache.head_dim,
            cache.pages.data_ptr() + layer * cache.layer_bytes, cache.num_pages, cache.page_size,
            cache.page_table.data_ptr(), cache.ld_table, max_context, scale, window, sinks,
            out.data_ptr(), ld_out, status.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size(), stream))
    return out, status


def kv_prompt_attention(cache: KVCache, q: torch.Tensor, cu_seqlens: torch.Tensor,
                        context_lens: torch.Tensor, *, max_context: int, total_context: int,
                        layer: int = 0, scale: float | None = None, window: int = 0,
                        sinks: int = 0, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None):
    """spec_kv_prompt_attention: attention of whole prompts over the cache, any number of
    rows per request (append them first).  max_context bounds a request's context plus
    rows, total_context their sum over the requests.  scale defaults to head_dim ** -0.5.
    Returns (out [rows, heads, D], status[B]).

    Rows of no request stay as `out` holds them (undefined without `out`); `out` has no element
    in common with q (columns of one wider tensor are fine).  Without
    `workspace` the scratch of the largest call so far stays with the stream: the requests'
    cache in bf16 for the most part (spec_kv_prompt_workspace_bytes)."""
    batch = _kv_batch(cache, cu_seqlens)
    code = _dtype_code(q)
    rows, heads, ld_q = _heads_of(q, "q", cache, q.dtype)
    _check_ints(context_lens, "context_lens", cache.device, batch)
    if not 0 <= layer < cache.layers:
        raise ValueError(f"layer {layer} of {cache.layers}")
    if out is None:
        out = _out_like(q)
        ld_out = heads * cache.head_dim
    else:
        o_rows, o_heads, ld_out = _heads_of(out, "out", cache, q.dtype)
        if o_rows != rows or o_heads != heads:
            raise ValueError("out must match q's shape")
    # (ctypes would take the low bits of a larger number)
    if not (1 <= max_context <= 1 << 30 and 1 <= total_context <= 1 << 30 and rows < 1 << 31
            and 0 <= window <= 1 << 30 and 0 <= sinks <= 1 << 30):
        raise ValueError("max_context, total_context, window and sinks are at most 2^30")
    status = context_lens.new_empty(batch)
    scale = cache.head_dim ** -0.5 if scale is None else scale
    L = lib()
    need = L.spec_kv_prompt_workspace_bytes(code, batch, rows, heads, cache.kv_heads, cache.head_dim,
                                            max_context, total_context, window, sinks)
    if need == 0:
        raise ValueError("invalid sizes for spec_kv_prompt_attention")
    with _on(cache.device) as stream:
        ws = _kv_workspace(cache.device, need, workspace)
        _raise(L.spec_kv_prompt_attention(
            q.data_ptr(), ld_q, code, cu_seqlens.data_ptr(), context_lens.data_ptr(), batch, rows,
            heads, cache.kv_heads, cache.head_dim, cache.pages.data_ptr() + layer * cache.layer_bytes,
            cache.num_pages, cache.page_size, cache.page_table.data_ptr(), cache.ld_table,
            max_context, total_context, scale, window, sinks, out.data_ptr(), ld_out,
            status.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), stream))
    return out, status


def kv_attention_weights(cache: KVCache, q: torch.Tensor, cu_seqlens: torch.Tensor,
                         context_lens: torch.Tensor, *, max_k: int, max_context: int,
                         weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         row_counts: torch.Tensor | None = None, layer: int = 0,
                         scale: float | None = None, window: int = 0, sinks: int = 0,
                         workspace: torch.Tensor | None = None):
    """spec_kv_attention_weights: the attention weight that cached positions get from the rows
    q (as kv_append turned them) of each request, summed over its first row_counts[b] rows
    (None: all) and the query heads of each KV head, on top of `weights` (None: zeros).  After a
    verify and its drain, row_counts is accepted + 1, and the call goes before kv_release: all
    rows need their pages, counted or not.

    weights, out  float32 [B, kv_heads, L], L >= max_context: one layer's.  `out` defaults to
    `weights` itself, or to new memory.  Only positions below context_lens[b] + rows are written
    (new memory is 0 behind them).  Returns (out, status[B])."""
    batch = _kv_batch(cache, cu_seqlens)
    code = _dtype_code(q)
    rows, heads, ld_q = _heads_of(q, "q", cache, q.dtype)
    _check_ints(context_lens, "context_lens", cache.device, batch)
    _check_ints(row_counts, "row_counts", cache.device, batch)
    if not 0 <= layer < cache.layers:
        raise ValueError(f"layer {layer} of {cache.layers}")
    # (ctypes would take the low 32 bits of a larger number)
    if not (0 <= max_k <= MAX_K and 1 <= max_context <= 1 << 30 and 0 <= window <= 1 << 30
            and 0 <= sinks <= 1 << 30):
        raise ValueError(f"max_k is at most {MAX_K}, max_context, window and sinks at most 2^30")
    scale = cache.head_dim ** -0.5 if scale is None else scale
    L = lib()
    need = L.spec_kv_weights_workspace_bytes(code, batch, max_k, heads, cache.kv_heads,
                                             cache.head_dim, max_context, window, sinks)
    if need == 0:
        raise ValueError("invalid sizes for spec_kv_attention_weights")
    if out is None:
        out = weights if weights is not None else torch.zeros(
            batch, cache.kv_heads, max_context, dtype=torch.float32, device=cache.device)
    for t, name in ((out, "out"), (weights, "weights")):
        if t is not None and (t.dtype != torch.float32 or t.device != cache.device
                              or not t.is_contiguous() or t.dim() != 3 or t.shape[0] < batch
                              or t.shape[1] != cache.kv_heads or t.shape[2] < max_context
                              or t.shape[2] != out.shape[2]):
            raise ValueError(f"{name} must be a contiguous float32 tensor [{batch}, {cache.kv_heads}, "
                             f"at least {max_context}] on the cache's device")
    status = context_lens.new_empty(batch)
    with _on(cache.device) as stream:
        ws = _kv_workspace(cache.device, need, workspace)
        _raise(L.spec_kv_attention_weights(
            q.data_ptr(), ld_q, code, cu_seqlens.data_ptr(), context_lens.data_ptr(),
            _ptr(row_counts), batch, rows, max_k, heads, cache.kv_heads, cache.head_dim,
            cache.pages.data_ptr() + layer * cache.layer_bytes, cache.num_pages, cache.page_size,
            cache.page_table.data_ptr(), cache.ld_table, max_context, scale, window, sinks,
            _ptr(weights), out.data_ptr(), out.shape[2], status.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size(), stream))
    return out, status


def kv_evict(cache: KVCache, weights: torch.Tensor, budgets: torch.Tensor, *, sinks: int = 0,
             recent: int = 0, evicted: torch.Tensor | None = None):
    """spec_kv_evict: requests longer than budgets[b] (int32 [B], 0: no budget) keep that many
    positions: the first `sinks`, the last `recent`, and those of the largest weights between
    them, per layer and KV head.  What stays moves to the front, pages behind it are free.

    weights  float32 [layers, B, kv_heads, L], moved along; evicted int32 [B] or None, counted
    up by the positions that left (kv_append's position_offsets).  No other call changes them:
    set evicted[b] to 0 when slot b takes a new sequence, and after a kv_fork of an evicted
    request copy evicted[src] and weights[:, src] to dst.  Returns status[B]."""
    batch = budgets.numel()
    _check_ints(budgets, "budgets", cache.device, 1)
    _check_ints(evicted, "evicted", cache.device, batch)
    if batch > cache.requests:
        raise ValueError(f"{batch} requests, but the page table has {cache.requests}")
    if (weights.dtype != torch.float32 or weights.device != cache.device or weights.dim() != 4
            or not weights.is_contiguous()
            or weights.shape[:3] != (cache.layers, batch, cache.kv_heads)):
        raise ValueError(f"weights must be a contiguous float32 tensor [{cache.layers}, {batch}, "
                         f"{cache.kv_heads}, positions] on the cache's device")
    # (ctypes would take the low 32 bits of a larger number)
    if not (0 <= sinks <= 1 << 30 and 0 <= recent <= 1 << 30):
        raise ValueError("sinks and recent are at most 2^30")
    status = budgets.new_empty(batch)
    with _on(cache.device) as stream:
        _raise(lib().spec_kv_evict(
            budgets.data_ptr(), batch, sinks, recent, weights.data_ptr(), weights.shape[3],
            cache.kv_heads, cache.head_dim, cache.page_size, cache.seq_lens.data_ptr(),
            cache.page_table.data_ptr(), cache.ld_table, cache.ref_counts.data_ptr(),
            cache.num_pages, cache.pages.data_ptr(), cache.layers, cache.layer_bytes,
            _ptr(evicted), status.data_ptr(), stream))
    return status


def _pages_workspace(cache: KVCache, seqs: int, workspace):
    need = lib().spec_kv_pages_workspace_bytes(seqs, cache.num_pages)
    if need == 0:
        raise ValueError("invalid sizes: at most 1024 requests and 2^24 pages")
    return _kv_workspace(cache.device, need, workspace)


def kv_reserve(cache: KVCache, cu_seqlens: torch.Tensor, *, workspace: torch.Tensor | None = None):
    """spec_kv_reserve: pages for the rows of a call (shared last pages are
    copied).  Returns (context_lens[B], status[B])."""
    batch = _kv_batch(cache, cu_seqlens)
    context, status = cu_seqlens.new_empty(batch), cu_seqlens.new_empty(batch)
    with _on(cache.device) as stream:
        ws = _pages_workspace(cache, batch, workspace)
        _raise(lib().spec_kv_reserve(
            cu_seqlens.data_ptr(), batch, cache.page_size, cache.seq_lens.data_ptr(),
            cache.page_table.data_ptr(), cache.ld_table, cache.ref_counts.data_ptr(),
            cache.num_pages, cache.pages.data_ptr(), cache.page_bytes, cache.layers,
            cache.layer_bytes, context.data_ptr(), status.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size(), stream))
    return context, status


def kv_release(cache: KVCache, rollback: torch.Tensor, context_lens: torch.Tensor | None = None):
    """spec_kv_release: gives positions back (rollback as drain returns it, with
    the context_lens of the reserve before it).  Returns status[B]."""
    batch = rollback.numel()
    _check_ints(rollback, "rollback", cache.device, 1)
    _check_ints(context_lens, "context_lens", cache.device, batch)
    if batch > cache.requests:
        raise ValueError(f"{batch} requests, but the page table has {cache.requests}")
    status = rollback.new_empty(batch)
    with _on(cache.device) as stream:
        _raise(lib().spec_kv_release(
            rollback.data_ptr(), _ptr(context_lens), batch, cache.page_size,
            cache.seq_lens.data_ptr(), cache.page_table.data_ptr(), cache.ld_table,
            cache.ref_counts.data_ptr(), cache.num_pages, status.data_ptr(), stream))
    return status


def kv_fork(cache: KVCache, src: torch.Tensor, dst: torch.Tensor,
            lens: torch.Tensor | None = None):
    """spec_kv_fork: row dst[i] starts as the first lens[i] positions (None: all)
    of row src[i], sharing its pages.  Returns status[pairs]."""
    pairs = src.numel()
    _check_ints(src, "src", cache.device, 1)
    _check_ints(dst, "dst", cache.device, pairs)
    _check_ints(lens, "lens", cache.device, pairs)
    status = src.new_empty(pairs)
    with _on(cache.device) as stream:
        _raise(lib().spec_kv_fork(
            src.data_ptr(), dst.data_ptr(), _ptr(lens), pairs, cache.requests, cache.page_size,
            cache.seq_lens.data_ptr(), cache.page_table.data_ptr(), cache.ld_table,
            cache.ref_counts.data_ptr(), cache.num_pages, status.data_ptr(), stream))
    return status


def kv_compact(cache: KVCache, *, workspace: torch.Tensor | None = None):
    """spec_kv_compact: moves the pages in use to the front of the pool.
    Returns live (int32 [1]): pages live .. num_pages-1 are free afterwards."""
    live = cache.seq_lens.new_empty(1)
    with _on(cache.device) as stream:
        ws = _pages_workspace(cache, cache.requests, workspace)
        _raise(lib().spec_kv_compact(
            cache.requests, cache.page_size, cache.seq_lens.data_ptr(),
            cache.page_table.data_ptr(), cache.ld_table, cache.ref_counts.data_ptr(),
            cache.num_pages, cache.pages.data_ptr(), cache.page_bytes, cache.layers,
            cache.layer_bytes, live.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
            stream))
    return live


def workload_tensors(w, device) -> dict:
    """Device tensors of a synthetic workload (see synth.Workload)."""
    def rows(a, dt):
        if a is None:
            return None
        if dt == SV_BF16:
            return torch.from_numpy(a.view("int16")).to(device).view(torch.bfloat16)
        return torch.from_numpy(a).to(device)

    def vec(a, dtype):
        return None if a is None else torch.from_numpy(a).to(device=device, dtype=dtype)

    return dict(
        target=rows(w.target, w.target_dtype),
        draft=rows(w.draft, w.draft_dtype),
        draft_kind=vec(w.draft_kind, torch.int32),
        cu_seqlens=vec(w.cu_seqlens, torch.int32),
        draft_tokens=vec(w.draft_tokens, torch.int32),
        uniforms=vec(w.uniforms, torch.float32),
        temperature=vec(w.temperature, torch.float32),
        top_k=vec(w.top_k, torch.int32),
        top_p=vec(w.top_p, torch.float32),
    )
