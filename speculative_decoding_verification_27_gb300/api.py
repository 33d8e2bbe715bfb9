"""Python binding of libspecverify.so, with the C ABI's names.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors must be CUDA tensors; there is no CPU path, and a missing library is an
error, not a fallback. PyTorch supplies device memory and the current stream.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import struct
import threading
from typing import NamedTuple, Optional

import torch

from .build import LIB_PATH, ROOT

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_CUDA, SV_ERR_TIMEOUT, SV_ERR_UNIMPLEMENTED, SV_ERR_DATA = range(6)
SV_FP32, SV_BF16 = 0, 1
SV_MODE_SAMPLE, SV_MODE_GREEDY = 0, 1
SV_DATA_BAD_OFFSETS = 0x1
SV_DATA_BAD_TOKEN = 0x2
SV_DATA_EMPTY_ROW = 0x4
SV_DATA_BAD_MODE = 0x8
SV_DATA_DEGENERATE_RESIDUAL = 0x10
SV_DEV_COPY_TIMEOUT = 0x20
SV_DATA_BAD_LOGIT = 0x40
SV_DATA_BAD_PAGE = 0x80
SV_DATA_NO_PAGES = 0x100
SV_DATA_BAD_SEQ = 0x200
SV_ONEHOT_ROW_BYTES_DEFAULT = 128 * 1024  # sv_set_onehot_row_bytes' initial limit

HEADER = os.path.join(ROOT, "include", "spec_verify.h")

_lib = None


class SpecVerifyError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load the CUDA library (built in-tree by build.build_library())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it first "
            "(speculative_decoding_verification_27_gb300.build.build_library())")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.spec_verify_workspace_size.argtypes = [i32, i32, i32]
    lib.spec_verify_workspace_size.restype = sz
    lib.spec_verify.argtypes = [P, P, ctypes.c_int, i32, i32, P, P, P, P, f32, P, P, P, P, sz, P]
    lib.spec_verify.restype = ctypes.c_int
    lib.spec_verify_greedy.argtypes = [P, ctypes.c_int, i32, i32, P, P, P, P, P, sz, P]
    lib.spec_verify_greedy.restype = ctypes.c_int
    lib.ngram_propose.argtypes = [P, i64, P, i32, i32, i32, i32, P, P, P, P]
    lib.ngram_propose.restype = ctypes.c_int
    lib.sv_pack_drafts.argtypes = [P, P, i32, i32, P, P, P]
    lib.sv_pack_drafts.restype = ctypes.c_int
    lib.sv_token_logprobs.argtypes = [P, ctypes.c_int, i32, i64, i32, P, i32, P, P, f32, i32, P, P, P, P, P, P, P]
    lib.sv_token_logprobs.restype = ctypes.c_int
    lib.sv_cache_fork.argtypes = [P, P, i32, P, P, P, P]
    lib.sv_cache_free.argtypes = [P, P, i32, P, P, P]
    lib.sv_cache_reserve_workspace_size.argtypes = [i32]
    lib.sv_cache_reserve_workspace_size.restype = sz
    lib.sv_cache_reserve.argtypes = [P, P, i32, P, P, P, P, sz, P, P]
    lib.sv_cache_append.argtypes = [P, i32, i32, P, P, i64, i64, i32, P, i32, P, P, P, P]
    lib.sv_cache_commit.argtypes = [P, P, i32, P, P, P, P, P, P]
    lib.sv_window_attention_workspace_size.argtypes = [P, i32, i32]
    lib.sv_window_attention_workspace_size.restype = sz
    lib.sv_window_attention.argtypes = [P, i64, i32, i32, P, i32, P, i32, P, P, f32, P, i64, P, P, sz, P, P]
    for name in ("sv_cache_fork", "sv_cache_free", "sv_cache_reserve", "sv_cache_append", "sv_cache_commit",
                 "sv_window_attention"):
        getattr(lib, name).restype = ctypes.c_int
    lib.sv_check_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
    lib.sv_check_status.restype = ctypes.c_int
    lib.sv_status_string.argtypes = [ctypes.c_int]
    lib.sv_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def header_functions() -> list:
    """Names of the functions declared in include/spec_verify.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(\w+)\s*\(", text)) - {"defined", "if"})


def status_string(status: int) -> str:
    return load().sv_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != SV_OK:
        raise SpecVerifyError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("spec_verify tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("spec_verify tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SV_FP32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise ValueError("logits must be float32 or bfloat16")


def spec_verify_workspace_size(B: int, R_t: int, V: int) -> int:
    return int(load().spec_verify_workspace_size(int(B), int(R_t), int(V)))


def new_workspace(B: int, R_t: int, V: int, device="cuda") -> torch.Tensor:
    """Zero-filled workspace (the library leaves it zeroed after each call)."""
    return torch.zeros(spec_verify_workspace_size(B, R_t, V), dtype=torch.uint8, device=device)


# Default workspaces, one per (device, stream, entry point): calls on one
# stream run in order and the library leaves its counters at zero after each
# call, so one block serves every call whose workspace layout is the same.
# The layout follows (B, V) for spec_verify / spec_verify_greedy and (B, R_t,
# V) for spec_verify_filtered (its thresholds come first); when it changes,
# or the block is too small, the block is cleared (or grown to the next power
# of two and cleared) before the call. Calls with an unchanged layout clear
# nothing and allocate nothing.
_default_ws: dict = {}
default_workspace_clears = 0   # blocks allocated or cleared so far (each one fill launch)


def default_workspace(nbytes: int, device, stream=None, layout=None) -> torch.Tensor:
    """The cached workspace of `stream` (current stream if None) on `device`
    for calls with workspace layout `layout`, at least `nbytes` long. Calls
    that pass no workspace use it; pass it to sv_check_status to read the
    data-error bits of those calls."""
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    s = torch.cuda.current_stream(idx) if stream is None else stream
    global default_workspace_clears
    key = (idx, s.cuda_stream, layout[0] if layout else None)
    ent = _default_ws.get(key)
    if ent is None or ent[0].numel() < nbytes:
        default_workspace_clears += 1
        size = 1 << max(12, (int(nbytes) - 1).bit_length())
        with torch.cuda.stream(s):
            ent = [torch.zeros(size, dtype=torch.uint8, device=torch.device("cuda", idx)), layout]
        _default_ws[key] = ent
    elif ent[1] != layout:
        default_workspace_clears += 1
        with torch.cuda.stream(s):
            ent[0].zero_()
        ent[1] = layout
    return ent[0]


def reset_default_workspaces() -> None:
    """Drops the cached workspaces (needed only after SV_DEV_COPY_TIMEOUT,
    which leaves a workspace's counters set)."""
    _default_ws.clear()


def spec_verify(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                cu_draft: torch.Tensor, uniforms: torch.Tensor, temperature: float,
                mode: Optional[torch.Tensor] = None, *, out_tokens=None, out_len=None,
                out_probs=None, want_probs: bool = True, workspace=None, stream=None):
    """Lossless verify-and-commit. Returns (out_tokens, out_len, out_probs)."""
    lib = load()
    B = cu_draft.shape[0] - 1
    R_t = target.shape[0]
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.full((R_t,), -1, dtype=torch.int32, device=dev)
    if out_len is None:
        out_len = torch.zeros(B, dtype=torch.int32, device=dev)
    if out_probs is None and want_probs:
        out_probs = torch.empty((R_t, 2), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = default_workspace(spec_verify_workspace_size(B, R_t, target.shape[1]), dev, stream,
                                      ("verify", B, target.shape[1]))
    st = lib.spec_verify(_ptr(target), _ptr(draft), _dtype(target), int(target.shape[1]), int(B),
                         _ptr(draft_tokens), _ptr(cu_draft), _ptr(mode), _ptr(uniforms),
                         float(temperature), _ptr(out_tokens), _ptr(out_len), _ptr(out_probs),
                         _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spec_verify", st)
    return out_tokens, out_len, out_probs


SV_NOALLOC_SCRATCH_BYTES = 4 << 20


def _noalloc_fn():
    lib = load()
    fn = lib.spec_verify_noalloc
    P = ctypes.c_void_p
    fn.argtypes = [P, P, ctypes.c_int, ctypes.c_int32, ctypes.c_int32, P, P, P, P, ctypes.c_float,
                   P, P, P, P, P]
    fn.restype = ctypes.c_int
    return fn


def spec_verify_noalloc(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                        cu_draft: torch.Tensor, uniforms: torch.Tensor, temperature: float,
                        mode: Optional[torch.Tensor], out_tokens: torch.Tensor, out_len: torch.Tensor,
                        out_probs: Optional[torch.Tensor] = None,
                        status_out: Optional[torch.Tensor] = None, stream=None):
    """spec_verify on the library's fixed scratch block: no workspace argument
    and no allocation. Outputs are the caller's. Calls on one device must not
    overlap.

    status_out: a one-element int32 CUDA tensor that receives the call's
    SV_DATA_* / SV_DEV_* bits (0 = clean). With None the bits are dropped:
    a call with bad device data (offsets, tokens) then raises nothing and its
    outputs are unspecified, and the block's own status word cannot be read
    afterwards. Pass one whenever the inputs are not known to be valid."""
    B = cu_draft.shape[0] - 1
    st = _noalloc_fn()(_ptr(target), _ptr(draft), _dtype(target), int(target.shape[1]), int(B),
                       _ptr(draft_tokens), _ptr(cu_draft), _ptr(mode), _ptr(uniforms),
                       float(temperature), _ptr(out_tokens), _ptr(out_len), _ptr(out_probs),
                       _ptr(status_out), _stream(stream))
    _check("spec_verify_noalloc", st)
    return out_tokens, out_len, out_probs


def spec_verify_greedy(target: torch.Tensor, draft_tokens: torch.Tensor, cu_draft: torch.Tensor, *,
                       out_tokens=None, out_len=None, workspace=None, stream=None):
    """Strict (greedy) verify-and-commit. Returns (out_tokens, out_len)."""
    lib = load()
    B = cu_draft.shape[0] - 1
    R_t = target.shape[0]
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.full((R_t,), -1, dtype=torch.int32, device=dev)
    if out_len is None:
        out_len = torch.zeros(B, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = default_workspace(spec_verify_workspace_size(B, R_t, target.shape[1]), dev, stream,
                                      ("verify", B, target.shape[1]))
    st = lib.spec_verify_greedy(_ptr(target), _dtype(target), int(target.shape[1]), int(B),
                                _ptr(draft_tokens), _ptr(cu_draft), _ptr(out_tokens), _ptr(out_len),
                                _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spec_verify_greedy", st)
    return out_tokens, out_len


def ngram_propose(histories: torch.Tensor, hist_len: torch.Tensor, min_n: int, max_n: int,
                  max_tokens: int, *, out_tokens=None, out_count=None, out_n=None, stream=None):
    """N-gram / prompt-lookup proposer. Returns (out_tokens [B, max_tokens], out_count, out_n)."""
    lib = load()
    B, stride = histories.shape
    dev = histories.device
    if out_tokens is None:
        out_tokens = torch.empty((B, max_tokens), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty(B, dtype=torch.int32, device=dev)
    if out_n is None:
        out_n = torch.empty(B, dtype=torch.int32, device=dev)
    st = lib.ngram_propose(_ptr(histories), int(stride), _ptr(hist_len), int(B), int(min_n),
                           int(max_n), int(max_tokens), _ptr(out_tokens), _ptr(out_count),
                           _ptr(out_n), _stream(stream))
    _check("ngram_propose", st)
    return out_tokens, out_count, out_n


SV_SUFFIX_MAX_OCC = 256


def suffix_propose(histories: torch.Tensor, hist_len: torch.Tensor, min_n: int, max_n: int,
                   max_tokens: int, min_share: float = 0.5, max_occ: int = SV_SUFFIX_MAX_OCC, *,
                   out_tokens=None, out_count=None, out_n=None, stream=None):
    """Frequency-ranked suffix proposer. Returns (out_tokens [B, max_tokens], out_count, out_n)."""
    lib = load()
    fn = lib.suffix_propose
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    fn.argtypes = [P, ctypes.c_int64, P, i32, i32, i32, i32, ctypes.c_float, i32, P, P, P, P]
    fn.restype = ctypes.c_int
    B, stride = histories.shape
    dev = histories.device
    if out_tokens is None:
        out_tokens = torch.empty((B, max_tokens), dtype=torch.int32, device=dev)
    if out_count is None:
        out_count = torch.empty(B, dtype=torch.int32, device=dev)
    if out_n is None:
        out_n = torch.empty(B, dtype=torch.int32, device=dev)
    st = fn(_ptr(histories), int(stride), _ptr(hist_len), int(B), int(min_n), int(max_n),
            int(max_tokens), float(min_share), int(max_occ), _ptr(out_tokens), _ptr(out_count),
            _ptr(out_n), _stream(stream))
    _check("suffix_propose", st)
    return out_tokens, out_count, out_n


def sv_pack_drafts(tokens: torch.Tensor, counts: torch.Tensor, max_tokens: int, *, cu_draft=None,
                   packed=None, stream=None):
    """(cu_draft [B+1], packed [B*max_tokens]) from padded proposals and their counts."""
    lib = load()
    B = counts.shape[0]
    dev = counts.device
    if cu_draft is None:
        cu_draft = torch.empty(B + 1, dtype=torch.int32, device=dev)
    if packed is None:
        packed = torch.empty(max(B * max_tokens, 1), dtype=torch.int32, device=dev)
    st = lib.sv_pack_drafts(_ptr(tokens), _ptr(counts), int(B), int(max_tokens), _ptr(cu_draft),
                            _ptr(packed), _stream(stream))
    _check("sv_pack_drafts", st)
    return cu_draft, packed


def sv_check_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronize, read and clear the device status word; returns the SV_DATA_* bits."""
    bits = ctypes.c_uint32(0)
    st = load().sv_check_status(_ptr(workspace), _stream(stream), ctypes.byref(bits))
    if st not in (SV_OK, SV_ERR_DATA, SV_ERR_TIMEOUT):
        raise SpecVerifyError("sv_check_status", st)
    return int(bits.value)


# ---------------------------------------------------------------------------
# Acceptance statistics and the draft-length controller
# ---------------------------------------------------------------------------
SV_METRICS_MAX_POS = 32
_METRIC_SCALARS = ("rounds", "rounds_with_draft", "drafted", "accepted", "committed")
_METRIC_WORDS = len(_METRIC_SCALARS) + 3 * SV_METRICS_MAX_POS


def new_metrics(device="cuda") -> torch.Tensor:
    """A zeroed sv_metrics block on the device (64-bit counters)."""
    return torch.zeros(_METRIC_WORDS, dtype=torch.int64, device=device)


def sv_accumulate_metrics(cu_draft: torch.Tensor, out_len: torch.Tensor, metrics: torch.Tensor,
                          stream=None) -> torch.Tensor:
    """Adds one verify call's rounds to `metrics` (see new_metrics)."""
    lib = load()
    fn = lib.sv_accumulate_metrics
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    if metrics.numel() != _METRIC_WORDS or metrics.dtype != torch.int64:
        raise ValueError("metrics must come from new_metrics()")
    _check("sv_accumulate_metrics", fn(_ptr(cu_draft), _ptr(out_len), int(out_len.numel()),
                                       _ptr(metrics), _stream(stream)))
    return metrics


def metrics_dict(metrics: torch.Tensor) -> dict:
    """The counters as a host dict (keys as in the header's sv_metrics)."""
    v = [int(x) for x in metrics.cpu().tolist()]
    d = dict(zip(_METRIC_SCALARS, v[:5]))
    P = SV_METRICS_MAX_POS
    d["offered"], d["reached"], d["accepted_at"] = v[5:5 + P], v[5 + P:5 + 2 * P], v[5 + 2 * P:5 + 3 * P]
    return d


class _Adapt(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("min_k", ctypes.c_int32), ("max_k", ctypes.c_int32),
                ("k", ctypes.c_int32), ("count", ctypes.c_int32), ("next", ctypes.c_int32),
                ("target", ctypes.c_double), ("ratio", ctypes.c_double * 1024)]


class AdaptiveDraftLength:
    """The library's sliding-window draft-length controller (host code)."""

    def __init__(self, window=100, min_k=1, max_k=10, target=0.7, initial_k=5):
        lib = load()
        lib.sv_adapt_init.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_double, ctypes.c_int32]
        lib.sv_adapt_init.restype = ctypes.c_int
        lib.sv_adapt_update.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32]
        lib.sv_adapt_update.restype = ctypes.c_int
        lib.sv_adapt_draft_length.argtypes = [ctypes.c_void_p]
        lib.sv_adapt_draft_length.restype = ctypes.c_int32
        self._lib = lib
        self._s = _Adapt()
        _check("sv_adapt_init", lib.sv_adapt_init(ctypes.byref(self._s), window, min_k, max_k,
                                                  float(target), initial_k))

    def update(self, draft_len: int, accepted_len: int) -> int:
        _check("sv_adapt_update", self._lib.sv_adapt_update(ctypes.byref(self._s), draft_len, accepted_len))
        return self.draft_length

    @property
    def draft_length(self) -> int:
        return int(self._lib.sv_adapt_draft_length(ctypes.byref(self._s)))


# ---------------------------------------------------------------------------
# Top-k / top-p filtered verify
# ---------------------------------------------------------------------------
def spec_verify_filtered_workspace_size(B: int, R_t: int, V: int) -> int:
    lib = load()
    lib.spec_verify_filtered_workspace_size.argtypes = [ctypes.c_int32] * 3
    lib.spec_verify_filtered_workspace_size.restype = ctypes.c_size_t
    return int(lib.spec_verify_filtered_workspace_size(int(B), int(R_t), int(V)))


def spec_verify_filtered(target: torch.Tensor, draft: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                         cu_draft: torch.Tensor, uniforms: torch.Tensor, temperature: float,
                         top_k: int = 0, top_p: float = 1.0, mode: Optional[torch.Tensor] = None, *,
                         out_tokens=None, out_len=None, out_probs=None, want_probs: bool = True,
                         workspace=None, stream=None):
    """Verify-and-commit on top-k / top-p filtered distributions.
    Returns (out_tokens, out_len, out_probs)."""
    lib = load()
    fn = lib.spec_verify_filtered
    P = ctypes.c_void_p
    fn.argtypes = [P, P, ctypes.c_int, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P, P,
                   ctypes.c_float, ctypes.c_int32, ctypes.c_float, P, P, P, P, ctypes.c_size_t, P]
    fn.restype = ctypes.c_int
    B = cu_draft.shape[0] - 1
    R_t = target.shape[0]
    V = target.shape[1]
    dev = target.device
    if out_tokens is None:
        out_tokens = torch.full((R_t,), -1, dtype=torch.int32, device=dev)
    if out_len is None:
        out_len = torch.zeros(B, dtype=torch.int32, device=dev)
    if out_probs is None and want_probs:
        out_probs = torch.empty((R_t, 2), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = default_workspace(spec_verify_filtered_workspace_size(B, R_t, V), dev, stream,
                                      ("filtered", B, R_t, V))
    st = fn(_ptr(target), _ptr(draft), _dtype(target), int(V), int(B), int(R_t), _ptr(draft_tokens),
            _ptr(cu_draft), _ptr(mode), _ptr(uniforms), float(temperature), int(top_k), float(top_p),
            _ptr(out_tokens), _ptr(out_len), _ptr(out_probs), _ptr(workspace), workspace.numel(),
            _stream(stream))
    _check("spec_verify_filtered", st)
    return out_tokens, out_len, out_probs


def sv_set_onehot_row_bytes(nbytes: int) -> int:
    """Largest row (V * element size, in bytes) that spec_verify runs with
    the one-CTA-per-row kernel for one-hot batches (0: never; negative: only
    read); returns the previous limit. Process-wide."""
    lib = load()
    lib.sv_set_onehot_row_bytes.argtypes = [ctypes.c_int32]
    lib.sv_set_onehot_row_bytes.restype = ctypes.c_int32
    return int(lib.sv_set_onehot_row_bytes(int(nbytes)))


def sv_set_cluster_rows(rows: int) -> int:
    """Largest workspace (in target rows) that spec_verify runs with the
    cluster kernel (0: never; negative: only read); returns the previous
    threshold. Process-wide."""
    lib = load()
    lib.sv_set_cluster_rows.argtypes = [ctypes.c_int32]
    lib.sv_set_cluster_rows.restype = ctypes.c_int32
    return int(lib.sv_set_cluster_rows(int(rows)))


SV_SELECT_UNIFORM, SV_SELECT_LONGEST_BIASED = 0, 1


def sv_select_candidates(cu_cand: torch.Tensor, out_len: torch.Tensor, policy: int,
                         u_select: Optional[torch.Tensor] = None, *, best=None, best_len=None,
                         stream=None):
    """Per request, the kept candidate under `policy` (SV_SELECT_UNIFORM needs
    one selection uniform per request in u_select; SV_SELECT_LONGEST_BIASED
    is not distribution-preserving). Returns (best, best_len)."""
    lib = load()
    fn = lib.sv_select_candidates
    P = ctypes.c_void_p
    fn.argtypes = [P, P, ctypes.c_int32, ctypes.c_int32, P, P, P, P]
    fn.restype = ctypes.c_int
    B = cu_cand.shape[0] - 1
    if best is None:
        best = torch.empty(B, dtype=torch.int32, device=cu_cand.device)
    if best_len is None:
        best_len = torch.empty(B, dtype=torch.int32, device=cu_cand.device)
    _check("sv_select_candidates", fn(_ptr(cu_cand), _ptr(out_len), int(B), int(policy), _ptr(u_select),
                                      _ptr(best), _ptr(best_len), _stream(stream)))
    return best, best_len


# ---------------------------------------------------------------------------
# Log probabilities of given tokens
# ---------------------------------------------------------------------------
SV_LOGPROBS_MAX_TOP = 32


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]       # [R] float32, ln p(token)
    rank: Optional[torch.Tensor]          # [R] int32, 1 = the largest logit
    entropy: Optional[torch.Tensor]       # [R] float32
    top_ids: Optional[torch.Tensor]       # [R, n_top] int32, -1 where fewer are left
    top_logprobs: Optional[torch.Tensor]  # [R, n_top] float32


def _raw_stream(device: int) -> int:
    """The current stream of a device as an address."""
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)  # the same without a Stream object


def _launch(name: str, t: torch.Tensor, stream, *args):
    """Calls the library on t's device and stream (the current one if None)."""
    fn = getattr(_lib or load(), name)
    device = t.get_device()
    s = _raw_stream(device) if stream is None else stream.cuda_stream
    if device == torch.cuda.current_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(device):
            st = fn(*args, s)
    if st:
        raise SpecVerifyError(name, st)


def _new(make, shape, dtype, like: torch.Tensor, stream):
    """An output tensor beside `like`, owned by the stream that writes it."""
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _vec(t: Optional[torch.Tensor], name: str, dtype, shape: tuple):
    """Address of a contiguous tensor of that type and shape (whose device _on_one_device looks at); None stays None."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_one_device(t: torch.Tensor, *others: Optional[torch.Tensor]):
    """The kernels run on t's device and read the addresses of all."""
    device = t.get_device()
    for x in others:
        if x is not None and x.get_device() != device:
            raise ValueError("the tensors of a call must lie on one CUDA device")


def sv_token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, cu_draft=None, out_len=None,
                      temperature: float = 1.0, n_top: int = 0, out_logprob=None, out_rank=None, out_entropy=None,
                      out_top_ids=None, out_top_logprobs=None, status=None, stream=None) -> TokenLogprobs:
    """Log probability, rank, entropy and top alternatives of every row, or,
    with the cu_draft and out_len of a verify call (and its out_tokens as
    `tokens`), of the committed rows only: the other rows of given outputs
    keep their values, those of outputs made here are zero. `logits` may have
    a row stride. `status`: a one-element int32 CUDA tensor that collects the
    data-error bits."""
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA matrix with contiguous rows")
    R, V = logits.shape
    ld = logits.stride(0) if R > 1 else max(V, 1)
    n_top = int(n_top)
    f32, i32 = torch.float32, torch.int32
    if (cu_draft is None) != (out_len is None):
        raise ValueError("cu_draft and out_len come together")
    B = 0 if out_len is None else out_len.shape[0]
    make = torch.empty if out_len is None else torch.zeros
    if tokens is not None and out_logprob is None:
        out_logprob = _new(make, R, f32, logits, stream)
    if tokens is not None and out_rank is None:
        out_rank = _new(make, R, i32, logits, stream)
    if out_entropy is None:
        out_entropy = _new(make, R, f32, logits, stream)
    if n_top > 0 and out_top_ids is None:
        out_top_ids = _new(make, (R, n_top), i32, logits, stream)
    if n_top > 0 and out_top_logprobs is None:
        out_top_logprobs = _new(make, (R, n_top), f32, logits, stream)
    rows, tops = (R,), (R, n_top)
    _on_one_device(logits, tokens, cu_draft, out_len, out_logprob, out_rank, out_entropy, out_top_ids, out_top_logprobs, status)
    _launch("sv_token_logprobs", logits, stream, logits.data_ptr(), _dtype(logits), V, ld, R,
            _vec(tokens, "tokens", i32, rows), B, _vec(cu_draft, "cu_draft", i32, (B + 1,)),
            _vec(out_len, "out_len", i32, (B,)), temperature, n_top, _vec(out_logprob, "out_logprob", f32, rows),
            _vec(out_rank, "out_rank", i32, rows), _vec(out_entropy, "out_entropy", f32, rows),
            _vec(out_top_ids, "out_top_ids", i32, tops), _vec(out_top_logprobs, "out_top_logprobs", f32, tops),
            _vec(status, "status", i32, (1,)))
    return TokenLogprobs(out_logprob, out_rank, out_entropy, out_top_ids, out_top_logprobs)


# ---------------------------------------------------------------------------
# The paged key-value cache around the verify step
# ---------------------------------------------------------------------------
SV_CACHE_MAX_SEQS = 16384


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n_layers", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_ref", ctypes.c_void_p),
                ("free_bits", ctypes.c_void_p)]


class _Sequences(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_pages", ctypes.c_int32),
                ("n", ctypes.c_int32), ("ctx_len", ctypes.c_void_p)]


_pack_sequences = struct.Struct("@PqiiP").pack  # _Sequences as bytes: the library reads it during the call only


def _steps(t: torch.Tensor) -> list:
    """The strides that are taken: a dimension of one element takes no step, and its stride may be anything."""
    return [s if m > 1 else 0 for s, m in zip(t.stride(), t.shape)]


def _heads_contiguous(t: torch.Tensor) -> bool:
    """Whether the last two dimensions, heads and their elements, lie together."""
    heads, D = t.shape[-2:]
    step, one = t.stride()[-2:]
    return one == 1 and (step == D or heads == 1)


class _Scratch:
    """Scratch of the calls on one stream, whose kernels run in order. A call
    of two launches hands its results over in the block, so no other thread's
    launch on the stream may come between them: the lock is held over the
    whole call (and may be taken again by a handler that interrupts it)."""
    __slots__ = ("lock", "block")

    def __init__(self):
        self.lock = threading.RLock()
        self.block = None


class KVCache:
    """The pages of a key-value cache: `k` and `v` are [n_layers, n_pages,
    page_size, n_kv_heads, head_dim] views with equal strides (any order of
    the first four dimensions in memory, the last contiguous). page_ref
    [n_pages] int32 counts a page's holders, free_bits [ceil(n_pages / 32)]
    int32 has a bit set per free page; without them the cache starts empty."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_ref=None, free_bits=None):
        if k.dim() != 5 or k.shape != v.shape or _steps(k) != _steps(v) or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must be [layers, pages, page_size, kv_heads, head_dim] with equal strides")
        if not k.is_cuda or (k.shape[4] > 1 and k.stride(4) != 1):
            raise ValueError("k and v must be CUDA tensors with a contiguous last dimension")
        if (page_ref is None) != (free_bits is None):
            raise ValueError("page_ref and free_bits come together")
        n, words = k.shape[1], -(-k.shape[1] // 32)
        if page_ref is None:
            page_ref = torch.zeros(n, dtype=torch.int32, device=k.device)
            free_bits = torch.full((words,), -1, dtype=torch.int32, device=k.device)
            if n % 32:
                free_bits[-1] = (1 << n % 32) - 1
        _on_one_device(k, page_ref, free_bits)
        self.k, self.v, self.page_ref, self.free_bits = k, v, page_ref, free_bits
        self.n_layers, self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = k.shape
        self._c = _Cache(k.data_ptr(), v.data_ptr(), _dtype(k), *k.shape, *_steps(k)[:4],
                         _vec(page_ref, "page_ref", torch.int32, (n,)), _vec(free_bits, "free_bits", torch.int32, (words,)))
        self._ref = ctypes.byref(self._c)
        self._attention_bytes = load().sv_window_attention_workspace_size(self._ref, self.n_kv_heads, 0)
        self._scratches: dict = {}

    def _scratch(self, stream) -> _Scratch:
        """What calls on `stream` share. A call that is being captured gets
        scratch of its graph's own."""
        device = self.k.get_device()
        if stream is not None:
            key = stream.cuda_stream
            with torch.cuda.stream(stream):
                capturing = torch.cuda.is_current_stream_capturing()
        else:
            key = _raw_stream(device)
            if device == torch.cuda.current_device():
                capturing = torch.cuda.is_current_stream_capturing()
            else:
                with torch.cuda.device(device):
                    capturing = torch.cuda.is_current_stream_capturing()
        if capturing:
            return _Scratch()
        return self._scratches.get(key) or self._scratches.setdefault(key, _Scratch())

    def _launch_with_scratch(self, nbytes: int, stream, call):
        """call(workspace) with at least nbytes of the stream's scratch."""
        scratch = self._scratch(stream)
        with scratch.lock:
            if scratch.block is None or scratch.block.numel() < nbytes:
                scratch.block = _new(torch.empty, nbytes, torch.uint8, self.k, stream)
            call(scratch.block)


def _seqs(page_table: torch.Tensor, ctx_len: torch.Tensor) -> bytes:
    n, width = page_table.shape
    stride, step = page_table.stride()
    if page_table.dtype != torch.int32 or (step != 1 and width > 1):
        raise ValueError("page_table must be an int32 matrix with contiguous rows")
    return _pack_sequences(page_table.data_ptr(), stride if n > 1 else max(width, 1), width, n,
                           _vec(ctx_len, "ctx_len", torch.int32, (n,)))


def _windows(n: int, cu_draft, cu_cand):
    """(n_cand, cu_draft, cu_cand) as the library takes them."""
    if cu_draft is None:
        if cu_cand is not None:
            raise ValueError("cu_cand needs cu_draft")
        return n, None, None
    n_cand = cu_draft.shape[0] - 1
    if cu_cand is None and n_cand != n:
        raise ValueError("cu_draft has an offset per sequence and one more")
    return n_cand, _vec(cu_draft, "cu_draft", torch.int32, (n_cand + 1,)), _vec(cu_cand, "cu_cand", torch.int32, (n + 1,))


def sv_cache_fork(cache: KVCache, page_table: torch.Tensor, ctx_len: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, *,
                  status=None, stream=None) -> None:
    """Sequences dst[i] (empty) become copies of src[i] that share its pages."""
    N = src.shape[0]
    _on_one_device(cache.k, page_table, ctx_len, src, dst, status)
    _launch("sv_cache_fork", cache.k, stream, cache._ref, _seqs(page_table, ctx_len), N, _vec(src, "src", torch.int32, (N,)),
            _vec(dst, "dst", torch.int32, (N,)), _vec(status, "status", torch.int32, (1,)))


def sv_cache_free(cache: KVCache, page_table: torch.Tensor, ctx_len: torch.Tensor, which: torch.Tensor, *, status=None,
                  stream=None) -> None:
    """Ends the sequences `which`: their pages are released."""
    N = which.shape[0]
    _on_one_device(cache.k, page_table, ctx_len, which, status)
    _launch("sv_cache_free", cache.k, stream, cache._ref, _seqs(page_table, ctx_len), N,
            _vec(which, "which", torch.int32, (N,)), _vec(status, "status", torch.int32, (1,)))


@functools.lru_cache(maxsize=1024)
def _reserve_bytes(n: int) -> int:
    return max(int(load().sv_cache_reserve_workspace_size(n)), 16)


def sv_cache_reserve(cache: KVCache, page_table: torch.Tensor, ctx_len: torch.Tensor, cu_draft=None, cu_cand=None, *,
                     granted=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """Pages for every sequence's window. Returns `granted` [n]: the window's
    rows, or 0 for a sequence that got no room."""
    n = page_table.shape[0]
    if granted is None:
        granted = _new(torch.empty, n, torch.int32, page_table, stream)
    _on_one_device(cache.k, page_table, ctx_len, cu_draft, cu_cand, granted, workspace, status)

    def call(ws):
        _launch("sv_cache_reserve", cache.k, stream, cache._ref, _seqs(page_table, ctx_len), *_windows(n, cu_draft, cu_cand),
                _vec(granted, "granted", torch.int32, (n,)), _ptr(ws), ws.numel(), _vec(status, "status", torch.int32, (1,)))

    if workspace is None:
        cache._launch_with_scratch(_reserve_bytes(n), stream, call)
    else:
        call(workspace)
    return granted


def sv_cache_append(cache: KVCache, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor,
                    ctx_len: torch.Tensor, cu_draft=None, cu_cand=None, *, status=None, stream=None) -> None:
    """Writes the windows' keys and values to their pages: [R, kv_heads,
    head_dim] for one layer, or [n_layers, R, kv_heads, head_dim] for the
    layers from `layer` on."""
    if k_new.dim() == 3:
        k_new, v_new = k_new[None], v_new[None]
    L, R = k_new.shape[:2]
    want = (L, R, cache.n_kv_heads, cache.head_dim)
    strides = k_new.stride()
    if k_new.shape != want or v_new.shape != want or (v_new.stride() != strides and _steps(v_new) != _steps(k_new)) or \
            (strides[2:] != (cache.head_dim, 1) and not _heads_contiguous(k_new)) or \
            k_new.dtype != cache.k.dtype or v_new.dtype != cache.k.dtype:
        raise ValueError("k_new and v_new must be [n_layers, R, kv_heads, head_dim] of the cache's dtype, alike "
                         "in strides, with contiguous heads")
    _on_one_device(cache.k, k_new, v_new, page_table, ctx_len, cu_draft, cu_cand, status)
    _launch("sv_cache_append", cache.k, stream, cache._ref, int(layer), L, k_new.data_ptr(), v_new.data_ptr(),
            strides[0] if L > 1 else 0, strides[1] if R > 1 else 0, R, _seqs(page_table, ctx_len),
            *_windows(page_table.shape[0], cu_draft, cu_cand), _vec(status, "status", torch.int32, (1,)))


def sv_cache_commit(cache: KVCache, page_table: torch.Tensor, ctx_len: torch.Tensor, cu_draft, out_len: torch.Tensor,
                    cu_cand=None, best=None, *, status=None, stream=None) -> None:
    """Keeps the committed rows of every window (candidate best[b]'s first
    out_len rows, moved to the window's front) and releases the pages behind
    them; ctx_len grows by the rows kept."""
    n = page_table.shape[0]
    if (cu_cand is None) != (best is None):
        raise ValueError("cu_cand and best come together")
    win = _windows(n, cu_draft, cu_cand)
    _on_one_device(cache.k, page_table, ctx_len, cu_draft, out_len, cu_cand, best, status)
    _launch("sv_cache_commit", cache.k, stream, cache._ref, _seqs(page_table, ctx_len), *win,
            _vec(best, "best", torch.int32, (n,)), _vec(out_len, "out_len", torch.int32, (win[0],)),
            _vec(status, "status", torch.int32, (1,)))


def sv_window_attention(q: torch.Tensor, cache: KVCache, layer: int, page_table: torch.Tensor, ctx_len: torch.Tensor,
                        cu_draft=None, cu_cand=None, *, scale: Optional[float] = None, out=None, out_lse=None,
                        want_lse: bool = False, workspace=None, status=None, stream=None):
    """Attention of every window (q [R, q_heads, head_dim]) over its history
    and itself, whose keys and values are in their pages. Returns (out, lse);
    rows of no window keep the values of a given `out`, and are zero in one
    made here. scale: 1 / sqrt(head_dim) if None."""
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.dtype != cache.k.dtype:
        raise ValueError("q must be [R, q_heads, head_dim] of the cache's dtype")
    R, heads, D = q.shape
    if out is None:
        out = _new(torch.zeros, (R, heads, D), q.dtype, q, stream)
    if out.shape != q.shape or out.dtype != q.dtype or (q.stride()[1:] != (D, 1) and not _heads_contiguous(q)) or \
            (out.stride()[1:] != (D, 1) and not _heads_contiguous(out)):
        raise ValueError("q and out must be [R, q_heads, head_dim] with contiguous heads")
    if out_lse is None and want_lse:
        out_lse = _new(torch.zeros, (R, heads), torch.float32, q, stream)
    _on_one_device(cache.k, q, page_table, ctx_len, cu_draft, cu_cand, out, out_lse, workspace, status)

    def call(ws):
        _launch("sv_window_attention", q, stream, q.data_ptr(), q.stride(0) if R > 1 else heads * D, heads, R, cache._ref,
                int(layer), _seqs(page_table, ctx_len), *_windows(page_table.shape[0], cu_draft, cu_cand),
                D ** -0.5 if scale is None else float(scale), out.data_ptr(), out.stride(0) if R > 1 else heads * D,
                _vec(out_lse, "out_lse", torch.float32, (R, heads)), _ptr(ws), ws.numel(),
                _vec(status, "status", torch.int32, (1,)))

    if workspace is None:
        cache._launch_with_scratch(cache._attention_bytes, stream, call)
    else:
        call(workspace)
    return out, out_lse
