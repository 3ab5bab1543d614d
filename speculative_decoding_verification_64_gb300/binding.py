"""ctypes binding of ``libspecdec.so`` (argument marshalling only).

Every step of the verify path runs in the library's CUDA kernels; this module
checks tensor shapes, dtypes and devices, allocates outputs and the workspace
with torch (device memory and streams are PyTorch's only role) and passes raw
device pointers to the C ABI declared in ``include/specdec.h``.  There is no
CPU fallback: if the library is missing or a call fails, an exception says so.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
from typing import Optional

import torch
from torch.autograd.forward_ad import unpack_dual

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecdec.so")

F32 = 0
BF16 = 1
OK = 0
ROW_BAD_TOKEN = 1
ROW_BAD_Q = 2
ROW_NONFINITE = 4
ROW_BAD_TEMP = 8
ROW_BAD_TREE = 16
ROW_INTERNAL = 32
ROW_BAD_CACHE = 64
ROW_BAD_FILTER = 128

_lib = None

_EXPORTS = {
    "specdec_abi_version": ([], ctypes.c_int),
    "specdec_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "specdec_workspace_size": ([ctypes.c_int] * 4, ctypes.c_size_t),
    "specdec_philox_uniforms": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_ulonglong,
                                 ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p],
                                ctypes.c_int),
    "specdec_row_entropy": ([ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p,
                             ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                             ctypes.c_void_p], ctypes.c_int),
    "specdec_verify_linear_launches": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "specdec_verify_linear_path": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "specdec_final_mass": ([ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int,
                            ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p],
                           ctypes.c_int),
    "specdec_row_alpha": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                           ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                           ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "specdec_path_logprob": ([ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                              ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                              ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int),
    "specdec_verify_linear_topk": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_void_p], ctypes.c_int),
    "specdec_row_stats": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                           ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                           ctypes.c_uint, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p],
                          ctypes.c_int),
    "specdec_verify_linear": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                              [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 +
                              [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p],
                              ctypes.c_int),
    "specdec_linear_finalize": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                                [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 +
                                [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p],
                                ctypes.c_int),
    "specdec_verify_tree": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                            [ctypes.c_void_p] * 4 + [ctypes.c_int] * 4 +
                            [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p],
                            ctypes.c_int),
    "specdec_verify_linear_static": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                                     [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 +
                                     [ctypes.c_void_p] * 7, ctypes.c_int),
    "specdec_linear_staging_size": ([ctypes.c_int] * 4, ctypes.c_size_t),
    "specdec_tree_staging_size": ([ctypes.c_int] * 5, ctypes.c_size_t),
    "specdec_verify_linear_host": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                                   [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 +
                                   [ctypes.c_void_p] * 7 + [ctypes.c_size_t, ctypes.c_void_p],
                                   ctypes.c_int),
    "specdec_verify_tree_host": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                                 [ctypes.c_void_p] * 4 + [ctypes.c_int] * 4 +
                                 [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p],
                                 ctypes.c_int),
    "specdec_tree_finalize": ([ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] +
                              [ctypes.c_void_p] * 4 + [ctypes.c_int] * 4 +
                              [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p],
                              ctypes.c_int),
    "specdec_rope": ([ctypes.c_void_p] * 2 + [ctypes.c_int] + [ctypes.c_longlong] * 2 +
                     [ctypes.c_void_p] * 4 + [ctypes.c_int] * 6 +
                     [ctypes.c_uint, ctypes.c_float] + [ctypes.c_void_p] * 3, ctypes.c_int),
    "specdec_kv_append": ([ctypes.c_void_p] * 2 + [ctypes.c_int] + [ctypes.c_longlong] * 2 +
                          [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                           ctypes.c_void_p, ctypes.c_int, ctypes.c_int] + [ctypes.c_void_p] * 3,
                          ctypes.c_int),
    "specdec_attend_workspace_size": ([ctypes.c_int] * 6, ctypes.c_size_t),
    "specdec_attend": ([ctypes.c_void_p] * 3 + [ctypes.c_int] + [ctypes.c_longlong] * 3 +
                       [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 + [ctypes.c_float] * 2 +
                       [ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 4 +
                       [ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "specdec_sample": ([ctypes.c_void_p, ctypes.c_int] + [ctypes.c_longlong] * 2 +
                       [ctypes.c_void_p] * 5 + [ctypes.c_int] * 4 + [ctypes.c_uint] +
                       [ctypes.c_void_p] * 2 + [ctypes.c_longlong] * 2 + [ctypes.c_void_p] * 3,
                       ctypes.c_int),
    "specdec_top_logits_workspace_size": ([ctypes.c_int] * 4, ctypes.c_size_t),
    "specdec_top_logits": ([ctypes.c_void_p, ctypes.c_int] + [ctypes.c_longlong] * 2 +
                           [ctypes.c_float] + [ctypes.c_int] * 4 + [ctypes.c_void_p] * 5 +
                           [ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "specdec_distill": ([ctypes.c_void_p, ctypes.c_int] + [ctypes.c_longlong] * 2 +
                        [ctypes.c_void_p] * 4 + [ctypes.c_float] + [ctypes.c_int] * 4 +
                        [ctypes.c_void_p] * 2 + [ctypes.c_longlong] * 2 + [ctypes.c_void_p] * 2,
                        ctypes.c_int),
    "specdec_distill_backward": ([ctypes.c_void_p, ctypes.c_int] + [ctypes.c_longlong] * 2 +
                                 [ctypes.c_void_p] * 5 + [ctypes.c_float] + [ctypes.c_int] * 4 +
                                 [ctypes.c_void_p] + [ctypes.c_longlong] * 2 + [ctypes.c_void_p],
                                 ctypes.c_int),
}


class SpecdecError(RuntimeError):
    pass


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load ``libspecdec.so``; raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise SpecdecError(
            f"{p} is missing: build it with __graft_entry__.build() or "
            "`python -m speculative_decoding_verification_64_gb300.build`")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _EXPORTS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().specdec_status_string(int(code)).decode()


def _check(rc: int, what: str):
    if rc != OK:
        raise SpecdecError(f"{what} failed: {status_string(rc)} (code {rc})")


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"logits/q must be float32 or bfloat16, got {t.dtype}")


def workspace_size(B: int, rows_per_request: int, V: int, dtype: int) -> int:
    return int(load_library().specdec_workspace_size(B, rows_per_request, V, dtype))


def alloc_workspace(B: int, rows_per_request: int, V: int, dtype: int,
                    device="cuda") -> torch.Tensor:
    n = max(workspace_size(B, rows_per_request, V, dtype), 256)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_HERE_AND_NOW = contextlib.nullcontext()


def _on(stream):
    """Where a call on ``stream`` makes its outputs and workspaces: with that stream current,
    so that torch's allocator hands their memory out again in its order, and not to other
    streams while the call's kernels still use it."""
    return _HERE_AND_NOW if stream is None else torch.cuda.stream(stream)


def _cuda(**tensors):
    """Every given tensor (None skipped) must live on one CUDA device, the
    current one: the library reads and writes device memory only (it has no
    CPU path), launches on the current device, and the binding passes that
    device's current stream."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other arrays on {dev}")
        dev = t.device
    if dev is not None:
        cur = torch.cuda.current_device()
        if (dev.index if dev.index is not None else cur) != cur:
            raise ValueError(f"the arrays are on {dev}, but the current device is cuda:{cur}: "
                             f"call under torch.cuda.device({dev.index})")


def _req(t: torch.Tensor, name: str, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


@dataclasses.dataclass
class LinearOut:
    n_accepted: torch.Tensor   # int32 [B]
    out_tokens: torch.Tensor   # int32 [B, gamma+1]
    final_token: torch.Tensor  # int32 [B]
    is_bonus: torch.Tensor     # uint8 [B]
    row_status: torch.Tensor   # int32 [B]
    p_draft: Optional[torch.Tensor]  # float32 [B, gamma]

    @staticmethod
    def empty(B, gamma, device, with_p=True):
        z = dict(dtype=torch.int32, device=device)
        return LinearOut(torch.empty(B, **z), torch.empty(B, gamma + 1, **z),
                         torch.empty(B, **z), torch.empty(B, dtype=torch.uint8, device=device),
                         torch.empty(B, **z),
                         torch.empty(B, gamma, dtype=torch.float32, device=device)
                         if with_p else None)


@dataclasses.dataclass
class TreeOut:
    n_accepted: torch.Tensor   # int32 [B]
    path_nodes: torch.Tensor   # int32 [B, max_depth+1]
    out_tokens: torch.Tensor   # int32 [B, max_depth+1]
    final_token: torch.Tensor  # int32 [B]
    is_bonus: torch.Tensor     # uint8 [B]
    row_status: torch.Tensor   # int32 [B]
    p_node: Optional[torch.Tensor]   # float32 [B, N]

    @staticmethod
    def empty(B, N, max_depth, device, with_p=True):
        z = dict(dtype=torch.int32, device=device)
        D1 = max_depth + 1
        return TreeOut(torch.empty(B, **z), torch.empty(B, D1, **z), torch.empty(B, D1, **z),
                       torch.empty(B, **z), torch.empty(B, dtype=torch.uint8, device=device),
                       torch.empty(B, **z),
                       torch.empty(B, N, dtype=torch.float32, device=device) if with_p else None)


def _linear_args(logits, q, draft_tokens, temperature, uniforms, out, workspace, stream):
    _cuda(logits=logits, q=q, draft_tokens=draft_tokens, temperature=temperature,
          uniforms=uniforms, workspace=workspace,
          **({} if out is None else {k: v for k, v in vars(out).items()}))
    B, R, V = logits.shape
    gamma = R - 1
    dev = logits.device
    dt = dtype_code(logits)
    _req(q, "q", logits.dtype, (B, gamma, V), dev)
    _req(logits, "logits", logits.dtype, (B, R, V), dev)
    _req(draft_tokens, "draft_tokens", torch.int32, (B, gamma), dev)
    _req(temperature, "temperature", torch.float32, (B,), dev)
    _req(uniforms, "uniforms", torch.float32, (B, R), dev)
    if out is None or workspace is None:
        with _on(stream):
            out = out if out is not None else LinearOut.empty(B, gamma, dev)
            workspace = workspace if workspace is not None else alloc_workspace(B, R, V, dt, dev)
    return B, gamma, V, dt, out, workspace


def verify_linear(logits: torch.Tensor, q: torch.Tensor, draft_tokens: torch.Tensor,
                  temperature: torch.Tensor, uniforms: torch.Tensor,
                  out: Optional[LinearOut] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> LinearOut:
    """Linear verify step (``specdec_verify_linear``) on CUDA tensors."""
    B, gamma, V, dt, out, ws = _linear_args(logits, q, draft_tokens, temperature, uniforms,
                                            out, workspace, stream)
    lib = load_library()
    rc = lib.specdec_verify_linear(
        _ptr(logits), _ptr(q), dt, _ptr(draft_tokens), _ptr(temperature), _ptr(uniforms),
        B, gamma, V, _ptr(out.n_accepted), _ptr(out.out_tokens), _ptr(out.final_token),
        _ptr(out.is_bonus), _ptr(out.row_status), _ptr(out.p_draft), _ptr(ws), ws.numel(),
        _stream_ptr(stream))
    _check(rc, "specdec_verify_linear")
    return out


STATS_ENTROPY = 1


def verify_linear_topk(logits: torch.Tensor, q: torch.Tensor, draft_tokens: torch.Tensor,
                       temperature: torch.Tensor, uniforms: torch.Tensor, topk: int,
                       out: Optional[LinearOut] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> LinearOut:
    """Linear verify with the top-k residual approximation (``specdec_verify_linear_topk``)."""
    B, gamma, V, dt, out, ws = _linear_args(logits, q, draft_tokens, temperature, uniforms,
                                            out, workspace, stream)
    rc = load_library().specdec_verify_linear_topk(
        _ptr(logits), _ptr(q), dt, _ptr(draft_tokens), _ptr(temperature), _ptr(uniforms),
        B, gamma, V, int(topk), _ptr(out.n_accepted), _ptr(out.out_tokens),
        _ptr(out.final_token), _ptr(out.is_bonus), _ptr(out.row_status), _ptr(out.p_draft),
        _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(rc, "specdec_verify_linear_topk")
    return out


def row_stats(logits: torch.Tensor, temperature: torch.Tensor, workspace: torch.Tensor,
              q: Optional[torch.Tensor] = None, draft_tokens: Optional[torch.Tensor] = None,
              entropy: bool = False, stream=None) -> None:
    """Phase 1 only (``specdec_row_stats``): logits [B, R, V] -> stage partials in the
    workspace.  For the linear form pass q and draft_tokens too (phase 2 needs the
    drafted tokens' logits and q values, gathered here).  ``entropy`` keeps the sums
    ``row_entropy`` reads."""
    _cuda(logits=logits, temperature=temperature, workspace=workspace, q=q,
          draft_tokens=draft_tokens)
    B, R, V = logits.shape
    rc = load_library().specdec_row_stats(
        _ptr(logits), _ptr(q), dtype_code(logits), _ptr(draft_tokens), _ptr(temperature), B, R, V,
        STATS_ENTROPY if entropy else 0, _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc, "specdec_row_stats")


def linear_finalize(logits, q, draft_tokens, temperature, uniforms, out: LinearOut,
                    workspace: torch.Tensor, stream=None) -> LinearOut:
    """Phase 2 of the linear form (``specdec_linear_finalize``)."""
    B, gamma, V, dt, out, ws = _linear_args(logits, q, draft_tokens, temperature, uniforms,
                                            out, workspace, stream)
    rc = load_library().specdec_linear_finalize(
        _ptr(logits), _ptr(q), dt, _ptr(draft_tokens), _ptr(temperature), _ptr(uniforms),
        B, gamma, V, _ptr(out.n_accepted), _ptr(out.out_tokens), _ptr(out.final_token),
        _ptr(out.is_bonus), _ptr(out.row_status), _ptr(out.p_draft), _ptr(ws), ws.numel(),
        _stream_ptr(stream))
    _check(rc, "specdec_linear_finalize")
    return out


def _tree_args(logits, q, node_tokens, parent, temperature, uniforms, max_depth, out,
               workspace, stream):
    _cuda(logits=logits, q=q, node_tokens=node_tokens, parent=parent, temperature=temperature,
          uniforms=uniforms, workspace=workspace,
          **({} if out is None else {k: v for k, v in vars(out).items()}))
    B, N, V = logits.shape
    dev = logits.device
    dt = dtype_code(logits)
    _req(q, "q", logits.dtype, (B, N, V), dev)
    _req(logits, "logits", logits.dtype, (B, N, V), dev)
    _req(node_tokens, "node_tokens", torch.int32, (B, N), dev)
    _req(parent, "parent", torch.int32, (B, N), dev)
    _req(temperature, "temperature", torch.float32, (B,), dev)
    _req(uniforms, "uniforms", torch.float32, (B, N), dev)
    if out is None or workspace is None:
        with _on(stream):
            out = out if out is not None else TreeOut.empty(B, N, max_depth, dev)
            workspace = workspace if workspace is not None else alloc_workspace(B, N, V, dt, dev)
    return B, N, V, dt, out, workspace


def verify_tree(logits, q, node_tokens, parent, temperature, uniforms, max_depth: int,
                out: Optional[TreeOut] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> TreeOut:
    """Token-tree verify step (``specdec_verify_tree``) on CUDA tensors."""
    B, N, V, dt, out, ws = _tree_args(logits, q, node_tokens, parent, temperature, uniforms,
                                      max_depth, out, workspace, stream)
    rc = load_library().specdec_verify_tree(
        _ptr(logits), _ptr(q), dt, _ptr(node_tokens), _ptr(parent), _ptr(temperature),
        _ptr(uniforms), B, N, V, max_depth, _ptr(out.n_accepted), _ptr(out.path_nodes),
        _ptr(out.out_tokens), _ptr(out.final_token), _ptr(out.is_bonus), _ptr(out.row_status),
        _ptr(out.p_node), _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(rc, "specdec_verify_tree")
    return out


def tree_finalize(logits, q, node_tokens, parent, temperature, uniforms, max_depth: int,
                  out: TreeOut, workspace: torch.Tensor, stream=None) -> TreeOut:
    """Phase 2 of the tree form (``specdec_tree_finalize``)."""
    B, N, V, dt, out, ws = _tree_args(logits, q, node_tokens, parent, temperature, uniforms,
                                      max_depth, out, workspace, stream)
    rc = load_library().specdec_tree_finalize(
        _ptr(logits), _ptr(q), dt, _ptr(node_tokens), _ptr(parent), _ptr(temperature),
        _ptr(uniforms), B, N, V, max_depth, _ptr(out.n_accepted), _ptr(out.path_nodes),
        _ptr(out.out_tokens), _ptr(out.final_token), _ptr(out.is_bonus), _ptr(out.row_status),
        _ptr(out.p_node), _ptr(ws), ws.numel(), _stream_ptr(stream))
    _check(rc, "specdec_tree_finalize")
    return out


# ---------------------------------------------------------------------------
# host-buffer calls: inputs and outputs in host memory, a device staging buffer
# ---------------------------------------------------------------------------

def linear_staging_size(B: int, gamma: int, V: int, dtype: int) -> int:
    return int(load_library().specdec_linear_staging_size(B, gamma, V, dtype))


def tree_staging_size(B: int, N: int, V: int, max_depth: int, dtype: int) -> int:
    return int(load_library().specdec_tree_staging_size(B, N, V, max_depth, dtype))


def _staging(nbytes: int, staging, device, stream) -> torch.Tensor:
    if staging is None:
        with _on(stream):
            return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if staging.device.type != "cuda" or staging.dtype != torch.uint8:
        raise ValueError("staging must be a uint8 CUDA tensor")
    _cuda(staging=staging)
    return staging


def _host_out(out, make):
    """A result container in page-locked host memory (made when None)."""
    if out is None:
        out = make()
        for k, v in vars(out).items():
            if v is not None:
                setattr(out, k, v.pin_memory())
    return out


def verify_linear_host(logits: torch.Tensor, q: torch.Tensor, draft_tokens: torch.Tensor,
                       temperature: torch.Tensor, uniforms: torch.Tensor,
                       out: Optional[LinearOut] = None, staging: Optional[torch.Tensor] = None,
                       stream=None, sync: bool = True, device="cuda") -> LinearOut:
    """Linear verify of host tensors (``specdec_verify_linear_host``): inputs and the
    returned outputs live in host memory (page-locked keeps the copies
    asynchronous); ``staging`` is device memory of ``linear_staging_size`` bytes.
    With ``sync=False`` the outputs are valid only after ``stream`` has reached
    the call."""
    cpu = torch.device("cpu")
    B, R, V = logits.shape
    gamma = R - 1
    dt = dtype_code(logits)
    _req(logits, "logits", logits.dtype, (B, R, V), cpu)
    _req(q, "q", logits.dtype, (B, gamma, V), cpu)
    _req(draft_tokens, "draft_tokens", torch.int32, (B, gamma), cpu)
    _req(temperature, "temperature", torch.float32, (B,), cpu)
    _req(uniforms, "uniforms", torch.float32, (B, R), cpu)
    out = _host_out(out, lambda: LinearOut.empty(B, gamma, cpu))
    st = _staging(linear_staging_size(B, gamma, V, dt), staging, device, stream)
    s = stream if stream is not None else torch.cuda.current_stream(st.device)
    rc = load_library().specdec_verify_linear_host(
        _ptr(logits), _ptr(q), dt, _ptr(draft_tokens), _ptr(temperature), _ptr(uniforms),
        B, gamma, V, _ptr(out.n_accepted), _ptr(out.out_tokens), _ptr(out.final_token),
        _ptr(out.is_bonus), _ptr(out.row_status), _ptr(out.p_draft), _ptr(st), st.numel(),
        ctypes.c_void_p(s.cuda_stream))
    _check(rc, "specdec_verify_linear_host")
    if sync:
        s.synchronize()
    return out


def verify_tree_host(logits, q, node_tokens, parent, temperature, uniforms, max_depth: int,
                     out: Optional[TreeOut] = None, staging: Optional[torch.Tensor] = None,
                     stream=None, sync: bool = True, device="cuda") -> TreeOut:
    """Token-tree verify of host tensors (``specdec_verify_tree_host``); as
    ``verify_linear_host``, with ``tree_staging_size`` bytes of staging."""
    cpu = torch.device("cpu")
    B, N, V = logits.shape
    dt = dtype_code(logits)
    _req(logits, "logits", logits.dtype, (B, N, V), cpu)
    _req(q, "q", logits.dtype, (B, N, V), cpu)
    _req(node_tokens, "node_tokens", torch.int32, (B, N), cpu)
    _req(parent, "parent", torch.int32, (B, N), cpu)
    _req(temperature, "temperature", torch.float32, (B,), cpu)
    _req(uniforms, "uniforms", torch.float32, (B, N), cpu)
    out = _host_out(out, lambda: TreeOut.empty(B, N, max_depth, cpu))
    st = _staging(tree_staging_size(B, N, V, max_depth, dt), staging, device, stream)
    s = stream if stream is not None else torch.cuda.current_stream(st.device)
    rc = load_library().specdec_verify_tree_host(
        _ptr(logits), _ptr(q), dt, _ptr(node_tokens), _ptr(parent), _ptr(temperature),
        _ptr(uniforms), B, N, V, max_depth, _ptr(out.n_accepted), _ptr(out.path_nodes),
        _ptr(out.out_tokens), _ptr(out.final_token), _ptr(out.is_bonus), _ptr(out.row_status),
        _ptr(out.p_node), _ptr(st), st.numel(), ctypes.c_void_p(s.cuda_stream))
    _check(rc, "specdec_verify_tree_host")
    if sync:
        s.synchronize()
    return out


def to_host(a, bf16: bool = False, pin: bool = True) -> torch.Tensor:
    """numpy array -> CPU tensor (page-locked by default); uint16 arrays with
    ``bf16`` are bfloat16 bits."""
    import numpy as np
    a = np.ascontiguousarray(a)
    t = torch.from_numpy(a.view(np.int16) if bf16 else a)
    t = t.view(torch.bfloat16) if bf16 else t
    return t.pin_memory() if pin else t.clone()


def linear_inputs_to_host(w, pin: bool = True):
    bf = w.dtype == "bf16"
    return (to_host(w.logits, bf, pin), to_host(w.q, bf, pin), to_host(w.draft_tokens, pin=pin),
            to_host(w.temperature, pin=pin), to_host(w.uniforms, pin=pin))


def tree_inputs_to_host(w, pin: bool = True):
    bf = w.dtype == "bf16"
    return (to_host(w.logits, bf, pin), to_host(w.q, bf, pin), to_host(w.node_tokens, pin=pin),
            to_host(w.parent, pin=pin), to_host(w.temperature, pin=pin),
            to_host(w.uniforms, pin=pin))


# ---------------------------------------------------------------------------
# host <-> device marshalling for numpy workloads
# ---------------------------------------------------------------------------

def to_device(a, device="cuda", bf16: bool = False) -> torch.Tensor:
    """numpy array -> CUDA tensor; uint16 arrays with ``bf16`` are bfloat16 bits."""
    import numpy as np
    a = np.ascontiguousarray(a)
    if bf16:
        t = torch.from_numpy(a.view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(a)
    return t.to(device)


def linear_inputs_to_device(w, device="cuda"):
    """A ``workloads.LinearWorkload`` as CUDA tensors (logits, q, tokens, T, u)."""
    bf = w.dtype == "bf16"
    return (to_device(w.logits, device, bf), to_device(w.q, device, bf),
            to_device(w.draft_tokens, device), to_device(w.temperature, device),
            to_device(w.uniforms, device))


def tree_inputs_to_device(w, device="cuda"):
    """A ``workloads.TreeWorkload`` as CUDA tensors (logits, q, tokens, parent, T, u)."""
    bf = w.dtype == "bf16"
    return (to_device(w.logits, device, bf), to_device(w.q, device, bf),
            to_device(w.node_tokens, device), to_device(w.parent, device),
            to_device(w.temperature, device), to_device(w.uniforms, device))


def philox_uniforms(key, counter, first_word: int, n: int, device="cuda", stream=None) -> torch.Tensor:
    """float32 uniforms of the Philox4x64-10 words [first_word, first_word + n) of the
    stream (key, counter), made on the device (``specdec_philox_uniforms``).  key: 2
    words, counter: 4 words (e.g. the state of ``numpy.random.Philox(seed)``)."""
    import numpy as np
    k = np.ascontiguousarray(np.asarray(key, dtype=np.uint64).reshape(-1))
    c = np.ascontiguousarray(np.asarray(counter, dtype=np.uint64).reshape(-1))
    if k.size != 2 or c.size != 4:
        raise ValueError("key must hold 2 and counter 4 64-bit words")
    with _on(stream):
        out = torch.empty(int(n), dtype=torch.float32, device=device)
    rc = load_library().specdec_philox_uniforms(k.ctypes.data, c.ctypes.data, int(first_word),
                                                int(n), _ptr(out) if n > 0 else None,
                                                _stream_ptr(stream))
    _check(rc, "specdec_philox_uniforms")
    return out



def row_entropy(logits: torch.Tensor, temperature: torch.Tensor, workspace: torch.Tensor,
                stream=None) -> torch.Tensor:
    """Entropies [B, R] of the target rows of ``logits`` from the workspace of a
    ``row_stats(..., entropy=True)`` call on those logits (``specdec_row_entropy``)."""
    _cuda(logits=logits, temperature=temperature, workspace=workspace)
    B, R, V = logits.shape
    with _on(stream):
        out = torch.empty((B, R), dtype=torch.float32, device=logits.device)
    rc = load_library().specdec_row_entropy(_ptr(workspace), workspace.numel(), dtype_code(logits),
                                            _ptr(temperature), B, R, V, _ptr(out),
                                            _stream_ptr(stream))
    _check(rc, "specdec_row_entropy")
    return out


def verify_linear_launches(logits: torch.Tensor, q: torch.Tensor) -> int:
    """Kernels ``verify_linear`` launches for these inputs: 1 (a small batch, one
    launch) or 2 (the stats pass, then the draw)."""
    B, R, V = logits.shape
    return int(load_library().specdec_verify_linear_launches(B, R - 1, V, dtype_code(logits),
                                                             _ptr(logits), _ptr(q)))


def final_mass(workspace: torch.Tensor, B: int, rows_per_request: int, V: int, dtype: int,
               stream=None) -> torch.Tensor:
    """Normaliser [B] of each request's final draw in the last verify call on
    ``workspace`` (``specdec_final_mass``; NaN where nothing was drawn)."""
    _cuda(workspace=workspace)
    with _on(stream):
        out = torch.empty(B, dtype=torch.float32, device=workspace.device)
    rc = load_library().specdec_final_mass(_ptr(workspace), workspace.numel(), B,
                                           rows_per_request, V, dtype,
                                           _ptr(out) if B > 0 else None, _stream_ptr(stream))
    _check(rc, "specdec_final_mass")
    return out


PATH_NONE, PATH_SMALL_ONE_LAUNCH, PATH_TWO_LAUNCHES = 0, 1, 3
PATH_KERNELS = {PATH_SMALL_ONE_LAUNCH: "small_verify_kernel", PATH_TWO_LAUNCHES: "row_stats_kernel"}


def verify_linear_path(logits: torch.Tensor, q: torch.Tensor) -> int:
    """The path ``verify_linear`` takes for these inputs (``PATH_*``): a small
    batch in one launch, or two launches."""
    B, R, V = logits.shape
    return int(load_library().specdec_verify_linear_path(B, R - 1, V, dtype_code(logits),
                                                         _ptr(logits), _ptr(q)))


def row_alpha(logits: torch.Tensor, q: torch.Tensor, temperature: torch.Tensor,
              workspace: torch.Tensor, stream=None) -> torch.Tensor:
    """Acceptance rates [B, gamma], sum_v min(p_i, q_i) of every drafted row, from the
    logits [B, gamma+1, V], q [B, gamma, V] and the workspace of a ``row_stats`` call on
    those logits (``specdec_row_alpha``)."""
    _cuda(logits=logits, q=q, temperature=temperature, workspace=workspace)
    B, R, V = logits.shape
    gamma = R - 1
    with _on(stream):
        out = torch.empty((B, gamma), dtype=torch.float32, device=logits.device)
    rc = load_library().specdec_row_alpha(_ptr(logits), _ptr(q), dtype_code(logits),
                                          _ptr(temperature), B, gamma, V, _ptr(workspace),
                                          workspace.numel(), _ptr(out), _stream_ptr(stream))
    _check(rc, "specdec_row_alpha")
    return out


def path_logprob(logits: torch.Tensor, temperature: torch.Tensor, out_tokens: torch.Tensor,
                 n_accepted: torch.Tensor, workspace: torch.Tensor,
                 path_nodes: Optional[torch.Tensor] = None,
                 row_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Log-probabilities [B] of the emitted paths (``specdec_path_logprob``)."""
    _cuda(logits=logits, temperature=temperature, out_tokens=out_tokens, n_accepted=n_accepted,
          workspace=workspace, path_nodes=path_nodes, row_status=row_status)
    B, R, V = logits.shape
    with _on(stream):
        out = torch.empty(B, dtype=torch.float32, device=logits.device)
    rc = load_library().specdec_path_logprob(
        _ptr(logits), dtype_code(logits), _ptr(temperature), _ptr(out_tokens), _ptr(n_accepted),
        _ptr(path_nodes), _ptr(row_status), B, R, V, out_tokens.shape[1], _ptr(workspace),
        workspace.numel(), _ptr(out), _stream_ptr(stream))
    _check(rc, "specdec_path_logprob")
    return out


# ---------------------------------------------------------------------------
# the attention side of the step: rotary positions, the 8-bit cache, attention
# ---------------------------------------------------------------------------

ROPE_INTERLEAVED, ROPE_BACKWARD = 1, 2


class _CacheStruct(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "block_table",
                                                "length")] +
                [(n, ctypes.c_int) for n in ("n_blocks", "max_blocks", "block", "Hkv", "D")])


@dataclasses.dataclass
class KVCache:
    """A paged cache in 8 bits (``specdec_kv_cache``): token j of request b is slot
    j % block of block ``block_table[b, j // block]``; value = code * scale."""
    k: torch.Tensor            # float8_e4m3fn [n_blocks, Hkv, block, D]
    v: torch.Tensor            # float8_e4m3fn [n_blocks, Hkv, block, D]
    k_scale: torch.Tensor      # float32 [n_blocks, Hkv]
    v_scale: torch.Tensor      # float32 [n_blocks, Hkv]
    block_table: torch.Tensor  # int32 [B, max_blocks]
    length: torch.Tensor       # int32 [B]

    @staticmethod
    def empty(B: int, max_blocks: int, n_blocks: int, block: int, Hkv: int, D: int,
              device="cuda") -> "KVCache":
        """An empty cache: no request holds a token and no table entry a block (-1)."""
        f8 = torch.float8_e4m3fn
        shape = (n_blocks, Hkv, block, D)
        return KVCache(torch.empty(shape, dtype=torch.uint8, device=device).view(f8),
                       torch.empty(shape, dtype=torch.uint8, device=device).view(f8),
                       torch.zeros(n_blocks, Hkv, device=device),
                       torch.zeros(n_blocks, Hkv, device=device),
                       torch.full((B, max_blocks), -1, dtype=torch.int32, device=device),
                       torch.zeros(B, dtype=torch.int32, device=device))


@dataclasses.dataclass
class AppendOut:
    length: torch.Tensor      # int32 [B]: the cache's length with the new tokens
    row_status: torch.Tensor  # int32 [B]


@dataclasses.dataclass
class AttendOut:
    out: torch.Tensor            # [B, N, Hq, D] in q's dtype
    lse: Optional[torch.Tensor]  # float32 [B, N, Hq]
    row_status: torch.Tensor     # int32 [B]


def _raw(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _raw_stream(stream) -> int:
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


# torch's own lookup of the current stream without making a Stream object, where it has one
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(stream, tensors, names):
    """The raw stream of a call on these tensors (None skipped), which all have to live on the
    current device.  These calls run once a layer and step, some on a single token, so their
    checks are the plain attribute reads that cost least; ``_cuda`` words the error."""
    dev = tensors[0].get_device()  # -1: host memory
    for t in tensors:
        if t is not None and t.get_device() != dev:
            dev = -1
            break
    if dev < 0 or dev != torch.cuda.current_device():
        _cuda(**dict(zip(names, tensors)))
    if stream is None and _current_raw_stream is not None:
        return _current_raw_stream(dev)
    return _raw_stream(stream)


def _tokens4(t: torch.Tensor, name: str, dtype, B: int, N: int, H, D: int) -> int:
    """Elements between consecutive tokens of a [B, N, H, D] tensor (H None: any) whose heads
    and elements are contiguous (a whole tensor, or heads of a fused projection)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != N or shape[3] != D or \
            (H is not None and shape[2] != H):
        raise ValueError(f"{name} must have shape [{B}, {N}, {'heads' if H is None else H}, {D}], "
                         f"got {tuple(shape)}")
    s = t.stride()
    H = shape[2]
    at = s[1] if N > 1 else s[0] if B > 1 else H * D
    if (s[3] != 1 and D > 1) or (s[2] != D and H > 1) or (B > 1 and N > 1 and s[0] != N * at):
        raise ValueError(f"{name}: heads and elements must be contiguous and tokens one stride "
                         f"apart, got strides {s}")
    return at


def _flat(t: torch.Tensor, name: str, dtype, shape):
    """A contiguous tensor of this type and shape (a tuple)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _req(t, name, dtype, shape, t.device)


_CACHE_NAMES = ("cache.k", "cache.v", "cache.k_scale", "cache.v_scale", "cache.block_table",
                "cache.length")


def _cache_struct(c: KVCache, B: int) -> _CacheStruct:
    k, v, ks, vs, table, length = c.k, c.v, c.k_scale, c.v_scale, c.block_table, c.length
    shape = k.shape
    if len(shape) != 4:
        raise ValueError(f"cache.k must be [n_blocks, Hkv, block, D], got {tuple(shape)}")
    nb, Hkv, block, D = shape
    f8 = torch.float8_e4m3fn
    _flat(k, "cache.k", f8, shape)
    _flat(v, "cache.v", f8, shape)
    _flat(ks, "cache.k_scale", torch.float32, (nb, Hkv))
    _flat(vs, "cache.v_scale", torch.float32, (nb, Hkv))
    if table.dim() != 2:
        raise ValueError(f"cache.block_table must be [B, max_blocks], got {tuple(table.shape)}")
    width = table.shape[1]
    _flat(table, "cache.block_table", torch.int32, (B, width))
    _flat(length, "cache.length", torch.int32, (B,))
    return _CacheStruct(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                        table.data_ptr(), length.data_ptr(), nb, width, block, Hkv, D)


def rope_frequencies(rot: int, theta: float = 10000.0, factor: float = 1.0,
                     original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device="cuda") -> torch.Tensor:
    """Frequencies of ``rope`` in units of 2^-64 turns a position, int64 [rot / 2]: pair i
    turns by theta^(-2i/rot) radians a position.  ``factor`` > 1 stretches them for a
    context ``factor`` times longer: all pairs alike (position interpolation), or, given
    the ``original_length`` that a model was trained on, only those that turn fewer than
    ``beta_slow`` times over it, with a linear ramp up to ``beta_fast`` turns
    (interpolation by frequency band)."""
    import math
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and positive, got {rot}")
    words = []
    for i in range(rot // 2):
        turns = theta ** (-2.0 * i / rot) / (2.0 * math.pi)
        if factor != 1.0:
            keep = 0.0
            if original_length > 0:
                # the ramp is linear in the pair's index, from where a pair turns
                # beta_fast times over the original length to where it turns beta_slow times,
                # be that among the pairs or before the first or past the last
                def at(n):
                    return rot * math.log(original_length / (n * 2.0 * math.pi)) / \
                        (2.0 * math.log(theta))
                low, high = math.floor(at(beta_fast)), math.ceil(at(beta_slow))
                keep = 1.0 - min(1.0, max(0.0, (i - low) / max(high - low, 1e-3)))
            turns = turns * keep + turns / factor * (1.0 - keep)
        word = int(math.ldexp(turns, 64)) % 2 ** 64
        words.append(word - 2 ** 64 if word >= 2 ** 63 else word)
    return torch.tensor(words, dtype=torch.int64, device=device)


def rope(q: torch.Tensor, k: Optional[torch.Tensor], freq: torch.Tensor,
         positions: Optional[torch.Tensor] = None, base: Optional[torch.Tensor] = None,
         parent: Optional[torch.Tensor] = None, interleaved: bool = False,
         backward: bool = False, magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions (``specdec_rope``) of q [B, N, Hq, D] and k [B, N, Hk, D] (or None):
    returns the turned (q, k).  Positions are ``positions`` [B, N], or ``base`` [B] plus the
    depth of each node of ``parent`` [B, N] (a chain without it).  ``backward``: the
    gradient, from dq and dk; it is also what autograd takes for q and k that need one
    (no q_out or k_out then)."""
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        if q_out is not None or k_out is not None:
            raise ValueError("q_out and k_out cannot be given where q or k requires a gradient")
        with _on(stream):
            return _Rope.apply(q, k, freq, positions, base, parent, interleaved, backward, magnitude)
    raw = _here(stream, (q, k, freq, positions, base, parent, q_out, k_out),
                ("q", "k", "freq", "positions", "base", "parent", "q_out", "k_out"))
    dt = dtype_code(q)
    if q.dim() != 4:
        raise ValueError(f"q must be [B, N, Hq, D], got {tuple(q.shape)}")
    B, N, Hq, D = q.shape
    q_at = _tokens4(q, "q", q.dtype, B, N, Hq, D)
    Hk = k_at = 0
    if k is not None:
        k_at, Hk = _tokens4(k, "k", q.dtype, B, N, None, D), k.shape[2]
    half = freq.numel()
    _flat(freq, "freq", torch.int64, (half,))
    if positions is not None:
        _flat(positions, "positions", torch.int32, (B, N))
    if base is not None:
        _flat(base, "base", torch.int32, (B,))
    if parent is not None:
        _flat(parent, "parent", torch.int32, (B, N))
    if q_out is None:
        with _on(stream):
            q_out = torch.empty((B, N, Hq, D), dtype=q.dtype, device=q.device)
    else:
        _flat(q_out, "q_out", q.dtype, (B, N, Hq, D))
    if k is None:
        k_out = None
    elif k_out is None:
        with _on(stream):
            k_out = torch.empty((B, N, Hk, D), dtype=q.dtype, device=q.device)
    else:
        _flat(k_out, "k_out", q.dtype, (B, N, Hk, D))
    rc = load_library().specdec_rope(
        q.data_ptr(), _raw(k), dt, q_at, k_at, freq.data_ptr(), _raw(positions), _raw(base),
        _raw(parent), B, N, Hq, Hk, D, 2 * half,
        (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_BACKWARD if backward else 0), magnitude,
        q_out.data_ptr(), _raw(k_out), raw)
    _check(rc, "specdec_rope")
    return q_out, k_out


class _Rope(torch.autograd.Function):
    """``rope`` under autograd: the map is linear, its transpose the same call."""

    @staticmethod
    def forward(ctx, q, k, freq, positions, base, parent, interleaved, backward, magnitude):
        ctx.save_for_backward(freq, positions, base, parent)
        ctx.how = interleaved, not backward, magnitude
        return rope(q, k, freq, positions, base, parent, interleaved, backward, magnitude)

    @staticmethod
    def backward(ctx, dq, dk):
        if dk is not None and not ctx.needs_input_grad[1]:
            dk = None
        q, k = rope(dq.contiguous(), None if dk is None else dk.contiguous(), *ctx.saved_tensors, *ctx.how)
        return (q, k) + (None,) * 7


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache,
              count: Optional[torch.Tensor] = None, extra: int = 0,
              path: Optional[torch.Tensor] = None, out: Optional[AppendOut] = None,
              stream=None) -> AppendOut:
    """Append tokens of k, v [B, N, Hkv, D] to the cache (``specdec_kv_append``): of request b
    the first ``count[b] + extra`` nodes (N + extra without count) of ``path`` [B, path_len]
    or of 0 .. N-1.  After a verify step: ``count=r.n_accepted, extra=1`` and, for a tree,
    ``path=r.path_nodes``.  ``cache.length`` is left alone: set it to the result's
    ``length`` for the next step.  (No gradient passes through the cache.)"""
    raw = _here(stream, (k, v, count, path, cache.k, cache.v, cache.k_scale, cache.v_scale,
                         cache.block_table, cache.length) +
                (() if out is None else (out.length, out.row_status)),
                ("k", "v", "count", "path") + _CACHE_NAMES + ("out.length", "out.row_status"))
    dt = dtype_code(k)
    if k.dim() != 4:
        raise ValueError(f"k must be [B, N, Hkv, D], got {tuple(k.shape)}")
    B, N = k.shape[:2]
    c = _cache_struct(cache, B)
    k_at = _tokens4(k, "k", k.dtype, B, N, c.Hkv, c.D)
    v_at = _tokens4(v, "v", k.dtype, B, N, c.Hkv, c.D)
    if count is not None:
        _flat(count, "count", torch.int32, (B,))
    if path is not None:
        _flat(path, "path", torch.int32, (B, path.shape[-1]))
    if out is None:
        with _on(stream):
            out = AppendOut(torch.empty(B, dtype=torch.int32, device=k.device),
                            torch.empty(B, dtype=torch.int32, device=k.device))
    else:
        _flat(out.length, "out.length", torch.int32, (B,))
        _flat(out.row_status, "out.row_status", torch.int32, (B,))
    rc = load_library().specdec_kv_append(
        k.data_ptr(), v.data_ptr(), dt, k_at, v_at, _raw(count), extra, _raw(path),
        path.shape[1] if path is not None else 0, ctypes.addressof(c), B, N,
        out.length.data_ptr(), out.row_status.data_ptr(), raw)
    _check(rc, "specdec_kv_append")
    return out


def attend_workspace_size(B: int, N: int, Hq: int, Hkv: int, D: int, dtype: int) -> int:
    return int(load_library().specdec_attend_workspace_size(B, N, Hq, Hkv, D, dtype))


def alloc_attend_workspace(q: torch.Tensor, cache: KVCache) -> torch.Tensor:
    """The workspace of ``attend`` for queries of q's shape on this cache."""
    B, N, Hq, D = q.shape
    n = attend_workspace_size(B, N, Hq, cache.k.shape[1], D, dtype_code(q))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: KVCache,
           parent: Optional[torch.Tensor] = None, n_nodes: Optional[torch.Tensor] = None,
           scale: Optional[float] = None, softcap: float = 0.0,
           slopes: Optional[torch.Tensor] = None, window: int = 0,
           out: Optional[AttendOut] = None, workspace: Optional[torch.Tensor] = None,
           stream=None) -> AttendOut:
    """Attention of drafted tokens (``specdec_attend``): q [B, N, Hq, D] over the request's
    cached tokens and, by the chain or the tree ``parent`` [B, N], over the drafted tokens'
    own k, v [B, N, Hkv, D].  ``scale`` defaults to D ** -0.5.  (Inference only: the result
    carries no gradient.)"""
    raw = _here(stream, (q, k, v, parent, n_nodes, slopes, workspace, cache.k, cache.v,
                         cache.k_scale, cache.v_scale, cache.block_table, cache.length) +
                (() if out is None else (out.out, out.lse, out.row_status)),
                ("q", "k", "v", "parent", "n_nodes", "slopes", "workspace") + _CACHE_NAMES +
                ("out.out", "out.lse", "out.row_status"))
    dtype = q.dtype
    dt = dtype_code(q)
    if q.dim() != 4:
        raise ValueError(f"q must be [B, N, Hq, D], got {tuple(q.shape)}")
    B, N, Hq, D = q.shape
    c = _cache_struct(cache, B)
    if D != c.D:
        raise ValueError(f"q has heads of {D} elements, the cache of {c.D}")
    q_at = _tokens4(q, "q", dtype, B, N, Hq, D)
    k_at = _tokens4(k, "k", dtype, B, N, c.Hkv, D)
    v_at = _tokens4(v, "v", dtype, B, N, c.Hkv, D)
    if parent is not None:
        _flat(parent, "parent", torch.int32, (B, N))
    if n_nodes is not None:
        _flat(n_nodes, "n_nodes", torch.int32, (B,))
    if slopes is not None:
        _flat(slopes, "slopes", torch.float32, (Hq,))
    if out is None:
        dev = q.device
        with _on(stream):
            out = AttendOut(torch.empty((B, N, Hq, D), dtype=dtype, device=dev),
                            torch.empty((B, N, Hq), dtype=torch.float32, device=dev),
                            torch.empty(B, dtype=torch.int32, device=dev))
    else:
        _flat(out.out, "out.out", dtype, (B, N, Hq, D))
        if out.lse is not None:
            _flat(out.lse, "out.lse", torch.float32, (B, N, Hq))
        _flat(out.row_status, "out.row_status", torch.int32, (B,))
    if workspace is None:
        with _on(stream):
            workspace = alloc_attend_workspace(q, cache)
    rc = load_library().specdec_attend(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, q_at, k_at, v_at, _raw(parent),
        _raw(n_nodes), ctypes.addressof(c), B, N, Hq, D ** -0.5 if scale is None else scale,
        softcap, _raw(slopes), window, out.out.data_ptr(), _raw(out.lse),
        out.row_status.data_ptr(), workspace.data_ptr(), workspace.numel(), raw)
    _check(rc, "specdec_attend")
    return out


# ---------------------------------------------------------------------------
# the draft side of the step: sampling, records of the target's rows, distillation
# ---------------------------------------------------------------------------

SAMPLE_LOGITS = 1


@dataclasses.dataclass
class SampleOut:
    tokens: Optional[torch.Tensor]  # int32 [B, R, S]
    rows: Optional[torch.Tensor]    # [B, R, V] in the logits' dtype
    kept: torch.Tensor              # int32 [B, R]
    row_status: torch.Tensor        # int32 [B, R]


@dataclasses.dataclass
class TopOut:
    values: torch.Tensor      # float32 [B, R, K], largest first
    ids: torch.Tensor         # int32 [B, R, K]
    lse: torch.Tensor         # float32 [B, R]
    row_status: torch.Tensor  # int32 [B, R]


@dataclasses.dataclass
class DistillOut:
    loss: torch.Tensor            # float32 [B, R]
    grad: Optional[torch.Tensor]  # [B, R, V] in the logits' dtype
    row_status: torch.Tensor      # int32 [B, R]


def _rows3(t: torch.Tensor, name: str, dtype, shape):
    """The strides, in elements, of requests and of rows of a [B, R, V] tensor whose rows are
    contiguous (``shape`` None: any)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [B, R, V], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous, got strides {s}")
    return s[0], s[1]


def _sample(logits, temperature, uniforms, top_k, top_p, min_p, rows, flags, out, stream):
    raw = _here(stream, (logits, temperature, uniforms, top_k, top_p, min_p) +
                (() if out is None else (out.tokens, out.rows, out.kept, out.row_status)),
                ("logits", "temperature", "uniforms", "top_k", "top_p", "min_p", "out.tokens",
                 "out.rows", "out.kept", "out.row_status"))
    dtype = logits.dtype
    dt = dtype_code(logits)
    request, row = _rows3(logits, "logits", dtype, None)
    B, R, V = logits.shape
    _flat(temperature, "temperature", torch.float32, (B,))
    if top_k is not None:
        _flat(top_k, "top_k", torch.int32, (B,))
    if top_p is not None:
        _flat(top_p, "top_p", torch.float32, (B,))
    if min_p is not None:
        _flat(min_p, "min_p", torch.float32, (B,))
    S = 0
    if uniforms is not None:
        if uniforms.dim() != 3:
            raise ValueError(f"uniforms must be [B, R, S], got {tuple(uniforms.shape)}")
        S = uniforms.shape[2]
        _flat(uniforms, "uniforms", torch.float32, (B, R, S))
    if out is None:
        dev = logits.device
        with _on(stream):
            out = SampleOut(
                None if uniforms is None else torch.empty((B, R, S), dtype=torch.int32, device=dev),
                torch.empty((B, R, V), dtype=dtype, device=dev) if rows else None,
                torch.empty((B, R), dtype=torch.int32, device=dev),
                torch.empty((B, R), dtype=torch.int32, device=dev))
    else:
        if uniforms is not None:
            if out.tokens is None:
                raise ValueError("out.tokens is missing")
            _flat(out.tokens, "out.tokens", torch.int32, (B, R, S))
        _flat(out.kept, "out.kept", torch.int32, (B, R))
        _flat(out.row_status, "out.row_status", torch.int32, (B, R))
    to_request = to_row = 0
    if out.rows is not None:
        to_request, to_row = _rows3(out.rows, "out.rows", dtype, logits.shape)
    rc = load_library().specdec_sample(
        logits.data_ptr(), dt, request, row, temperature.data_ptr(), _raw(top_k), _raw(top_p),
        _raw(min_p), uniforms.data_ptr() if S else None, B, R, V, S, flags,
        out.tokens.data_ptr() if S else None, _raw(out.rows), to_request, to_row,
        out.kept.data_ptr(), out.row_status.data_ptr(), raw)
    _check(rc, "specdec_sample")
    return out


def sample(logits: torch.Tensor, temperature: torch.Tensor, uniforms: torch.Tensor,
           top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
           min_p: Optional[torch.Tensor] = None, probs: bool = True,
           out: Optional[SampleOut] = None, stream=None) -> SampleOut:
    """S tokens of every row of logits [B, R, V] from uniforms [B, R, S], under every request's
    temperature and filters [B] (``specdec_sample``): ``out.tokens`` [B, R, S] and, with
    ``probs``, ``out.rows`` [B, R, V], the distributions that they were drawn from: drafted
    tokens and q of the verify calls.  An ``out`` of the caller's decides by its ``rows``,
    which may be a slice such as ``q[:, i:i + 1]``, or None."""
    return _sample(logits, temperature, uniforms, top_k, top_p, min_p, probs, 0, out, stream)


def filter_logits(logits: torch.Tensor, temperature: torch.Tensor,
                  top_k: Optional[torch.Tensor] = None, top_p: Optional[torch.Tensor] = None,
                  min_p: Optional[torch.Tensor] = None, out: Optional[SampleOut] = None,
                  stream=None) -> SampleOut:
    """``out.rows`` [B, R, V]: the logits of what the filters of ``sample`` keep, -infinity for
    the rest (``specdec_sample`` with SPECDEC_SAMPLE_LOGITS).  A verify call on the target's
    rows so filtered, at the same temperature, emits tokens of the filtered distribution.
    ``out.rows`` may be the logits themselves."""
    return _sample(logits, temperature, None, top_k, top_p, min_p, True, SAMPLE_LOGITS, out, stream)


def top_logits_workspace_size(B: int, R: int, V: int, dtype: int) -> int:
    return int(load_library().specdec_top_logits_workspace_size(B, R, V, dtype))


def top_logits(logits: torch.Tensor, k: int, temperature: float = 1.0,
               out: Optional[TopOut] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> TopOut:
    """The k largest of every row of logits [B, R, V] (largest first, equal ones by index)
    and its log-sum-exp at ``temperature`` (``specdec_top_logits``): the record of a target's
    row that ``distill`` learns from."""
    raw = _here(stream, (logits, workspace) +
                (() if out is None else (out.values, out.ids, out.lse, out.row_status)),
                ("logits", "workspace", "out.values", "out.ids", "out.lse", "out.row_status"))
    dt = dtype_code(logits)
    request, row = _rows3(logits, "logits", logits.dtype, None)
    B, R, V = logits.shape
    dev = logits.device
    if out is None:
        with _on(stream):
            out = TopOut(torch.empty((B, R, k), dtype=torch.float32, device=dev),
                         torch.empty((B, R, k), dtype=torch.int32, device=dev),
                         torch.empty((B, R), dtype=torch.float32, device=dev),
                         torch.empty((B, R), dtype=torch.int32, device=dev))
    else:
        _flat(out.values, "out.values", torch.float32, (B, R, k))
        _flat(out.ids, "out.ids", torch.int32, (B, R, k))
        _flat(out.lse, "out.lse", torch.float32, (B, R))
        _flat(out.row_status, "out.row_status", torch.int32, (B, R))
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(max(top_logits_workspace_size(B, R, V, dt), 256),
                                    dtype=torch.uint8, device=dev)
    rc = load_library().specdec_top_logits(
        logits.data_ptr(), dt, request, row, temperature, B, R, V, k, out.values.data_ptr(),
        out.ids.data_ptr(), out.lse.data_ptr(), out.row_status.data_ptr(), workspace.data_ptr(),
        workspace.numel(), raw)
    _check(rc, "specdec_top_logits")
    return out


def _distill_rows(logits, ids, teacher, lse, weight):
    """The checked sizes and strides of a distillation's inputs."""
    dt = dtype_code(logits)
    request, row = _rows3(logits, "logits", logits.dtype, None)
    B, R, V = logits.shape
    if ids.dim() != 3:
        raise ValueError(f"ids must be [B, R, K], got {tuple(ids.shape)}")
    K = ids.shape[2]
    _flat(ids, "ids", torch.int32, (B, R, K))
    _flat(teacher, "teacher", torch.float32, (B, R, K))
    if lse is not None:
        _flat(lse, "lse", torch.float32, (B, R))
    if weight is not None:
        _flat(weight, "weight", torch.float32, (B, R))
    return dt, request, row, B, R, V, K


def distill(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
            lse: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
            temperature: float = 1.0, grad: bool = True, out: Optional[DistillOut] = None,
            stream=None) -> DistillOut:
    """Divergence of the draft's rows of logits [B, R, V] from a teacher's records (ids int32
    and logits float32 [B, R, K], with the rows' ``lse`` [B, R] or renormalised over their
    entries), and ``weight`` times its gradient (``specdec_distill``).  An ``out`` of the
    caller's decides by its ``grad``, which may be the logits themselves, or None.
    ``distill_loss`` is the same under autograd."""
    raw = _here(stream, (logits, ids, teacher, lse, weight) +
                (() if out is None else (out.loss, out.grad, out.row_status)),
                ("logits", "ids", "teacher", "lse", "weight", "out.loss", "out.grad", "out.row_status"))
    dt, request, row, B, R, V, K = _distill_rows(logits, ids, teacher, lse, weight)
    dev = logits.device
    if out is None:
        with _on(stream):
            out = DistillOut(torch.empty((B, R), dtype=torch.float32, device=dev),
                             torch.empty((B, R, V), dtype=logits.dtype, device=dev) if grad else None,
                             torch.empty((B, R), dtype=torch.int32, device=dev))
    else:
        _flat(out.loss, "out.loss", torch.float32, (B, R))
        _flat(out.row_status, "out.row_status", torch.int32, (B, R))
    g_request = g_row = 0
    if out.grad is not None:
        g_request, g_row = _rows3(out.grad, "out.grad", logits.dtype, logits.shape)
    rc = load_library().specdec_distill(
        logits.data_ptr(), dt, request, row, ids.data_ptr(), teacher.data_ptr(), _raw(lse),
        _raw(weight), temperature, B, R, V, K, out.loss.data_ptr(), _raw(out.grad), g_request,
        g_row, out.row_status.data_ptr(), raw)
    _check(rc, "specdec_distill")
    return out


def distill_loss(logits: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                 lse: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                 temperature: float = 1.0, stream=None) -> torch.Tensor:
    """``weight`` times the divergences of ``distill``, float32 [B, R], under autograd (for the
    logits and the weights).  The logits' gradient is made with the loss, from one look at
    them, and holds for rows whose incoming gradient is 1, as under ``.sum()``: a mean is
    cheaper as weights of 1 / n than as a division afterwards.  A weight's gradient is its
    row's divergence, for which rows of weight 0 are looked at too where the weights require
    one.  A malformed row's loss and gradients are NaN.  The teacher is a constant: a ``teacher``
    or ``lse`` that requires a gradient is refused, and so are tangents (forward mode)."""
    if torch.is_grad_enabled():
        for name, t in (("teacher", teacher), ("lse", lse)):
            if t is not None and t.requires_grad:
                raise ValueError(f"distill_loss has no gradient for {name}: pass {name}.detach()")
    learn = torch.is_grad_enabled() and (logits.requires_grad or
                                         (weight is not None and weight.requires_grad))
    with _on(stream):
        # (torch refuses tangents there, where no form of them is defined)
        if learn or any(t is not None and unpack_dual(t).tangent is not None
                        for t in (logits, teacher, lse, weight)):
            return _Distill.apply(logits, ids, teacher, lse, weight, temperature)
        loss = distill(logits, ids, teacher, lse, weight, temperature, grad=False).loss
        return loss if weight is None else loss * weight


class _Distill(torch.autograd.Function):
    """``distill`` under autograd.  The first backward turns the forward's gradient into its
    own, in place; a second one (over a retained graph) makes it anew.  It is saved like the inputs,
    so that hooks on saved tensors (offloading, checkpoints) have it too."""

    @staticmethod
    def forward(ctx, logits, ids, teacher, lse, weight, temperature):
        r = distill(logits, ids, teacher, lse, weight, temperature, grad=ctx.needs_input_grad[0])
        loss = None
        if ctx.needs_input_grad[4]:  # the rows of weight 0 have theirs too
            alone = (weight == 0).float()
            loss = r.loss + distill(logits, ids, teacher, lse, alone, temperature, grad=False).loss
        ctx.save_for_backward(logits, ids, teacher, lse, weight, loss, r.grad)
        ctx.temperature, ctx.spent = temperature, False
        return r.loss if weight is None else r.loss * weight

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        logits, ids, teacher, lse, weight, loss, grad = ctx.saved_tensors
        dloss = dloss.contiguous()
        dweight = None if loss is None else dloss * loss
        if not ctx.needs_input_grad[0]:
            grad = None
        elif ctx.spent:
            w = dloss if weight is None else torch.where(weight == 0, weight, dloss * weight)
            grad = distill(logits, ids, teacher, lse, w, ctx.temperature).grad
        else:
            ctx.spent = True
            _distill_backward(logits, ids, teacher, lse, weight, ctx.temperature, dloss, grad)
            grad = grad.data  # (the caller's: what becomes of it is no change of a saved tensor)
        return grad, None, None, None, dweight, None


def _distill_backward(logits, ids, teacher, lse, weight, temperature, dloss, grad):
    """A forward's gradient becomes ``dloss`` times itself (``specdec_distill_backward``)."""
    raw = _here(None, (logits, ids, teacher, lse, weight, dloss, grad),
                ("logits", "ids", "teacher", "lse", "weight", "dloss", "grad"))
    dt, request, row, B, R, V, K = _distill_rows(logits, ids, teacher, lse, weight)
    g_request, g_row = _rows3(grad, "grad", logits.dtype, logits.shape)
    _flat(dloss, "dloss", torch.float32, (B, R))
    rc = load_library().specdec_distill_backward(
        logits.data_ptr(), dt, request, row, ids.data_ptr(), teacher.data_ptr(), _raw(lse),
        _raw(weight), dloss.data_ptr(), temperature, B, R, V, K, grad.data_ptr(), g_request, g_row,
        raw)
    _check(rc, "specdec_distill_backward")
