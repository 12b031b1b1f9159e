"""Python binding of libdrafthead.so (the reduced-vocabulary NVFP4 draft head).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch provides device memory and the current stream. If the compiled
library is missing, every call raises; there is no fallback.

Names follow the C ABI in include/drafthead.h:
  draft_head_build_index   keep mask -> dh_idx (padded to N % 64 == 0)
  nvfp4_quantize_rows      gather + NVFP4 quantisation of W[dh_idx]
  fp8_quantize_rows        gather + per-tensor FP8 E4M3 quantisation
  fp8_quantize_activations per-token FP8 E4M3 codes of hidden states (W8A8)
  DraftHead.top_tokens     get_top_tokens: dh_idx[argmax_n (W_q h)]
  DraftHead.compute_logits compute_logits: -inf row + logits at dh_idx
  NVFP4Linear              nvfp4_linear: an MTP-block linear, y = x W'^T
  DraftHead.top_keys       draft_head_top_keys: a vocabulary shard's argmax keys
  keys_to_ids              draft_head_keys_to_ids: combined keys -> target ids
  NVFP4Matmul              nvfp4_matmul: y = x W'^T for many tokens, activations
                           quantised to NVFP4 per token (W4A4)
  draft_head_row_map       dh_idx -> column of every target id
  token_logprobs           draft_head_token_logprobs: log-probabilities of given
                           tokens, entropy, normaliser, top alternatives
  distill_topk             draft_head_distill: distillation loss and gradient
  (_forward, _backward)    the loss alone; the gradient from its normaliser
  DistillTopK              the same as a torch.autograd function
A call given stream= works and allocates on that stream: its arguments have to be
ready there, and its results are, for what follows on it.
The vocabulary-sharded head (the local-argmax exchange) is in .sharded.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import NamedTuple

import numpy as np
import torch

from . import build as _build

DH_OK, DH_ERR_ARG, DH_ERR_SHAPE, DH_ERR_ALIGN, DH_ERR_WORKSPACE, DH_ERR_CUDA = 0, 1, 2, 3, 4, 5
DH_FMT_NVFP4, DH_FMT_FP8, DH_FMT_BF16, DH_FMT_NVFP4_PACKED, DH_FMT_FP8_W8A8 = 1, 2, 3, 4, 5
DH_MAX_M = 16
DH_WORKSPACE_ALIGN = 256
DH_DEVERR_IDX = 1
DH_DEVERR_TIMEOUT = 2
DH_DEVERR_UNFINISHED = 4
DH_HEAD_IDX_ASCENDING = 1
DH_T_BF16, DH_T_F16, DH_T_F32 = 1, 2, 3
DH_MAX_TOP, DH_MAX_TEACHER = 128, 512

EXPORTS = (
    "draft_head_build_index", "draft_head_quantize_workspace_bytes", "nvfp4_quantize_rows",
    "fp8_quantize_rows", "draft_head_workspace_bytes", "draft_head_workspace_init",
    "draft_head_top_tokens", "draft_head_compute_logits", "draft_head_read_device_error",
    "draft_head_status_string", "draft_head_abi_version", "draft_head_top_tokens_static",
    "nvfp4_pack_head", "fp8_quantize_activations", "draft_head_last_cuda_error", "nvfp4_linear",
    "draft_head_wait_probe", "draft_head_top_tokens_host", "draft_head_top_keys", "draft_head_keys_to_ids",
    "draft_head_static_read_device_error", "draft_head_row_map", "draft_head_token_logprobs", "draft_head_distill",
    "draft_head_distill_backward", "nvfp4_matmul_packed_bytes", "nvfp4_pack_matmul", "nvfp4_matmul_workspace_bytes",
    "nvfp4_matmul", "nvfp4_matmul_wait_probe",
)

_lib = None


class DraftHeadError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().draft_head_status_string(status).decode() if _lib is not None else str(status)
        self.cuda_error = 0
        if status == DH_ERR_CUDA and _lib is not None:
            name = C.c_char_p()
            self.cuda_error = _lib.draft_head_last_cuda_error(C.byref(name))
            msg += f": {name.value.decode() if name.value else self.cuda_error}"
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


class dh_head_t(C.Structure):
    _fields_ = [("fmt", C.c_int), ("V", C.c_int), ("K", C.c_int), ("N", C.c_int),
                ("n_kept", C.c_int), ("q", C.c_void_p), ("sf", C.c_void_p),
                ("scale", C.c_void_p), ("idx", C.c_void_p), ("flags", C.c_uint)]


class dh_logits_t(C.Structure):
    _fields_ = [("z", C.c_void_p), ("type", C.c_int), ("M", C.c_int), ("C", C.c_int), ("ld", C.c_int64),
                ("temperature", C.c_float), ("row_of", C.c_void_p), ("V", C.c_int), ("idx", C.c_void_p)]


# a dh_logits_t as bytes: built once per call, in a sixth of the time of the ctypes structure
_pack_logits = struct.Struct("@PiiiqfPiP").pack
assert struct.calcsize("@PiiiqfPiP") == C.sizeof(dh_logits_t)


class dh_matmul_t(C.Structure):
    _fields_ = [("N", C.c_int), ("K", C.c_int), ("packed", C.c_void_p), ("scale", C.c_void_p)]


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """Load libdrafthead.so (built by ``nvfp4_draft_head_gb300.build``); raises if absent."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libdrafthead.so is not built ({path}); run "
                               "`python -m nvfp4_draft_head_gb300.build`")
        L = C.CDLL(path)
        P, I, S = C.c_void_p, C.c_int, C.c_size_t
        L.draft_head_build_index.argtypes = [P, I, P, I, P, P]
        L.draft_head_quantize_workspace_bytes.argtypes = []
        L.draft_head_quantize_workspace_bytes.restype = S
        L.nvfp4_quantize_rows.argtypes = [P, I, I, P, I, P, P, P, P, S, P]
        L.fp8_quantize_rows.argtypes = [P, I, I, P, I, P, P, P, S, P]
        L.draft_head_workspace_bytes.argtypes = [C.POINTER(dh_head_t), I]
        L.draft_head_workspace_bytes.restype = S
        L.draft_head_workspace_init.argtypes = [P, S, P]
        L.draft_head_top_tokens.argtypes = [C.POINTER(dh_head_t), P, I, P, P, P, S, P]
        L.draft_head_top_tokens_host.argtypes = [C.POINTER(dh_head_t), P, I, P, P, P, S, P]
        L.draft_head_compute_logits.argtypes = [C.POINTER(dh_head_t), P, I, P, P, S, P]
        L.draft_head_read_device_error.argtypes = [P, P, P]
        L.draft_head_status_string.argtypes = [I]
        L.draft_head_status_string.restype = C.c_char_p
        L.draft_head_abi_version.argtypes = []
        L.draft_head_top_tokens_static.argtypes = [C.POINTER(dh_head_t), P, I, P, P, P]
        L.nvfp4_pack_head.argtypes = [P, P, I, I, P, P]
        L.fp8_quantize_activations.argtypes = [P, I, I, P, P, P]
        L.draft_head_last_cuda_error.argtypes = [C.POINTER(C.c_char_p)]
        L.nvfp4_linear.argtypes = [C.POINTER(dh_head_t), P, I, P, P, S, P]
        L.draft_head_wait_probe.argtypes = [P, S, I, C.c_uint, P]
        L.draft_head_top_keys.argtypes = [C.POINTER(dh_head_t), P, I, P, P, S, P]
        L.draft_head_keys_to_ids.argtypes = [P, I, P, P, P]
        L.draft_head_static_read_device_error.argtypes = [P, P]
        # (a dh_logits_t as its bytes, or by reference)
        L.draft_head_row_map.argtypes = [P, I, P, I, P]
        L.draft_head_token_logprobs.argtypes = [P, P, I, P, P, P, I, P, P, P]
        L.draft_head_distill.argtypes = [P, P, P, I, I, P, P, P, P, C.c_int64, P]
        L.draft_head_distill_backward.argtypes = [P, P, P, I, I, P, P, P, C.c_int64, P]
        L.nvfp4_matmul_packed_bytes.argtypes = [I, I]
        L.nvfp4_matmul_packed_bytes.restype = S
        L.nvfp4_pack_matmul.argtypes = [P, P, I, I, P, P]
        L.nvfp4_matmul_workspace_bytes.argtypes = [I, I]
        L.nvfp4_matmul_workspace_bytes.restype = S
        L.nvfp4_matmul.argtypes = [C.POINTER(dh_matmul_t), P, I, C.c_int64, I, P, I, C.c_int64, P, S, P, P]
        L.nvfp4_matmul_wait_probe.argtypes = [C.POINTER(dh_matmul_t), P, I, P, P, S, I, C.c_uint, P, P]
        _lib = L
    return _lib


def _check(fn: str, st: int):
    if st != DH_OK:
        raise DraftHeadError(fn, st)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None) -> int:
    """cudaStream_t of `stream`, or of the current stream (without building a
    Stream object: this runs once per draft step)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _keep_for(stream, *values) -> None:
    """Tensors (of any values) used on `stream`, not their own, stay allocated until its work is done."""
    for t in values:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)


def _on_stream(stream, call, *args):
    """call(*args) with `stream` current, for a caller that asked for it: what the
    call allocates comes from that stream's own pool (a block of the caller's
    stream may still be in use by work pending there) and is filled on it. The
    arguments stay allocated for `stream`'s work, the results for the caller's."""
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(*args)
    _keep_for(stream, *args)
    _keep_for(here, *(out if isinstance(out, tuple) else (out,)))
    return out


def _workspace(nbytes: int, device) -> torch.Tensor:
    """Zeroed device buffer whose data pointer is DH_WORKSPACE_ALIGN-aligned."""
    buf = torch.zeros(nbytes + DH_WORKSPACE_ALIGN, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % DH_WORKSPACE_ALIGN
    return buf[off: off + nbytes]


# ---------------------------------------------------------------- head build --

def draft_head_build_index(keep) -> tuple[np.ndarray, int]:
    """(dh_idx int32[N], n_kept) from a host keep mask (numpy or CPU tensor)."""
    keep = np.ascontiguousarray(np.asarray(keep).astype(np.uint8))
    V = keep.size
    idx = np.empty(V + 64, dtype=np.int32)
    nk, N = C.c_int(), C.c_int()
    _check("draft_head_build_index",
           lib().draft_head_build_index(keep.ctypes.data, V, idx.ctypes.data, idx.size,
                                        C.byref(nk), C.byref(N)))
    return idx[: N.value].copy(), nk.value


def _gather_args(W: torch.Tensor, idx: torch.Tensor):
    if W.dtype != torch.bfloat16 or W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous [V, K] bfloat16 CUDA tensor")
    if idx.dtype != torch.int32 or idx.dim() != 1 or idx.device != W.device:
        raise ValueError("idx must be an int32 vector on W's device")
    return W.shape[0], W.shape[1], idx.numel()


def nvfp4_quantize_rows(W: torch.Tensor, idx: torch.Tensor, stream=None):
    """(q uint8[N, K/2], sf uint8[N, K/16], g float32[1]) of the rows W[idx]."""
    if stream is not None:
        return _on_stream(stream, nvfp4_quantize_rows, W, idx)
    V, K, N = _gather_args(W, idx)
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    sf = torch.empty((N, K // 16), dtype=torch.uint8, device=W.device)
    g = torch.empty(1, dtype=torch.float32, device=W.device)
    nb = lib().draft_head_quantize_workspace_bytes()
    ws = _workspace(nb, W.device)
    _check("nvfp4_quantize_rows",
           lib().nvfp4_quantize_rows(W.data_ptr(), V, K, idx.data_ptr(), N, q.data_ptr(),
                                     sf.data_ptr(), g.data_ptr(), ws.data_ptr(), nb, _stream()))
    _raise_device_error(ws, "nvfp4_quantize_rows")
    return q, sf, g


def fp8_quantize_rows(W: torch.Tensor, idx: torch.Tensor, stream=None):
    """(q uint8[N, K] E4M3 codes, scale float32[1]) of the rows W[idx]."""
    if stream is not None:
        return _on_stream(stream, fp8_quantize_rows, W, idx)
    V, K, N = _gather_args(W, idx)
    q = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    s = torch.empty(1, dtype=torch.float32, device=W.device)
    nb = lib().draft_head_quantize_workspace_bytes()
    ws = _workspace(nb, W.device)
    _check("fp8_quantize_rows",
           lib().fp8_quantize_rows(W.data_ptr(), V, K, idx.data_ptr(), N, q.data_ptr(),
                                   s.data_ptr(), ws.data_ptr(), nb, _stream()))
    _raise_device_error(ws, "fp8_quantize_rows")
    return q, s


def nvfp4_pack_head(q: torch.Tensor, sf: torch.Tensor, stream=None) -> torch.Tensor:
    """Tile-major copy of an NVFP4 head (DH_FMT_NVFP4_PACKED): uint8 [N/16, K/128, 1152]."""
    if stream is not None:
        return _on_stream(stream, nvfp4_pack_head, q, sf)
    N, Kh = q.shape
    K = 2 * Kh
    if sf.shape != (N, K // 16) or q.dtype != torch.uint8 or sf.dtype != torch.uint8:
        raise ValueError("q must be uint8 [N, K/2] and sf uint8 [N, K/16]")
    packed = torch.empty((N // 16, K // 128, 1152), dtype=torch.uint8, device=q.device)
    _check("nvfp4_pack_head",
           lib().nvfp4_pack_head(q.data_ptr(), sf.data_ptr(), N, K, packed.data_ptr(), _stream()))
    return packed


def fp8_quantize_activations(h: torch.Tensor, stream=None):
    """(qx uint8[M, K] E4M3 codes, sx float32[M] scales): per-token dynamic FP8
    quantisation of BF16 hidden states, as the W8A8 head's draft step does it."""
    if stream is not None:
        return _on_stream(stream, fp8_quantize_activations, h)
    if h.dtype != torch.bfloat16 or h.dim() != 2 or not h.is_cuda or not h.is_contiguous():
        raise ValueError("h must be a contiguous [M, K] bfloat16 CUDA tensor")
    M, K = h.shape
    qx = torch.empty((M, K), dtype=torch.uint8, device=h.device)
    sx = torch.empty(M, dtype=torch.float32, device=h.device)
    _check("fp8_quantize_activations",
           lib().fp8_quantize_activations(h.data_ptr(), M, K, qx.data_ptr(), sx.data_ptr(), _stream()))
    return qx, sx


def draft_head_read_device_error(ws: torch.Tensor, stream=None) -> int:
    err = C.c_int()
    _check("draft_head_read_device_error",
           lib().draft_head_read_device_error(ws.data_ptr(), C.byref(err), _stream(stream)))
    return err.value


def draft_head_static_read_device_error(stream=None) -> int:
    """Read and clear the static scratch's device error word (synchronises)."""
    err = C.c_int(0)
    _check("draft_head_static_read_device_error",
           lib().draft_head_static_read_device_error(C.byref(err), _stream(stream)))
    return err.value


def draft_head_wait_probe(ws: torch.Tensor | None, kind: int, rounds: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test on workspace ws, or on the static
    scratch of draft_head_top_tokens_static when ws is None (kind 0: a global
    word nothing writes, 1: an mbarrier nothing arrives on)."""
    _check("draft_head_wait_probe",
           lib().draft_head_wait_probe(_ptr(ws), 0 if ws is None else ws.numel(), kind, rounds,
                                       _stream(stream)))


def _raise_device_error(ws, fn):
    err = draft_head_read_device_error(ws)
    if err:
        raise RuntimeError(f"{fn}: device error word {err:#x} (a dh_idx entry outside [0, V))")


# ---------------------------------------------------------------- draft step --

class DraftHead:
    """A quantised draft head plus its workspace; tensors stay owned by torch.

    fmt: DH_FMT_NVFP4 (q, sf, scale=g), DH_FMT_NVFP4_PACKED (tile-major q, scale=g),
    DH_FMT_FP8 / DH_FMT_FP8_W8A8 (q, scale) or DH_FMT_BF16 (q = the BF16
    weights, idx may be None for a full-vocabulary head).
    """

    def __init__(self, fmt: int, V: int, q: torch.Tensor, idx: torch.Tensor | None, n_kept: int,
                 sf: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                 idx_ascending: bool = False):
        self.fmt, self.V, self.n_kept = fmt, int(V), int(n_kept)
        self.flags = DH_HEAD_IDX_ASCENDING if idx_ascending else 0
        self.q, self.sf, self.scale, self.idx = q, sf, scale, idx
        self.N = q.shape[0]
        if fmt == DH_FMT_NVFP4_PACKED:        # [N/16, K/128, 1152]
            self.N = q.shape[0] * 16
            self.K = q.shape[1] * 128
        elif fmt == DH_FMT_NVFP4:
            self.K = q.shape[1] * 2
        elif fmt in (DH_FMT_FP8, DH_FMT_FP8_W8A8):
            self.K = q.shape[1]
        else:
            self.K = q.shape[1] if q.dtype == torch.bfloat16 else q.shape[1] // 2
        self.desc = dh_head_t(fmt, self.V, self.K, self.N, self.n_kept, _ptr(q), _ptr(sf),
                              _ptr(scale), _ptr(idx), self.flags)
        self.ws_bytes = lib().draft_head_workspace_bytes(C.byref(self.desc), DH_MAX_M)
        self.ws = _workspace(self.ws_bytes, q.device)
        _check("draft_head_workspace_init",
               lib().draft_head_workspace_init(self.ws.data_ptr(), self.ws_bytes, _stream()))

    def with_storage(self, q: torch.Tensor, sf: torch.Tensor | None = None) -> "DraftHead":
        """The same head (same scale, idx, workspace) read from another copy of q / sf."""
        other = object.__new__(DraftHead)
        other.__dict__.update(self.__dict__)
        other.q, other.sf = q, (sf if sf is not None else self.sf)
        other.desc = dh_head_t(self.fmt, self.V, self.K, self.N, self.n_kept, _ptr(other.q),
                               _ptr(other.sf), _ptr(self.scale), _ptr(self.idx), self.flags)
        return other

    def top_tokens(self, h: torch.Tensor, ids: torch.Tensor | None = None,
                   top: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """get_top_tokens: int32[M] target ids of the argmax over kept rows."""
        if ids is None and stream is not None:
            return _on_stream(stream, self.top_tokens, h, None, top)
        M = self._check_h(h)
        if ids is None:
            ids = torch.empty(M, dtype=torch.int32, device=h.device)
        _check("draft_head_top_tokens",
               lib().draft_head_top_tokens(C.byref(self.desc), h.data_ptr(), M, ids.data_ptr(),
                                           _ptr(top), self.ws.data_ptr(), self.ws_bytes,
                                           _stream(stream)))
        return ids

    def top_keys(self, h: torch.Tensor, keys: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """This head as one vocabulary shard: int64[M] argmax keys (largest
        logit, then lowest target id) whose maximum over shards is the whole
        head's; needs an ascending dh_idx."""
        if keys is None and stream is not None:
            return _on_stream(stream, self.top_keys, h)
        M = self._check_h(h)
        if keys is None:
            keys = torch.empty(M, dtype=torch.int64, device=h.device)
        _check("draft_head_top_keys",
               lib().draft_head_top_keys(C.byref(self.desc), h.data_ptr(), M, keys.data_ptr(),
                                         self.ws.data_ptr(), self.ws_bytes, _stream(stream)))
        return keys

    def top_tokens_host(self, h: torch.Tensor, ids: torch.Tensor | None = None,
                        top: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """get_top_tokens on host tensors: h a CPU bfloat16 [M, K] tensor; ids
        (returned) a CPU int32 [M] tensor; top an optional CPU float32 [M] tensor.
        One C call enqueues the copy of h to the device, the draft step and the
        copies back; the results are valid once the stream synchronises. Pinned
        tensors keep the copies asynchronous."""
        if h.device.type != "cpu":
            raise ValueError("h must be a host (CPU) tensor")
        M = self._check_h(h)
        if ids is None:
            ids = torch.empty(M, dtype=torch.int32, pin_memory=h.is_pinned())
        elif ids.device.type != "cpu" or ids.dtype != torch.int32 or ids.numel() != M or not ids.is_contiguous():
            raise ValueError(f"ids must be a contiguous CPU torch.int32 tensor of {M} elements")
        if top is not None and (top.device.type != "cpu" or top.dtype != torch.float32 or top.numel() != M
                                or not top.is_contiguous()):
            raise ValueError(f"top must be a contiguous CPU torch.float32 tensor of {M} elements")
        _check("draft_head_top_tokens_host",
               lib().draft_head_top_tokens_host(C.byref(self.desc), h.data_ptr(), M, ids.data_ptr(),
                                                _ptr(top), self.ws.data_ptr(), self.ws_bytes,
                                                _stream(stream)))
        return ids

    def compute_logits(self, h: torch.Tensor, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
        """compute_logits: float32[M, V], -inf outside the kept ids."""
        if out is None and stream is not None:
            return _on_stream(stream, self.compute_logits, h)
        M = self._check_h(h)
        if out is None:
            out = torch.empty((M, self.V), dtype=torch.float32, device=h.device)
        _check("draft_head_compute_logits",
               lib().draft_head_compute_logits(C.byref(self.desc), h.data_ptr(), M, out.data_ptr(),
                                               self.ws.data_ptr(), self.ws_bytes, _stream(stream)))
        return out

    def device_error(self, stream=None) -> int:
        return draft_head_read_device_error(self.ws, stream)

    def _check_h(self, h: torch.Tensor) -> int:
        if h.dtype != torch.bfloat16 or h.dim() != 2 or h.shape[1] != self.K or not h.is_contiguous():
            raise ValueError(f"h must be a contiguous [M, {self.K}] bfloat16 tensor")
        return h.shape[0]


def keys_to_ids(keys: torch.Tensor, ids: torch.Tensor | None = None, top: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Target ids (and, into `top`, the winning logits) of argmax keys."""
    if ids is None and stream is not None:
        return _on_stream(stream, keys_to_ids, keys, None, top)
    M = keys.numel()
    if keys.dtype != torch.int64 or not keys.is_contiguous():
        raise ValueError("keys must be a contiguous int64 tensor")
    if ids is None:
        ids = torch.empty(M, dtype=torch.int32, device=keys.device)
    _check("draft_head_keys_to_ids",
           lib().draft_head_keys_to_ids(keys.data_ptr(), M, ids.data_ptr(), _ptr(top), _stream(stream)))
    return ids


def nvfp4_head(W: torch.Tensor, keep, packed: bool = True, stream=None) -> DraftHead:
    """Build an NVFP4 draft head from a BF16 target head and a host keep mask
    (repacked tile-major unless packed=False)."""
    idx_np, nk = draft_head_build_index(keep)
    idx = torch.from_numpy(idx_np).to(W.device)
    q, sf, g = nvfp4_quantize_rows(W, idx, stream)
    if packed and (W.shape[1] % 128 == 0):
        qp = nvfp4_pack_head(q, sf, stream)
        return DraftHead(DH_FMT_NVFP4_PACKED, W.shape[0], qp, idx, nk, scale=g, idx_ascending=True)
    return DraftHead(DH_FMT_NVFP4, W.shape[0], q, idx, nk, sf=sf, scale=g, idx_ascending=True)


def fp8_head(W: torch.Tensor, keep, w8a8: bool = False, stream=None) -> DraftHead:
    """Build a per-tensor FP8 draft head from a BF16 target head and a host keep
    mask: W8A16 (BF16 hidden states), or W8A8 (per-token FP8 hidden states)."""
    idx_np, nk = draft_head_build_index(keep)
    idx = torch.from_numpy(idx_np).to(W.device)
    q, s = fp8_quantize_rows(W, idx, stream)
    return DraftHead(DH_FMT_FP8_W8A8 if w8a8 else DH_FMT_FP8, W.shape[0], q, idx, nk, scale=s,
                     idx_ascending=True)


class NVFP4Linear:
    """An NVFP4 W4A16 linear layer (an MTP-block linear): weight W [N, K] BF16
    quantised with the head's recipe and repacked tile-major; forward(x) =
    x W'^T in fp32. N % 64 == 0."""

    def __init__(self, W: torch.Tensor, stream=None):
        if stream is not None:
            _on_stream(stream, self.__init__, W)
            return _keep_for(torch.cuda.current_stream(stream.device), self.q, self.sf, self.g, self.packed, self.ws)
        N, K = W.shape
        idx = torch.arange(N, dtype=torch.int32, device=W.device)
        q, sf, g = nvfp4_quantize_rows(W, idx)
        self.q, self.sf, self.g = q, sf, g
        self.packed = nvfp4_pack_head(q, sf)
        self.N, self.K = N, K
        self.desc = dh_head_t(DH_FMT_NVFP4_PACKED, N, K, N, N, _ptr(self.packed), None, _ptr(g), None, 0)
        self.ws_bytes = lib().draft_head_workspace_bytes(C.byref(self.desc), DH_MAX_M)
        self.ws = _workspace(self.ws_bytes, W.device)

    def with_storage(self, packed: torch.Tensor) -> "NVFP4Linear":
        """The same layer read from another copy of its packed bytes."""
        other = object.__new__(NVFP4Linear)
        other.__dict__.update(self.__dict__)
        other.packed = packed
        other.desc = dh_head_t(DH_FMT_NVFP4_PACKED, self.N, self.K, self.N, self.N, _ptr(packed), None,
                               _ptr(self.g), None, 0)
        return other

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.K or not x.is_contiguous():
            raise ValueError(f"x must be a contiguous [M, {self.K}] bfloat16 tensor")
        if y is None and stream is not None:
            return _on_stream(stream, self.forward, x)
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float32, device=x.device)
        _check("nvfp4_linear",
               lib().nvfp4_linear(C.byref(self.desc), x.data_ptr(), M, y.data_ptr(), self.ws.data_ptr(),
                                  self.ws_bytes, _stream(stream)))
        return y

    __call__ = forward

    def device_error(self, stream=None) -> int:
        return draft_head_read_device_error(self.ws, stream)


def bf16_full_head(W: torch.Tensor) -> DraftHead:
    """The stock full-vocabulary BF16 head (the row is the id)."""
    return DraftHead(DH_FMT_BF16, W.shape[0], W, None, W.shape[0])


def bf16_truncated_head(W: torch.Tensor, n_rows: int) -> DraftHead:
    """A truncated BF16 draft head: the first n_rows rows of the target head
    (ids 0 .. n_rows-1, n_rows % 64 == 0), read in place; compute_logits still
    writes full-vocabulary rows (-inf past n_rows)."""
    if n_rows % 64 or not 0 < n_rows <= W.shape[0]:
        raise ValueError("n_rows must be a multiple of 64 within the head")
    return DraftHead(DH_FMT_BF16, W.shape[0], W[:n_rows], None, n_rows)


# --------------------------------------------------- operators on many tokens --

_TYPES = {torch.bfloat16: DH_T_BF16, torch.float16: DH_T_F16, torch.float32: DH_T_F32}


def _vector(t: torch.Tensor | None, name: str, dtype: torch.dtype, n: int | None, device) -> None:
    if t is not None and (t.dtype != dtype or t.device != device or not t.is_contiguous() or (n is not None and t.numel() != n)):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor{'' if n is None else f' of {n} elements'} on {device}")


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(t: torch.Tensor) -> int:
    """cudaStream_t of the current stream; t's device has to be the current one, where
    the library launches."""
    device = t.get_device()
    if device != _current_device():
        raise ValueError(f"the tensors are on cuda:{device}, which is not the device of the call: make it the current device "
                         "(torch.cuda.device) and pass a stream of that device")
    return _raw_stream(device) if _raw_stream is not None else _stream()


def _no_gradient(t: torch.Tensor, name: str) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} require a gradient, which this operator does not have: detach them, or call it under torch.no_grad()")


class NVFP4Matmul:
    """An NVFP4 weight for many-token products: forward(x) = x W'^T with x
    quantised to NVFP4 per token (W4A4) and fp32 accumulation. q uint8 [N, K/2],
    sf uint8 [N, K/16] and g float32 [1] as from nvfp4_quantize_rows; N % 64 == 0,
    K % 16 == 0. No gradient: an x that requires one is refused.

    These are not the logits of the draft step: for up to 16 tokens NVFP4Linear and
    DraftHead keep the activations in bfloat16 (W4A16). Four-bit activations change a
    logit by about a tenth of the logits' spread (a 64,064 x 2,560 head on normal
    hidden states: rms 0.096 of the standard deviation; 0.16 where one channel in 211
    is 30 times the rest), so what is scored here is the W4A4 head: for acceptance
    rates and rejection sampling of a served W4A16 head take DraftHead.compute_logits."""

    def __init__(self, q: torch.Tensor, sf: torch.Tensor, g: torch.Tensor, stream=None):
        if stream is not None:
            _on_stream(stream, self.__init__, q, sf, g)
            return _keep_for(torch.cuda.current_stream(stream.device), self.packed, self.error)
        if q.dtype != torch.uint8 or q.dim() != 2 or not q.is_cuda or not q.is_contiguous():
            raise ValueError("q must be a contiguous [N, K/2] uint8 CUDA tensor")
        self.N, self.K = q.shape[0], 2 * q.shape[1]
        if sf.shape != (self.N, self.K // 16):
            raise ValueError(f"sf must be uint8 [{self.N}, {self.K // 16}]")
        _vector(sf, "sf", torch.uint8, None, q.device)
        _vector(g, "g", torch.float32, 1, q.device)
        self.g = g
        nb = lib().nvfp4_matmul_packed_bytes(self.N, self.K)
        if nb == 0:
            raise DraftHeadError("nvfp4_matmul_packed_bytes", DH_ERR_SHAPE)
        self.packed = torch.empty(nb, dtype=torch.uint8, device=q.device)
        _check("nvfp4_pack_matmul",
               lib().nvfp4_pack_matmul(q.data_ptr(), sf.data_ptr(), self.N, self.K, self.packed.data_ptr(), _stream_of(q)))
        self.error = torch.zeros(1, dtype=torch.int32, device=q.device)
        self.desc = dh_matmul_t(self.N, self.K, self.packed.data_ptr(), g.data_ptr())
        self.desc_ref, self.error_ptr = C.byref(self.desc), self.error.data_ptr()

    @classmethod
    def from_weight(cls, W: torch.Tensor, idx: torch.Tensor | None = None, stream=None) -> "NVFP4Matmul":
        """Quantise the rows W[idx] (all rows without idx) of a bfloat16 weight [V, K]."""
        if stream is not None:
            new = _on_stream(stream, cls.from_weight, W, idx)
            _keep_for(torch.cuda.current_stream(stream.device), new.packed, new.g, new.error)
            return new
        if W.is_cuda:
            _stream_of(W)   # refuses before the first launch
        if idx is None:
            idx = torch.arange(W.shape[0], dtype=torch.int32, device=W.device)
        return cls(*nvfp4_quantize_rows(W, idx))

    def forward(self, x: torch.Tensor, y: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                stream=None) -> torch.Tensor:
        """y [M, N] (out_dtype: bfloat16, float16 or float32, or a given tensor's
        type) = x W'^T for x [M, K] (bfloat16, float16 or float32, rows may be strided)."""
        if stream is not None:
            _keep_for(stream, self.packed, self.g, self.error)
            return _on_stream(stream, self.forward, x, y, out_dtype)
        if x.dim() != 2 or x.shape[1] != self.K or x.dtype not in _TYPES or x.device != self.packed.device or \
                x.stride(1) != 1 or (x.shape[0] > 1 and x.stride(0) < self.K):
            raise ValueError(f"x must be a [M, {self.K}] bfloat16, float16 or float32 tensor with contiguous rows")
        _no_gradient(x, "the activations")
        M = x.shape[0]
        if y is None:
            if out_dtype not in _TYPES:
                raise ValueError("out_dtype must be bfloat16, float16 or float32")
            y = torch.empty((M, self.N), dtype=out_dtype, device=x.device)
        elif y.shape != (M, self.N) or y.dtype not in _TYPES or y.device != x.device or y.stride(1) != 1 or \
                (M > 1 and y.stride(0) < self.N):
            raise ValueError(f"y must be a [{M}, {self.N}] bfloat16, float16 or float32 tensor with contiguous rows")
        if M == 0:
            return y
        L = lib()
        nb = L.nvfp4_matmul_workspace_bytes(M, self.K)
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device)   # the allocator's blocks are 512-byte aligned
        _check("nvfp4_matmul",
               L.nvfp4_matmul(self.desc_ref, x.data_ptr(), _TYPES[x.dtype], x.stride(0), M, y.data_ptr(),
                                  _TYPES[y.dtype], y.stride(0), ws.data_ptr(), nb, self.error_ptr, _stream_of(x)))
        return y

    __call__ = forward

    def wait_probe(self, x: torch.Tensor, role: int, rounds: int) -> None:
        """Enqueue the self-test of the product's bounded waits on x [M, K] (bfloat16,
        contiguous): `role` of the kernel's warps does nothing (see nvfp4_matmul_wait_probe);
        device_error() tells how it ended."""
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.K or x.device != self.packed.device or \
                not x.is_contiguous():
            raise ValueError(f"x must be a contiguous [M, {self.K}] bfloat16 tensor")
        M = x.shape[0]
        y = torch.empty((M, self.N), dtype=torch.bfloat16, device=x.device)
        nb = lib().nvfp4_matmul_workspace_bytes(M, self.K)
        ws = torch.empty(nb, dtype=torch.uint8, device=x.device)
        _check("nvfp4_matmul_wait_probe",
               lib().nvfp4_matmul_wait_probe(self.desc_ref, x.data_ptr(), M, y.data_ptr(), ws.data_ptr(), nb, role, rounds,
                                             self.error_ptr, _stream_of(x)))

    def device_error(self) -> int:
        """Read and clear the device error word (waits for the device: products may be
        pending on any stream)."""
        torch.cuda.synchronize(self.error.device)
        err = int(self.error.item())
        if err:
            self.error.zero_()
        return err


def _logits_desc(logits: torch.Tensor, temperature: float, row_of: torch.Tensor | None,
                 idx: torch.Tensor | None = None) -> bytes:
    """The dh_logits_t of logits [M, C], as bytes."""
    dtype = _TYPES.get(logits.dtype)
    if logits.dim() != 2 or dtype is None or not logits.is_cuda:
        raise ValueError("logits must be a [M, C] bfloat16, float16 or float32 CUDA tensor")
    M, n = logits.shape
    ld, step = logits.stride()
    if (step != 1 and n > 1) or (M > 1 and ld < n):
        raise ValueError("logits rows must be contiguous and must not overlap")
    V = 0
    if row_of is not None:
        _vector(row_of, "row_of", torch.int32, None, logits.device)
        V = row_of.numel()
    if idx is not None:
        _vector(idx, "idx", torch.int32, None, logits.device)
        if idx.numel() < n:
            raise ValueError(f"idx must hold the ids of all {n} columns")
    try:
        return _pack_logits(logits.data_ptr(), dtype, M, n, ld, temperature, _ptr(row_of) or 0, V, _ptr(idx) or 0)
    except (struct.error, OverflowError):   # a size past 32 bits, a temperature that fp32 does not hold or no number
        raise DraftHeadError("dh_logits_t", DH_ERR_SHAPE if max(M, n, V) >= 2 ** 31 else DH_ERR_ARG) from None


def draft_head_row_map(idx: torch.Tensor, n_kept: int, V: int, stream=None) -> torch.Tensor:
    """int32[V]: the head row (logits column) of every target id, -1 for ids that
    are not kept; the row_of argument of the operators below."""
    if stream is not None:
        return _on_stream(stream, draft_head_row_map, idx, n_kept, V)
    if idx.dtype != torch.int32 or idx.dim() != 1 or not idx.is_cuda or not idx.is_contiguous() or idx.numel() < n_kept:
        raise ValueError(f"idx must be a contiguous int32 CUDA vector of at least {n_kept} elements")
    row_of = torch.empty(V, dtype=torch.int32, device=idx.device)
    _check("draft_head_row_map",
           lib().draft_head_row_map(idx.data_ptr(), n_kept, row_of.data_ptr(), V, _stream_of(idx)))
    return row_of


class TokenLogprobs(NamedTuple):
    """Results of token_logprobs for M rows: logp float32 [M, G] (None without
    tokens), entropy and lse float32 [M], top_logp float32 and top_ids int32 [M, top_k]."""
    logp: torch.Tensor | None
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logp: torch.Tensor
    top_ids: torch.Tensor


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top_k: int = 0, temperature: float = 1.0,
                   idx: torch.Tensor | None = None, row_of: torch.Tensor | None = None, stream=None) -> TokenLogprobs:
    """Log-probabilities of `tokens` (int32 [M] or [M, G]), entropy, normaliser and
    the top_k alternatives of logits rows [M, C] (rows may be strided; pass
    logits[:, :n_kept] to leave a head's padding rows out). With row_of
    (draft_head_row_map) tokens are target ids, with idx (dh_idx) the alternatives
    are returned as target ids; without them both are columns. A token without a
    column has log-probability -inf; alternatives past the last logit above -inf
    have id -1. No gradient: logits that require one are refused. See
    draft_head_token_logprobs."""
    if stream is not None:
        return _on_stream(stream, token_logprobs, logits, tokens, top_k, temperature, idx, row_of)
    _no_gradient(logits, "the logits")
    d = _logits_desc(logits, temperature, row_of, idx)
    M, dev, f32 = logits.shape[0], logits.device, torch.float32
    G = 0
    if tokens is not None:
        if tokens.dim() not in (1, 2) or tokens.shape[0] != M:
            raise ValueError(f"tokens must be an int32 tensor [{M}] or [{M}, G]")
        _vector(tokens, "tokens", torch.int32, None, dev)
        G = 1 if tokens.dim() == 1 else tokens.shape[1]
    if not 0 <= top_k <= DH_MAX_TOP:
        raise ValueError(f"top_k must lie in 0 .. {DH_MAX_TOP}")
    logp = None if tokens is None else torch.empty(tokens.shape, dtype=f32, device=dev)
    entropy, lse = torch.empty(M, dtype=f32, device=dev), torch.empty(M, dtype=f32, device=dev)
    top_logp = torch.empty((M, top_k), dtype=f32, device=dev)
    top_ids = torch.empty((M, top_k), dtype=torch.int32, device=dev)
    if M > 0:
        _check("draft_head_token_logprobs",
               lib().draft_head_token_logprobs(d, _ptr(tokens), G, _ptr(logp), entropy.data_ptr(), lse.data_ptr(), top_k,
                                               top_logp.data_ptr(), top_ids.data_ptr(), _stream_of(logits)))
    return TokenLogprobs(logp, entropy, lse, top_logp, top_ids)


def _teacher(logits, ids, val):
    shape = ids.shape
    if len(shape) != 2 or shape[0] != logits.shape[0] or val.shape != shape:
        raise ValueError(f"teacher ids and logits must be [{logits.shape[0]}, K] tensors")
    _vector(ids, "teacher ids", torch.int32, None, logits.device)
    if val.dtype not in _TYPES:
        raise ValueError("teacher logits must be bfloat16, float16 or float32")
    _vector(val, "teacher logits", val.dtype, None, logits.device)
    if not 1 <= ids.shape[1] <= DH_MAX_TEACHER:
        raise ValueError(f"a row takes 1 .. {DH_MAX_TEACHER} teacher entries")
    return ids.shape[1], _TYPES[val.dtype]


def _gradient(logits: torch.Tensor, out: torch.Tensor | None) -> torch.Tensor:
    """The caller's gradient buffer, checked, or a new one with the logits' row stride."""
    M, n = logits.shape
    if out is None:
        ld = logits.stride(0)
        if not n <= ld <= 2 * n:     # one row, or rows far apart: whole 16-byte vectors per row
            ld = (n + 7) // 8 * 8
        return torch.empty_strided((M, n), (ld, 1), dtype=logits.dtype, device=logits.device)
    if out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device or \
            (out.stride(1) != 1 and n > 1) or (M > 1 and out.stride(0) < n):
        raise ValueError("the gradient must be a tensor of the logits' shape, type and device with contiguous rows")
    return out


def distill_topk(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, temperature: float = 1.0,
                 weights: torch.Tensor | None = None, row_of: torch.Tensor | None = None,
                 dlogits: torch.Tensor | None = None, stream=None):
    """(loss float32 [M], dlogits [M, C]): per-row distillation loss of the
    student's logits [M, C] from the teacher's top K ids (int32 [M, K]) and logits
    [M, K], and the gradient of its sum, in one kernel. Ids are target ids with
    row_of, columns without it; entries without a column, and masked (-inf) ones,
    leave the teacher's distribution. weights: float32 [M], 0 for rows to leave
    out. dlogits may be the logits tensor itself. The loss has no autograd graph
    (the gradient is at hand; DistillTopK is the differentiable form). See
    draft_head_distill."""
    if stream is not None:
        return _on_stream(stream, distill_topk, logits, teacher_ids, teacher_logits, temperature, weights, row_of, dlogits)
    d = _logits_desc(logits, temperature, row_of)
    K, vt = _teacher(logits, teacher_ids, teacher_logits)
    _vector(weights, "weights", torch.float32, logits.shape[0], logits.device)
    dz = _gradient(logits, dlogits)
    loss = torch.empty(logits.shape[0], dtype=torch.float32, device=logits.device)
    if logits.shape[0] > 0:
        _check("draft_head_distill",
               lib().draft_head_distill(d, teacher_ids.data_ptr(), teacher_logits.data_ptr(), vt, K, _ptr(weights),
                                        loss.data_ptr(), None, dz.data_ptr(), dz.stride(0), _stream_of(logits)))
    return loss, dz


def distill_topk_forward(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                         temperature: float = 1.0, weights: torch.Tensor | None = None,
                         row_of: torch.Tensor | None = None, stream=None):
    """(loss, lse), both float32 [M]: the loss of distill_topk alone, and the
    student's normaliser for distill_topk_backward."""
    if stream is not None:
        return _on_stream(stream, distill_topk_forward, logits, teacher_ids, teacher_logits, temperature, weights, row_of)
    d = _logits_desc(logits, temperature, row_of)
    K, vt = _teacher(logits, teacher_ids, teacher_logits)
    _vector(weights, "weights", torch.float32, logits.shape[0], logits.device)
    M, dev = logits.shape[0], logits.device
    loss, lse = torch.empty(M, dtype=torch.float32, device=dev), torch.empty(M, dtype=torch.float32, device=dev)
    if logits.shape[0] > 0:
        _check("draft_head_distill",
               lib().draft_head_distill(d, teacher_ids.data_ptr(), teacher_logits.data_ptr(), vt, K, _ptr(weights),
                                        loss.data_ptr(), lse.data_ptr(), None, 0, _stream_of(logits)))
    return loss, lse


def distill_topk_backward(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, lse: torch.Tensor,
                          weights: torch.Tensor | None = None, temperature: float = 1.0,
                          row_of: torch.Tensor | None = None, dlogits: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """dlogits [M, C] from distill_topk_forward's lse; weights: float32 [M], the
    upstream gradient of each row's loss times the forward's weight."""
    if stream is not None:
        return _on_stream(stream, distill_topk_backward, logits, teacher_ids, teacher_logits, lse, weights, temperature, row_of,
                          dlogits)
    d = _logits_desc(logits, temperature, row_of)
    K, vt = _teacher(logits, teacher_ids, teacher_logits)
    _vector(lse, "lse", torch.float32, logits.shape[0], logits.device)
    _vector(weights, "weights", torch.float32, logits.shape[0], logits.device)
    dz = _gradient(logits, dlogits)
    if logits.shape[0] > 0:
        _check("draft_head_distill_backward",
               lib().draft_head_distill_backward(d, teacher_ids.data_ptr(), teacher_logits.data_ptr(), vt, K,
                                                 lse.data_ptr(), _ptr(weights), dz.data_ptr(), dz.stride(0),
                                                 _stream_of(logits)))
    return dz


class _Refuse(torch.autograd.Function):
    """A tensor whose gradient is refused: a backward pass that comes back to it, or
    by it to the sources that it was computed from, raises."""

    @staticmethod
    def forward(ctx, message, tensor, *sources):
        ctx.message = message
        return tensor.view_as(tensor)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(ctx.message)


class DistillTopK(torch.autograd.Function):
    """loss [M] = DistillTopK.apply(logits, teacher_ids, teacher_logits, temperature,
    weights, row_of); differentiable once in the logits and the weights (the teacher
    is a constant: a backward pass that would reach its logits raises, detach them). A
    weight's derivative is the loss that its row has at weight 1."""

    @classmethod
    def apply(cls, logits, teacher_ids, teacher_logits, *rest):
        if teacher_logits.requires_grad and torch.is_grad_enabled():
            teacher_logits = _Refuse.apply("DistillTopK has no gradient for the teacher's logits: detach them", teacher_logits)
        return super().apply(logits, teacher_ids, teacher_logits, *rest)

    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_logits, temperature=1.0, weights=None, row_of=None):
        loss, lse = distill_topk_forward(logits, teacher_ids, teacher_logits, temperature, weights, row_of)
        ctx.save_for_backward(logits, teacher_ids, teacher_logits, lse, weights, row_of)
        ctx.temperature = temperature
        return loss

    @staticmethod
    def backward(ctx, dloss):
        logits, ids, val, lse, weights, row_of = ctx.saved_tensors
        dz = dw = None
        with torch.no_grad():
            up = dloss.float()
            if ctx.needs_input_grad[0]:
                w = (up if weights is None else up * weights).contiguous()
                dz = distill_topk_backward(logits, ids, val, lse, w, ctx.temperature, row_of)
            if weights is not None and ctx.needs_input_grad[4]:
                dw = up * distill_topk_forward(logits, ids, val, ctx.temperature, None, row_of)[0]
        if torch.is_grad_enabled():   # the caller asked for the gradients' graph
            dz, dw = (None if d is None else _Refuse.apply("DistillTopK is differentiable once: its gradient has no derivative",
                                                           d, logits, dloss, weights) for d in (dz, dw))
        return dz, None, None, None, dw, None
