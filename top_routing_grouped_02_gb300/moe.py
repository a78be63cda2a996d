"""Thin ctypes binding over libmoe.so (include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. (The sub-block calls at the end of the file marshal in _native.so.) Tensors must be contiguous CUDA tensors of the dtype each call names;
their ``data_ptr()`` and the current torch stream are passed straight through.
There is no fallback: if libmoe.so is missing or a call fails, a ``MoeError``
is raised.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe.h")

MOE_OK = 0
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_ARCH", 5: "MOE_ERR_CUDA",
          6: "MOE_ERR_DEVICE_TIMEOUT", 7: "MOE_ERR_DEVICE_CHECK"}
# Kernels each call enqueues; the gate/up GEMM launches one more (a row gather)
# when it runs on CTA pairs, the router's backward one fewer when T is too
# short to split into chunks, moe_ffn one for few tokens, moe_permute one kernel instead of three for
# T <= 65536, moe_linear_backward one to four (moe.h), the norms' backward one without weights'
# gradients, and the whole-layer calls depend on the shape (forward_launches).
LAUNCHES = {"moe_route": 2, "moe_route_logits": 1, "moe_permute": 3, "moe_gemm_gate_up": 1,
            "moe_gemm_gate_up_train": 1, "moe_backward_dh": 2, "moe_backward_dx": 2,
            "moe_backward_router": 5, "moe_backward_dw": 5,
            "moe_gemm_down": 1, "moe_combine": 1, "moe_round_routing": 3, "moe_combine_rows": 1,
            "moe_layernorm": 1, "moe_layernorm_backward": 2, "moe_dropout": 1,
            "moe_dropout_backward": 1, "moe_ffn": 2, "moe_ffn_train": 2, "moe_ffn_backward": 3,
            "moe_linear": 1, "moe_linear_train": 1, "moe_linear_backward": 3,
            "moe_block_norm": 1, "moe_block_norm_backward": 2, "moe_rmsnorm": 1,
            "moe_rmsnorm_backward": 2, "moe_dispatch": 1, "moe_combine_weighted": 1, "moe_combine_weighted_backward": 1}
TILE_M = 128


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)}")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_L = ctypes.c_int64
_U = ctypes.c_uint64
_F = ctypes.c_float
_D = ctypes.c_double
_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_abi_version": (_I, []),
    "moe_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_forward_launches": (_I, [_I, _I, _I, _I, _I, _I]),
    "moe_expert_mlp_launches": (_I, [_I, _I, _I, _I, _I, _I]),
    "moe_workspace_init": (_I, [_P, _SZ, _P]),
    "moe_route": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_route_logits": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_permute": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_permute_noalloc": (_I, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "moe_gemm_gate_up": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_gemm_down": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_gemm_gate_up_train": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ,
                                    _P]),
    "moe_backward_dh": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                             _SZ, _P]),
    "moe_backward_dx": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_backward_router": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P,
                                 _P, _SZ, _P]),
    "moe_backward_dw_scratch_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_backward_dw": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P,
                             _P, _SZ, _P]),
    "moe_expert_mlp": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ,
                            _P]),
    "moe_combine": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "moe_forward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ,
                         _P]),
    "moe_forward_traced": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                _SZ, _P, ctypes.POINTER(_P), _I]),
    "moe_forward_host": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ,
                              _P]),
    "moe_sync_check": (_I, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "moe_selftest_wait_timeout": (_I, [_P, _SZ, _P]),
    "moe_selftest_layernorm_withhold": (_I, [_L]),
    "moe_forward_host_stream": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                     _I, _P, _SZ, _P, _P, _P]),
    "moe_layernorm_forward": (_I, [_P, _L, _P, _P, _L, _I, _F, _I, _I, _P, _L, _P, _P, _P]),
    "moe_layernorm_scratch_bytes": (_SZ, [_L, _I]),
    "moe_layernorm_backward": (_I, [_P, _L, _P, _L, _P, _P, _P, _P, _L, _L, _I, _I, _I, _P, _L, _P,
                                    _P, _P, _SZ, _P]),
    "moe_dropout": (_I, [_P, _L, _P, _L, _L, _I, _D, _U, _U, _P, _I, _P, _L, _P]),
    "moe_dropout_backward": (_I, [_P, _L, _L, _I, _D, _U, _U, _P, _I, _P, _L, _P]),
    "moe_ffn_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_ffn_saved_floats": (_SZ, [_I, _I]),
    "moe_ffn_workspace_init": (_I, [_P, _SZ, _P]),
    "moe_ffn_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_ffn_forward_train": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ,
                                   _P]),
    "moe_ffn_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                              _P, _SZ, _P]),
    "moe_linear_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_linear_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_linear_forward_train": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_linear_backward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_block_norm_forward": (_I, [_P, _L, _P, _L, _P, _L, _I, _P, _P, _F, _I, _L, _I, _F, _I, _I,
                                    _P, _L, _P, _L, _P, _P, _P]),
    "moe_block_norm_scratch_bytes": (_SZ, [_L, _I]),
    "moe_block_norm_backward": (_I, [_P, _L, _P, _L, _P, _L, _P, _L, _P, _L, _I, _P, _P, _F, _I, _P,
                                     _P, _L, _I, _I, _I, _P, _L, _P, _L, _P, _L, _P, _P, _P, _SZ,
                                     _P]),
    "moe_dispatch": (_I, [_P, _L, _P, _L, _I, _I, _I, _P, _L, _L, _P]),
    "moe_combine_weighted": (_I, [_P, _L, _L, _P, _P, _P, _L, _L, _I, _I, _I, _P, _L, _P]),
    "moe_combine_weighted_backward": (_I, [_P, _L, _P, _L, _L, _P, _P, _L, _I, _I, _I, _P, _L, _P,
                                           _P]),
    "moe_round_capacity": (ctypes.c_int64, [_I, _I, _I, _I]),
    "moe_round_workspace_bytes": (_SZ, [_I, _I]),
    "moe_round_routing": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                               _P]),
    "moe_combine_rows": (_I, [_P, _P, _I, _I, _I, ctypes.c_int64, _P, _P]),
    "moe_workspace_bytes_rounded": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_forward_rounded": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ,
                                 _P]),
    "moe_forward_rounded_traced": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P,
                                        _SZ, _P, ctypes.POINTER(_P), _I]),
}


def header_symbols() -> list[str]:
    """Entry points declared in include/moe.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]+?\b(moe_\w+)\s*\(", text, re.M)))


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def moe_workspace_bytes(T: int, d: int, E: int, K: int, n: int) -> int:
    return int(lib().moe_workspace_bytes(T, d, E, K, n))


def forward_launches(T: int, d: int, E: int, K: int, n: int, rounded: bool = False,
                     part: str = "forward") -> int:
    """Kernels moe_forward (or moe_forward_rounded) enqueues for this shape on the
    current device under the current environment (host only); part="expert_mlp":
    the expert GEMMs' share (1 when fused)."""
    fn = lib().moe_forward_launches if part == "forward" else lib().moe_expert_mlp_launches
    v = int(fn(T, d, E, K, n, int(rounded)))
    if v < 0:
        raise ValueError("invalid layer shape")
    return v


def workspace(T: int, d: int, E: int, K: int, n: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor (uint8) for this layer shape."""
    nbytes = moe_workspace_bytes(T, d, E, K, n)
    if nbytes == 0:
        raise ValueError("invalid layer shape")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check("moe_workspace_init", lib().moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)))


def moe_route(X, Wr, K: int, bias=None, renorm: bool = True, stream=None, logits=None):
    """(topk_idx [T,K] int32, topk_w [T,K] fp32, counts [E] int32); the router
    logits [T,E] fp32 land in `logits` (allocated when not given)."""
    T, d = X.shape
    E = Wr.shape[1]
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=X.device)
    idx = torch.empty((T, K), dtype=torch.int32, device=X.device)
    w = torch.empty((T, K), dtype=torch.float32, device=X.device)
    counts = torch.empty(E, dtype=torch.int32, device=X.device)
    _check("moe_route", lib().moe_route(
        _ptr(X, torch.bfloat16, "X"), _ptr(Wr, torch.float32, "Wr"), _ptr(bias, torch.float32, "bias"),
        T, d, E, K, int(bool(renorm)), _ptr(logits, torch.float32, "logits"), _ptr(idx), _ptr(w),
        _ptr(counts), _stream(stream)))
    return idx, w, counts


def moe_route_logits(logits, K: int, renorm: bool = True, stream=None):
    T, E = logits.shape
    idx = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    counts = torch.empty(E, dtype=torch.int32, device=logits.device)
    _check("moe_route_logits", lib().moe_route_logits(
        _ptr(logits, torch.float32, "logits"), T, E, K, int(bool(renorm)), _ptr(idx), _ptr(w),
        _ptr(counts), _stream(stream)))
    return idx, w, counts


def moe_permute(topk_idx, E: int, counts=None, ws=None, stream=None) -> dict:
    T, K = topk_idx.shape
    R = T * K
    dev = topk_idx.device
    if ws is None:
        ws = workspace(T, 0, E, K, 0, dev)
    out = dict(
        offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
        perm_token=torch.empty(R, dtype=torch.int32, device=dev),
        perm_slot=torch.empty(R, dtype=torch.int32, device=dev),
        row_of_slot=torch.empty(R, dtype=torch.int32, device=dev),
        tiles=torch.zeros((R // TILE_M + E, 4), dtype=torch.int32, device=dev),
        num_tiles=torch.empty(1, dtype=torch.int32, device=dev),
    )
    _check("moe_permute", lib().moe_permute(
        _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(counts, torch.int32, "counts"), T, E, K,
        _ptr(out["offsets"]), _ptr(out["perm_token"]), _ptr(out["perm_slot"]),
        _ptr(out["row_of_slot"]), _ptr(out["tiles"]), _ptr(out["num_tiles"]), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def moe_permute_noalloc(topk_idx, E: int, counts=None, out: dict | None = None, stream=None) -> dict:
    """moe_permute without a workspace: the library uses its built-in 4 MiB
    scratch array, so this call allocates no device memory of its own. `out`
    may hold preallocated output tensors (same keys as moe_permute returns)."""
    T, K = topk_idx.shape
    R = T * K
    dev = topk_idx.device
    if out is None:
        out = dict(
            offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            perm_token=torch.empty(R, dtype=torch.int32, device=dev),
            perm_slot=torch.empty(R, dtype=torch.int32, device=dev),
            row_of_slot=torch.empty(R, dtype=torch.int32, device=dev),
            tiles=torch.zeros((R // TILE_M + E, 4), dtype=torch.int32, device=dev),
            num_tiles=torch.empty(1, dtype=torch.int32, device=dev),
        )
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(
        _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(counts, torch.int32, "counts"), T, E, K,
        _ptr(out["offsets"]), _ptr(out["perm_token"]), _ptr(out["perm_slot"]),
        _ptr(out["row_of_slot"]), _ptr(out["tiles"]), _ptr(out["num_tiles"]), _stream(stream)))
    return out


def moe_gemm_gate_up(X, W1, W3, perm_token, offsets, K: int, ws=None, stream=None):
    T, d = X.shape
    E, _, n = W1.shape
    if ws is None:
        ws = workspace(T, d, E, K, n, X.device)
    H = torch.empty((T * K, n), dtype=torch.bfloat16, device=X.device)
    _check("moe_gemm_gate_up", lib().moe_gemm_gate_up(
        _ptr(X, torch.bfloat16, "X"), _ptr(W1, torch.bfloat16, "W1"), _ptr(W3, torch.bfloat16, "W3"),
        _ptr(perm_token, torch.int32), _ptr(offsets, torch.int32), T, d, E, K, n, _ptr(H),
        _ptr(ws), ws.numel(), _stream(stream)))
    return H


def moe_gemm_gate_up_train(X, W1, W3, perm_token, offsets, K: int, ws=None, stream=None):
    """(H [T*K, n] bf16, A1, A3 [T*K, n] fp32): H as moe_gemm_gate_up gives it
    and the pre-activations x W1[e], x W3[e] of every grouped row."""
    T, d = X.shape
    E, _, n = W1.shape
    if ws is None:
        ws = workspace(T, d, E, K, n, X.device)
    H = torch.empty((T * K, n), dtype=torch.bfloat16, device=X.device)
    A1, A3 = (torch.empty((T * K, n), dtype=torch.float32, device=X.device) for _ in range(2))
    _check("moe_gemm_gate_up_train", lib().moe_gemm_gate_up_train(
        _ptr(X, torch.bfloat16, "X"), _ptr(W1, torch.bfloat16, "W1"), _ptr(W3, torch.bfloat16, "W3"),
        _ptr(perm_token, torch.int32, "perm_token"), _ptr(offsets, torch.int32, "offsets"),
        T, d, E, K, n, _ptr(H), _ptr(A1), _ptr(A3), _ptr(ws), ws.numel(), _stream(stream)))
    return H, A1, A3


def moe_backward_dh(dY, W2, A1, A3, topk_w, perm_token, perm_slot, offsets, K: int, ws=None,
                    stream=None):
    """(dA1, dA3 [T*K, n] bf16, dS [T*K] fp32) of the grouped rows: the backward's
    dH step with the routing-weight gradient."""
    T, d = dY.shape
    E, n, _ = W2.shape
    if ws is None:
        ws = workspace(T, d, E, K, n, dY.device)
    dA1, dA3 = (torch.empty((T * K, n), dtype=torch.bfloat16, device=dY.device) for _ in range(2))
    dS = torch.zeros(T * K, dtype=torch.float32, device=dY.device)
    _check("moe_backward_dh", lib().moe_backward_dh(
        _ptr(dY, torch.bfloat16, "dY"), _ptr(W2, torch.bfloat16, "W2"), _ptr(A1, torch.float32, "A1"),
        _ptr(A3, torch.float32, "A3"), _ptr(topk_w, torch.float32, "topk_w"),
        _ptr(perm_token, torch.int32, "perm_token"), _ptr(perm_slot, torch.int32, "perm_slot"),
        _ptr(offsets, torch.int32, "offsets"), T, d, E, K, n, _ptr(dA1), _ptr(dA3), _ptr(dS),
        _ptr(ws), ws.numel(), _stream(stream)))
    return dA1, dA3, dS


def moe_backward_dx(dA1, dA3, W1, W3, offsets, row_of_slot, K: int, ws=None, stream=None):
    """(dXg [T*K, d] bf16 grouped rows, dX [T, d] bf16): the experts' share of the
    input gradient."""
    R, n = dA1.shape
    E, d, _ = W1.shape
    T = R // K
    if ws is None:
        ws = torch.zeros(256, dtype=torch.uint8, device=dA1.device)
    dXg = torch.empty((R, d), dtype=torch.bfloat16, device=dA1.device)
    dX = torch.empty((T, d), dtype=torch.bfloat16, device=dA1.device)
    _check("moe_backward_dx", lib().moe_backward_dx(
        _ptr(dA1, torch.bfloat16, "dA1"), _ptr(dA3, torch.bfloat16, "dA3"),
        _ptr(W1, torch.bfloat16, "W1"), _ptr(W3, torch.bfloat16, "W3"),
        _ptr(offsets, torch.int32, "offsets"), _ptr(row_of_slot, torch.int32, "row_of_slot"),
        T, d, E, K, n, _ptr(dXg), _ptr(dX), _ptr(ws), ws.numel(), _stream(stream)))
    return dXg, dX


def moe_backward_router(X, Wr, logits, topk_idx, dS, row_of_slot, dXg, renorm: bool = True,
                        ws=None, stream=None) -> dict:
    """The router's backward and the full input gradient: dict of dX [T, d] bf16,
    dL [T, E], dWr [d, E], dbias [E] fp32."""
    T, d = X.shape
    E = Wr.shape[1]
    K = topk_idx.shape[1]
    if ws is None:
        ws = workspace(T, d, E, K, 0, X.device)
    out = dict(dX=torch.empty((T, d), dtype=torch.bfloat16, device=X.device),
               dL=torch.empty((T, E), dtype=torch.float32, device=X.device),
               dWr=torch.empty((d, E), dtype=torch.float32, device=X.device),
               dbias=torch.empty(E, dtype=torch.float32, device=X.device))
    _check("moe_backward_router", lib().moe_backward_router(
        _ptr(X, torch.bfloat16, "X"), _ptr(Wr, torch.float32, "Wr"),
        _ptr(logits, torch.float32, "logits"), _ptr(topk_idx, torch.int32, "topk_idx"),
        _ptr(dS, torch.float32, "dS"), _ptr(row_of_slot, torch.int32, "row_of_slot"),
        T, d, E, K, int(bool(renorm)), _ptr(dXg, torch.bfloat16, "dXg"), _ptr(out["dX"]),
        _ptr(out["dL"]), _ptr(out["dWr"]), _ptr(out["dbias"]), _ptr(ws), ws.numel(),
        _stream(stream)))
    return out


def moe_backward_dw(X, dY, H, dA1, dA3, topk_w, perm_token, perm_slot, offsets, K: int,
                    scratch=None, stream=None) -> dict:
    """Weight gradients dW1, dW3 [E, d, n] and dW2 [E, n, d], fp32."""
    T, d = X.shape
    E = offsets.shape[0] - 1
    n = dA1.shape[1]
    if scratch is None:
        nbytes = int(lib().moe_backward_dw_scratch_bytes(T, d, E, K))
        scratch = torch.zeros(nbytes, dtype=torch.uint8, device=X.device)
    out = dict(dW1=torch.empty((E, d, n), dtype=torch.float32, device=X.device),
               dW3=torch.empty((E, d, n), dtype=torch.float32, device=X.device),
               dW2=torch.empty((E, n, d), dtype=torch.float32, device=X.device))
    _check("moe_backward_dw", lib().moe_backward_dw(
        _ptr(X, torch.bfloat16, "X"), _ptr(dY, torch.bfloat16, "dY"), _ptr(H, torch.bfloat16, "H"),
        _ptr(dA1, torch.bfloat16, "dA1"), _ptr(dA3, torch.bfloat16, "dA3"),
        _ptr(topk_w, torch.float32, "topk_w"), _ptr(perm_token, torch.int32, "perm_token"),
        _ptr(perm_slot, torch.int32, "perm_slot"), _ptr(offsets, torch.int32, "offsets"),
        T, d, E, K, n, _ptr(out["dW1"]), _ptr(out["dW3"]), _ptr(out["dW2"]), _ptr(scratch),
        scratch.numel(), _stream(stream)))
    out["scratch"] = scratch
    return out


def moe_gemm_down(H, W2, topk_w, perm_slot, offsets, T: int, K: int, ws=None, stream=None):
    E, n, d = W2.shape
    if ws is None:
        ws = workspace(T, d, E, K, n, H.device)
    Z = torch.empty((T * K, d), dtype=torch.bfloat16, device=H.device)
    _check("moe_gemm_down", lib().moe_gemm_down(
        _ptr(H, torch.bfloat16, "H"), _ptr(W2, torch.bfloat16, "W2"), _ptr(topk_w, torch.float32),
        _ptr(perm_slot, torch.int32), _ptr(offsets, torch.int32), T, d, E, K, n, _ptr(Z),
        _ptr(ws), ws.numel(), _stream(stream)))
    return Z


def moe_expert_mlp(X, W1, W3, W2, topk_w, perm_token, perm_slot, offsets, K: int, ws=None,
                   stream=None):
    T, d = X.shape
    E, _, n = W1.shape
    if ws is None:
        ws = workspace(T, d, E, K, n, X.device)
    H = torch.empty((T * K, n), dtype=torch.bfloat16, device=X.device)
    Z = torch.empty((T * K, d), dtype=torch.bfloat16, device=X.device)
    _check("moe_expert_mlp", lib().moe_expert_mlp(
        _ptr(X, torch.bfloat16), _ptr(W1, torch.bfloat16), _ptr(W3, torch.bfloat16),
        _ptr(W2, torch.bfloat16), _ptr(topk_w, torch.float32), _ptr(perm_token, torch.int32),
        _ptr(perm_slot, torch.int32), _ptr(offsets, torch.int32), T, d, E, K, n, _ptr(H), _ptr(Z),
        _ptr(ws), ws.numel(), _stream(stream)))
    return H, Z


def moe_combine(Z, row_of_slot, K: int, stream=None):
    R, d = Z.shape
    T = row_of_slot.numel() // K
    Y = torch.empty((T, d), dtype=torch.bfloat16, device=Z.device)
    _check("moe_combine", lib().moe_combine(
        _ptr(Z, torch.bfloat16, "Z"), _ptr(row_of_slot, torch.int32), T, K, d, _ptr(Y),
        _stream(stream)))
    return Y


def moe_forward(X, Wr, W1, W3, W2, K: int, bias=None, renorm: bool = True, ws=None, Y=None,
                topk_idx=None, topk_w=None, stream=None, events=None):
    """Y [T,d] bf16 for the whole layer. Optional topk_idx/topk_w receive the
    routing; `events` (list of torch.cuda.Event) are recorded between stages."""
    T, d = X.shape
    E, _, n = W1.shape
    if ws is None:
        ws = workspace(T, d, E, K, n, X.device)
    if Y is None:
        Y = torch.empty((T, d), dtype=torch.bfloat16, device=X.device)
    args = (_ptr(X, torch.bfloat16, "X"), _ptr(Wr, torch.float32, "Wr"),
            _ptr(bias, torch.float32, "bias"), _ptr(W1, torch.bfloat16, "W1"),
            _ptr(W3, torch.bfloat16, "W3"), _ptr(W2, torch.bfloat16, "W2"), T, d, E, K, n,
            int(bool(renorm)), _ptr(Y, torch.bfloat16, "Y"), _ptr(topk_idx, torch.int32),
            _ptr(topk_w, torch.float32), _ptr(ws), ws.numel(), _stream(stream))
    if events:
        for e in events:
            if e.cuda_event == 0:  # torch creates the CUDA event on first record
                e.record()
        arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
        _check("moe_forward_traced", lib().moe_forward_traced(*args, arr, len(events)))
    else:
        _check("moe_forward", lib().moe_forward(*args))
    return Y


def moe_forward_host(X_host, Y_host, X_dev, Y_dev, Wr, W1, W3, W2, K: int, bias=None,
                     renorm: bool = True, ws=None, stream=None):
    """End to end from host memory (X_host/Y_host CPU bf16 tensors, ideally pinned);
    returns after Y_host holds the result."""
    T, d = X_host.shape
    E, _, n = W1.shape
    for name, t in (("X_host", X_host), ("Y_host", Y_host)):
        if t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be a contiguous CPU bf16 tensor")
    if ws is None:
        ws = workspace(T, d, E, K, n, X_dev.device)
    _check("moe_forward_host", lib().moe_forward_host(
        ctypes.c_void_p(X_host.data_ptr()), ctypes.c_void_p(Y_host.data_ptr()),
        _ptr(X_dev, torch.bfloat16), _ptr(Y_dev, torch.bfloat16), _ptr(Wr, torch.float32),
        _ptr(bias, torch.float32), _ptr(W1, torch.bfloat16), _ptr(W3, torch.bfloat16),
        _ptr(W2, torch.bfloat16), T, d, E, K, n, int(bool(renorm)), _ptr(ws), ws.numel(),
        _stream(stream)))
    return Y_host


def moe_forward_host_stream(X_host, Y_host, X_dev2, Y_dev2, Wr, W1, W3, W2, K: int, bias=None,
                            renorm: bool = True, ws=None, stream=None, h2d_stream=None,
                            d2h_stream=None):
    """n batches from host memory with copies overlapped: X_host / Y_host are CPU
    bf16 [n, T, d] (pinned), X_dev2 / Y_dev2 CUDA bf16 [2, T, d]. Returns after
    Y_host holds every output."""
    nb, T, d = X_host.shape
    E, _, n = W1.shape
    for name, t in (("X_host", X_host), ("Y_host", Y_host)):
        if t.is_cuda or not t.is_contiguous() or t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be a contiguous CPU bf16 tensor")
    if tuple(X_dev2.shape) != (2, T, d) or tuple(Y_dev2.shape) != (2, T, d):
        raise ValueError("X_dev2 / Y_dev2 must be [2, T, d]")
    if ws is None:
        ws = workspace(T, d, E, K, n, X_dev2.device)
    if stream is None:
        stream = torch.cuda.current_stream()
    h2d_stream = h2d_stream or torch.cuda.Stream(device=X_dev2.device)
    d2h_stream = d2h_stream or torch.cuda.Stream(device=X_dev2.device)
    _check("moe_forward_host_stream", lib().moe_forward_host_stream(
        ctypes.c_void_p(X_host.data_ptr()), ctypes.c_void_p(Y_host.data_ptr()), nb,
        _ptr(X_dev2, torch.bfloat16), _ptr(Y_dev2, torch.bfloat16), _ptr(Wr, torch.float32),
        _ptr(bias, torch.float32), _ptr(W1, torch.bfloat16), _ptr(W3, torch.bfloat16),
        _ptr(W2, torch.bfloat16), T, d, E, K, n, int(bool(renorm)), _ptr(ws), ws.numel(),
        _stream(stream), _stream(h2d_stream), _stream(d2h_stream)))
    return Y_host


def moe_selftest_wait_timeout(ws, stream=None):
    """Enqueue the bounded-wait self-test (sets MOE_DEVERR_TIMEOUT after ~1 s)."""
    _check("moe_selftest_wait_timeout", lib().moe_selftest_wait_timeout(
        _ptr(ws), ws.numel(), _stream(stream)))


def moe_selftest_layernorm_withhold(row: int):
    """This thread's next layer or block norm call never gets row `row` (a wait of ~1 s runs out)."""
    _check("moe_selftest_layernorm_withhold", lib().moe_selftest_layernorm_withhold(row))


def moe_sync_check(ws, stream=None):
    """(status, raw error word) after waiting for the stream; clears the word."""
    word = ctypes.c_uint32(0)
    st = lib().moe_sync_check(_ptr(ws), _stream(stream), ctypes.byref(word))
    return int(st), int(word.value)


# ------------------------------------------------------------ Token Rounding

def moe_round_capacity(T: int, E: int, K: int, M: int = TILE_M) -> int:
    return int(lib().moe_round_capacity(T, E, K, M))


def moe_round_routing(logits, topk_idx, counts, M: int = TILE_M, renorm: bool = True, ws=None,
                      stream=None) -> dict:
    """Token Rounding of a top-K routing (outputs of moe_route). Returns counts,
    offsets, perm_token [capacity], row_map [T,E], row_w [capacity], tiles and
    num_tiles; offsets[E] entries of perm_token/row_w are meaningful."""
    T, E = logits.shape
    K = topk_idx.shape[1]
    dev = logits.device
    cap = moe_round_capacity(T, E, K, M)
    if cap < 0:
        raise ValueError("invalid Token Rounding shape")
    if ws is None:
        ws = torch.zeros(int(lib().moe_round_workspace_bytes(T, E)), dtype=torch.uint8, device=dev)
    out = dict(
        counts=torch.empty(E, dtype=torch.int32, device=dev),
        offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
        perm_token=torch.full((max(cap, 1),), -1, dtype=torch.int32, device=dev),
        row_map=torch.empty((T, E), dtype=torch.int32, device=dev),
        row_w=torch.zeros(max(cap, 1), dtype=torch.float32, device=dev),
        tiles=torch.zeros((cap // TILE_M + E, 4), dtype=torch.int32, device=dev),
        num_tiles=torch.empty(1, dtype=torch.int32, device=dev),
    )
    _check("moe_round_routing", lib().moe_round_routing(
        _ptr(logits, torch.float32, "logits"), _ptr(topk_idx, torch.int32, "topk_idx"),
        _ptr(counts, torch.int32, "counts"), T, E, K, M, int(bool(renorm)),
        _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["perm_token"]), _ptr(out["row_map"]),
        _ptr(out["row_w"]), _ptr(out["tiles"]), _ptr(out["num_tiles"]), _ptr(ws), ws.numel(),
        _stream(stream)))
    out["ws"] = ws
    return out


def moe_combine_rows(Z, row_map, stream=None):
    R, d = Z.shape
    T, E = row_map.shape
    Y = torch.empty((T, d), dtype=torch.bfloat16, device=Z.device)
    _check("moe_combine_rows", lib().moe_combine_rows(
        _ptr(Z, torch.bfloat16, "Z"), _ptr(row_map, torch.int32, "row_map"), T, E, d, R,
        _ptr(Y), _stream(stream)))
    return Y


def workspace_rounded(T: int, d: int, E: int, K: int, n: int, device=None) -> torch.Tensor:
    """A zeroed workspace tensor for moe_forward_rounded."""
    nbytes = int(lib().moe_workspace_bytes_rounded(T, d, E, K, n))
    if nbytes == 0:
        raise ValueError("invalid layer shape")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def moe_forward_rounded(X, Wr, W1, W3, W2, K: int, bias=None, renorm: bool = True, ws=None,
                        Y=None, row_map=None, stream=None, events=None):
    """Y [T,d] bf16 for the layer under Token Rounding (tile size 128). An optional
    row_map [T,E] int32 receives each (token, expert) row or -1."""
    T, d = X.shape
    E, _, n = W1.shape
    if ws is None:
        ws = workspace_rounded(T, d, E, K, n, X.device)
    if Y is None:
        Y = torch.empty((T, d), dtype=torch.bfloat16, device=X.device)
    args = (_ptr(X, torch.bfloat16, "X"), _ptr(Wr, torch.float32, "Wr"),
            _ptr(bias, torch.float32, "bias"), _ptr(W1, torch.bfloat16, "W1"),
            _ptr(W3, torch.bfloat16, "W3"), _ptr(W2, torch.bfloat16, "W2"), T, d, E, K, n,
            int(bool(renorm)), _ptr(Y, torch.bfloat16, "Y"), _ptr(row_map, torch.int32, "row_map"),
            _ptr(ws), ws.numel(), _stream(stream))
    if events:
        for e in events:
            if e.cuda_event == 0:
                e.record()
        arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
        _check("moe_forward_rounded_traced", lib().moe_forward_rounded_traced(*args, arr,
                                                                               len(events)))
    else:
        _check("moe_forward_rounded", lib().moe_forward_rounded(*args))
    return Y


# ------------------------------------- layer norm, residual dropout, dense block

_nat = None


def _native():
    """The compiled entry points of the calls below (csrc/binding.cpp): checks,
    allocation of outputs and the library call."""
    global _nat
    if _nat is None:
        lib()
        try:
            from . import _native as nat
        except ImportError as e:
            raise RuntimeError(f"_native.so is not built or cannot be loaded ({e}); run "
                               "__graft_entry__.build()") from e
        nat.set_error(MoeError)
        _nat = nat
    return _nat


def moe_layernorm(x, gamma=None, beta=None, eps: float = 1e-5, stats: bool = False, y=None,
                  stream=None):
    """y = layer norm of x along its last dimension (gamma, beta: [d] of x's type or
    fp32, or None); stats=True: (y, mean, rstd), the fp32 row statistics that the
    backward takes."""
    return _native().layernorm(x, gamma, beta, eps, stats, y, stream)


def moe_layernorm_backward(dy, x, gamma, mean, rstd, dres=None, wdtype=None, dx=None, scratch=None,
                           stream=None):
    """(dx, dgamma, dbeta) of moe_layernorm, with `dres` (the gradient that reaches
    x by the residual branch) added to dx when given. dgamma and dbeta have gamma's
    type, or wdtype (default fp32) without gamma."""
    if gamma is None and wdtype not in (None, torch.float32, x.dtype):
        raise TypeError(f"weight gradients are {x.dtype} or fp32, got {wdtype}")
    return _native().layernorm_backward(dy, x, gamma, mean, rstd, dres, wdtype is not x.dtype, dx,
                                        scratch, stream)


def moe_dropout(x, p: float, seed: int, offset: int = 0, residual=None, offset_dev=None, y=None,
                stream=None):
    """residual + dropout(x): the mask is a function of (seed, offset, element), see
    moe.h; offset_dev: a one-element int64 CUDA tensor added to offset."""
    return _native().dropout(x, p, seed, offset, residual, offset_dev, y, stream)


def moe_dropout_backward(dy, p: float, seed: int, offset: int = 0, offset_dev=None, dx=None,
                         stream=None):
    """The gradient of moe_dropout with respect to x (the residual's is dy)."""
    return _native().dropout_backward(dy, p, seed, offset, offset_dev, dx, stream)


ACTS = {"silu": 0, "gelu": 1}


def ffn_workspace(T: int, d: int, n: int, train: bool = False, device=None, stream=None):
    """A workspace (uint8, control words zeroed) of the dense block's calls for up to
    T tokens; train: of moe_ffn_train and moe_ffn_backward too. It lies on `device`
    (default: the given stream's, else the current one)."""
    nbytes = int(lib().moe_ffn_workspace_bytes(T, d, n, int(train)))
    if nbytes == 0:
        raise ValueError("invalid feed-forward shape")
    return _control_workspace(nbytes, device, stream)


def _control_workspace(nbytes: int, device, stream):
    device = None if device is None else torch.device(device)
    if device is not None:
        if device.type != "cuda":
            raise ValueError("the workspace lies on a CUDA device")
        if stream is not None and device.index not in (None, stream.device_index):
            raise ValueError("stream must belong to the workspace's device")
    # its memory is the stream's, as a temporary's reuse follows that order
    with torch.cuda.device(device if stream is None else stream.device), torch.cuda.stream(stream):
        ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        _check("moe_ffn_workspace_init", lib().moe_ffn_workspace_init(
            ws.data_ptr(), nbytes, _stream(stream)))
    return ws


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    return ACTS[act]


def _ffn_ws(ws, x, W1, train, stream):
    if ws is not None:
        return ws
    if not x.is_cuda or x.dim() < 1 or W1.dim() != 2 or W1.numel() == 0:
        raise ValueError("x must be a CUDA tensor [..., d] and W1 [d, n]")
    d, n = W1.shape
    return ffn_workspace(x.numel() // d, d, n, train, x.device, stream)


def moe_ffn(x, W1, W3, W2, act: str = "silu", ws=None, Y=None, stream=None):
    """Y = (act(x W1) * (x W3)) W2 of x [..., d] (bf16 or fp16); act "silu" or "gelu"
    (the tanh form). ws: ffn_workspace, kept between calls."""
    return _native().ffn(x, W1, W3, W2, _act(act), _ffn_ws(ws, x, W1, False, stream), Y, stream)


def moe_ffn_train(x, W1, W3, W2, act: str = "silu", ws=None, stream=None):
    """(Y, H, F1, F3): moe_ffn's Y and what moe_ffn_backward takes (F1, F3: fp32 in the
    blocks that moe.h describes). ws: ffn_workspace(..., train=True)."""
    return _native().ffn_train(x, W1, W3, W2, _act(act), _ffn_ws(ws, x, W1, True, stream), stream)


def moe_ffn_backward(dY, x, W1, W3, W2, H, F1, F3, act: str = "silu", need_dx: bool = True,
                     need_dw: bool = True, ws=None, stream=None):
    """(dX, dW1, dW3, dW2) of moe_ffn_train, all of x's type (None where not asked
    for). ws: ffn_workspace(..., train=True)."""
    return _native().ffn_backward(dY, x, W1, W3, W2, H, F1, F3, _act(act), need_dx, need_dw,
                                  _ffn_ws(ws, x, W1, True, stream), stream)

# ------------------------------------------- a dense projection with its epilogue


def linear_workspace(T: int, k: int, n: int, train: bool = False, device=None, stream=None):
    """A workspace (uint8, control words zeroed) of the projection calls for up to T tokens;
    train: of moe_linear_train and moe_linear_backward too. Where it lies: as ffn_workspace."""
    nbytes = int(lib().moe_linear_workspace_bytes(T, k, n, int(train)))
    if nbytes == 0:
        raise ValueError("invalid projection shape")
    return _control_workspace(nbytes, device, stream)


def _linear_act(act) -> int:
    return 2 if act is None else _act(act)


def _linear_ws(ws, x, W, train, stream):
    if ws is not None:
        return ws
    if not x.is_cuda or x.dim() < 1 or W.dim() != 2 or W.numel() == 0:
        raise ValueError("x must be a CUDA tensor [..., k] and W [k, n]")
    k, n = W.shape
    return linear_workspace(x.numel() // k, k, n, train, x.device, stream)


def moe_linear(x, W, bias=None, act=None, residual=None, ws=None, Y=None, stream=None):
    """Y = act(x W + bias) + residual of x [..., k] (bf16 or fp16); act None, "silu" or "gelu"
    (the tanh form), bias [n] of x's type or fp32. Y may be residual. ws: linear_workspace, kept
    between calls."""
    return _native().linear(x, W, bias, _linear_act(act), residual, _linear_ws(ws, x, W, False, stream), Y,
                            stream)


def moe_linear_train(x, W, bias=None, act=None, residual=None, ws=None, stream=None):
    """(Y, F): moe_linear's Y and F = act'(x W + bias), which moe_linear_backward takes (fp32 in
    the blocks that moe.h describes; None without an activation). ws: linear_workspace(..., train=True)."""
    return _native().linear_train(x, W, bias, _linear_act(act), residual, _linear_ws(ws, x, W, True, stream),
                                  stream)


def moe_linear_backward(dY, x, W, F, bias_dtype=None, need_dx: bool = True, need_dw: bool = True, ws=None,
                        stream=None):
    """(dX, dW, dbias) of moe_linear_train, of x's type, dbias of bias_dtype (x's type or fp32;
    None: there was no bias); None where not asked for. The residual's gradient is dY. ws:
    linear_workspace(..., train=True)."""
    if bias_dtype not in (None, torch.float32, x.dtype):
        raise TypeError(f"the bias' gradient is {x.dtype} or fp32, got {bias_dtype}")
    return _native().linear_backward(dY, x, W, F, None if bias_dtype is None else bias_dtype is not x.dtype,
                                     need_dx, need_dw, _linear_ws(ws, x, W, True, stream), stream)


# --------------------------------------------------- the norms around a block


def moe_block_norm(x, b, post=None, pre=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
                   post_norm: bool = True, pre_norm: bool = True, stats: bool = False, y=None, u=None,
                   stream=None):
    """(y, u): y = scale x + sigmoid(gate) post rms(b), the stream behind a block whose output
    is b, and u = pre rms(y), the input of the next one (None without pre_norm; without
    post_norm, post scales b itself). gate: like x, or one fp32 value a row, or None (no gate);
    post, pre [d] of x's type or fp32, or None. stats=True: (y, u, rstd_post, rstd_pre), the
    fp32 row statistics that the backward takes. y may be x."""
    if b is None:
        raise TypeError("b must be a tensor (moe_rmsnorm is the norm alone)")
    return _native().block_norm(x, b, post, pre, gate, scale, eps, post_norm, pre_norm, stats, y, u, stream)


def moe_block_norm_backward(dy, du, x, b, post, pre, rstd_post, rstd_pre, gate=None,
                            scale: float = 1.0, wdtype=None, dx=None, db=None, scratch=None,
                            stream=None):
    """(dx, db, dgate, dpost, dpre) of moe_block_norm, with dy the gradient that reaches y by the
    stream (or None) and du that of u; rstd_post and rstd_pre are None where the forward had no
    such norm. dgate is None without a gate, dpre without the pre norm. dpost and dpre have the
    weights' type, or wdtype (default fp32) without weights."""
    if post is None and pre is None and wdtype not in (None, torch.float32, x.dtype):
        raise TypeError(f"weight gradients are {x.dtype} or fp32, got {wdtype}")
    if b is None:
        raise TypeError("b must be a tensor (moe_rmsnorm_backward is the norm alone)")
    return _native().block_norm_backward(dy, du, x, b, post, pre, rstd_post, rstd_pre, gate,
                                         scale, wdtype is not x.dtype, dx, db, scratch, stream)


def moe_rmsnorm(x, gamma=None, eps: float = 1e-6, stats: bool = False, y=None, stream=None):
    """y = gamma x / sqrt(mean(x^2) + eps) along the last dimension (gamma: [d] of x's type or
    fp32, or None); stats=True: (y, rstd), the fp32 row statistics that the backward takes."""
    out = _native().block_norm(x, None, None, gamma, None, 1.0, eps, False, True, stats, None, y, stream)
    return (out[1], out[3]) if stats else out[1]


def moe_rmsnorm_backward(dy, x, gamma, rstd, dres=None, wdtype=None, dx=None, scratch=None,
                         stream=None):
    """(dx, dgamma) of moe_rmsnorm, with `dres` (the gradient that reaches x by the residual
    branch) added to dx when given. dgamma has gamma's type, or wdtype (default fp32) without
    gamma."""
    if gamma is None and wdtype not in (None, torch.float32, x.dtype):
        raise TypeError(f"weight gradients are {x.dtype} or fp32, got {wdtype}")
    if not torch.is_tensor(dy) or not torch.is_tensor(rstd):
        raise TypeError("dy and rstd must be tensors")
    out = _native().block_norm_backward(dres, dy, x, None, None, gamma, None, rstd, None, 1.0,
                                        wdtype is not x.dtype, dx, None, scratch, stream)
    return out[0], out[4]


# ------------------------- rows sorted by expert and back, for experts of any kind


def moe_dispatch(x, row_of_slot, K: int, xg=None, stream=None):
    """xg [T*K, d]: every token's row of x [..., d] at the rows of its K slots, with
    row_of_slot as moe_permute gives it (a value outside xg's rows: no row). Rows that no
    slot names are left as they were: not defined in a new xg."""
    return _native().dispatch(x, row_of_slot, K, xg, stream)


def moe_dispatch_backward(dxg, row_of_slot, K: int, residual=None, dx=None, stream=None):
    """dx [T, d]: the sum of dxg over each token's rows (+ residual, a gradient that reaches
    x by another branch)."""
    return _native().combine_weighted(dxg, row_of_slot, int(K), residual, dx, stream)


def moe_combine_weighted(z, row_of_slot, w, residual=None, y=None, stream=None):
    """y [T, d] = sum over k of w[t, k] times the row of slot (t, k) of z [rows, d]
    (+ residual); w [T, K] fp32 as moe_route gives it. y may be residual."""
    if not torch.is_tensor(w):
        raise TypeError("w must be a tensor")
    return _native().combine_weighted(z, row_of_slot, w, residual, y, stream)


def moe_combine_weighted_backward(dy, z, row_of_slot, w, dz=None, stream=None):
    """(dz [rows, d], dw [T, K] fp32) of moe_combine_weighted (the residual's gradient is
    dy). Rows of dz that no slot names are left as they were: not defined in a new dz."""
    return _native().combine_weighted_backward(dy, z, row_of_slot, w, dz, stream)
