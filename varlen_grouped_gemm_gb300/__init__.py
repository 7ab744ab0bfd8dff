"""GB300 (sm_103a) MoE expert-layer hot path — Python binding of the C ABI in ``include/moe.h``.

Argument marshalling only: every step of the path (routing, grouping, grouped
GEMMs, combine, backward) runs in the CUDA library ``lib/libvgg_moe.so``.
PyTorch supplies device memory and streams.  There is no CPU fallback: when
the library is missing, every call raises.

The functions carry the C names (``moe_route``, ``moe_permute``,
``moe_grouped_gemm_fwd``, ``moe_combine``, ``moe_backward``); sizes are taken
from the tensors' shapes.  ``Buffers`` allocates every tensor the path needs
for one configuration, and ``forward_backward`` runs the whole path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libvgg_moe.so")

# The symbols declared in include/moe.h.
EXPORTS = (
    "moe_create", "moe_destroy", "moe_status_str", "moe_get_error", "moe_set_wait_timeout", "moe_set_cta_pairs",
    "moe_pair_capacity", "moe_workspace_bytes", "moe_route", "moe_permute", "moe_grouped_gemm_fwd",
    "moe_combine", "moe_backward", "moe_profile_enable", "moe_profile_read", "moe_test_gemm_varlen_m",
    "moe_test_gemm_varlen_k", "moe_test_wait_timeout", "moe_permute_noalloc", "moe_permute_capacity",
    "moe_capacity_workspace_bytes", "moe_quantize_rows_e4m3", "moe_grouped_gemm_fwd_e4m3",
    "moe_quantize_dx_weights_e4m3", "moe_quantize_dact_weights_e4m3", "moe_backward_e4m3",
    "moe_expert_capacity", "moe_test_gemm_varlen_k_dual", "moe_test_gemm_varlen_m_dual",
    "moe_mx_sf_cols", "moe_mx_weight_sf_bytes", "moe_mx_act_sf_bytes", "moe_quantize_rows_mx",
    "moe_quantize_weights_mx", "moe_grouped_gemm_fwd_mx", "moe_quantize_bwd_weights_mx", "moe_backward_mx",
    "moe_mx_dw_ws_bytes", "moe_add_rmsnorm", "moe_add_rmsnorm_workspace_bytes", "moe_add_rmsnorm_backward",
    "moe_balance_loss", "moe_balance_loss_workspace_bytes", "moe_router_backward",
    "moe_router_backward_workspace_bytes", "moe_few_workspace_bytes", "moe_forward_few", "moe_forward_few_e4m3",
    "moe_keep_rows8", "moe_read_rows8", "moe_grouped_gemm_fwd_kept8", "moe_grouped_gemm_fwd_e4m3_kept8",
    "moe_grouped_gemm_fwd_mx_kept8", "moe_kept8_workspace_bytes", "moe_backward_kept8", "moe_backward_e4m3_kept8",
    "moe_backward_mx_kept8",
)

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_DEVICE, MOE_ERR_DEVICE_TIMEOUT = range(6)
DEV_OK, DEV_BAD_EXPERT, DEV_DUP_EXPERT, DEV_BAD_OFFSETS, DEV_TIMEOUT, DEV_CAPACITY = range(6)

_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
_SZ = ctypes.c_size_t
_F = ctypes.c_float


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run varlen_grouped_gemm_gb300/build.py or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_create.argtypes = [ctypes.POINTER(_P), _I]
        L.moe_destroy.argtypes = [_P]
        L.moe_status_str.argtypes = [_I]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_get_error.argtypes = [_P, ctypes.POINTER(_I)]
        L.moe_set_wait_timeout.argtypes = [_P, ctypes.c_ulonglong]
        L.moe_set_cta_pairs.argtypes = [_P, _I, _I]
        L.moe_pair_capacity.argtypes = [_I, _I, _I, _I]
        L.moe_pair_capacity.restype = _LL
        L.moe_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
        L.moe_workspace_bytes.restype = _SZ
        L.moe_route.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_permute.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_grouped_gemm_fwd.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P, _P, _P, _P, _P,
                                           _P, _SZ, _P]
        L.moe_combine.argtypes = [_P, _P, _P, _P, _I, _I, _LL, _P, _P]
        L.moe_backward.argtypes = [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _LL, _P, _P, _P, _P, _P,
                                   _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _SZ, _P]
        L.moe_test_gemm_varlen_m.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _LL, _P, _P, _P]
        L.moe_test_gemm_varlen_k.argtypes = [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P]
        L.moe_test_wait_timeout.argtypes = [_P, ctypes.c_ulonglong, _P]
        L.moe_expert_capacity.argtypes = [_I, _I, _I, ctypes.c_double]
        L.moe_expert_capacity.restype = _LL
        L.moe_test_gemm_varlen_k_dual.argtypes = [_P, _P, _P, _I, _P, _I, _I, _I, _I, _LL, _P, _P, _I, _P, _P]
        L.moe_test_gemm_varlen_m_dual.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P]
        L.moe_permute_noalloc.argtypes = [_P, _P, _P, _I, _I, _I, _LL, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_permute_capacity.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _LL, _P, _P, _P, _P, _P, _P, _P, _P, _SZ,
                                           _P]
        L.moe_capacity_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
        L.moe_capacity_workspace_bytes.restype = _SZ
        L.moe_quantize_rows_e4m3.argtypes = [_P, _P, _LL, _I, _P, _P, _P]
        L.moe_grouped_gemm_fwd_e4m3.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P,
                                                _P, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_quantize_dx_weights_e4m3.argtypes = [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P]
        L.moe_quantize_dact_weights_e4m3.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P]
        L.moe_backward_e4m3.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _LL,
                                        _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I,
                                        _P, _P, _P, _P, _SZ, _P]
        L.moe_mx_sf_cols.argtypes = [_I]
        L.moe_mx_sf_cols.restype = _LL
        L.moe_mx_weight_sf_bytes.argtypes = [_I, _I, _I, _I]
        L.moe_mx_weight_sf_bytes.restype = _LL
        L.moe_mx_act_sf_bytes.argtypes = [_LL, _I, _I]
        L.moe_mx_act_sf_bytes.restype = _LL
        L.moe_mx_dw_ws_bytes.argtypes = [_I, _I, _I, _LL]
        L.moe_mx_dw_ws_bytes.restype = _SZ
        L.moe_quantize_rows_mx.argtypes = [_P, _P, _LL, _I, _P, _P, _P]
        L.moe_quantize_weights_mx.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]
        L.moe_grouped_gemm_fwd_mx.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P, _P,
                                              _P, _P, _P, _P, _P, _P]
        L.moe_quantize_bwd_weights_mx.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]
        L.moe_backward_mx.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _LL, _P, _P,
                                      _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P,
                                      _SZ, _P, _SZ, _P]
        L.moe_add_rmsnorm.argtypes = [_P, _P, _LL, _P, _LL, _I, _P, _I, _LL, _I, _F, _P, _LL, _P, _LL, _P, _I, _P, _P, _P]
        L.moe_add_rmsnorm_workspace_bytes.argtypes = [_LL, _I]
        L.moe_add_rmsnorm_workspace_bytes.restype = _SZ
        L.moe_add_rmsnorm_backward.argtypes = [_P, _P, _LL, _P, _LL, _I, _P, _I, _P, _P, _LL, _LL, _I, _P, _LL, _P, _LL,
                                               _P, _P, _SZ, _P]
        L.moe_balance_loss_workspace_bytes.argtypes = [_LL, _I, _I]
        L.moe_balance_loss_workspace_bytes.restype = _SZ
        L.moe_balance_loss.argtypes = [_P, _P, _P, _P, _P, _LL, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_router_backward_workspace_bytes.argtypes = [_I, _I, _I]
        L.moe_router_backward_workspace_bytes.restype = _SZ
        L.moe_router_backward.argtypes = [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]
        L.moe_keep_rows8.argtypes = [_P, _P, _LL, _I, _P, _P, _P]
        L.moe_read_rows8.argtypes = [_P, _P, _P, _LL, _I, _P, _P]
        L.moe_grouped_gemm_fwd_kept8.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                                 _P, _SZ, _P]
        L.moe_grouped_gemm_fwd_e4m3_kept8.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P,
                                                      _P, _P, _P, _P, _P, _P, _P, _P, _P]
        L.moe_grouped_gemm_fwd_mx_kept8.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _LL, _P, _P, _P, _P, _P,
                                                    _P, _P, _P, _P, _P, _P, _P]
        L.moe_kept8_workspace_bytes.argtypes = [_I, _I, _I, _I, _LL]
        L.moe_kept8_workspace_bytes.restype = _SZ
        L.moe_backward_kept8.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _LL] + [_P] * 7 + \
            [_P] * 8 + [_I, _P, _P, _P, _P, _SZ, _P]
        L.moe_backward_e4m3_kept8.argtypes = [_P] * 13 + [_I, _I, _I, _I, _I, _I, _LL] + [_P] * 7 + [_P] * 12 + \
            [_I, _P, _P, _P, _P, _SZ, _P]
        L.moe_backward_mx_kept8.argtypes = [_P] * 13 + [_I, _I, _I, _I, _I, _I, _LL] + [_P] * 7 + [_P] * 12 + \
            [_I, _P, _P, _P, _P, _SZ, _P, _SZ, _P]
        L.moe_few_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
        L.moe_few_workspace_bytes.restype = _SZ
        L.moe_forward_few.argtypes = [_P, _P, _LL, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _LL, _P, _SZ, _P]
        L.moe_forward_few_e4m3.argtypes = [_P, _P, _LL, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P,
                                           _LL, _P, _SZ, _P]
        L.moe_profile_enable.argtypes = [_P, _I]
        L.moe_profile_read.argtypes = [_P, _I, ctypes.c_char_p, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(_LL), ctypes.POINTER(_I)]
        _lib = L
    return _lib


def status_str(code: int) -> str:
    return lib().moe_status_str(code).decode()


def _check(name: str, rc: int):
    if rc != MOE_OK:
        raise RuntimeError(f"{name} failed: {status_str(rc)} (status {rc})")


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the raw handle of the current stream: building a Stream object takes longer than a launch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Context:
    """A library context on one device (owns the device error word)."""

    def __init__(self, device: int = 0):
        self.device = device
        h = _P()
        _check("moe_create", lib().moe_create(ctypes.byref(h), device))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            lib().moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_wait_timeout(self, ns: int):
        _check("moe_set_wait_timeout", lib().moe_set_wait_timeout(self.handle, int(ns)))

    def set_cta_pairs(self, varlen_m: bool, varlen_k: bool):
        """CTA pairs (two CTAs per 256-row tile) for the tiled varlen-M and the weight-gradient GEMMs."""
        _check("moe_set_cta_pairs", lib().moe_set_cta_pairs(self.handle, int(varlen_m), int(varlen_k)))


@dataclass
class Kept8:
    """Rows kept in 8 bits for the backward: codes ``q`` int8 [rows, cols] and bf16 scales ``scale`` [rows, cols / 32]."""

    q: torch.Tensor
    scale: torch.Tensor

    @staticmethod
    def empty(rows: int, cols: int, device="cuda") -> "Kept8":
        if cols % 32:
            raise ValueError(f"kept rows are whole blocks of 32 columns, got {cols}")
        return Kept8(torch.zeros((rows, cols), dtype=torch.int8, device=device),
                     torch.zeros((rows, cols // 32), dtype=torch.bfloat16, device=device))

    @property
    def shape(self):
        return self.q.shape

    def pointers(self, ctx: "Context", shape, name: str):
        """(codes, scales) of rows of the given shape on the context's device."""
        rows, cols = shape
        if cols % 32:
            raise ValueError(f"{name}: kept rows are whole blocks of 32 columns, got {cols}")
        return (_flat(ctx, self.q, (rows, cols), torch.int8, f"{name}.q"),
                _flat(ctx, self.scale, (rows, cols // 32), torch.bfloat16, f"{name}.scale"))


def _kept_pair(ctx, H, U, shape):
    """Pointers of H and U where they are kept in 8 bits, None where they are fp32 tensors (or absent)."""
    if not isinstance(H, Kept8) and not isinstance(U, Kept8):
        return None
    if not (isinstance(H, Kept8) and isinstance(U, Kept8)):
        raise ValueError("H and U are kept in the same way: both fp32 or both Kept8")
    return (*H.pointers(ctx, shape, "H"), *U.pointers(ctx, shape, "U"))


def _kept_x(ctx, X, T, d):
    """(X, its codes, their scales) for a backward from kept activations: X a bf16 tensor or Kept8."""
    if isinstance(X, Kept8):
        return (None, *X.pointers(ctx, (T, d), "X"))
    return (_ptr(X, torch.bfloat16, "X"), None, None)


def moe_profile_enable(ctx: Context, enable: bool = True):
    _check("moe_profile_enable", lib().moe_profile_enable(ctx.handle, 1 if enable else 0))


def moe_profile_read(ctx: Context) -> dict[str, tuple[float, int]]:
    """{kernel label: (total ms, launches)} since the last read (waits for the recorded events)."""
    nmax = 64
    names = ctypes.create_string_buffer(32 * nmax)
    ms = (ctypes.c_double * nmax)()
    cnt = (_LL * nmax)()
    n = _I(0)
    _check("moe_profile_read", lib().moe_profile_read(ctx.handle, nmax, names, ms, cnt, ctypes.byref(n)))
    out = {}
    for i in range(min(n.value, nmax)):
        label = names.raw[32 * i:32 * i + 32].split(b"\0", 1)[0].decode()
        out[label] = (ms[i], int(cnt[i]))
    return out


def moe_get_error(ctx: Context) -> tuple[int, int]:
    """(status, device error code); synchronizes the device and clears the code."""
    code = _I(0)
    rc = lib().moe_get_error(ctx.handle, ctypes.byref(code))
    return rc, code.value


def moe_pair_capacity(T: int, E: int, K: int, m_tile: int = 0) -> int:
    return int(lib().moe_pair_capacity(T, E, K, m_tile))


def moe_workspace_bytes(T: int, d: int, E: int, n: int, K: int, m_tile: int = 0) -> int:
    return int(lib().moe_workspace_bytes(T, d, E, n, K, m_tile))


def _ws(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def moe_route(ctx, X, W_r, bias, K, logits, scores, topk_ids, topk_w, ws=None, stream=None):
    T, d = X.shape
    E = W_r.shape[1]
    wp, wb = _ws(ws)
    _check("moe_route", lib().moe_route(
        ctx.handle, _ptr(X, torch.bfloat16, "X"), _ptr(W_r, torch.bfloat16, "W_r"),
        _ptr(bias, torch.float32, "bias"), T, d, E, K, _ptr(logits, torch.float32, "logits"),
        _ptr(scores, torch.float32, "scores"), _ptr(topk_ids, torch.int32, "topk_ids"),
        _ptr(topk_w, torch.float32, "topk_w"), wp, wb, _stream(stream)))


def moe_permute(ctx, topk_ids, topk_w, logits, scores, E, m_tile, counts, offsets, sorted_tok, sorted_w,
                tok_ptr, tok_pairs, P_out, ws, stream=None):
    T, K = topk_ids.shape
    cap = sorted_tok.numel()
    wp, wb = _ws(ws)
    _check("moe_permute", lib().moe_permute(
        ctx.handle, _ptr(topk_ids, torch.int32), _ptr(topk_w, torch.float32), _ptr(logits, torch.float32),
        _ptr(scores, torch.float32), T, E, K, m_tile, cap, _ptr(counts, torch.int32),
        _ptr(offsets, torch.int32), _ptr(sorted_tok, torch.int32), _ptr(sorted_w, torch.float32),
        _ptr(tok_ptr, torch.int32), _ptr(tok_pairs, torch.int32), _ptr(P_out, torch.int32), wp, wb,
        _stream(stream)))


def moe_permute_noalloc(ctx, topk_ids, topk_w, E, counts, offsets, sorted_tok, sorted_w, tok_ptr, tok_pairs, P_out,
                        stream=None):
    """moe_permute (plain top-K) with its scratch in a fixed array inside the library: for callers
    that cannot allocate device memory.  At most 32768 tokens and 512 experts."""
    T, K = topk_ids.shape
    _check("moe_permute_noalloc", lib().moe_permute_noalloc(
        ctx.handle, _ptr(topk_ids, torch.int32), _ptr(topk_w, torch.float32), T, E, K, sorted_tok.numel(),
        _ptr(counts, torch.int32), _ptr(offsets, torch.int32), _ptr(sorted_tok, torch.int32),
        _ptr(sorted_w, torch.float32), _ptr(tok_ptr, torch.int32), _ptr(tok_pairs, torch.int32),
        _ptr(P_out, torch.int32), _stream(stream)))


POLICIES = {"position": 0, "probs": 1}


def expert_capacity(T: int, E: int, K: int, capacity_factor: float) -> int:
    """Slots per expert of the capacity dispatch (the library's moe_expert_capacity)."""
    C = int(lib().moe_expert_capacity(T, E, K, float(capacity_factor)))
    if C < 1:
        raise ValueError(f"moe_expert_capacity: invalid arguments T={T} E={E} K={K} cf={capacity_factor}")
    return C


def moe_permute_capacity(ctx, topk_ids, topk_w, E, C, policy, counts, offsets, sorted_tok, sorted_w, tok_ptr,
                         tok_pairs, P_out, ws, stream=None):
    """Capacity (drop/pad) dispatch: expert e keeps at most C pairs in slots [e C, (e+1) C)."""
    T, K = topk_ids.shape
    wp, wb = _ws(ws)
    _check("moe_permute_capacity", lib().moe_permute_capacity(
        ctx.handle, _ptr(topk_ids, torch.int32), _ptr(topk_w, torch.float32), T, E, K, C, POLICIES[policy],
        sorted_tok.numel(), _ptr(counts, torch.int32), _ptr(offsets, torch.int32), _ptr(sorted_tok, torch.int32),
        _ptr(sorted_w, torch.float32), _ptr(tok_ptr, torch.int32), _ptr(tok_pairs, torch.int32),
        _ptr(P_out, torch.int32), wp, wb, _stream(stream)))


def moe_capacity_workspace_bytes(T: int, d: int, E: int, n: int, K: int, C: int) -> int:
    return int(lib().moe_capacity_workspace_bytes(T, d, E, n, K, C))


def moe_grouped_gemm_fwd(ctx, X, W_gate, W_up, W_down, offsets, sorted_tok, sorted_w, H, U, A, Yw, ws=None,
                         stream=None):
    """The experts' products of every pair; H and U fp32 [cap, n], Kept8 (8 bits), or None (forward only)."""
    T, d = X.shape
    E, n, _ = W_gate.shape
    cap = sorted_tok.numel()
    wp, wb = _ws(ws)
    bf = torch.bfloat16
    head = (ctx.handle, _ptr(X, bf), _ptr(W_gate, bf), _ptr(W_up, bf), _ptr(W_down, bf), T, d, E, n, cap,
            _ptr(offsets, torch.int32), _ptr(sorted_tok, torch.int32), _ptr(sorted_w, torch.float32))
    tail = (_ptr(A, bf), _ptr(Yw, bf), wp, wb, _stream(stream))
    kept = _kept_pair(ctx, H, U, (cap, n))
    if kept:
        _check("moe_grouped_gemm_fwd_kept8", lib().moe_grouped_gemm_fwd_kept8(*head, *kept, *tail))
    else:
        _check("moe_grouped_gemm_fwd", lib().moe_grouped_gemm_fwd(
            *head, _ptr(H, torch.float32), _ptr(U, torch.float32), *tail))


def moe_keep_rows8(ctx, M, kept: Kept8, stream=None):
    """M [rows, cols] bf16 as codes and scales (one for 32 columns) into ``kept``."""
    rows, cols = M.shape
    q, scale = kept.pointers(ctx, (rows, cols), "kept")
    _check("moe_keep_rows8", lib().moe_keep_rows8(
        ctx.handle, _flat(ctx, M, (rows, cols), torch.bfloat16, "M"), rows, cols, q, scale, _stream(stream)))


def moe_read_rows8(ctx, kept: Kept8, M, stream=None):
    """The values that ``kept`` stands for into M [rows, cols] bf16."""
    rows, cols = M.shape
    q, scale = kept.pointers(ctx, (rows, cols), "kept")
    _check("moe_read_rows8", lib().moe_read_rows8(
        ctx.handle, q, scale, rows, cols, _flat(ctx, M, (rows, cols), torch.bfloat16, "M"), _stream(stream)))


def moe_quantize_rows_e4m3(ctx, M, q, scales, stream=None):
    """Per-row e4m3 codes (uint8, shaped like M) and fp32 scales (one per row of M's last axis)."""
    cols = M.shape[-1]
    rows = M.numel() // cols
    if q.shape != M.shape or scales.numel() != rows:
        raise ValueError("q must be shaped like M and scales hold one value per row")
    _check("moe_quantize_rows_e4m3", lib().moe_quantize_rows_e4m3(
        ctx.handle, _ptr(M, torch.bfloat16), rows, cols, _ptr(q, torch.uint8), _ptr(scales, torch.float32),
        _stream(stream)))


def moe_grouped_gemm_fwd_e4m3(ctx, Xq, x_scale, Wg_q, wg_scale, Wu_q, wu_scale, W_down, offsets, sorted_tok,
                              sorted_w, H, U, A, Yw, Wd_q=None, wd_scale=None, Aq=None, a_scale=None, stream=None):
    """e4m3 gate/up; the down projection in bf16 (W_down) or, given Wd_q / wd_scale and the Aq / a_scale
    buffers, in e4m3."""
    T, d = Xq.shape
    E, n, _ = Wg_q.shape
    cap = sorted_tok.numel()
    u8, f32 = torch.uint8, torch.float32
    head = (ctx.handle, _ptr(Xq, u8), _ptr(x_scale, f32), _ptr(Wg_q, u8), _ptr(wg_scale, f32), _ptr(Wu_q, u8),
            _ptr(wu_scale, f32), _ptr(W_down, torch.bfloat16), _ptr(Wd_q, u8), _ptr(wd_scale, f32), T, d, E, n, cap,
            _ptr(offsets, torch.int32), _ptr(sorted_tok, torch.int32), _ptr(sorted_w, f32))
    tail = (_ptr(A, torch.bfloat16), _ptr(Aq, u8), _ptr(a_scale, f32), _ptr(Yw, torch.bfloat16), _stream(stream))
    kept = _kept_pair(ctx, H, U, (cap, n))
    if kept:
        _check("moe_grouped_gemm_fwd_e4m3_kept8", lib().moe_grouped_gemm_fwd_e4m3_kept8(*head, *kept, *tail))
    else:
        _check("moe_grouped_gemm_fwd_e4m3", lib().moe_grouped_gemm_fwd_e4m3(*head, _ptr(H, f32), _ptr(U, f32), *tail))


def mx_sf_cols(cols: int) -> int:
    """Bytes per row of a row-major block-scale array (the library's moe_mx_sf_cols)."""
    return int(lib().moe_mx_sf_cols(cols))


def mx_weight_sf_bytes(E: int, d: int, n: int, which: int) -> int:
    """Bytes of the weight scale blocks: which = 0 the W_gate / W_up pair, 1 W_down."""
    b = int(lib().moe_mx_weight_sf_bytes(E, d, n, which))
    if b <= 0:
        raise ValueError(f"moe_mx_weight_sf_bytes: invalid arguments E={E} d={d} n={n} which={which}")
    return b


def mx_dw_ws_bytes(d: int, E: int, n: int, cap: int) -> int:
    """Bytes of the block-scaled weight gradients' workspace (``moe_mx_dw_ws_bytes``)."""
    b = int(lib().moe_mx_dw_ws_bytes(d, E, n, cap))
    if b <= 0:
        raise ValueError(f"moe_mx_dw_ws_bytes: invalid arguments d={d} E={E} n={n} cap={cap}")
    return b


def mx_act_sf_bytes(cap: int, E: int, n: int) -> int:
    """Bytes of the activation scale blocks of the block-scaled down projection."""
    b = int(lib().moe_mx_act_sf_bytes(cap, E, n))
    if b <= 0:
        raise ValueError(f"moe_mx_act_sf_bytes: invalid arguments cap={cap} E={E} n={n}")
    return b


def moe_quantize_rows_mx(ctx, M, q, sf, stream=None):
    """Block-scaled codes (uint8, shaped like M) and row-major scale bytes [rows, mx_sf_cols(cols)]."""
    cols = M.shape[-1]
    rows = M.numel() // cols
    if q.shape != M.shape or sf.numel() != rows * mx_sf_cols(cols):
        raise ValueError("q must be shaped like M and sf hold mx_sf_cols(cols) bytes per row")
    _check("moe_quantize_rows_mx", lib().moe_quantize_rows_mx(
        ctx.handle, _ptr(M, torch.bfloat16), rows, cols, _ptr(q, torch.uint8), _ptr(sf, torch.uint8),
        _stream(stream)))


def moe_quantize_weights_mx(ctx, W_gate, W_up, W_down, Wg_q, Wu_q, gu_sf, Wd_q, dn_sf, stream=None):
    E, n, d = W_gate.shape
    bf, u8 = torch.bfloat16, torch.uint8
    _check("moe_quantize_weights_mx", lib().moe_quantize_weights_mx(
        ctx.handle, _ptr(W_gate, bf), _ptr(W_up, bf), _ptr(W_down, bf), E, d, n, _ptr(Wg_q, u8), _ptr(Wu_q, u8),
        _ptr(gu_sf, u8), _ptr(Wd_q, u8), _ptr(dn_sf, u8), _stream(stream)))


def moe_grouped_gemm_fwd_mx(ctx, Xq, x_sf, w, offsets, sorted_tok, sorted_w, H, U, x_sf_tiles, Aq, a_sf, Yw,
                            stream=None):
    """Block-scaled gate/up (+ SwiGLU, A quantized in the epilogue) and down projection; ``w`` is MxWeights,
    ``x_sf_tiles`` scratch of mx_act_sf_bytes(cap, E, d) bytes."""
    T, d = Xq.shape
    E, n, _ = w.Wg_q.shape
    cap = sorted_tok.numel()
    u8, f32 = torch.uint8, torch.float32
    head = (ctx.handle, _ptr(Xq, u8), _ptr(x_sf, u8), _ptr(w.Wg_q, u8), _ptr(w.Wu_q, u8), _ptr(w.gu_sf, u8),
            _ptr(w.Wd_q, u8), _ptr(w.dn_sf, u8), T, d, E, n, cap, _ptr(offsets, torch.int32),
            _ptr(sorted_tok, torch.int32), _ptr(sorted_w, f32))
    tail = (_ptr(x_sf_tiles, u8), _ptr(Aq, u8), _ptr(a_sf, u8), _ptr(Yw, torch.bfloat16), _stream(stream))
    kept = _kept_pair(ctx, H, U, (cap, n))
    if kept:
        _check("moe_grouped_gemm_fwd_mx_kept8", lib().moe_grouped_gemm_fwd_mx_kept8(*head, *kept, *tail))
    else:
        _check("moe_grouped_gemm_fwd_mx", lib().moe_grouped_gemm_fwd_mx(*head, _ptr(H, f32), _ptr(U, f32), *tail))


def moe_combine(ctx, Yw, tok_ptr, tok_pairs, O, stream=None):
    T, d = O.shape
    _check("moe_combine", lib().moe_combine(
        ctx.handle, _ptr(Yw, torch.bfloat16), _ptr(tok_ptr, torch.int32), _ptr(tok_pairs, torch.int32), T, d,
        tok_pairs.numel(), _ptr(O, torch.bfloat16), _stream(stream)))


def moe_backward(ctx, dO, X, W_r, W_gate, W_up, W_down, K, m_tile, topk_ids, topk_w, offsets, sorted_tok,
                 sorted_w, tok_ptr, tok_pairs, H, U, dX, dW_gate, dW_up, dW_down, dS, dlogits, dW_r, ws,
                 stream=None):
    """Gradients of the layer.  With H and U as Kept8 (``ws`` of moe_kept8_workspace_bytes) X may be Kept8, too."""
    T, d = X.shape
    E, n, _ = W_gate.shape
    cap = sorted_tok.numel()
    wp, wb = _ws(ws)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    dw_fp32 = 1 if dW_gate.dtype == f32 else 0
    mid = (_ptr(W_r, bf), _ptr(W_gate, bf), _ptr(W_up, bf), _ptr(W_down, bf), T, d, E, n, K, m_tile, cap, _ptr(topk_ids, i32),
           _ptr(topk_w, f32), _ptr(offsets, i32), _ptr(sorted_tok, i32), _ptr(sorted_w, f32), _ptr(tok_ptr, i32),
           _ptr(tok_pairs, i32))
    tail = (_ptr(dX, bf), _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down), dw_fp32, _ptr(dS, f32), _ptr(dlogits, f32),
            _ptr(dW_r, f32), wp, wb, _stream(stream))
    kept = _kept_pair(ctx, H, U, (cap, n))
    if kept:
        _check("moe_backward_kept8", lib().moe_backward_kept8(
            ctx.handle, _ptr(dO, bf), *_kept_x(ctx, X, T, d), *mid, *kept, *tail))
    else:
        _check("moe_backward", lib().moe_backward(
            ctx.handle, _ptr(dO, bf), _ptr(_plain_x(X), bf), *mid, _ptr(H, f32), _ptr(U, f32), *tail))


def _plain_x(X):
    if isinstance(X, Kept8):
        raise ValueError("X kept in 8 bits goes with H and U kept in 8 bits")
    return X


def moe_kept8_workspace_bytes(T: int, d: int, E: int, n: int, K: int, m_tile: int = 0, cap: int | None = None) -> int:
    """Bytes of the workspace of a backward from activations kept in 8 bits (``cap``: the pair arrays' length where it is
    not moe_pair_capacity(T, E, K, m_tile))."""
    b = int(lib().moe_kept8_workspace_bytes(T, d, E, n, moe_pair_capacity(T, E, K, m_tile) if cap is None else cap))
    if b <= 0:
        raise ValueError(f"moe_kept8_workspace_bytes: invalid arguments T={T} d={d} E={E} n={n} K={K} m_tile={m_tile} cap={cap}")
    return b


def moe_quantize_dx_weights_e4m3(ctx, W_gate, W_up, Wgu_q, wgu_scale, stream=None):
    """[W_gate; W_up]^T per expert ([E, d, 2n]) as e4m3 codes with one scale per row (the dX GEMM's B)."""
    E, n, d = W_gate.shape
    tmp = torch.empty((E, d, 2 * n), dtype=torch.bfloat16, device=W_gate.device)
    _check("moe_quantize_dx_weights_e4m3", lib().moe_quantize_dx_weights_e4m3(
        ctx.handle, _ptr(W_gate, torch.bfloat16), _ptr(W_up, torch.bfloat16), E, n, d, _ptr(tmp, torch.bfloat16),
        _ptr(Wgu_q, torch.uint8), _ptr(wgu_scale, torch.float32), _stream(stream)))
    return tmp  # the caller keeps it alive until the stream has run the call


def moe_quantize_dact_weights_e4m3(ctx, W_down, Wdt_q, wdt_scale, stream=None):
    """W_down^T per expert ([E, n, d]) as e4m3 codes with one scale per row (the dSwiGLU GEMM's B)."""
    E, d, n = W_down.shape
    tmp = torch.empty((E, n, d), dtype=torch.bfloat16, device=W_down.device)
    _check("moe_quantize_dact_weights_e4m3", lib().moe_quantize_dact_weights_e4m3(
        ctx.handle, _ptr(W_down, torch.bfloat16), E, n, d, _ptr(tmp, torch.bfloat16), _ptr(Wdt_q, torch.uint8),
        _ptr(wdt_scale, torch.float32), _stream(stream)))
    return tmp  # the caller keeps it alive until the stream has run the call


def moe_backward_e4m3(ctx, dO, X, W_r, W_gate, W_up, W_down, Wgu_q, wgu_scale, Wdt_q, wdt_scale, K, m_tile, topk_ids,
                      topk_w, offsets, sorted_tok, sorted_w, tok_ptr, tok_pairs, H, U, HUq, hu_scale, dOq, do_scale,
                      dX, dW_gate, dW_up, dW_down, dS, dlogits, dW_r, ws, stream=None):
    T, d = X.shape
    E, n, _ = W_gate.shape
    cap = sorted_tok.numel()
    wp, wb = _ws(ws)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    dw_fp32 = 1 if dW_gate.dtype == torch.float32 else 0
    mid = (_ptr(W_r, bf), _ptr(W_gate, bf), _ptr(W_up, bf), _ptr(W_down, bf), _ptr(Wgu_q, torch.uint8), _ptr(wgu_scale, f32),
           _ptr(Wdt_q, torch.uint8), _ptr(wdt_scale, f32), T, d, E, n, K, m_tile, cap, _ptr(topk_ids, i32), _ptr(topk_w, f32),
           _ptr(offsets, i32), _ptr(sorted_tok, i32), _ptr(sorted_w, f32), _ptr(tok_ptr, i32), _ptr(tok_pairs, i32))
    tail = (_ptr(HUq, torch.uint8), _ptr(hu_scale, f32), _ptr(dOq, torch.uint8), _ptr(do_scale, f32), _ptr(dX, bf),
            _ptr(dW_gate), _ptr(dW_up), _ptr(dW_down), dw_fp32, _ptr(dS, f32), _ptr(dlogits, f32), _ptr(dW_r, f32), wp, wb,
            _stream(stream))
    kept = _kept_pair(ctx, H, U, (cap, n))
    if kept:
        _check("moe_backward_e4m3_kept8", lib().moe_backward_e4m3_kept8(
            ctx.handle, _ptr(dO, bf), *_kept_x(ctx, X, T, d), *mid, *kept, *tail))
    else:
        _check("moe_backward_e4m3", lib().moe_backward_e4m3(
            ctx.handle, _ptr(dO, bf), _ptr(_plain_x(X), bf), *mid, _ptr(H, f32), _ptr(U, f32), *tail))


# ------------------------------------------------------------------ around the layer


def _refuse(t, shape, dtype, name, ctx, what=""):
    raise ValueError(f"{name} must be a {what}{tuple(shape)} {dtype} tensor on CUDA device {ctx.device}, got "
                     f"{tuple(t.shape)} {t.dtype} with strides {t.stride()} on {t.device}")


def _rows(ctx, t: torch.Tensor | None, shape, dtype, name):
    """(pointer, row stride) of a [T, d] tensor whose columns are contiguous; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != ctx.device or t.shape != shape:
        _refuse(t, shape, dtype, name, ctx)
    if t.is_contiguous():
        return t.data_ptr(), shape[1]
    ld, one = t.stride()
    if (one != 1 and shape[1] > 1) or (ld < shape[1] and shape[0] > 1):
        _refuse(t, shape, dtype, name, ctx, "row-strided ")
    return t.data_ptr(), max(ld, shape[1])


def _flat(ctx, t: torch.Tensor | None, shape, dtype, name):
    """Pointer of a contiguous tensor of the given shape; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != ctx.device or t.shape != shape or not t.is_contiguous():
        _refuse(t, shape, dtype, name, ctx, "contiguous ")
    return t.data_ptr()


def _scratch(ctx, ws: torch.Tensor):
    """(pointer, bytes) of a workspace."""
    if ws.get_device() != ctx.device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on CUDA device {ctx.device}")
    return ws.data_ptr(), ws.nbytes


def _stream_type(t: torch.Tensor, name):
    """1 for an fp32 tensor, 0 for bf16."""
    if t.dtype == torch.float32:
        return 1
    if t.dtype == torch.bfloat16:
        return 0
    raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")


def moe_add_rmsnorm(ctx, x, residual, weight, eps, h, y, rstd=None, q=None, scales=None, stream=None):
    """h = residual + x, y = rmsnorm(h) * weight (bf16) and, with ``q`` and ``scales``, y's e4m3 codes: ``scales`` fp32
    [T] gives one scale a row (the per-row FP8 forward), uint8 [T, mx_sf_cols(d)] one power of two for 32 columns
    (the block-scaled forward).  ``residual`` and ``h`` are bf16 or fp32, ``weight`` bf16 or fp32; 2-D tensors may
    have any row stride.  ``x`` None: no addition (``h`` may then be None); ``y`` may be None when codes are
    written; ``rstd`` [T] is kept for the backward.  ``h`` may be ``residual`` and ``y`` may be ``x``."""
    shape = residual.shape
    if len(shape) != 2:
        raise ValueError(f"residual must be [T, d], got {tuple(shape)}")
    T, d = shape
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    rt = _stream_type(residual, "residual")
    (px, lx), (pr, lr) = _rows(ctx, x, shape, bf, "x"), _rows(ctx, residual, shape, residual.dtype, "residual")
    (ph, lh), (py, ly) = _rows(ctx, h, shape, residual.dtype, "h"), _rows(ctx, y, shape, bf, "y")
    wt = _stream_type(weight, "weight")
    form, ps = 0, None
    if q is not None or scales is not None:
        if q is None or scales is None:
            raise ValueError("q and scales go together")
        form = 1 if scales.dtype == f32 else 2
        ps = _flat(ctx, scales, (T,), f32, "scales") if form == 1 else _flat(ctx, scales, (T, 4 * -(-d // 128)), u8, "scales")
    _check("moe_add_rmsnorm", lib().moe_add_rmsnorm(
        ctx.handle, px, lx, pr, lr, rt, _flat(ctx, weight, (d,), weight.dtype, "weight"), wt, T, d, eps, ph, lh, py, ly,
        _flat(ctx, rstd, (T,), f32, "rstd"), form, _flat(ctx, q, shape, u8, "q"), ps, _stream(stream)))


def moe_add_rmsnorm_workspace_bytes(T: int, d: int) -> int:
    """Bytes of the norm backward's workspace."""
    b = int(lib().moe_add_rmsnorm_workspace_bytes(T, d))
    if b <= 0:
        raise ValueError(f"moe_add_rmsnorm_workspace_bytes: invalid arguments T={T} d={d}")
    return b


def moe_add_rmsnorm_backward(ctx, dy, h, weight, rstd, dh, dx, dresidual, dweight, ws, stream=None):
    """Gradients of moe_add_rmsnorm for ``dy`` (of y) and ``dh`` (of h along the residual stream, or None): the input's,
    as ``dx`` (bf16) and / or ``dresidual`` (the stream's type), and ``dweight`` [d] fp32.  ``ws``: uint8 of
    moe_add_rmsnorm_workspace_bytes(T, d)."""
    shape = h.shape
    if len(shape) != 2:
        raise ValueError(f"h must be [T, d], got {tuple(shape)}")
    T, d = shape
    bf, f32 = torch.bfloat16, torch.float32
    rt = _stream_type(h, "h")
    (pdy, ldy), (ph, lh) = _rows(ctx, dy, shape, bf, "dy"), _rows(ctx, h, shape, h.dtype, "h")
    (pdh, ldh), (pdx, ldx) = _rows(ctx, dh, shape, h.dtype, "dh"), _rows(ctx, dx, shape, bf, "dx")
    pdr, ldr = _rows(ctx, dresidual, shape, h.dtype, "dresidual")
    wt = _stream_type(weight, "weight")
    wp, wb = _scratch(ctx, ws)
    _check("moe_add_rmsnorm_backward", lib().moe_add_rmsnorm_backward(
        ctx.handle, pdy, ldy, ph, lh, rt, _flat(ctx, weight, (d,), weight.dtype, "weight"), wt,
        _flat(ctx, rstd, (T,), f32, "rstd"), pdh, ldh, T, d, pdx, ldx, pdr, ldr, _flat(ctx, dweight, (d,), f32, "dweight"), wp, wb,
        _stream(stream)))


def moe_balance_loss_workspace_bytes(T: int, E: int, B: int = 1) -> int:
    """Bytes of moe_balance_loss's workspace for B sequences."""
    b = int(lib().moe_balance_loss_workspace_bytes(T, E, B))
    if b <= 0:
        raise ValueError(f"moe_balance_loss_workspace_bytes: invalid arguments T={T} E={E} B={B}")
    return b


def moe_balance_loss(ctx, logits, topk_ids, balance_coef, z_coef, loss, counts, probs, dlogits, ws, mask=None,
                     seq_offsets=None, dloss=None, stream=None):
    """Balance loss and z loss of the router over the sequences of a packed batch: ``loss`` [3] = (balance_coef *
    balance + z_coef * z, balance, z), per sequence and expert the ``counts`` [B, E] int32 of the choices and the mean
    probabilities ``probs`` [B, E], and with ``dlogits`` [T, E] the gradient of loss[0] times ``dloss`` (a device
    scalar, None for 1).  ``mask`` [T] bool or uint8: tokens that count; ``seq_offsets`` [B + 1] int32.  ``ws``: uint8
    of moe_balance_loss_workspace_bytes(T, E, B)."""
    if logits.dim() != 2 or topk_ids.dim() != 2 or counts.dim() != 2:
        raise ValueError("logits, topk_ids and counts must be [T, E], [T, K] and [B, E]")
    T, E = logits.shape
    K, B = topk_ids.shape[1], counts.shape[0]
    f32, i32 = torch.float32, torch.int32
    if mask is not None and mask.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"mask must be bool or uint8, got {mask.dtype}")
    if seq_offsets is None and B != 1:
        raise ValueError(f"{B} sequences need seq_offsets")
    wp, wb = _scratch(ctx, ws)
    _check("moe_balance_loss", lib().moe_balance_loss(
        ctx.handle, _flat(ctx, logits, (T, E), f32, "logits"), _flat(ctx, topk_ids, (T, K), i32, "topk_ids"),
        _flat(ctx, mask, (T,), None if mask is None else mask.dtype, "mask"),
        _flat(ctx, seq_offsets, (B + 1,), i32, "seq_offsets"), T, E, K, B, balance_coef, z_coef,
        None if dloss is None else _flat(ctx, dloss.reshape(-1), (1,), f32, "dloss"), _flat(ctx, loss, (3,), f32, "loss"),
        _flat(ctx, counts, (B, E), i32, "counts"), _flat(ctx, probs, (B, E), f32, "probs"),
        _flat(ctx, dlogits, (T, E), f32, "dlogits"), wp, wb, _stream(stream)))


def moe_router_backward_workspace_bytes(T: int, d: int, E: int) -> int:
    """Bytes of moe_router_backward's workspace."""
    b = int(lib().moe_router_backward_workspace_bytes(T, d, E))
    if b <= 0:
        raise ValueError(f"moe_router_backward_workspace_bytes: invalid arguments T={T} d={d} E={E}")
    return b


def moe_router_backward(ctx, dlogits, X, W_r, dX_in, dW_r_in, dX, dW_r, ws, stream=None):
    """dX = dX_in + dlogits W_r^T (bf16) and dW_r = dW_r_in + X^T dlogits (fp32): what an additional loss on the router
    logits adds to the gradients that the layer's backward left.  ``dX_in`` / ``dW_r_in`` None: zero; an output may be
    its own input, and None skips its product.  ``ws``: uint8 of moe_router_backward_workspace_bytes(T, d, E)."""
    if dlogits.dim() != 2 or X.dim() != 2:
        raise ValueError("dlogits and X must be [T, E] and [T, d]")
    T, E = dlogits.shape
    d = X.shape[1]
    bf, f32 = torch.bfloat16, torch.float32
    wp, wb = _scratch(ctx, ws)
    _check("moe_router_backward", lib().moe_router_backward(
        ctx.handle, _flat(ctx, dlogits, (T, E), f32, "dlogits"), _flat(ctx, X, (T, d), bf, "X"), _flat(ctx, W_r, (d, E), bf, "W_r"), T, d,
        E, _flat(ctx, dX_in, (T, d), bf, "dX_in"), _flat(ctx, dW_r_in, (d, E), f32, "dW_r_in"), _flat(ctx, dX, (T, d), bf, "dX"),
        _flat(ctx, dW_r, (d, E), f32, "dW_r"), wp, wb, _stream(stream)))


# ------------------------------------------------------------------ a few tokens


def moe_few_workspace_bytes(T: int, d: int, E: int, n: int, K: int) -> int:
    """Bytes of the workspace of moe_forward_few and moe_forward_few_e4m3."""
    b = int(lib().moe_few_workspace_bytes(T, d, E, n, K))
    if b <= 0:
        raise ValueError(f"moe_few_workspace_bytes: invalid arguments T={T} d={d} E={E} n={n} K={K}")
    return b


def _few(ctx, X, W_r, bias, W_gate, W_up, W_down, dtype, K, O, topk_ids, topk_w, ws):
    """Sizes and checked pointers common to both forms of the layer for a few tokens."""
    if X.dim() != 2 or W_gate.dim() != 3:
        raise ValueError(f"X must be [T, d] and W_gate [E, n, d], got {tuple(X.shape)} and {tuple(W_gate.shape)}")
    T, d = X.shape
    E, n = W_gate.shape[:2]
    bf, f32 = torch.bfloat16, torch.float32
    px, lx = _rows(ctx, X, (T, d), bf, "X")
    po, lo = _rows(ctx, O, (T, d), bf, "O")
    head = (ctx.handle, px, lx, _flat(ctx, W_r, (d, E), bf, "W_r"), _flat(ctx, bias, (E,), f32, "bias"))
    weights = (_flat(ctx, W_gate, (E, n, d), dtype, "W_gate"), _flat(ctx, W_up, (E, n, d), dtype, "W_up"),
               _flat(ctx, W_down, (E, d, n), dtype, "W_down"))
    wp, wb = _scratch(ctx, ws)
    tail = (T, d, E, n, K, _flat(ctx, topk_ids, (T, K), torch.int32, "topk_ids"), _flat(ctx, topk_w, (T, K), f32, "topk_w"),
            po, lo, wp, wb)
    return head, weights, tail


def moe_forward_few(ctx, X, W_r, bias, W_gate, W_up, W_down, K, O, topk_ids, topk_w, ws, stream=None):
    """The whole layer for up to 64 tokens: ``topk_ids`` and ``topk_w`` [T, K] as moe_route gives them, ``O`` [T, d] bf16.
    ``X`` and ``O`` may have any row stride (a multiple of 8 and 4 elements).  ``ws``: uint8 of
    moe_few_workspace_bytes(T, d, E, n, K), one for each call that may overlap another."""
    head, w, tail = _few(ctx, X, W_r, bias, W_gate, W_up, W_down, torch.bfloat16, K, O, topk_ids, topk_w, ws)
    _check("moe_forward_few", lib().moe_forward_few(*head, *w, *tail, _stream(stream)))


def moe_forward_few_e4m3(ctx, X, W_r, bias, w8, K, O, topk_ids, topk_w, ws, stream=None):
    """moe_forward_few on e4m3 weights (``w8``: E4m3Weights with W_down's codes); the call quantizes X and the activations."""
    if w8.Wd_q is None:
        raise ValueError("moe_forward_few_e4m3 needs W_down's codes (E4m3Weights.quantize with W_down)")
    head, (g, u, dn), tail = _few(ctx, X, W_r, bias, w8.Wg_q, w8.Wu_q, w8.Wd_q, torch.uint8, K, O, topk_ids, topk_w, ws)
    E, n, d = w8.Wg_q.shape
    f32 = torch.float32
    _check("moe_forward_few_e4m3", lib().moe_forward_few_e4m3(
        *head, g, _flat(ctx, w8.wg_scale, (E, n), f32, "wg_scale"), u, _flat(ctx, w8.wu_scale, (E, n), f32, "wu_scale"),
        dn, _flat(ctx, w8.wd_scale, (E, d), f32, "wd_scale"), *tail, _stream(stream)))


@dataclass
class FewBuffers:
    """Outputs and workspace of the layer for up to T tokens (a decoding step of T sequences), T <= 64."""

    O: torch.Tensor         # [T, d] bf16
    topk_ids: torch.Tensor  # [T, K] int32
    topk_w: torch.Tensor    # [T, K] fp32
    ws: torch.Tensor

    @staticmethod
    def allocate(T, d, E, n, K, device="cuda") -> "FewBuffers":
        return FewBuffers(torch.zeros((T, d), dtype=torch.bfloat16, device=device),
                          torch.zeros((T, K), dtype=torch.int32, device=device), torch.zeros((T, K), device=device),
                          torch.empty(moe_few_workspace_bytes(T, d, E, n, K), dtype=torch.uint8, device=device))


def forward_few(ctx, X, W_r, bias, weights, buf: FewBuffers, stream=None):
    """The layer for the few tokens of X [T, d], at most those that ``buf`` has room for; the output is ``buf.O[:T]``.
    ``weights``: (W_gate, W_up, W_down) in bf16, or E4m3Weights."""
    T, K = X.shape[0], buf.topk_ids.shape[1]
    out = K, buf.O[:T], buf.topk_ids[:T], buf.topk_w[:T], buf.ws, stream
    if isinstance(weights, E4m3Weights):
        moe_forward_few_e4m3(ctx, X, W_r, bias, weights, *out)
    else:
        moe_forward_few(ctx, X, W_r, bias, *weights, *out)


def moe_test_gemm_varlen_m(ctx, A, idx, B, b_kmajor, offsets, D, stream=None):
    G = B.shape[0]
    K = A.shape[1]
    N = B.shape[1] if b_kmajor else B.shape[2]
    _check("moe_test_gemm_varlen_m", lib().moe_test_gemm_varlen_m(
        ctx.handle, _ptr(A, torch.bfloat16), _ptr(idx, torch.int32), _ptr(B, torch.bfloat16), int(b_kmajor), G,
        A.shape[0], K, N, D.shape[0], _ptr(offsets, torch.int32), _ptr(D, torch.float32), _stream(stream)))


def moe_test_gemm_varlen_k(ctx, A, idx_a, B, idx_b, offsets, D, cap, stream=None):
    G, M, N = D.shape
    _check("moe_test_gemm_varlen_k", lib().moe_test_gemm_varlen_k(
        ctx.handle, _ptr(A, torch.bfloat16), _ptr(idx_a, torch.int32), A.shape[0], _ptr(B, torch.bfloat16),
        _ptr(idx_b, torch.int32), B.shape[0], G, M, N, cap, _ptr(offsets, torch.int32), _ptr(D, torch.float32),
        _stream(stream)))


def moe_test_gemm_varlen_m_dual(ctx, A_hi, A_lo, B, offsets, D, stream=None):
    """Test export: per group and sorted row, (A_hi + A_lo) B[e]^T (B is [G, N, K]); D is [cap, N] fp32."""
    G, N, K = B.shape
    _check("moe_test_gemm_varlen_m_dual", lib().moe_test_gemm_varlen_m_dual(
        ctx.handle, _ptr(A_hi, torch.bfloat16), _ptr(A_lo, torch.bfloat16), _ptr(B, torch.bfloat16), G,
        A_hi.shape[0], K, N, D.shape[0], _ptr(offsets, torch.int32), _ptr(D, torch.float32), _stream(stream)))


def moe_test_gemm_varlen_k_dual(ctx, A_hi, A_lo, B, offsets, D, cap, trans=False, b_offsets=None, stream=None):
    """Test export: per group, (A_hi + A_lo)^T B over the group's rows (D [G, M, N], or [G, N, M] with trans);
    b_offsets: B's rows in the padded layout (groups rounded up to 16 rows, zero rows in between)."""
    G = D.shape[0]
    M = A_hi.shape[1]
    N = B.shape[1]
    _check("moe_test_gemm_varlen_k_dual", lib().moe_test_gemm_varlen_k_dual(
        ctx.handle, _ptr(A_hi, torch.bfloat16), _ptr(A_lo, torch.bfloat16), A_hi.shape[0], _ptr(B, torch.bfloat16),
        B.shape[0], G, M, N, cap, _ptr(offsets, torch.int32), _ptr(b_offsets, torch.int32), int(bool(trans)),
        _ptr(D, torch.float32), _stream(stream)))


def moe_test_wait_timeout(ctx, timeout_ns: int, stream=None):
    _check("moe_test_wait_timeout", lib().moe_test_wait_timeout(ctx.handle, int(timeout_ns), _stream(stream)))


# ------------------------------------------------------------------ buffers and the whole path


@dataclass
class Buffers:
    """Every device tensor of one forward + backward for sizes (T, d, E, n, K, m_tile)."""

    T: int
    d: int
    E: int
    n: int
    K: int
    m_tile: int
    cap: int
    logits: torch.Tensor
    scores: torch.Tensor | None
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    sorted_tok: torch.Tensor
    sorted_w: torch.Tensor
    tok_ptr: torch.Tensor
    tok_pairs: torch.Tensor
    P: torch.Tensor
    H: torch.Tensor | Kept8
    U: torch.Tensor | Kept8
    A: torch.Tensor
    Yw: torch.Tensor
    O: torch.Tensor
    dX: torch.Tensor | None
    dW_gate: torch.Tensor | None
    dW_up: torch.Tensor | None
    dW_down: torch.Tensor | None
    dS: torch.Tensor | None
    dlogits: torch.Tensor | None
    dW_r: torch.Tensor | None
    ws: torch.Tensor
    capacity: int = 0          # capacity dispatch: slots per expert (0 = ragged)
    drop_policy: str = "position"
    xq: torch.Tensor | None = None  # e4m3 forward: X's codes [T, d] and per-token scales [T]
    xs: torch.Tensor | None = None
    aq: torch.Tensor | None = None  # e4m3 down projection: A's codes [cap, n] and per-row scales [cap]
    as_: torch.Tensor | None = None
    huq: torch.Tensor | None = None  # e4m3 dX GEMM: [dH | dU] codes [cap, 2n] and per-row scales [cap]
    hus: torch.Tensor | None = None
    doq: torch.Tensor | None = None  # e4m3 dSwiGLU GEMM: sorted dO codes [cap, d] and per-row scales [cap]
    dos: torch.Tensor | None = None
    mxq: torch.Tensor | None = None  # block-scaled forward: X's codes [T, d] and scales [T, mx_sf_cols(d)]
    mxsf: torch.Tensor | None = None
    maq: torch.Tensor | None = None  # block-scaled down projection: A's codes [cap, n] and scale blocks
    masf: torch.Tensor | None = None
    mxsft: torch.Tensor | None = None  # block-scaled gate/up: the gathered X rows' scales per sorted row tile
    mdoq: torch.Tensor | None = None  # block-scaled backward: sorted dO codes [cap, d], their scales per row tile,
    mdosft: torch.Tensor | None = None  # [dH | dU] codes [cap, 2n] and their scale blocks
    mhuq: torch.Tensor | None = None
    mhusf: torch.Tensor | None = None
    mdw: torch.Tensor | None = None  # block-scaled weight gradients' workspace (moe_mx_dw_ws_bytes), on first use
    xk: Kept8 | None = None  # activations kept in 8 bits: X (H and U are Kept8, too)

    @staticmethod
    def allocate(T, d, E, n, K, m_tile=0, backward=True, dW_dtype=torch.bfloat16, device="cuda", capacity=0,
                 drop_policy="position", capacity_factor=0.0, e4m3=False, mx=False, kept8=False):
        """Buffers for one configuration; capacity > 0 (or capacity_factor > 0, giving
        ceil(capacity_factor * T * K / E)) selects the capacity (drop/pad) dispatch with that many slots per
        expert (pair-indexed arrays sized E * capacity).  ``kept8``: the forwards keep X, H and U in 8 bits (Kept8) for the
        backward, which then takes None for X."""
        if capacity_factor and not capacity:
            capacity = expert_capacity(T, E, K, capacity_factor)
        if capacity and m_tile:
            raise ValueError("token rounding and the capacity dispatch are exclusive")
        cap = E * capacity if capacity else moe_pair_capacity(T, E, K, m_tile)
        f32, i32, bf = torch.float32, torch.int32, torch.bfloat16

        def z(shape, dt):
            return torch.zeros(shape, dtype=dt, device=device)

        ws_bytes = moe_capacity_workspace_bytes(T, d, E, n, K, capacity) if capacity else \
            moe_workspace_bytes(T, d, E, n, K, m_tile)
        if ws_bytes == 0:
            raise ValueError(f"unsupported sizes T={T} d={d} E={E} n={n} K={K}")
        if kept8:
            ws_bytes = max(ws_bytes, moe_kept8_workspace_bytes(T, d, E, n, K, cap=cap))
        return Buffers(
            T, d, E, n, K, m_tile, cap,
            logits=z((T, E), f32), scores=z((T, E), f32) if m_tile else None,
            topk_ids=z((T, K), i32), topk_w=z((T, K), f32), counts=z((E,), i32), offsets=z((E + 1,), i32),
            sorted_tok=z((cap,), i32), sorted_w=z((cap,), f32), tok_ptr=z((T + 1,), i32),
            tok_pairs=z((cap,), i32), P=z((1,), i32),
            H=Kept8.empty(cap, n, device) if kept8 else z((cap, n), f32),
            U=Kept8.empty(cap, n, device) if kept8 else z((cap, n), f32), xk=Kept8.empty(T, d, device) if kept8 else None, A=z((cap, n), bf), Yw=z((cap, d), bf), O=z((T, d), bf),
            dX=z((T, d), bf) if backward else None,
            dW_gate=z((E, n, d), dW_dtype) if backward else None,
            dW_up=z((E, n, d), dW_dtype) if backward else None,
            dW_down=z((E, d, n), dW_dtype) if backward else None,
            dS=z((cap,), f32) if backward else None, dlogits=z((T, E), f32) if backward else None,
            dW_r=z((d, E), f32) if backward else None,
            ws=torch.empty(ws_bytes, dtype=torch.uint8, device=device), capacity=capacity, drop_policy=drop_policy,
            xq=z((T, d), torch.uint8) if e4m3 else None, xs=z((T,), f32) if e4m3 else None,
            aq=z((cap, n), torch.uint8) if e4m3 else None, as_=z((cap,), f32) if e4m3 else None,
            huq=z((cap, 2 * n), torch.uint8) if (e4m3 and backward) else None,
            hus=z((cap,), f32) if (e4m3 and backward) else None,
            doq=z((cap, d), torch.uint8) if (e4m3 and backward) else None,
            dos=z((cap,), f32) if (e4m3 and backward) else None,
            mxq=z((T, d), torch.uint8) if mx else None, mxsf=z((T, mx_sf_cols(d)), torch.uint8) if mx else None,
            maq=z((cap, n), torch.uint8) if mx else None,
            masf=z((mx_act_sf_bytes(cap, E, n),), torch.uint8) if mx else None,
            mxsft=z((mx_act_sf_bytes(cap, E, d),), torch.uint8) if mx else None,
            mdoq=z((cap, d), torch.uint8) if (mx and backward) else None,
            mdosft=z((mx_act_sf_bytes(cap, E, d),), torch.uint8) if (mx and backward) else None,
            mhuq=z((cap, 2 * n), torch.uint8) if (mx and backward) else None,
            mhusf=z((mx_act_sf_bytes(cap, E, 2 * n),), torch.uint8) if (mx and backward) else None)


def _keep_x(ctx, X, buf: Buffers, cache, stream):
    if cache and buf.xk is not None:
        moe_keep_rows8(ctx, X, buf.xk, stream)


def _kept_input(X, buf: Buffers):
    """The backward's X: the caller's, or the one kept in 8 bits."""
    if X is None and buf.xk is None:
        raise ValueError("the backward needs X (buffers allocated with kept8=True keep it)")
    return buf.xk if X is None else X


def forward(ctx, X, W_r, bias, W_gate, W_up, W_down, buf: Buffers, stream=None, cache=True):
    """Routing, grouping, grouped GEMMs and combine; the output is ``buf.O``.  ``cache=False``: forward only,
    the activations that the backward needs (H and U; with ``kept8`` buffers X, too) are not written."""
    moe_route(ctx, X, W_r, bias, buf.K, buf.logits, buf.scores, buf.topk_ids, buf.topk_w, buf.ws, stream)
    if buf.capacity:
        moe_permute_capacity(ctx, buf.topk_ids, buf.topk_w, buf.E, buf.capacity, buf.drop_policy, buf.counts,
                             buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.P, buf.ws,
                             stream)
    else:
        moe_permute(ctx, buf.topk_ids, buf.topk_w, buf.logits, buf.scores, buf.E, buf.m_tile, buf.counts,
                    buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.P, buf.ws, stream)
    _keep_x(ctx, X, buf, cache, stream)
    moe_grouped_gemm_fwd(ctx, X, W_gate, W_up, W_down, buf.offsets, buf.sorted_tok, buf.sorted_w,
                         buf.H if cache else None, buf.U if cache else None, buf.A, buf.Yw, buf.ws, stream)
    moe_combine(ctx, buf.Yw, buf.tok_ptr, buf.tok_pairs, buf.O, stream)


@dataclass
class MxWeights:
    """The expert weights as block-scaled e4m3 (1 x 32 blocks along each row, power-of-two scales): codes
    Wg_q, Wu_q [E, n, d], Wd_q [E, d, n] (uint8) and the scale blocks the GEMMs read (gu_sf, dn_sf)."""

    Wg_q: torch.Tensor
    Wu_q: torch.Tensor
    gu_sf: torch.Tensor
    Wd_q: torch.Tensor
    dn_sf: torch.Tensor
    Wdt_q: torch.Tensor | None = None  # the backward: W_down^T codes [E, n, d] and scale blocks
    wdt_sf: torch.Tensor | None = None
    Wgu_q: torch.Tensor | None = None  # [W_gate; W_up]^T codes [E, d, 2n] and scale blocks
    wgu_sf: torch.Tensor | None = None

    @staticmethod
    def quantize(ctx, W_gate, W_up, W_down, stream=None, backward=False) -> "MxWeights":
        """The forward's codes and scale blocks; with ``backward`` also the two backward operands."""
        E, n, d = W_gate.shape
        dev = W_gate.device
        u8 = torch.uint8
        w = MxWeights(torch.empty((E, n, d), dtype=u8, device=dev), torch.empty((E, n, d), dtype=u8, device=dev),
                      torch.empty(mx_weight_sf_bytes(E, d, n, 0), dtype=u8, device=dev),
                      torch.empty((E, d, n), dtype=u8, device=dev),
                      torch.empty(mx_weight_sf_bytes(E, d, n, 1), dtype=u8, device=dev))
        moe_quantize_weights_mx(ctx, W_gate, W_up, W_down, w.Wg_q, w.Wu_q, w.gu_sf, w.Wd_q, w.dn_sf, stream)
        if backward:
            w.Wdt_q = torch.empty((E, n, d), dtype=u8, device=dev)
            w.wdt_sf = torch.empty(mx_weight_sf_bytes(E, d, n, 2), dtype=u8, device=dev)
            w.Wgu_q = torch.empty((E, d, 2 * n), dtype=u8, device=dev)
            w.wgu_sf = torch.empty(mx_weight_sf_bytes(E, d, n, 3), dtype=u8, device=dev)
            tmp = torch.empty((E, d, 2 * n), dtype=torch.bfloat16, device=dev)
            _check("moe_quantize_bwd_weights_mx", lib().moe_quantize_bwd_weights_mx(
                ctx.handle, _ptr(W_gate, torch.bfloat16), _ptr(W_up, torch.bfloat16), _ptr(W_down, torch.bfloat16),
                E, d, n, _ptr(tmp), _ptr(w.Wdt_q, u8), _ptr(w.wdt_sf, u8), _ptr(w.Wgu_q, u8), _ptr(w.wgu_sf, u8),
                _stream(stream)))
            torch.cuda.synchronize(dev)  # the scratch copy may go once the call has run
            del tmp
        return w


@dataclass
class E4m3Weights:
    """W_gate and W_up as e4m3 codes [E, n, d] (uint8) with one fp32 scale per output channel [E, n]; with
    W_down given, W_down as codes [E, d, n] with scales [E, d] too (the e4m3 down projection)."""

    Wg_q: torch.Tensor
    wg_scale: torch.Tensor
    Wu_q: torch.Tensor
    wu_scale: torch.Tensor
    Wd_q: torch.Tensor | None = None
    wd_scale: torch.Tensor | None = None
    Wgu_q: torch.Tensor | None = None  # the e4m3 dX GEMM: [W_gate; W_up]^T codes [E, d, 2n], scales [E, d]
    wgu_scale: torch.Tensor | None = None
    Wdt_q: torch.Tensor | None = None  # the e4m3 dSwiGLU GEMM: W_down^T codes [E, n, d], scales [E, n]
    wdt_scale: torch.Tensor | None = None

    @staticmethod
    def quantize(ctx, W_gate, W_up, W_down=None, stream=None, backward=False) -> "E4m3Weights":
        """The forward's codes (W_down's too when given); with ``backward`` also the two backward copies
        ([W_gate; W_up]^T for the dX GEMM, W_down^T for the dSwiGLU GEMM; W_down required)."""
        E, n, d = W_gate.shape
        dev = W_gate.device
        w = E4m3Weights(torch.empty((E, n, d), dtype=torch.uint8, device=dev),
                        torch.empty((E, n), dtype=torch.float32, device=dev),
                        torch.empty((E, n, d), dtype=torch.uint8, device=dev),
                        torch.empty((E, n), dtype=torch.float32, device=dev))
        moe_quantize_rows_e4m3(ctx, W_gate, w.Wg_q, w.wg_scale, stream)
        moe_quantize_rows_e4m3(ctx, W_up, w.Wu_q, w.wu_scale, stream)
        if W_down is not None:
            w.Wd_q = torch.empty((E, d, n), dtype=torch.uint8, device=dev)
            w.wd_scale = torch.empty((E, d), dtype=torch.float32, device=dev)
            moe_quantize_rows_e4m3(ctx, W_down, w.Wd_q, w.wd_scale, stream)
        if backward:
            if W_down is None:
                raise ValueError("the backward codes need W_down")
            w.Wgu_q = torch.empty((E, d, 2 * n), dtype=torch.uint8, device=dev)
            w.wgu_scale = torch.empty((E, d), dtype=torch.float32, device=dev)
            tmp = moe_quantize_dx_weights_e4m3(ctx, W_gate, W_up, w.Wgu_q, w.wgu_scale, stream)
            w.Wdt_q = torch.empty((E, n, d), dtype=torch.uint8, device=dev)
            w.wdt_scale = torch.empty((E, n), dtype=torch.float32, device=dev)
            tmp2 = moe_quantize_dact_weights_e4m3(ctx, W_down, w.Wdt_q, w.wdt_scale, stream)
            torch.cuda.synchronize(dev)  # the scratch copies may go once the calls have run
            del tmp, tmp2
        return w


def forward_e4m3(ctx, X, W_r, bias, w8: E4m3Weights, W_down, buf: Buffers, stream=None, cache=True, quantized=False):
    """The forward with the gate/up GEMM on e4m3 operands (``buf`` allocated with ``e4m3=True``): routing and
    grouping as ``forward``, X quantized per token, then the e4m3 grouped GEMMs and the combine.  When ``w8``
    holds W_down's codes the down projection runs on e4m3 operands too (``W_down`` may then be None).
    ``cache=False``: forward only (H, U not written).  ``quantized=True``: ``buf.xq`` and ``buf.xs`` already hold X's
    codes and scales (as moe_add_rmsnorm writes them); X itself serves the routing."""
    if buf.xq is None:
        raise ValueError("buffers were allocated without e4m3=True")
    moe_route(ctx, X, W_r, bias, buf.K, buf.logits, buf.scores, buf.topk_ids, buf.topk_w, buf.ws, stream)
    if buf.capacity:
        moe_permute_capacity(ctx, buf.topk_ids, buf.topk_w, buf.E, buf.capacity, buf.drop_policy, buf.counts,
                             buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.P, buf.ws,
                             stream)
    else:
        moe_permute(ctx, buf.topk_ids, buf.topk_w, buf.logits, buf.scores, buf.E, buf.m_tile, buf.counts,
                    buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.P, buf.ws, stream)
    if not quantized:
        moe_quantize_rows_e4m3(ctx, X, buf.xq, buf.xs, stream)
    _keep_x(ctx, X, buf, cache, stream)
    moe_grouped_gemm_fwd_e4m3(ctx, buf.xq, buf.xs, w8.Wg_q, w8.wg_scale, w8.Wu_q, w8.wu_scale,
                              None if w8.Wd_q is not None else W_down, buf.offsets, buf.sorted_tok, buf.sorted_w,
                              buf.H if cache else None, buf.U if cache else None, buf.A, buf.Yw, Wd_q=w8.Wd_q,
                              wd_scale=w8.wd_scale,
                              Aq=buf.aq if w8.Wd_q is not None else None,
                              a_scale=buf.as_ if w8.Wd_q is not None else None, stream=stream)
    moe_combine(ctx, buf.Yw, buf.tok_ptr, buf.tok_pairs, buf.O, stream)


def forward_mx(ctx, X, W_r, bias, wmx: MxWeights, buf: Buffers, stream=None, cache=True, quantized=False):
    """The forward on block-scaled e4m3 operands (``buf`` allocated with ``mx=True``): routing and grouping as
    ``forward``, X quantized in 1 x 32 blocks, the gate/up GEMM (whose epilogue quantizes A), the down
    projection and the combine.  ``cache=False``: forward only (H, U not written).  ``quantized=True``: ``buf.mxq`` and
    ``buf.mxsf`` already hold X's codes and scales (as moe_add_rmsnorm writes them)."""
    if buf.mxq is None:
        raise ValueError("buffers were allocated without mx=True")
    moe_route(ctx, X, W_r, bias, buf.K, buf.logits, buf.scores, buf.topk_ids, buf.topk_w, buf.ws, stream)
    if buf.capacity:
        moe_permute_capacity(ctx, buf.topk_ids, buf.topk_w, buf.E, buf.capacity, buf.drop_policy, buf.counts,
                             buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.P, buf.ws,
                             stream)
    else:
        moe_permute(ctx, buf.topk_ids, buf.topk_w, buf.logits, buf.scores, buf.E, buf.m_tile, buf.counts,
                    buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.P, buf.ws, stream)
    if not quantized:
        moe_quantize_rows_mx(ctx, X, buf.mxq, buf.mxsf, stream)
    _keep_x(ctx, X, buf, cache, stream)
    moe_grouped_gemm_fwd_mx(ctx, buf.mxq, buf.mxsf, wmx, buf.offsets, buf.sorted_tok, buf.sorted_w,
                            buf.H if cache else None, buf.U if cache else None, buf.mxsft, buf.maq, buf.masf, buf.Yw,
                            stream)
    moe_combine(ctx, buf.Yw, buf.tok_ptr, buf.tok_pairs, buf.O, stream)


def backward_mx(ctx, dO, X, W_r, W_gate, W_up, W_down, wmx: MxWeights, buf: Buffers, stream=None, dw=False):
    """The backward with the dSwiGLU and dX GEMMs on block-scaled operands (``wmx`` quantized with
    ``backward=True``, ``buf`` allocated with ``mx=True``); with ``dw`` the weight gradients too (blocks of 32
    tokens of one expert), else they stay bf16 on dH, dU, A' rounded once to bf16.  The block-scaled weight
    gradients are slower on one GB300 (c2 step 1.20 against 0.94 ms): with short per-expert reductions the
    GEMMs are bound by per-tile work, not by the tensor cores, and their operands take a transposing
    quantization pass."""
    if wmx.Wdt_q is None or buf.mhuq is None:
        raise ValueError("block-scaled backward needs MxWeights.quantize(..., backward=True) and Buffers(mx=True)")
    X = _kept_input(X, buf)
    T, d = X.shape
    E, n, _ = W_gate.shape
    cap = buf.sorted_tok.numel()
    wp, wb = _ws(buf.ws)
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    dw_fp32 = 1 if buf.dW_gate.dtype == f32 else 0
    if dw and buf.mdw is None:
        buf.mdw = torch.empty(mx_dw_ws_bytes(d, E, n, cap), dtype=u8, device=dO.device)
    mid = (_ptr(W_r, bf), _ptr(W_gate, bf), _ptr(W_up, bf), _ptr(W_down, bf), _ptr(wmx.Wdt_q, u8), _ptr(wmx.wdt_sf, u8),
           _ptr(wmx.Wgu_q, u8), _ptr(wmx.wgu_sf, u8), T, d, E, n, buf.K, buf.m_tile, cap, _ptr(buf.topk_ids, i32),
           _ptr(buf.topk_w, f32), _ptr(buf.offsets, i32), _ptr(buf.sorted_tok, i32), _ptr(buf.sorted_w, f32),
           _ptr(buf.tok_ptr, i32), _ptr(buf.tok_pairs, i32))
    tail = (_ptr(buf.mdoq, u8), _ptr(buf.mdosft, u8), _ptr(buf.mhuq, u8), _ptr(buf.mhusf, u8), _ptr(buf.dX, bf),
            _ptr(buf.dW_gate), _ptr(buf.dW_up), _ptr(buf.dW_down), dw_fp32, _ptr(buf.dS, f32), _ptr(buf.dlogits, f32),
            _ptr(buf.dW_r, f32), wp, wb, _ptr(buf.mdw, u8) if dw else None, buf.mdw.numel() if dw else 0, _stream(stream))
    kept = _kept_pair(ctx, buf.H, buf.U, (cap, n))
    if kept:
        _check("moe_backward_mx_kept8", lib().moe_backward_mx_kept8(
            ctx.handle, _ptr(dO, bf), *_kept_x(ctx, X, T, d), *mid, *kept, *tail))
    else:
        _check("moe_backward_mx", lib().moe_backward_mx(
            ctx.handle, _ptr(dO, bf), _ptr(_plain_x(X), bf), *mid, _ptr(buf.H, f32), _ptr(buf.U, f32), *tail))


def backward_e4m3(ctx, dO, X, W_r, W_gate, W_up, W_down, w8: E4m3Weights, buf: Buffers, stream=None, dx=True,
                  dact=True):
    """The backward with the dX GEMM (``dx``) and the dSwiGLU GEMM (``dact``) on e4m3 operands (``w8`` quantized
    with ``backward=True``, ``buf`` allocated with ``e4m3=True``); the weight gradients stay bf16, on dH, dU and
    A' rounded once to bf16.  Measured on one GB300, the e4m3 training step is faster than bf16 by 1.55x at
    d = 7168, n = 2048, 1.23x at d = 2048, n = 512 and 1.07x at d = 1536, n = 256 (where the per-row
    quantization passes take most of what the shorter GEMMs save)."""
    if w8.Wgu_q is None or buf.huq is None:
        raise ValueError("e4m3 backward needs E4m3Weights.quantize(..., backward=True) and Buffers(e4m3=True)")
    X = _kept_input(X, buf)
    moe_backward_e4m3(ctx, dO, X, W_r, W_gate, W_up, W_down, w8.Wgu_q if dx else None, w8.wgu_scale if dx else None,
                      w8.Wdt_q if dact else None, w8.wdt_scale if dact else None, buf.K, buf.m_tile, buf.topk_ids,
                      buf.topk_w, buf.offsets, buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.H, buf.U,
                      buf.huq if dx else None, buf.hus if dx else None, buf.doq if dact else None,
                      buf.dos if dact else None, buf.dX, buf.dW_gate, buf.dW_up, buf.dW_down, buf.dS, buf.dlogits,
                      buf.dW_r, buf.ws, stream)


def backward(ctx, dO, X, W_r, W_gate, W_up, W_down, buf: Buffers, stream=None):
    """Gradients into ``buf``; X None: the X that a forward on ``kept8`` buffers kept."""
    moe_backward(ctx, dO, _kept_input(X, buf), W_r, W_gate, W_up, W_down, buf.K, buf.m_tile, buf.topk_ids, buf.topk_w, buf.offsets,
                 buf.sorted_tok, buf.sorted_w, buf.tok_ptr, buf.tok_pairs, buf.H, buf.U, buf.dX, buf.dW_gate,
                 buf.dW_up, buf.dW_down, buf.dS, buf.dlogits, buf.dW_r, buf.ws, stream)


class StepGraph:
    """One forward + backward (``backward=False``: the forward) captured as a CUDA graph for fixed tensors and
    buffers.  The library's host work (argument checks, tensor-map encoding, launch configuration) runs once, at
    capture; ``replay()`` launches the whole step at once on the current stream.  New inputs are copied into the
    captured tensors (same addresses) before a replay; outputs land in ``buf`` as with the eager calls."""

    def __init__(self, ctx, X, W_r, bias, W_gate, W_up, W_down, dO, buf: Buffers, backward=True):
        def run():
            if backward:
                forward_backward(ctx, X, W_r, bias, W_gate, W_up, W_down, dO, buf)
            else:
                forward(ctx, X, W_r, bias, W_gate, W_up, W_down, buf)
        side = torch.cuda.Stream(device=X.device)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # one eager pass outside the capture (first-use configuration)
            run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize(X.device)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            run()
        torch.cuda.synchronize(X.device)

    def replay(self):
        self.graph.replay()


def forward_backward(ctx, X, W_r, bias, W_gate, W_up, W_down, dO, buf: Buffers, stream=None):
    forward(ctx, X, W_r, bias, W_gate, W_up, W_down, buf, stream)
    backward(ctx, dO, X, W_r, W_gate, W_up, W_down, buf, stream)
