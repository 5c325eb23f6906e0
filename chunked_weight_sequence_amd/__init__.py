"""Chunked test-time-training fast-weight scan for MI355X (gfx950): Python binding.

A thin ctypes layer over ``libttt_mi355x.so`` (declared in ``include/ttt_mi355x.h``). It only
marshals arguments: PyTorch supplies device memory and the current HIP stream, and every step of
the computation runs in the library's HIP kernels. There is no fallback of any kind: if the
library is missing or the tensors are not on the GPU, the call raises.

    O, W = chunk_scan(Z, Vhat, W0, chunk=512, eta=1e-4)          # In-Place TTT
    O, W, loss = linear_minibatch(Q, K, V, minibatch=16, eta=0.1)  # TTT-Linear
    cache = surprisal_route(loss, K, V, chunk=64)                 # SR-TTT routing
    Vhat = lm_target(X0, conv_w, W_target, chunk=512)            # In-Place TTT target

The attention half of a block, over a packed prompt and then token by token:

    inv_freq, rope_scale = rope_frequencies(128, base=1e6)
    q, k = qk_norm_rope(Q, K, pos, inv_freq, V=V, K_cache=Kc, V_cache=Vc, slots=slots)
    O = attention_packed(q, k, V, cu_seqlens)
    O = attention_decode(q, Kc, Vc, page_table, lengths, page_size=64)

or prompts in pieces, mixed with single tokens, over the same cache:

    O = attention_paged(q, Kc, Vc, cu_q, page_table, lengths, page_size=64)

Between the halves, and fast weights that forget:

    y, _, x = add_rms_norm(O, weight, residual=x)
    O, states = gated_delta_packed(Q, K, V, g, beta, cu_seqlens, state=states, slots=slots)
    O, states = gated_delta_decode(Q, K, V, g, beta, states, slots=slots)
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

__all__ = [
    "lib", "library_path", "TTTError", "abi_version", "status_string",
    "chunk_scan", "chunk_scan_workspace_bytes", "chunk_scan_profile",
    "linear_minibatch", "surprisal_route", "lm_target", "gated_z", "cache_readout", "chunk_scan_docs",
    "chunk_scan_handover_timeouts", "scan_test_overrides", "chunk_scan_noalloc",
    "rope_frequencies", "qk_norm_rope", "attention_packed", "attention_decode",
    "attention_paged", "add_rms_norm", "gated_delta_packed", "gated_delta_decode", "EXPORTED",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libttt_mi355x.so")

TTT_F32, TTT_BF16 = 0, 1
ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
SCAN_PHASES = ("stage", "corr", "update", "apply")

# name -> (restype, argtypes); mirrors include/ttt_mi355x.h
_p, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_d, _ll = ctypes.c_double, ctypes.c_longlong
_SCAN_ARGS = [_p, _p, _i, _p, _i, _p, _i, _p, _i, _i, _i, _i, _i, _f, _p, _sz, _p]
EXPORTED = {
    "ttt_chunk_scan": (_i, _SCAN_ARGS),
    "ttt_chunk_scan_workspace": (_sz, [_i, _i, _i, _i, _i, _i]),
    "ttt_chunk_scan_workspace_min": (_sz, [_i, _i, _i, _i, _i, _i]),
    "ttt_chunk_scan_noalloc": (_i, _SCAN_ARGS[:14] + [_p]),
    "ttt_chunk_scan_profile": (_i, _SCAN_ARGS + [_p, _p]),
    "ttt_chunk_scan_docs": (_i, _SCAN_ARGS[:14] + [_p, _p, _f] + _SCAN_ARGS[14:]),
    "ttt_chunk_scan_docs_workspace": (_sz, [_i, _i, _i, _i, _i, _i, _f]),
    "ttt_linear_minibatch": (_i, [_p, _p, _p, _i, _p, _p, _i, _p, _p,
                                  _i, _i, _i, _i, _i, _f, _p]),
    "ttt_surprisal_route": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _f, _f, _i,
                                 _p, _p, _p, _p, _p, _p, _p, _p]),
    "ttt_lm_target": (_i, [_p, _i, _p, _i, _p, _p, _i, _i, _i, _i, _i, _i, _p, _sz, _p]),
    "ttt_lm_target_workspace": (_sz, [_i, _i, _i, _i]),
    "ttt_gated_z": (_i, [_p, _i, _p, _p, _i, _i, _i, _i, _i, _p]),
    "ttt_cache_readout": (_i, [_p, _p, _p, _i, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _f,
                               _p]),
    "ttt_chunk_scan_handover_timeouts": (_i, [_i, _i, _i, _i, _i, _i, _p, _sz, _p, _p]),
    "ttt_scan_test_overrides": (_i, [_i, _i, _i]),
    "ttt_rope_frequencies": (_i, [_p, _i, _d, _i, _d, _i, _d, _d, _p]),
    "ttt_qk_norm_rope": (_i, [_p, _ll, _p, _ll, _p, _ll, _i, _p, _p, _f, _p, _p, _i, _i, _f,
                              _p, _ll, _p, _ll, _p, _p, _p, _ll, _i, _i, _i, _i, _p]),
    "ttt_attention_packed": (_i, [_p, _ll, _p, _ll, _p, _ll, _i, _p, _ll, _p, _p, _p,
                                  _i, _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p]),
    "ttt_attention_packed_workspace": (_sz, [_i, _i, _i, _i, _i, _i]),
    "ttt_attention_decode": (_i, [_p, _ll, _p, _p, _i, _p, _ll, _p, _p, _i, _i, _i, _p,
                                  _i, _i, _i, _i, _f, _i, _p, _sz, _p]),
    "ttt_attention_decode_workspace": (_sz, [_i, _i, _i, _i, _i, _i]),
    "ttt_attention_paged": (_i, [_p, _ll, _p, _p, _i, _p, _ll, _p, _p, _p, _i, _i, _i, _p,
                                 _i, _i, _i, _i, _i, _f, _i, _p, _sz, _p]),
    "ttt_attention_paged_workspace": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "ttt_add_rms_norm": (_i, [_p, _ll, _p, _ll, _i, _p, _f, _p, _ll, _p, _ll, _p, _i, _i, _i, _p]),
    "ttt_gated_delta_decode": (_i, [_p, _ll, _p, _ll, _p, _ll, _i, _p, _p, _p, _ll, _p, _p, _p, _ll,
                                    _i, _i, _i, _i, _i, _f, _i, _f, _p]),
    "ttt_gated_delta_packed": (_i, [_p, _ll, _p, _ll, _p, _ll, _i, _p, _p, _p, _ll, _p, _p, _p, _ll, _p,
                                    _i, _i, _i, _i, _i, _i, _f, _i, _f, _p, _sz, _p]),
    "ttt_gated_delta_packed_workspace": (_sz, [_i, _i, _i, _i, _i, _i]),
    "ttt_status_string": (ctypes.c_char_p, [_i]),
    "ttt_abi_version": (_i, []),
}

_lib = None


class TTTError(RuntimeError):
    """A non-OK status returned by the library."""


def lib() -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise TTTError(f"{library_path} is missing: build it with "
                           "`python -m chunked_weight_sequence_amd.build` (no fallback exists)")
        handle = ctypes.CDLL(library_path)
        for name, (res, args) in EXPORTED.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def abi_version() -> int:
    return lib().ttt_abi_version()


def status_string(code: int) -> str:
    return lib().ttt_status_string(code).decode()


def _check(code: int) -> None:
    if code != 0:
        raise TTTError(status_string(code))


# ---------------------------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    """Library dtype code of a tensor or a torch.dtype."""
    torch = _torch()
    dt = t if isinstance(t, torch.dtype) else t.dtype
    if dt is torch.bfloat16:
        return TTT_BF16
    if dt is torch.float32:
        return TTT_F32
    raise TypeError(f"unsupported dtype {dt}: use float32 or bfloat16")


def _dev(t, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    torch = _torch()
    return torch.cuda.current_stream(t.device).cuda_stream


def _as3(t):
    return t if t.dim() == 3 else t.unsqueeze(0)


def chunk_scan_workspace_bytes(B, T, d_ff, d_model, chunk, dtype, minimum: bool = False) -> int:
    """Workspace bytes of chunk_scan for one pass, or (minimum=True) the least it accepts (bf16:
    segments of one group of chunks plus an fp32 state)."""
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    f = lib().ttt_chunk_scan_workspace_min if minimum else lib().ttt_chunk_scan_workspace
    return f(B, T, d_ff, d_model, chunk, code)


def _need(t, name: str, shape, dtype, device):
    """Checks that an output tensor passed in by the caller has exactly the shape, dtype and
    device the kernels will write (the C ABI sees only its pointer)."""
    _dev(t, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _scan_prepare(Z, Vhat, W0, chunk, eta, out_dtype, O, W_final, workspace, final_state):
    torch = _torch()
    Z3, V3 = _dev(_as3(Z), "Z"), _dev(_as3(Vhat), "Vhat")
    B, T, F = Z3.shape
    D = V3.shape[2]
    dev = Z3.device
    if V3.shape[:2] != (B, T):
        raise ValueError("Z and Vhat must agree on [B, T]")
    if V3.dtype != Z3.dtype:
        raise TypeError(f"Vhat must have Z's dtype {Z3.dtype}, got {V3.dtype}")
    if V3.device != dev:
        raise ValueError("Z and Vhat must be on one device")
    _dev(W0, "W0")
    if W0.dtype != torch.float32:
        raise TypeError("W0 must be float32")
    if W0.device != dev:
        raise ValueError("W0 must be on Z's device")
    if tuple(W0.shape) == (D, F):
        shared = 1
    elif tuple(W0.shape) == (B, D, F):
        shared = 0
    else:
        raise ValueError(f"W0 must be [d_model, d_ff] = [{D}, {F}] or [B, d_model, d_ff] = "
                         f"[{B}, {D}, {F}], got {tuple(W0.shape)}")
    out_dtype = out_dtype or Z3.dtype
    if O is None:
        O = torch.empty((B, T, D), dtype=out_dtype, device=dev)
    else:
        O = _as3(O)
        _need(O, "O", (B, T, D), None, dev)
        _dtype_code(O)
    if W_final is None and final_state:
        W_final = torch.empty((B, D, F), dtype=torch.float32, device=dev)
    if W_final is not None:
        # [B, d_model, d_ff], or [d_model, d_ff] for a single sequence (e.g. W0 itself)
        want = (D, F) if (W_final.dim() == 2 and B == 1) else (B, D, F)
        _need(W_final, "W_final", want, torch.float32, dev)
    code = _dtype_code(Z3)
    need = lib().ttt_chunk_scan_workspace(B, T, F, D, chunk, code)
    if workspace is False:       # the caller sizes its own workspace
        workspace = None
    elif workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _dev(workspace, "workspace")
        if workspace.device != dev:
            raise ValueError("workspace must be on Z's device")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [_ptr(Z3), _ptr(V3), code, _ptr(W0), shared, _ptr(O), _dtype_code(O),
            _ptr(W_final), B, T, F, D, chunk, float(eta), _ptr(workspace),
            ws_bytes, _stream(Z3)]
    return args, O, W_final


def chunk_scan(Z, Vhat, W0, chunk: int, eta: float, *, out_dtype=None, O=None, W_final=None,
               workspace=None, final_state: bool = True):
    """In-Place TTT scan. Z [B,T,d_ff] or [T,d_ff], Vhat [B,T,d_model] (same dtype), W0
    [d_model,d_ff] fp32 (shared) or [B,d_model,d_ff]. Returns (O [B,T,d_model], W_final
    [B,d_model,d_ff] or None)."""
    args, O, W_final = _scan_prepare(Z, Vhat, W0, chunk, eta, out_dtype, O, W_final, workspace,
                                     final_state)
    _check(lib().ttt_chunk_scan(*args))
    return O, W_final


def chunk_scan_noalloc(Z, Vhat, W0, chunk: int, eta: float, *, O, W_final=None):
    """ttt_chunk_scan_noalloc: the scan with its workspace taken from the library's static device
    scratch (no allocation by the library; O and W_final are the caller's). Returns (O, W_final)."""
    args, O, W_final = _scan_prepare(Z, Vhat, W0, chunk, eta, None, O, W_final, False, False)
    _check(lib().ttt_chunk_scan_noalloc(*(args[:14] + [args[16]])))
    return O, W_final


def chunk_scan_docs(Z, Vhat, W0, chunk: int, eta: float, *, doc_starts=None, clip_tau=0.0,
                    out_dtype=None, O=None, W_final=None, workspace=None,
                    final_state: bool = True):
    """chunk_scan with document-boundary resets and per-chunk update clipping. doc_starts: None
    or one list per sequence of chunk-aligned token offsets in (0, T) where a new document
    begins; clip_tau: absolute Frobenius threshold per chunk delta (<= 0: off). Returns
    (O, W_final)."""
    args, O, W_final = _scan_prepare(Z, Vhat, W0, chunk, eta, out_dtype, O, W_final, False,
                                     final_state)
    B, T, F, D, code = args[8], args[9], args[10], args[11], args[2]
    torch = _torch()
    need = lib().ttt_chunk_scan_docs_workspace(B, T, F, D, chunk, code, float(clip_tau))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=O.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    counts = starts = None
    if doc_starts is not None:
        if len(doc_starts) != B:
            raise ValueError("doc_starts needs one list per sequence")
        flat = [int(x) for d in doc_starts for x in d]
        counts = (ctypes.c_int * B)(*[len(d) for d in doc_starts])
        starts = (ctypes.c_int * max(1, len(flat)))(*flat)
    args = args[:14] + [None if starts is None else ctypes.addressof(starts),
                        None if counts is None else ctypes.addressof(counts), float(clip_tau),
                        _ptr(workspace), ws_bytes, args[16]]
    _check(lib().ttt_chunk_scan_docs(*args))
    return O, W_final


def chunk_scan_handover_timeouts(workspace, B, T, d_ff, d_model, chunk, dtype):
    """How many state-chain hand-over waits ran out (and were recomputed) in the last scan call
    that used `workspace` with these sizes: a device int32 tensor of one element, written on the
    current stream (no synchronisation)."""
    torch = _torch()
    _dev(workspace, "workspace")
    count = torch.empty(4, dtype=torch.int32, device=workspace.device)
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    _check(lib().ttt_chunk_scan_handover_timeouts(
        B, T, d_ff, d_model, chunk, code, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(count), _stream(workspace)))
    return count[:1]


def scan_test_overrides(group_tokens: int = 0, token_split: int = -1, spin_limit: int = -1):
    """FOR TESTS ONLY: process-wide schedule overrides of the bf16 scan (see the header);
    scan_test_overrides() restores the defaults."""
    _check(lib().ttt_scan_test_overrides(int(group_tokens), int(token_split), int(spin_limit)))


def chunk_scan_profile(Z, Vhat, W0, chunk: int, eta: float, *, out_dtype=None, O=None,
                       W_final=None, workspace=None, final_state: bool = True):
    """chunk_scan with per-phase HIP-event timing; synchronises. Returns (O, W_final, {phase:
    (ms, launches)})."""
    args, O, W_final = _scan_prepare(Z, Vhat, W0, chunk, eta, out_dtype, O, W_final, workspace,
                                     final_state)
    ms = (ctypes.c_float * 4)()
    n = (ctypes.c_int * 4)()
    _check(lib().ttt_chunk_scan_profile(*args, ctypes.addressof(ms), ctypes.addressof(n)))
    return O, W_final, {p: (ms[i], n[i]) for i, p in enumerate(SCAN_PHASES)}


def linear_minibatch(Q, K, V, minibatch: int, eta: float, *, W0=None, out_dtype=None,
                     with_loss: bool = True, final_state: bool = True, O=None, W_final=None,
                     loss=None):
    """TTT-Linear mini-batch GD. Q, K, V [B,T,H,dh]; W0 [B,H,dh,dh] fp32 or None (zeros).
    Returns (O [B,T,H,dh], W_final [B,H,dh,dh] or None, loss [B,T,H] or None)."""
    torch = _torch()
    for t, n in ((Q, "Q"), (K, "K"), (V, "V")):
        _dev(t, n)
    if not (Q.shape == K.shape == V.shape) or Q.dim() != 4:
        raise ValueError("Q, K, V must share one [B, T, H, dh] shape")
    if not (Q.dtype == K.dtype == V.dtype):
        raise TypeError("Q, K, V must share one dtype")
    B, T, H, dh = Q.shape
    dev = Q.device
    if W0 is not None:
        _dev(W0, "W0")
        if W0.dtype != torch.float32 or tuple(W0.shape) != (B, H, dh, dh):
            raise ValueError("W0 must be float32 [B, H, dh, dh]")
    for t, n in ((K, "K"), (V, "V")):
        if t.device != dev:
            raise ValueError(f"{n} must be on Q's device")
    if W0 is not None and W0.device != dev:
        raise ValueError("W0 must be on Q's device")
    if O is None:
        O = torch.empty((B, T, H, dh), dtype=out_dtype or Q.dtype, device=dev)
    else:
        _need(O, "O", (B, T, H, dh), out_dtype, dev)
        _dtype_code(O)
    if W_final is None and final_state:
        W_final = torch.empty((B, H, dh, dh), dtype=torch.float32, device=dev)
    elif W_final is not None:
        _need(W_final, "W_final", (B, H, dh, dh), torch.float32, dev)
    if loss is None and with_loss:
        loss = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    elif loss is not None:
        _need(loss, "loss", (B, T, H), torch.float32, dev)
    _check(lib().ttt_linear_minibatch(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(Q), _ptr(W0),
                                      _ptr(O), _dtype_code(O), _ptr(W_final), _ptr(loss),
                                      B, T, H, dh, minibatch, float(eta), _stream(Q)))
    return O, W_final, loss


def surprisal_route(loss, K, V, chunk: int, *, pct: float = 0.95, ema: float = 0.9,
                    ratio: float = 0.8, capacity: int = 256, want_kv: bool = True,
                    want_mask: bool = True, out: dict | None = None):
    """SR-TTT routing. loss [B,T,H] fp32; K, V [B,T,H,dh] or [B,T,H*dh]. Returns a dict with
    tau [B,T/chunk], mask [B,T] uint8, idx [B,cap] int32, k/v [B,cap,H*dh], count [B],
    total [B]. `out` may pass that dict back in to reuse its tensors (same shapes)."""
    torch = _torch()
    _dev(loss, "loss")
    if loss.dtype != torch.float32 or loss.dim() != 3:
        raise ValueError("loss must be float32 [B, T, H]")
    B, T, H = loss.shape
    _dev(K, "K")
    _dev(V, "V")
    dev = loss.device
    if K.dim() < 3 or tuple(K.shape[:2]) != (B, T) or K.shape != V.shape or K.dtype != V.dtype:
        raise ValueError("K and V must share one [B, T, H, dh] or [B, T, H*dh] shape and dtype, "
                         "with loss's B and T")
    if K.device != dev or V.device != dev:
        raise ValueError("K and V must be on loss's device")
    row = K[0, 0].numel()
    if row % H:
        raise ValueError("K rows must hold H * dh elements")
    dh = row // H
    if out is not None:
        torch_i32, torch_f32 = torch.int32, torch.float32
        want = {"tau": ((B, T // chunk), torch_f32), "idx": ((B, capacity), torch_i32),
                "count": ((B,), torch_i32), "total": ((B,), torch_i32)}
        for name, (shape, dt) in want.items():
            _need(out[name], f"out[{name!r}]", shape, dt, dev)
        for name in ("k", "v"):
            if out.get(name) is not None:
                _need(out[name], f"out[{name!r}]", (B, capacity, row), K.dtype, dev)
        if out.get("mask") is not None:
            _need(out["mask"], "out['mask']", (B, T), torch.uint8, dev)
    else:
        out = {
        "tau": torch.empty((B, T // chunk), dtype=torch.float32, device=dev),
        "mask": torch.empty((B, T), dtype=torch.uint8, device=dev) if want_mask else None,
        "idx": torch.empty((B, capacity), dtype=torch.int32, device=dev),
        "k": torch.empty((B, capacity, row), dtype=K.dtype, device=dev) if want_kv else None,
        "v": torch.empty((B, capacity, row), dtype=V.dtype, device=dev) if want_kv else None,
        "count": torch.empty(B, dtype=torch.int32, device=dev),
        "total": torch.empty(B, dtype=torch.int32, device=dev),
        }
    _check(lib().ttt_surprisal_route(
        _ptr(loss), _ptr(K), _ptr(V), _dtype_code(K), B, T, H, dh, chunk, float(pct),
        float(ema), float(ratio), capacity, _ptr(out["tau"]), _ptr(out["mask"]),
        _ptr(out["idx"]), _ptr(out["k"]), _ptr(out["v"]), _ptr(out["count"]),
        _ptr(out["total"]), _stream(loss)))
    return out


def lm_target(X0, conv_w, W_target, chunk: int, *, out_dtype=None, V_hat=None, workspace=None):
    """LM-aligned target V_hat = Conv1D(X0) W_target with chunk-end padding. X0 [B,T,d_in] or
    [T,d_in] bf16; conv_w [width, d_in] fp32 (offsets +1 .. +width); W_target [d_in, d_out]
    bf16. Returns V_hat [B,T,d_out] (bf16 unless out_dtype / V_hat say otherwise)."""
    torch = _torch()
    X0 = _as3(_dev(X0, "X0"))
    _dev(conv_w, "conv_w")
    _dev(W_target, "W_target")
    if conv_w.dtype != torch.float32 or conv_w.dim() != 2:
        raise ValueError("conv_w must be float32 [width, d_in]")
    if W_target.dim() != 2:
        raise ValueError("W_target must be [d_in, d_out]")
    B, T, d_in = X0.shape
    width = conv_w.shape[0]
    d_out = W_target.shape[1]
    if conv_w.shape[1] != d_in or W_target.shape[0] != d_in:
        raise ValueError("conv_w and W_target must match X0's d_in")
    if _dtype_code(W_target) != TTT_BF16:
        raise ValueError("W_target must be bfloat16")
    if V_hat is None:
        od = out_dtype or torch.bfloat16
        V_hat = torch.empty((B, T, d_out), dtype=od, device=X0.device)
    need = lib().ttt_lm_target_workspace(B, T, d_in, d_out)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=X0.device)
    _check(lib().ttt_lm_target(
        _ptr(X0), _dtype_code(X0), _ptr(conv_w), width, _ptr(W_target), _ptr(_dev(V_hat, "V_hat")),
        _dtype_code(V_hat), B, T, d_in, d_out, chunk, _ptr(workspace), workspace.numel(),
        _stream(X0)))
    return V_hat


def gated_z(X, W_gu, *, out_dtype=None, Z=None):
    """Gated-MLP activation Z = SiLU(X W_gate) * (X W_up). X [B,T,d_model] or [T,d_model] bf16;
    W_gu [2 d_ff, d_model] bf16 in linear-layer storage: rows 0 .. d_ff-1 are W_gate^T, rows
    d_ff .. 2 d_ff-1 are W_up^T. Returns Z [B,T,d_ff] (bf16 unless out_dtype / Z say otherwise)."""
    torch = _torch()
    X = _as3(_dev(X, "X"))
    _dev(W_gu, "W_gu")
    if W_gu.dim() != 2 or W_gu.shape[0] % 2:
        raise ValueError("W_gu must be [2 d_ff, d_model]")
    if _dtype_code(W_gu) != TTT_BF16:
        raise ValueError("W_gu must be bfloat16")
    B, T, d_model = X.shape
    d_ff = W_gu.shape[0] // 2
    if W_gu.shape[1] != d_model:
        raise ValueError("W_gu rows must have X's d_model entries")
    if Z is None:
        Z = torch.empty((B, T, d_ff), dtype=out_dtype or torch.bfloat16, device=X.device)
    _check(lib().ttt_gated_z(_ptr(X), _dtype_code(X), _ptr(W_gu), _ptr(_dev(Z, "Z")),
                             _dtype_code(Z), B, T, d_model, d_ff, _stream(X)))
    return Z


def cache_readout(Q, K, V, routed_mask, ttt_out, alpha, H: int, chunk: int, capacity: int,
                  scale=None, *, out=None):
    """SR residual-cache readout: out = ttt_out + clamp(alpha, 0, 1) * softmax attention of Q
    over the cache each token's routing chunk starts with. Q, K, V [B,T,H*dh] bf16;
    routed_mask [B,T] uint8; ttt_out [B,T,H*dh] bf16 or fp32; alpha [H*dh] fp32. `out` may be
    ttt_out (in place). Returns out."""
    torch = _torch()
    Q, K, V, ttt_out = (_as3(_dev(t, n)) for t, n in
                        ((Q, "Q"), (K, "K"), (V, "V"), (ttt_out, "ttt_out")))
    _dev(routed_mask, "routed_mask")
    _dev(alpha, "alpha")
    B, T, HD = Q.shape
    if HD % H:
        raise ValueError("Q's last dimension must be H * dh")
    dh = HD // H
    for t, n in ((K, "K"), (V, "V"), (ttt_out, "ttt_out")):
        if tuple(t.shape) != (B, T, HD):
            raise ValueError(f"{n} must have Q's shape")
    if routed_mask.dtype != torch.uint8 or routed_mask.numel() != B * T:
        raise ValueError("routed_mask must be uint8 [B, T]")
    if alpha.dtype != torch.float32 or alpha.numel() != HD:
        raise ValueError("alpha must be float32 [H * dh]")
    if out is None:
        out = torch.empty_like(ttt_out)
    if scale is None:
        scale = 1.0 / dh ** 0.5
    _check(lib().ttt_cache_readout(
        _ptr(Q), _ptr(K), _ptr(V), _dtype_code(Q), _ptr(routed_mask), _ptr(ttt_out),
        _ptr(_dev(out, "out")), _dtype_code(out), _ptr(alpha), B, T, H, dh, chunk, capacity,
        float(scale), _stream(Q)))
    return out


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str | None = None,
                     factor: float = 1.0, original_length: int = 0, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device=None):
    """Frequencies of a rotation of `rot` channels for qk_norm_rope: (inv_freq [rot / 2] float64 on
    `device` (default: the current GPU), rope_scale). scaling: None, "linear", "ntk" or "yarn"
    (which needs original_length, the context the model was trained with)."""
    torch = _torch()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)}, got {scaling!r}")
    rot = _int_in(rot, "rot", 2, 256)
    original_length = _int_in(original_length, "original_length", 0, (1 << 31) - 1)
    out = (ctypes.c_double * (rot // 2))()
    scale = ctypes.c_float(1.0)
    _check(lib().ttt_rope_frequencies(ctypes.addressof(out), rot, float(base),
                                      ROPE_SCALINGS[scaling], float(factor), original_length,
                                      float(beta_fast), float(beta_slow),
                                      ctypes.addressof(scale)))
    return (torch.tensor(list(out), dtype=torch.float64, device=device or "cuda"), scale.value)


def _rows(t, name: str, heads=None, dh=None, dtype=None, device=None, n=None):
    """Checks a [tokens, heads, dh] GPU tensor whose tokens may lie apart (a slice of one buffer);
    returns its token stride in elements."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dh], got {tuple(shape)}")
    N, H, D = shape
    if device is None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if N >= 1 << 31:
            raise ValueError(f"{name} has too many tokens: {N}")
    else:
        if (n is not None and N != n) or (heads is not None and H != heads) or D != dh:
            raise ValueError(f"{name} must be [{n}, {heads}, {dh}], got {tuple(shape)}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")
    if (stride[2] != 1 and D > 1) or (stride[1] != D and H > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return stride[0] if N > 1 else H * D


def _vec(t, name: str, shape, dtype, device):
    """Checks a dense tensor of exactly this shape, dtype and device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on {device}, got "
                         f"{tuple(t.shape)} on {t.device}")


def _int_in(value, name: str, lo: int, hi: int) -> int:
    """An argument that the C ABI takes as an int: refused where ctypes would cut it."""
    value = operator.index(value)
    if not lo <= value <= hi:
        raise ValueError(f"{name} must lie in [{lo}, {hi}], got {value}")
    return value


@functools.lru_cache(maxsize=1)
def _device_calls(internals=None):
    """(the current device's index, a device's current stream as a handle). torch's own functions where it
    has them, since torch.cuda.current_stream() builds an object, 4 us of a 16 us call; they are not part
    of its interface, so the public ones otherwise."""
    torch = _torch()
    internals = torch._C if internals is None else internals
    return (getattr(internals, "_cuda_getDevice", None) or torch.cuda.current_device,
            getattr(internals, "_cuda_getCurrentRawStream", None) or
            (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _launch(fn, args, device):
    """Calls fn(*args, stream) with `device` current and its current stream; checks the status."""
    current, stream = _device_calls()
    index = device.index
    if current() == index:
        code = fn(*args, stream(index))
    else:
        with _torch().cuda.device(device):
            code = fn(*args, stream(index))
    if code != 0:
        raise TTTError(status_string(code))


def qk_norm_rope(Q, K, pos, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                 layout: str = "half", rope_scale: float = 1.0, V=None, K_cache=None,
                 V_cache=None, slots=None, Q_out=None, K_out=None):
    """Per-head RMS norm (where a weight is given) and rotation of Q [N,Hq,dh] and K [N,Hkv,dh]
    (bf16 or fp32; tokens may be slices of one buffer) at positions pos [N] int32. inv_freq
    [rot / 2] float64 and rope_scale as from rope_frequencies; layout "half" or "interleaved".
    With slots [N] int32, token t's rotated K row and its V row are also written to row slots[t] of
    K_cache and V_cache [n_slots,Hkv,dh] (slots outside are skipped; the others must be distinct).
    Q_out / K_out may be Q / K (in place). Returns (Q_out, K_out)."""
    torch = _torch()
    qs = _rows(Q, "Q")
    N, Hq, dh = Q.shape
    dt, dev = Q.dtype, Q.device
    code = _dtype_code(dt)
    ks = _rows(K, "K", None, dh, dt, dev, N)
    Hkv = K.shape[1]
    _vec(pos, "pos", (N,), torch.int32, dev)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    half = inv_freq.shape[0]
    _vec(inv_freq, "inv_freq", (half,), torch.float64, dev)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _vec(w, name, (dh,), torch.float32, dev)
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {list(ROPE_LAYOUTS)}, got {layout!r}")
    vs = n_slots = 0
    if slots is not None:
        if V is None or K_cache is None or V_cache is None:
            raise ValueError("slots needs V, K_cache and V_cache")
        _vec(slots, "slots", (N,), torch.int32, dev)
        vs = _rows(V, "V", Hkv, dh, dt, dev, N)
        if K_cache.dim() != 3:
            raise ValueError(f"K_cache must be [n_slots, Hkv, dh], got {tuple(K_cache.shape)}")
        n_slots = K_cache.shape[0]
        _vec(K_cache, "K_cache", (n_slots, Hkv, dh), dt, dev)
        _vec(V_cache, "V_cache", (n_slots, Hkv, dh), dt, dev)
    elif V is not None or K_cache is not None or V_cache is not None:
        raise ValueError("V, K_cache and V_cache are for a call with slots")
    if Q_out is None:
        Q_out, qos = torch.empty_like(Q), Hq * dh  # contiguous, also of a slice
    else:
        qos = _rows(Q_out, "Q_out", Hq, dh, dt, dev, N)
    if K_out is None:
        K_out, kos = torch.empty_like(K), Hkv * dh
    else:
        kos = _rows(K_out, "K_out", Hkv, dh, dt, dev, N)
    _launch(lib().ttt_qk_norm_rope,
            (Q.data_ptr(), qs, K.data_ptr(), ks, _ptr(V), vs, code, _ptr(q_weight),
             _ptr(k_weight), eps, pos.data_ptr(), inv_freq.data_ptr() if half else None, 2 * half,
             ROPE_LAYOUTS[layout], rope_scale, Q_out.data_ptr(), qos, K_out.data_ptr(), kos,
             _ptr(K_cache), _ptr(V_cache), _ptr(slots), n_slots, N, Hq, Hkv, dh), dev)
    return Q_out, K_out


def attention_packed(Q, K, V, cu_q, cu_k=None, *, scale=None, window: int = 0, O=None,
                     with_lse: bool = False, lse=None, workspace=None):
    """Causal attention over packed sequences. Q [Nq,Hq,dh], K and V [Nk,Hkv,dh] bf16 (tokens may
    be slices of one buffer), dh 64 or 128, Hq a multiple of Hkv; cu_q, cu_k [n_seq + 1] int32
    offsets on the GPU (cu_k None: the same as cu_q). A sequence's last query stands at its last
    key; window > 0 limits every query to the last `window` keys up to its own. scale: 1 / sqrt(dh)
    by default. Returns O [Nq,Hq,dh], with (with_lse, or lse given) lse [Nq,Hq] fp32 beside it."""
    torch = _torch()
    qs = _rows(Q, "Q")
    Nq, Hq, dh = Q.shape
    dt, dev = Q.dtype, Q.device
    ks = _rows(K, "K", None, dh, dt, dev)
    Nk, Hkv, _ = K.shape
    if Nk >= 1 << 31:
        raise ValueError(f"K has too many tokens: {Nk}")
    vs = _rows(V, "V", Hkv, dh, dt, dev, Nk)
    if cu_q.dim() != 1:
        raise ValueError(f"cu_q must be [n_seq + 1], got {tuple(cu_q.shape)}")
    n_seq = cu_q.shape[0] - 1
    _vec(cu_q, "cu_q", (n_seq + 1,), torch.int32, dev)
    if cu_k is None:
        cu_k = cu_q
    else:
        _vec(cu_k, "cu_k", (n_seq + 1,), torch.int32, dev)
    if O is None:
        O, os_ = torch.empty_like(Q), Hq * dh
    else:
        os_ = _rows(O, "O", Hq, dh, dt, dev, Nq)
    window = _int_in(window, "window", 0, 1 << 30)
    if lse is not None:
        _vec(lse, "lse", (Nq, Hq), torch.float32, dev)
    elif with_lse:
        lse = torch.empty(Nq, Hq, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(workspace, _workspace_bytes(
        "ttt_attention_packed_workspace", n_seq, Nq, Nk, Hq, Hkv, dh), dev)
    _launch(lib().ttt_attention_packed,
            (Q.data_ptr(), qs, K.data_ptr(), ks, V.data_ptr(), vs, _dtype_code(dt), O.data_ptr(),
             os_, _ptr(lse), cu_q.data_ptr(), cu_k.data_ptr(), n_seq, Nq, Nk, Hq, Hkv, dh,
             dh ** -0.5 if scale is None else scale, window, _ptr(ws), ws_bytes), dev)
    return O if lse is None else (O, lse)


def attention_decode(Q, K_cache, V_cache, page_table, lengths, page_size: int, *, scale=None,
                     window: int = 0, O=None, with_lse: bool = False, lse=None, workspace=None):
    """One-token attention over a paged cache. Q [S,Hq,dh] bf16; K_cache, V_cache
    [n_slots,Hkv,dh] (rows of page p: p * page_size ..; rows behind the last whole page are not read, and
    tokens of a page that is not there are left out); page_table [S,max_pages] int32;
    lengths [S] int32: cached tokens of each sequence, its query's own among them. Returns
    O [S,Hq,dh], with (with_lse, or lse given) lse [S,Hq] fp32 beside it."""
    torch = _torch()
    qs = _rows(Q, "Q")
    S, Hq, dh = Q.shape
    dt, dev = Q.dtype, Q.device
    if K_cache.dim() != 3:
        raise ValueError(f"K_cache must be [n_slots, Hkv, dh], got {tuple(K_cache.shape)}")
    n_slots, Hkv = K_cache.shape[0], K_cache.shape[1]
    _vec(K_cache, "K_cache", (n_slots, Hkv, dh), dt, dev)
    _vec(V_cache, "V_cache", (n_slots, Hkv, dh), dt, dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seq, max_pages]")
    max_pages = page_table.shape[1]
    _vec(page_table, "page_table", (S, max_pages), torch.int32, dev)
    _vec(lengths, "lengths", (S,), torch.int32, dev)
    page_size = _int_in(page_size, "page_size", 1, 65536)
    window = _int_in(window, "window", 0, 1 << 30)
    if O is None:
        O, os_ = torch.empty_like(Q), Hq * dh
    else:
        os_ = _rows(O, "O", Hq, dh, dt, dev, S)
    if lse is not None:
        _vec(lse, "lse", (S, Hq), torch.float32, dev)
    elif with_lse:
        lse = torch.empty(S, Hq, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(workspace, _workspace_bytes(
        "ttt_attention_decode_workspace", S, max_pages, page_size, Hq, Hkv, dh), dev)
    _launch(lib().ttt_attention_decode,
            (Q.data_ptr(), qs, K_cache.data_ptr(), V_cache.data_ptr(), _dtype_code(dt),
             O.data_ptr(), os_, _ptr(lse), page_table.data_ptr(), max_pages, page_size,
             n_slots // page_size, lengths.data_ptr(), S, Hq, Hkv, dh,
             dh ** -0.5 if scale is None else scale, window, _ptr(ws), ws_bytes), dev)
    return O if lse is None else (O, lse)


def attention_paged(Q, K_cache, V_cache, cu_q, page_table, lengths, page_size: int, *, scale=None,
                    window: int = 0, O=None, with_lse: bool = False, lse=None, workspace=None):
    """Attention of new tokens over a paged cache that holds them already. Q [Nq,Hq,dh] bf16, the tokens of
    sequence s from cu_q[s] to cu_q[s+1] (cu_q [n_seq + 1] int32 on the GPU; any numbers of them, 0 and 1
    too); lengths [n_seq] int32: the cached tokens of each sequence, of which the last is its last query's
    own. The caches, page_table [n_seq,max_pages] and page_size as in attention_decode; what a query sees,
    window and the results as in attention_packed."""
    torch = _torch()
    qs = _rows(Q, "Q")
    Nq, Hq, dh = Q.shape
    dt, dev = Q.dtype, Q.device
    if K_cache.dim() != 3:
        raise ValueError(f"K_cache must be [n_slots, Hkv, dh], got {tuple(K_cache.shape)}")
    n_slots, Hkv = K_cache.shape[0], K_cache.shape[1]
    _vec(K_cache, "K_cache", (n_slots, Hkv, dh), dt, dev)
    _vec(V_cache, "V_cache", (n_slots, Hkv, dh), dt, dev)
    if cu_q.dim() != 1:
        raise ValueError(f"cu_q must be [n_seq + 1], got {tuple(cu_q.shape)}")
    n_seq = cu_q.shape[0] - 1
    _vec(cu_q, "cu_q", (n_seq + 1,), torch.int32, dev)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n_seq, max_pages]")
    max_pages = page_table.shape[1]
    _vec(page_table, "page_table", (n_seq, max_pages), torch.int32, dev)
    _vec(lengths, "lengths", (n_seq,), torch.int32, dev)
    page_size = _int_in(page_size, "page_size", 1, 65536)
    window = _int_in(window, "window", 0, 1 << 30)
    if O is None:
        O, os_ = torch.empty_like(Q), Hq * dh
    else:
        os_ = _rows(O, "O", Hq, dh, dt, dev, Nq)
    if lse is not None:
        _vec(lse, "lse", (Nq, Hq), torch.float32, dev)
    elif with_lse:
        lse = torch.empty(Nq, Hq, dtype=torch.float32, device=dev)
    ws, ws_bytes = _workspace(workspace, _workspace_bytes(
        "ttt_attention_paged_workspace", n_seq, Nq, max_pages, page_size, Hq, Hkv, dh), dev)
    _launch(lib().ttt_attention_paged,
            (Q.data_ptr(), qs, K_cache.data_ptr(), V_cache.data_ptr(), _dtype_code(dt), O.data_ptr(), os_,
             _ptr(lse), cu_q.data_ptr(), page_table.data_ptr(), max_pages, page_size, n_slots // page_size,
             lengths.data_ptr(), n_seq, Nq, Hq, Hkv, dh, dh ** -0.5 if scale is None else scale, window,
             _ptr(ws), ws_bytes), dev)
    return O if lse is None else (O, lse)


def _row_stride(t, name: str, N, D):
    """The row stride in elements of an [N, D] tensor whose rows are contiguous."""
    stride = t.stride()
    if stride[1] != 1 and D > 1:
        raise ValueError(f"{name}: a row must be contiguous")
    return stride[0] if N > 1 else D


def _matrix(t, name: str, N, D, dtype, device):
    """Checks a [N, D] GPU tensor whose rows may lie apart; returns its row stride in elements."""
    if t.shape != (N, D):
        raise ValueError(f"{name} must be [{N}, {D}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return _row_stride(t, name, N, D)


def add_rms_norm(X, weight=None, *, residual=None, eps: float = 1e-6, e4m3: bool = False, group: int = 0,
                 S=None, Y=None, scales=None):
    """RMS norm of X [N,D] (bf16 or fp32; rows may be slices of one buffer), or of X + residual, times weight
    [D] fp32. Returns (Y, scales, S): Y [N,D] in X's dtype and scales None, or (e4m3) Y in
    torch.float8_e4m3fn with the fp32 scales it was divided by, one a row ([N]) or one for each `group`
    channels ([N, D / group]); S [N,D] the sum X + residual, None without a residual. S may be X or
    residual (in place)."""
    torch = _torch()
    if X.dim() != 2 or not X.is_cuda:
        raise ValueError("X must be a [N, D] GPU tensor")
    N, D = X.shape
    dt, dev = X.dtype, X.device
    code = _dtype_code(dt)
    if N >= 1 << 31 or D >= 1 << 31:
        raise ValueError(f"X is too large: {(N, D)}")
    xs = _row_stride(X, "X", N, D)
    rs = ss = 0
    if residual is not None:
        rs = _matrix(residual, "residual", N, D, dt, dev)
        if S is None:
            S, ss = torch.empty_like(X), D  # contiguous, also of a slice
        else:
            ss = _matrix(S, "S", N, D, dt, dev)
    elif S is not None:
        raise ValueError("S is for a call with a residual")
    if weight is not None:
        _vec(weight, "weight", (D,), torch.float32, dev)
    group = _int_in(group, "group", 0, 1 << 30)
    out = torch.float8_e4m3fn if e4m3 else dt
    if Y is None:
        Y, ys = torch.empty_like(X, dtype=out), D
    else:
        ys = _matrix(Y, "Y", N, D, out, dev)
    if e4m3:
        if group and D % group:
            raise ValueError(f"group must divide D = {D}, got {group}")
        shape = (N, D // group) if group else (N,)
        if scales is None:
            scales = torch.empty(shape, dtype=torch.float32, device=dev)
        else:
            _vec(scales, "scales", shape, torch.float32, dev)
    elif scales is not None or group:
        raise ValueError("scales and group are for an output in e4m3")
    _launch(lib().ttt_add_rms_norm,
            (X.data_ptr(), xs, _ptr(residual), rs, code, _ptr(weight), eps, _ptr(S), ss, Y.data_ptr(), ys,
             _ptr(scales), group, N, D), dev)
    return Y, scales, S


def _delta_inputs(Q, K, V, g, beta, O):
    """Checks the tensors that both calls of the gated delta rule take; returns (O, the arguments up to it,
    tokens, Hk, Hv, dk, dv)."""
    torch = _torch()
    qs = _rows(Q, "Q")
    N, Hk, dk = Q.shape
    dt, dev = Q.dtype, Q.device
    ks = _rows(K, "K", Hk, dk, dt, dev, N)
    if V.dim() != 3:
        raise ValueError(f"V must be [tokens, heads, dv], got {tuple(V.shape)}")
    Hv, dv = V.shape[1:]
    vs = _rows(V, "V", Hv, dv, dt, dev, N)
    _vec(g, "g", (N, Hv), torch.float32, dev)
    _vec(beta, "beta", (N, Hv), torch.float32, dev)
    if O is None:
        O, os_ = torch.empty_like(V), Hv * dv  # contiguous, also of a slice
    else:
        os_ = _rows(O, "O", Hv, dv, dt, dev, N)
    return O, (Q.data_ptr(), qs, K.data_ptr(), ks, V.data_ptr(), vs, _dtype_code(dt), g.data_ptr(),
               beta.data_ptr(), O.data_ptr(), os_), N, Hk, Hv, dk, dv


def _delta_states(state, state_out, slots, n_seq, Hv, dk, dv, device):
    """Checks the pools of states; returns how many slots they have."""
    torch = _torch()
    n_slots = None
    for t, name in ((state, "state"), (state_out, "state_out")):
        if t is None:
            continue
        if t.dim() != 4:
            raise ValueError(f"{name} must be [n_slots, Hv, dk, dv], got {tuple(t.shape)}")
        n_slots = t.shape[0] if n_slots is None else n_slots
        _vec(t, name, (n_slots, Hv, dk, dv), torch.float32, device)
    if slots is not None:
        _vec(slots, "slots", (n_seq,), torch.int32, device)
    elif n_slots is not None and n_slots < n_seq:
        raise ValueError(f"{n_seq} sequences need as many states, got {n_slots}")
    return n_slots or 0


def gated_delta_packed(Q, K, V, g, beta, cu, *, state=None, state_out=None, slots=None, scale=None,
                       normalize: bool = True, norm_eps: float = 1e-6, final_state: bool = True, O=None,
                       workspace=None):
    """The gated delta rule (see gated_delta_decode) over packed sequences: Q, K [N,Hk,dk], V [N,Hv,dv] bf16,
    g and beta [N,Hv] fp32, the tokens of sequence s from cu[s] to cu[s+1] (cu [n_seq + 1] int32 on the GPU; may
    be empty). Sequences start from their slots of state [n_slots,Hv,dk,dv] fp32 (None: from zero) and leave
    their last states in state_out: in state itself if that is None, in a new [n_seq,Hv,dk,dv] if there is
    neither, nowhere with final_state=False. Returns (O [N,Hv,dv], state_out or None)."""
    torch = _torch()
    O, args, N, Hk, Hv, dk, dv = _delta_inputs(Q, K, V, g, beta, O)
    dev = Q.device
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError(f"cu must be [n_seq + 1], got {tuple(cu.shape)}")
    n_seq = cu.shape[0] - 1
    _vec(cu, "cu", (n_seq + 1,), torch.int32, dev)
    if not final_state:
        if state_out is not None:
            raise ValueError("state_out is for a call with final_state")
    elif state_out is None and state is not None:
        state_out = state
    elif state_out is None:
        if slots is not None:
            raise ValueError("slots needs state or state_out")
        state_out = torch.empty((n_seq, Hv, dk, dv), dtype=torch.float32, device=dev)
    n_slots = _delta_states(state, state_out, slots, n_seq, Hv, dk, dv, dev)
    ws, ws_bytes = _workspace(workspace, _workspace_bytes(
        "ttt_gated_delta_packed_workspace", n_seq, N, Hk, Hv, dk, dv), dev)
    _launch(lib().ttt_gated_delta_packed,
            args + (_ptr(state), _ptr(state_out), _ptr(slots), n_slots, cu.data_ptr(), n_seq, N, Hk, Hv, dk, dv,
                    dk ** -0.5 if scale is None else scale, int(bool(normalize)), norm_eps, _ptr(ws), ws_bytes),
            dev)
    return O, state_out


def gated_delta_decode(Q, K, V, g, beta, state, *, state_out=None, slots=None, scale=None,
                       normalize: bool = True, norm_eps: float = 1e-6, O=None):
    """The gated delta rule for one token of each of S sequences: per value head, with a = exp(g),
    u = beta (v - a W^T k), W <- a W + k u^T, o = scale W^T q; q and k divided by their norm first
    (normalize). Q, K [S,Hk,dk], V [S,Hv,dv] bf16 (tokens may be slices of one buffer), g and beta [S,Hv] fp32;
    state [n_slots,Hv,dk,dv] fp32 (None: all start at zero), of which sequence s has slot slots[s] (int32; slots
    None: s; outside: starts at zero, nothing kept). The new states go to the same slots of state_out, in place if
    that is None.
    scale: 1 / sqrt(dk) by default. Returns (O [S,Hv,dv], state_out)."""
    O, args, S, Hk, Hv, dk, dv = _delta_inputs(Q, K, V, g, beta, O)
    state_out = state if state_out is None else state_out
    n_slots = _delta_states(state, state_out, slots, S, Hv, dk, dv, Q.device)
    _launch(lib().ttt_gated_delta_decode,
            args + (_ptr(state), _ptr(state_out), _ptr(slots), n_slots, S, Hk, Hv, dk, dv,
                    dk ** -0.5 if scale is None else scale, int(bool(normalize)), norm_eps), Q.device)
    return O, state_out


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(query: str, *sizes) -> int:
    """A workspace query of the library, which depends on the sizes only (0.2 instead of 0.4 us)."""
    return getattr(lib(), query)(*sizes)


def _workspace(given, need: int, device):
    """The caller's workspace, or a new one of `need` bytes (None where nothing is needed)."""
    if given is not None:
        if not given.is_cuda or not given.is_contiguous() or given.device != device:
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        return given, given.numel() * given.element_size()
    if need == 0:
        return None, 0
    return _torch().empty(need, dtype=_torch().uint8, device=device), need
