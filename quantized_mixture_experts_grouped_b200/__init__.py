"""Python binding of libmoe_w4a16.so, the fused grouped W4A16 MoE FFN layer for sm_100a.

Argument marshalling only: every step of the layer runs in the library's CUDA kernels. The
functions carry the C ABI's names (include/moe_w4a16.h) and take torch tensors for device
memory and torch streams; torch provides memory, streams and nothing else. There is no CPU
fallback: importing this package without the built library raises.

Method: "Every Expert Counts: ExactMoE for Memory-Efficient W4A16 Inference", Abstract.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_w4a16.so")

MOE_OK, MOE_ERR_ARG, MOE_ERR_SHAPE, MOE_ERR_CUDA, MOE_ERR_TIMEOUT = 0, 1, 2, 3, 4
MOE_PATH_AUTO, MOE_PATH_SIMPLE, MOE_PATH_DECODE, MOE_PATH_GROUPED, MOE_PATH_SEQUENTIAL = 0, 1, 2, 3, 4
MOE_FLAG_ACCUMULATE = 0x100
MOE_DTYPE_BF16, MOE_DTYPE_F16, MOE_DTYPE_F32 = 0, 1, 2
MOE_NORM_Y, MOE_NORM_NEXT = 1, 2
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_FULL = 0, 1, 2, 3
PATHS = {"auto": MOE_PATH_AUTO, "simple": MOE_PATH_SIMPLE, "decode": MOE_PATH_DECODE,
         "grouped": MOE_PATH_GROUPED, "sequential": MOE_PATH_SEQUENTIAL}


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python quantized_mixture_experts_grouped_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    c = ctypes
    P, I, Z, L64, F = c.c_void_p, c.c_int, c.c_size_t, c.c_int64, c.c_float
    sig = {
        "moe_abi_version": ([], I),
        "moe_packed_layout_version": ([], I),
        "moe_last_error_string": ([], c.c_char_p),
        "moe_launch_count": ([], c.c_ulonglong),
        "moe_debug_set_decode_trace": ([P], None),
        "moe_debug_set_wait_limit": ([c.c_ulonglong, I], None),
        "moe_packed_bytes": ([I, I], Z),
        "moe_scales_count": ([I, I], Z),
        "moe_quantize_pack": ([P, I, I, I, P, P, P], I),
        "moe_route_topk": ([P, I, I, I, P, P, P], I),
        "moe_permute_scratch_count": ([I, I, I], Z),
        "moe_permute": ([P, I, I, I, P, P, P, P, P, P], I),
        "moe_workspace_bytes": ([I, I, I, I, I, c.POINTER(Z)], I),
        "moe_workspace_init": ([P, Z, P], I),
        "moe_workspace_status": ([P, P, c.POINTER(I)], I),
        "moe_w4a16_ffn": ([P, I, I, I, I, I, P, P, P, P, P, P, P, P, Z, P, I, P], I),
        "moe_w4a16_layer": ([P, P, I, I, I, I, I, P, P, P, P, P, P, P, P, Z, P, I, P], I),
        "moe_w4a16_layer_noalloc": ([P, P, I, I, I, I, I, P, P, P, P, P, P, P, P, I, P], I),
        "moe_noalloc_status": ([P, c.POINTER(I)], I),
        "moe_bf16_ffn": ([P, I, I, I, I, I, P, P, P, P, P, P, Z, P, I, P], I),
        "moe_bf16_layer": ([P, P, I, I, I, I, I, P, P, P, P, P, P, Z, P, I, P], I),
        "moe_dispatch": ([P, L64, I, P, I, I, I, I, P, P, P, P, P, L64, P], I),
        "moe_dispatch_backward": ([P, L64, I, P, I, I, I, P, L64, P], I),
        "moe_combine": ([P, L64, I, P, P, I, I, I, P, L64, I, P], I),
        "moe_combine_backward": ([P, L64, I, P, L64, I, P, P, I, I, I, P, L64, P, P], I),
        "moe_route_topk_backward": ([P, P, P, I, I, I, P, L64, I, P], I),
        "moe_norm_workspace_bytes": ([I, I, c.POINTER(Z)], I),
        "moe_norm_pre": ([P, L64, I, P, F, I, I, P, L64, P], I),
        "moe_norm_pre_backward": ([P, L64, P, L64, I, P, F, I, I, P, L64, P, L64, P, P, Z, P], I),
        "moe_norm_post": ([P, L64, P, L64, I, P, P, L64, I, F, F, I, I, I, P, L64, P, P, L64, P], I),
        "moe_combine_norm_post": ([P, L64, I, P, P, I, P, L64, I, P, P, L64, I, F, F, I, I, I, P, L64, P, P, L64,
                                   P, L64, P], I),
        "moe_norm_post_backward": ([P, L64, P, L64, I, P, P, L64, I, F, F, I, I, I, P, L64, P, P, L64, P, L64,
                                    P, L64, P, P, L64, P, P, Z, P], I),
        "moe_slot_cache_create": ([I, I, I, I, P, P, P, P, P, P, P, P, c.POINTER(P)], I),
        "moe_slot_cache_destroy": ([P], None),
        "moe_slot_cache_fail_copy_after": ([P, I], None),
        "moe_slot_cache_dry_run": ([P, I], None),
        "slot_table_update": ([P, P, P, P, c.POINTER(I), P, P, P], I),
        "slot_table_update_ex": ([P, P, P, P, c.POINTER(I), P, P, P, I, P], I),
        "moe_slot_cache_state": ([P, P, P], c.c_int64),
        "moe_slot_cache_layer": ([P, P, P, I, I, P, P, P, P, Z, P, I, P, P, c.POINTER(I), c.POINTER(I)], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


lib = _load()


class _NotLoaded:
    """Stands for the native binding where it does not load: every row operator's call raises, the calls
    that go through ctypes (the W4A16 and BF16 layers) work."""

    def __init__(self, why: str):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"the native binding _rows.so is missing or does not load ({self._why}); build it with "
                          "`python quantized_mixture_experts_grouped_b200/build.py`")


try:
    from . import _rows            # native argument marshalling of the row operators
    _built_for = getattr(_rows, "built_for", "an earlier one")
    if _built_for != torch.__version__.split("+")[0]:
        raise ImportError(f"built for torch {_built_for}, not {torch.__version__}")
    _rows.set_error(MoeError)
except ImportError as e:
    _rows = _NotLoaded(str(e))


def _err(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, lib.moe_last_error_string().decode())


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def moe_abi_version() -> int:
    return lib.moe_abi_version()


def moe_launch_count() -> int:
    return lib.moe_launch_count()


def moe_debug_set_wait_limit(cycles: int, extra_arrivals: int = 0):
    """Testing aid: bounded-wait limit of the single-token decode kernel (0 = default) and extra
    arrivals its exchange waits for (> 0 makes that wait run out)."""
    lib.moe_debug_set_wait_limit(cycles, extra_arrivals)


def moe_packed_bytes(N: int, K: int) -> int:
    return lib.moe_packed_bytes(N, K)


def moe_scales_count(N: int, K: int) -> int:
    return lib.moe_scales_count(N, K)


def moe_quantize_pack(w_bf16: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, stream=None):
    """w_bf16 [E][N][K] bf16 -> packed uint8 [E][N*K/2], scales bf16 [E][N*K/128]."""
    E, N, K = w_bf16.shape
    _err(lib.moe_quantize_pack(_p(w_bf16), E, N, K, _p(packed), _p(scales), _s(stream)))


def moe_route_topk(logits: torch.Tensor, k: int, idx: torch.Tensor, wts: torch.Tensor, stream=None):
    T, E = logits.shape
    _err(lib.moe_route_topk(_p(logits), T, E, k, _p(idx), _p(wts), _s(stream)))


def moe_permute_scratch_count(T: int, k: int, E: int) -> int:
    return lib.moe_permute_scratch_count(T, k, E)


def moe_permute(idx, E: int, counts, offsets, perm, inv, scratch, stream=None):
    T, k = idx.shape
    _err(lib.moe_permute(_p(idx), T, k, E, _p(counts), _p(offsets), _p(perm), _p(inv), _p(scratch), _s(stream)))


def moe_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    out = ctypes.c_size_t(0)
    _err(lib.moe_workspace_bytes(T, H, I, E, k, ctypes.byref(out)))
    return out.value


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _err(lib.moe_workspace_init(_p(ws), ws.numel() * ws.element_size(), _s(stream)))


def moe_workspace_status(ws: torch.Tensor, stream=None) -> int:
    st = ctypes.c_int(0)
    _err(lib.moe_workspace_status(_p(ws), _s(stream), ctypes.byref(st)))
    return st.value


def moe_w4a16_ffn(x, idx, wts, w13, s13, w2, s2, H: int, I: int, E: int, ws, out, slot_of_expert=None,
                  flags: int = MOE_PATH_AUTO, stream=None):
    T, k = idx.shape
    _err(lib.moe_w4a16_ffn(_p(x), T, H, I, E, k, _p(idx), _p(wts), _p(w13), _p(s13), _p(w2), _p(s2),
                           _p(slot_of_expert), _p(ws), ws.numel() * ws.element_size(), _p(out), flags, _s(stream)))


def moe_w4a16_layer(x, logits, k: int, w13, s13, w2, s2, H: int, I: int, idx, wts, ws, out,
                    slot_of_expert=None, flags: int = MOE_PATH_AUTO, stream=None):
    T, E = logits.shape
    _err(lib.moe_w4a16_layer(_p(x), _p(logits), T, H, I, E, k, _p(w13), _p(s13), _p(w2), _p(s2),
                             _p(slot_of_expert), _p(idx), _p(wts), _p(ws), ws.numel() * ws.element_size(),
                             _p(out), flags, _s(stream)))


def moe_w4a16_layer_noalloc(x, logits, k: int, w13, s13, w2, s2, H: int, I: int, idx, wts, out,
                            slot_of_expert=None, flags: int = MOE_PATH_AUTO, stream=None):
    """moe_w4a16_layer with the library's static device scratch as its workspace (no allocation)."""
    T, E = logits.shape
    _err(lib.moe_w4a16_layer_noalloc(_p(x), _p(logits), T, H, I, E, k, _p(w13), _p(s13), _p(w2), _p(s2),
                                     _p(slot_of_expert), _p(idx), _p(wts), _p(out), flags, _s(stream)))


def moe_bf16_ffn(x, idx, wts, w13, w2, H: int, I: int, E: int, ws, out, slot_of_expert=None,
                 flags: int = MOE_PATH_AUTO, stream=None):
    """The layer's FFN on unquantised bf16 experts: w13 [slots][2I][H], w2 [slots][H][I] (bf16)."""
    T, k = idx.shape
    _err(lib.moe_bf16_ffn(_p(x), T, H, I, E, k, _p(idx), _p(wts), _p(w13), _p(w2), _p(slot_of_expert),
                          _p(ws), ws.numel() * ws.element_size(), _p(out), flags, _s(stream)))


def moe_bf16_layer(x, logits, k: int, w13, w2, H: int, I: int, idx, wts, ws, out, slot_of_expert=None,
                   flags: int = MOE_PATH_AUTO, stream=None):
    T, E = logits.shape
    _err(lib.moe_bf16_layer(_p(x), _p(logits), T, H, I, E, k, _p(w13), _p(w2), _p(slot_of_expert), _p(idx),
                            _p(wts), _p(ws), ws.numel() * ws.element_size(), _p(out), flags, _s(stream)))


# ---- rows sorted by expert and back, the router's gradient, norms around a block. These calls take
# the sizes, types and row strides from the tensors and check them (MoeError, MOE_ERR_ARG) in the
# native module _rows (csrc/binding.cpp); every tensor lives on one CUDA device, whose current
# stream is the default.


def moe_dispatch(x, idx, E: int, counts, offsets, perm, inv, xp, stream=None):
    """Sorts the token-expert pairs of idx (int32 [T][k]) by expert and writes each token's row of x
    [T][H] to its pairs' rows of xp [T*k][H]. counts [E], offsets [E+1], perm [T*k], inv [T][k] (int32)."""
    _rows.dispatch(x, idx, E, counts, offsets, perm, inv, xp, stream)


def moe_dispatch_backward(dxp, inv, dx, stream=None):
    """dx[t] = sum of the rows of dxp [T*k][H] that moe_dispatch filled from token t."""
    _rows.dispatch_backward(dxp, inv, dx, stream)


def moe_combine(yp, inv, wts, out, stream=None):
    """out[t] = sum_j wts[t][j] * yp[inv[t][j]]; yp [T*k][H] of out's type or fp32, wts fp32 [T][k]."""
    _rows.combine(yp, inv, wts, out, stream)


def moe_combine_backward(dout, yp, inv, wts, dyp=None, dwts=None, stream=None):
    """Gradients of moe_combine: dyp (rows like yp), dwts (fp32 [T][k]); either may be None. yp may be
    None when dwts is."""
    _rows.combine_backward(dout, yp, inv, wts, dyp, dwts, stream)


def moe_route_topk_backward(idx, wts, dwts, dlogits, stream=None):
    """Gradient of moe_route_topk's weights towards the logits: dlogits [T][E], 0 where not chosen. idx: the
    router's own ids, also of choices dropped after it (their logits have a gradient too)."""
    _rows.route_topk_backward(idx, wts, dwts, dlogits, stream)


def moe_norm_workspace_bytes(T: int, H: int) -> int:
    out = ctypes.c_size_t(0)
    _err(lib.moe_norm_workspace_bytes(T, H, ctypes.byref(out)))
    return out.value


def moe_norm_pre(h, w, eps: float, x, stream=None):
    """x = h / sqrt(mean(h^2) + eps) * w, row by row; w [H] or None."""
    _rows.norm_pre(h, w, eps, x, stream)


def moe_norm_pre_backward(dx, h, w, eps: float, dh, dres=None, dw=None, ws=None, stream=None):
    """Gradients of moe_norm_pre: dh (plus the residual path's dres), dw (fp32 [H]). dw needs ws, a
    workspace of moe_norm_workspace_bytes. dh may be dres."""
    _rows.norm_pre_backward(dx, h, w, eps, dh, dres, dw, ws, stream)


def moe_norm_post(y, h, h_out, eps: float, alpha: float = 1.0, norm_y: bool = True, w=None, gate=None, w_next=None,
                  x_next=None, stream=None):
    """h_out = alpha * h + gate * u with u = rms(y) * w (norm_y) or y, and with x_next given
    x_next = rms(h_out) * w_next. gate: None, [H], fp32 [T][1] or [T] (one value per token), or [T][H].
    fp32 rows with T = H take a single dimension as [H]. h_out may be h."""
    _rows.norm_post(y, h, h_out, eps, alpha, norm_y, w, gate, w_next, x_next, stream)


def moe_combine_norm_post(yp, inv, wts, h, h_out, eps: float, alpha: float = 1.0, norm_y: bool = True, w=None,
                          gate=None, w_next=None, x_next=None, y_out=None, stream=None):
    """moe_combine and moe_norm_post in one launch; y_out (optional) keeps the combined rows."""
    _rows.combine_norm_post(yp, inv, wts, h, h_out, eps, alpha, norm_y, w, gate, w_next, x_next, y_out, stream)


def moe_norm_post_backward(dh_out, y, dh, dy, eps: float, alpha: float = 1.0, norm_y: bool = True, w=None, dw=None,
                           gate=None, dgate=None, h_out=None, w_next=None, dx_next=None, dw_next=None, ws=None,
                           stream=None):
    """Gradients of moe_norm_post: dh, dy, and where given dw, dw_next (fp32 [H]) and dgate (fp32 [H], fp32
    [T][1] or [T], or rows, as the gate is). With dx_next given, h_out is the forward's output. Gradients of
    vectors need ws, a workspace of moe_norm_workspace_bytes. dh may be dh_out."""
    _rows.norm_post_backward(dh_out, y, dh, dy, eps, alpha, norm_y, w, dw, gate, dgate, h_out, w_next, dx_next,
                             dw_next, ws, stream)


def moe_noalloc_status(stream=None) -> int:
    """Reads and clears the device status word of the static array of moe_w4a16_layer_noalloc."""
    st = ctypes.c_int(0)
    _err(lib.moe_noalloc_status(_s(stream), ctypes.byref(st)))
    return st.value


class SlotCache:
    """Owner of a moe_slot_cache handle (one layer's GPU slot pool over a pinned host bank)."""

    def __init__(self, E: int, S: int, H: int, I: int, bank, pool):
        self.E, self.S, self.H, self.I = E, S, H, I
        self.bank, self.pool = bank, pool          # keep the memory alive
        h = ctypes.c_void_p(0)
        _err(lib.moe_slot_cache_create(E, S, H, I, *(_p(t) for t in bank), *(_p(t) for t in pool),
                                       ctypes.byref(h)))
        self.handle = h

    def close(self):
        if self.handle:
            lib.moe_slot_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def fail_copy_after(self, n: int):
        lib.moe_slot_cache_fail_copy_after(self.handle, n)

    def dry_run(self, dry: bool = True):
        """Plan and commit refills without copying (testing the policy without a GPU)."""
        lib.moe_slot_cache_dry_run(self.handle, int(dry))

    def state(self):
        import numpy as np
        se = np.zeros(self.S, np.int32)
        lu = np.zeros(self.S, np.int64)
        clock = lib.moe_slot_cache_state(self.handle, se.ctypes.data_as(ctypes.c_void_p),
                                         lu.ctypes.data_as(ctypes.c_void_p))
        return se, lu, clock

    def slot_table_update(self, needed_mask, wave_table, misses, copy_stream, reuse_ok=None, loaded=None):
        """needed_mask: numpy uint64 [ceil(E/64)] (updated); wave_table: numpy int32 [E];
        misses: numpy int32 [S]. Returns the number of misses."""
        n = ctypes.c_int(0)
        ev = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
        _err(lib.slot_table_update(self.handle, needed_mask.ctypes.data_as(ctypes.c_void_p),
                                   wave_table.ctypes.data_as(ctypes.c_void_p), misses.ctypes.data_as(ctypes.c_void_p),
                                   ctypes.byref(n), _s(copy_stream), ev(reuse_ok), ev(loaded)))
        return n.value

    def layer(self, x, logits, k: int, idx, wts, wave_tables, ws, out, path: int = MOE_PATH_AUTO,
              stream=None, copy_stream=None):
        T = logits.shape[0]
        nw, nl = ctypes.c_int(0), ctypes.c_int(0)
        _err(lib.moe_slot_cache_layer(self.handle, _p(x), _p(logits), T, k, _p(idx), _p(wts), _p(wave_tables),
                                      _p(ws), ws.numel() * ws.element_size(), _p(out), path, _s(stream),
                                      _s(copy_stream), ctypes.byref(nw), ctypes.byref(nl)))
        return nw.value, nl.value


def alloc_bank(E: int, N: int, K: int, device="cuda", pinned: bool = False):
    """Zeroed (packed uint8 [E][N*K/2], scales bf16 [E][N*K/128]) buffers for E matrices."""
    kw = dict(device=device) if not pinned else dict(device="cpu", pin_memory=True)
    packed = torch.zeros((E, moe_packed_bytes(N, K)), dtype=torch.uint8, **kw)
    scales = torch.zeros((E, moe_scales_count(N, K)), dtype=torch.bfloat16, **kw)
    return packed, scales


def alloc_workspace(T: int, H: int, I: int, E: int, k: int, device="cuda", stream=None) -> torch.Tensor:
    ws = torch.empty(moe_workspace_bytes(T, H, I, E, k), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws
