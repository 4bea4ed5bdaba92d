"""ctypes binding of libarmt.so (include/armt.h), same entry-point names.

Argument marshalling only: every step of the forward pass runs in the
library's CUDA kernels.  PyTorch is used for device memory and streams.  If
the library has not been built, importing the binding raises; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

import numpy as np

from . import inputs as _inputs

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libarmt.so")

ARMT_OK = 0
STATUS_NAMES = {0: "ARMT_OK", 1: "ARMT_ERR_ARG", 2: "ARMT_ERR_SHAPE", 3: "ARMT_ERR_UNSUPPORTED",
                4: "ARMT_ERR_OOM", 5: "ARMT_ERR_CUDA", 6: "ARMT_ERR_TIMEOUT", 7: "ARMT_ERR_NO_DEVICE"}
ARMT_F32, ARMT_BF16 = 0, 1
PRECISION_BF16, PRECISION_BF16X2 = 0, 1
SCHEDULE_DIAGONAL, SCHEDULE_SEQUENTIAL, SCHEDULE_WAVEFRONT = 0, 1, 2
CACHE_BF16, CACHE_E4M3 = 0, 1
KERNEL_CLASSES = ("gemm_qkv", "gemm_o", "gemm_gateup", "gemm_down", "attention", "assoc_read",
                  "assoc_write", "norm", "other")

EXPORTED = ("armt_create", "armt_destroy", "armt_forward", "armt_forward_sequential",
            "armt_forward_batch", "armt_forward_host", "armt_grouped_gemm_bf16", "armt_segment_attention_bf16",
            "armt_segment_attention_bf16_noalloc", "armt_forward_full_attention", "armt_state_sizes",
            "armt_memory_bytes", "armt_lm_head", "armt_launch_count",
            "armt_set_profiling", "armt_set_profiling_mask", "armt_kernel_times", "armt_sync_status", "armt_status_string",
            "armt_last_error", "armt_block_sync_status", "armt_noalloc_sync_status", "armt_backward",
            "armt_backward_stats", "armt_set_tracing", "armt_cache_write_bf16", "armt_cache_read_bf16",
            "armt_paged_attention_bf16", "armt_paged_attention_workspace", "armt_token_probs",
            "armt_verify_drafts")


class ArmtError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")


class armt_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("ffn_dim", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("seg_len", ctypes.c_int32),
                ("n_mem", ctypes.c_int32), ("key_dim", ctypes.c_int32),
                ("dpfp_nu", ctypes.c_int32), ("norm_eps", ctypes.c_float),
                ("assoc_eps", ctypes.c_float), ("rope_base", ctypes.c_double),
                ("dtype", ctypes.c_int32), ("precision", ctypes.c_int32)]


_WKEYS = ("embed", "mem", "wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "a_wq", "a_wk",
          "a_wv", "a_wbeta", "norm1", "norm2", "norm_f")


class armt_weights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in _WKEYS] + [("on_device", ctypes.c_int32)]


GRAD_KEYS = _WKEYS + ("mem_A", "mem_z")


class armt_grads(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in GRAD_KEYS]


class armt_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("type", ctypes.c_int32)]


class armt_paged_batch(ctypes.Structure):
    _fields_ = [("row_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_rows", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("max_new", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libarmt.so; raises FileNotFoundError when it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} not built: run python -m recurrent_memory_transformer_gb300.build")
    lib = ctypes.CDLL(path)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    S = ctypes.c_int
    lib.armt_create.argtypes = [ctypes.POINTER(armt_config), ctypes.POINTER(armt_weights), P,
                                ctypes.POINTER(P)]
    lib.armt_destroy.argtypes = [P]
    for fn in (lib.armt_forward, lib.armt_forward_sequential):
        fn.argtypes = [P, P, I64, P, P, P, I32, P]
    lib.armt_forward_batch.argtypes = [P, P, I32, I64, P, P, P, I32, I32, P]
    lib.armt_forward_host.argtypes = [P, P, I64, P, P, P, I32, I32, P]
    lib.armt_forward_full_attention.argtypes = [P, P, I64, P, P]
    lib.armt_grouped_gemm_bf16.argtypes = [P, P, P, I32, I32, I32, I32, P]
    lib.armt_segment_attention_bf16.argtypes = [P, P, P, I32, I32, I32, I32, I32, P]
    lib.armt_segment_attention_bf16_noalloc.argtypes = [P, P, I32, I32, I32, I32, I32, P]
    lib.armt_state_sizes.argtypes = [P, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    lib.armt_lm_head.argtypes = [P, P, I64, P, P, P]
    lib.armt_memory_bytes.argtypes = [P, ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(I64)]
    lib.armt_launch_count.argtypes = [P, I64, I32, ctypes.POINTER(I64)]
    lib.armt_set_profiling.argtypes = [P, I32]
    lib.armt_set_tracing.argtypes = [P, I32]
    lib.armt_set_profiling_mask.argtypes = [P, ctypes.c_uint32]
    lib.armt_kernel_times.argtypes = [P, ctypes.POINTER(I64), ctypes.POINTER(ctypes.c_double), I32]
    lib.armt_sync_status.argtypes = [P, P]
    lib.armt_block_sync_status.argtypes = [P]
    lib.armt_noalloc_sync_status.argtypes = [P]
    lib.armt_backward.argtypes = [P, P, I64, P, P, P, P, P, P, P, P, ctypes.POINTER(armt_grads), P]
    lib.armt_backward_stats.argtypes = [P, ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(ctypes.c_double)]
    CACHE, BATCH = ctypes.POINTER(armt_kv_cache), ctypes.POINTER(armt_paged_batch)
    lib.armt_cache_write_bf16.argtypes = [P, I64, P, I64, CACHE, BATCH, P]
    lib.armt_cache_read_bf16.argtypes = [CACHE, BATCH, P, I64, P, I64, P]
    lib.armt_paged_attention_bf16.argtypes = [P, I64, CACHE, BATCH, I32, ctypes.c_float, P, I64, P, I64, P]
    lib.armt_paged_attention_workspace.argtypes = [CACHE, BATCH, I32, ctypes.POINTER(I64)]
    lib.armt_token_probs.argtypes = [P, I64, P, I64, I32, P, I64, P]
    lib.armt_verify_drafts.argtypes = [P, I64, P, I64, P, P, P, I32, I64, I32, P, P, P]
    for name in EXPORTED:
        getattr(lib, name).restype = S
    lib.armt_status_string.restype = ctypes.c_char_p
    lib.armt_status_string.argtypes = [S]
    lib.armt_last_error.restype = ctypes.c_char_p
    lib.armt_last_error.argtypes = []
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != ARMT_OK:
        detail = _lib.armt_last_error().decode(errors="replace")
        raise ArmtError(status, where, detail)


def make_config(cfg: "_inputs.ArmtConfig") -> armt_config:
    return armt_config(cfg.n_layers, cfg.d_model, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim,
                       cfg.ffn_dim, cfg.vocab, cfg.seg_len, cfg.n_mem, cfg.key_dim, cfg.dpfp_nu,
                       cfg.norm_eps, cfg.assoc_eps, cfg.rope_base,
                       ARMT_BF16 if cfg.dtype == "bf16" else ARMT_F32,
                       PRECISION_BF16X2 if cfg.precision == "bf16x2" else PRECISION_BF16)


def _stream_ptr(stream) -> Optional[int]:
    if stream is None:
        import torch
        # the raw handle, without the Stream object around it (0.3 instead of 3 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return getattr(stream, "cuda_stream", stream)


def _ptr(t) -> int:
    return t.data_ptr()


def host_weight_arrays(cfg, weights: Dict[str, np.ndarray]) -> Dict[str, np.ndarray]:
    """Contiguous host arrays in the model's element type (fp32, or bf16 bits as uint16)."""
    out = {}
    for k in _WKEYS:
        a = np.ascontiguousarray(weights[k], dtype=np.float32)
        out[k] = _inputs.bf16_bits(a) if cfg.dtype == "bf16" else a
    return out


def device_weight_tensors(cfg, weights: Dict[str, np.ndarray], device="cuda"):
    """Device tensors in the model's element type (exact: inputs are bf16-representable)."""
    import torch
    dt = torch.bfloat16 if cfg.dtype == "bf16" else torch.float32
    return {k: torch.from_numpy(np.ascontiguousarray(weights[k], dtype=np.float32)).to(device).to(dt)
            for k in _WKEYS}


class Model:
    """Owns one armt_model; wraps the forward entry points."""

    def __init__(self, cfg, weights, stream=None):
        """`weights`: dict of numpy arrays (host path) or torch tensors on the device."""
        lib = load_library()
        self.cfg = cfg
        self._c = make_config(cfg)
        w = armt_weights()
        keep = []
        first = weights["embed"]
        on_device = hasattr(first, "is_cuda") and first.is_cuda
        if on_device:
            for k in _WKEYS:
                t = weights[k].contiguous()
                keep.append(t)
                setattr(w, k, t.data_ptr())
        else:
            arrs = host_weight_arrays(cfg, weights)
            for k in _WKEYS:
                keep.append(arrs[k])
                setattr(w, k, arrs[k].ctypes.data)
        w.on_device = 1 if on_device else 0
        h = ctypes.c_void_p()
        _check(lib.armt_create(ctypes.byref(self._c), ctypes.byref(w), _stream_ptr(stream),
                               ctypes.byref(h)), "armt_create")
        self._h = h
        a, z = ctypes.c_int64(), ctypes.c_int64()
        _check(lib.armt_state_sizes(h, ctypes.byref(a), ctypes.byref(z)), "armt_state_sizes")
        self.a_elems, self.z_elems = a.value, z.value

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _check(_lib.armt_destroy(self._h), "armt_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def armt_forward(self, tokens, n_segments, hidden_out, mem_A, mem_z, mem_in_valid=0,
                     stream=None, schedule=SCHEDULE_DIAGONAL):
        fn = _lib.armt_forward if schedule == SCHEDULE_DIAGONAL else _lib.armt_forward_sequential
        _check(fn(self._h, _ptr(tokens), int(n_segments), _ptr(hidden_out), _ptr(mem_A),
                  _ptr(mem_z), int(mem_in_valid), _stream_ptr(stream)),
               "armt_forward" if schedule == SCHEDULE_DIAGONAL else "armt_forward_sequential")

    def armt_forward_sequential(self, tokens, n_segments, hidden_out, mem_A, mem_z, mem_in_valid=0,
                                stream=None):
        self.armt_forward(tokens, n_segments, hidden_out, mem_A, mem_z, mem_in_valid, stream,
                          SCHEDULE_SEQUENTIAL)

    def armt_forward_batch(self, tokens, hidden_out, mem_A, mem_z, mem_in_valid=0,
                           schedule=SCHEDULE_DIAGONAL, stream=None):
        """tokens int32 [B, N] (device), hidden fp32 [B, N, d], state [L, B, d, P] and [L, B, P]."""
        B_, N = tokens.shape
        _check(_lib.armt_forward_batch(self._h, _ptr(tokens), int(B_), int(N), _ptr(hidden_out),
                                       _ptr(mem_A), _ptr(mem_z), int(mem_in_valid), int(schedule),
                                       _stream_ptr(stream)), "armt_forward_batch")

    def forward_batch(self, tokens, schedule=SCHEDULE_DIAGONAL, mem_A=None, mem_z=None, stream=None):
        """Allocates outputs with torch; tokens int32 [B, N] on the device (N any
        positive count: a short last segment is allowed).  Returns (hidden
        [B, N, d], A [L, B, d, P], z [L, B, P])."""
        import torch
        dev = tokens.device
        B_, N = tokens.shape
        L, d, P = self.cfg.n_layers, self.cfg.d_model, self.cfg.phi_dim
        hidden = torch.empty((B_, N, d), dtype=torch.float32, device=dev)
        valid = mem_A is not None
        A = mem_A.clone() if valid else torch.empty((L, B_, d, P), dtype=torch.float32, device=dev)
        z = mem_z.clone() if valid else torch.empty((L, B_, P), dtype=torch.float32, device=dev)
        self.armt_forward_batch(tokens, hidden, A, z, 1 if valid else 0, schedule, stream)
        return hidden, A.view(L, B_, d, P), z.view(L, B_, P)

    def armt_forward_host(self, tokens: np.ndarray, n_segments, hidden_out: np.ndarray,
                          mem_A: np.ndarray, mem_z: np.ndarray, mem_in_valid=0,
                          schedule=SCHEDULE_DIAGONAL, stream=None):
        """Host-buffer forward (numpy arrays or pinned CPU tensors); synchronous."""
        def hp(x):
            return x.data_ptr() if hasattr(x, "data_ptr") else x.ctypes.data
        _check(_lib.armt_forward_host(self._h, hp(tokens), int(n_segments), hp(hidden_out),
                                      hp(mem_A), hp(mem_z), int(mem_in_valid), int(schedule),
                                      _stream_ptr(stream)), "armt_forward_host")

    def forward(self, tokens, n_segments, schedule=SCHEDULE_DIAGONAL, mem_A=None, mem_z=None,
                stream=None):
        """Allocates outputs with torch and runs one forward; returns (hidden, A, z)."""
        import torch
        dev = tokens.device
        hidden = torch.empty((n_segments * self.cfg.seg_len, self.cfg.d_model), dtype=torch.float32,
                             device=dev)
        valid = mem_A is not None
        A = mem_A.clone() if valid else torch.empty(self.a_elems, dtype=torch.float32, device=dev)
        z = mem_z.clone() if valid else torch.empty(self.z_elems, dtype=torch.float32, device=dev)
        self.armt_forward(tokens, n_segments, hidden, A, z, 1 if valid else 0, stream, schedule)
        L, d, P = self.cfg.n_layers, self.cfg.d_model, self.cfg.phi_dim
        return hidden, A.view(L, d, P), z.view(L, P)

    def armt_backward(self, tokens, grads, mem_A0=None, mem_z0=None, cot_hidden=None, cot_A=None,
                      cot_z=None, hidden_out=None, mem_A_out=None, mem_z_out=None, stream=None):
        """Device tensors (None where the header allows NULL); grads: dict of
        fp32 device tensors keyed like the weights (+ optional mem_A, mem_z)."""
        g = armt_grads()
        for k in GRAD_KEYS:
            t = grads.get(k)
            setattr(g, k, None if t is None else _ptr(t))

        def opt(t):
            return None if t is None else _ptr(t)
        _check(_lib.armt_backward(self._h, _ptr(tokens), int(tokens.numel()), opt(mem_A0), opt(mem_z0),
                                  opt(cot_hidden), opt(cot_A), opt(cot_z), opt(hidden_out), opt(mem_A_out),
                                  opt(mem_z_out), ctypes.byref(g), _stream_ptr(stream)), "armt_backward")

    def armt_backward_stats(self):
        """(kernel launches, algorithmic FLOPs) of the last backward, and its workspace bytes."""
        a, b, f = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_double()
        _check(_lib.armt_backward_stats(self._h, ctypes.byref(a), ctypes.byref(b), ctypes.byref(f)),
               "armt_backward_stats")
        return a.value, f.value, b.value

    def backward(self, tokens, cot_hidden=None, cot_A=None, cot_z=None, mem_A0=None, mem_z0=None,
                 state_grads=False, stream=None):
        """Allocates the gradients with torch; returns (grads dict, (hidden, A, z))."""
        import torch
        c, dev = self.cfg, tokens.device
        L, d, P = c.n_layers, c.d_model, c.phi_dim
        shapes = _inputs.weight_shapes(c)
        grads = {k: torch.empty(shapes[k], dtype=torch.float32, device=dev) for k in _WKEYS}
        if state_grads:
            grads["mem_A"] = torch.empty((L, d, P), dtype=torch.float32, device=dev)
            grads["mem_z"] = torch.empty((L, P), dtype=torch.float32, device=dev)
        hidden = torch.empty((tokens.numel(), d), dtype=torch.float32, device=dev)
        A = torch.empty((L, d, P), dtype=torch.float32, device=dev)
        z = torch.empty((L, P), dtype=torch.float32, device=dev)
        self.armt_backward(tokens, grads, mem_A0, mem_z0, cot_hidden, cot_A, cot_z, hidden, A, z, stream)
        return grads, (hidden, A, z)

    def armt_set_tracing(self, enable=True):
        """NVTX ranges around every step (forward diagonals or cells, backward diagonals)."""
        _check(_lib.armt_set_tracing(self._h, 1 if enable else 0), "armt_set_tracing")

    def armt_forward_full_attention(self, tokens, hidden_out, stream=None):
        """Plain causal LLaMA over all tokens (no memory), same weights."""
        _check(_lib.armt_forward_full_attention(self._h, _ptr(tokens), int(tokens.numel()),
                                                _ptr(hidden_out), _stream_ptr(stream)),
               "armt_forward_full_attention")

    def armt_lm_head(self, hidden, logits, w_head=None, stream=None):
        """logits fp32 [rows, vocab] = hidden fp32 [rows, d] @ head^T (head: w_head or the tied embedding)."""
        _check(_lib.armt_lm_head(self._h, _ptr(hidden), int(hidden.shape[0]),
                                 None if w_head is None else _ptr(w_head), _ptr(logits),
                                 _stream_ptr(stream)), "armt_lm_head")

    def armt_memory_bytes(self):
        """(weights, workspace, full_workspace): device bytes the library holds for this model."""
        w, ws, fw = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(_lib.armt_memory_bytes(self._h, ctypes.byref(w), ctypes.byref(ws), ctypes.byref(fw)),
               "armt_memory_bytes")
        return w.value, ws.value, fw.value

    def armt_launch_count(self, n_segments, schedule=SCHEDULE_DIAGONAL) -> int:
        n = ctypes.c_int64()
        _check(_lib.armt_launch_count(self._h, int(n_segments), int(schedule), ctypes.byref(n)),
               "armt_launch_count")
        return n.value

    def armt_set_profiling(self, enable: bool):
        _check(_lib.armt_set_profiling(self._h, 1 if enable else 0), "armt_set_profiling")

    def armt_set_profiling_mask(self, classes):
        """Time only the launches of the named kernel classes (KERNEL_CLASSES); [] turns it off."""
        mask = 0
        for c in classes:
            mask |= 1 << KERNEL_CLASSES.index(c)
        _check(_lib.armt_set_profiling_mask(self._h, mask), "armt_set_profiling_mask")

    def armt_kernel_times(self):
        n = len(KERNEL_CLASSES)
        launches = (ctypes.c_int64 * n)()
        ms = (ctypes.c_double * n)()
        _check(_lib.armt_kernel_times(self._h, launches, ms, n), "armt_kernel_times")
        return {KERNEL_CLASSES[i]: (launches[i], ms[i]) for i in range(n)}

    def armt_sync_status(self, stream=None):
        _check(_lib.armt_sync_status(self._h, _stream_ptr(stream)), "armt_sync_status")


def armt_grouped_gemm_bf16(A, B, C, stream=None):
    """C[g] = A[g] @ B[g]^T: A bf16 [G,M,K], B bf16 [G,N,K], C fp32 [G,M,N] (torch, cuda)."""
    lib = load_library()
    G, M, K = A.shape
    N = B.shape[1]
    _check(lib.armt_grouped_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), G, M, N, K, _stream_ptr(stream)),
           "armt_grouped_gemm_bf16")


def armt_segment_attention_bf16(qk, vt, out, Hq, Hkv, stream=None):
    """Causal GQA per cell: qk bf16 [G,T,(Hq+Hkv)*hd], vt bf16 [G,Hkv,hd,T], out bf16 [G,T,Hq*hd]."""
    lib = load_library()
    G, T, _ = qk.shape
    hd = vt.shape[2]
    _check(lib.armt_segment_attention_bf16(_ptr(qk), _ptr(vt), _ptr(out), G, T, Hq, Hkv, hd,
                                           _stream_ptr(stream)), "armt_segment_attention_bf16")


def armt_segment_attention_bf16_noalloc(qkv, out, Hq, Hkv, hd, stream=None):
    """Same attention from the fused row layout qkv bf16 [G,T,(Hq+2Hkv)*hd]; allocates nothing."""
    lib = load_library()
    G, T, _ = qkv.shape
    _check(lib.armt_segment_attention_bf16_noalloc(_ptr(qkv), _ptr(out), G, T, Hq, Hkv, hd,
                                                   _stream_ptr(stream)),
           "armt_segment_attention_bf16_noalloc")


def armt_block_sync_status(stream=None):
    """Raises ArmtError(ARMT_ERR_TIMEOUT) if a building block's bounded wait gave up on this device."""
    lib = load_library()
    _check(lib.armt_block_sync_status(_stream_ptr(stream)), "armt_block_sync_status")


def armt_noalloc_sync_status(stream=None):
    """Raises ArmtError(ARMT_ERR_TIMEOUT) if the no-allocation attention's bounded wait gave up."""
    lib = load_library()
    _check(lib.armt_noalloc_sync_status(_stream_ptr(stream)), "armt_noalloc_sync_status")


# ------------------------------------------------------------- serving --

# These calls are made once a token, so what Python adds to them counts: torch
# is looked up once (an import statement in a function is 0.2 us), and a tensor
# is asked for as little as its check needs.
_torch = None


def _with_torch():
    global _torch
    if _torch is None:
        import torch
        load_library()
        _torch = torch
    return _torch


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _raw_stream(stream, dev):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev)
    return getattr(stream, "cuda_stream", stream)


def _rows(t, heads, hd, n_rows, dev, what):
    """Row stride of a [n_rows, heads, hd] bf16 tensor on device `dev` whose rows are each contiguous."""
    if t.dtype is not _torch.bfloat16 or t.shape != (n_rows, heads, hd) or t.get_device() != dev:
        raise ValueError(f"{what}: a bf16 tensor of shape {(n_rows, heads, hd)} on the current CUDA device is needed")
    row, head, one = t.stride()
    if one != 1 or (head != hd and heads > 1):
        raise ValueError(f"{what}: the heads of a row must be contiguous")
    return row if n_rows > 1 else heads * hd


def _current(*owners):
    """The current device, which every tensor of a call has to be on."""
    dev = _with_torch().cuda.current_device()
    for o in owners:
        if o.device_index != dev:
            raise ValueError("the cache and the batch must be on the current CUDA device")
    return dev


class KvCache:
    """A paged cache over the caller's pools (torch, cuda), for the calls below.

    k, v: [n_pages, n_kv_heads, page_size, head_dim], bf16, or float8_e4m3fn
    (or uint8) with k_scale, v_scale: uint8 [n_pages, n_kv_heads, page_size].
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        _need(k.is_cuda and v.is_cuda and k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and
              k.is_contiguous() and v.is_contiguous() and k.device == v.device,
              "k, v: contiguous 4-D CUDA tensors alike")
        codes = k.dtype in (torch.float8_e4m3fn, torch.uint8)
        _need(codes or k.dtype == torch.bfloat16, f"no cache of {k.dtype}")
        for s in (k_scale, v_scale):
            _need((s is not None) == codes, "k_scale and v_scale go with 8-bit pools, and only with them")
            _need(s is None or (s.dtype == torch.uint8 and s.shape == k.shape[:3] and s.is_contiguous() and
                                s.device == k.device), "scales: contiguous uint8 [n_pages, n_kv_heads, page_size]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.type = CACHE_E4M3 if codes else CACHE_BF16
        self.device_index = k.get_device()
        self._c = armt_kv_cache(_ptr(k), _ptr(v), None if k_scale is None else _ptr(k_scale),
                                None if v_scale is None else _ptr(v_scale), self.n_pages, self.page_size,
                                self.n_kv_heads, self.head_dim, self.type)
        self._ref = ctypes.byref(self._c)

    @staticmethod
    def allocate(n_pages, page_size, n_kv_heads, head_dim, type=CACHE_BF16, device="cuda"):
        """Pools of zeros (e4m3: scale bytes 0), allocated with torch."""
        import torch
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        if type == CACHE_BF16:
            return KvCache(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        _need(type == CACHE_E4M3, f"no cache type {type}")
        pools = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        return KvCache(*pools, *(torch.zeros(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)))


class PagedBatch:
    """The sequences of a call: int32 CUDA tensors row_start [n_seqs + 1], kv_len
    [n_seqs] and page_table [n_seqs, width].  They are read when the kernels
    run, so they may be updated in place between calls (also of a CUDA graph);
    n_rows and max_new are upper bounds fixed here."""

    def __init__(self, row_start, kv_len, page_table, n_rows, max_new):
        import torch
        for t, d in ((row_start, 1), (kv_len, 1), (page_table, 2)):
            _need(t.is_cuda and t.dtype == torch.int32 and t.dim() == d and t.is_contiguous(),
                  "row_start, kv_len, page_table: contiguous int32 CUDA tensors")
        n = kv_len.shape[0]
        _need(row_start.shape[0] == n + 1 and page_table.shape[0] == n,
              "row_start has one entry more than kv_len, page_table as many rows")
        self.row_start, self.kv_len, self.page_table = row_start, kv_len, page_table
        self.n_seqs, self.n_rows, self.max_new = n, int(n_rows), int(max_new)
        self.device_index = kv_len.get_device()
        _need(row_start.get_device() == page_table.get_device() == self.device_index, "one device for all three")
        self._c = armt_paged_batch(_ptr(row_start), _ptr(kv_len), _ptr(page_table), self.n_rows, n,
                                   page_table.shape[1], self.max_new)
        self._ref = ctypes.byref(self._c)


def armt_cache_write_bf16(k, v, cache, batch, stream=None):
    """Writes the batch's new rows, k and v bf16 [n_rows, n_kv_heads, head_dim] (rows may be
    strided, as slices of fused q|k|v rows are), into the cache."""
    dev = _current(cache, batch)
    ks = _rows(k, cache.n_kv_heads, cache.head_dim, batch.n_rows, dev, "k")
    vs = _rows(v, cache.n_kv_heads, cache.head_dim, batch.n_rows, dev, "v")
    _check(_lib.armt_cache_write_bf16(_ptr(k), ks, _ptr(v), vs, cache._ref, batch._ref, _raw_stream(stream, dev)),
           "armt_cache_write_bf16")


def armt_cache_read_bf16(cache, batch, k, v, stream=None):
    """Copies the rows at the batch's positions out of the cache into k and v."""
    dev = _current(cache, batch)
    ks = _rows(k, cache.n_kv_heads, cache.head_dim, batch.n_rows, dev, "k")
    vs = _rows(v, cache.n_kv_heads, cache.head_dim, batch.n_rows, dev, "v")
    _check(_lib.armt_cache_read_bf16(cache._ref, batch._ref, _ptr(k), ks, _ptr(v), vs, _raw_stream(stream, dev)),
           "armt_cache_read_bf16")


def armt_paged_attention_workspace(cache, batch, n_q_heads) -> int:
    """Bytes of workspace that armt_paged_attention_bf16 needs for this batch."""
    n = ctypes.c_int64()
    _check(load_library().armt_paged_attention_workspace(cache._ref, batch._ref, int(n_q_heads), ctypes.byref(n)),
           "armt_paged_attention_workspace")
    return n.value


def paged_attention_workspace(cache, batch, n_q_heads):
    """That workspace, allocated with torch.  One for the batch with the most new rows a sequence
    serves all calls with these heads on a stream, over either type of cache; calls that may overlap
    on the device need one each."""
    import torch
    return torch.empty(armt_paged_attention_workspace(cache, batch, n_q_heads), dtype=torch.uint8,
                       device=cache.k.device)


def armt_paged_attention_bf16(q, cache, batch, out, workspace, scale=None, stream=None):
    """Causal attention of the batch's new rows over the cache, which holds theirs too: q, out
    bf16 [n_rows, n_q_heads, head_dim] (rows may be strided); scale: 1 / sqrt(head_dim) if None."""
    heads, hd = q.shape[1], cache.head_dim
    dev = _current(cache, batch)
    qs = _rows(q, heads, hd, batch.n_rows, dev, "q")
    os_ = _rows(out, heads, hd, batch.n_rows, dev, "out")
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the current CUDA device is needed")
    _check(_lib.armt_paged_attention_bf16(_ptr(q), qs, cache._ref, batch._ref, heads,
                                         hd ** -0.5 if scale is None else scale, _ptr(out), os_, _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _raw_stream(stream, dev)),
           "armt_paged_attention_bf16")


def _vocab_rows(t, dev, what):
    if t.dtype is not _torch.float32 or t.dim() != 2 or t.get_device() != dev:
        raise ValueError(f"{what}: a 2-D fp32 tensor on the current CUDA device is needed")
    rows, width = t.shape
    row, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return row if rows > 1 else max(row, width)


def _vector(t, n, dtype, dev, what):
    if t.dtype is not dtype or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor of {n} {dtype} on the current CUDA device is needed")
    return t.data_ptr()


def armt_token_probs(logits, probs, temperature=None, stream=None):
    """probs = softmax(logits / temperature) by rows, fp32 [rows, vocab] (views of wider rows are
    fine; probs may be logits); temperature: fp32 [rows] or None for 1; <= 0 asks for the greedy choice."""
    dev = _current()
    li, lo = _vocab_rows(logits, dev, "logits"), _vocab_rows(probs, dev, "probs")
    rows, vocab = logits.shape
    if probs.shape != (rows, vocab):
        raise ValueError("logits and probs must have one shape")
    t = None if temperature is None else _vector(temperature, rows, _torch.float32, dev, "temperature")
    _check(_lib.armt_token_probs(_ptr(logits), li, t, rows, vocab, _ptr(probs), lo, _raw_stream(stream, dev)),
           "armt_token_probs")


def armt_verify_drafts(target, draft, tokens, start, uniform, n_accepted, out_tokens, stream=None):
    """Checks drafted tokens: target fp32 [drafts + seqs, vocab], draft fp32 [drafts, vocab] or None
    (certain drafts), tokens int32 [drafts], start int32 [seqs + 1], uniform fp32 [drafts + seqs];
    writes n_accepted int32 [seqs] and out_tokens int32 [drafts + seqs]."""
    n_drafts, n_seqs = tokens.shape[0], start.shape[0] - 1
    dev, rows = _current(), n_drafts + n_seqs
    i32 = _torch.int32
    lt = _vocab_rows(target, dev, "target")
    ld = 0 if draft is None else _vocab_rows(draft, dev, "draft")
    if target.shape[0] != rows or (draft is not None and draft.shape != (n_drafts, target.shape[1])):
        raise ValueError("target has a row for each draft and one more for each sequence, draft one for each draft")
    _check(_lib.armt_verify_drafts(_ptr(target), lt, None if draft is None else _ptr(draft), ld,
                                  _vector(tokens, n_drafts, i32, dev, "tokens"),
                                  _vector(start, n_seqs + 1, i32, dev, "start"),
                                  _vector(uniform, rows, _torch.float32, dev, "uniform"), n_seqs, n_drafts,
                                  target.shape[1], _vector(n_accepted, n_seqs, i32, dev, "n_accepted"),
                                  _vector(out_tokens, rows, i32, dev, "out_tokens"), _raw_stream(stream, dev)),
           "armt_verify_drafts")
