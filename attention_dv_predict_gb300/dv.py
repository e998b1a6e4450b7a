"""Python binding of libdv.so (include/dv.h): argument marshalling only.

Every computation runs in the library's CUDA kernels.  PyTorch supplies
device memory and streams.  Importing this module fails if the library has
not been built (``python -m attention_dv_predict_gb300.build``); there is no
fallback.
"""

from __future__ import annotations

import ctypes as C
import os
from typing import Dict, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m attention_dv_predict_gb300.build` "
        "(the sparse layer decode has no CPU fallback)")

_lib = C.CDLL(LIB_PATH)

DV_OK, DV_ERR_INVALID_ARG, DV_ERR_UNSUPPORTED, DV_ERR_CUDA = 0, 1, 2, 3
DV_ERR_TIMEOUT, DV_ERR_WORKSPACE, DV_ERR_DEVICE_INDEX, DV_ERR_SCRATCH_LIMIT = 4, 5, 6, 7
DV_F32, DV_F16, DV_I8 = 0, 1, 2
DV_LAYERNORM, DV_RMSNORM = 0, 1
DV_MLP_RELU, DV_MLP_SWIGLU = 0, 1
DV_MAX_BATCH = 32
DV_KV_MAX_BATCH = 256
DV_TREE_MAX_TOKENS = 64

WEIGHT_FIELDS = ("ln1_g", "ln1_b", "w_qkv", "b_qkv", "w_oT", "b_o", "ln2_g", "ln2_b",
                 "w1", "b1", "w2T", "b2", "pred_h", "pred_a", "pred_b")


class LayerDesc(C.Structure):
    _fields_ = [("d_model", C.c_int32), ("n_heads", C.c_int32), ("head_dim", C.c_int32),
                ("d_ffn", C.c_int32), ("pred_rank", C.c_int32), ("dtype", C.c_int32),
                ("norm", C.c_int32), ("ln_eps", C.c_float), ("kv_cap", C.c_int32),
                ("neuron_block", C.c_int32), ("mlp", C.c_int32)]


class LayerWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in WEIGHT_FIELDS]


class Selection(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("idx_h", "idx_n", "u_h", "n_u_h", "u_n", "n_u_n")]


class KvDesc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_heads", "n_kv_heads", "head_dim", "kv_cap", "dtype",
                                         "block")]


class KvCachePointers(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "k_mean",
                                          "k_mean_scale")]


class KvRows(C.Structure):
    _fields_ = [("p", C.c_void_p), ("dtype", C.c_int32), ("stride_b", C.c_int64),
                ("stride_t", C.c_int64), ("stride_h", C.c_int64)]


_P = C.c_void_p
_I = C.c_int
_SZ = C.c_size_t
_D = C.POINTER(LayerDesc)
_W = C.POINTER(LayerWeights)
_S = C.POINTER(Selection)
_KD = C.POINTER(KvDesc)
_KC = C.POINTER(KvCachePointers)
_KR = C.POINTER(KvRows)

_SIGS = {
    "dv_status_string": ([_I], C.c_char_p),
    "dv_cuda_error": ([], _I),
    "dv_abi_version": ([], _I),
    "dv_set_row_kernel": ([_I], _I),
    "dv_workspace_size": ([_D, _I], _SZ),
    "dv_workspace_init": ([_P, _SZ, _P], _I),
    "dv_check": ([_P, _SZ, _P], _I),
    "dv_layer_decode_launches": ([_D, _I], _I),
    "dv_layer_decode_persistent_ok": ([_D, _I], _I),
    "dv_mlp_one_pass": ([_D, _I, _I], _I),
    "dv_predict_topk": ([_D, _W, _P, _I, _I, _I, _S, _P, _P, _P, _SZ, _P], _I),
    "dv_predict_topk_noalloc": ([_D, _W, _P, _I, _I, _I, _S, _P, _P, _P], _I),
    "dv_sparse_attn": ([_D, _W, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _SZ, _P], _I),
    "dv_sparse_mlp": ([_D, _W, _P, _I, _P, _P, _I, _P, _P, _SZ, _P], _I),
    "dv_layer_decode": ([_D, _W, _P, _P, _I, _I, _I, _P, _P, _I, _S, _P, _P, _P, _SZ, _P], _I),
    "dv_layer_decode_persistent": ([_D, _W, _P, _P, _I, _I, _I, _P, _P, _I, _S, _P, _P, _P, _SZ,
                                    _P], _I),
    "dv_layer_decode_chained": ([_D, _W, _P, _P, _I, _I, _I, _P, _P, _I, _S, _P, _P, _P, _SZ,
                                 _P], _I),
    "dv_layer_decode_stamped": ([_D, _W, _P, _P, _I, _I, _I, _P, _P, _I, _S, _P, _P, _P, _SZ,
                                 _I, _P, _I, _P], _I),
    "dv_layer_decode_presel": ([_D, _W, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _P,
                                _SZ, _P], _I),
    "dv_layer_decode_traced": ([_D, _W, _P, _P, _I, _I, _I, _P, _P, _I, _S, _P, _P, _P, _SZ,
                                C.POINTER(_P), _I, _P], _I),
    "dv_layer_decode_host": ([_D, _W, _P, _P, _I, _I, _I, _P, _P, _I, _S, _P, _P, _SZ, _P], _I),
    "dv_hbm_copy": ([_P, _P, _SZ, _P], _I),
    "dv_test_hold_wait": ([_P, _SZ, _I, _I, _P], _I),
    "dv_set_tree_kernel": ([_I], _I),
    "dv_kv_workspace_size": ([_KD, _I, _I], _SZ),
    "dv_kv_append": ([_KD, _KC, _KR, _KR, _I, _I, _P, _P, _P, _SZ, _P], _I),
    "dv_kv_read": ([_KD, _KC, _I, _I, _P, _I, _P, _P, _P, _SZ, _P], _I),
    "dv_kv_keep": ([_KD, _KC, _I, _I, _P, _P, _P, _P, _SZ, _P], _I),
    "dv_tree_attn": ([_KD, _KC, _KR, _I, _I, _P, _P, _P, C.c_float, _P, _P, _I, _P, _P, _SZ, _P],
                     _I),
    "dv_block_topk": ([_KD, _KC, _KR, _I, _P, _I, _I, _I, _P, _P, _SZ, _P], _I),
    "dv_block_attn": ([_KD, _KC, _KR, _I, _P, _P, _I, C.c_float, _P, _P, _SZ, _P], _I),
}
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = tuple(_SIGS)


class DvError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        extra = f", cudaError {cuda_error}" if cuda_error else ""
        super().__init__(f"{fn}: {status_string(status)} ({status}{extra})")


def status_string(status: int) -> str:
    return _lib.dv_status_string(int(status)).decode()


def abi_version() -> int:
    return _lib.dv_abi_version()


def _check(fn: str, status: int):
    if status == DV_ERR_CUDA:
        raise DvError(fn, status, int(_lib.dv_cuda_error()))
    if status != DV_OK:
        raise DvError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return C.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


# ---------------------------------------------------------------------------


def make_desc(d_model, n_heads, head_dim, d_ffn, pred_rank, dtype, kv_cap,
              norm=DV_LAYERNORM, ln_eps=1e-5, neuron_block=0, mlp=0) -> LayerDesc:
    return LayerDesc(d_model, n_heads, head_dim, d_ffn, pred_rank, dtype, norm, ln_eps, kv_cap,
                     neuron_block, mlp)


def desc_from_config(cfg, kv_cap: Optional[int] = None) -> LayerDesc:
    """LayerDesc from a ``dv_inputs.LayerConfig`` (read by attribute)."""
    cap = cfg.kv_len + 1 if kv_cap is None else kv_cap
    return make_desc(cfg.d_model, cfg.n_heads, cfg.head_dim, cfg.d_ffn, cfg.pred_rank,
                     DV_F32 if cfg.dtype == "f32" else DV_F16, cap,
                     DV_LAYERNORM if cfg.norm == "layernorm" else DV_RMSNORM, cfg.ln_eps,
                     getattr(cfg, "neuron_block", 0),
                     1 if getattr(cfg, "mlp", "relu") == "swiglu" else 0)


class Layer:
    """One layer's device weights plus the C struct pointing at them."""

    def __init__(self, desc: LayerDesc, weights: Dict[str, torch.Tensor]):
        self.desc = desc
        self.weights = {n: weights[n].contiguous() for n in WEIGHT_FIELDS}
        for n, t in self.weights.items():
            if not t.is_cuda:
                raise ValueError(f"weight {n} must be a CUDA tensor")
        self.c = LayerWeights(*[_ptr(self.weights[n]) for n in WEIGHT_FIELDS])


class Workspace:
    """Device workspace sized for (desc, batch), zeroed once."""

    def __init__(self, desc: LayerDesc, batch: int, device=None, stream=None):
        n = workspace_size(desc, batch)
        if n == 0:
            raise DvError("dv_workspace_size", DV_ERR_INVALID_ARG)
        # torch's caching allocator returns 512-byte aligned blocks
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buf.data_ptr()) % 256
        self.ptr = self.buf.data_ptr() + off
        self.nbytes = n
        _check("dv_workspace_init", _lib.dv_workspace_init(C.c_void_p(self.ptr), n,
                                                            _stream(stream)))

    @property
    def cptr(self):
        return C.c_void_p(self.ptr)


class SelectionBuffers:
    """Device buffers for one selection (per-row top-k and unions)."""

    def __init__(self, desc: LayerDesc, batch: int, k_heads: int, k_neurons: int, device=None):
        dev = device or "cuda"
        H, N = desc.n_heads, desc.d_ffn
        self.batch, self.k_heads, self.k_neurons = batch, k_heads, k_neurons
        self.max_u_h = min(H, batch * k_heads)
        self.max_u_n = min(N, batch * k_neurons)
        self.idx_h = torch.empty((batch, k_heads), dtype=torch.int32, device=dev)
        self.idx_n = torch.empty((batch, k_neurons), dtype=torch.int32, device=dev)
        self.u_h = torch.empty(self.max_u_h, dtype=torch.int32, device=dev)
        self.u_n = torch.empty(self.max_u_n, dtype=torch.int32, device=dev)
        self.n_u_h = torch.zeros(1, dtype=torch.int32, device=dev)
        self.n_u_n = torch.zeros(1, dtype=torch.int32, device=dev)
        self.c = Selection(_ptr(self.idx_h), _ptr(self.idx_n), _ptr(self.u_h), _ptr(self.n_u_h),
                           _ptr(self.u_n), _ptr(self.n_u_n))

    def unions(self):
        """(u_h, u_n) trimmed to their device counts (synchronises)."""
        nh, nn = int(self.n_u_h.item()), int(self.n_u_n.item())
        return self.u_h[:nh], self.u_n[:nn]


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI).


def workspace_size(desc: LayerDesc, batch: int) -> int:
    return int(_lib.dv_workspace_size(C.byref(desc), int(batch)))


def dv_set_row_kernel(variant: int) -> None:
    """0: fc1 rows on mma.sync (default); 1: on tcgen05 (binary16, ReLU, B >= 9)."""
    _check("dv_set_row_kernel", _lib.dv_set_row_kernel(int(variant)))


def dv_check(ws: Workspace, stream=None) -> int:
    return int(_lib.dv_check(ws.cptr, ws.nbytes, _stream(stream)))


def dv_layer_decode_launches(desc: LayerDesc, batch: int) -> int:
    return int(_lib.dv_layer_decode_launches(C.byref(desc), int(batch)))


def dv_mlp_one_pass(desc: LayerDesc, batch: int, max_u_n: int) -> bool:
    """The MLP half runs as one pass plus the partials' sum (two kernels)."""
    return bool(_lib.dv_mlp_one_pass(C.byref(desc), int(batch), int(max_u_n)))


def dv_layer_decode_persistent_ok(desc: LayerDesc, batch: int) -> bool:
    return bool(_lib.dv_layer_decode_persistent_ok(C.byref(desc), int(batch)))


def dv_predict_topk(layer: Layer, x_pred: torch.Tensor, k_heads: int, k_neurons: int,
                    sel: SelectionBuffers, ws: Workspace, scores_h: Optional[torch.Tensor] = None,
                    scores_n: Optional[torch.Tensor] = None, stream=None):
    B = x_pred.shape[0]
    _check("dv_predict_topk", _lib.dv_predict_topk(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x_pred), B, k_heads, k_neurons,
        C.byref(sel.c), _ptr(scores_h), _ptr(scores_n), ws.cptr, ws.nbytes, _stream(stream)))


def dv_predict_topk_noalloc(layer: Layer, x_pred: torch.Tensor, k_heads: int, k_neurons: int,
                            sel: SelectionBuffers, scores_h: Optional[torch.Tensor] = None,
                            scores_n: Optional[torch.Tensor] = None, stream=None):
    B = x_pred.shape[0]
    _check("dv_predict_topk_noalloc", _lib.dv_predict_topk_noalloc(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x_pred), B, k_heads, k_neurons,
        C.byref(sel.c), _ptr(scores_h), _ptr(scores_n), _stream(stream)))


def dv_sparse_attn(layer: Layer, x: torch.Tensor, u_h: torch.Tensor, n_u_h: torch.Tensor,
                   k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int, h1: torch.Tensor,
                   ws: Workspace, max_u_h: Optional[int] = None, stream=None):
    B = x.shape[0]
    m = u_h.numel() if max_u_h is None else max_u_h
    _check("dv_sparse_attn", _lib.dv_sparse_attn(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), B, _ptr(u_h), _ptr(n_u_h), m,
        _ptr(k_cache), _ptr(v_cache), kv_len, _ptr(h1), ws.cptr, ws.nbytes, _stream(stream)))


def dv_sparse_mlp(layer: Layer, h1: torch.Tensor, u_n: torch.Tensor, n_u_n: torch.Tensor,
                  y: torch.Tensor, ws: Workspace, max_u_n: Optional[int] = None, stream=None):
    B = h1.shape[0]
    m = u_n.numel() if max_u_n is None else max_u_n
    _check("dv_sparse_mlp", _lib.dv_sparse_mlp(
        C.byref(layer.desc), C.byref(layer.c), _ptr(h1), B, _ptr(u_n), _ptr(n_u_n), m, _ptr(y),
        ws.cptr, ws.nbytes, _stream(stream)))


def dv_layer_decode(layer: Layer, x: torch.Tensor, k_heads: int, k_neurons: int,
                    k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                    sel: SelectionBuffers, y: torch.Tensor, ws: Workspace,
                    x_pred: Optional[torch.Tensor] = None, h1: Optional[torch.Tensor] = None,
                    stream=None):
    B = x.shape[0]
    _check("dv_layer_decode", _lib.dv_layer_decode(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), _ptr(x_pred), B, k_heads, k_neurons,
        _ptr(k_cache), _ptr(v_cache), kv_len, C.byref(sel.c), _ptr(h1), _ptr(y), ws.cptr,
        ws.nbytes, _stream(stream)))


def dv_layer_decode_chained(layer: Layer, x: torch.Tensor, k_heads: int, k_neurons: int,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                            sel: SelectionBuffers, y: torch.Tensor, ws: Workspace,
                            x_pred: Optional[torch.Tensor] = None,
                            h1: Optional[torch.Tensor] = None, stream=None):
    """dv_layer_decode as the seven chained kernels (every shape and batch)."""
    B = x.shape[0]
    _check("dv_layer_decode_chained", _lib.dv_layer_decode_chained(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), _ptr(x_pred), B, k_heads, k_neurons,
        _ptr(k_cache), _ptr(v_cache), kv_len, C.byref(sel.c), _ptr(h1), _ptr(y), ws.cptr,
        ws.nbytes, _stream(stream)))


def dv_layer_decode_stamped(layer: Layer, x: torch.Tensor, k_heads: int, k_neurons: int,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                            sel: SelectionBuffers, y: torch.Tensor, ws: Workspace,
                            stamps: torch.Tensor, x_pred: Optional[torch.Tensor] = None,
                            h1: Optional[torch.Tensor] = None, persistent: bool = False,
                            stream=None):
    """The decode with its timeline in ``stamps`` (int64): [7, SMs, 8] for the
    chain, [SMs, 32] for the persistent streaming kernel."""
    B = x.shape[0]
    _check("dv_layer_decode_stamped", _lib.dv_layer_decode_stamped(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), _ptr(x_pred), B, k_heads, k_neurons,
        _ptr(k_cache), _ptr(v_cache), kv_len, C.byref(sel.c), _ptr(h1), _ptr(y), ws.cptr,
        ws.nbytes, int(bool(persistent)), _ptr(stamps), stamps.numel(), _stream(stream)))


def dv_layer_decode_persistent(layer: Layer, x: torch.Tensor, k_heads: int, k_neurons: int,
                               k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                               sel: SelectionBuffers, y: torch.Tensor, ws: Workspace,
                               x_pred: Optional[torch.Tensor] = None,
                               h1: Optional[torch.Tensor] = None, stream=None):
    """dv_layer_decode through the streaming kernel only (see dv_layer_decode_persistent_ok)."""
    B = x.shape[0]
    _check("dv_layer_decode_persistent", _lib.dv_layer_decode_persistent(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), _ptr(x_pred), B, k_heads, k_neurons,
        _ptr(k_cache), _ptr(v_cache), kv_len, C.byref(sel.c), _ptr(h1), _ptr(y), ws.cptr,
        ws.nbytes, _stream(stream)))


def dv_layer_decode_presel(layer: Layer, x: torch.Tensor, sel: SelectionBuffers,
                           k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                           y: torch.Tensor, ws: Workspace, h1: Optional[torch.Tensor] = None,
                           stream=None):
    """Layer decode on the unions already in ``sel`` (e.g. from a lookahead predictor)."""
    B = x.shape[0]
    _check("dv_layer_decode_presel", _lib.dv_layer_decode_presel(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), B, _ptr(sel.u_h), _ptr(sel.n_u_h),
        sel.max_u_h, _ptr(sel.u_n), _ptr(sel.n_u_n), sel.max_u_n, _ptr(k_cache), _ptr(v_cache),
        kv_len, _ptr(h1), _ptr(y), ws.cptr, ws.nbytes, _stream(stream)))


def dv_layer_decode_traced(layer: Layer, x: torch.Tensor, k_heads: int, k_neurons: int,
                           k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                           sel: SelectionBuffers, y: torch.Tensor, ws: Workspace,
                           events: Sequence[torch.cuda.Event],
                           x_pred: Optional[torch.Tensor] = None,
                           h1: Optional[torch.Tensor] = None, stream=None):
    B = x.shape[0]
    s = stream if stream is not None else torch.cuda.current_stream()
    for e in events:  # torch creates the CUDA event on its first record
        if e.cuda_event == 0:
            e.record(s)
    arr = (C.c_void_p * len(events))(*[C.c_void_p(e.cuda_event) for e in events])
    _check("dv_layer_decode_traced", _lib.dv_layer_decode_traced(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x), _ptr(x_pred), B, k_heads, k_neurons,
        _ptr(k_cache), _ptr(v_cache), kv_len, C.byref(sel.c), _ptr(h1), _ptr(y), ws.cptr,
        ws.nbytes, arr, len(events), _stream(stream)))


def dv_layer_decode_host(layer: Layer, x_host: torch.Tensor, k_heads: int, k_neurons: int,
                         k_cache: torch.Tensor, v_cache: torch.Tensor, kv_len: int,
                         y_host: torch.Tensor, ws: Workspace,
                         sel: Optional[SelectionBuffers] = None,
                         x_pred_host: Optional[torch.Tensor] = None, stream=None):
    """Host activations in and out (pinned CPU tensors give async copies); synchronous."""
    for t in (x_host, y_host) + ((x_pred_host,) if x_pred_host is not None else ()):
        if t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError("host activations must be contiguous float32 CPU tensors")
    B = x_host.shape[0]
    _check("dv_layer_decode_host", _lib.dv_layer_decode_host(
        C.byref(layer.desc), C.byref(layer.c), _ptr(x_host), _ptr(x_pred_host), B, k_heads,
        k_neurons, _ptr(k_cache), _ptr(v_cache), kv_len,
        C.byref(sel.c) if sel is not None else None, _ptr(y_host), ws.cptr, ws.nbytes,
        _stream(stream)))


def dv_test_hold_wait(ws: Workspace, wait_id: int, budget_us: int, stream=None):
    """Test support: make the next streaming decode's wait `wait_id` run out."""
    _check("dv_test_hold_wait", _lib.dv_test_hold_wait(ws.cptr, ws.nbytes, int(wait_id),
                                                        int(budget_us), _stream(stream)))


def dv_hbm_copy(dst: torch.Tensor, src: torch.Tensor, nbytes: Optional[int] = None, stream=None):
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    _check("dv_hbm_copy", _lib.dv_hbm_copy(_ptr(dst), _ptr(src), n, _stream(stream)))


# ---------------------------------------------------------------------------
# KV-cache operators.


_TORCH_DTYPE = {DV_F32: torch.float32, DV_F16: torch.float16, DV_I8: torch.int8}
_ROW_DTYPE = {torch.float32: DV_F32, torch.float16: DV_F16}


def make_kv_desc(n_heads, n_kv_heads, head_dim, kv_cap, dtype, block=0) -> KvDesc:
    return KvDesc(n_heads, n_kv_heads, head_dim, kv_cap, dtype, block)


def kv_workspace_size(desc: KvDesc, batch: int, tokens: int = 1) -> int:
    return int(_lib.dv_kv_workspace_size(C.byref(desc), int(batch), int(tokens)))


def _kv_tensors(desc: KvDesc, batch: int):
    """Shape and type of each of a cache's tensors."""
    B, H, cap, D = batch, desc.n_kv_heads, desc.kv_cap, desc.head_dim
    t = {n: ((B, H, cap, D), _TORCH_DTYPE[desc.dtype]) for n in ("k", "v")}
    if desc.dtype == DV_I8:
        t.update({n: ((B, H, cap), torch.float32) for n in ("k_scale", "v_scale")})
    if desc.block:
        nb = cap // desc.block
        t["k_mean"] = ((B, H, nb, D), torch.int8)
        t["k_mean_scale"] = ((B, H, nb), torch.float32)
    return t


def _raw_stream(device_index: int) -> int:
    """The current stream's handle (without a Stream object around it, where torch offers that)."""
    return torch.cuda.current_stream(device_index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


class KvCache:
    """The tensors of one KV cache (attributes ``k``, ``v``, and where the
    descriptor has them ``k_scale``, ``v_scale``, ``k_mean``,
    ``k_mean_scale``) plus the C struct pointing at them.  ``tensors``: use
    these instead of allocating (zeroed) ones."""

    def __init__(self, desc: KvDesc, batch: int, device=None,
                 tensors: Optional[Dict[str, torch.Tensor]] = None):
        if kv_workspace_size(desc, batch) == 0:
            raise DvError("dv_kv_workspace_size", DV_ERR_INVALID_ARG)
        self.desc, self.batch = desc, batch
        want = _kv_tensors(desc, batch)
        if tensors is None:
            dev = device or "cuda"
            tensors = {n: torch.zeros(shape, dtype=dt, device=dev)
                       for n, (shape, dt) in want.items()}
        if set(tensors) != set(want):
            raise ValueError(f"this cache has the tensors {sorted(want)}, got {sorted(tensors)}")
        self.device = tensors["k"].device
        self.device_index = tensors["k"].get_device()
        for n, (shape, dt) in want.items():
            t = tensors[n]
            if (tuple(t.shape) != shape or t.dtype != dt or not t.is_cuda
                    or not t.is_contiguous() or t.device != self.device):
                raise ValueError(f"cache tensor {n} must be a contiguous CUDA tensor {shape} of "
                                 f"{dt} on one device")
            setattr(self, n, t)
        self.c = KvCachePointers(*[_ptr(getattr(self, n, None)) if n in want else None
                                   for n, _ in KvCachePointers._fields_])
        self._refs = (C.byref(self.desc), C.byref(self.c))


class KvWorkspace(Workspace):
    """Device workspace of the KV-cache operators, zeroed once: for caches of
    ``desc`` with up to ``tokens`` query tokens a row."""

    def __init__(self, desc: KvDesc, batch: int, tokens: int = 1, device=None, stream=None):
        n = kv_workspace_size(desc, batch, tokens)
        if n == 0:
            raise DvError("dv_kv_workspace_size", DV_ERR_INVALID_ARG)
        self.buf = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        self.device = self.buf.device
        self.device_index = self.buf.get_device()
        off = (-self.buf.data_ptr()) % 256
        self.ptr = self.buf.data_ptr() + off
        self.nbytes = n
        with torch.cuda.device(self.device):
            _check("dv_workspace_init", _lib.dv_workspace_init(C.c_void_p(self.ptr), n,
                                                                _stream(stream)))


def _kv_dev(cache: KvCache, ws: KvWorkspace, stream):
    """The stream of a call; its device must be the cache's and the current one."""
    dev = cache.device_index
    if ws.device_index != dev:
        raise ValueError("the workspace is not on the cache's device")
    if torch.cuda.current_device() != dev:
        raise ValueError("the cache is not on the current device (torch.cuda.device)")
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError("the stream is not of the cache's device")
    return stream.cuda_stream


def _kv_dim(name: str, t: torch.Tensor, ndim: int, dim: int) -> int:
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    return t.shape[dim]


def _kv_tensor(name: str, t: Optional[torch.Tensor], cache: KvCache, shape, dtype):
    if t is None:
        return None
    if (t.dtype != dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != cache.device_index):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on the "
                         "cache's device")
    return t.data_ptr()


def _kv_rows(name: str, t: torch.Tensor, cache: KvCache, shape) -> KvRows:
    dt = _ROW_DTYPE.get(t.dtype)
    s = t.stride()
    if (dt is None or t.shape != shape or t.get_device() != cache.device_index
            or (s[-1] != 1 and shape[-1] != 1)):
        raise ValueError(f"{name} must be a float32 or float16 tensor {shape} on the "
                         "cache's device, contiguous in its last dimension")
    # (a dimension of one row is never stepped over: its stride says nothing)
    if len(shape) == 4:
        return KvRows(t.data_ptr(), dt, s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0,
                      s[2] if shape[2] > 1 else 0)
    return KvRows(t.data_ptr(), dt, s[0] if shape[0] > 1 else 0, 0, s[1] if shape[1] > 1 else 0)


def dv_kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, lens: torch.Tensor,
                 ws: KvWorkspace, n_tok: Optional[torch.Tensor] = None, stream=None):
    """Write k, v [B, T, Hkv, D] (any strides over the first three) at positions lens[b] + t."""
    d, B, T = cache.desc, cache.batch, _kv_dim("k", k, 4, 1)
    st = _kv_dev(cache, ws, stream)
    shape = (B, T, d.n_kv_heads, d.head_dim)
    _check("dv_kv_append", _lib.dv_kv_append(
        *cache._refs, C.byref(_kv_rows("k", k, cache, shape)),
        C.byref(_kv_rows("v", v, cache, shape)), B, T,
        _kv_tensor("lens", lens, cache, (B,), torch.int32),
        _kv_tensor("n_tok", n_tok, cache, (B,), torch.int32), ws.ptr, ws.nbytes, st))


def dv_kv_read(cache: KvCache, start: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
               ws: KvWorkspace, stream=None):
    """Positions start[b] .. start[b] + T - 1 into k_out, v_out [B, Hkv, T, D] (float32/float16)."""
    d, B, T = cache.desc, cache.batch, _kv_dim("k_out", k_out, 4, 2)
    st = _kv_dev(cache, ws, stream)
    if k_out.dtype not in _ROW_DTYPE:
        raise ValueError("k_out must be float32 or float16")
    shape = (B, d.n_kv_heads, T, d.head_dim)
    _check("dv_kv_read", _lib.dv_kv_read(
        *cache._refs, B, T, _kv_tensor("start", start, cache, (B,), torch.int32),
        _ROW_DTYPE[k_out.dtype], _kv_tensor("k_out", k_out, cache, shape, k_out.dtype),
        _kv_tensor("v_out", v_out, cache, shape, k_out.dtype), ws.ptr, ws.nbytes, st))


def dv_kv_keep(cache: KvCache, lens: torch.Tensor, path: torch.Tensor, n_keep: torch.Tensor,
               ws: KvWorkspace, stream=None):
    """Move position lens[b] + path[b, i] to lens[b] + i for i < n_keep[b] (path [B, T] ascending)."""
    B, T = cache.batch, _kv_dim("path", path, 2, 1)
    st = _kv_dev(cache, ws, stream)
    _check("dv_kv_keep", _lib.dv_kv_keep(
        *cache._refs, B, T, _kv_tensor("lens", lens, cache, (B,), torch.int32),
        _kv_tensor("path", path, cache, (B, T), torch.int32),
        _kv_tensor("n_keep", n_keep, cache, (B,), torch.int32), ws.ptr, ws.nbytes, st))


def dv_tree_attn(cache: KvCache, q: torch.Tensor, lens: torch.Tensor, out: torch.Tensor,
                 ws: KvWorkspace, mask: Optional[torch.Tensor] = None,
                 n_tok: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                 u_h: Optional[torch.Tensor] = None, n_u_h: Optional[torch.Tensor] = None,
                 stream=None):
    """Attention of q [B, T, H, D] over the cache; mask [B, T] int64 (bit j: sees drafted token j).

    scale: head_dim ** -0.5 by default.  u_h, n_u_h: a device list of KV heads and its length."""
    d, B, T = cache.desc, cache.batch, _kv_dim("q", q, 4, 1)
    st = _kv_dev(cache, ws, stream)
    shape = (B, T, d.n_heads, d.head_dim)
    if (u_h is None) != (n_u_h is None):
        raise ValueError("u_h and n_u_h go together")
    m = 0 if u_h is None else u_h.numel()
    _check("dv_tree_attn", _lib.dv_tree_attn(
        *cache._refs, C.byref(_kv_rows("q", q, cache, shape)), B, T,
        _kv_tensor("lens", lens, cache, (B,), torch.int32),
        _kv_tensor("n_tok", n_tok, cache, (B,), torch.int32),
        _kv_tensor("mask", mask, cache, (B, T), torch.int64),
        d.head_dim ** -0.5 if scale is None else scale,
        _kv_tensor("u_h", u_h, cache, (m,), torch.int32),
        _kv_tensor("n_u_h", n_u_h, cache, (1,), torch.int32), m,
        _kv_tensor("out", out, cache, shape, torch.float32), ws.ptr, ws.nbytes, st))


def dv_set_tree_kernel(variant: int) -> None:
    """dv_tree_attn above 8 query rows a KV head: 0 by rule, 1 mma.sync, 2 tcgen05."""
    _check("dv_set_tree_kernel", _lib.dv_set_tree_kernel(int(variant)))


def dv_block_topk(cache: KvCache, q: torch.Tensor, lens: torch.Tensor, idx: torch.Tensor,
                  ws: KvWorkspace, n_first: int = 1, n_last: int = 1, stream=None):
    """The idx.shape[2] blocks each query of q [B, H, D] attends to, into idx [B, H, k] (-1 behind)."""
    d, B, k = cache.desc, cache.batch, _kv_dim("idx", idx, 3, 2)
    st = _kv_dev(cache, ws, stream)
    _check("dv_block_topk", _lib.dv_block_topk(
        *cache._refs, C.byref(_kv_rows("q", q, cache, (B, d.n_heads, d.head_dim))), B,
        _kv_tensor("lens", lens, cache, (B,), torch.int32), k, n_first, n_last,
        _kv_tensor("idx", idx, cache, (B, d.n_heads, k), torch.int32), ws.ptr, ws.nbytes, st))


def dv_block_attn(cache: KvCache, q: torch.Tensor, lens: torch.Tensor, idx: torch.Tensor,
                  out: torch.Tensor, ws: KvWorkspace, scale: Optional[float] = None, stream=None):
    """Attention of q [B, H, D] over the blocks listed in idx [B, H, k], into out [B, H, D]."""
    d, B, k = cache.desc, cache.batch, _kv_dim("idx", idx, 3, 2)
    st = _kv_dev(cache, ws, stream)
    shape = (B, d.n_heads, d.head_dim)
    _check("dv_block_attn", _lib.dv_block_attn(
        *cache._refs, C.byref(_kv_rows("q", q, cache, shape)), B,
        _kv_tensor("lens", lens, cache, (B,), torch.int32),
        _kv_tensor("idx", idx, cache, (B, d.n_heads, k), torch.int32), k,
        d.head_dim ** -0.5 if scale is None else scale,
        _kv_tensor("out", out, cache, shape, torch.float32), ws.ptr, ws.nbytes, st))
