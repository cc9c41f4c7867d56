"""Python binding of libpi_ffn.so: activation-sparse FFN decode on one GB300 (sm_103a).

Argument marshalling only. Every step of the path runs in the CUDA kernels of
libpi_ffn.so (built in-tree by ``_build.py``); there is no CPU or PyTorch
fallback, and importing this package fails if the library has not been built.

The raw C-ABI calls keep their names (``pi_ffn_create``, ``pi_predict``,
``pi_sparse_ffn``, ``pi_decode_stack``, ``pi_hot_first_order``,
``pi_permute_rows``, ``pi_get_status``, ...) and take device pointers (ints)
or CUDA torch tensors. ``SparseFFN`` wraps a handle for torch users.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpi_ffn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python activation_sparse_decode_pi_gb300/_build.py` "
        "(or __graft_entry__.build()); there is no fallback path")

_lib = ctypes.CDLL(LIB_PATH)

PI_OK, PI_ERR_INVALID_ARG, PI_ERR_UNSUPPORTED, PI_ERR_CUDA, PI_ERR_OOM, PI_ERR_TIMEOUT, PI_ERR_DEVICE_CHECK = range(7)
PI_FFN_GATED_RELU, PI_FFN_RELU = 0, 1
PI_F32, PI_BF16, PI_F16, PI_INT4_G128 = 0, 1, 2, 3
DTYPES = {"f32": PI_F32, "bf16": PI_BF16, "f16": PI_F16, "int4g128": PI_INT4_G128}
KINDS = {"gated": PI_FFN_GATED_RELU, "relu": PI_FFN_RELU}

# every symbol include/pi_ffn.h and include/pi_kv.h declare
EXPORTS = (
    "pi_ffn_create", "pi_ffn_destroy", "pi_predict", "pi_sparse_ffn", "pi_decode_stack",
    "pi_hot_first_order", "pi_permute_rows", "pi_get_status", "pi_status_string", "pi_abi_version",
    "pi_profile_begin", "pi_profile_end", "pi_sparse_ffn_noalloc", "pi_selftest_grid_barrier",
    "pi_selftest_umma", "pi_ffn_set_hot_neurons", "pi_ffn_set_hot_prefix", "pi_decode_stack_layers",
    "pi_ffn_set_phase_trace",
    "pi_kv_create", "pi_kv_destroy", "pi_kv_get_status", "pi_kv_reserve", "pi_kv_append", "pi_kv_attend",
    "pi_kv_fork", "pi_kv_free", "pi_kv_trim", "pi_kv_copy_pages", "pi_kv_compact",
)
PI_STACK_PHASES = 8
STACK_PHASE_NAMES = ("layer_start", "hidden_done", "logits_start", "list_ready", "first_rows", "ffn_done",
                     "reduce_start", "reduce_done")
PI_NOALLOC_SCRATCH_BYTES = 16 << 20
KERNEL_KINDS = ("rms", "pred_hidden", "pred_logits", "ffn_h", "ffn_down", "reduce", "decode_stack", "pred_fused")


class PiFfnDesc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("f", ctypes.c_int32), ("r", ctypes.c_int32),
                ("n_layers", ctypes.c_int32), ("max_batch", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("pdtype", ctypes.c_int32), ("tau_logit", ctypes.c_float)]


class PiLayerWeights(ctypes.Structure):
    _fields_ = [("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down_t", ctypes.c_void_p),
                ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
                ("b_gate", ctypes.c_void_p), ("p1_t", ctypes.c_void_p), ("p2_t", ctypes.c_void_p),
                ("b_pred", ctypes.c_void_p)]


class PiKvDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class PiKvLayer(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class PiKvState(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("length", ctypes.c_void_p), ("ref", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_lib.pi_ffn_create.restype = ctypes.c_int
_lib.pi_ffn_create.argtypes = [ctypes.POINTER(_P), ctypes.POINTER(PiFfnDesc), ctypes.POINTER(PiLayerWeights)]
_lib.pi_ffn_destroy.restype = None
_lib.pi_ffn_destroy.argtypes = [_P]
_lib.pi_predict.restype = ctypes.c_int
_lib.pi_predict.argtypes = [_P, _I32, _P, _I32, _P, _P, _P]
_lib.pi_sparse_ffn.restype = ctypes.c_int
_lib.pi_sparse_ffn.argtypes = [_P, _I32, _P, _I32, _P, _P, _P, _P]
_lib.pi_decode_stack.restype = ctypes.c_int
_lib.pi_decode_stack.argtypes = [_P, _P, _I32, _P, _P, _P, _P]
_lib.pi_decode_stack_layers.restype = ctypes.c_int
_lib.pi_decode_stack_layers.argtypes = [_P, _P, _I32, _P, _P, _P, _P, _P]
_lib.pi_ffn_set_phase_trace.restype = ctypes.c_int
_lib.pi_ffn_set_phase_trace.argtypes = [_P, _P, _I64]
_lib.pi_hot_first_order.restype = ctypes.c_int
_lib.pi_hot_first_order.argtypes = [_P, _I32, _P, _P]
_lib.pi_permute_rows.restype = ctypes.c_int
_lib.pi_permute_rows.argtypes = [_P, _P, _P, _I64, _I64, _P, _P]
_lib.pi_get_status.restype = ctypes.c_int
_lib.pi_get_status.argtypes = [_P]
_lib.pi_status_string.restype = ctypes.c_char_p
_lib.pi_status_string.argtypes = [ctypes.c_int]
_lib.pi_abi_version.restype = _I32
_lib.pi_abi_version.argtypes = []
_lib.pi_sparse_ffn_noalloc.restype = ctypes.c_int
_lib.pi_sparse_ffn_noalloc.argtypes = [ctypes.POINTER(PiFfnDesc), ctypes.POINTER(PiLayerWeights), _P, _I32, _P, _P,
                                       _P, _P, _P]
_lib.pi_selftest_grid_barrier.restype = ctypes.c_int
_lib.pi_selftest_grid_barrier.argtypes = [_P, _I32, _P]
_lib.pi_ffn_set_hot_prefix.restype = ctypes.c_int
_lib.pi_ffn_set_hot_prefix.argtypes = [_P, _I32]
_lib.pi_ffn_set_hot_neurons.restype = ctypes.c_int
_lib.pi_ffn_set_hot_neurons.argtypes = [_P, _I32]
_lib.pi_selftest_umma.restype = ctypes.c_int
_lib.pi_selftest_umma.argtypes = [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P]
_lib.pi_profile_begin.restype = ctypes.c_int
_lib.pi_profile_begin.argtypes = [_P]
_lib.pi_profile_end.restype = ctypes.c_int
_lib.pi_profile_end.argtypes = [_P, _P, _P, _I32]
_F32 = ctypes.c_float
for _name, _args in {
    "pi_kv_create": [ctypes.POINTER(_P), ctypes.POINTER(PiKvDesc), ctypes.POINTER(PiKvLayer),
                     ctypes.POINTER(PiKvState)],
    "pi_kv_get_status": [_P],
    "pi_kv_reserve": [_P, _P, _P, _I32, _P],
    "pi_kv_append": [_P, _I32, _P, _P, _I32, _I32, _P, _P, _I64, _I32, _P],
    "pi_kv_attend": [_P, _I32, _P, _P, _I32, _I32, _P, _I64, _P, _I64, _P, _I32, _F32, _I32, _I32, _P],
    "pi_kv_fork": [_P, _P, _P, _I32, _P],
    "pi_kv_free": [_P, _P, _I32, _P],
    "pi_kv_trim": [_P, _P, _I32, _I32, _I32, _P],
    "pi_kv_copy_pages": [_P, _P, _P, _I32, _P],
    "pi_kv_compact": [_P, _P, _P],
}.items():
    getattr(_lib, _name).restype = ctypes.c_int
    getattr(_lib, _name).argtypes = _args
_lib.pi_kv_destroy.restype = None
_lib.pi_kv_destroy.argtypes = [_P]


class PiError(RuntimeError):
    def __init__(self, code: int, call: str):
        self.code = code
        super().__init__(f"{call}: {pi_status_string(code)} ({code})")


def pi_status_string(code: int) -> str:
    return _lib.pi_status_string(code).decode()


def pi_abi_version() -> int:
    return _lib.pi_abi_version()


def _ptr(x):
    """Device pointer of a CUDA tensor, an int, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None   # the current CUDA stream's handle, without building a torch.cuda.Stream


def _stream(s):
    if s is None:
        global _current_stream
        if _current_stream is None:
            import torch

            torch.cuda.current_stream()   # initialises CUDA
            raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            _current_stream = lambda: raw(device())
        return _current_stream()
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(code: int, call: str):
    if code != PI_OK:
        raise PiError(code, call)


def pi_ffn_create(desc: PiFfnDesc, layers) -> int:
    arr = (PiLayerWeights * len(layers))(*layers)
    h = _P()
    _check(_lib.pi_ffn_create(ctypes.byref(h), ctypes.byref(desc), arr), "pi_ffn_create")
    return h.value


def pi_ffn_destroy(h: int) -> None:
    _lib.pi_ffn_destroy(h)


def pi_predict(h, layer, u, B, idx, count, stream=None) -> None:
    _check(_lib.pi_predict(h, layer, _ptr(u), B, _ptr(idx), _ptr(count), _stream(stream)), "pi_predict")


def pi_sparse_ffn(h, layer, u, B, idx, count, y, stream=None) -> None:
    _check(_lib.pi_sparse_ffn(h, layer, _ptr(u), B, _ptr(idx), _ptr(count), _ptr(y), _stream(stream)),
           "pi_sparse_ffn")


def pi_decode_stack(h, x0, B, x_out, counts=None, idx_out=None, stream=None) -> None:
    _check(_lib.pi_decode_stack(h, _ptr(x0), B, _ptr(x_out), _ptr(counts), _ptr(idx_out), _stream(stream)),
           "pi_decode_stack")


def pi_decode_stack_layers(h, x0, B, x_out, counts, idx_out, x_layers, stream=None) -> None:
    _check(_lib.pi_decode_stack_layers(h, _ptr(x0), B, _ptr(x_out), _ptr(counts), _ptr(idx_out), _ptr(x_layers),
                                       _stream(stream)), "pi_decode_stack_layers")


def pi_ffn_set_phase_trace(h, stamps, n_stamps=0) -> None:
    _check(_lib.pi_ffn_set_phase_trace(h, _ptr(stamps), n_stamps), "pi_ffn_set_phase_trace")


def pi_sparse_ffn_noalloc(desc, layer, u, B, idx, count, y, status=None, stream=None) -> None:
    """pi_sparse_ffn without a handle and without any device allocation (static library scratch)."""
    _check(_lib.pi_sparse_ffn_noalloc(ctypes.byref(desc), ctypes.byref(layer), _ptr(u), B, _ptr(idx), _ptr(count),
                                      _ptr(y), _ptr(status), _stream(stream)), "pi_sparse_ffn_noalloc")


def pi_selftest_grid_barrier(work, extra, stream=None) -> None:
    _check(_lib.pi_selftest_grid_barrier(_ptr(work), extra, _stream(stream)), "pi_selftest_grid_barrier")


def pi_ffn_set_hot_prefix(h, hot_prefix) -> None:
    _check(_lib.pi_ffn_set_hot_prefix(h, hot_prefix), "pi_ffn_set_hot_prefix")


def pi_ffn_set_hot_neurons(h, n_hot) -> None:
    _check(_lib.pi_ffn_set_hot_neurons(h, n_hot), "pi_ffn_set_hot_neurons")


def pi_selftest_umma(a, b, d, mode, n, k, dtype, status, stream=None) -> None:
    _check(_lib.pi_selftest_umma(_ptr(a), _ptr(b), _ptr(d), mode, n, k, dtype, _ptr(status), _stream(stream)),
           "pi_selftest_umma")


def pi_hot_first_order(counts, f, perm, stream=None) -> None:
    _check(_lib.pi_hot_first_order(_ptr(counts), f, _ptr(perm), _stream(stream)), "pi_hot_first_order")


def pi_permute_rows(src, dst, perm, rows, row_bytes, err=None, stream=None) -> None:
    _check(_lib.pi_permute_rows(_ptr(src), _ptr(dst), _ptr(perm), rows, row_bytes, _ptr(err), _stream(stream)),
           "pi_permute_rows")


def pi_get_status(h) -> int:
    return _lib.pi_get_status(h)


def pi_profile_begin(h) -> None:
    _check(_lib.pi_profile_begin(h), "pi_profile_begin")


def pi_profile_end(h) -> dict:
    """{kernel kind: (total ms, launches)} since pi_profile_begin."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int32 * n)()
    _check(_lib.pi_profile_end(h, ms, cnt, n), "pi_profile_end")
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}


def pi_kv_create(desc: PiKvDesc, layers, state: PiKvState) -> int:
    arr = (PiKvLayer * len(layers))(*layers)
    h = _P()
    _check(_lib.pi_kv_create(ctypes.byref(h), ctypes.byref(desc), arr, ctypes.byref(state)), "pi_kv_create")
    return h.value


def pi_kv_destroy(h: int) -> None:
    _lib.pi_kv_destroy(h)


def pi_kv_get_status(h) -> int:
    return _lib.pi_kv_get_status(h)


def pi_kv_reserve(h, seqs, tok_start, n, stream=None) -> None:
    _check(_lib.pi_kv_reserve(h, _ptr(seqs), _ptr(tok_start), n, _stream(stream)), "pi_kv_reserve")


def pi_kv_append(h, layer, seqs, tok_start, n, n_tokens, k_new, v_new, ld, dtype, stream=None) -> None:
    _check(_lib.pi_kv_append(h, layer, _ptr(seqs), _ptr(tok_start), n, n_tokens, _ptr(k_new), _ptr(v_new), ld, dtype,
                             _stream(stream)), "pi_kv_append")


def pi_kv_attend(h, layer, seqs, tok_start, n, n_tokens, q, ld_q, out, ld_out, lse, dtype, scale, window=0, sinks=0,
                 stream=None) -> None:
    _check(_lib.pi_kv_attend(h, layer, _ptr(seqs), _ptr(tok_start), n, n_tokens, _ptr(q), ld_q, _ptr(out), ld_out,
                             _ptr(lse), dtype, scale, window, sinks, _stream(stream)), "pi_kv_attend")


def pi_kv_fork(h, src, dst, n, stream=None) -> None:
    _check(_lib.pi_kv_fork(h, _ptr(src), _ptr(dst), n, _stream(stream)), "pi_kv_fork")


def pi_kv_free(h, seqs, n, stream=None) -> None:
    _check(_lib.pi_kv_free(h, _ptr(seqs), n, _stream(stream)), "pi_kv_free")


def pi_kv_trim(h, seqs, n, window, sinks=0, stream=None) -> None:
    _check(_lib.pi_kv_trim(h, _ptr(seqs), n, window, sinks, _stream(stream)), "pi_kv_trim")


def pi_kv_copy_pages(h, src, dst, n, stream=None) -> None:
    _check(_lib.pi_kv_copy_pages(h, _ptr(src), _ptr(dst), n, _stream(stream)), "pi_kv_copy_pages")


def pi_kv_compact(h, n_live=None, stream=None) -> None:
    _check(_lib.pi_kv_compact(h, _ptr(n_live), _stream(stream)), "pi_kv_compact")


# ------------------------------------------------------------------------------------------------
# torch conveniences (still only marshalling: each call is one C-ABI call)
# ------------------------------------------------------------------------------------------------

PER_NEURON = ("w_gate", "w_up", "w_down_t", "s_gate", "s_up", "s_down", "b_gate", "p2_t", "b_pred", "counts", "p")


def hot_first_order(counts):
    """perm (int32, device) for a CUDA tensor of per-neuron activation counts."""
    import torch

    c = counts.to(torch.int32).contiguous()
    perm = torch.empty_like(c)
    pi_hot_first_order(c, c.numel(), perm)
    return perm


def permute_rows(src, perm):
    """dst[k] = src[perm[k]] for a CUDA tensor (rows along dim 0)."""
    import torch

    s = src.contiguous()
    dst = torch.empty_like(s)
    rows = s.shape[0]
    row_bytes = s.numel() * s.element_size() // max(rows, 1)
    pi_permute_rows(s, dst, perm, rows, row_bytes)
    return dst


def apply_hot_first(layer: dict) -> tuple[dict, object]:
    """Offline hot-first reorder of one layer (every per-neuron array) by its profiling counts."""
    perm = hot_first_order(layer["counts"])
    out = dict(layer)
    for k in PER_NEURON:
        v = layer.get(k)
        if v is not None and hasattr(v, "is_cuda") and v.is_cuda:
            out[k] = permute_rows(v, perm)
    return out, perm


def layer_weights(layer: dict) -> PiLayerWeights:
    g = lambda k: _ptr(layer.get(k))
    return PiLayerWeights(g("w_gate"), g("w_up"), g("w_down_t"), g("s_gate"), g("s_up"), g("s_down"),
                          g("b_gate"), g("p1_t"), g("p2_t"), g("b_pred"))


class SparseFFN:
    """A pi_ffn handle over CUDA tensors (kept referenced for the handle's lifetime)."""

    def __init__(self, layers, *, d, f, r, kind, wdtype, pdtype, max_batch=1, tau=0.0):
        self.layers = list(layers)
        self.desc = PiFfnDesc(d, f, r, len(self.layers), max_batch, KINDS[kind], DTYPES[wdtype], DTYPES[pdtype],
                              tau)
        self.h = pi_ffn_create(self.desc, [layer_weights(L) for L in self.layers])

    @classmethod
    def from_workload(cls, w, layers, max_batch=1, tau=0.0):
        return cls(layers, d=w.d, f=w.f, r=w.r, kind=w.kind, wdtype=w.wdtype, pdtype=w.pdtype,
                   max_batch=max_batch, tau=tau)

    def predict(self, layer, u, idx=None, count=None, stream=None):
        import torch

        B = u.shape[0]
        idx = torch.empty(self.desc.f, dtype=torch.int32, device=u.device) if idx is None else idx
        count = torch.empty(1, dtype=torch.int32, device=u.device) if count is None else count
        pi_predict(self.h, layer, u, B, idx, count, stream)
        return idx, count

    def sparse_ffn(self, layer, u, idx, count, y=None, stream=None):
        import torch

        y = torch.empty_like(u) if y is None else y
        pi_sparse_ffn(self.h, layer, u, u.shape[0], idx, count, y, stream)
        return y

    def decode_stack(self, x0, x_out=None, counts=None, idx_out=None, stream=None):
        import torch

        x_out = torch.empty_like(x0) if x_out is None else x_out
        pi_decode_stack(self.h, x0, x0.shape[0], x_out, counts, idx_out, stream)
        return x_out

    def decode_stack_layers(self, x0, counts=None, idx_out=None, stream=None):
        """(x_out, x_layers): one decode step, and every layer's output (row l = x_{l+1})."""
        import torch

        B = x0.shape[0]
        x_out = torch.empty_like(x0)
        x_layers = torch.empty((self.desc.n_layers, B, self.desc.d), dtype=torch.float32, device=x0.device)
        pi_decode_stack_layers(self.h, x0, B, x_out, counts, idx_out, x_layers, stream)
        return x_out, x_layers

    def set_phase_trace(self, stamps) -> None:
        """Phase stamps of the persistent step into `stamps` (int64 CUDA tensor
        [n_layers, PI_STACK_PHASES, n_sm]); None turns them off."""
        pi_ffn_set_phase_trace(self.h, stamps, 0 if stamps is None else stamps.numel())

    def set_hot_neurons(self, n_hot: int) -> None:
        pi_ffn_set_hot_neurons(self.h, n_hot)

    def set_hot_prefix(self, hot_prefix: int) -> None:
        pi_ffn_set_hot_prefix(self.h, hot_prefix)

    def status(self) -> int:
        return pi_get_status(self.h)

    def close(self):
        if self.h:
            pi_ffn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_TORCH_DTYPES = None


def _act_dtype(x) -> int:
    """pi_dtype_t of an activation tensor."""
    global _TORCH_DTYPES
    if _TORCH_DTYPES is None:
        import torch

        _TORCH_DTYPES = {torch.float32: PI_F32, torch.bfloat16: PI_BF16, torch.float16: PI_F16}
    try:
        return _TORCH_DTYPES[x.dtype]
    except KeyError:
        raise PiError(PI_ERR_UNSUPPORTED, f"dtype {x.dtype}") from None


_INT32 = None


def _i32(x, name, n=None):
    """A call's index tensor: int32, contiguous, on the GPU (its values are checked by the kernels). Its address."""
    global _INT32
    if _INT32 is None:
        import torch

        _INT32 = torch.int32
    shape = x.shape
    if x.dtype is not _INT32 or len(shape) != 1 or not x.is_cuda or (shape[0] > 1 and x.stride(0) != 1):
        raise ValueError(f"{name}: a contiguous 1-D int32 CUDA tensor")
    if n is not None and shape[0] != n:
        raise ValueError(f"{name}: {n} entries, got {shape[0]}")
    return x.data_ptr()


def _token_rows(x, heads, dim, name):
    """Row stride of a [tokens, heads, dim] tensor whose rows lie [heads, dim] contiguous (a slice of a fused
    projection is fine)."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or not x.is_cuda:
        raise ValueError(f"{name}: a [tokens, {heads}, {dim}] CUDA tensor, got {tuple(shape)}")
    row, head, one = x.stride()
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{name}: the heads of a token lie next to each other")
    return row if shape[0] > 1 else heads * dim


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to `stream` (a torch stream or a handle; None: the current one), so that memory which
    work on another stream may still use is not taken for it."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class KVCache:
    """A pi_kv handle over CUDA tensors (kept referenced for the handle's lifetime): a paged e4m3 key/value cache.

    layers: per layer a dict of ``k``, ``v`` (float8_e4m3fn [pages, kv heads, page tokens, dim]) and ``k_scale``,
    ``v_scale`` (fp32 [pages, kv heads]); table (int32 [sequences, columns], -1 for no page), length (int32
    [sequences]), ref (int32 [pages]). ``KVCache.empty`` makes them. A step is one ``reserve``, then per layer
    ``append`` and ``attend``; ``seqs`` names the call's sequences and ``tok_start`` where each one's new tokens
    begin in the call's token arrays (one entry more than seqs).
    """

    def __init__(self, layers, table, length, ref, *, n_heads):
        import torch

        self.layers, self.table, self.length, self.ref = list(layers), table, length, ref
        k = self.layers[0]["k"]
        n_pages, kv_heads, page, dim = k.shape
        for L in self.layers:
            for name in ("k", "v"):
                if L[name].dtype is not torch.float8_e4m3fn or L[name].shape != k.shape or not L[name].is_contiguous():
                    raise ValueError(f"{name}: contiguous float8_e4m3fn of one shape for all layers")
            for name in ("k_scale", "v_scale"):
                x = L[name]
                if x.dtype is not torch.float32 or tuple(x.shape) != (n_pages, kv_heads) or not x.is_contiguous():
                    raise ValueError(f"{name}: contiguous fp32 [{n_pages}, {kv_heads}]")
        for name, x, dims in (("table", table, 2), ("length", length, 1), ("ref", ref, 1)):
            if x.dtype is not torch.int32 or x.dim() != dims or not x.is_contiguous():
                raise ValueError(f"{name}: a contiguous int32 tensor of {dims} dimension(s)")
        if length.shape[0] != table.shape[0] or ref.shape[0] != n_pages:
            raise ValueError("length has an entry for each table row, ref one for each page")
        self.n_heads, self.n_kv_heads, self.head_dim, self.page_tokens = n_heads, kv_heads, dim, page
        self.desc = PiKvDesc(len(self.layers), n_heads, kv_heads, dim, page, n_pages, table.shape[0], table.shape[1])
        self.h = None
        self.h = pi_kv_create(self.desc, [PiKvLayer(*(_ptr(L[x]) for x in ("k", "v", "k_scale", "v_scale")))
                                          for L in self.layers], PiKvState(_ptr(table), _ptr(length), _ptr(ref)))

    @classmethod
    def empty(cls, n_layers, n_heads, n_kv_heads, head_dim, page_tokens, n_pages, max_seqs, max_tokens, device="cuda"):
        """A new cache: room for n_pages pages of page_tokens positions, max_seqs sequences of up to max_tokens."""
        import torch

        def pool():
            return torch.zeros((n_pages, n_kv_heads, page_tokens, head_dim), dtype=torch.uint8,
                               device=device).view(torch.float8_e4m3fn)

        def scale():
            return torch.zeros((n_pages, n_kv_heads), dtype=torch.float32, device=device)

        layers = [dict(k=pool(), v=pool(), k_scale=scale(), v_scale=scale()) for _ in range(n_layers)]
        columns = -(-max_tokens // page_tokens)
        i32 = dict(dtype=torch.int32, device=device)
        return cls(layers, torch.full((max_seqs, columns), -1, **i32), torch.zeros(max_seqs, **i32),
                   torch.zeros(n_pages, **i32), n_heads=n_heads)

    def reserve(self, seqs, tok_start, stream=None) -> None:
        """The sequences grow by their new tokens (lengths, pages)."""
        n = seqs.shape[0]
        pi_kv_reserve(self.h, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, stream)

    def append(self, layer, seqs, tok_start, k_new, v_new, stream=None) -> None:
        """Keys and values [tokens, kv heads, dim] (fp32, bf16 or fp16) of the sequences' last positions."""
        n, T = seqs.shape[0], k_new.shape[0]
        ld = _token_rows(k_new, self.n_kv_heads, self.head_dim, "k_new")
        if _token_rows(v_new, self.n_kv_heads, self.head_dim, "v_new") != ld or v_new.dtype is not k_new.dtype or \
                v_new.shape[0] != T:
            raise ValueError("k_new and v_new: one shape, type and row stride")
        pi_kv_append(self.h, layer, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, T, k_new.data_ptr(),
                     v_new.data_ptr(), ld, _act_dtype(k_new), stream)

    def attend(self, layer, seqs, tok_start, q, out=None, lse=None, *, scale=None, window=0, sinks=0, stream=None):
        """Attention of q [tokens, heads, dim], the sequences' last positions, over their cache; returns out
        (q's type). window > 0: only the last `window` positions and the first `sinks` are seen. lse: fp32
        [tokens, heads], filled with the log of each row's sum of exponentials."""
        n, T, heads, dim = seqs.shape[0], q.shape[0], self.n_heads, self.head_dim
        ld, dtype = _token_rows(q, heads, dim, "q"), _act_dtype(q)
        if out is None:
            out, ld_out = _empty((T, heads, dim), q.dtype, q.device, stream), heads * dim
        else:
            ld_out = _token_rows(out, heads, dim, "out")
            if out.dtype is not q.dtype or out.shape[0] != T:
                raise ValueError("out: q's type and number of tokens")
        if lse is not None:
            if _act_dtype(lse) != PI_F32 or tuple(lse.shape) != (T, heads) or not lse.is_contiguous():
                raise ValueError(f"lse: contiguous fp32 [{T}, {heads}]")
            lse = lse.data_ptr()
        pi_kv_attend(self.h, layer, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, T, q.data_ptr(), ld,
                     out.data_ptr(), ld_out, lse, dtype, dim ** -0.5 if scale is None else scale, window, sinks, stream)
        return out

    def fork(self, src, dst, stream=None) -> None:
        """dst[i] becomes a copy of sequence src[i] that shares its full pages."""
        n = src.shape[0]
        pi_kv_fork(self.h, _i32(src, "src"), _i32(dst, "dst", n), n, stream)

    def free(self, seqs, stream=None) -> None:
        """Give back the sequences' pages."""
        pi_kv_free(self.h, _i32(seqs, "seqs"), seqs.shape[0], stream)

    def trim(self, seqs, window, sinks=0, stream=None) -> None:
        """Give back the pages that a sliding window with first tokens no longer sees."""
        pi_kv_trim(self.h, _i32(seqs, "seqs"), seqs.shape[0], window, sinks, stream)

    def copy_pages(self, src, dst, stream=None) -> None:
        """Copy pages src[i] to dst[i] in every layer (table and counts stay)."""
        n = src.shape[0]
        pi_kv_copy_pages(self.h, _i32(src, "src"), _i32(dst, "dst", n), n, stream)

    def compact(self, stream=None):
        """Move the used pages to the lowest ids; returns their number (int32 [1], on the GPU)."""
        live = _empty(1, self.ref.dtype, self.ref.device, stream)
        pi_kv_compact(self.h, live.data_ptr(), stream)
        return live

    def status(self) -> int:
        return pi_kv_get_status(self.h)

    def close(self):
        if self.h:
            pi_kv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
