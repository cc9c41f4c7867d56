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

# every symbol that the headers in include/ declare
EXPORTS = (
    "pi_ffn_create", "pi_ffn_destroy", "pi_predict", "pi_sparse_ffn", "pi_decode_stack",
    "pi_hot_first_order", "pi_permute_rows", "pi_get_status", "pi_status_string", "pi_abi_version",
    "pi_profile_begin", "pi_profile_end", "pi_sparse_ffn_noalloc", "pi_selftest_grid_barrier",
    "pi_selftest_umma", "pi_ffn_set_hot_neurons", "pi_ffn_set_hot_prefix", "pi_decode_stack_layers",
    "pi_ffn_set_phase_trace",
    "pi_kv_create", "pi_kv_destroy", "pi_kv_get_status", "pi_kv_reserve", "pi_kv_append", "pi_kv_attend",
    "pi_kv_fork", "pi_kv_free", "pi_kv_trim", "pi_kv_copy_pages", "pi_kv_compact",
    "pi_kv_append_rotated", "pi_kv_share", "pi_kv_attend_shared", "pi_rotate", "pi_int4_linear",
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


class PiRotary(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("amp", ctypes.c_float), ("eps", ctypes.c_float)]


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
    "pi_kv_append_rotated": [_P, _I32, _P, _P, _I32, _I32, ctypes.POINTER(PiRotary), _P, _I64, _P, _I64, _P, _P, _I64,
                             _I32, _P],
    "pi_kv_share": [_P, _P, _P, _I32, _P, _I32, _P, _P],
    "pi_kv_attend_shared": [_P, _I32, _P, _P, _I32, _I32, _P, _I32, _P, _I64, _P, _I64, _P, _I32, _F32, _P, _P],
    "pi_rotate": [ctypes.POINTER(PiRotary), _P, _I32, _I32, _I32, _I32, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _P],
    "pi_int4_linear": [_P, _P, _P, _I32, _I32, _P, _I64, _I32, _P, _I64, _P, _I64, _I32, _P],
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


def pi_kv_append_rotated(h, layer, seqs, tok_start, n, n_tokens, rotary, q, ld_q, q_out, ld_q_out, k_new, v_new, ld, dtype,
                         stream=None) -> None:
    _check(_lib.pi_kv_append_rotated(h, layer, _ptr(seqs), _ptr(tok_start), n, n_tokens, ctypes.byref(rotary), _ptr(q),
                                     ld_q, _ptr(q_out), ld_q_out, _ptr(k_new), _ptr(v_new), ld, dtype, _stream(stream)),
           "pi_kv_append_rotated")


def pi_kv_share(h, seqs, tok_start, n, group_start, n_groups, plan, stream=None) -> None:
    _check(_lib.pi_kv_share(h, _ptr(seqs), _ptr(tok_start), n, _ptr(group_start), n_groups, _ptr(plan), _stream(stream)),
           "pi_kv_share")


def pi_kv_attend_shared(h, layer, seqs, tok_start, n, n_tokens, plan, n_groups, q, ld_q, out, ld_out, lse, dtype, scale,
                        work, stream=None) -> None:
    _check(_lib.pi_kv_attend_shared(h, layer, _ptr(seqs), _ptr(tok_start), n, n_tokens, _ptr(plan), n_groups, _ptr(q), ld_q,
                                    _ptr(out), ld_out, _ptr(lse), dtype, scale, _ptr(work), _stream(stream)),
           "pi_kv_attend_shared")


def pi_rotate(rotary, pos, n_tokens, n_heads, n_kv_heads, head_dim, q, ld_q, q_out, ld_q_out, k, ld_k, k_out, ld_k_out,
              dtype, stream=None) -> None:
    _check(_lib.pi_rotate(ctypes.byref(rotary), _ptr(pos), n_tokens, n_heads, n_kv_heads, head_dim, _ptr(q), ld_q,
                          _ptr(q_out), ld_q_out, _ptr(k), ld_k, _ptr(k_out), ld_k_out, dtype, _stream(stream)),
           "pi_rotate")


def pi_int4_linear(w, s, bias, n, k, x, ld_x, rows, add, ld_add, y, ld_y, dtype, stream=None) -> None:
    _check(_lib.pi_int4_linear(_ptr(w), _ptr(s), _ptr(bias), n, k, _ptr(x), ld_x, rows, _ptr(add), ld_add, _ptr(y), ld_y,
                               dtype, _stream(stream)), "pi_int4_linear")


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


def _empty_like(x, shape, stream):
    """A new tensor of x's type on x's device that belongs to `stream` (see _empty)."""
    return x.new_empty(shape) if stream is None else _empty(shape, x.dtype, x.device, stream)


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


def _rows(x, width, name):
    """Row stride of a [rows, width] tensor with contiguous rows."""
    shape = x.shape
    if len(shape) != 2 or shape[1] != width or not x.is_cuda or (width > 1 and x.stride(1) != 1):
        raise ValueError(f"{name}: a [rows, {width}] CUDA tensor with contiguous rows, got {tuple(shape)}")
    return x.stride(0) if shape[0] > 1 else width


class Int4Linear:
    """y = x W^T (+ bias) (+ add) with 4-bit weights in the format of SparseFFN's (group 128), for 1 to 256 rows.

    w: uint8 [n, k / 2] (two's-complement nibbles, the even element low), s: fp16 [n, k / 128], bias: fp32 [n] or None
    (kept referenced).
    """

    def __init__(self, w, s, bias=None):
        import torch

        if w.dtype is not torch.uint8 or w.dim() != 2 or not w.is_contiguous():
            raise ValueError("w: contiguous uint8 [n, k / 2]")
        self.n, self.k = w.shape[0], 2 * w.shape[1]
        if s.dtype is not torch.float16 or tuple(s.shape) != (self.n, self.k // 128) or not s.is_contiguous():
            raise ValueError(f"s: contiguous fp16 [{self.n}, {self.k // 128}]")
        if bias is not None and (bias.dtype is not torch.float32 or tuple(bias.shape) != (self.n,) or not bias.is_contiguous()):
            raise ValueError(f"bias: contiguous fp32 [{self.n}]")
        self.w, self.s, self.bias = w, s, bias
        self._weights = w.data_ptr(), s.data_ptr(), _ptr(bias), self.n, self.k

    def __call__(self, x, out=None, add=None, stream=None):
        """x [rows, k] (fp32, bf16 or fp16); add: x's type, [rows, n]; out: likewise, and may be add itself."""
        rows, n = x.shape[0], self.n
        ld_x, dtype, ld_add = _rows(x, self.k, "x"), _act_dtype(x), 0
        if add is not None:
            ld_add = _rows(add, n, "add")
            if add.dtype is not x.dtype or add.shape[0] != rows:
                raise ValueError("add: x's type and number of rows")
            add = add.data_ptr()
        if out is None:
            out, ld_out = _empty_like(x, (rows, n), stream), n
        else:
            ld_out = _rows(out, n, "out")
            if out.dtype is not x.dtype or out.shape[0] != rows:
                raise ValueError("out: x's type and number of rows")
        code = _lib.pi_int4_linear(*self._weights, x.data_ptr(), ld_x, rows, add, ld_add, out.data_ptr(), ld_out, dtype,
                                   _stream(stream))
        if code:
            _check(code, "pi_int4_linear")
        return out


def rotary_frequencies(rot_dim, base=10000.0, *, stretch=1.0, trained=None, slow=1.0, fast=32.0):
    """Radians per position of the rot_dim / 2 pairs: base^(-2 i / rot_dim), for contexts `stretch` times the trained
    length. trained None: every frequency over stretch. Else pairs that turn at least `fast` times within `trained`
    positions keep theirs, those that turn at most `slow` times get it over stretch, and in between the two are mixed
    in proportion."""
    import math

    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        keep = 0.0
        if trained is not None:
            keep = min(1.0, max(0.0, (trained * f / (2 * math.pi) - slow) / (fast - slow)))
        out.append(f * (keep + (1.0 - keep) / stretch))
    return out


def _pi_bits(n):
    """pi * 2^n to the nearest integer but one: 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (n + 32)

    def atan_of_inverse(q):
        total, term, k = 0, one // q, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= q * q
            k += 2
        return total

    return (16 * atan_of_inverse(5) - 4 * atan_of_inverse(239)) >> 32


def rotary_turns(freq):
    """Each frequency (radians per position) as a fraction of a turn per position in units of 2^-64, exactly rounded
    from the given double: what pi_rotary_t's `turns` holds. Ints in [0, 2^64)."""
    bits = 256
    turn = 2 * _pi_bits(bits)
    out = []
    for f in freq:
        num, den = float(f).as_integer_ratio()
        num, den = num << (64 + bits), den * turn
        out.append((2 * num + den) // (2 * den) % (1 << 64))
    return out


class Rotary:
    """Norm (optional) and position rotation of query and key heads, for ``rotate`` and ``KVCache.append_rotated``.

    freq: radians per position of each pair (any doubles; ``rotary_frequencies`` has the usual ones); the first
    2 len(freq) elements of a head are turned, in pairs (i, i + len(freq)) or, interleaved, (2 i, 2 i + 1), and multiplied by
    amp. norm: each head is divided by its root mean square first; q_norm, k_norm: fp32 [head_dim] weights, None: ones.
    """

    def __init__(self, freq, head_dim, *, interleaved=False, amp=1.0, norm=False, q_norm=None, k_norm=None, eps=1e-6,
                 device="cuda"):
        import torch

        turns = [t - (1 << 64) if t >= 1 << 63 else t for t in rotary_turns(freq)]
        self.head_dim, self.q_norm, self.k_norm = head_dim, q_norm, k_norm
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is None:
                continue
            if w.dtype is not torch.float32 or tuple(w.shape) != (head_dim,) or not w.is_contiguous():
                raise ValueError(f"{name}: contiguous fp32 [{head_dim}]")
            if not norm:
                raise ValueError(f"{name}: weights of a norm that is off")
        self.turns = torch.tensor(turns, dtype=torch.int64).to(device)
        self.desc = PiRotary(_ptr(self.turns) if turns else None, _ptr(q_norm), _ptr(k_norm), 2 * len(turns), int(interleaved),
                             int(norm), amp, eps)
        self._desc = ctypes.byref(self.desc)

    def rotate(self, pos, q, k=None, q_out=None, k_out=None, stream=None):
        """(q_out, k_out): q [tokens, heads, dim] and k [tokens, kv heads, dim] (fp32, bf16 or fp16) at positions pos
        (int32 [tokens]). q_out and k_out may be q and k themselves."""
        shape, dtype = q.shape, _act_dtype(q)
        if len(shape) != 3:
            raise ValueError("q: [tokens, heads, dim]")
        T, heads, dim = shape[0], shape[1], self.head_dim
        ld_q = _token_rows(q, heads, dim, "q")
        if q_out is None:
            q_out, ld_q_out = _empty_like(q, (T, heads, dim), stream), heads * dim
        else:
            ld_q_out = self._out(q_out, q, heads, "q_out")
        kv_heads = ld_k = ld_k_out = 0
        k_at = k_out_at = None
        if k is None:
            k_out = None
        else:
            shape = k.shape
            if len(shape) != 3 or shape[0] != T or k.dtype is not q.dtype:
                raise ValueError("k: [tokens, kv heads, dim] of q's type and number of tokens")
            kv_heads = shape[1]
            ld_k = _token_rows(k, kv_heads, dim, "k")
            if k_out is None:
                k_out, ld_k_out = _empty_like(k, (T, kv_heads, dim), stream), kv_heads * dim
            else:
                ld_k_out = self._out(k_out, k, kv_heads, "k_out")
            k_at, k_out_at = k.data_ptr(), k_out.data_ptr()
        code = _lib.pi_rotate(self._desc, _i32(pos, "pos", T), T, heads, kv_heads, dim, q.data_ptr(), ld_q, q_out.data_ptr(),
                              ld_q_out, k_at, ld_k, k_out_at, ld_k_out, dtype, _stream(stream))
        if code:
            _check(code, "pi_rotate")
        return q_out, k_out

    def _out(self, out, x, heads, name):
        """Row stride of an output given for x."""
        if out.dtype is not x.dtype or out.shape[0] != x.shape[0]:
            raise ValueError(f"{name}: its input's type and number of tokens")
        return _token_rows(out, heads, self.head_dim, name)


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
        self._f32 = self.layers[0]["k_scale"]
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

    def append_rotated(self, layer, seqs, tok_start, rotary, q, k_new, v_new, q_out=None, stream=None):
        """append with rotary's norm and rotation in the same pass: keys are turned by their positions before they are
        coded; returns q_out, q [tokens, heads, dim] turned likewise (q_out may be q itself)."""
        n, T, heads, dim = seqs.shape[0], q.shape[0], self.n_heads, self.head_dim
        if rotary.head_dim != dim:
            raise ValueError(f"rotary: made for heads of {rotary.head_dim}, not {dim}")
        ld_q, ld, dtype = _token_rows(q, heads, dim, "q"), _token_rows(k_new, self.n_kv_heads, dim, "k_new"), _act_dtype(q)
        if _token_rows(v_new, self.n_kv_heads, dim, "v_new") != ld or v_new.dtype is not k_new.dtype or \
                k_new.dtype is not q.dtype or v_new.shape[0] != T or k_new.shape[0] != T:
            raise ValueError("q, k_new and v_new: one type and number of tokens, the latter two one row stride")
        if q_out is None:
            q_out, ld_out = _empty_like(q, (T, heads, dim), stream), heads * dim
        else:
            ld_out = rotary._out(q_out, q, heads, "q_out")
        code = _lib.pi_kv_append_rotated(self.h, layer, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, T,
                                         rotary._desc, q.data_ptr(), ld_q, q_out.data_ptr(), ld_out, k_new.data_ptr(),
                                         v_new.data_ptr(), ld, dtype, _stream(stream))
        if code:
            _check(code, "pi_kv_append_rotated")
        return q_out

    def attend(self, layer, seqs, tok_start, q, out=None, lse=None, *, scale=None, window=0, sinks=0, stream=None):
        """Attention of q [tokens, heads, dim], the sequences' last positions, over their cache; returns out
        (q's type). window > 0: only the last `window` positions and the first `sinks` are seen. lse: fp32
        [tokens, heads], filled with the log of each row's sum of exponentials."""
        n, T = seqs.shape[0], q.shape[0]
        out, args = self._attend_args(q, out, lse, stream)
        pi_kv_attend(self.h, layer, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, T, *args,
                     self.head_dim ** -0.5 if scale is None else scale, window, sinks, stream)
        return out

    def _attend_args(self, q, out, lse, stream):
        """out (made where it is None), and the addresses and strides of q, out and lse with q's type."""
        T, heads, dim = q.shape[0], self.n_heads, self.head_dim
        ld, dtype = _token_rows(q, heads, dim, "q"), _act_dtype(q)
        if out is None:
            out, ld_out = _empty_like(q, (T, heads, dim), stream), heads * dim
        else:
            ld_out = _token_rows(out, heads, dim, "out")
            if out.dtype is not q.dtype or out.shape[0] != T:
                raise ValueError("out: q's type and number of tokens")
        if lse is not None:
            if _act_dtype(lse) != PI_F32 or tuple(lse.shape) != (T, heads) or not lse.is_contiguous():
                raise ValueError(f"lse: contiguous fp32 [{T}, {heads}]")
            lse = lse.data_ptr()
        return out, (q.data_ptr(), ld, out.data_ptr(), ld_out, lse, dtype)

    def share(self, seqs, tok_start, group_start, stream=None):
        """What groups of the call's sequences share (group g: group_start[g] .. group_start[g + 1] of seqs), for
        attend_shared: an int32 tensor. It serves every layer and later steps of the same seqs and tok_start while the
        sequences only grow."""
        n, groups = seqs.shape[0], group_start.shape[0] - 1
        plan = _empty(3 * (n + groups) + 2, group_start.dtype, group_start.device, stream)
        pi_kv_share(self.h, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, _i32(group_start, "group_start"),
                    groups, plan.data_ptr(), stream)
        return plan

    def attend_shared(self, layer, seqs, tok_start, plan, q, out=None, lse=None, *, scale=None, work=None, stream=None):
        """attend (without a window) with the plan's shared prefixes read once for all sequences of a group. work: fp32, at
        least tokens * heads * (dim + 2) elements to use in between."""
        n, T = seqs.shape[0], q.shape[0]
        groups = (plan.shape[0] - 2) // 3 - n if plan.dim() == 1 else -1
        if groups < 0 or groups > n:
            raise ValueError(f"plan: what share returned for these {n} sequences")
        out, args = self._attend_args(q, out, lse, stream)
        room = T * self.n_heads * (self.head_dim + 2)
        if work is None:
            work = _empty_like(self._f32, (room,), stream)
        elif _act_dtype(work) != PI_F32 or work.numel() < room or not work.is_contiguous():
            raise ValueError(f"work: contiguous fp32 of {room} elements")
        code = _lib.pi_kv_attend_shared(self.h, layer, _i32(seqs, "seqs"), _i32(tok_start, "tok_start", n + 1), n, T,
                                        _i32(plan, "plan", 3 * (n + groups) + 2), groups, *args,
                                        self.head_dim ** -0.5 if scale is None else scale, work.data_ptr(), _stream(stream))
        if code:
            _check(code, "pi_kv_attend_shared")
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
