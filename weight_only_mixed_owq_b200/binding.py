"""ctypes binding of libowq_b200.so (include/owq.h): same names, argument marshalling only.

Every function here forwards to the C ABI; PyTorch is used only to allocate device memory
and to name streams.  There is no CPU fallback: if the library is missing this module
raises at import time.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# OWQ_LIB_VARIANT=bounds loads the debug-bounds build (libowq_b200_bounds.so) built beside it
VARIANTS = {"": "libowq_b200.so", "bounds": "libowq_b200_bounds.so"}
_variant = os.environ.get("OWQ_LIB_VARIANT", "")
if _variant not in VARIANTS:
    raise ImportError(f"OWQ_LIB_VARIANT={_variant!r}: expected one of {sorted(VARIANTS)}")
LIB_PATH = os.path.join(PKG, VARIANTS[_variant])

OWQ_OK = 0
STATUS_NAMES = {
    0: "OWQ_OK", 1: "OWQ_ERR_NULL", 2: "OWQ_ERR_SHAPE", 3: "OWQ_ERR_BITS", 4: "OWQ_ERR_GROUP",
    5: "OWQ_ERR_INDEX", 6: "OWQ_ERR_ALIGN", 7: "OWQ_ERR_CUDA", 8: "OWQ_ERR_TIMEOUT",
    9: "OWQ_ERR_NOMEM", 10: "OWQ_ERR_HANDLE", 11: "OWQ_ERR_DEVICE", 12: "OWQ_ERR_ARG", 13: "OWQ_ERR_BOUNDS",
}
OWQ_ACT_SILU, OWQ_ACT_GELU, OWQ_ACT_GELU_TANH = 0, 1, 2
OWQ_F32, OWQ_F16, OWQ_BF16 = 0, 1, 2
OWQ_GATED_FORWARD, OWQ_GATED_INPUT_GRAD, OWQ_GATED_BACKWARD = 0, 1, 2
OWQ_INJECT_NONE, OWQ_INJECT_GEMV_TAG, OWQ_INJECT_GEMM_ARRIVE, OWQ_INJECT_BOUNDS = 0, 1, 2, 3
OWQ_INJECT_CLIP, OWQ_INJECT_GATED = 4, 5

# (name, restype, argtypes) of every exported symbol of include/owq.h
_P, _I, _SZ, _S = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t), ctypes.c_char_p
PROTOTYPES = [
    ("owq_quantize", _I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    ("owq_quantize_noalloc", _I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    ("owq_pack", _I, [_P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _P, ctypes.POINTER(_P)]),
    ("owq_search_params", _I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
    ("owq_optq", _I, [_P, _P, _I, _I, _I, _I, _I, _P, _I, _P, _P, ctypes.c_double, _P, _P, _P]),
    ("owq_quantize_optq", _I, [_P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_double, _P, _P, _P, _P, _P, _P]),
    ("owq_storage_words", _I, [_I, _I, _I, ctypes.POINTER(_I)]),
    ("owq_storage_pack", _I, [_P, _I, _I, _I, _P, _I, _P, _P]),
    ("owq_storage_unpack", _I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _P]),
    ("owq_pack_storage", _I, [_P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _P, ctypes.POINTER(_P)]),
    ("owq_gemv", _I, [_P, _P, _P, _I, _P]),
    ("owq_gemv_multi", _I, [ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(_P), _I, _I, _P]),
    ("owq_gemm", _I, [_P, _P, _P, _I, _P]),
    ("owq_gemm_plan", _I, [_I, _I, _I, _I, ctypes.POINTER(_I)]),
    ("owq_weak_grad", _I, [_P, _P, _P, _P, _I, _P]),
    ("owq_input_grad", _I, [_P, _P, _P, _I, _P]),
    ("owq_gated_gemv", _I, [_P, _P, _I, _P, _P, _I, _P]),
    ("owq_gated_workspace", _I, [_P, _P, _I, _SZ]),
    ("owq_gated_plan", _I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I)]),
    ("owq_gated_gemm", _I, [_P, _P, _I, _P, _P, _I, _P, ctypes.c_size_t, _P]),
    ("owq_gated_grad", _I, [_P, _P, _I, _P, _P, _P, _P, _I, _P, ctypes.c_size_t, _P]),
    ("owq_gated_backward", _I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _P, ctypes.c_size_t, _P]),
    ("owq_gated_input_grad", _I, [_P, _P, _P, _P, _P, _I, _P, ctypes.c_size_t, _P]),
    ("owq_clip_create", _I, [_P, _I, _P, ctypes.POINTER(_P)]),
    ("owq_clip_grads", _I, [_P, ctypes.c_float, _P, _P]),
    ("owq_clip_free", _I, [_P]),
    ("owq_dequant", _I, [_P, _P, _P, _P]),
    ("owq_layer_info", _I, [_P] + [ctypes.POINTER(_I)] * 5),
    ("owq_layer_bytes", _I, [_P, _SZ, _SZ, _SZ, _SZ]),
    ("owq_layer_free", _I, [_P]),
    ("owq_device_status", _I, []),
    ("owq_debug_inject", _I, [_I, ctypes.c_longlong]),
    ("owq_status_string", _S, [_I]),
    ("owq_version", _S, []),
]


class OwqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m weight_only_mixed_owq_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, res, args in PROTOTYPES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def _ptr(a) -> int | None:
    """Device address of a tensor (or an int address, or None)."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        try:
            import torch
            if torch.cuda.is_available():
                return torch.cuda.current_stream().cuda_stream
        except Exception:
            pass
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str) -> None:
    if st != OWQ_OK:
        raise OwqError(st, where)


# ------------------------------------------------------------------ raw C-ABI mirrors
def owq_quantize(W, X, N, K, T, bits, group, k, codes, scales, zeros, idx, w_weak, stream=None) -> int:
    return LIB.owq_quantize(_ptr(W), _ptr(X), N, K, T, bits, group, k, _ptr(codes), _ptr(scales),
                            _ptr(zeros), _ptr(idx), _ptr(w_weak), _stream(stream))


def owq_quantize_noalloc(W, X, N, K, T, bits, group, k, codes, scales, zeros, idx, w_weak, stream=None) -> int:
    return LIB.owq_quantize_noalloc(_ptr(W), _ptr(X), N, K, T, bits, group, k, _ptr(codes), _ptr(scales),
                                    _ptr(zeros), _ptr(idx), _ptr(w_weak), _stream(stream))


def owq_pack(codes, N, K, bits, group, scales, zeros, idx, k, w_weak, stream=None):
    """Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = LIB.owq_pack(_ptr(codes), N, K, bits, group, _ptr(scales), _ptr(zeros), _ptr(idx), k,
                      _ptr(w_weak), _stream(stream), ctypes.byref(h))
    return st, h.value


def owq_search_params(W, N, K, bits, group, idx, k, scales, zeros, stream=None) -> int:
    return LIB.owq_search_params(_ptr(W), N, K, bits, group, _ptr(idx), k, _ptr(scales), _ptr(zeros), _stream(stream))


def owq_optq(W, X, N, K, T, bits, group, idx, k, scales, zeros, damp, codes, w_weak, stream=None) -> int:
    return LIB.owq_optq(_ptr(W), _ptr(X), N, K, T, bits, group, _ptr(idx), k, _ptr(scales), _ptr(zeros),
                        float(damp), _ptr(codes), _ptr(w_weak), _stream(stream))


def owq_quantize_optq(W, X, N, K, T, bits, group, k, damp, codes, scales, zeros, idx, w_weak, stream=None) -> int:
    return LIB.owq_quantize_optq(_ptr(W), _ptr(X), N, K, T, bits, group, k, float(damp), _ptr(codes), _ptr(scales),
                                 _ptr(zeros), _ptr(idx), _ptr(w_weak), _stream(stream))


def owq_storage_words(K, bits, k):
    """Returns (status, uint32 words per row of the storage-favoured stream)."""
    w = ctypes.c_int()
    st = LIB.owq_storage_words(K, bits, k, ctypes.byref(w))
    return st, w.value


def owq_storage_pack(codes, N, K, bits, idx, k, words, stream=None) -> int:
    return LIB.owq_storage_pack(_ptr(codes), N, K, bits, _ptr(idx), k, _ptr(words), _stream(stream))


def owq_storage_unpack(words, N, K, bits, group, idx, k, zeros, codes, stream=None) -> int:
    return LIB.owq_storage_unpack(_ptr(words), N, K, bits, group, _ptr(idx), k, _ptr(zeros), _ptr(codes),
                                  _stream(stream))


def owq_pack_storage(words, N, K, bits, group, scales, zeros, idx, k, w_weak, stream=None):
    """Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = LIB.owq_pack_storage(_ptr(words), N, K, bits, group, _ptr(scales), _ptr(zeros), _ptr(idx), k,
                              _ptr(w_weak), _stream(stream), ctypes.byref(h))
    return st, h.value


def owq_gemv(layer, x, y, M, stream=None) -> int:
    return LIB.owq_gemv(layer, _ptr(x), _ptr(y), M, _stream(stream))


def owq_gemv_multi(layers, xs, ys, M, stream=None) -> int:
    n = len(layers)
    arr_l = (ctypes.c_void_p * n)(*layers)
    arr_x = (ctypes.c_void_p * n)(*[_ptr(v) for v in xs])
    arr_y = (ctypes.c_void_p * n)(*[_ptr(v) for v in ys])
    return LIB.owq_gemv_multi(arr_l, arr_x, arr_y, n, M, _stream(stream))


def owq_gemm(layer, x, y, M, stream=None) -> int:
    return LIB.owq_gemm(layer, _ptr(x), _ptr(y), M, _stream(stream))


def owq_gemm_plan(N, K, M, sms):
    """Returns (status, {tile_tokens, splits, tail_tiles, tail_splits}): owq_gemm's launch shape."""
    out = (ctypes.c_int * 4)()
    st = LIB.owq_gemm_plan(N, K, M, sms, out)
    return st, dict(zip(("tile_tokens", "splits", "tail_tiles", "tail_splits"), out))


def owq_weak_grad(layer, x, dy, dw_weak, M, stream=None) -> int:
    return LIB.owq_weak_grad(layer, _ptr(x), _ptr(dy), _ptr(dw_weak), M, _stream(stream))


def owq_input_grad(layer, dy, dx, M, stream=None) -> int:
    return LIB.owq_input_grad(layer, _ptr(dy), _ptr(dx), M, _stream(stream))


def owq_gated_gemv(gate, up, act, x, h, M, stream=None) -> int:
    return LIB.owq_gated_gemv(gate, up, act, _ptr(x), _ptr(h), M, _stream(stream))


def owq_gated_workspace(gate, up, M):
    """Returns (status, bytes)."""
    n = ctypes.c_size_t()
    st = LIB.owq_gated_workspace(gate, up, M, ctypes.byref(n))
    return st, n.value


def owq_gated_plan(N, K, M, sms, product):
    """Returns (status, {tile_tokens, tiles, whole, splits, steps}): a gated product's launch shape."""
    out = (ctypes.c_int * 5)()
    st = LIB.owq_gated_plan(N, K, M, sms, product, out)
    return st, dict(zip(("tile_tokens", "tiles", "whole", "splits", "steps"), out))


def owq_gated_gemm(gate, up, act, x, h, M, ws, ws_bytes, stream=None) -> int:
    return LIB.owq_gated_gemm(gate, up, act, _ptr(x), _ptr(h), M, _ptr(ws), ws_bytes, _stream(stream))


def owq_gated_grad(gate, up, act, x, dh, dgate, dup, M, ws, ws_bytes, stream=None) -> int:
    return LIB.owq_gated_grad(gate, up, act, _ptr(x), _ptr(dh), _ptr(dgate), _ptr(dup), M, _ptr(ws), ws_bytes,
                              _stream(stream))


def owq_gated_input_grad(gate, up, dgate, dup, dx, M, ws, ws_bytes, stream=None) -> int:
    return LIB.owq_gated_input_grad(gate, up, _ptr(dgate), _ptr(dup), _ptr(dx), M, _ptr(ws), ws_bytes, _stream(stream))


def owq_gated_backward(gate, up, act, x, dh, dgate, dup, dx, M, ws, ws_bytes, stream=None) -> int:
    return LIB.owq_gated_backward(gate, up, act, _ptr(x), _ptr(dh), _ptr(dgate), _ptr(dup), _ptr(dx), M, _ptr(ws), ws_bytes,
                                  _stream(stream))


class OwqGrad(ctypes.Structure):
    """owq_grad_t: one gradient tensor of owq_clip_create."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_longlong), ("dtype", ctypes.c_int)]


def owq_clip_create(grads, count, stream=None):
    """grads: a ctypes array of OwqGrad (or None).  Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = LIB.owq_clip_create(grads, count, _stream(stream), ctypes.byref(h))
    return st, h.value


def owq_clip_grads(clip, max_norm, norm, stream=None) -> int:
    return LIB.owq_clip_grads(clip, float(max_norm), _ptr(norm), _stream(stream))


def owq_clip_free(clip) -> int:
    return LIB.owq_clip_free(clip)


def owq_dequant(layer, w_hat, codes=None, stream=None) -> int:
    return LIB.owq_dequant(layer, _ptr(w_hat), _ptr(codes), _stream(stream))


def owq_layer_info(layer):
    vals = [ctypes.c_int() for _ in range(5)]
    st = LIB.owq_layer_info(layer, *[ctypes.byref(v) for v in vals])
    return st, tuple(v.value for v in vals)


def owq_layer_bytes(layer):
    vals = [ctypes.c_size_t() for _ in range(4)]
    st = LIB.owq_layer_bytes(layer, *[ctypes.byref(v) for v in vals])
    return st, dict(zip(("packed", "scales_zeros", "weak", "idx"), (v.value for v in vals)))


def owq_layer_free(layer) -> int:
    return LIB.owq_layer_free(layer)


def owq_device_status() -> int:
    return LIB.owq_device_status()


def owq_debug_inject(what: int, wait_cycles: int) -> int:
    return LIB.owq_debug_inject(what, wait_cycles)


def owq_status_string(st: int) -> str:
    return LIB.owq_status_string(st).decode()


def owq_version() -> str:
    return LIB.owq_version().decode()


# ------------------------------------------------------------------ torch-facing helpers
def quantize(W, X, bits: int, group: int, k: int, stream=None) -> dict:
    """Run owq_quantize on fp16 CUDA tensors W (N x K) and X (T x K); allocates the outputs."""
    import torch
    N, K = W.shape
    T = X.shape[0]
    dev = W.device
    out = {
        "codes": torch.empty((N, K), dtype=torch.uint8, device=dev),
        "scales": torch.empty((N, K // group), dtype=torch.float16, device=dev),
        "zeros": torch.empty((N, K // group), dtype=torch.float16, device=dev),
        "idx": torch.empty((k,), dtype=torch.int32, device=dev),
        "w_weak": torch.empty((N, k), dtype=torch.float16, device=dev),
    }
    _check(owq_quantize(W, X, N, K, T, bits, group, k, out["codes"], out["scales"], out["zeros"],
                        out["idx"] if k else None, out["w_weak"] if k else None, stream), "owq_quantize")
    return out


class OwqLayer:
    """A packed layer owned by the C library (freed on close() / garbage collection)."""

    def __init__(self, codes, scales, zeros, idx, w_weak, bits: int, group: int, stream=None):
        N, K = codes.shape
        k = 0 if idx is None else int(idx.numel())
        st, h = owq_pack(codes, N, K, bits, group, scales, zeros, idx if k else None, k,
                         w_weak if k else None, stream)
        _check(st, "owq_pack")
        self.handle = h
        self.N, self.K, self.bits, self.group, self.k = N, K, bits, group, k

    def gemv(self, x, y=None, stream=None):
        import torch
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=x.device)
        _check(owq_gemv(self.handle, x, y, M, stream), "owq_gemv")
        return y

    def gemm(self, x, y=None, stream=None):
        import torch
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=x.device)
        _check(owq_gemm(self.handle, x, y, M, stream), "owq_gemm")
        return y

    def weak_grad(self, x, dy, dw=None, stream=None):
        """dW_weak = dy^T x[:, idx] (fp32 N x k)."""
        import torch
        M = x.shape[0]
        if dw is None:
            dw = torch.empty((self.N, self.k), dtype=torch.float32, device=x.device)
        _check(owq_weak_grad(self.handle, x, dy, dw if self.k else None, M, stream), "owq_weak_grad")
        return dw

    def input_grad(self, dy, dx=None, stream=None):
        """dX = dy W_eff (fp16 M x K)."""
        import torch
        M = dy.shape[0]
        if dx is None:
            dx = torch.empty((M, self.K), dtype=torch.float16, device=dy.device)
        _check(owq_input_grad(self.handle, dy, dx, M, stream), "owq_input_grad")
        return dx

    def dequant(self, with_codes: bool = False, stream=None):
        import torch
        dev = torch.device("cuda")
        w = torch.empty((self.N, self.K), dtype=torch.float16, device=dev)
        c = torch.empty((self.N, self.K), dtype=torch.uint8, device=dev) if with_codes else None
        _check(owq_dequant(self.handle, w, c, stream), "owq_dequant")
        return (w, c) if with_codes else w

    def nbytes(self) -> dict:
        st, b = owq_layer_bytes(self.handle)
        _check(st, "owq_layer_bytes")
        return b

    def close(self):
        if getattr(self, "handle", None):
            owq_layer_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def quantize_optq(W, X, bits: int, group: int, k: int, damp: float = 0.01, stream=None) -> dict:
    """Run owq_quantize_optq (selection, parameter search, OPTQ with the weak columns last) on
    fp16 CUDA tensors W (N x K) and X (T x K); allocates the outputs."""
    import torch
    N, K = W.shape
    T = X.shape[0]
    dev = W.device
    out = {
        "codes": torch.empty((N, K), dtype=torch.uint8, device=dev),
        "scales": torch.empty((N, K // group), dtype=torch.float16, device=dev),
        "zeros": torch.empty((N, K // group), dtype=torch.float16, device=dev),
        "idx": torch.empty((k,), dtype=torch.int32, device=dev),
        "w_weak": torch.empty((N, k), dtype=torch.float16, device=dev),
    }
    _check(owq_quantize_optq(W, X, N, K, T, bits, group, k, damp, out["codes"], out["scales"], out["zeros"],
                             out["idx"] if k else None, out["w_weak"] if k else None, stream), "owq_quantize_optq")
    return out


def quantize_pack(W, X, bits: int, group: int, k: int, stream=None) -> tuple[OwqLayer, dict]:
    """owq_quantize then owq_pack (both on the GPU)."""
    q = quantize(W, X, bits, group, k, stream)
    layer = OwqLayer(q["codes"], q["scales"], q["zeros"], q["idx"], q["w_weak"], bits, group, stream)
    return layer, q


def _check_tensor(t, name: str, shape, dtype, device=None) -> None:
    """A contiguous CUDA tensor of this shape and type (ValueError otherwise)."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _raw_stream(torch, index: int) -> int:
    """The current stream's handle on device `index` (torch.cuda.current_stream builds an object
    for it, which costs more than a launch)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _run_on(torch, device, stream, fn):
    """fn(stream handle) with `device` current and, for an explicit stream (a torch stream or a
    raw handle), that stream current too, so that what fn allocates belongs to it."""
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(device):
            return _run_on(torch, device, stream, fn)
    if stream is None:
        return fn(_raw_stream(torch, index))
    ext = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(ext):
        return fn(ext.cuda_stream)


class OwqGated:
    """The gated block h = act(x Wg^T) * (x Wu^T) of two packed layers of one shape (see
    owq_gated_gemv and the calls after it in include/owq.h), with its backward pass.  act:
    "silu", "gelu" (erf) or "gelu_tanh".  Nothing is kept between calls; tensors are fp16,
    contiguous, on the layers' device, and a given output or `stream` is used as it is."""

    ACTS = {"silu": OWQ_ACT_SILU, "gelu": OWQ_ACT_GELU, "gelu_tanh": OWQ_ACT_GELU_TANH}

    def __init__(self, gate: OwqLayer, up: OwqLayer, act: str = "silu"):
        import torch
        if act not in self.ACTS:
            raise ValueError(f"act {act!r}: expected one of {sorted(self.ACTS)}")
        for what in ("N", "K", "bits", "group"):
            if getattr(gate, what) != getattr(up, what):
                raise ValueError(f"gate and up differ in {what}: {getattr(gate, what)} and {getattr(up, what)}")
        self.gate, self.up, self.act = gate, up, self.ACTS[act]
        self.N, self.K = gate.N, gate.K
        self._torch, self._half = torch, torch.float16
        self._ws_size = (0, 0)   # (M, bytes) of the last workspace

    def _rows(self, t, name: str, width: int) -> int:
        if t.dim() != 2:
            raise ValueError(f"{name}: expected 2 dimensions, got {tuple(t.shape)}")
        M = t.shape[0]
        if t.dtype != self._half or t.shape[1] != width or not t.is_cuda or not t.is_contiguous():
            _check_tensor(t, name, (M, width), self._half)
        return M

    def _with(self, t, name: str, M: int, width: int, like) -> None:
        if t.shape != (M, width) or t.dtype != self._half or t.device != like.device or not t.is_contiguous():
            _check_tensor(t, name, (M, width), self._half, like.device)

    def _out(self, t, name: str, M: int, width: int, like):
        if t is None:
            return like.new_empty((M, width))
        self._with(t, name, M, width, like)
        return t

    def _workspace(self, M: int, like):
        last, n = self._ws_size
        if last != M:
            st, n = owq_gated_workspace(self.gate.handle, self.up.handle, M)
            _check(st, "owq_gated_workspace")
            self._ws_size = (M, n)
        return like.new_empty((n,), dtype=self._torch.uint8), n

    def gemv(self, x, h=None, stream=None):
        """h for 1 to 16 tokens (x: M x K)."""
        M = self._rows(x, "x", self.K)

        def go(s):
            y = self._out(h, "h", M, self.N, x)
            _check(LIB.owq_gated_gemv(self.gate.handle, self.up.handle, self.act, x.data_ptr(), y.data_ptr(), M, s),
                   "owq_gated_gemv")
            return y
        return _run_on(self._torch, x.device, stream, go)

    def gemm(self, x, h=None, stream=None):
        """h for any number of tokens (tuned for 64 and more)."""
        M = self._rows(x, "x", self.K)

        def go(s):
            ws, n = self._workspace(M, x)
            y = self._out(h, "h", M, self.N, x)
            _check(LIB.owq_gated_gemm(self.gate.handle, self.up.handle, self.act, x.data_ptr(), y.data_ptr(), M, ws.data_ptr(), n, s),
                   "owq_gated_gemm")
            return y
        return _run_on(self._torch, x.device, stream, go)

    def _grad(self, x, dh, dgate, dup, M, ws, n, s):
        g, u = self._out(dgate, "dgate", M, self.N, x), self._out(dup, "dup", M, self.N, x)
        _check(LIB.owq_gated_grad(self.gate.handle, self.up.handle, self.act, x.data_ptr(), dh.data_ptr(), g.data_ptr(),
                                  u.data_ptr(), M, ws.data_ptr(), n, s), "owq_gated_grad")
        return g, u

    def _input_grad(self, dgate, dup, dx, M, ws, n, s):
        d = self._out(dx, "dx", M, self.K, dgate)
        _check(LIB.owq_gated_input_grad(self.gate.handle, self.up.handle, dgate.data_ptr(), dup.data_ptr(), d.data_ptr(), M,
                                        ws.data_ptr(), n, s), "owq_gated_input_grad")
        return d

    def grad(self, x, dh, dgate=None, dup=None, stream=None):
        """(dgate, dup): the gradients of x Wg^T and x Wu^T, recomputed from x."""
        M = self._rows(x, "x", self.K)
        self._with(dh, "dh", M, self.N, x)
        return _run_on(self._torch, x.device, stream, lambda s: self._grad(x, dh, dgate, dup, M, *self._workspace(M, x), s))

    def input_grad(self, dgate, dup, dx=None, stream=None):
        """dx = dgate Wg + dup Wu."""
        M = self._rows(dgate, "dgate", self.N)
        self._with(dup, "dup", M, self.N, dgate)
        return _run_on(self._torch, dgate.device, stream,
                       lambda s: self._input_grad(dgate, dup, dx, M, *self._workspace(M, dgate), s))

    def backward(self, x, dh, dx=None, dgate=None, dup=None, stream=None):
        """(dx, dgate, dup) from the gradient dh of h (up to 32 tokens dx comes from dgate and dup
        before their rounding, beyond it is input_grad(dgate, dup)).  The weak blocks' gradients follow with
        gate.weak_grad(x, dgate) and up.weak_grad(x, dup)."""
        M = self._rows(x, "x", self.K)
        self._with(dh, "dh", M, self.N, x)

        def go(s):
            ws, n = self._workspace(M, x)
            g, u, d = self._out(dgate, "dgate", M, self.N, x), self._out(dup, "dup", M, self.N, x), self._out(dx, "dx", M, self.K, x)
            _check(LIB.owq_gated_backward(self.gate.handle, self.up.handle, self.act, x.data_ptr(), dh.data_ptr(), g.data_ptr(),
                                          u.data_ptr(), d.data_ptr(), M, ws.data_ptr(), n, s), "owq_gated_backward")
            return d, g, u
        return _run_on(self._torch, x.device, stream, go)


class OwqGradClip:
    """The gradient tensors that a step clips together (see owq_clip_create in include/owq.h):
    fp32, fp16 or bf16, contiguous, on one device.  `outs` takes the clipped values (None: in
    place).  Calling it with max_norm returns the global norm, a device tensor of one fp32.

    The list holds the tensors' addresses: a step refills the same tensors (weak_grad(..., dw=t));
    gradients that are made anew each step want clip_grads, which makes a list for one call.  Calls
    of one list must be ordered (one stream, or synchronised).  A norm that is not finite clips
    nothing: the caller reads it and skips the step (torch's clip_grad_norm_ would write zeros or
    NaN)."""

    def __init__(self, grads, outs=None, stream=None):
        import torch
        self.handle = None
        self._torch = torch
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        kinds = {torch.float32: OWQ_F32, torch.float16: OWQ_F16, torch.bfloat16: OWQ_BF16}
        if len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.grads)} gradients and {len(self.outs)} outputs")
        self.device = self.grads[0].device if self.grads else torch.device("cuda", torch.cuda.current_device())
        table = (OwqGrad * max(1, len(self.grads)))()
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if g.dtype not in kinds:
                raise ValueError(f"gradient {i}: {g.dtype}, expected float32, float16 or bfloat16")
            _check_tensor(g, f"gradient {i}", g.shape, g.dtype, self.device)
            if o is not g:
                _check_tensor(o, f"output {i}", g.shape, g.dtype, self.device)
            table[i] = OwqGrad(g.data_ptr(), o.data_ptr(), g.numel(), kinds[g.dtype])
        st, self.handle = _run_on(torch, self.device, stream, lambda s: owq_clip_create(table, len(self.grads), s))
        _check(st, "owq_clip_create")

    def __call__(self, max_norm: float, norm=None, stream=None):
        torch = self._torch

        def go(s):
            n = torch.empty(1, dtype=torch.float32, device=self.device) if norm is None else norm
            if norm is not None:
                _check_tensor(n, "norm", (1,), torch.float32, self.device)
            _check(LIB.owq_clip_grads(self.handle, max_norm, n.data_ptr(), s), "owq_clip_grads")
            return n
        return _run_on(torch, self.device, stream, go)

    def close(self):
        if getattr(self, "handle", None):
            owq_clip_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def clip_grads(grads, max_norm: float, outs=None, stream=None):
    """OwqGradClip for one call: returns the norm (synchronises: the list is made and released)."""
    clip = OwqGradClip(grads, outs, stream)
    norm = clip(max_norm, stream=stream)
    clip.close()
    return norm
