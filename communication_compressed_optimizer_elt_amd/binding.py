"""ctypes binding of libdemo (include/demo.h): argument marshalling only.

Every computation runs in the HIP kernels of libdemo.so; this module turns
PyTorch tensors into device pointers and the current HIP stream, checks that
each tensor is a contiguous device tensor of the dtype and size the call
reads or writes (so no kernel can run past it), and raises on error codes.
There is no fallback: if libdemo.so is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdemo.so")

ABI_VERSION = 1
CHUNK = 32
SCHEME_DCT, SCHEME_RANDOM, SCHEME_STRIDE, SCHEME_DILOCO = 0, 1, 2, 3
VAL_TERNARY, VAL_F16, VAL_F32 = 0, 1, 2
DTYPE_F32, DTYPE_F16, DTYPE_BF16 = 0, 1, 2
FMT_E4M3, FMT_E5M2 = 0, 1
BLOCK = 128
BLOCK_MAX_K = 1 << 22
BLOCK_MAX_WORKSPACE = 64 << 20
NORM_MAX_COLS = 16384
MAX_TENSORS = 65536
MX_BLOCK = 32
OK, EINVAL, EALIGN, EUNSUPPORTED, EHIP, EABI = 0, -1, -2, -3, -4, -5

SYMBOLS = ("demo_abi_version", "demo_strerror", "demo_payload_layout", "demo_encode",
           "demo_decode_apply", "demo_random_select", "demo_encode_adamw", "demo_decode_apply_adamw",
           "demo_payload_validate", "demo_dropout", "demo_dropout_backward", "demo_block_layout",
           "demo_block_quantize", "demo_block_workspace", "demo_block_matmul", "demo_rms_norm",
           "demo_rms_norm_workspace", "demo_rms_norm_backward", "demo_grad_workspace", "demo_grad_norm",
           "demo_grad_clip", "demo_mx_layout", "demo_mx_quantize", "demo_mx_dequantize", "demo_mx_workspace",
           "demo_mx_matmul")


class DemoError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


class demo_cfg(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("scheme", ctypes.c_uint32),
        ("chunk", ctypes.c_uint32),
        ("k", ctypes.c_uint32),
        ("period", ctypes.c_uint32),
        ("sign", ctypes.c_uint32),
        ("value_fmt", ctypes.c_uint32),
        ("beta", ctypes.c_float),
        ("lr", ctypes.c_float),
        ("reserved", ctypes.c_uint32),
        ("seed", ctypes.c_uint64),
        ("step", ctypes.c_uint64),
        ("chunk_offset", ctypes.c_uint64),
    ]


class demo_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("idx_off", "idx_bytes", "nz_off", "neg_off", "plane_bytes",
                                                "val_off", "val_bytes", "total_bytes")]

    def as_dict(self) -> dict:
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class demo_adamw(ctypes.Structure):
    _fields_ = [("beta2", ctypes.c_float), ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]


class demo_dropout_cfg(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("p", ctypes.c_float), ("site", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("seed", ctypes.c_uint64), ("step", ctypes.c_uint64),
                ("chunk_offset", ctypes.c_uint64)]


class demo_operand(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("pitch", "scale_off", "scale_pitch", "total_bytes")]

    def as_dict(self) -> dict:
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class demo_block_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("abi_version", "fmt", "tile", "dtype")]


class demo_product_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("abi_version", "fmt_a", "fmt_b", "dtype")]


class demo_norm_cfg(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_uint32), ("fmt", ctypes.c_uint32),
                ("eps", ctypes.c_float)]


class demo_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_elems", ctypes.c_uint64), ("dtype", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class demo_mx_cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("abi_version", "tile", "dtype", "reserved")]


@dataclass
class Dropout:
    """Python view of demo_dropout_cfg."""

    p: float = 0.1
    seed: int = 0
    step: int = 0
    site: int = 0
    chunk_offset: int = 0
    abi_version: int = ABI_VERSION
    reserved: int = 0

    def c(self) -> demo_dropout_cfg:
        return demo_dropout_cfg(self.abi_version, self.p, self.site, self.reserved, self.seed, self.step,
                                self.chunk_offset)


@dataclass
class Block:
    """Python view of demo_block_cfg; the source's type comes from the tensor."""

    fmt: int = FMT_E4M3
    tile: int = 0
    abi_version: int = ABI_VERSION

    def c(self, dtype: int) -> demo_block_cfg:
        return demo_block_cfg(self.abi_version, self.fmt, self.tile, dtype)


@dataclass
class Product:
    """Python view of demo_product_cfg; the result's type comes from the tensor."""

    fmt_a: int = FMT_E4M3
    fmt_b: int = FMT_E4M3
    abi_version: int = ABI_VERSION

    def c(self, dtype: int = DTYPE_F32) -> demo_product_cfg:
        return demo_product_cfg(self.abi_version, self.fmt_a, self.fmt_b, dtype)


@dataclass
class Norm:
    """Python view of demo_norm_cfg; the matrices' type comes from the tensors."""

    eps: float = 1e-6
    fmt: int = FMT_E4M3
    abi_version: int = ABI_VERSION

    def c(self, dtype: int = DTYPE_F32) -> demo_norm_cfg:
        return demo_norm_cfg(self.abi_version, dtype, self.fmt, self.eps)


@dataclass
class Mx:
    """Python view of demo_mx_cfg; the matrix' type comes from the tensor."""

    tile: int = 0
    abi_version: int = ABI_VERSION
    reserved: int = 0

    def c(self, dtype: int = DTYPE_F32) -> demo_mx_cfg:
        return demo_mx_cfg(self.abi_version, self.tile, dtype, self.reserved)


@dataclass
class AdamW:
    """Python view of demo_adamw (Decoupled AdamW; beta1 is Config.beta)."""

    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01
    reserved: int = 0

    def c(self) -> demo_adamw:
        return demo_adamw(self.beta2, self.eps, self.weight_decay, self.reserved)


@dataclass
class Config:
    """Python view of demo_cfg."""

    scheme: int = SCHEME_DCT
    k: int = 1
    period: int = 16
    sign: int = 1
    value_fmt: int = VAL_TERNARY
    beta: float = 0.9
    lr: float = 1e-3
    seed: int = 0
    step: int = 0
    chunk_offset: int = 0
    chunk: int = CHUNK
    abi_version: int = ABI_VERSION
    reserved: int = 0

    def c(self) -> demo_cfg:
        return demo_cfg(self.abi_version, self.scheme, self.chunk, self.k, self.period, self.sign,
                        self.value_fmt, self.beta, self.lr, self.reserved, self.seed, self.step,
                        self.chunk_offset)


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built (run __graft_entry__.build())")
        # torch brings a HIP runtime of its own: loaded first, libdemo binds to it;
        # loaded second, there would be two, and no launch on torch's streams works
        try:
            import torch  # noqa: F401
        except ImportError:  # raw addresses and the calls that need no GPU
            pass
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        L.demo_abi_version.argtypes = []
        L.demo_abi_version.restype = ctypes.c_int
        L.demo_strerror.argtypes = [ctypes.c_int]
        L.demo_strerror.restype = ctypes.c_char_p
        L.demo_payload_layout.argtypes = [ctypes.POINTER(demo_cfg), ctypes.c_uint64, ctypes.POINTER(demo_layout)]
        L.demo_payload_layout.restype = ctypes.c_int
        L.demo_encode.argtypes = [ctypes.POINTER(demo_cfg), ctypes.c_uint64, P, P, P, P, P]
        L.demo_encode.restype = ctypes.c_int
        L.demo_decode_apply.argtypes = [ctypes.POINTER(demo_cfg), ctypes.c_uint64, P, P, ctypes.c_uint64,
                                        ctypes.c_uint32, P]
        L.demo_decode_apply.restype = ctypes.c_int
        L.demo_random_select.argtypes = [ctypes.POINTER(demo_cfg), ctypes.c_uint64, ctypes.c_uint64,
                                         ctypes.c_uint64, P, P]
        L.demo_random_select.restype = ctypes.c_int
        L.demo_encode_adamw.argtypes = [ctypes.POINTER(demo_cfg), ctypes.POINTER(demo_adamw), ctypes.c_uint64,
                                        P, P, P, P, P, P]
        L.demo_encode_adamw.restype = ctypes.c_int
        L.demo_decode_apply_adamw.argtypes = [ctypes.POINTER(demo_cfg), ctypes.POINTER(demo_adamw),
                                              ctypes.c_uint64, P, P, P, ctypes.c_uint64, ctypes.c_uint32, P]
        L.demo_decode_apply_adamw.restype = ctypes.c_int
        L.demo_payload_validate.argtypes = [ctypes.POINTER(demo_cfg), ctypes.c_uint64, P, P, P]
        L.demo_payload_validate.restype = ctypes.c_int
        U32, U64 = ctypes.c_uint32, ctypes.c_uint64
        drop, prod = ctypes.POINTER(demo_dropout_cfg), ctypes.POINTER(demo_product_cfg)
        L.demo_dropout.argtypes = [drop, U32, U64, P, P, P, P]
        L.demo_dropout_backward.argtypes = [drop, U32, U64, P, P, P]
        L.demo_block_layout.argtypes = [U64, U64, ctypes.POINTER(demo_operand)]
        L.demo_block_quantize.argtypes = [ctypes.POINTER(demo_block_cfg), U64, U64, P, U64, drop, P, P, P]
        L.demo_block_workspace.argtypes = [prod, U64, U64, U64, ctypes.POINTER(U64)]
        L.demo_block_matmul.argtypes = [prod, U64, U64, U64, P, P, P, U64, P, U64, drop, P, U64, P]
        norm, mx = ctypes.POINTER(demo_norm_cfg), ctypes.POINTER(demo_mx_cfg)
        tensors = ctypes.POINTER(demo_tensor)
        L.demo_rms_norm.argtypes = [norm, U64, U64, P, U64, P, U64, P, P, U64, P, U64, P, P, P, P]
        L.demo_rms_norm_workspace.argtypes = [norm, U64, U64, ctypes.POINTER(U64)]
        L.demo_rms_norm_backward.argtypes = [norm, U64, U64, P, U64, P, U64, P, P, P, U64, P, U64, P, P, P, U64, P]
        L.demo_grad_workspace.argtypes = [U32, tensors, ctypes.POINTER(U64)]
        L.demo_grad_norm.argtypes = [U32, tensors, P, P, U64, P]
        L.demo_grad_clip.argtypes = [U32, tensors, tensors, P, ctypes.c_double, P, P]
        L.demo_mx_layout.argtypes = [U64, U64, ctypes.POINTER(demo_operand)]
        L.demo_mx_quantize.argtypes = [mx, U64, U64, P, U64, drop, P, P, P]
        L.demo_mx_dequantize.argtypes = [mx, U64, U64, P, P, U64, P]
        L.demo_mx_workspace.argtypes = [mx, U64, U64, U64, ctypes.POINTER(U64)]
        L.demo_mx_matmul.argtypes = [mx, U64, U64, U64, P, P, P, U64, P, U64, drop, P, U64, P]
        for name in SYMBOLS[SYMBOLS.index("demo_dropout"):]:
            getattr(L, name).restype = ctypes.c_int
        if L.demo_abi_version() != ABI_VERSION:
            raise RuntimeError("libdemo.so ABI version mismatch")
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().demo_strerror(code).decode()


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise DemoError(rc, what)


def _buf(t, what: str, nbytes: int, fp32: bool = False, elem: int = 0) -> int | None:
    """Address of t after checking that the kernels stay inside it: a
    contiguous device tensor of at least nbytes bytes (float32 where fp32,
    elements of `elem` bytes where given).  None stays None; an int is taken
    as a raw device address, unchecked."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if fp32 and str(t.dtype) != "torch.float32":
        raise TypeError(f"{what}: expected float32, got {t.dtype}")
    if elem and t.element_size() != elem:
        raise TypeError(f"{what}: expected {elem}-byte elements, got {t.dtype}")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{what}: holds {have} bytes, the call needs {nbytes}")
    return t.data_ptr()


def _payload_bytes(c, n_elems: int) -> int:
    """One replica's payload size, 0 if the configuration is invalid (the call
    itself then returns the error code)."""
    out = demo_layout()
    if lib().demo_payload_layout(ctypes.byref(c), max(int(n_elems), 0), ctypes.byref(out)) != OK:
        return 0
    return int(out.total_bytes)


def _sends(c) -> bool:
    """Whether this step writes and reads payloads (DiLoCo only on sync steps)."""
    return c.scheme != SCHEME_DILOCO or (c.period >= 1 and c.step % c.period == c.period - 1)


_current = None  # device -> the handle of its current stream
_device = None  # () -> the current device


def _look_up() -> None:
    """The calls behind torch's own: making a Stream object takes 2.7 us."""
    global _current, _device
    import torch

    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _current = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _stream(stream, device: int | None = None) -> int | None:
    """Handle of a stream; None: the current one of `device`, or of the current device."""
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _current is None:
        _look_up()
    if device is None:
        import torch

        device = torch.cuda.current_device()
    return _current(device)


def _cfg(cfg) -> demo_cfg:
    return cfg.c() if isinstance(cfg, Config) else cfg


# --------------------------------------------------------------------------- #
# the C ABI, one Python function per entry point                              #
# --------------------------------------------------------------------------- #

def demo_abi_version() -> int:
    return int(lib().demo_abi_version())


def demo_strerror(code: int) -> str:
    return strerror(code)


def demo_payload_layout(cfg, n_elems: int) -> dict:
    out = demo_layout()
    c = _cfg(cfg)
    _check(lib().demo_payload_layout(ctypes.byref(c), n_elems, ctypes.byref(out)), "demo_payload_layout")
    return out.as_dict()


def demo_encode(cfg, n_elems: int, grad, momentum, payload_out, q_out=None, stream=None) -> None:
    c = _cfg(cfg)
    nb = 4 * max(int(n_elems), 0)
    pb = _payload_bytes(c, n_elems) if _sends(c) else 0
    _check(lib().demo_encode(ctypes.byref(c), n_elems, _buf(grad, "grad", nb, True),
                             _buf(momentum, "momentum", nb, True), _buf(payload_out, "payload_out", pb),
                             _buf(q_out, "q_out", nb, True), _stream(stream)), "demo_encode")


def demo_decode_apply(cfg, n_elems: int, params, payloads, stride: int, R: int, stream=None) -> None:
    c = _cfg(cfg)
    nb = 4 * max(int(n_elems), 0)
    pb = (max(int(R), 1) - 1) * int(stride) + _payload_bytes(c, n_elems) if _sends(c) else 0
    _check(lib().demo_decode_apply(ctypes.byref(c), n_elems, _buf(params, "params", nb, True),
                                   _buf(payloads, "payloads", pb), stride, R, _stream(stream)), "demo_decode_apply")


def demo_random_select(cfg, seed: int, step: int, n_chunks: int, masks_out, stream=None) -> None:
    c = _cfg(cfg)
    _check(lib().demo_random_select(ctypes.byref(c), seed, step, n_chunks,
                                    _buf(masks_out, "masks_out", 4 * max(int(n_chunks), 0), elem=4),
                                    _stream(stream)), "demo_random_select")


def demo_payload_validate(cfg, n_elems: int, payload, violations_out, stream=None) -> None:
    """violations_out: device int64 tensor of at least one element; the count
    is written asynchronously on the stream."""
    c = _cfg(cfg)
    pb = _payload_bytes(c, n_elems) if _sends(c) else 0
    _check(lib().demo_payload_validate(ctypes.byref(c), n_elems, _buf(payload, "payload", pb),
                                       _buf(violations_out, "violations_out", 8, elem=8), _stream(stream)),
           "demo_payload_validate")


def demo_encode_adamw(cfg, adamw, n_elems: int, grad, moment1, moment2, payload_out, q_out=None,
                      stream=None) -> None:
    c = _cfg(cfg)
    w = adamw.c() if isinstance(adamw, AdamW) else adamw
    nb = 4 * max(int(n_elems), 0)
    pb = _payload_bytes(c, n_elems) if _sends(c) else 0
    _check(lib().demo_encode_adamw(ctypes.byref(c), ctypes.byref(w), n_elems, _buf(grad, "grad", nb, True),
                                   _buf(moment1, "moment1", nb, True), _buf(moment2, "moment2", nb, True),
                                   _buf(payload_out, "payload_out", pb), _buf(q_out, "q_out", nb, True),
                                   _stream(stream)), "demo_encode_adamw")


def demo_decode_apply_adamw(cfg, adamw, n_elems: int, params, moment2, payloads, stride: int, R: int,
                            stream=None) -> None:
    c = _cfg(cfg)
    w = adamw.c() if isinstance(adamw, AdamW) else adamw
    nb = 4 * max(int(n_elems), 0)
    pb = (max(int(R), 1) - 1) * int(stride) + _payload_bytes(c, n_elems) if _sends(c) else 0
    _check(lib().demo_decode_apply_adamw(ctypes.byref(c), ctypes.byref(w), n_elems,
                                         _buf(params, "params", nb, True), _buf(moment2, "moment2", nb, True),
                                         _buf(payloads, "payloads", pb), stride, R, _stream(stream)),
           "demo_decode_apply_adamw")


_dtypes: dict = {}  # torch dtype -> DTYPE_*


def _dtype(t, what: str) -> int:
    d = _dtypes.get(t.dtype)
    if d is None:
        import torch

        _dtypes.update({torch.float32: DTYPE_F32, torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16})
        d = _dtypes.get(t.dtype)
        if d is None:
            raise TypeError(f"{what}: expected float32, float16 or bfloat16, got {t.dtype}")
    return d


def _here(t, what: str) -> int:
    """The current device, whose stream the call is queued on: t is on it."""
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a device tensor")
    if _device is None:
        _look_up()
    dev = _device()
    if t.get_device() != dev:
        raise ValueError(f"{what}: on device {t.get_device()}, not the current one")
    return dev


def _flat(t, what: str, like, dev: int) -> int:
    """Address of a contiguous tensor on device dev with like's type and size."""
    if t.get_device() != dev:
        _here(t, what)
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if t.dtype != like.dtype:
        raise TypeError(f"{what}: expected {like.dtype}, got {t.dtype}")
    if t.numel() != like.numel():
        raise ValueError(f"{what}: holds {t.numel()} elements, not {like.numel()}")
    return t.data_ptr()


def _matrix(t, what: str, dev: int, shape=None, dtype=None) -> tuple[int, int]:
    """(address, row pitch) of a matrix on device dev with neighbouring columns."""
    if t.get_device() != dev:
        _here(t, what)
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{what}: expected a matrix{'' if shape is None else ' of %d x %d' % shape}, "
                         f"got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    rows, cols = t.shape
    pitch, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{what}: expected neighbouring columns, got stride {step}")
    if rows > 1 and pitch < cols:
        raise ValueError(f"{what}: rows overlap (row stride {pitch}, {cols} columns)")
    return t.data_ptr(), pitch if rows > 1 else max(cols, 1)


@functools.lru_cache(maxsize=1024)
def _operand_bytes(rows: int, cols: int) -> int:
    return demo_block_layout(rows, cols)["total_bytes"]


def _operand_buf(t, what: str, rows: int, cols: int, dev: int) -> int | None:
    if t is None:
        return None
    if t.get_device() != dev:
        _here(t, what)
    return _buf(t, what, _operand_bytes(rows, cols))


def _ref(c):
    return None if c is None else ctypes.byref(c.c() if isinstance(c, Dropout) else c)


def demo_dropout(cfg, x, y, residual=None, stream=None) -> None:
    """y = residual + dropout(x); x, y and residual are contiguous tensors of
    one type and size."""
    dtype, dev = _dtype(x, "x"), _here(x, "x")
    _check(lib().demo_dropout(_ref(cfg), dtype, x.numel(), _flat(x, "x", x, dev),
                              None if residual is None else _flat(residual, "residual", x, dev),
                              _flat(y, "y", x, dev), _stream(stream, dev)), "demo_dropout")


def demo_dropout_backward(cfg, dy, dx, stream=None) -> None:
    """dx = the gradient of demo_dropout for x under the same cfg."""
    dtype, dev = _dtype(dy, "dy"), _here(dy, "dy")
    _check(lib().demo_dropout_backward(_ref(cfg), dtype, dy.numel(), _flat(dy, "dy", dy, dev),
                                       _flat(dx, "dx", dy, dev), _stream(stream, dev)), "demo_dropout_backward")


def demo_block_layout(rows: int, cols: int) -> dict:
    out = demo_operand()
    _check(lib().demo_block_layout(rows, cols, ctypes.byref(out)), "demo_block_layout")
    return out.as_dict()


def demo_block_quantize(cfg, src, operand=None, operand_t=None, dropout=None, stream=None) -> None:
    """src: a matrix with neighbouring columns (rows may have a pitch);
    operand and operand_t: device buffers of demo_block_layout(rows, cols) and
    demo_block_layout(cols, rows) bytes."""
    dev = _here(src, "src")
    addr, ld = _matrix(src, "src", dev)
    rows, cols = src.shape
    c = cfg.c(_dtype(src, "src")) if isinstance(cfg, Block) else cfg
    _check(lib().demo_block_quantize(ctypes.byref(c), rows, cols, addr, ld, _ref(dropout),
                                     _operand_buf(operand, "operand", rows, cols, dev),
                                     _operand_buf(operand_t, "operand_t", cols, rows, dev), _stream(stream, dev)),
           "demo_block_quantize")


def demo_block_workspace(cfg, m: int, n: int, k: int, dtype: int = DTYPE_F32) -> int:
    """Bytes of workspace of a product whose result has the type dtype."""
    out = ctypes.c_uint64()
    c = cfg.c(dtype) if isinstance(cfg, Product) else cfg
    _check(lib().demo_block_workspace(ctypes.byref(c), m, n, k, ctypes.byref(out)), "demo_block_workspace")
    return int(out.value)


def demo_block_matmul(cfg, m: int, n: int, k: int, a, b, c, addend=None, dropout=None, workspace=None,
                      stream=None) -> None:
    """c = addend + dropout(a b^T) for operands a (m x k) and b (n x k); c and
    addend are m x n matrices of one type with neighbouring columns."""
    dev = _here(c, "c")
    addr, ldc = _matrix(c, "c", dev, (m, n))
    add, lda = (None, 0) if addend is None else _matrix(addend, "addend", dev, (m, n), c.dtype)
    cc = cfg.c(_dtype(c, "c")) if isinstance(cfg, Product) else cfg
    work, have = None, 0
    if workspace is not None:
        if workspace.get_device() != dev:
            _here(workspace, "workspace")
        work, have = _buf(workspace, "workspace", 0), workspace.numel() * workspace.element_size()
    _check(lib().demo_block_matmul(ctypes.byref(cc), m, n, k, _operand_buf(a, "a", m, k, dev),
                                   _operand_buf(b, "b", n, k, dev), addr, ldc, add, lda, _ref(dropout), work, have,
                                   _stream(stream, dev)), "demo_block_matmul")


def _vector(t, what: str, dev: int, n: int) -> int | None:
    """Address of a contiguous fp32 vector of n elements on device dev."""
    if t is None:
        return None
    if t.get_device() != dev:
        _here(t, what)
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if _dtype(t, what) != DTYPE_F32:
        raise TypeError(f"{what}: expected float32, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{what}: holds {t.numel()} elements, not {n}")
    return t.data_ptr()


def _maybe_matrix(t, what: str, dev: int, like) -> tuple[int | None, int]:
    return (None, 0) if t is None else _matrix(t, what, dev, tuple(like.shape), like.dtype)


def _workspace(t, dev: int) -> tuple[int | None, int]:
    if t is None:
        return None, 0
    if t.get_device() != dev:
        _here(t, "workspace")
    if not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def demo_rms_norm(cfg, x, weight, y=None, residual=None, h=None, rstd=None, operand=None, operand_t=None,
                  stream=None) -> None:
    """h = residual + x, y = h / rms(h) * weight.  x, residual, h and y are
    matrices of one type and size with neighbouring columns; weight and rstd
    fp32 vectors; operand and operand_t device buffers of
    demo_block_layout(rows, cols) and demo_block_layout(cols, rows) bytes."""
    dev = _here(x, "x")
    addr, ld = _matrix(x, "x", dev)
    rows, cols = x.shape
    res, ld_res = _maybe_matrix(residual, "residual", dev, x)
    to_h, ld_h = _maybe_matrix(h, "h", dev, x)
    to_y, ld_y = _maybe_matrix(y, "y", dev, x)
    c = cfg.c(_dtype(x, "x")) if isinstance(cfg, Norm) else cfg
    _check(lib().demo_rms_norm(ctypes.byref(c), rows, cols, addr, ld, res, ld_res, _vector(weight, "weight", dev, cols),
                               to_h, ld_h, to_y, ld_y, _vector(rstd, "rstd", dev, rows),
                               _operand_buf(operand, "operand", rows, cols, dev),
                               _operand_buf(operand_t, "operand_t", cols, rows, dev), _stream(stream, dev)),
           "demo_rms_norm")


def demo_rms_norm_workspace(cfg, rows: int, cols: int) -> int:
    """Bytes of workspace of demo_rms_norm_backward where dweight is wanted."""
    out = ctypes.c_uint64()
    c = cfg.c() if isinstance(cfg, Norm) else cfg
    _check(lib().demo_rms_norm_workspace(ctypes.byref(c), rows, cols, ctypes.byref(out)), "demo_rms_norm_workspace")
    return int(out.value)


def demo_rms_norm_backward(cfg, dy, h, weight, rstd, dx, dresidual=None, dweight=None, addend=None, workspace=None,
                           stream=None) -> None:
    """dx and dweight = addend + ... of demo_rms_norm, from its h and rstd (h is
    x where there was no residual).  dy, h, dresidual and dx are matrices of one
    type and size with neighbouring columns, the rest fp32 vectors."""
    dev = _here(dy, "dy")
    addr, ld = _matrix(dy, "dy", dev)
    rows, cols = dy.shape
    at_h, ld_h = _matrix(h, "h", dev, (rows, cols), dy.dtype)
    res, ld_res = _maybe_matrix(dresidual, "dresidual", dev, dy)
    to, ld_dx = _matrix(dx, "dx", dev, (rows, cols), dy.dtype)
    c = cfg.c(_dtype(dy, "dy")) if isinstance(cfg, Norm) else cfg
    work, have = _workspace(workspace, dev)
    _check(lib().demo_rms_norm_backward(ctypes.byref(c), rows, cols, addr, ld, at_h, ld_h,
                                        _vector(weight, "weight", dev, cols), _vector(rstd, "rstd", dev, rows), res,
                                        ld_res, to, ld_dx, _vector(dweight, "dweight", dev, cols),
                                        _vector(addend, "addend", dev, cols), work, have, _stream(stream, dev)),
           "demo_rms_norm_backward")


class Tensors:
    """A list of gradients for demo_grad_norm and demo_grad_clip: contiguous
    device tensors of one device, held here with the table that the library
    reads.  A program makes it once for tensors that stay where they are."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.device = None
        if len(self.tensors) > MAX_TENSORS:
            raise ValueError(f"tensors: {len(self.tensors)} of them, at most {MAX_TENSORS}")
        self.table = (demo_tensor * max(len(self.tensors), 1))()
        for i, t in enumerate(self.tensors):
            what = f"tensors[{i}]"
            if not t.is_cuda:
                raise ValueError(f"{what}: expected a device tensor")
            if self.device is None:
                self.device = t.get_device()
            if t.get_device() != self.device:
                raise ValueError(f"{what}: on device {t.get_device()}, tensors[0] on {self.device}")
            if not t.is_contiguous():
                raise ValueError(f"{what}: expected a contiguous tensor")
            self.table[i] = demo_tensor(t.data_ptr() or None, t.numel(), _dtype(t, what), 0)

    def __len__(self) -> int:
        return len(self.tensors)

    def check(self, what: str, dev: int) -> None:
        if self.device not in (None, dev):
            raise ValueError(f"{what}: on device {self.device}, not the current one")


def _tensors(t, what: str, dev: int) -> Tensors:
    t = t if isinstance(t, Tensors) else Tensors(t)
    t.check(what, dev)
    return t


@functools.lru_cache(maxsize=None)
def _torch():
    import torch

    return torch


def _scalar(t, what: str, dev: int, dtype: str) -> int | None:
    """Address of a device tensor whose first element a call reads or writes."""
    if t is None:
        return None
    if t.get_device() != dev:
        _here(t, what)
    if t.dtype != getattr(_torch(), dtype):
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.numel() < 1:
        raise ValueError(f"{what}: holds nothing, the call needs one element")
    return t.data_ptr()


def demo_grad_workspace(tensors) -> int:
    """Bytes of workspace of demo_grad_norm for a list of tensors."""
    out = ctypes.c_uint64()
    t = tensors if isinstance(tensors, Tensors) else Tensors(tensors)
    _check(lib().demo_grad_workspace(len(t), t.table, ctypes.byref(out)), "demo_grad_workspace")
    return int(out.value)


def demo_grad_norm(tensors, sumsq, workspace=None, stream=None) -> None:
    """sumsq[0] = sum of the squares of all elements: tensors is a Tensors or a
    list of tensors, sumsq a float64 device tensor."""
    dev = _here(sumsq, "sumsq")
    t = _tensors(tensors, "tensors", dev)
    work, have = _workspace(workspace, dev)
    _check(lib().demo_grad_norm(len(t), t.table, _scalar(sumsq, "sumsq", dev, "float64"), work, have,
                                _stream(stream, dev)), "demo_grad_norm")


def demo_grad_clip(src, sumsq, max_norm: float, dst=None, norm=None, stream=None) -> None:
    """dst[i] = min(1, max_norm / (sqrt(sumsq[0]) + 1e-6)) * src[i] for two lists
    (Tensors or lists) of tensors; dst None: in place.  norm[0] (float32) =
    sqrt(sumsq[0])."""
    dev = _here(sumsq, "sumsq")
    s = _tensors(src, "src", dev)
    d = None if dst is None else _tensors(dst, "dst", dev)
    if d is not None and len(d) != len(s):
        raise ValueError(f"dst: {len(d)} tensors, src has {len(s)}")
    _check(lib().demo_grad_clip(len(s), s.table, None if d is None else d.table,
                                _scalar(sumsq, "sumsq", dev, "float64"), max_norm,
                                _scalar(norm, "norm", dev, "float32"), _stream(stream, dev)), "demo_grad_clip")


def demo_mx_layout(rows: int, cols: int) -> dict:
    out = demo_operand()
    _check(lib().demo_mx_layout(rows, cols, ctypes.byref(out)), "demo_mx_layout")
    return out.as_dict()


@functools.lru_cache(maxsize=1024)
def _mx_bytes(rows: int, cols: int) -> int:
    return demo_mx_layout(rows, cols)["total_bytes"]


def _mx_buf(t, what: str, rows: int, cols: int, dev: int) -> int | None:
    if t is None:
        return None
    if t.get_device() != dev:
        _here(t, what)
    return _buf(t, what, _mx_bytes(rows, cols))


def demo_mx_quantize(cfg, src, operand=None, operand_t=None, dropout=None, stream=None) -> None:
    """src: a matrix with neighbouring columns (rows may have a pitch);
    operand and operand_t: device buffers of demo_mx_layout(rows, cols) and
    demo_mx_layout(cols, rows) bytes."""
    dev = _here(src, "src")
    addr, ld = _matrix(src, "src", dev)
    rows, cols = src.shape
    c = cfg.c(_dtype(src, "src")) if isinstance(cfg, Mx) else cfg
    _check(lib().demo_mx_quantize(ctypes.byref(c), rows, cols, addr, ld, _ref(dropout),
                                  _mx_buf(operand, "operand", rows, cols, dev),
                                  _mx_buf(operand_t, "operand_t", cols, rows, dev), _stream(stream, dev)),
           "demo_mx_quantize")


def demo_mx_dequantize(operand, dst, stream=None) -> None:
    """dst (a matrix with neighbouring columns) = the values of the operand of
    its size."""
    dev = _here(dst, "dst")
    addr, ld = _matrix(dst, "dst", dev)
    rows, cols = dst.shape
    c = demo_mx_cfg(ABI_VERSION, 0, _dtype(dst, "dst"), 0)
    _check(lib().demo_mx_dequantize(ctypes.byref(c), rows, cols, _mx_buf(operand, "operand", rows, cols, dev), addr, ld,
                                    _stream(stream, dev)), "demo_mx_dequantize")


def demo_mx_workspace(cfg, m: int, n: int, k: int, dtype: int = DTYPE_F32) -> int:
    """Bytes of workspace of a product whose result has the type dtype."""
    out = ctypes.c_uint64()
    c = cfg.c(dtype) if isinstance(cfg, Mx) else cfg
    _check(lib().demo_mx_workspace(ctypes.byref(c), m, n, k, ctypes.byref(out)), "demo_mx_workspace")
    return int(out.value)


def demo_mx_matmul(cfg, m: int, n: int, k: int, a, b, c, addend=None, dropout=None, workspace=None,
                   stream=None) -> None:
    """c = addend + dropout(a b^T) for 4-bit operands a (m x k) and b (n x k); c
    and addend are m x n matrices of one type with neighbouring columns."""
    dev = _here(c, "c")
    addr, ldc = _matrix(c, "c", dev, (m, n))
    add, lda = _maybe_matrix(addend, "addend", dev, c)
    cc = cfg.c(_dtype(c, "c")) if isinstance(cfg, Mx) else cfg
    work, have = _workspace(workspace, dev)
    _check(lib().demo_mx_matmul(ctypes.byref(cc), m, n, k, _mx_buf(a, "a", m, k, dev), _mx_buf(b, "b", n, k, dev),
                                addr, ldc, add, lda, _ref(dropout), work, have, _stream(stream, dev)),
           "demo_mx_matmul")


# raw return codes (tests of the boundary's validation)
def raw_encode(cfg, n_elems, grad, momentum, payload_out, q_out=None, stream=0) -> int:
    c = _cfg(cfg)
    return int(lib().demo_encode(ctypes.byref(c), n_elems, grad, momentum, payload_out, q_out, stream))


def raw_decode_apply(cfg, n_elems, params, payloads, stride, R, stream=0) -> int:
    c = _cfg(cfg)
    return int(lib().demo_decode_apply(ctypes.byref(c), n_elems, params, payloads, stride, R, stream))


def raw_random_select(cfg, seed, step, n_chunks, masks_out, stream=0) -> int:
    c = _cfg(cfg)
    return int(lib().demo_random_select(ctypes.byref(c), seed, step, n_chunks, masks_out, stream))


def raw_payload_layout(cfg, n_elems) -> tuple[int, dict]:
    out = demo_layout()
    c = _cfg(cfg)
    rc = int(lib().demo_payload_layout(ctypes.byref(c), n_elems, ctypes.byref(out)))
    return rc, out.as_dict()


def raw_encode_adamw(cfg, adamw, n_elems, grad, moment1, moment2, payload_out, q_out=None, stream=0) -> int:
    c = _cfg(cfg)
    w = adamw.c() if isinstance(adamw, AdamW) else adamw
    wp = None if adamw is None else ctypes.byref(w)
    return int(lib().demo_encode_adamw(ctypes.byref(c), wp, n_elems, grad, moment1, moment2, payload_out, q_out,
                                       stream))


def raw_decode_apply_adamw(cfg, adamw, n_elems, params, moment2, payloads, stride, R, stream=0) -> int:
    c = _cfg(cfg)
    w = adamw.c() if isinstance(adamw, AdamW) else adamw
    wp = None if adamw is None else ctypes.byref(w)
    return int(lib().demo_decode_apply_adamw(ctypes.byref(c), wp, n_elems, params, moment2, payloads, stride, R,
                                             stream))


def raw_payload_validate(cfg, n_elems, payload, violations_out, stream=0) -> int:
    c = _cfg(cfg)
    return int(lib().demo_payload_validate(ctypes.byref(c), n_elems, payload, violations_out, stream))


def raw_dropout(cfg, dtype, n_elems, x, residual, y, stream=0) -> int:
    return int(lib().demo_dropout(_ref(cfg), dtype, n_elems, x, residual, y, stream))


def raw_dropout_backward(cfg, dtype, n_elems, dy, dx, stream=0) -> int:
    return int(lib().demo_dropout_backward(_ref(cfg), dtype, n_elems, dy, dx, stream))


def raw_block_layout(rows, cols) -> tuple[int, dict]:
    out = demo_operand()
    rc = int(lib().demo_block_layout(rows, cols, ctypes.byref(out)))
    return rc, out.as_dict()


def raw_block_quantize(cfg, rows, cols, src, ld, dropout, operand, operand_t, stream=0) -> int:
    return int(lib().demo_block_quantize(None if cfg is None else ctypes.byref(cfg), rows, cols, src, ld,
                                         _ref(dropout), operand, operand_t, stream))


def raw_block_workspace(cfg, m, n, k) -> tuple[int, int]:
    out = ctypes.c_uint64()
    rc = int(lib().demo_block_workspace(None if cfg is None else ctypes.byref(cfg), m, n, k, ctypes.byref(out)))
    return rc, int(out.value)


def raw_block_matmul(cfg, m, n, k, a, b, c, ldc, addend=None, ld_addend=0, dropout=None, workspace=None,
                     workspace_bytes=0, stream=0) -> int:
    return int(lib().demo_block_matmul(None if cfg is None else ctypes.byref(cfg), m, n, k, a, b, c, ldc, addend,
                                       ld_addend, _ref(dropout), workspace, workspace_bytes, stream))


def _byref(c):
    return None if c is None else ctypes.byref(c)


def raw_rms_norm(cfg, rows, cols, x, ld_x, residual, ld_residual, weight, h=None, ld_h=0, y=None, ld_y=0, rstd=None,
                 operand=None, operand_t=None, stream=0) -> int:
    return int(lib().demo_rms_norm(_byref(cfg), rows, cols, x, ld_x, residual, ld_residual, weight, h, ld_h, y, ld_y,
                                   rstd, operand, operand_t, stream))


def raw_rms_norm_workspace(cfg, rows, cols) -> tuple[int, int]:
    out = ctypes.c_uint64()
    rc = int(lib().demo_rms_norm_workspace(_byref(cfg), rows, cols, ctypes.byref(out)))
    return rc, int(out.value)


def raw_rms_norm_backward(cfg, rows, cols, dy, ld_dy, h, ld_h, weight, rstd, dresidual, ld_dresidual, dx, ld_dx,
                          dweight=None, addend=None, workspace=None, workspace_bytes=0, stream=0) -> int:
    return int(lib().demo_rms_norm_backward(_byref(cfg), rows, cols, dy, ld_dy, h, ld_h, weight, rstd, dresidual,
                                            ld_dresidual, dx, ld_dx, dweight, addend, workspace, workspace_bytes,
                                            stream))


def raw_tensors(*entries):
    """A table of (address, elements, type[, reserved]) entries."""
    return (demo_tensor * max(len(entries), 1))(*(demo_tensor(*(e if len(e) == 4 else (*e, 0))) for e in entries))


def raw_grad_workspace(count, tensors) -> tuple[int, int]:
    out = ctypes.c_uint64()
    rc = int(lib().demo_grad_workspace(count, tensors, ctypes.byref(out)))
    return rc, int(out.value)


def raw_grad_norm(count, tensors, sumsq, workspace=None, workspace_bytes=0, stream=0) -> int:
    return int(lib().demo_grad_norm(count, tensors, sumsq, workspace, workspace_bytes, stream))


def raw_grad_clip(count, src, dst, sumsq, max_norm, norm=None, stream=0) -> int:
    return int(lib().demo_grad_clip(count, src, dst, sumsq, max_norm, norm, stream))


def raw_mx_layout(rows, cols) -> tuple[int, dict]:
    out = demo_operand()
    rc = int(lib().demo_mx_layout(rows, cols, ctypes.byref(out)))
    return rc, out.as_dict()


def raw_mx_quantize(cfg, rows, cols, src, ld, dropout, operand, operand_t, stream=0) -> int:
    return int(lib().demo_mx_quantize(_byref(cfg), rows, cols, src, ld, _ref(dropout), operand, operand_t, stream))


def raw_mx_dequantize(cfg, rows, cols, operand, dst, ld, stream=0) -> int:
    return int(lib().demo_mx_dequantize(_byref(cfg), rows, cols, operand, dst, ld, stream))


def raw_mx_workspace(cfg, m, n, k) -> tuple[int, int]:
    out = ctypes.c_uint64()
    rc = int(lib().demo_mx_workspace(_byref(cfg), m, n, k, ctypes.byref(out)))
    return rc, int(out.value)


def raw_mx_matmul(cfg, m, n, k, a, b, c, ldc, addend=None, ld_addend=0, dropout=None, workspace=None,
                  workspace_bytes=0, stream=0) -> int:
    return int(lib().demo_mx_matmul(_byref(cfg), m, n, k, a, b, c, ldc, addend, ld_addend, _ref(dropout), workspace,
                                    workspace_bytes, stream))
