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
OK, EINVAL, EALIGN, EUNSUPPORTED, EHIP, EABI = 0, -1, -2, -3, -4, -5

SYMBOLS = ("demo_abi_version", "demo_strerror", "demo_payload_layout", "demo_encode",
           "demo_decode_apply", "demo_random_select", "demo_encode_adamw", "demo_decode_apply_adamw",
           "demo_payload_validate", "demo_dropout", "demo_dropout_backward", "demo_block_layout",
           "demo_block_quantize", "demo_block_workspace", "demo_block_matmul")


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
        for name in ("demo_dropout", "demo_dropout_backward", "demo_block_layout", "demo_block_quantize",
                     "demo_block_workspace", "demo_block_matmul"):
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
