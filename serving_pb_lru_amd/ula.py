"""Python binding of libula.so: argument marshalling only.

Every step of the residency path runs in the HIP kernels behind the C ABI in
include/ula.h; this module turns torch tensors and numpy arrays into pointers
and sizes, and error codes into exceptions. PyTorch supplies the device
workspace and the streams. There is no fallback: without the built library
every call raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import List, Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libula.so")

ERROR_NAMES = {0: "OK", -1: "EINVAL", -2: "ERANGE", -3: "EDUP", -4: "EHOSTFULL",
               -5: "ECAPACITY", -6: "ENOTRESIDENT", -7: "ESTATE", -8: "EHIP", -9: "EBUSY",
               -10: "ETOOBIG"}


POLICY_PBLRU, POLICY_LRU = 0, 1
PLACE_LOWEST, PLACE_RING = 0, 1


class UlaConfig(ctypes.Structure):
    _fields_ = [("num_groups", ctypes.c_int32), ("layers_per_group", ctypes.c_int32),
                ("row_bytes", ctypes.c_int32), ("ring_buckets", ctypes.c_int32),
                ("logical_capacity", ctypes.c_int32), ("gpu_slots", ctypes.c_int32),
                ("host_slots", ctypes.c_int32), ("max_sets", ctypes.c_int32),
                ("max_k", ctypes.c_int32), ("max_append", ctypes.c_int32), ("policy", ctypes.c_int32),
                ("placement", ctypes.c_int32)]


class UlaStepStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("unique", "hits", "misses", "evictions", "from_free", "invalid")]

    def as_tuple(self):
        return (self.unique, self.hits, self.misses, self.evictions, self.from_free, self.invalid)


class UlaStateHost(ctypes.Structure):
    _fields_ = [("map", ctypes.c_void_p), ("gown", ctypes.c_void_p), ("hown", ctypes.c_void_p),
                ("bitsets", ctypes.c_void_p), ("cur", ctypes.c_int32), ("flag", ctypes.c_int64),
                ("last", UlaStepStats), ("stamps", ctypes.c_void_p)]


BF16, FP16, FP32 = 0, 1, 2
ROWS_LATENT, ROWS_HEADS = 0, 1
LATENT_CHANNELS, ROPE_CHANNELS = 512, 64


class RowFormat(ctypes.Structure):
    """What a row's bytes hold (ula_row_format); see latent_rows and head_rows."""
    _fields_ = [("kind", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_tokens", ctypes.c_int32)]

    @property
    def row_bytes(self) -> int:
        return lib().ula_row_format_bytes(ctypes.byref(self))


class UlaAttendArgs(ctypes.Structure):
    _fields_ = [("rows", RowFormat), ("type", ctypes.c_int32), ("heads", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("q_set_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_set_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class UlaTreeArgs(ctypes.Structure):
    _fields_ = [("attend", UlaAttendArgs), ("nodes", ctypes.c_int32), ("q_node_stride", ctypes.c_int64),
                ("out_node_stride", ctypes.c_int64), ("drafts", ctypes.c_void_p), ("visible", ctypes.c_void_p)]


class UlaWeighArgs(ctypes.Structure):
    _fields_ = [("rows", RowFormat), ("type", ctypes.c_int32), ("nodes", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_set_stride", ctypes.c_int64),
                ("q_node_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("lse", ctypes.c_void_p),
                ("shares", ctypes.c_void_p), ("scores", ctypes.c_void_p)]


class UlaLightestArgs(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_void_p), ("capacity", ctypes.c_int32), ("ranges", ctypes.c_int32),
                ("first", ctypes.c_void_p), ("last", ctypes.c_void_p), ("count", ctypes.c_void_p), ("most", ctypes.c_int32),
                ("mark", ctypes.c_int32), ("out", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class UlaRotary(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 3), ("interleaved", ctypes.c_int32),
                ("theta", ctypes.c_double)]


class UlaPackArgs(ctypes.Structure):
    _fields_ = [("rows", RowFormat), ("type", ctypes.c_int32), ("n", ctypes.c_int32), ("layers", ctypes.c_int32),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("a_stride", ctypes.c_int64 * 4),
                ("b_stride", ctypes.c_int64 * 4), ("positions", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("rotary", UlaRotary)]


class UlaRotateArgs(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("n", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("x", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("x_stride", ctypes.c_int64 * 2), ("out_stride", ctypes.c_int64 * 2), ("positions", ctypes.c_void_p),
                ("rotary", UlaRotary)]


class UlaNormArgs(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("n", ctypes.c_int32), ("dim", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("k_heads", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("weight_type", ctypes.c_int32),
                ("eps", ctypes.c_float), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("k_out", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 2), ("k_stride", ctypes.c_int64 * 2),
                ("q_out_stride", ctypes.c_int64 * 2), ("k_out_stride", ctypes.c_int64 * 2),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("rotary", UlaRotary)]


class UlaError(RuntimeError):
    def __init__(self, code: int, where: str, text: str):
        self.code = code
        self.name = ERROR_NAMES.get(code, str(code))
        super().__init__(f"{where}: {self.name} ({text})")


_lib = None

# (name, restype, argtypes) of every symbol include/ula.h declares
SIGNATURES = [
    ("ula_device_bytes", ctypes.c_size_t, [ctypes.POINTER(UlaConfig)]),
    ("ula_host_bytes", ctypes.c_size_t, [ctypes.POINTER(UlaConfig)]),
    ("ula_init", ctypes.c_int, [ctypes.POINTER(UlaConfig), ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.c_uint64, ctypes.POINTER(ctypes.c_void_p)]),
    ("ula_init_static", ctypes.c_int, [ctypes.POINTER(UlaConfig), ctypes.c_void_p, ctypes.c_uint64,
                                       ctypes.POINTER(ctypes.c_void_p)]),
    ("ula_row_format_bytes", ctypes.c_size_t, [ctypes.POINTER(RowFormat)]),
    ("ula_pack_rows", ctypes.c_int, [ctypes.POINTER(UlaPackArgs), ctypes.c_void_p, ctypes.c_uint64]),
    ("ula_rotate", ctypes.c_int, [ctypes.POINTER(UlaRotateArgs), ctypes.c_uint64]),
    ("ula_norm_rotate", ctypes.c_int, [ctypes.POINTER(UlaNormArgs), ctypes.c_uint64]),
    ("ula_attend_bytes", ctypes.c_size_t, [ctypes.POINTER(RowFormat), ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]),
    ("ula_attend", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.c_void_p, ctypes.POINTER(UlaAttendArgs), ctypes.c_uint64]),
    ("ula_attend_tree_bytes", ctypes.c_size_t, [ctypes.POINTER(RowFormat), ctypes.c_int32, ctypes.c_int32,
                                                ctypes.c_int32, ctypes.c_int32]),
    ("ula_attend_tree", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.POINTER(UlaTreeArgs), ctypes.c_uint64]),
    ("ula_weigh", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                 ctypes.c_void_p, ctypes.POINTER(UlaWeighArgs), ctypes.c_uint64]),
    ("ula_lightest_bytes", ctypes.c_size_t, [ctypes.POINTER(UlaLightestArgs)]),
    ("ula_lightest", ctypes.c_int, [ctypes.POINTER(UlaLightestArgs), ctypes.c_uint64]),
    ("ula_fork", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                ctypes.c_uint64]),
    ("ula_rename", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.c_uint64]),
    ("ula_append", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64]),
    ("ula_release", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                   ctypes.c_uint64]),
    ("ula_step", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                ctypes.c_void_p, ctypes.c_uint64]),
    ("ula_append_step", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_void_p, ctypes.c_uint64]),
    ("ula_gather", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                  ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64]),
    ("ula_gather_layers", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_uint64]),
    ("ula_sync", ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    ("ula_export_state", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(UlaStateHost)]),
    ("ula_read_rows", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p]),
    ("ula_flag_address", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.POINTER(ctypes.c_void_p)]),
    ("ula_set_timing", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32]),
    ("ula_read_timing", ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    ("ula_read_gather_timing", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_double),
                                              ctypes.POINTER(ctypes.c_int64)]),
    ("ula_read_link_timing", ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_double),
                                            ctypes.POINTER(ctypes.c_int64)]),
    ("ula_destroy", ctypes.c_int, [ctypes.c_void_p]),
    ("ula_strerror", ctypes.c_char_p, [ctypes.c_int]),
    ("ula_host_alloc", ctypes.c_void_p, [ctypes.c_size_t]),
    ("ula_host_free", ctypes.c_int, [ctypes.c_void_p]),
]


def lib() -> ctypes.CDLL:
    """Load libula.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with serving_pb_lru_amd.build.build()")
        # torch ships its own HIP runtime under the same soname as the one this
        # library links; importing torch first makes the library bind to that
        # runtime (loaded the other way round, the process ends up with two HIP
        # runtimes and device calls fail)
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int, where: str) -> None:
    if rc != 0:
        raise UlaError(rc, where, lib().ula_strerror(rc).decode())


_DTYPES = {x: f"torch.{x}" for x in ("uint8", "int32", "int64", "float32")}


def _dev(t, dtype: str, count: int, what: str) -> int:
    """Device pointer of a contiguous CUDA tensor of `dtype` holding at least
    `count` elements; raises ValueError otherwise (the library takes plain
    pointers and would read or write past a smaller buffer)."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{what}: a CUDA tensor is required")
    if str(t.dtype) != _DTYPES[dtype]:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {_DTYPES[dtype]}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: the tensor must be contiguous")
    if t.numel() < count:
        raise ValueError(f"{what}: {t.numel()} elements, at least {count} needed")
    return t.data_ptr()


def _shaped(t, dtype: str, shape, what: str) -> int:
    """_dev for a tensor of exactly this shape: another one would be read, or written, as something else."""
    ptr = _dev(t, dtype, 0, what)
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ptr


def _sets(sel):
    """(n_sets, k) of a selection tensor [n_sets][k] or [k]."""
    return (1, sel.shape[0]) if sel.dim() == 1 else tuple(sel.shape)


def _stream(stream) -> int:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def latent_rows() -> RowFormat:
    """656-byte rows of one shared representation: 512 e4m3 channels, 64 bf16 rotary channels,
    one fp32 scale per 128 channels."""
    return RowFormat(ROWS_LATENT, 0, 0, 0)


def head_rows(kv_heads: int, head_dim: int, block_tokens: int = 1) -> RowFormat:
    """Rows of block_tokens tokens' e4m3 keys and values of every KV head, with an fp32 scale
    for each block and head."""
    fmt = RowFormat(ROWS_HEADS, kv_heads, head_dim, block_tokens)
    if not fmt.row_bytes:
        raise UlaError(-1, "head_rows", "kv_heads >= 1, head_dim 64 or 128, block_tokens 1, 2, 4, 8 or 16, "
                                        "and at most 4096 bytes a row")
    return fmt


_TYPES = {"torch.bfloat16": BF16, "torch.float16": FP16, "torch.float32": FP32}


def _tensor(t, shape, what: str, types=(BF16, FP16, FP32)):
    """(pointer, type code, strides) of a CUDA tensor of the given shape (None: any size)
    whose last dimension is contiguous."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{what}: a CUDA tensor is required")
    code = _TYPES.get(str(t.dtype))
    if code not in types:
        raise ValueError(f"{what}: dtype {t.dtype} is not supported")
    real, strides = t.shape, t.stride()
    if len(real) != len(shape):
        raise ValueError(f"{what}: shape {tuple(real)}, expected {tuple(shape)} (None: any)")
    for n, m in zip(shape, real):
        if n is not None and n != m:
            raise ValueError(f"{what}: shape {tuple(real)}, expected {tuple(shape)} (None: any)")
    if strides[-1] != 1 and real[-1] > 1 and t.numel():
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), code, strides


def _host_ints(x, what: str) -> np.ndarray:
    """A one-dimensional int32 array of integers that fit it."""
    if isinstance(x, np.ndarray) and x.dtype == np.int32 and x.ndim == 1 and x.flags.c_contiguous:
        return x
    y = np.asarray(x)
    if y.ndim != 1 or (y.size and y.dtype.kind not in "iu"):
        raise ValueError(f"{what}: a list of integers is required")
    z = np.ascontiguousarray(y, dtype=np.int32)
    if (z != y).any():
        raise ValueError(f"{what}: an integer outside 32 bits")
    return z


def _same_device(first, *others) -> None:
    device = first.device
    for t in others:
        if t is not None and t.device != device:
            raise ValueError(f"tensors on {device} and {t.device}")


def _no_gradient(what: str, *tensors) -> None:
    """Refuses tensors whose history autograd would expect the result to carry: these calls record none."""
    import torch
    if torch.is_grad_enabled():
        for t in tensors:
            if getattr(t, "requires_grad", False):
                raise ValueError(f"{what}: a tensor requires a gradient, which this call does not record "
                                 "(detach it, or call under torch.no_grad())")


class _On:
    """Makes a tensor's device current and `stream` (None: that device's current stream) the
    stream that what is allocated inside belongs to; as a context it gives the stream's handle.
    On another stream than the caller's, `inputs` are kept from reuse until that stream is done
    with them, and what give() names until the caller's stream is."""

    def __init__(self, device, stream, *inputs):
        import torch
        if getattr(stream, "device", device) != device:
            raise ValueError(f"tensors on {device}, a stream of {stream.device}")
        # the handle alone: a decode step's call is bound by the host, and a Stream object costs 2 us
        current = torch._C._cuda_getCurrentRawStream(device.index)
        here = torch._C._cuda_getDevice() == device.index
        self.handle = current if stream is None else _stream(stream)
        self.ctx = None
        if not here or self.handle != current:
            if not hasattr(stream, "cuda_stream"):
                # handle 0 is the device's default stream, which has no external form
                stream = (torch.cuda.ExternalStream(self.handle, device=device) if self.handle
                          else torch.cuda.default_stream(device))
            self.ctx = torch.cuda.stream(stream)
            self.caller = torch.cuda.current_stream(device)
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def give(self, *outputs) -> None:
        if self.ctx is not None:
            for t in outputs:
                t.record_stream(self.caller)

    def __enter__(self) -> int:
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _rotary(positions, sections, theta, interleaved, pairs: int, lead, what: str):
    """(tensor to keep, pointer, UlaRotary) of int32 positions [*lead][axes] (or [*lead] for one
    axis); (None, None, zeros) without positions."""
    r = UlaRotary()
    if positions is None:
        return None, None, r
    if positions.dim() == len(lead):
        positions = positions.unsqueeze(-1)
    shape = tuple(positions.shape)
    axes = shape[-1]
    if shape[:-1] != lead or not 1 <= axes <= 3:
        raise ValueError(f"{what} positions: shape {shape}, expected {tuple(lead)} and 1 to 3 axes")
    sections = (pairs,) if sections is None and axes == 1 else sections
    if sections is None or len(sections) != axes:
        raise ValueError(f"{what}: one section for each of the {axes} axes is required")
    ptr = _dev(positions, "int32", 0, f"{what} positions")   # of that shape: no fewer elements
    r.axes, r.interleaved, r.theta = axes, int(bool(interleaved)), float(theta)
    for i, s in enumerate(sections):
        r.sections[i] = int(s)
    return positions, ptr, r


def pack_rows(fmt: RowFormat, a, b, positions=None, sections=None, theta: float = 10000.0, interleaved: bool = False,
              counts=None, out=None, stream=None):
    """Rows [n][layers][fmt.row_bytes] (uint8) from bf16, fp16 or fp32 tensors: latent channels
    [n][layers][512] and rotary channels [n][layers][64], or for heads rows keys and values
    [n][layers][block_tokens][kv_heads][head_dim] with `counts` (int32 [n], tokens in use).
    With int32 positions ([n][axes], heads rows [n][block_tokens][axes]) the rotary channels, or
    the whole keys, are turned first; sections: pairs of each axis. No gradient is recorded:
    inputs that require one are refused."""
    import torch
    _no_gradient("pack_rows", a, b)
    args = UlaPackArgs()
    args.rows = fmt
    row_bytes = fmt.row_bytes
    if not row_bytes:
        raise UlaError(-1, "pack_rows", "invalid row format")
    latent = fmt.kind == ROWS_LATENT
    if latent:
        if a.dim() != 3:
            raise ValueError(f"pack_rows latent: shape {tuple(a.shape)}, expected (None, None, {LATENT_CHANNELS})")
        n, layers = a.shape[:2]
        args.a, args.type, st_a = _tensor(a, (None, None, LATENT_CHANNELS), "pack_rows latent")
        args.b, type_b, st_b = _tensor(b, (n, layers, ROPE_CHANNELS), "pack_rows rotary channels")
        pairs, lead = ROPE_CHANNELS // 2, (n,)
        if counts is not None:
            raise ValueError("pack_rows counts: heads rows only")
    else:
        shape = (None, None, fmt.block_tokens, fmt.kv_heads, fmt.head_dim)
        args.a, args.type, st_a = _tensor(a, shape, "pack_rows keys")
        n, layers = a.shape[:2]
        args.b, type_b, st_b = _tensor(b, (n, layers, *shape[2:]), "pack_rows values")
        pairs, lead = fmt.head_dim // 2, (n, fmt.block_tokens)
        if counts is not None:
            args.count = _dev(counts, "int32", n, "pack_rows counts")
    if type_b != args.type:
        raise ValueError(f"pack_rows: dtypes {a.dtype} and {b.dtype}")
    for i, (x, y) in enumerate(zip(st_a[:-1], st_b[:-1])):
        args.a_stride[i], args.b_stride[i] = x, y
    args.n, args.layers = n, layers
    _keep, args.positions, args.rotary = _rotary(positions, sections, theta, interleaved, pairs, lead, "pack_rows")
    _same_device(a, b, positions, counts, out)
    on = _On(a.device, stream, a, b, positions, counts, out)
    with on as s:
        if out is None:
            out = torch.empty((n, layers, row_bytes), dtype=torch.uint8, device=a.device)
            on.give(out)
        ptr = _dev(out, "uint8", n * layers * row_bytes, "pack_rows out")
        _check(lib().ula_pack_rows(ctypes.byref(args), ptr, s), "ula_pack_rows")
    return out


def rotate(x, positions, sections=None, theta: float = 10000.0, interleaved: bool = False, inverse: bool = False,
           out=None, stream=None):
    """x [n][heads][dim] turned by int32 positions [n][axes] (or [n]); inverse turns back,
    which is also the gradient of the turn; it is not recorded, so an x that requires one is refused.
    out: a tensor of x's shape and dtype, x itself for in place."""
    import torch
    _no_gradient("rotate", x, out)
    args = UlaRotateArgs()
    args.x, args.type, st = _tensor(x, (None, None, None), "rotate x")
    args.n, args.heads, args.dim = x.shape
    _keep, args.positions, args.rotary = _rotary(positions, sections, theta, interleaved, x.shape[2] // 2,
                                                 (x.shape[0],), "rotate")
    if args.positions is None and x.shape[0]:
        raise ValueError("rotate positions: required")
    args.inverse = int(bool(inverse))
    _same_device(x, positions, out)
    on = _On(x.device, stream, x, positions, out)
    with on as s:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            on.give(out)
        args.out, code, st_out = _tensor(out, x.shape, "rotate out")
        if code != args.type:
            raise ValueError(f"rotate out: dtype {out.dtype}, expected {x.dtype}")
        for i in range(2):
            args.x_stride[i], args.out_stride[i] = st[i], st_out[i]
        _check(lib().ula_rotate(ctypes.byref(args), s), "ula_rotate")
    return out


def norm_rotate(q, k=None, q_weight=None, k_weight=None, positions=None, sections=None, theta: float = 10000.0,
                interleaved: bool = False, rotary: Optional[int] = None, eps: float = 1e-6, out=None, stream=None):
    """(q, k) with each head's channels divided by their root mean square (eps, 2^-126 to 2^96, inside the root) times the weights,
    and the first `rotary` channels (default: all) turned by int32 positions [n][axes] (or [n]; none: norms
    alone), in one launch. q [n][heads][dim], k [n][kv_heads][dim] or None, bf16, fp16 or fp32; weights [dim] in
    that type or fp32, or None for ones. out: a pair of tensors shaped as q and k, themselves for in place. No
    gradient is recorded: tensors that require one are refused."""
    q_out, k_out = out if out is not None else (None, None)
    _no_gradient("norm_rotate", q, k, q_weight, k_weight, q_out, k_out)
    q_ptr, code, st_q = _tensor(q, (None, None, None), "norm_rotate q")
    n, heads, dim = q.shape
    k_ptr, kv, st_k = None, 0, (0, 0)
    if k is not None:
        k_ptr, code_k, st_k = _tensor(k, (n, None, dim), "norm_rotate k")
        if code_k != code:
            raise ValueError(f"norm_rotate: dtypes {q.dtype} and {k.dtype}")
        kv = k.shape[1]
    elif k_weight is not None or k_out is not None:
        raise ValueError("norm_rotate: a weight or result of keys, but no keys")
    if out is not None and (q_out is None or (k_out is None) != (k is None)):
        raise ValueError("norm_rotate out: a result for each of q and k is required")
    weight_type, qw, kw = code, None, None
    if q_weight is not None:
        qw, weight_type, _ = _tensor(q_weight, (dim,), "norm_rotate q_weight", (code, FP32))
    if k_weight is not None:
        kw, weight_type, _ = _tensor(k_weight, (dim,), "norm_rotate k_weight", (code, FP32))
        if q_weight is not None and q_weight.dtype != k_weight.dtype:
            raise ValueError(f"norm_rotate: weights of {q_weight.dtype} and {k_weight.dtype}")
    if positions is None:
        if rotary:
            raise ValueError("norm_rotate positions: required")
        rotary = 0
    elif rotary is None:
        rotary = dim
    _keep, pos, turn = _rotary(positions if rotary else None, sections, theta, interleaved, rotary // 2, (n,), "norm_rotate")
    _same_device(q, k, q_weight, k_weight, positions, q_out, k_out)
    on = _On(q.device, stream, q, k, q_weight, k_weight, positions, q_out, k_out)
    with on as s:
        if out is None:
            q_out = q.new_empty((n, heads, dim))
            on.give(q_out)
            qo, st_qo, ko, st_ko = q_out.data_ptr(), (heads * dim, dim), None, (0, 0)
            if k is not None:
                k_out = q.new_empty((n, kv, dim))
                on.give(k_out)
                ko, st_ko = k_out.data_ptr(), (kv * dim, dim)
        else:
            qo, code_out, st_qo = _tensor(q_out, (n, heads, dim), "norm_rotate q_out")
            ko, code_k, st_ko = (None, code, (0, 0)) if k is None else _tensor(k_out, (n, kv, dim), "norm_rotate k_out")
            if code_out != code or code_k != code:
                raise ValueError(f"norm_rotate out: dtype other than {q.dtype}")
        args = UlaNormArgs(code, n, dim, heads, kv, rotary, weight_type, eps, q_ptr, k_ptr, qo, ko, st_q[:2], st_k[:2],
                           st_qo[:2], st_ko[:2], qw, kw, pos, turn)
        _check(lib().ula_norm_rotate(ctypes.byref(args), s), "ula_norm_rotate")
    return q_out, k_out


def lightest(scores, first, last, n, most: Optional[int] = None, mark: bool = False, out=None, stream=None):
    """Of each range of addresses first[i] .. last[i] - 1 the n[i] entries of least score (ties: lowest address), as
    int32 [ranges][most] in ascending order, -1 behind them: what Engine.release takes, once on the host. scores:
    int64 CUDA tensor by address, as Engine.weigh adds to; negative ones are entries that are not there. first, last, n: host
    integers (arrays or lists; n may be one number). most: columns, by default the largest n. mark: the scores of
    those chosen become -1."""
    import torch
    first, last = _host_ints(first, "lightest first"), _host_ints(last, "lightest last")
    n = _host_ints(np.full(first.shape, n) if np.ndim(n) == 0 else n, "lightest n")
    if first.shape != last.shape or first.shape != n.shape:
        raise ValueError(f"lightest: {first.size} first, {last.size} last addresses and {n.size} counts")
    args = UlaLightestArgs()
    args.scores = _dev(scores, "int64", 0, "lightest scores")
    if scores.numel() >= 1 << 31:
        raise ValueError("lightest scores: 2^31 or more")
    args.capacity, args.ranges = scores.numel(), first.size
    args.first, args.last, args.count = first.ctypes.data, last.ctypes.data, n.ctypes.data
    args.most = (int(n.max()) if n.size else 0) if most is None else most
    args.mark = int(bool(mark))
    if out is not None:
        args.out = _shaped(out, "int32", (first.size, max(args.most, 0)), "lightest out")
    _same_device(scores, out)
    on = _On(scores.device, stream, scores, out)
    with on as s:
        if out is None:
            out = torch.empty((first.size, max(args.most, 0)), dtype=torch.int32, device=scores.device)
            on.give(out)
            args.out = out.data_ptr()
        args.workspace_bytes = lib().ula_lightest_bytes(ctypes.byref(args))
        if args.workspace_bytes:
            work = torch.empty(args.workspace_bytes, dtype=torch.uint8, device=scores.device)
            args.workspace = work.data_ptr()
        _check(lib().ula_lightest(ctypes.byref(args), s), "ula_lightest")
    return out


def tree_masks(parents) -> np.ndarray:
    """Masks for attend_tree (int64, shaped as `parents`, [nodes] or [n_sets][nodes], at most 64 nodes) of trees
    given by each node's parent, an earlier node's number or -1 for a root: bit j of a node is set for each node j
    on its way to the root, itself too. numpy in, numpy out."""
    parents = np.asarray(parents)
    if parents.dtype.kind not in "iu" or parents.ndim not in (1, 2):
        raise ValueError("tree_masks: integers [nodes] or [n_sets][nodes] are required")
    nodes = parents.shape[-1]
    if nodes > 64:
        raise ValueError(f"tree_masks: {nodes} nodes, at most 64")
    rows = parents.reshape(parents.size // nodes if nodes else 0, nodes).astype(np.int64)
    if ((rows < -1) | (rows >= np.arange(nodes))).any():
        raise ValueError("tree_masks: a parent is an earlier node's number or -1")
    out = np.zeros(rows.shape, np.uint64)
    each = np.arange(len(rows))
    for t in range(nodes):
        above = np.where(rows[:, t] >= 0, out[each, np.maximum(rows[:, t], 0)], np.uint64(0))
        out[:, t] = above | np.uint64(1 << t)
    return out.view(np.int64).reshape(parents.shape)


class Engine:
    """One engine context: per group a GPU pool, a pinned host pool and PB-LRU state."""

    def __init__(self, num_groups: int, layers: int, row_bytes: int, ring: int, logical_capacity: int,
                 gpu_slots: int, host_slots: int, max_sets: int, max_k: int, max_append: int = 4096,
                 device: str = "cuda", stream=None, policy: int = 0, static_workspace: bool = False,
                 placement: int = 0):
        """policy: POLICY_PBLRU (0) or POLICY_LRU (1). static_workspace: take the device
        workspace from the library's static array (ula_init_static) instead of a torch
        allocation. placement: PLACE_LOWEST (0) or PLACE_RING (1) for appended entries."""
        import torch
        self.cfg = UlaConfig(num_groups, layers, row_bytes, ring, logical_capacity, gpu_slots,
                             host_slots, max_sets, max_k, max_append, policy, placement)
        self.policy = policy
        L = lib()
        nbytes = L.ula_device_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise UlaError(-1, "ula_device_bytes", "invalid configuration")
        self.device_bytes = nbytes
        self.host_bytes = L.ula_host_bytes(ctypes.byref(self.cfg))
        self.ws = None if static_workspace else torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = torch.device("cuda", torch.cuda.current_device()) if static_workspace else self.ws.device
        self.host = None
        if self.host_bytes:
            self.host = L.ula_host_alloc(self.host_bytes)
            if not self.host:
                raise UlaError(-8, "ula_host_alloc", f"could not pin {self.host_bytes} bytes")
        self.ctx = ctypes.c_void_p()
        if static_workspace:
            rc = L.ula_init_static(ctypes.byref(self.cfg), self.host, _stream(stream), ctypes.byref(self.ctx))
            if rc:
                L.ula_host_free(self.host)
                self.host = None
            _check(rc, "ula_init_static")
        else:
            _check(L.ula_init(ctypes.byref(self.cfg), self.ws.data_ptr(), self.host, _stream(stream),
                              ctypes.byref(self.ctx)), "ula_init")
        self.num_groups, self.layers, self.row_bytes, self.ring = num_groups, layers, row_bytes, ring
        self.N, self.P, self.H = logical_capacity, gpu_slots, host_slots

    # -- calls ---------------------------------------------------------------
    def _rows(self, las, rows, what):
        """(pointer, on_device, keep) for the appended rows [n][layers][row_bytes];
        `keep` holds a host copy alive for the duration of the call."""
        n = las.size * self.layers * self.row_bytes
        if hasattr(rows, "is_cuda") and rows.is_cuda:
            return (_dev(rows, "uint8", n, what) if las.size else None), 1, None
        rows = np.ascontiguousarray(rows, dtype=np.uint8)
        if rows.size < n:
            raise ValueError(f"{what}: {rows.size} row bytes, at least {n} needed")
        return (rows.ctypes.data if las.size else None), 0, rows

    def append(self, group: int, las: np.ndarray, rows, stream=None) -> None:
        """rows: torch CUDA uint8 tensor or numpy uint8 array [n][layers][row_bytes]."""
        las = np.ascontiguousarray(las, dtype=np.int32)
        ptr, on_dev, _keep = self._rows(las, rows, "ula_append rows")
        _check(lib().ula_append(self.ctx, group, las.size, las.ctypes.data, ptr, on_dev,
                                _stream(stream)), "ula_append")

    def release(self, group: int, las: np.ndarray, stream=None) -> None:
        """Give back the slots of finished entries (they become absent)."""
        las = np.ascontiguousarray(las, dtype=np.int32)
        _check(lib().ula_release(self.ctx, group, las.size, las.ctypes.data, _stream(stream)),
               "ula_release")

    def fork(self, group: int, src: int, dst: int, n: int, stream=None) -> None:
        """Copy entries src .. src + n - 1 to the new addresses dst .. dst + n - 1."""
        with _On(self.device, stream) as s:
            _check(lib().ula_fork(self.ctx, group, src, dst, n, s), "ula_fork")

    def rename(self, group: int, src: int, dst: int, n: int, stream=None) -> None:
        """Give entries src .. src + n - 1 the addresses dst .. dst + n - 1; no row moves."""
        with _On(self.device, stream) as s:
            _check(lib().ula_rename(self.ctx, group, src, dst, n, s), "ula_rename")

    def step(self, group: int, sel, stream=None) -> None:
        """sel: torch CUDA int32 tensor [n_sets][k] (or [k] for one set)."""
        n_sets, k = _sets(sel)
        _check(lib().ula_step(self.ctx, group, n_sets, k, _dev(sel, "int32", n_sets * k, "ula_step sel"),
                              _stream(stream)), "ula_step")

    def append_step(self, group: int, las: np.ndarray, rows, sel, stream=None) -> None:
        """append(group, las, rows) then step(group, sel), in fewer launches."""
        las = np.ascontiguousarray(las, dtype=np.int32)
        ptr, on_dev, _keep = self._rows(las, rows, "ula_append_step rows")
        n_sets, k = _sets(sel)
        _check(lib().ula_append_step(self.ctx, group, las.size, las.ctypes.data if las.size else None,
                                     ptr, on_dev, n_sets, k,
                                     _dev(sel, "int32", n_sets * k, "ula_append_step sel"),
                                     _stream(stream)), "ula_append_step")

    def gather(self, group: int, layer: int, sel, out=None, stream=None):
        import torch
        n_sets, k = _sets(sel)
        if out is None:
            out = torch.empty((n_sets, k, self.row_bytes), dtype=torch.uint8, device=sel.device)
        _check(lib().ula_gather(self.ctx, group, layer, n_sets, k,
                                _dev(sel, "int32", n_sets * k, "ula_gather sel"),
                                _dev(out, "uint8", n_sets * k * self.row_bytes, "ula_gather out"),
                                _stream(stream)), "ula_gather")
        return out

    def gather_layers(self, group: int, layer0: int, n_layers: int, sel, out=None, stream=None):
        """Layers layer0 .. layer0 + n_layers - 1 in one launch: out[i] is gather(layer0 + i)."""
        import torch
        n_sets, k = _sets(sel)
        if out is None:
            out = torch.empty((max(n_layers, 0), n_sets, k, self.row_bytes), dtype=torch.uint8,
                              device=sel.device)
        _check(lib().ula_gather_layers(
            self.ctx, group, layer0, n_layers, n_sets, k,
            _dev(sel, "int32", n_sets * k, "ula_gather_layers sel"),
            _dev(out, "uint8", max(n_layers, 0) * n_sets * k * self.row_bytes, "ula_gather_layers out"),
            _stream(stream)), "ula_gather_layers")
        return out

    def attend(self, group: int, layer: int, sel, q, fmt: RowFormat, scale: Optional[float] = None, out=None,
               lse=None, stream=None):
        """(out, lse): attention of q [n_sets][heads][576 or head_dim] (bf16 or fp16) over the selected
        entries' rows of one layer, which are in format `fmt`. out [n_sets][heads][512 or head_dim] in
        q's dtype, lse fp32 [n_sets][heads]. scale: factor of the logits, default 1 / sqrt(q's width);
        pass it for latent rows, whose models scale by a head's width before absorption, not by 576.
        The workspace of a split call is allocated here, on the call's stream. No gradient is recorded:
        a q that requires one is refused."""
        import torch
        _no_gradient("ula_attend", q, out, lse)
        n_sets, k = _sets(sel)
        args = UlaAttendArgs()
        args.rows = fmt
        latent = fmt.kind == ROWS_LATENT
        width = LATENT_CHANNELS + ROPE_CHANNELS if latent else fmt.head_dim
        back = LATENT_CHANNELS if latent else fmt.head_dim
        if q.dim() != 3:
            raise ValueError(f"ula_attend q: shape {tuple(q.shape)}, expected ({n_sets}, None, {width})")
        heads = q.shape[1]
        args.q, args.type, st = _tensor(q, (n_sets, None, width), "ula_attend q", (BF16, FP16))
        args.q_set_stride, args.q_head_stride, args.heads = st[0], st[1], heads
        args.scale = 1.0 / width ** 0.5 if scale is None else scale
        _same_device(q, sel, out, lse, self)
        on = _On(q.device, stream, q, sel, out, lse)
        with on as s:
            if out is None:
                out = torch.empty((n_sets, heads, back), dtype=q.dtype, device=q.device)
                on.give(out)
            args.out, code, st = _tensor(out, (n_sets, heads, back), "ula_attend out")
            if code != args.type:
                raise ValueError(f"ula_attend out: dtype {out.dtype}, expected {q.dtype}")
            args.out_set_stride, args.out_head_stride = st[0], st[1]
            if lse is None:
                lse = torch.empty((n_sets, heads), dtype=torch.float32, device=q.device)
                on.give(lse)
            args.lse = _dev(lse, "float32", n_sets * heads, "ula_attend lse")
            args.workspace_bytes = lib().ula_attend_bytes(ctypes.byref(fmt), n_sets, k, heads)
            if args.workspace_bytes:
                work = torch.empty(args.workspace_bytes, dtype=torch.uint8, device=q.device)
                args.workspace = work.data_ptr()
            _check(lib().ula_attend(self.ctx, group, layer, n_sets, k,
                                    _dev(sel, "int32", n_sets * k, "ula_attend sel"), ctypes.byref(args), s),
                   "ula_attend")
        return out, lse

    def attend_tree(self, group: int, layer: int, sel, q, fmt: RowFormat, drafts, visible, scale: Optional[float] = None,
                    out=None, lse=None, stream=None):
        """(out, lse): attention of a tree of drafted tokens per set. q [n_sets][nodes][heads][576 or head_dim]
        (bf16 or fp16, at most 64 nodes); every node attends to the set's selected entries and to the drafted
        tokens whose bit its mask `visible` (int64 [n_sets][nodes], see tree_masks) has. drafts: their rows, not
        appended yet, as pack_rows gives them: uint8 [n_sets * ceil(nodes / block_tokens)][layers][row_bytes].
        out [n_sets][nodes][heads][512 or head_dim], lse fp32 [n_sets][nodes][heads]; the rest as for attend."""
        import torch
        _no_gradient("ula_attend_tree", q, out, lse)
        n_sets, k = _sets(sel)
        latent = fmt.kind == ROWS_LATENT
        width = LATENT_CHANNELS + ROPE_CHANNELS if latent else fmt.head_dim
        back = LATENT_CHANNELS if latent else fmt.head_dim
        if q.dim() != 4:
            raise ValueError(f"ula_attend_tree q: shape {tuple(q.shape)}, expected ({n_sets}, None, None, {width})")
        nodes, heads = q.shape[1:3]
        q_ptr, code, st = _tensor(q, (n_sets, None, None, width), "ula_attend_tree q", (BF16, FP16))
        per_set = nodes if latent else -(-nodes // max(fmt.block_tokens, 1))
        drafts_ptr = _shaped(drafts, "uint8", (n_sets * per_set, self.layers, self.row_bytes), "ula_attend_tree drafts")
        visible_ptr = _shaped(visible, "int64", (n_sets, nodes), "ula_attend_tree visible")
        if lse is not None:
            lse_ptr = _shaped(lse, "float32", (n_sets, nodes, heads), "ula_attend_tree lse")
        _same_device(q, sel, drafts, visible, out, lse, self)
        on = _On(q.device, stream, q, sel, drafts, visible, out, lse)
        with on as s:
            if out is None:
                out = q.new_empty((n_sets, nodes, heads, back))
                on.give(out)
                out_ptr, st_out = out.data_ptr(), (nodes * heads * back, heads * back, back)
            else:
                out_ptr, code_out, st_out = _tensor(out, (n_sets, nodes, heads, back), "ula_attend_tree out")
                if code_out != code:
                    raise ValueError(f"ula_attend_tree out: dtype {out.dtype}, expected {q.dtype}")
            if lse is None:
                lse = q.new_empty((n_sets, nodes, heads), dtype=torch.float32)
                on.give(lse)
                lse_ptr = lse.data_ptr()
            need = lib().ula_attend_tree_bytes(ctypes.byref(fmt), n_sets, k, nodes, heads)
            work = q.new_empty(need, dtype=torch.uint8) if need else None
            args = UlaTreeArgs(UlaAttendArgs(fmt, code, heads, 1.0 / width ** 0.5 if scale is None else scale, q_ptr, st[0],
                                             st[2], out_ptr, st_out[0], st_out[2], lse_ptr,
                                             work.data_ptr() if need else None, need),
                               nodes, st[1], st_out[1], drafts_ptr, visible_ptr)
            _check(lib().ula_attend_tree(self.ctx, group, layer, n_sets, k,
                                         _dev(sel, "int32", n_sets * k, "ula_attend_tree sel"), ctypes.byref(args), s),
                   "ula_attend_tree")
        return out, lse

    def weigh(self, group: int, layer: int, sel, q, lse, fmt: RowFormat, scores=None, scale: Optional[float] = None,
              out=None, stream=None):
        """The softmax weight that each selected entry got in the attention that gave `lse`, summed over the query
        rows: fp32 [n_sets][k] (out, if given). q [n_sets][heads][576 or head_dim] with lse [n_sets][heads], or with
        a dimension of nodes in front of the heads, as attend and attend_tree take and give them; scale as there.
        scores: int64 [logical_capacity] in units of 2^-32, to which each entry's weight is added at its address,
        whatever is there: weigh every layer before lightest marks, since a marked -1 would be a score again."""
        _no_gradient("ula_weigh", q, lse, out)
        n_sets, k = _sets(sel)
        width = LATENT_CHANNELS + ROPE_CHANNELS if fmt.kind == ROWS_LATENT else fmt.head_dim
        if q.dim() not in (3, 4):
            raise ValueError(f"ula_weigh q: shape {tuple(q.shape)}, expected ({n_sets}, None, {width}) or one more dimension")
        q_ptr, code, st = _tensor(q, (n_sets, *(None,) * (q.dim() - 2), width), "ula_weigh q", (BF16, FP16))
        nodes, heads = (1, q.shape[1]) if q.dim() == 3 else q.shape[1:3]
        lse_ptr = _shaped(lse, "float32", q.shape[:-1], "ula_weigh lse")
        if out is not None:
            out_ptr = _shaped(out, "float32", (n_sets, k), "ula_weigh out")
        scores_ptr = None if scores is None else _dev(scores, "int64", self.N, "ula_weigh scores")
        _same_device(q, sel, lse, scores, out, self)
        on = _On(q.device, stream, q, sel, lse, scores, out)
        with on as s:
            if out is None:
                out = lse.new_empty((n_sets, k))
                on.give(out)
                out_ptr = out.data_ptr()
            args = UlaWeighArgs(fmt, code, nodes, heads, 1.0 / width ** 0.5 if scale is None else scale, q_ptr, st[0], st[1],
                                st[-2], lse_ptr, out_ptr, scores_ptr)
            _check(lib().ula_weigh(self.ctx, group, layer, n_sets, k, _dev(sel, "int32", n_sets * k, "ula_weigh sel"),
                                   ctypes.byref(args), s), "ula_weigh")
        return out

    def sync(self, stream=None) -> List[tuple]:
        st = (UlaStepStats * self.num_groups)()
        _check(lib().ula_sync(self.ctx, _stream(stream), st), "ula_sync")
        return [s.as_tuple() for s in st]

    def sync_code(self, stream=None) -> int:
        """ula_sync's return code without raising (for error-path tests)."""
        return lib().ula_sync(self.ctx, _stream(stream), None)

    def export_state(self, group: int) -> dict:
        W = (self.P + 31) // 32
        out = dict(map=np.empty(self.N, np.uint32), gown=np.empty(self.P, np.int32),
                   hown=np.empty(max(self.H, 1), np.int32),
                   bitsets=np.empty((self.ring + 2, W), np.uint32))
        stamps = np.empty(self.P, np.int32) if self.policy == POLICY_LRU else None
        sh = UlaStateHost(out["map"].ctypes.data, out["gown"].ctypes.data, out["hown"].ctypes.data,
                          out["bitsets"].ctypes.data, 0, 0, UlaStepStats(),
                          stamps.ctypes.data if stamps is not None else None)
        _check(lib().ula_export_state(self.ctx, group, ctypes.byref(sh)), "ula_export_state")
        out["hown"] = out["hown"][: self.H]
        out["cur"] = int(sh.cur)
        out["flag"] = int(sh.flag)
        out["stats"] = sh.last.as_tuple()
        if stamps is not None:
            out["stamps"] = stamps
        return out

    def read_rows(self, group: int, las: np.ndarray) -> np.ndarray:
        las = np.ascontiguousarray(las, dtype=np.int32)
        out = np.empty((las.size, self.layers, self.row_bytes), dtype=np.uint8)
        _check(lib().ula_read_rows(self.ctx, group, las.size, las.ctypes.data, out.ctypes.data),
               "ula_read_rows")
        return out

    def flag_address(self, group: int) -> int:
        p = ctypes.c_void_p()
        _check(lib().ula_flag_address(self.ctx, group, ctypes.byref(p)), "ula_flag_address")
        return p.value

    TIMING_STEP = 1      # phase events of every step (read_timing)
    TIMING_GATHER = 2    # kernel time of every gather (read_gather_timing)
    TIMING_LINK = 4      # kernel time of every step's host-link launch (read_link_timing)

    def set_timing(self, flags) -> None:
        """flags: an OR of TIMING_STEP and TIMING_GATHER (True means TIMING_STEP)."""
        flags = self.TIMING_STEP if flags is True else int(flags)
        _check(lib().ula_set_timing(self.ctx, flags), "ula_set_timing")

    def read_timing(self, group: int) -> List[float]:
        ms = (ctypes.c_float * 3)()
        _check(lib().ula_read_timing(self.ctx, group, ms), "ula_read_timing")
        return list(ms)

    def read_gather_timing(self) -> tuple:
        """(summed gather kernel milliseconds, launches) since the last read."""
        ms, n = ctypes.c_double(), ctypes.c_int64()
        _check(lib().ula_read_gather_timing(self.ctx, ctypes.byref(ms), ctypes.byref(n)),
               "ula_read_gather_timing")
        return ms.value, n.value

    def read_link_timing(self) -> tuple:
        """(summed host-link launch milliseconds, launches) since the last read."""
        ms, n = ctypes.c_double(), ctypes.c_int64()
        _check(lib().ula_read_link_timing(self.ctx, ctypes.byref(ms), ctypes.byref(n)),
               "ula_read_link_timing")
        return ms.value, n.value

    def close(self) -> None:
        if getattr(self, "ctx", None) is not None and self.ctx.value:
            import torch
            torch.cuda.synchronize()
            lib().ula_destroy(self.ctx)
            self.ctx = None
        if getattr(self, "host", None):
            lib().ula_host_free(self.host)
            self.host = None
        self.ws = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
