"""ctypes binding of libcsa.so: argument marshalling only.

Every function here checks each tensor's dtype and shape against the layer
and the call (the C ABI sees only untyped pointers, so a wrong dtype or shape
would otherwise be read as garbage) and that it is a contiguous CUDA tensor,
all before anything is allocated or enqueued; then it passes raw device
pointers and the current CUDA stream to the C ABI declared in include/csa.h
and turns a non-zero csa_status into an exception.  All arithmetic runs in the
library's CUDA kernels; there is no CPU path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct
import sysconfig
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libcsa.so")
_TENSORS_PATH = os.path.join(_HERE, "_lib", "libcsa_tensors.so")
_CHECKS_PATH = os.path.join(_HERE, "_lib", "csa_checks" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

CSA_F32, CSA_BF16 = 0, 1
OP_COMPRESS, OP_INDEX_TOPK, OP_ATTEND_DECODE, OP_ATTEND_PREFILL, OP_COMPRESS_PAIR = 0, 1, 2, 3, 4
OP_COMPRESS_VARLEN, OP_ATTEND_PREFILL_VARLEN = 5, 6
OP_COMPRESS_TREE, OP_ATTEND_TREE, OP_INDEX_SCORES_TREE = 7, 8, 9
OP_ATTEND_PAGES = 10
FP8_ROW_BYTES = 144  # CSA_FP8_ROW_BYTES: 128 E4M3 codes, the fp32 scale, 12 zero bytes
DEV_CAPACITY, DEV_STATE, DEV_RANGE, DEV_ROLLBACK = 1, 2, 4, 8
CSA_OK, CSA_ERR_ARG, CSA_ERR_UNSUPPORTED, CSA_ERR_CUDA, CSA_ERR_WORKSPACE = 0, 1, 2, 3, 4
STATUS = {0: "CSA_OK", 1: "CSA_ERR_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_CUDA", 4: "CSA_ERR_WORKSPACE"}
EXPORTS = ("csa_kernel_launches", "csa_frontier_slots", "csa_workspace_size", "csa_compress_append", "csa_index_topk",
           "csa_attend_decode", "csa_attend_prefill_chunk", "csa_status_string", "csa_static_scratch_bytes",
           "csa_index_topk_static", "csa_index_topk_overlapped", "csa_advance_positions",
           "csa_compress_append_pair", "csa_trim", "csa_index_topk_verify", "csa_attend_verify",
           "csa_compress_append_varlen", "csa_attend_prefill_varlen", "csa_index_rows_fp8", "csa_norm_rope",
           "csa_compress_tree", "csa_index_scores_tree", "csa_attend_tree", "csa_commit_tree", "csa_add_norm",
           "csa_append_pages", "csa_attend_pages")


class CSAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


class _Layer(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int), ("R", ctypes.c_int),
                ("W", ctypes.c_int), ("ratio", ctypes.c_int), ("Hi", ctypes.c_int), ("Di", ctypes.c_int),
                ("topk", ctypes.c_int), ("X", ctypes.c_int), ("scale", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("rollback", ctypes.c_int), ("index_fp8", ctypes.c_int)]


class _Comp(ctypes.Structure):
    _fields_ = [("wkv", ctypes.c_void_p), ("wgate", ctypes.c_void_p), ("ape", ctypes.c_void_p),
                ("norm_w", ctypes.c_void_p), ("d", ctypes.c_int)]


class _Rows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int), ("norm", ctypes.c_int),
                ("x_stride", ctypes.c_longlong)]


# the same layouts for struct.pack, a few microseconds a call cheaper than building ctypes structures
_COMP_FMT, _ROWS_FMT, _PAGES_FMT = "@4Pi0P", "@3P3iq", "@2P2i"


_lib = None
_addresses = None  # csrc/checks.c: what _ptrs does, in C
_plain = None  # csrc/checks.c: whole calls on plain tensors; with the addresses of the library's functions
_at = {}


def _tensors(path: str = _TENSORS_PATH) -> int:
    """Address of csa_tensor (csrc/tensors.cpp) where it was built for this very torch, whose layout of a tensor it has
    compiled in; otherwise 0, and the checks ask tensors by their attributes."""
    if not os.path.exists(path):
        return 0
    try:
        lib = ctypes.CDLL(path)  # (stays loaded: nothing unloads it)
        built_for = lib.csa_tensors_torch
        built_for.argtypes, built_for.restype = [], ctypes.c_char_p
        if built_for().decode() != f"{torch.__version__} {torch.version.git_version}":
            return 0
        return ctypes.cast(lib.csa_tensor, ctypes.c_void_p).value
    except (OSError, AttributeError):  # it needs what this torch has not; an older build that does not say
        return 0


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libcsa.so (built by build.py); raises if it is missing."""
    global _lib, _addresses, _plain
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"CSA CUDA library not built: {path} is missing "
                          "(run deepseek_v4_compressed_csa_gb300.build.build())")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.csa_frontier_slots.argtypes = [i32]
    lib.csa_frontier_slots.restype = i32
    lib.csa_kernel_launches.argtypes = []
    lib.csa_kernel_launches.restype = ctypes.c_ulonglong
    lib.csa_status_string.argtypes = [i32]
    lib.csa_status_string.restype = ctypes.c_char_p
    lib.csa_workspace_size.argtypes = [vp, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.csa_workspace_size.restype = i32
    lib.csa_compress_append.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.csa_compress_append.restype = i32
    lib.csa_index_topk.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.csa_index_topk.restype = i32
    lib.csa_index_topk_overlapped.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    lib.csa_index_topk_overlapped.restype = i32
    lib.csa_static_scratch_bytes.argtypes = []
    lib.csa_static_scratch_bytes.restype = sz
    lib.csa_index_topk_static.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.csa_index_topk_static.restype = i32
    lib.csa_attend_decode.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.csa_attend_decode.restype = i32
    lib.csa_attend_prefill_chunk.argtypes = [vp, vp, vp, vp, vp, vp, i32, ctypes.c_int32, vp, vp, vp, i32, vp, vp,
                                             vp, vp, vp, sz, vp, vp]
    lib.csa_attend_prefill_chunk.restype = i32
    lib.csa_compress_append_pair.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, i32, vp, vp, vp,
                                             sz, vp, vp]
    lib.csa_compress_append_pair.restype = i32
    lib.csa_advance_positions.argtypes = [vp, i32, i32, vp]
    lib.csa_advance_positions.restype = i32
    lib.csa_trim.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.csa_trim.restype = i32
    lib.csa_index_topk_verify.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.csa_index_topk_verify.restype = i32
    lib.csa_attend_verify.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.csa_attend_verify.restype = i32
    lib.csa_compress_append_varlen.argtypes = [vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.csa_compress_append_varlen.restype = i32
    lib.csa_attend_prefill_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, vp, i32, vp, vp,
                                              vp, vp, vp, sz, vp, vp]
    lib.csa_attend_prefill_varlen.restype = i32
    lib.csa_index_rows_fp8.argtypes = [vp, vp, ctypes.c_longlong, vp, vp]
    lib.csa_index_rows_fp8.restype = i32
    lib.csa_norm_rope.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
    lib.csa_norm_rope.restype = i32
    lib.csa_compress_tree.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.csa_compress_tree.restype = i32
    lib.csa_index_scores_tree.argtypes = [vp, vp, vp, i32, i32, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp, vp]
    lib.csa_index_scores_tree.restype = i32
    lib.csa_attend_tree.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                    vp]
    lib.csa_attend_tree.restype = i32
    lib.csa_commit_tree.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                    i32, vp, vp, vp, vp]
    lib.csa_commit_tree.restype = i32
    i64 = ctypes.c_longlong
    lib.csa_add_norm.argtypes = [vp, vp, i64, vp, i64, vp, i64, i32, vp, vp, vp, vp, i32, vp]
    lib.csa_add_norm.restype = i32
    lib.csa_append_pages.argtypes = [vp, vp, vp, i64, i64, i32, i32, vp, i32, vp, vp, vp, i32, vp, vp, vp]
    lib.csa_append_pages.restype = i32
    lib.csa_attend_pages.argtypes = [vp, vp, vp, i32, i32, vp, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz,
                                     vp, vp]
    lib.csa_attend_pages.restype = i32
    if os.path.exists(_CHECKS_PATH):  # (not built where Python's headers are missing)
        spec = importlib.util.spec_from_file_location("csa_checks", _CHECKS_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _addresses = module.addresses
        module.setup(torch.float32, torch.uint8, torch.int32, torch._C._cuda_getCurrentRawStream,
                     torch._C._cuda_getDevice)
        module.tensors(_tensors())
        for name in ("add_norm", "append_pages", "attend_pages"):
            _at[name] = ctypes.cast(getattr(lib, "csa_" + name), ctypes.c_void_p).value
        _plain = module
    _lib = lib
    return lib


@dataclass(frozen=True)
class Layer:
    """Mirror of csa_layer.  dtype: torch.bfloat16 or torch.float32 (model dtype).  rollback: tokens csa_trim may
    rewind; the window ring then has W + rollback slots and each frontier ring frontier_slots(ratio) + rollback.
    index_fp8: the index pool holds fp8 rows, a uint8 tensor [B, cap, FP8_ROW_BYTES]."""

    dtype: torch.dtype
    H: int
    D: int
    R: int
    W: int
    ratio: int
    Hi: int
    Di: int
    topk: int
    X: int
    scale: float = 0.0
    rms_eps: float = 1e-6
    rollback: int = 0
    index_fp8: bool = False

    @property
    def ring_slots(self) -> int:
        return self.W + self.rollback

    @property
    def lanes(self) -> int:
        return 2 if self.ratio == 4 else 1

    @property
    def has_indexer(self) -> bool:
        return self.ratio == 4

    def _c(self) -> _Layer:
        code = CSA_BF16 if self.dtype == torch.bfloat16 else CSA_F32
        return _Layer(code, self.H, self.D, self.R, self.W, self.ratio, self.Hi, self.Di, self.topk, self.X,
                      float(self.scale), float(self.rms_eps), int(self.rollback), int(self.index_fp8))

    def _packed(self) -> bytes:
        """The bytes of the C struct (kept: the fields are frozen)."""
        p = self.__dict__.get("_bytes")
        if p is None:
            p = bytes(self._c())
            object.__setattr__(self, "_bytes", p)
        return p

    def pool_spec(self, d: int):
        """(dtype, row length) of a pool with rows of d values: fp8 index rows are FP8_ROW_BYTES bytes."""
        if self.index_fp8 and d == self.Di:
            return torch.uint8, FP8_ROW_BYTES
        return self.dtype, d


@dataclass
class Compressor:
    """Device weights of one compressor: wkv, wgate [L*d, X] model dtype; ape [ratio, L*d] fp32; norm_w [d] fp32."""

    wkv: torch.Tensor
    wgate: torch.Tensor
    ape: torch.Tensor
    norm_w: torch.Tensor
    d: int

    def _c(self) -> _Comp:
        return _Comp(_ptr(self.wkv), _ptr(self.wgate), _ptr(self.ape), _ptr(self.norm_w), self.d)


def _expect(name: str, t, dtype: torch.dtype, shape=None, optional: bool = False):
    """Raise TypeError / ValueError unless ``t`` has ``dtype`` and (when given) exactly ``shape``."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _expect_err(err):
    if err is not None:
        _expect("err", err, torch.int32)
        if err.numel() < 1:
            raise ValueError("err must hold at least one int32")


def _expect_comp(layer: "Layer", comp: "Compressor", which: str):
    L, d = layer.lanes, comp.d
    _expect(f"{which}.wkv", comp.wkv, layer.dtype, (L * d, layer.X))
    _expect(f"{which}.wgate", comp.wgate, layer.dtype, (L * d, layer.X))
    _expect(f"{which}.ape", comp.ape, torch.float32, (layer.ratio, L * d))
    _expect(f"{which}.norm_w", comp.norm_w, torch.float32, (d,))


def _expect_pool(name: str, layer: "Layer", pool, d: int, B=None, dims: int = 3):
    """pool [B, cap, row] (dims 3) or [cap, row] (dims 2) in the layer's pool format for rows of d values."""
    dt, row = layer.pool_spec(d)
    _expect(name, pool, dt)
    lead = () if B is None or dims == 2 else (B,)
    if pool.dim() != dims or pool.shape[-1] != row or tuple(pool.shape[:len(lead)]) != lead:
        want = "[cap, %d]" % row if dims == 2 else "[%s, cap, %d]" % ("B" if B is None else B, row)
        raise ValueError(f"{name}: shape {tuple(pool.shape)}, expected {want}")


def _frontier_len(layer: "Layer") -> int:
    return (2 * layer.ratio if layer.ratio == 4 else layer.ratio) + layer.rollback


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("CSA tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("CSA tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(fn: str, code: int):
    if code != 0:
        raise CSAError(fn, code)


def kernel_launches() -> int:
    """Kernels enqueued by the library so far in this process."""
    return int(load_library().csa_kernel_launches())


def advance_positions(pos, by: int = 1, stream=None):
    """pos[b] += by for every sequence (int32 device tensor), on the library's launch path."""
    _expect("pos", pos, torch.int32, (pos.numel(),) if isinstance(pos, torch.Tensor) else None)
    _check("csa_advance_positions", load_library().csa_advance_positions(_ptr(pos), pos.numel(), by,
                                                                         _stream(stream)))


def index_rows_fp8(layer: Layer, src, dst, stream=None):
    """csa_index_rows_fp8: src [..., Di] model-dtype index rows -> dst [..., FP8_ROW_BYTES] uint8 fp8 rows (same
    leading shape); the layer has index_fp8 set."""
    _expect("src", src, layer.dtype)
    if src.dim() < 1 or src.shape[-1] != layer.Di:
        raise ValueError(f"src: shape {tuple(src.shape)}, expected [..., {layer.Di}]")
    _expect("dst", dst, torch.uint8, tuple(src.shape[:-1]) + (FP8_ROW_BYTES,))
    n = src.numel() // layer.Di
    L = layer._c()
    _check("csa_index_rows_fp8", load_library().csa_index_rows_fp8(ctypes.byref(L), _ptr(src), n, _ptr(dst),
                                                                   _stream(stream)))


def frontier_slots(ratio: int) -> int:
    return load_library().csa_frontier_slots(ratio)


def trim(layer: Layer, n_back, pos, n_rows_a, n_rows_i, hw, err=None, stream=None):
    """csa_trim: rewind each sequence b by n_back[b] tokens (int32 device tensors [B]; n_rows_i None for layers
    without an indexer; hw: the high-water positions, caller-owned).  Returns the device error word tensor."""
    B = pos.numel() if isinstance(pos, torch.Tensor) else 0
    for name, t in (("n_back", n_back), ("pos", pos), ("n_rows_a", n_rows_a), ("hw", hw)):
        _expect(name, t, torch.int32, (B,))
    _expect("n_rows_i", n_rows_i, torch.int32, (B,), optional=not layer.has_indexer)
    _expect_err(err)
    err = _err(err, pos.device, stream)
    L = layer._c()
    _check("csa_trim", load_library().csa_trim(ctypes.byref(L), B, _ptr(n_back), _ptr(pos), _ptr(n_rows_a),
                                               _ptr(n_rows_i), _ptr(hw), _ptr(err), _stream(stream)))
    return err


def workspace_size(layer: Layer, op: int, B: int, T: int, cap: int) -> int:
    n = ctypes.c_size_t(0)
    L = layer._c()
    _check("csa_workspace_size", load_library().csa_workspace_size(ctypes.byref(L), op, B, T, cap, ctypes.byref(n)))
    return int(n.value)


def _new(device, stream, new, *size, dtype):
    """A tensor of the call's own: allocated, and zeroed where it is, on the stream that will use it (torch's, or any
    object with its handle as cuda_stream)."""
    if stream is None:
        return new(*size, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        return new(*size, dtype=dtype, device=device)


def _ws(layer, op, B, T, cap, ws, device, stream):
    need = workspace_size(layer, op, B, T, cap)
    if ws is None:
        ws = _new(device, stream, torch.empty, max(need, 256), dtype=torch.uint8)
    return ws, ws.numel() * ws.element_size()


def _err(err, device, stream):
    return _new(device, stream, torch.zeros, 1, dtype=torch.int32) if err is None else err


def compress_append(layer: Layer, comp: Compressor, x, pos, frontier, pool, n_rows, inv_freq, ws=None, err=None,
                    stream=None):
    """csa_compress_append; x [B,T,X]; returns the device error word tensor."""
    _expect("x", x, layer.dtype)
    if x.dim() != 3 or x.shape[2] != layer.X:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [B, T, {layer.X}]")
    B, T = x.shape[0], x.shape[1]
    _expect_comp(layer, comp, "comp")
    _expect_pool("pool", layer, pool, comp.d, B)
    cap = pool.shape[1]
    _expect("pos", pos, torch.int32, (B,))
    _expect("frontier", frontier, layer.dtype, (B, _frontier_len(layer), 2 * layer.lanes * comp.d))
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect_err(err)
    ws, nb = _ws(layer, OP_COMPRESS, B, T, cap, ws, x.device, stream)
    err = _err(err, x.device, stream)
    L, C = layer._c(), comp._c()
    _check("csa_compress_append", load_library().csa_compress_append(
        ctypes.byref(L), ctypes.byref(C), _ptr(x), B, T, _ptr(pos), _ptr(frontier), _ptr(pool), cap, _ptr(n_rows),
        _ptr(inv_freq), _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def compress_append_pair(layer: Layer, comp_a: Compressor, comp_i: Compressor, x, pos, frontier_a, pool_a, n_rows_a,
                         frontier_i, pool_i, n_rows_i, inv_freq, ws=None, err=None, stream=None):
    """csa_compress_append_pair (attention pool, then index pool, same tokens); returns the error word tensor."""
    _expect("x", x, layer.dtype)
    if x.dim() != 3 or x.shape[2] != layer.X:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [B, T, {layer.X}]")
    B, T = x.shape[0], x.shape[1]
    _expect_comp(layer, comp_a, "comp_a")
    _expect_comp(layer, comp_i, "comp_i")
    F = _frontier_len(layer)
    for nm, pl, fr, nr, d in (("a", pool_a, frontier_a, n_rows_a, comp_a.d), ("i", pool_i, frontier_i, n_rows_i,
                                                                               comp_i.d)):
        _expect_pool(f"pool_{nm}", layer, pl, d, B)
        _expect(f"frontier_{nm}", fr, layer.dtype, (B, F, 2 * layer.lanes * d))
        _expect(f"n_rows_{nm}", nr, torch.int32, (B,))
    _expect("pos", pos, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect_err(err)
    cap_a, cap_i = pool_a.shape[1], pool_i.shape[1]
    ws, nb = _ws(layer, OP_COMPRESS_PAIR, B, T, max(cap_a, cap_i), ws, x.device, stream)
    err = _err(err, x.device, stream)
    L, Ca, Ci = layer._c(), comp_a._c(), comp_i._c()
    _check("csa_compress_append_pair", load_library().csa_compress_append_pair(
        ctypes.byref(L), ctypes.byref(Ca), ctypes.byref(Ci), _ptr(x), B, T, _ptr(pos), _ptr(frontier_a),
        _ptr(pool_a), cap_a, _ptr(n_rows_a), _ptr(frontier_i), _ptr(pool_i), cap_i, _ptr(n_rows_i), _ptr(inv_freq),
        _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def _expect_index(layer: Layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, err):
    _expect("iq", iq, layer.dtype)
    if iq.dim() != 3 or iq.shape[1:] != (layer.Hi, layer.Di):
        raise ValueError(f"iq: shape {tuple(iq.shape)}, expected [B, {layer.Hi}, {layer.Di}]")
    B = iq.shape[0]
    _expect("iw", iw, layer.dtype, (B, layer.Hi))
    _expect_pool("ikeys", layer, ikeys, layer.Di, B)
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("pos", pos, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect("sel", sel, torch.int32, (B, layer.topk))
    _expect("n_sel", n_sel, torch.int32, (B,))
    _expect_err(err)


def index_topk(layer: Layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, ws=None, err=None, stream=None):
    _expect_index(layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, err)
    B, cap = iq.shape[0], ikeys.shape[1]
    ws, nb = _ws(layer, OP_INDEX_TOPK, B, 1, cap, ws, iq.device, stream)
    err = _err(err, iq.device, stream)
    L = layer._c()
    _check("csa_index_topk", load_library().csa_index_topk(
        ctypes.byref(L), _ptr(iq), _ptr(iw), B, _ptr(ikeys), cap, _ptr(n_rows), _ptr(pos), _ptr(inv_freq),
        _ptr(sel), _ptr(n_sel), _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def index_topk_overlapped(layer: Layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, pool_ready=None, ws=None,
                          err=None, stream=None):
    """csa_index_topk_overlapped: the scan of the rows complete before the token is enqueued at once; the
    rest waits for `pool_ready` (a torch.cuda.Event recorded after the index pool's compress call)."""
    _expect_index(layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, err)
    B, cap = iq.shape[0], ikeys.shape[1]
    ws, nb = _ws(layer, OP_INDEX_TOPK, B, 1, cap, ws, iq.device, stream)
    err = _err(err, iq.device, stream)
    L = layer._c()
    ev = pool_ready.cuda_event if pool_ready is not None else None
    _check("csa_index_topk_overlapped", load_library().csa_index_topk_overlapped(
        ctypes.byref(L), _ptr(iq), _ptr(iw), B, _ptr(ikeys), cap, _ptr(n_rows), _ptr(pos), _ptr(inv_freq),
        _ptr(sel), _ptr(n_sel), _ptr(ws), nb, _ptr(err), _stream(stream), ev))
    return err


def index_topk_static(layer: Layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, err=None, stream=None):
    """csa_index_topk_static: the decode indexer with the library's own fixed scratch array (no workspace)."""
    _expect_index(layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, err)
    B, cap = iq.shape[0], ikeys.shape[1]
    err = _err(err, iq.device, stream)
    L = layer._c()
    _check("csa_index_topk_static", load_library().csa_index_topk_static(
        ctypes.byref(L), _ptr(iq), _ptr(iw), B, _ptr(ikeys), cap, _ptr(n_rows), _ptr(pos), _ptr(inv_freq),
        _ptr(sel), _ptr(n_sel), _ptr(err), _stream(stream)))
    return err


def static_scratch_bytes() -> int:
    return int(load_library().csa_static_scratch_bytes())


def attend_decode(layer: Layer, q, kv_new, sink, window, pool, n_rows, sel, n_sel, pos, inv_freq, out, ws=None,
                  err=None, stream=None):
    _expect("q", q, layer.dtype)
    if q.dim() != 3 or q.shape[1:] != (layer.H, layer.D):
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [B, {layer.H}, {layer.D}]")
    B = q.shape[0]
    _expect("kv_new", kv_new, layer.dtype, (B, layer.D))
    _expect("sink", sink, torch.float32, (layer.H,))
    _expect("window", window, layer.dtype, (B, layer.ring_slots, layer.D))
    _expect("pool", pool, layer.dtype)
    if pool.dim() != 3 or pool.shape[0] != B or pool.shape[2] != layer.D:
        raise ValueError(f"pool: shape {tuple(pool.shape)}, expected [{B}, cap, {layer.D}]")
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("sel", sel, torch.int32, (B, layer.topk), optional=True)
    _expect("n_sel", n_sel, torch.int32, (B,), optional=sel is None)
    _expect("pos", pos, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect("out", out, layer.dtype, (B, layer.H, layer.D))
    _expect_err(err)
    cap = pool.shape[1]
    ws, nb = _ws(layer, OP_ATTEND_DECODE, B, 1, cap, ws, q.device, stream)
    err = _err(err, q.device, stream)
    L = layer._c()
    _check("csa_attend_decode", load_library().csa_attend_decode(
        ctypes.byref(L), _ptr(q), _ptr(kv_new), _ptr(sink), B, _ptr(window), _ptr(pool), cap, _ptr(n_rows),
        _ptr(sel), _ptr(n_sel), _ptr(pos), _ptr(inv_freq), _ptr(out), _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def attend_prefill_chunk(layer: Layer, q, kv_new, iq, iw, sink, pos0: int, window, pool, ikeys, n_rows, inv_freq,
                         out, sel_out=None, ws=None, err=None, stream=None):
    _expect("q", q, layer.dtype)
    if q.dim() != 3 or q.shape[1:] != (layer.H, layer.D):
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [T, {layer.H}, {layer.D}]")
    T = q.shape[0]
    _expect("kv_new", kv_new, layer.dtype, (T, layer.D))
    if layer.has_indexer:
        _expect("iq", iq, layer.dtype, (T, layer.Hi, layer.Di))
        _expect("iw", iw, layer.dtype, (T, layer.Hi))
        _expect_pool("ikeys", layer, ikeys, layer.Di, dims=2)
    _expect("sink", sink, torch.float32, (layer.H,))
    _expect("window", window, layer.dtype, (layer.ring_slots, layer.D))
    _expect("pool", pool, layer.dtype)
    if pool.dim() != 2 or pool.shape[1] != layer.D:
        raise ValueError(f"pool: shape {tuple(pool.shape)}, expected [cap, {layer.D}]")
    _expect("n_rows", n_rows, torch.int32, (1,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect("out", out, layer.dtype, (T, layer.H, layer.D))
    _expect("sel_out", sel_out, torch.int32, (T, layer.topk), optional=True)
    _expect_err(err)
    cap = pool.shape[-2]
    ws, nb = _ws(layer, OP_ATTEND_PREFILL, 1, T, cap, ws, q.device, stream)
    err = _err(err, q.device, stream)
    L = layer._c()
    _check("csa_attend_prefill_chunk", load_library().csa_attend_prefill_chunk(
        ctypes.byref(L), _ptr(q), _ptr(kv_new), _ptr(iq), _ptr(iw), _ptr(sink), T, int(pos0), _ptr(window),
        _ptr(pool), _ptr(ikeys), cap, _ptr(n_rows), _ptr(inv_freq), _ptr(out), _ptr(sel_out), _ptr(ws), nb,
        _ptr(err), _stream(stream)))
    return err


def _expect_varlen(cu_seqlens, B: int, N: int, T_max: int):
    _expect("cu_seqlens", cu_seqlens, torch.int32, (B + 1,))
    if not 1 <= int(T_max) <= N:
        raise ValueError(f"T_max = {T_max}: expected 1 <= T_max <= N = {N}")


def compress_append_varlen(layer: Layer, comp: Compressor, x, cu_seqlens, T_max: int, pos, frontier, pool, n_rows,
                           inv_freq, ws=None, err=None, stream=None):
    """csa_compress_append_varlen; x [N, X] packs B chunks, sequence b's rows cu_seqlens[b] .. cu_seqlens[b+1]-1
    (device int32 [B+1]); T_max (host) bounds every chunk's length."""
    _expect("x", x, layer.dtype)
    if x.dim() != 2 or x.shape[1] != layer.X:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [N, {layer.X}]")
    N = x.shape[0]
    _expect_pool("pool", layer, pool, comp.d)
    B, cap = pool.shape[0], pool.shape[1]
    _expect_varlen(cu_seqlens, B, N, T_max)
    _expect_comp(layer, comp, "comp")
    _expect("pos", pos, torch.int32, (B,))
    _expect("frontier", frontier, layer.dtype, (B, _frontier_len(layer), 2 * layer.lanes * comp.d))
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect_err(err)
    ws, nb = _ws(layer, OP_COMPRESS_VARLEN, B, N, cap, ws, x.device, stream)
    err = _err(err, x.device, stream)
    L, C = layer._c(), comp._c()
    _check("csa_compress_append_varlen", load_library().csa_compress_append_varlen(
        ctypes.byref(L), ctypes.byref(C), _ptr(x), B, _ptr(cu_seqlens), N, int(T_max), _ptr(pos), _ptr(frontier),
        _ptr(pool), cap, _ptr(n_rows), _ptr(inv_freq), _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def attend_prefill_varlen(layer: Layer, q, kv_new, iq, iw, sink, cu_seqlens, T_max: int, pos, window, pool, ikeys,
                          n_rows, inv_freq, out, sel_out=None, ws=None, err=None, stream=None):
    """csa_attend_prefill_varlen; q [N, H, D], kv_new [N, D], iq [N, Hi, Di], iw [N, Hi], out [N, H, D] pack B
    chunks (rows cu_seqlens[b] .. cu_seqlens[b+1]-1 at positions pos[b] ..); window [B, W+rollback, D], pool
    [B, cap, D], ikeys [B, cap, Di], n_rows [B]."""
    _expect("q", q, layer.dtype)
    if q.dim() != 3 or q.shape[1:] != (layer.H, layer.D):
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [N, {layer.H}, {layer.D}]")
    N = q.shape[0]
    _expect("pool", pool, layer.dtype)
    if pool.dim() != 3 or pool.shape[2] != layer.D:
        raise ValueError(f"pool: shape {tuple(pool.shape)}, expected [B, cap, {layer.D}]")
    B, cap = pool.shape[0], pool.shape[1]
    _expect_varlen(cu_seqlens, B, N, T_max)
    _expect("kv_new", kv_new, layer.dtype, (N, layer.D))
    if layer.has_indexer:
        _expect("iq", iq, layer.dtype, (N, layer.Hi, layer.Di))
        _expect("iw", iw, layer.dtype, (N, layer.Hi))
        _expect_pool("ikeys", layer, ikeys, layer.Di, B)
        if ikeys.shape[1] != cap:
            raise ValueError(f"ikeys: shape {tuple(ikeys.shape)}, expected [{B}, {cap}, {layer.pool_spec(layer.Di)[1]}]")
    _expect("sink", sink, torch.float32, (layer.H,))
    _expect("pos", pos, torch.int32, (B,))
    _expect("window", window, layer.dtype, (B, layer.ring_slots, layer.D))
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect("out", out, layer.dtype, (N, layer.H, layer.D))
    _expect("sel_out", sel_out, torch.int32, (N, layer.topk), optional=True)
    _expect_err(err)
    ws, nb = _ws(layer, OP_ATTEND_PREFILL_VARLEN, B, N, cap, ws, q.device, stream)
    err = _err(err, q.device, stream)
    L = layer._c()
    _check("csa_attend_prefill_varlen", load_library().csa_attend_prefill_varlen(
        ctypes.byref(L), _ptr(q), _ptr(kv_new), _ptr(iq), _ptr(iw), _ptr(sink), B, _ptr(cu_seqlens), N, int(T_max),
        _ptr(pos), _ptr(window), _ptr(pool), _ptr(ikeys), cap, _ptr(n_rows), _ptr(inv_freq), _ptr(out), _ptr(sel_out),
        _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def index_topk_verify(layer: Layer, iq, iw, ikeys, n_rows, pos, inv_freq, sel, n_sel, ws=None, err=None,
                      stream=None):
    """csa_index_topk_verify: iq [B, T, Hi, Di], iw [B, T, Hi]; sel [B, T, topk], n_sel [B, T]; pos [B] is the
    position of each block's first token."""
    _expect("iq", iq, layer.dtype)
    if iq.dim() != 4 or iq.shape[2:] != (layer.Hi, layer.Di):
        raise ValueError(f"iq: shape {tuple(iq.shape)}, expected [B, T, {layer.Hi}, {layer.Di}]")
    B, T = iq.shape[0], iq.shape[1]
    _expect("iw", iw, layer.dtype, (B, T, layer.Hi))
    _expect_pool("ikeys", layer, ikeys, layer.Di, B)
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("pos", pos, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect("sel", sel, torch.int32, (B, T, layer.topk))
    _expect("n_sel", n_sel, torch.int32, (B, T))
    _expect_err(err)
    cap = ikeys.shape[1]
    ws, nb = _ws(layer, OP_INDEX_TOPK, B * T, 1, cap, ws, iq.device, stream)
    err = _err(err, iq.device, stream)
    L = layer._c()
    _check("csa_index_topk_verify", load_library().csa_index_topk_verify(
        ctypes.byref(L), _ptr(iq), _ptr(iw), B, T, _ptr(ikeys), cap, _ptr(n_rows), _ptr(pos), _ptr(inv_freq),
        _ptr(sel), _ptr(n_sel), _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def attend_verify(layer: Layer, q, kv_new, sink, window, pool, n_rows, sel, n_sel, pos, inv_freq, out, ws=None,
                  err=None, stream=None):
    """csa_attend_verify: q [B, T, H, D], kv_new [B, T, D], out [B, T, H, D]; the block's tokens are written to the
    window ring first (the layer needs rollback >= T - 1)."""
    _expect("q", q, layer.dtype)
    if q.dim() != 4 or q.shape[2:] != (layer.H, layer.D):
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [B, T, {layer.H}, {layer.D}]")
    B, T = q.shape[0], q.shape[1]
    _expect("kv_new", kv_new, layer.dtype, (B, T, layer.D))
    _expect("sink", sink, torch.float32, (layer.H,))
    _expect("window", window, layer.dtype, (B, layer.ring_slots, layer.D))
    _expect("pool", pool, layer.dtype)
    if pool.dim() != 3 or pool.shape[0] != B or pool.shape[2] != layer.D:
        raise ValueError(f"pool: shape {tuple(pool.shape)}, expected [{B}, cap, {layer.D}]")
    _expect("n_rows", n_rows, torch.int32, (B,))
    _expect("sel", sel, torch.int32, (B, T, layer.topk))
    _expect("n_sel", n_sel, torch.int32, (B, T))
    _expect("pos", pos, torch.int32, (B,))
    _expect("inv_freq", inv_freq, torch.float32, (layer.R // 2,))
    _expect("out", out, layer.dtype, (B, T, layer.H, layer.D))
    _expect_err(err)
    cap = pool.shape[1]
    ws, nb = _ws(layer, OP_ATTEND_DECODE, B * T, 1, cap, ws, q.device, stream)
    err = _err(err, q.device, stream)
    L = layer._c()
    _check("csa_attend_verify", load_library().csa_attend_verify(
        ctypes.byref(L), _ptr(q), _ptr(kv_new), _ptr(sink), B, T, _ptr(window), _ptr(pool), cap, _ptr(n_rows),
        _ptr(sel), _ptr(n_sel), _ptr(pos), _ptr(inv_freq), _ptr(out), _ptr(ws), nb, _ptr(err), _stream(stream)))
    return err


def _refuse(name: str, t, dtype, shape, dev):
    """Raise what is wrong with one tensor of a tree call."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required") if t is None else TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: CSA tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: CSA tensors must be contiguous")
    raise ValueError(f"{name}: on device {t.get_device()}, the call's tensors are on device {dev}")


def _ptrs(dev: int, *specs) -> list:
    """Addresses of a tree call's tensors, each spec (name, tensor, dtype, shape), after checks of type, shape, device
    and contiguity."""
    if _addresses is not None:
        out = _addresses(dev, *specs)
        if type(out) is list:
            return out
        _refuse(*out, dev)
    out = []
    for name, t, dtype, shape in specs:
        try:
            if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
                out.append(t.data_ptr())
                continue
        except AttributeError:  # no tensor
            pass
        _refuse(name, t, dtype, shape, dev)
    return out


def _tree_err(err, dev, stream):
    if err is None:
        return _new(f"cuda:{dev}", stream, torch.zeros, 1, dtype=torch.int32)
    if not (isinstance(err, torch.Tensor) and err.dtype is torch.int32 and err.numel() >= 1):
        _expect_err(err)
    if err.get_device() != dev:
        raise ValueError(f"err: expected a tensor on device {dev}")
    return err


def _tree_ws(layer, op, B, T, cap, ws, dev, stream):
    """The caller's workspace (the library checks its size), or a new one."""
    if ws is None:
        ws = _new(f"cuda:{dev}", stream, torch.empty, max(workspace_size(layer, op, B, T, cap), 256), dtype=torch.uint8)
    elif not isinstance(ws, torch.Tensor) or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on device {dev}")
    return ws, ws.numel() * ws.element_size()


def _tree_call(fn: str, dev: int, stream, *args):
    """The C call on the tensors' device, on `stream` or that device's current stream."""
    f = getattr(_lib or load_library(), fn)
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        code = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            code = f(*args, raw)
    if code:
        raise CSAError(fn, code)


def _tree_dims(name: str, t, tail: tuple):
    """(B, T, device) of a tensor [B, T, *tail]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 2 + len(tail) or shape[2:] != tail:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [B, T{''.join(', %d' % n for n in tail)}]")
    if not t.is_cuda:
        raise ValueError(f"{name}: CSA tensors must live on a CUDA device")
    return shape[0], shape[1], t.get_device()


def _tree_comp(layer: Layer, comp: Compressor, which: str, dev: int) -> bytes:
    """The bytes of a compressor's C struct after the checks of its weights."""
    n, d = layer.lanes * comp.d, comp.d
    return struct.pack(_COMP_FMT, *_ptrs(
        dev, (f"{which}.wkv", comp.wkv, layer.dtype, (n, layer.X)),
        (f"{which}.wgate", comp.wgate, layer.dtype, (n, layer.X)),
        (f"{which}.ape", comp.ape, torch.float32, (layer.ratio, n)),
        (f"{which}.norm_w", comp.norm_w, torch.float32, (d,))), d)


class RowOutputs(list):
    """norm_rope's outputs, a list of tensors; `err` is the call's device error word tensor."""

    def __init__(self, outs, err):
        super().__init__(outs)
        self.err = err


def norm_rope(layer: Layer, xs, pos=None, inv_freq=None, parent=None, weights=None, norm=None, outs=None, err=None,
              stream=None):
    """csa_norm_rope: every head row of the tensors xs (up to four, each [B, T, heads, dim] or [B, T, dim]) RMS-normed
    (norm[k], default True; weights[k] fp32 [dim] or None) and rotated to its token's position: pos[b] + depth in the
    tree `parent` [B, T], or pos[b] + i without one.  inv_freq None: no rotation (for the calls that rotate by
    themselves).  An x may be a slice of a wider tensor: its heads contiguous, one stride from token to token, at least
    a token's size (an expanded tensor is refused).
    Returns the outputs (`outs`, or new tensors; a new tensor's rows of unused tree slots are zeros) as a list whose `err`
    is the device error word tensor; rows of tokens that it reports (pos[b] < 0, an inconsistent tree) are not written, and
    in a new tensor hold nothing defined unless it has tree slots."""
    n = len(xs)
    if not 1 <= n <= 4:
        raise ValueError(f"norm_rope takes 1 to 4 tensors, got {n}")
    if (weights is not None and len(weights) != n) or (norm is not None and len(norm) != n) or (
            outs is not None and len(outs) != n):
        raise ValueError("weights, norm and outs need one entry per tensor")
    x = xs[0]
    if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4):
        raise ValueError("xs: expected tensors [B, T, heads, dim] or [B, T, dim]")
    B, T = x.shape[:2]
    dev = x.get_device()
    if outs is None:
        new = torch.empty if parent is None else torch.zeros
        outs = [_new(x.device, stream, new, x.shape, dtype=x.dtype) for x in xs]
    rows = b""
    dtype = layer.dtype
    for k in range(n):
        x, out = xs[k], outs[k]
        if not isinstance(x, torch.Tensor) or x.dim() not in (3, 4) or x.shape[:2] != (B, T):
            raise ValueError(f"xs[{k}]: expected [{B}, {T}, heads, dim] or [{B}, {T}, dim]")
        if x.dtype is not dtype:
            raise TypeError(f"xs[{k}]: dtype {x.dtype}, expected {dtype}")
        if not x.is_cuda or x.get_device() != dev:
            raise ValueError(f"xs[{k}]: expected a CUDA tensor on device {dev}")
        shape = x.shape
        heads, dim = (1 if len(shape) == 3 else shape[2]), shape[-1]
        stride = 0
        if not x.is_contiguous():
            st = x.stride()
            stride = st[1] if T > 1 else (st[0] if B > 1 else 0)
            # (a stride below a token's size: a broadcast tensor, or tokens over one another; 0 is 'dense' to the library)
            if st[-1] != 1 or (len(shape) == 4 and heads > 1 and st[2] != dim) or (
                    T > 1 and B > 1 and st[0] != T * st[1]) or (B * T > 1 and stride < heads * dim):
                raise ValueError(f"xs[{k}]: strides {st}; heads must be contiguous, tokens one stride of at least a "
                                 "token apart")
        if not (isinstance(out, torch.Tensor) and out.dtype is dtype and out.shape == shape
                and out.get_device() == dev and out.is_contiguous()):
            _refuse(f"outs[{k}]", out, dtype, shape, dev)
        w = None if weights is None else weights[k]
        p_w = 0 if w is None else _ptrs(dev, (f"weights[{k}]", w, torch.float32, (dim,)))[0]
        rows += struct.pack(_ROWS_FMT, x.data_ptr(), out.data_ptr(), p_w, heads, dim,
                            1 if norm is None or norm[k] else 0, stride)
    p_par = p_pos = p_frq = None
    if parent is not None:
        p_par, = _ptrs(dev, ("parent", parent, torch.int32, (B, T)))
    if inv_freq is not None:
        p_pos, p_frq = _ptrs(dev, ("pos", pos, torch.int32, (B,)),
                             ("inv_freq", inv_freq, torch.float32, (layer.R // 2,)))
    err = _tree_err(err, dev, stream)
    _tree_call("csa_norm_rope", dev, stream, layer._packed(), rows, n, B, T, p_par, p_pos, p_frq, err.data_ptr())
    return RowOutputs(outs, err)


def compress_tree(layer: Layer, comp_a: Compressor, x, parent, pos, frontier_a, proj_a, rows_a, inv_freq, comp_i=None,
                  frontier_i=None, proj_i=None, rows_i=None, ws=None, err=None, stream=None):
    """csa_compress_tree: x [B, T, X], parent [B, T]; writes proj_a [B, T, 2 L D], rows_a [B, T, D] and, with comp_i,
    the index pool's proj_i, rows_i.  The frontiers are read only.  Returns the device error word tensor."""
    dt, i32 = layer.dtype, torch.int32
    B, T, dev = _tree_dims("x", x, (layer.X,))
    F, wide = _frontier_len(layer), 2 * layer.lanes
    Ca = _tree_comp(layer, comp_a, "comp_a", dev)
    p_x, p_par, p_pos, p_fa, p_pa, p_ra, p_frq = _ptrs(
        dev, ("x", x, dt, (B, T, layer.X)), ("parent", parent, i32, (B, T)), ("pos", pos, i32, (B,)),
        ("frontier_a", frontier_a, dt, (B, F, wide * comp_a.d)), ("proj_a", proj_a, dt, (B, T, wide * comp_a.d)),
        ("rows_a", rows_a, dt, (B, T, comp_a.d)), ("inv_freq", inv_freq, torch.float32, (layer.R // 2,)))
    Ci = p_fi = p_pi = p_ri = None
    if comp_i is not None:
        Ci = _tree_comp(layer, comp_i, "comp_i", dev)
        row_dt, row = layer.pool_spec(comp_i.d)
        p_fi, p_pi, p_ri = _ptrs(dev, ("frontier_i", frontier_i, dt, (B, F, wide * comp_i.d)),
                                 ("proj_i", proj_i, dt, (B, T, wide * comp_i.d)), ("rows_i", rows_i, row_dt, (B, T, row)))
    elif not (frontier_i is None and proj_i is None and rows_i is None):
        raise ValueError("frontier_i, proj_i, rows_i come with comp_i")
    ws, nb = _tree_ws(layer, OP_COMPRESS_TREE, B, T, 1, ws, dev, stream)
    err = _tree_err(err, dev, stream)
    _tree_call("csa_compress_tree", dev, stream, layer._packed(), Ca, Ci, p_x, B, T, p_par, p_pos, p_fa, p_pa, p_ra,
               p_fi, p_pi, p_ri, p_frq, ws.data_ptr(), nb, err.data_ptr())
    return err


def index_scores_tree(layer: Layer, iq, iw, ikeys, rows_i, parent, n_rows, pos, scores, ws=None, err=None,
                      stream=None):
    """csa_index_scores_tree: rotated iq [B, T, Hi, Di], iw [B, T, Hi], ikeys [B, cap, Di], rows_i [B, T, Di] (both
    uint8 [..., FP8_ROW_BYTES] with index_fp8, which alone needs ws); writes scores [B, T, cap + T] (fp32).  Returns
    the device error word tensor."""
    dt, i32, Hi, Di = layer.dtype, torch.int32, layer.Hi, layer.Di
    B, T, dev = _tree_dims("iq", iq, (Hi, Di))
    if not isinstance(ikeys, torch.Tensor) or ikeys.dim() != 3:
        raise ValueError(f"ikeys: expected [{B}, cap, {Di}]")
    cap = ikeys.shape[1]
    key_dt, row = layer.pool_spec(Di)
    p = _ptrs(dev, ("iq", iq, dt, (B, T, Hi, Di)), ("iw", iw, dt, (B, T, Hi)), ("parent", parent, i32, (B, T)),
              ("ikeys", ikeys, key_dt, (B, cap, row)), ("rows_i", rows_i, key_dt, (B, T, row)),
              ("n_rows", n_rows, i32, (B,)), ("pos", pos, i32, (B,)),
              ("scores", scores, torch.float32, (B, T, cap + T)))
    p_ws, nb = None, 0
    if layer.index_fp8:
        ws, nb = _tree_ws(layer, OP_INDEX_SCORES_TREE, B, T, cap, ws, dev, stream)
        p_ws = ws.data_ptr()
    err = _tree_err(err, dev, stream)
    _tree_call("csa_index_scores_tree", dev, stream, layer._packed(), p[0], p[1], B, T, p[2], p[3], cap, p[4], p[5],
               p[6], p[7], p_ws, nb, err.data_ptr())
    return err


def attend_tree(layer: Layer, q, kv, sink, window, pool, rows_a, scores, parent, n_rows, pos, inv_freq, out,
                sel_out=None, ws=None, err=None, stream=None):
    """csa_attend_tree: rotated q [B, T, H, D] and kv [B, T, D]; scores [B, T, cap + T] of index_scores_tree, or None
    (every visible row); out [B, T, H, D]; sel_out [B, T, topk] int32 or None.  The cache is read only.  Returns the
    device error word tensor."""
    dt, i32, f32, H, D = layer.dtype, torch.int32, torch.float32, layer.H, layer.D
    B, T, dev = _tree_dims("q", q, (H, D))
    if not isinstance(pool, torch.Tensor) or pool.dim() != 3:
        raise ValueError(f"pool: expected [{B}, cap, {D}]")
    cap = pool.shape[1]
    p_q, p_kv, p_sink, p_par, p_win, p_pool, p_rows, p_n, p_pos, p_frq, p_out = _ptrs(
        dev, ("q", q, dt, (B, T, H, D)), ("kv", kv, dt, (B, T, D)), ("sink", sink, f32, (H,)),
        ("parent", parent, i32, (B, T)), ("window", window, dt, (B, layer.ring_slots, D)),
        ("pool", pool, dt, (B, cap, D)), ("rows_a", rows_a, dt, (B, T, D)), ("n_rows", n_rows, i32, (B,)),
        ("pos", pos, i32, (B,)), ("inv_freq", inv_freq, f32, (layer.R // 2,)), ("out", out, dt, (B, T, H, D)))
    p_sc = p_sel = None
    if scores is not None:
        p_sc, = _ptrs(dev, ("scores", scores, f32, (B, T, cap + T)))
    if sel_out is not None:
        p_sel, = _ptrs(dev, ("sel_out", sel_out, i32, (B, T, layer.topk)))
    ws, nb = _tree_ws(layer, OP_ATTEND_TREE, B, T, cap, ws, dev, stream)
    err = _tree_err(err, dev, stream)
    _tree_call("csa_attend_tree", dev, stream, layer._packed(), p_q, p_kv, p_sink, B, T, p_par, p_win, p_pool, cap,
               p_rows, p_sc, p_n, p_pos, p_frq, p_out, p_sel, ws.data_ptr(), nb, err.data_ptr())
    return err


def commit_tree(layer: Layer, parent, leaf, pos, n_rows_a, kv, window, proj_a, frontier_a, rows_a, pool_a,
                n_rows_i=None, proj_i=None, frontier_i=None, rows_i=None, pool_i=None, pos_out=None, n_rows_a_out=None,
                n_rows_i_out=None, err=None, stream=None):
    """csa_commit_tree: the path to leaf[b] (int32 [B]; -1: nothing accepted) enters the cache.  pos, n_rows_a and
    n_rows_i advance in place unless pos_out, n_rows_a_out, n_rows_i_out are given.  The index pool's arguments come
    together or not at all.  Returns the device error word tensor."""
    B, T, dev = _tree_dims("parent", parent, ())
    dt, i32, D, F, vec = layer.dtype, torch.int32, layer.D, _frontier_len(layer), (B,)
    wide = 2 * layer.lanes

    if not isinstance(pool_a, torch.Tensor) or pool_a.dim() != 3:
        raise ValueError(f"pool_a: expected [{B}, cap, {D}]")
    cap_a, wide_a = pool_a.shape[1], wide * D
    specs = [("parent", parent, i32, (B, T)), ("leaf", leaf, i32, vec), ("pos", pos, i32, vec),
             ("pos_out", pos if pos_out is None else pos_out, i32, vec), ("kv", kv, dt, (B, T, D)),
             ("window", window, dt, (B, layer.ring_slots, D)), ("proj_a", proj_a, dt, (B, T, wide_a)),
             ("frontier_a", frontier_a, dt, (B, F, wide_a)), ("rows_a", rows_a, dt, (B, T, D)),
             ("pool_a", pool_a, dt, (B, cap_a, D)), ("n_rows_a", n_rows_a, i32, vec),
             ("n_rows_a_out", n_rows_a if n_rows_a_out is None else n_rows_a_out, i32, vec)]
    if pool_i is not None:
        row_dt, row = layer.pool_spec(layer.Di)
        if not isinstance(pool_i, torch.Tensor) or pool_i.dim() != 3:
            raise ValueError(f"pool_i: expected [{B}, cap, {row}]")
        cap_i, wide_i = pool_i.shape[1], wide * layer.Di
        specs += (("proj_i", proj_i, dt, (B, T, wide_i)), ("frontier_i", frontier_i, dt, (B, F, wide_i)),
                  ("rows_i", rows_i, row_dt, (B, T, row)), ("pool_i", pool_i, row_dt, (B, cap_i, row)),
                  ("n_rows_i", n_rows_i, i32, vec),
                  ("n_rows_i_out", n_rows_i if n_rows_i_out is None else n_rows_i_out, i32, vec))
    elif any(t is not None for t in (n_rows_i, proj_i, frontier_i, rows_i, n_rows_i_out)):
        raise ValueError("n_rows_i, proj_i, frontier_i, rows_i, n_rows_i_out come with pool_i")
    p = _ptrs(dev, *specs)
    pi = (None, None, None, None, 0, None, None) if pool_i is None else (*p[12:16], cap_i, *p[16:])
    err = _tree_err(err, dev, stream)
    _tree_call("csa_commit_tree", dev, stream, layer._packed(), B, T, *p[:10], cap_a, *p[10:12], *pi, err.data_ptr())
    return err


def _row_stride(name: str, t, width: int) -> int:
    """Elements between the rows of a tensor [.., width] whose rows are one stride apart and contiguous themselves (0:
    dense)."""
    if t.is_contiguous():
        return 0
    shape, st = t.shape, t.stride()
    lead = [(n, k) for n, k in zip(shape[:-1], st[:-1]) if n != 1]
    ok = st[-1] == 1 or width == 1
    for (_, k), (n, inner) in zip(lead, lead[1:]):
        ok = ok and k == n * inner
    step = lead[-1][1] if lead else 0
    if not ok or (lead and step < width):
        raise ValueError(f"{name}: strides {st}; rows must be contiguous, one stride of at least a row apart")
    return step


class NormOutputs(tuple):
    """add_norm's outputs (out, residual_out, codes, scales); None for what was not asked for."""

    out = property(lambda self: self[0])
    residual = property(lambda self: self[1])
    codes = property(lambda self: self[2])
    scales = property(lambda self: self[3])


def add_norm(layer: Layer, x, residual=None, weight=None, group=None, out=None, residual_out=None, codes=None,
             scales=None, stream=None):
    """csa_add_norm: rows x [.., X] (+ residual [.., X]) RMS-normed (weight fp32 [X] or None); with `group` also in 8
    bits: codes uint8 [.., X] (E4M3) and scales fp32 [.., X / group], of groups of 8 to 256 values (a power of two) or
    whole rows (group = X).  Outputs are those given, or new tensors; out=False or residual_out=False leaves that one
    out (the latter also where there is no residual).  residual_out may be x or residual itself, and so may out.  Rows of
    x and residual may be a stride apart.  Returns (out, residual_out, codes, scales) as NormOutputs."""
    if _plain is not None:
        code = _plain.add_norm(_at["add_norm"], layer._packed(), layer.dtype, x, residual, weight, group, out,
                               residual_out, codes, scales, stream)
        if code is not None:
            if code:
                raise CSAError("csa_add_norm", code)
            return NormOutputs((None if out is False else out, None if residual_out is False else residual_out, codes,
                                scales))
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise TypeError("x: expected a tensor [.., X]")
    dtype, shape = layer.dtype, x.shape
    X = shape[-1]
    if x.dtype is not dtype:
        raise TypeError(f"x: dtype {x.dtype}, expected {dtype}")
    if not x.is_cuda:
        raise ValueError("x: CSA tensors must live on a CUDA device")
    if X > 16384:
        raise ValueError(f"x: rows of {X} values, at most 16384")
    dev = x.get_device()
    N = x.numel() // X if X else 0
    x_stride = _row_stride("x", x, X)
    if out is None:
        out = _new(x.device, stream, torch.empty, shape, dtype=dtype)
    if residual is None:
        if residual_out is not None and residual_out is not False:
            raise ValueError("residual_out comes with residual")
    elif residual_out is None:
        residual_out = _new(x.device, stream, torch.empty, shape, dtype=dtype)
    specs, r_stride = [], 0
    if residual is not None:
        if not (isinstance(residual, torch.Tensor) and residual.dtype is dtype and residual.shape == shape
                and residual.get_device() == dev):
            _refuse("residual", residual, dtype, shape, dev)
        r_stride = _row_stride("residual", residual, X)
    if weight is not None:
        specs.append(("weight", weight, torch.float32, (X,)))
    has_out, has_res = out is not False, residual_out is not None and residual_out is not False
    if has_out:
        specs.append(("out", out, dtype, shape))
    if has_res:
        specs.append(("residual_out", residual_out, dtype, shape))
    if group is not None:
        if group < 1 or X % group:
            raise ValueError(f"group = {group}: expected a divisor of {X}")
        few = (*shape[:-1], X // group)
        if codes is None:
            codes = _new(x.device, stream, torch.empty, shape, dtype=torch.uint8)
        if scales is None:
            scales = _new(x.device, stream, torch.empty, few, dtype=torch.float32)
        specs += (("codes", codes, torch.uint8, shape), ("scales", scales, torch.float32, few))
    elif codes is not None or scales is not None:
        raise ValueError("codes and scales come with group")
    p = iter(_ptrs(dev, *specs))
    p_w = next(p) if weight is not None else None
    p_out = next(p) if has_out else None
    p_res = next(p) if has_res else None
    p_codes, p_scales = (next(p), next(p)) if group is not None else (None, None)
    _tree_call("csa_add_norm", dev, stream, layer._packed(), x.data_ptr(), x_stride,
               None if residual is None else residual.data_ptr(), r_stride, p_w, N, X, p_out, p_res, p_codes, p_scales,
               group or 0)
    return NormOutputs((out if has_out else None, residual_out if has_res else None, codes, scales))


@dataclass(frozen=True)
class Pages:
    """A pool of cache pages in 8 bits (csa_pages): codes uint8 [n_pages, page_rows, D] (E4M3), scales fp32 [n_pages,
    page_rows]; a row stands for scale * code."""

    codes: torch.Tensor
    scales: torch.Tensor

    def _specs(self, layer: Layer) -> tuple:
        """What _ptrs checks of the pool's two tensors."""
        c = self.codes
        if not isinstance(c, torch.Tensor) or c.dim() != 3 or c.shape[2] != layer.D:
            raise ValueError(f"Pages.codes: expected a uint8 tensor [n_pages, page_rows, {layer.D}]")
        shape = c.shape
        return ("Pages.codes", c, torch.uint8, shape), ("Pages.scales", self.scales, torch.float32, shape[:2])

    def _packed(self, p_codes: int, p_scales: int) -> bytes:
        n, rows = self.scales.shape
        return struct.pack(_PAGES_FMT, p_codes, p_scales, n, rows)


def _table(name: str, t, B: int):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[0] != B:
        raise ValueError(f"{name}: expected an int32 tensor [{B}, pages of a sequence]")
    if t.shape[1] > 1 << 30:
        raise ValueError(f"{name}: {t.shape[1]} pages, at most 2^30 rows")
    return (name, t, torch.int32, t.shape)


def append_pages(layer: Layer, rows, pages: Pages, table, pos, n_new=None, weight=None, norm=False, inv_freq=None,
                 err=None, stream=None):
    """csa_append_pages: rows [B, T, D] become logical rows pos[b] .. pos[b] + n_new[b] - 1 (n_new None: T each) of the
    sequences' tables [B, width]: RMS-normed (norm, with weight fp32 [D] or None), rotated to those positions (inv_freq;
    None: not rotated) and put in 8 bits with a scale per row.  A token of rows is contiguous; tokens and sequences may be
    strides apart.  Compressed rows that compress_append put into its pool come as pool.gather(1, ..) at n_rows as it was before,
    ceil(T / ratio) of them, with n_new = n_rows - before: all on the device.  Returns the device error word tensor."""
    if _plain is not None:
        code = _plain.append_pages(_at["append_pages"], layer._packed(), layer.dtype, layer.D, layer.R // 2, rows,
                                   pages.codes, pages.scales, table, pos, n_new, weight, norm, inv_freq, err, stream)
        if code is not None:
            if code:
                raise CSAError("csa_append_pages", code)
            return err
    D, i32, f32 = layer.D, torch.int32, torch.float32
    B, T, dev = _tree_dims("rows", rows, (D,))
    if rows.dtype is not layer.dtype:
        raise TypeError(f"rows: dtype {rows.dtype}, expected {layer.dtype}")
    if B * T > 1 << 24:
        raise ValueError(f"rows: {B} x {T} tokens, at most 2^24 a call")
    stride_b = stride_t = 0
    if not rows.is_contiguous():
        st = rows.stride()
        if st[2] != 1 or (T > 1 and st[1] < D) or (B > 1 and st[0] < D):
            raise ValueError(f"rows: strides {st}; a token must be contiguous, tokens and sequences at least one apart")
        stride_t = st[1] if T > 1 else 0
        stride_b = st[0] if B > 1 else 0
    if weight is not None and not norm:
        raise ValueError("weight comes with norm")
    specs = [*pages._specs(layer), _table("table", table, B), ("pos", pos, i32, (B,))]
    if n_new is not None:
        specs.append(("n_new", n_new, i32, (B,)))
    if weight is not None:
        specs.append(("weight", weight, f32, (D,)))
    if inv_freq is not None:
        specs.append(("inv_freq", inv_freq, f32, (layer.R // 2,)))
    p = iter(_ptrs(dev, *specs))
    handle = pages._packed(next(p), next(p))
    p_table, p_pos = next(p), next(p)
    p_new = next(p) if n_new is not None else None
    p_w = next(p) if weight is not None else None
    p_frq = next(p) if inv_freq is not None else None
    err = _tree_err(err, dev, stream)
    _tree_call("csa_append_pages", dev, stream, layer._packed(), handle, rows.data_ptr(), stride_b, stride_t, B, T,
               p_table, table.shape[1], p_pos, p_new, p_w, 1 if norm else 0, p_frq, err.data_ptr())
    return err


def attend_pages(layer: Layer, q, pages: Pages, sink, pos, out, token_table=None, first=0, row_table=None, n_rows=None,
                 sel=None, n_sel=None, n_new=None, inv_freq=None, ws=None, err=None, stream=None):
    """csa_attend_pages: rotated q [B, T, H, D], query i of sequence b at pos[b] + i, over the rows of a paged cache: the
    last W tokens and the first `first` ones of token_table [B, width] (None: no tokens), and of row_table [B, width]
    (None: no compressed rows) the rows sel [B, T, topk] with counts n_sel [B, T], or without sel every visible row below
    n_rows [B].  sink fp32 [H] or None; n_new int32 [B]: the queries of each sequence (None: T); inv_freq: out
    [B, T, H, D] is rotated back (None: not).  Returns the device error word tensor."""
    if _plain is not None:
        code = _plain.attend_pages(_at["attend_pages"], layer._packed(), layer.dtype, layer.H, layer.D, layer.R // 2,
                                   layer.topk, q, pages.codes, pages.scales, sink, pos, out, token_table, first,
                                   row_table, n_rows, sel, n_sel, n_new, inv_freq, ws, err, stream)
        if code is not None:
            if code:
                raise CSAError("csa_attend_pages", code)
            return err
    dt, i32, f32, H, D = layer.dtype, torch.int32, torch.float32, layer.H, layer.D
    B, T, dev = _tree_dims("q", q, (H, D))
    if B * T > 1 << 16:
        raise ValueError(f"q: {B} x {T} queries, at most 2^16 a call")
    if not 0 <= first <= 0x7fffffff:
        raise ValueError(f"first = {first}: expected a count of tokens")
    if token_table is None and row_table is None:
        raise ValueError("attend_pages needs token_table, row_table, or both")
    if row_table is None and not (n_rows is None and sel is None and n_sel is None):
        raise ValueError("n_rows, sel, n_sel come with row_table")
    if (sel is None) != (n_sel is None):
        raise ValueError("sel and n_sel come together")
    specs = [*pages._specs(layer), ("q", q, dt, (B, T, H, D)), ("pos", pos, i32, (B,)), ("out", out, dt, (B, T, H, D))]
    if sink is not None:
        specs.append(("sink", sink, f32, (H,)))
    if token_table is not None:
        specs.append(_table("token_table", token_table, B))
    if row_table is not None:
        specs += (_table("row_table", row_table, B), ("n_rows", n_rows, i32, (B,)))
    if sel is not None:
        specs += (("sel", sel, i32, (B, T, layer.topk)), ("n_sel", n_sel, i32, (B, T)))
    if n_new is not None:
        specs.append(("n_new", n_new, i32, (B,)))
    if inv_freq is not None:
        specs.append(("inv_freq", inv_freq, f32, (layer.R // 2,)))
    p = iter(_ptrs(dev, *specs))
    handle = pages._packed(next(p), next(p))
    p_q, p_pos, p_out = next(p), next(p), next(p)
    p_sink = next(p) if sink is not None else None
    p_tok = next(p) if token_table is not None else None
    p_row, p_n = (next(p), next(p)) if row_table is not None else (None, None)
    p_sel, p_ns = (next(p), next(p)) if sel is not None else (None, None)
    p_new = next(p) if n_new is not None else None
    p_frq = next(p) if inv_freq is not None else None
    ws, nb = _tree_ws(layer, OP_ATTEND_PAGES, B, T, 1, ws, dev, stream)
    err = _tree_err(err, dev, stream)
    _tree_call("csa_attend_pages", dev, stream, layer._packed(), handle, p_q, B, T, p_sink, p_pos, p_new, p_tok,
               0 if p_tok is None else token_table.shape[1], first, p_row, 0 if p_row is None else row_table.shape[1],
               p_n, p_sel, p_ns, p_frq, p_out, ws.data_ptr(), nb, err.data_ptr())
    return err
