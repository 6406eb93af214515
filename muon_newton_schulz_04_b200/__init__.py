"""Python binding of the B200 Muon step library (include/muon.h).

Argument marshalling only: torch tensors are turned into raw pointers, sizes
and the current CUDA stream, and every entry point of the C ABI is called by
the same name.  All arithmetic runs in the CUDA kernels of libmuon_b200.so;
there is no fallback.  If the shared library is missing, the first call raises.

    import torch, muon_newton_schulz_04_b200 as mb
    opt = mb.Muon(mb.config(lr=0.02, weight_decay=0.1))
    opt.step([mb.Group(W=[w1, w2], G=[g1, g2], B=[b1, b2])])   # same-shape matrices per group
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct
from typing import List, Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon_b200.so")

MUON_OK, MUON_ERR_INVALID, MUON_ERR_UNSUPPORTED, MUON_ERR_OOM, MUON_ERR_CUDA, MUON_ERR_DEVICE_TIMEOUT = range(6)
MUON_BF16, MUON_FP32 = 0, 1
MUON_FILL_OUT, MUON_FILL_LSE, MUON_FILL_DQ, MUON_FILL_DK, MUON_FILL_DV = 1, 2, 4, 8, 16
PREC_BF16, PREC_FP32_DEBUG = 0, 1
SCALE_NONE, SCALE_MATCH_RMS, SCALE_CUSTOM = 0, 1, 2
NS_GRAM, NS_POLY, NS_UPDATE = 0, 1, 2


class MuonConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("eps", ctypes.c_float), ("rms_target", ctypes.c_float), ("nesterov", ctypes.c_int),
                ("ns_steps", ctypes.c_int), ("ns_a", ctypes.c_float), ("ns_b", ctypes.c_float),
                ("ns_c", ctypes.c_float), ("scale_mode", ctypes.c_int), ("precision", ctypes.c_int)]


class _Group(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("count", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("W", ctypes.POINTER(ctypes.c_void_p)), ("G", ctypes.POINTER(ctypes.c_void_p)),
                ("B", ctypes.POINTER(ctypes.c_void_p))]


class _OrthoGroup(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("count", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("M", ctypes.POINTER(ctypes.c_void_p)),
                ("O", ctypes.POINTER(ctypes.c_void_p))]


class _DirGroup(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("count", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("G", ctypes.POINTER(ctypes.c_void_p)), ("B", ctypes.POINTER(ctypes.c_void_p)),
                ("O", ctypes.POINTER(ctypes.c_void_p))]


class _ApplyGroup(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("count", ctypes.c_int),
                ("o_dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("W", ctypes.POINTER(ctypes.c_void_p)), ("O", ctypes.POINTER(ctypes.c_void_p))]


class _PhaseArgs(ctypes.Structure):
    _fields_ = [("phase", ctypes.c_int), ("precision", ctypes.c_int), ("m", ctypes.c_int), ("n", ctypes.c_int),
                ("count", ctypes.c_int), ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("x_op", ctypes.c_void_p), ("a_in", ctypes.c_void_p), ("x_master", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("out_op", ctypes.c_void_p)]


class _Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class _AttentionArgs(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int), ("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("total_q", ctypes.c_int), ("total_k", ctypes.c_int),
                ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("q", _Heads), ("k", _Heads), ("v", _Heads), ("out", _Heads),
                ("lse", ctypes.c_void_p), ("max_logits", ctypes.c_void_p)]


class _AttentionGradArgs(ctypes.Structure):
    _fields_ = [("forward", _AttentionArgs), ("grad_out", _Heads), ("dq", _Heads), ("dk", _Heads), ("dv", _Heads),
                ("delta", ctypes.c_void_p)]


class _WeightGradArgs(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("dy", ctypes.c_void_p),
                ("dy_stride", ctypes.c_longlong), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("G", ctypes.c_void_p), ("grad_dtype", ctypes.c_int), ("accumulate", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


# the two attention structures as one pack call each (a third of the time of filling the
# ctypes structures field by field)
_ATTENTION_PACK = struct.Struct("@6i2Pf" + "P2q" * 4 + "2P")
_ATTENTION_GRAD_PACK = struct.Struct("@6i2Pf" + "P2q" * 4 + "2P" + "P2q" * 4 + "P")
assert (_ATTENTION_PACK.size, _ATTENTION_GRAD_PACK.size) == (ctypes.sizeof(_AttentionArgs),
                                                             ctypes.sizeof(_AttentionGradArgs))

_LIB: Optional[ctypes.CDLL] = None
_raw_stream = None
torch = None        # imported by the first handle: building the library and planning need no torch

# name -> (restype, argtypes)
_SIGNATURES = {
    "muon_config_default": (None, [ctypes.POINTER(MuonConfig)]),
    "muon_validate_config": (ctypes.c_int, [ctypes.POINTER(MuonConfig)]),
    "muon_validate_groups": (ctypes.c_int, [ctypes.POINTER(_Group), ctypes.c_int]),
    "muon_create": (ctypes.c_int, [ctypes.POINTER(MuonConfig), ctypes.c_int, ctypes.POINTER(ctypes.c_void_p)]),
    "muon_set_config": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(MuonConfig)]),
    "muon_set_memory_limit": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t]),
    "muon_memory_held": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
    "muon_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_Group), ctypes.c_int, ctypes.c_void_p]),
    "muon_step_host": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_Group), ctypes.c_int, ctypes.c_void_p]),
    "muon_step_direction": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_DirGroup), ctypes.c_int, ctypes.c_void_p]),
    "muon_apply": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_ApplyGroup), ctypes.c_int, ctypes.c_void_p]),
    "muon_orthogonalize": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_OrthoGroup), ctypes.c_int, ctypes.c_void_p]),
    "muon_ns_phase_run": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_PhaseArgs), ctypes.c_void_p]),
    "muon_qk_clip": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p]),
    "muon_qk_clip_grouped": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                                            ctypes.c_void_p]),
    "muon_validate_attention": (ctypes.c_int, [ctypes.POINTER(_AttentionArgs)]),
    "muon_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_AttentionArgs), ctypes.c_void_p]),
    "muon_validate_attention_grad": (ctypes.c_int, [ctypes.POINTER(_AttentionGradArgs)]),
    "muon_attention_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_AttentionGradArgs), ctypes.c_void_p]),
    "muon_attention_fill": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_AttentionArgs), ctypes.c_int,
                                           ctypes.c_void_p]),
    "muon_attention_backward_fill": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_AttentionGradArgs), ctypes.c_int,
                                                    ctypes.c_void_p]),
    "muon_checkpoint_store": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "muon_checkpoint_load": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                            ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong,
                                            ctypes.c_void_p]),
    "muon_weight_grad_workspace": (ctypes.c_int, [ctypes.POINTER(_WeightGradArgs), ctypes.POINTER(ctypes.c_size_t)]),
    "muon_validate_weight_grad": (ctypes.c_int, [ctypes.POINTER(_WeightGradArgs)]),
    "muon_weight_grad": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(_WeightGradArgs), ctypes.c_void_p]),
    "muon_sync": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "muon_last_norms": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_float), ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int), ctypes.c_void_p]),
    "muon_last_update_rms": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_float), ctypes.c_int,
                                            ctypes.POINTER(ctypes.c_int), ctypes.c_void_p]),
    "muon_last_update": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "muon_timing_enable": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "muon_timing_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int),
                                        ctypes.c_int, ctypes.c_void_p]),
    "muon_destroy": (ctypes.c_int, [ctypes.c_void_p]),
    "muon_last_error": (ctypes.c_char_p, [ctypes.c_void_p]),
    "muon_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "muon_momentum_norm_noalloc": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_int,
                                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_char_p, ctypes.c_int]),
    "muon_plan_units": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int)]),
    "muon_plan_tile_m": (ctypes.c_int, []),
    "muon_plan_tile_n": (ctypes.c_int, []),
    "muon_plan_tiles": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int), ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
}


def lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if libmuon_b200.so has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m muon_newton_schulz_04_b200.build` "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


class MuonError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{lib().muon_status_string(status).decode()}: {msg}")
        self.status = status


def config(**kw) -> MuonConfig:
    """Default configuration (lr 0.02, momentum 0.95 Nesterov, 5 steps, (3.4445, -4.775, 2.0315), eps 1e-7)
    with the given fields replaced."""
    c = MuonConfig()
    lib().muon_config_default(ctypes.byref(c))
    for k, v in kw.items():
        if k not in dict(MuonConfig._fields_):
            raise TypeError(f"unknown config field {k}")
        setattr(c, k, int(v) if isinstance(getattr(c, k), int) else float(v))
    return c


@dataclasses.dataclass
class Group:
    """Same-shape matrices: W (fp32, updated), G (bf16 or fp32), B (fp32 momentum, updated)."""
    W: Sequence
    G: Sequence
    B: Sequence
    scale: float = 1.0


def _import_torch():
    global torch
    if torch is None:
        import torch as module
        torch = module


CKPT_BLOCK = 32     # values of an 8-bit checkpoint that share a scale


@dataclasses.dataclass
class Checkpoint:
    """An activation in 8 bits (see muon_checkpoint_store): codes int8 [rows, cols rounded up to CKPT_BLOCK],
    scales uint8 [rows, that / CKPT_BLOCK]; value = code * 2**(scale - 133), NaN where the scale is 255."""
    codes: object
    scales: object
    cols: int

    @staticmethod
    def empty(rows: int, cols: int, device) -> "Checkpoint":
        _import_torch()
        blocks = -(-cols // CKPT_BLOCK)
        return Checkpoint(torch.empty(rows, blocks * CKPT_BLOCK, dtype=torch.int8, device=device),
                          torch.empty(rows, blocks, dtype=torch.uint8, device=device), cols)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]


def _check_checkpoint(ckpt: Checkpoint, device: int):
    rows, cols = ckpt.codes.shape
    blocks = -(-ckpt.cols // CKPT_BLOCK)
    if cols != blocks * CKPT_BLOCK or tuple(ckpt.scales.shape) != (rows, blocks):
        raise ValueError(f"a checkpoint of {rows} x {ckpt.cols} values has codes [{rows}, {blocks * CKPT_BLOCK}] and "
                         f"scales [{rows}, {blocks}], got {tuple(ckpt.codes.shape)} and {tuple(ckpt.scales.shape)}")
    if ckpt.codes.dtype != torch.int8 or ckpt.scales.dtype != torch.uint8:
        raise ValueError("expected int8 codes and uint8 scales")
    _check_dense("codes", ckpt.codes, device)
    _check_dense("scales", ckpt.scales, device)


def _check_dense(name: str, t, device: int):
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the handle on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_sizes(name: str, *sizes: int):
    """The C library takes sizes as int, and ctypes would cut larger ones off without a word."""
    if max(sizes) >= 1 << 31:
        raise ValueError(f"{name}: sizes must be below 2^31, got {' x '.join(map(str, sizes))}")


def _heads(name: str, t, shape, device: int):
    """(address, row stride, head stride) of a bf16 CUDA tensor [rows, heads, head_dim] of the given shape with a
    dense last dimension."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}, expected torch.bfloat16")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the handle on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    rows, heads, last = t.stride()
    if last != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    return t.data_ptr(), rows, heads


def _check_rows(name: str, t, device: int):
    """A 2-D CUDA tensor with dense rows; returns its row stride."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with dense rows")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the handle on cuda:{device}")
    return t.stride(0)


def _ptrs(ts) -> "ctypes.Array":
    arr = (ctypes.c_void_p * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = t.data_ptr()
    return arr


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    if t.dtype == torch.float32:
        return MUON_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check_tensors(ts, shape, on_cuda: bool, dtype=None, device: Optional[int] = None):
    """Same shape, dense, on the expected device kind and, when given, of one dtype
    (the library reads and writes these buffers as dense arrays of that type) and on
    CUDA device `device` (the kernels run on one device and take only its memory)."""
    for t in ts:
        if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"expected contiguous tensors of shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.is_cuda != on_cuda:
            raise ValueError("tensor on the wrong device kind")
        if on_cuda and device is not None and t.device.index != device:
            raise ValueError(f"tensor on cuda:{t.device.index}, expected cuda:{device}")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"expected {dtype} tensors, got {t.dtype}")


def _stream(stream, device: Optional[int] = None) -> int:
    """The raw cudaStream_t: the given stream, else the current stream of `device`
    (of the current device when None)."""
    global _raw_stream
    if stream is None:
        if _raw_stream is not None and device is not None:
            return _raw_stream(device)
        _import_torch()
        raw = torch.cuda.current_stream(device).cuda_stream
        # from now on (CUDA is initialised) what that asks, without the stream object: 1 us less a call
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """A new tensor on the device of `like` for work on `stream` (a torch stream, a raw cudaStream_t or None for the
    current one): the caching allocator reuses memory in the order of the stream that it was allocated on.  With `shape`
    None it has the shape and type of `like`.  (`empty_like` takes 1.3 us, `new_empty` 1.9, `torch.empty` 3.)"""
    if stream is None:
        if shape is None:
            return torch.empty_like(like, memory_format=torch.contiguous_format)
        return like.new_empty(shape, dtype=dtype)
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=like.device) if stream
                  else torch.cuda.default_stream(like.device))
    with torch.cuda.stream(stream):
        return _empty(shape, dtype, like, None)


class Muon:
    """A handle of the C library bound to one CUDA device."""

    def __init__(self, cfg: Optional[MuonConfig] = None, device: int = 0):
        _import_torch()
        self._h = ctypes.c_void_p()
        self.cfg = cfg if cfg is not None else config()
        st = lib().muon_create(ctypes.byref(self.cfg), int(device), ctypes.byref(self._h))
        if st != MUON_OK:
            raise MuonError(st, f"muon_create on device {device}")
        self.device = device
        self._keep = []

    # ------------------------------------------------------------------ helpers
    def _check(self, st: int, what: str):
        if st != MUON_OK:
            raise MuonError(st, f"{what}: {lib().muon_last_error(self._h).decode()}")

    def _groups(self, groups: List[Group], on_cuda: bool):
        arr = (_Group * len(groups))()
        keep = []
        for i, g in enumerate(groups):
            import torch
            rows, cols = g.W[0].shape
            _check_tensors(g.W, (rows, cols), on_cuda, torch.float32, self.device)
            _check_tensors(g.G, (rows, cols), on_cuda, g.G[0].dtype, self.device)
            _check_tensors(g.B, (rows, cols), on_cuda, torch.float32, self.device)
            if not (len(g.W) == len(g.G) == len(g.B)):
                raise ValueError("W, G and B lists differ in length")
            pw, pg, pb = _ptrs(g.W), _ptrs(g.G), _ptrs(g.B)
            keep += [pw, pg, pb]
            arr[i] = _Group(rows, cols, len(g.W), _dtype_code(g.G[0]), float(g.scale),
                            ctypes.cast(pw, ctypes.POINTER(ctypes.c_void_p)),
                            ctypes.cast(pg, ctypes.POINTER(ctypes.c_void_p)),
                            ctypes.cast(pb, ctypes.POINTER(ctypes.c_void_p)))
        return arr, keep

    # ------------------------------------------------------------------ API
    def set_config(self, cfg: MuonConfig):
        self._check(lib().muon_set_config(self._h, ctypes.byref(cfg)), "muon_set_config")
        self.cfg = cfg

    def set_memory_limit(self, nbytes: int):
        """Caps the device bytes the handle may hold (0: no cap); a call that would grow
        past it raises MuonError (MUON_ERR_OOM) before launching anything."""
        self._check(lib().muon_set_memory_limit(self._h, int(nbytes)), "muon_set_memory_limit")

    def memory_held(self) -> int:
        n = ctypes.c_size_t(0)
        self._check(lib().muon_memory_held(self._h, ctypes.byref(n)), "muon_memory_held")
        return n.value

    def step(self, groups: List[Group], stream=None):
        arr, keep = self._groups(groups, True)
        self._shapes = [(arr[i].rows, arr[i].cols, arr[i].count) for i in range(len(groups))]
        self._check(lib().muon_step(self._h, arr, len(groups), ctypes.c_void_p(_stream(stream, self.device))), "muon_step")

    def step_host(self, groups: List[Group], stream=None):
        arr, keep = self._groups(groups, False)
        self._shapes = [(arr[i].rows, arr[i].cols, arr[i].count) for i in range(len(groups))]
        self._check(lib().muon_step_host(self._h, arr, len(groups), ctypes.c_void_p(_stream(stream, self.device))), "muon_step_host")

    def step_direction(self, groups, stream=None):
        """groups: list of (G_list, B_list, O_list) of same-shape matrices.  B is updated
        and O (fp32 or bf16 tensors of W's shape) receives the Newton-Schulz direction;
        no weight is touched (see muon_step_direction)."""
        import torch
        arr = (_DirGroup * len(groups))()
        keep = []
        for i, (Gs, Bs, Os) in enumerate(groups):
            rows, cols = Bs[0].shape
            if not (len(Gs) == len(Bs) == len(Os)):
                raise ValueError("G, B and O lists differ in length")
            _check_tensors(Gs, (rows, cols), True, Gs[0].dtype, self.device)
            _check_tensors(Bs, (rows, cols), True, torch.float32, self.device)
            _check_tensors(Os, (rows, cols), True, Os[0].dtype, self.device)
            pg, pb, po = _ptrs(Gs), _ptrs(Bs), _ptrs(Os)
            keep += [pg, pb, po]
            arr[i] = _DirGroup(rows, cols, len(Bs), _dtype_code(Gs[0]), _dtype_code(Os[0]),
                               ctypes.cast(pg, ctypes.POINTER(ctypes.c_void_p)),
                               ctypes.cast(pb, ctypes.POINTER(ctypes.c_void_p)),
                               ctypes.cast(po, ctypes.POINTER(ctypes.c_void_p)))
        self._check(lib().muon_step_direction(self._h, arr, len(groups), ctypes.c_void_p(_stream(stream, self.device))),
                    "muon_step_direction")

    def apply(self, groups, stream=None):
        """groups: list of (W_list, O_list[, scale]) of same-shape matrices:
        W <- W - lr*wd*W - lr*s*O (see muon_apply); O fp32 or bf16."""
        import torch
        arr = (_ApplyGroup * len(groups))()
        keep = []
        for i, grp in enumerate(groups):
            Ws, Os = grp[0], grp[1]
            scale = float(grp[2]) if len(grp) > 2 else 1.0
            rows, cols = Ws[0].shape
            if len(Ws) != len(Os):
                raise ValueError("W and O lists differ in length")
            _check_tensors(Ws, (rows, cols), True, torch.float32, self.device)
            _check_tensors(Os, (rows, cols), True, Os[0].dtype, self.device)
            pw, po = _ptrs(Ws), _ptrs(Os)
            keep += [pw, po]
            arr[i] = _ApplyGroup(rows, cols, len(Ws), _dtype_code(Os[0]), scale,
                                 ctypes.cast(pw, ctypes.POINTER(ctypes.c_void_p)),
                                 ctypes.cast(po, ctypes.POINTER(ctypes.c_void_p)))
        self._check(lib().muon_apply(self._h, arr, len(groups), ctypes.c_void_p(_stream(stream, self.device))),
                    "muon_apply")

    def orthogonalize(self, groups, stream=None):
        """groups: list of (M_list, O_list); O = NS(M / (||M||_F + eps)), fp32 outputs."""
        arr = (_OrthoGroup * len(groups))()
        keep = []
        for i, (Ms, Os) in enumerate(groups):
            import torch
            rows, cols = Ms[0].shape
            _check_tensors(Ms, (rows, cols), True, Ms[0].dtype, self.device)
            _check_tensors(Os, (rows, cols), True, torch.float32, self.device)
            pm, po = _ptrs(Ms), _ptrs(Os)
            keep += [pm, po]
            arr[i] = _OrthoGroup(rows, cols, len(Ms), _dtype_code(Ms[0]),
                                 ctypes.cast(pm, ctypes.POINTER(ctypes.c_void_p)),
                                 ctypes.cast(po, ctypes.POINTER(ctypes.c_void_p)))
        self._check(lib().muon_orthogonalize(self._h, arr, len(groups), ctypes.c_void_p(_stream(stream, self.device))),
                    "muon_orthogonalize")

    def ns_phase(self, phase: int, precision: int, m: int, n: int, count: int, alpha: float, beta: float,
                 x_op=None, a_in=None, x_master=None, out=None, out_op=None, stream=None):
        for t in (x_op, a_in, x_master, out, out_op):
            if t is not None and (not t.is_cuda or t.device.index != self.device):
                raise ValueError(f"building-block buffers must be on cuda:{self.device}")
        p = lambda t: None if t is None else t.data_ptr()
        args = _PhaseArgs(phase, precision, m, n, count, alpha, beta, p(x_op), p(a_in), p(x_master), p(out), p(out_op))
        self._check(lib().muon_ns_phase_run(self._h, ctypes.byref(args), ctypes.c_void_p(_stream(stream, self.device))),
                    "muon_ns_phase_run")

    def qk_clip(self, Wq, Wk, max_logits, head_dim: int, tau: float, stream=None):
        """MuonClip's QK-Clip: rows of head h of Wq and Wk times sqrt(min(1, tau / max_logits[h]))."""
        import torch
        for name, t in (("Wq", Wq), ("Wk", Wk), ("max_logits", max_logits)):
            if t is None and name == "Wk":
                continue
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
            if t.device.index != self.device:
                raise ValueError(f"{name} is on cuda:{t.device.index}, the handle on cuda:{self.device}")
        n_heads = max_logits.numel()
        if Wq.dim() != 2:
            raise ValueError("Wq must be 2-D")
        rows, cols = Wq.shape
        if rows != n_heads * head_dim or (Wk is not None and tuple(Wk.shape) != (rows, cols)):
            raise ValueError("Wq / Wk must be (n_heads * head_dim) x cols")
        self._check(lib().muon_qk_clip(self._h, ctypes.c_void_p(Wq.data_ptr()),
                                       None if Wk is None else ctypes.c_void_p(Wk.data_ptr()),
                                       ctypes.c_void_p(max_logits.data_ptr()), n_heads, head_dim, cols, float(tau),
                                       ctypes.c_void_p(_stream(stream, self.device))), "muon_qk_clip")

    def qk_clip_grouped(self, Wq, Wk, max_logits, head_dim: int, tau: float, stream=None):
        """QK-Clip of a layer whose query heads share key heads (see muon_qk_clip_grouped): Wq fp32
        (n_heads * head_dim) x cols, Wk fp32 (n_kv_heads * head_dim) x cols, max_logits as `attention` leaves it."""
        for name, t in (("Wq", Wq), ("Wk", Wk), ("max_logits", max_logits)):
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
            if t.device.index != self.device:
                raise ValueError(f"{name} is on cuda:{t.device.index}, the handle on cuda:{self.device}")
        n_heads = max_logits.numel()
        if Wq.dim() != 2 or Wk.dim() != 2 or Wq.shape[1] != Wk.shape[1]:
            raise ValueError("Wq and Wk must be 2-D with the same number of columns")
        if head_dim <= 0 or Wq.shape[0] != n_heads * head_dim or Wk.shape[0] % head_dim != 0 or Wk.shape[0] == 0:
            raise ValueError("Wq must have n_heads * head_dim rows, Wk a multiple of head_dim")
        _check_sizes("Wq", *Wq.shape)
        self._check(lib().muon_qk_clip_grouped(self._h, Wq.data_ptr(), Wk.data_ptr(), max_logits.data_ptr(), n_heads,
                                               Wk.shape[0] // head_dim, head_dim, Wq.shape[1], float(tau),
                                               ctypes.c_void_p(_stream(stream, self.device))), "muon_qk_clip_grouped")

    def _attention_fields(self, q, k, v, cu_seqlens, cu_seqlens_k, scale, out, lse, max_logits):
        """The fields of _AttentionArgs in order."""
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("q and k must be [rows, heads, head_dim]")
        (tq, hq, d), (tk, hk, _) = q.shape, k.shape
        dev = self.device
        cu_k = cu_seqlens if cu_seqlens_k is None else cu_seqlens_k
        for name, t in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_k)):
            if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() < 1:
                raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor")
            _check_dense(name, t, dev)
        n = cu_seqlens.numel()
        if cu_k.numel() != n:
            raise ValueError("cu_seqlens and cu_seqlens_k must hold one entry more than there are sequences")
        if lse.dtype is not torch.float32 or lse.shape != (hq, tq):
            raise ValueError(f"lse must be float32 of shape {(hq, tq)}")
        _check_dense("lse", lse, dev)
        if max_logits is not None:
            if max_logits.dtype is not torch.float32 or max_logits.shape != (hq,):
                raise ValueError(f"max_logits must be float32 of shape {(hq,)}")
            _check_dense("max_logits", max_logits, dev)
        if scale is None:
            scale = d ** -0.5 if d > 0 else 1.0         # (heads without width are refused by the library)
        kv = (tk, hk, d)
        return (n - 1, hq, hk, d, tq, tk, cu_seqlens.data_ptr(), cu_k.data_ptr(), scale,
                *_heads("q", q, q.shape, dev), *_heads("k", k, kv, dev), *_heads("v", v, kv, dev),
                *_heads("out", out, q.shape, dev), lse.data_ptr(), 0 if max_logits is None else max_logits.data_ptr())

    def attention(self, q, k, v, cu_seqlens, out=None, lse=None, max_logits=None, scale: Optional[float] = None,
                  cu_seqlens_k=None, stream=None):
        """Causal attention over packed sequences (see muon_attention): q [rows, heads, head_dim] and k, v
        [rows, kv heads, head_dim] in bf16, cu_seqlens int32 [sequences + 1] on the device (cu_seqlens_k where the
        keys are packed otherwise), scale 1 / sqrt(head_dim) by default.  Writes out (layout of q), lse
        [heads, rows] fp32 and raises max_logits [heads] fp32 to the largest logit of each head, for qk_clip.
        Returns (out, lse).  Rows of no sequence are left as they are in buffers that are given, and are 0 (lse: -inf)
        in those that the call allocates: `weight_grad` and the next projection sum over all rows."""
        fill = 0
        if out is None:
            out, fill = _empty(None, None, q, stream), MUON_FILL_OUT
        if lse is None:
            lse = _empty((q.shape[1], q.shape[0]) if q.dim() == 3 else (0,), torch.float32, q, stream)
            fill |= MUON_FILL_LSE
        args = _AttentionArgs.from_buffer_copy(_ATTENTION_PACK.pack(
            *self._attention_fields(q, k, v, cu_seqlens, cu_seqlens_k, scale, out, lse, max_logits)))
        self._check(lib().muon_attention_fill(self._h, args, fill, _stream(stream, self.device)), "muon_attention")
        return out, lse

    def attention_backward(self, grad_out, q, k, v, out, lse, cu_seqlens, dq=None, dk=None, dv=None,
                           scale: Optional[float] = None, cu_seqlens_k=None, stream=None):
        """Gradients of `attention` (see muon_attention_backward) from its inputs, out and lse.  Returns
        (dq, dk, dv).  Rows of no sequence are left as they are in buffers that are given, and are 0 in those that the
        call allocates."""
        fields = self._attention_fields(q, k, v, cu_seqlens, cu_seqlens_k, scale, out, lse, None)
        fill = 0
        if dq is None:
            dq, fill = _empty(None, None, q, stream), MUON_FILL_DQ
        if dk is None:
            dk, fill = _empty(None, None, k, stream), fill | MUON_FILL_DK
        if dv is None:
            dv, fill = _empty(None, None, v, stream), fill | MUON_FILL_DV
        delta = _empty(None, None, lse, stream)
        dev = self.device
        args = _AttentionGradArgs.from_buffer_copy(_ATTENTION_GRAD_PACK.pack(
            *fields, *_heads("grad_out", grad_out, q.shape, dev), *_heads("dq", dq, q.shape, dev),
            *_heads("dk", dk, k.shape, dev), *_heads("dv", dv, v.shape, dev), delta.data_ptr()))
        self._check(lib().muon_attention_backward_fill(self._h, args, fill, _stream(stream, self.device)),
                    "muon_attention_backward")
        return dq, dk, dv

    def checkpoint(self, x, ckpt: Optional[Checkpoint] = None, stream=None) -> Checkpoint:
        """x (2-D, bf16 or fp32, dense rows) in 8 bits, for the backward pass (see muon_checkpoint_store)."""
        stride = _check_rows("x", x, self.device)
        code = _dtype_code(x)
        rows, cols = x.shape
        _check_sizes("x", rows, cols)
        if ckpt is None:
            blocks = -(-cols // CKPT_BLOCK)
            ckpt = Checkpoint(_empty((rows, blocks * CKPT_BLOCK), torch.int8, x, stream),
                              _empty((rows, blocks), torch.uint8, x, stream), cols)
        else:
            _check_checkpoint(ckpt, self.device)
            if (ckpt.rows, ckpt.cols) != (rows, cols):
                raise ValueError(f"the checkpoint holds {ckpt.rows} x {ckpt.cols} values, x is {rows} x {cols}")
        self._check(lib().muon_checkpoint_store(self._h, x.data_ptr(), code, rows, cols, stride, ckpt.codes.data_ptr(),
                                                ckpt.scales.data_ptr(), _stream(stream, self.device)),
                    "muon_checkpoint_store")
        return ckpt

    def checkpoint_load(self, ckpt: Checkpoint, out=None, stream=None):
        """The values of a checkpoint, written to `out` (bf16 or fp32, dense rows; bf16 when not given)."""
        _check_checkpoint(ckpt, self.device)
        rows, cols = ckpt.rows, ckpt.cols
        _check_sizes("the checkpoint", rows, cols)
        if out is None:
            out = _empty((rows, cols), torch.bfloat16, ckpt.codes, stream)
        stride = _check_rows("out", out, self.device)
        if tuple(out.shape) != (rows, cols):
            raise ValueError(f"the checkpoint holds {rows} x {cols} values, out is {tuple(out.shape)}")
        self._check(lib().muon_checkpoint_load(self._h, ckpt.codes.data_ptr(), ckpt.scales.data_ptr(), rows, cols,
                                               out.data_ptr(), _dtype_code(out), stride, _stream(stream, self.device)),
                    "muon_checkpoint_load")
        return out

    def weight_grad(self, dy, ckpt: Checkpoint, G, accumulate: bool = False, stream=None):
        """G = dy^T x^ (or G += with `accumulate`): the gradient of the weight of y = x W^T from the checkpoint of x
        (see muon_weight_grad).  dy bf16 [tokens, rows] with dense rows; G fp32 or bf16 [rows, cols], the gradient
        that `step` takes.  Returns G."""
        _check_checkpoint(ckpt, self.device)
        stride = _check_rows("dy", dy, self.device)
        if dy.dtype is not torch.bfloat16:
            raise TypeError(f"dy: unsupported dtype {dy.dtype}, expected torch.bfloat16")
        tokens, rows = dy.shape
        _check_sizes("weight_grad", tokens, rows, ckpt.cols)
        if tokens != ckpt.rows:
            raise ValueError(f"dy has {tokens} rows, the checkpoint {ckpt.rows}")
        if tuple(G.shape) != (rows, ckpt.cols):
            raise ValueError(f"G must be {rows} x {ckpt.cols}, got {tuple(G.shape)}")
        _check_dense("G", G, self.device)
        args = _WeightGradArgs(tokens, rows, ckpt.cols, dy.data_ptr(), stride, ckpt.codes.data_ptr(),
                               ckpt.scales.data_ptr(), G.data_ptr(), _dtype_code(G), 1 if accumulate else 0, None, 0)
        need = ctypes.c_size_t(0)
        if lib().muon_weight_grad_workspace(args, need) == MUON_OK and need.value:
            workspace = _empty((need.value,), torch.uint8, G, stream)
            args.workspace, args.workspace_bytes = workspace.data_ptr(), need.value
        self._check(lib().muon_weight_grad(self._h, args, _stream(stream, self.device)), "muon_weight_grad")
        return G

    def sync(self, stream=None):
        self._check(lib().muon_sync(self._h, ctypes.c_void_p(_stream(stream, self.device))), "muon_sync")

    def last_norms(self, stream=None) -> List[float]:
        n = ctypes.c_int(0)
        lib().muon_last_norms(self._h, None, 0, ctypes.byref(n), ctypes.c_void_p(_stream(stream, self.device)))
        buf = (ctypes.c_float * max(n.value, 1))()
        self._check(lib().muon_last_norms(self._h, buf, n.value, ctypes.byref(n), ctypes.c_void_p(_stream(stream, self.device))),
                    "muon_last_norms")
        return list(buf[: n.value])

    def last_update_rms(self, stream=None) -> List[float]:
        """Per matrix (groups in order), the RMS of the update lr * s * O of the last step."""
        n = ctypes.c_int(0)
        lib().muon_last_update_rms(self._h, None, 0, ctypes.byref(n), ctypes.c_void_p(_stream(stream, self.device)))
        buf = (ctypes.c_float * max(n.value, 1))()
        self._check(lib().muon_last_update_rms(self._h, buf, n.value, ctypes.byref(n),
                                               ctypes.c_void_p(_stream(stream, self.device))), "muon_last_update_rms")
        return list(buf[: n.value])

    def last_update(self, group: int, index: int, dst, stream=None):
        """O of matrix `index` of group `group` of the last step, written to dst (fp32,
        the matrix's rows x cols, contiguous, on the device)."""
        import torch
        shapes = getattr(self, "_shapes", None)
        if shapes is None or not (0 <= group < len(shapes)) or not (0 <= index < shapes[group][2]):
            raise ValueError(f"no matrix {index} in group {group} of the last call")
        _check_tensors([dst], shapes[group][:2], True, torch.float32, self.device)
        self._check(lib().muon_last_update(self._h, group, index, ctypes.c_void_p(dst.data_ptr()),
                                           ctypes.c_void_p(_stream(stream, self.device))), "muon_last_update")

    TIMING_KINDS = ("momentum_norm", "norm_finalize", "gram", "poly", "update", "apply")

    def timing(self, enable: bool = True):
        self._check(lib().muon_timing_enable(self._h, int(enable)), "muon_timing_enable")

    def timing_read(self, stream=None):
        """{phase: (total ms, launches)} since the last read (synchronises the stream)."""
        k = len(self.TIMING_KINDS)
        ms = (ctypes.c_double * k)()
        n = (ctypes.c_int * k)()
        self._check(lib().muon_timing_read(self._h, ms, n, k, ctypes.c_void_p(_stream(stream, self.device))), "muon_timing_read")
        return {name: (ms[i], n[i]) for i, name in enumerate(self.TIMING_KINDS)}

    def close(self):
        if self._h:
            lib().muon_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def momentum_norm_noalloc(G, B, norm_out, U_out=None, momentum: float = 0.95, nesterov: bool = True, stream=None):
    """Momentum phase of one matrix with no device allocation (see muon.h):
    B <- momentum*B + G in place, U_out = G + momentum*B (or B), norm_out[0] = ||U||_F."""
    import torch
    rows, cols = B.shape
    if not B.is_cuda:
        raise ValueError("B must be a CUDA tensor")
    dev = B.device.index
    _check_tensors([G], (rows, cols), True, None, dev)
    _check_tensors([B], (rows, cols), True, torch.float32, dev)
    if U_out is not None:
        _check_tensors([U_out], (rows, cols), True, torch.float32, dev)
    if norm_out.dtype != torch.float32 or not norm_out.is_cuda or norm_out.numel() < 1:
        raise ValueError("norm_out must be a float32 CUDA tensor with at least one element")
    if norm_out.device.index != dev:
        raise ValueError(f"norm_out is on cuda:{norm_out.device.index}, B on cuda:{dev}")
    err = ctypes.create_string_buffer(256)
    # the entry point works on the current device: make it B's for the call
    with torch.cuda.device(dev):
        st = lib().muon_momentum_norm_noalloc(rows, cols, _dtype_code(G), G.data_ptr(), B.data_ptr(),
                                              None if U_out is None else U_out.data_ptr(), float(momentum),
                                              int(nesterov), norm_out.data_ptr(), ctypes.c_void_p(_stream(stream)),
                                              err, 256)
    if st != MUON_OK:
        raise MuonError(st, f"muon_momentum_norm_noalloc: {err.value.decode()}")


def plan_tiles(shapes, phase: int):
    """Tile list of a grouped GEMM launch: [(group, matrix, tile_row, tile_col)] (host only)."""
    flat = (ctypes.c_int * (3 * len(shapes)))(*[int(v) for s in shapes for v in s])
    n = ctypes.c_int(0)
    lib().muon_plan_tiles(flat, len(shapes), phase, None, 0, ctypes.byref(n))
    out = (ctypes.c_int * (4 * max(n.value, 1)))()
    st = lib().muon_plan_tiles(flat, len(shapes), phase, out, n.value, ctypes.byref(n))
    if st != MUON_OK:
        raise MuonError(st, "muon_plan_tiles")
    return [tuple(out[4 * i: 4 * i + 4]) for i in range(n.value)]


def plan_units(shapes, phase: int, clusters: int, split: bool = False):
    """Work units of a two-CTA GEMM launch (host only): tuples (cluster, group, matrix,
    tile_row, tile_col, k_begin, k_end, kind, slot, nslots, n_half)."""
    flat = (ctypes.c_int * (3 * len(shapes)))(*[int(v) for s in shapes for v in s])
    n = ctypes.c_int(0)
    lib().muon_plan_units(flat, len(shapes), phase, clusters, int(split), None, 0, ctypes.byref(n))
    out = (ctypes.c_int * (11 * max(n.value, 1)))()
    st = lib().muon_plan_units(flat, len(shapes), phase, clusters, int(split), out, n.value, ctypes.byref(n))
    if st != MUON_OK:
        raise MuonError(st, "muon_plan_units")
    return [tuple(out[11 * i: 11 * i + 11]) for i in range(n.value)]


def tile_shape():
    return lib().muon_plan_tile_m(), lib().muon_plan_tile_n()
