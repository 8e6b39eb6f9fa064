"""ctypes binding of libmua.so (include/mua.h): argument marshalling only.

Every entry point of the C ABI is reachable here under the same name
(``library().mua_step`` ...); :class:`MicroAdam` wraps a handle with tensor
checks. Tensors are passed as raw device pointers, streams as
``torch.cuda.Stream.cuda_stream``.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmua.so")

MUA_OK = 0
MUA_ERR_ARG = -1
MUA_ERR_UNSUPPORTED = -2
MUA_ERR_ALIGN = -3
MUA_ERR_CUDA = -4
MUA_STATUS_NONFINITE = 1
MUA_STATUS_TIMEOUT = 2
MUA_F32 = 0
MUA_BF16 = 1

# Every symbol include/mua.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_i64, _i32, _u64, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_float
SIGNATURES = {
    "mua_create": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, ctypes.POINTER(_P)]),
    "mua_create_shard": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i64, _i64,
                                        ctypes.POINTER(_P)]),
    "mua_create_segmented": (ctypes.c_int, [ctypes.POINTER(_i64), _i32, _i32, _i32, _i32, _i32,
                                            ctypes.POINTER(_P)]),
    "mua_destroy": (None, [_P]),
    "mua_state_bytes": (_i64, [_P]),
    "mua_state_layout": (ctypes.c_int, [_P, ctypes.POINTER(_i64)]),
    "mua_step": (ctypes.c_int, [_P, _P, _P, _P, _f32, _f32, _f32, _f32, _f32, _i64, _u64, _P]),
    "mua_select": (ctypes.c_int, [_P, _P, _P, _P, _f32, _f32, _f32, _f32, _f32, _i64, _u64, _P,
                                  _P, _P]),
    "mua_minmax_offset": (_i64, [_P, _i64]),
    "mua_apply": (ctypes.c_int, [_P, _P, _P, _P, _f32, _f32, _f32, _f32, _f32, _i64, _u64, _P,
                                 _P, _P]),
    "mua_get_status": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "mua_step_launches": (ctypes.c_int, [_P, _i32]),
    "mua_step_bf16": (ctypes.c_int, [_P, _P, _P, _P, _f32, _f32, _f32, _f32, _f32, _i64, _u64,
                                     _P]),
    "mua_apply_bf16": (ctypes.c_int, [_P, _P, _P, _P, _f32, _f32, _f32, _f32, _f32, _i64, _u64,
                                      _P, _P, _P]),
    "mua_set_wait_limit_ns": (ctypes.c_int, [_P, _i64]),
    "mua_muon_create": (ctypes.c_int, [_i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_f32),
                                       ctypes.POINTER(_P)]),
    "mua_muon_destroy": (None, [_P]),
    "mua_muon_state_bytes": (_i64, [_P]),
    "mua_muon_workspace_bytes": (_i64, [_P]),
    "mua_muon_state_layout": (ctypes.c_int, [_P, ctypes.POINTER(_i64)]),
    "mua_muon_momentum": (ctypes.c_int, [_P, _P, _i32, _P, _P, _i32, _f32, _i32, _i64, _u64, _P]),
    "mua_muon_read": (ctypes.c_int, [_P, _P, _P, _i32, _P]),
    "mua_muon_write": (ctypes.c_int, [_P, _P, _i32, _P, _P]),
    "mua_muon_orthogonalize": (ctypes.c_int, [_P, _P, _i32, _i64, _i64, _P, _i64, _i64, _P, _f32,
                                              _P]),
    "mua_muon_step": (ctypes.c_int, [_P, _P, _i32, _P, _i32, _P, _P, _f32, _f32, _f32, _i32, _f32,
                                     _f32, _i64, _u64, _P]),
    "mua_muon_set_wait_limit_ns": (ctypes.c_int, [_P, _i64]),
    "mua_muon_get_status": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "mua_muon_last_cuda_error": (ctypes.c_char_p, []),
    "mua_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "mua_last_cuda_error": (ctypes.c_char_p, []),
    "mua_version": (ctypes.c_char_p, []),
}

_lib = None


class MuaError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = f"{what}: {strerror(code)} ({code})"
        if code == MUA_ERR_CUDA:
            last = (library().mua_muon_last_cuda_error if what.startswith("mua_muon")
                    else library().mua_last_cuda_error)
            msg += f" [{last().decode()}]"
        super().__init__(msg)
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load libmua.so; raises ImportError if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"{_LIB_PATH} is missing: build it with "
                              "`python compressed_state_optimizer_b200/build.py`")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def strerror(code: int) -> str:
    return library().mua_strerror(code).decode()


def _check(code: int, what: str):
    if code != MUA_OK:
        raise MuaError(code, what)


def _stream_ptr(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


@dataclass
class Layout:
    header: int
    codes: int
    window: int
    row_stride: int
    blocks: int
    bytes: int


class MicroAdam:
    """One MicroAdam problem: d parameters in blocks of B_d, k_b kept per block,
    a window of m rows, b = 4 bits (optionally one rank's shard of the blocks,
    or, with ``segments``, a tensor list whose tensors are cut into blocks one
    by one; ``d`` must then be their total length).

    The optimizer state is a caller-owned ``torch.uint8`` tensor of
    ``state_bytes`` bytes (see :meth:`new_state`), zero at t = 0.
    """

    def __init__(self, d: int, block_size: int = 16384, k_per_block: int | None = None,
                 window: int = 10, bits: int = 4, *, shard: tuple[int, int] | None = None,
                 segments=None):
        if k_per_block is None:
            k_per_block = max(1, math.ceil(block_size / 100 - 1e-9))
        lib = library()
        h = ctypes.c_void_p()
        self.segments = None if segments is None else [int(n) for n in segments]
        if self.segments is not None:
            if shard is not None or sum(self.segments) != d:
                raise ValueError("segments: whole vector only, lengths summing to d")
            arr = (_i64 * len(self.segments))(*self.segments)
            _check(lib.mua_create_segmented(arr, len(self.segments), block_size, k_per_block,
                                            window, bits, ctypes.byref(h)),
                   "mua_create_segmented")
        elif shard is None:
            _check(lib.mua_create(d, block_size, k_per_block, window, bits, ctypes.byref(h)),
                   "mua_create")
        else:
            _check(lib.mua_create_shard(d, block_size, k_per_block, window, bits, shard[0],
                                        shard[1], ctypes.byref(h)), "mua_create_shard")
        self._h = h
        self.d_total = d
        self.block_size = block_size
        self.k_per_block = k_per_block
        self.window = window
        self.bits = bits
        self.shard = shard
        self.state_bytes = int(lib.mua_state_bytes(h))
        arr = (ctypes.c_int64 * 6)()
        _check(lib.mua_state_layout(h, arr), "mua_state_layout")
        self.layout = Layout(*[int(x) for x in arr])
        nb_total = self.layout.blocks if self.segments is not None else -(-d // block_size)
        if shard is None:
            self.first_block, self.blocks = 0, nb_total
        else:
            self.first_block, self.blocks = shard
        self.offset = self.first_block * block_size
        self.d = min(d, (self.first_block + self.blocks) * block_size) - self.offset

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.mua_destroy(h)
            self._h = None

    # ------------------------------------------------------------ state
    def new_state(self, device="cuda"):
        import torch
        return torch.zeros(self.state_bytes, dtype=torch.uint8, device=device)

    def _check_tensors(self, params, grads, state):
        import torch
        if params is not None:
            assert params.dtype in (torch.float32, torch.bfloat16)
            assert params.is_cuda and params.is_contiguous()
            assert params.numel() == self.d, (params.numel(), self.d)
        assert grads.dtype == torch.bfloat16 and grads.is_cuda and grads.is_contiguous()
        assert grads.numel() == self.d
        assert state.dtype == torch.uint8 and state.is_cuda and state.numel() >= self.state_bytes

    # ------------------------------------------------------------ steps
    def step(self, params, grads, state, *, lr, beta1, beta2, eps, wd, t, seed, stream=None):
        """One full step t on ``stream`` (default: the current stream);
        ``params`` fp32 (mua_step) or bf16 (mua_step_bf16)."""
        import torch
        self._check_tensors(params, grads, state)
        name = "mua_step_bf16" if params.dtype == torch.bfloat16 else "mua_step"
        _check(getattr(library(), name)(self._h, params.data_ptr(), grads.data_ptr(),
                                        state.data_ptr(), lr, beta1, beta2, eps, wd, t, seed,
                                        _stream_ptr(stream)), name)

    def select(self, params, grads, state, *, lr, beta1, beta2, eps, wd, t, seed, mhat=None,
               vhat=None, stream=None):
        """First half of step t (Top-k, window row, min/max partials)."""
        self._half("mua_select", params, grads, state, lr, beta1, beta2, eps, wd, t, seed, mhat,
                   vhat, stream)

    def _half(self, name, params, grads, state, lr, beta1, beta2, eps, wd, t, seed, mhat, vhat,
              stream):
        import torch
        self._check_tensors(params, grads, state)
        if params is not None and params.dtype == torch.bfloat16:
            if name == "mua_select":
                params = None  # not touched by the select kernel
            else:
                name = name + "_bf16"
        for x in (mhat, vhat):
            if x is not None:
                assert x.is_cuda and x.numel() == self.d and x.is_contiguous()
        fn = getattr(library(), name)
        _check(fn(self._h, params.data_ptr() if params is not None else None, grads.data_ptr(),
                  state.data_ptr(), lr, beta1,
                  beta2, eps, wd, t, seed, mhat.data_ptr() if mhat is not None else None,
                  vhat.data_ptr() if vhat is not None else None, _stream_ptr(stream)), name)

    def minmax_offset(self, t: int) -> int:
        off = int(library().mua_minmax_offset(self._h, t))
        if off < 0:
            raise MuaError(off, "mua_minmax_offset")
        return off

    def apply(self, params, grads, state, *, lr, beta1, beta2, eps, wd, t, seed, mhat=None,
              vhat=None, stream=None):
        """Second half of step t (4-bit quantization of the residual and the
        AdamStats update of the parameters)."""
        self._half("mua_apply", params, grads, state, lr, beta1, beta2, eps, wd, t, seed, mhat,
                   vhat, stream)

    def step_launches(self, bf16_params: bool = False) -> int:
        """Kernel launches of one ``step`` on the current device (1: fused)."""
        n = int(library().mua_step_launches(self._h, 1 if bf16_params else 0))
        if n < 0:
            raise MuaError(n, "mua_step_launches")
        return n

    def set_wait_limit_ns(self, ns: int):
        """Bound on the fused step's grid-barrier wait (<= 0: give up at once)."""
        _check(library().mua_set_wait_limit_ns(self._h, int(ns)), "mua_set_wait_limit_ns")

    def status(self, state, stream=None) -> int:
        out = ctypes.c_int32()
        _check(library().mua_get_status(self._h, state.data_ptr(), _stream_ptr(stream),
                                        ctypes.byref(out)), "mua_get_status")
        return int(out.value)


@dataclass
class MuonLayout:
    header: int
    scales: int
    codes: int
    blocks: int
    bytes: int


class Muon:
    """One Muon problem: ``count`` matrices of ``rows x cols`` one after the
    other, their momentum held in ``bits`` = 8 or 4 bits per value, the update
    orthogonalised by ``steps`` Newton-Schulz products.

    ``coefficients``: (a, b, c) of the polynomial a + b x + c x^2 of every step,
    or a sequence of ``steps`` of them; default (3.4445, -4.7750, 2.0315).

    The state and the workspace are caller-owned ``torch.uint8`` tensors (see
    :meth:`new_state` and :meth:`new_workspace`). A workspace serves one call
    at a time; calls on several streams, or captured graphs that may overlap,
    take one each. Rounding draws go by (seed, t, place in the stack): give every
    stack a seed of its own. None of this is differentiable: tensors that would record a
    gradient are refused, except the parameters ``step`` updates in place.
    """

    def __init__(self, rows: int, cols: int, count: int = 1, *, bits: int = 8, steps: int = 5,
                 coefficients=None):
        lib = library()
        for name, v in (("rows", rows), ("cols", cols), ("count", count), ("bits", bits),
                        ("steps", steps)):
            if not -(1 << 31) <= v < 1 << 31:  # ctypes would pass its low half
                raise ValueError(f"{name}: {v} does not fit 32 bits")
        arr = None
        if coefficients is not None:
            c = list(coefficients)
            if len(c) == 3 and not hasattr(c[0], "__len__"):
                c = [c] * steps
            if len(c) != steps or any(len(x) != 3 for x in c):
                raise ValueError("coefficients: one (a, b, c), or one for each step")
            arr = (_f32 * (3 * steps))(*[float(v) for x in c for v in x])
        h = ctypes.c_void_p()
        _check(lib.mua_muon_create(rows, cols, count, bits, steps, arr, ctypes.byref(h)),
               "mua_muon_create")
        self._h = h
        self.rows, self.cols, self.count = rows, cols, count
        self.bits, self.steps = bits, steps
        self.d = rows * cols * count
        self.state_bytes = int(lib.mua_muon_state_bytes(h))
        self.workspace_bytes = int(lib.mua_muon_workspace_bytes(h))
        out = (ctypes.c_int64 * 5)()
        _check(lib.mua_muon_state_layout(h, out), "mua_muon_state_layout")
        self.layout = MuonLayout(*[int(x) for x in out])

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and _lib is not None:
            _lib.mua_muon_destroy(h)
            self._h = None

    # ------------------------------------------------------------ buffers
    def new_state(self, device="cuda"):
        import torch
        return torch.zeros(self.state_bytes, dtype=torch.uint8, device=device)

    def new_workspace(self, device="cuda"):
        import torch
        w = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
        w[:256].zero_()
        return w

    # ------------------------------------------------------------ checks
    @staticmethod
    def _type(x, what):
        import torch
        if x.dtype == torch.float32:
            return MUA_F32
        if x.dtype == torch.bfloat16:
            return MUA_BF16
        raise ValueError(f"{what}: float32 or bfloat16, not {x.dtype}")

    def _values(self, x, what):
        """A contiguous tensor of all count * rows * cols values."""
        if x.numel() != self.d or not x.is_contiguous():
            raise ValueError(f"{what}: {self.d} contiguous values, not shape {tuple(x.shape)} "
                             f"with strides {tuple(x.stride())}")
        return self._type(x, what)

    def _buffer(self, x, size, what):
        import torch
        if x.dtype is not torch.uint8 or x.numel() < size or not x.is_contiguous():
            raise ValueError(f"{what}: a contiguous uint8 tensor of at least {size} bytes")

    def _stack(self, x, what):
        """(matrix stride, row stride) of a [count, rows, cols] view."""
        shape = (self.count, self.rows, self.cols)
        if tuple(x.shape) != shape and not (self.count == 1 and tuple(x.shape) == shape[1:]):
            raise ValueError(f"{what}: shape {shape}, not {tuple(x.shape)}")
        if self.cols > 1 and x.stride(-1) != 1:
            raise ValueError(f"{what}: columns must be contiguous")
        row = x.stride(-2) if self.rows > 1 else self.cols
        return (x.stride(0) if self.count > 1 else self.rows * row), row

    def _launch(self, name, stream, tensors, args, params=None):
        """Call ``name(handle, *args, stream)`` on the tensors' device."""
        import torch
        index = tensors[0].get_device()
        grad = torch.is_grad_enabled()
        for x in tensors:
            if x.get_device() != index or index < 0:
                raise ValueError("tensors must be on one CUDA device")
            if grad and x.requires_grad and x is not params:
                raise ValueError("not differentiable: detach() the tensors")
        if stream is None:
            s = torch._C._cuda_getCurrentRawStream(index)
        elif stream.device.index == index:
            s = stream.cuda_stream
        else:
            raise ValueError(f"stream on {stream.device}, tensors on cuda:{index}")
        fn = getattr(library(), name)
        if torch.cuda.current_device() == index:
            code = fn(self._h, *args, s)
        else:
            with torch.cuda.device(index):
                code = fn(self._h, *args, s)
        if code != MUA_OK:
            raise MuaError(code, name)

    # ------------------------------------------------------------ operators
    def momentum(self, grads, state, direction, *, beta, nesterov=True, t, seed, stream=None):
        """The momentum update of step ``t``: ``grads`` (fp32 or bf16) into
        ``state``, the direction to ``direction`` (fp32 or bf16)."""
        gt, dt = self._values(grads, "grads"), self._values(direction, "direction")
        self._buffer(state, self.state_bytes, "state")
        self._launch("mua_muon_momentum", stream, (grads, state, direction),
                     (grads.data_ptr(), gt, state.data_ptr(), direction.data_ptr(), dt, beta,
                      nesterov, t, seed))

    def read_momentum(self, state, out, stream=None):
        """The momentum's values to ``out`` (fp32 or bf16)."""
        ot = self._values(out, "out")
        self._buffer(state, self.state_bytes, "state")
        self._launch("mua_muon_read", stream, (state, out),
                     (state.data_ptr(), out.data_ptr(), ot))

    def write_momentum(self, values, state, stream=None):
        """``values`` (fp32 or bf16) as the momentum, each to the nearest level of
        its block. A copy of the state, not its values, is the exact checkpoint."""
        vt = self._values(values, "values")
        self._buffer(state, self.state_bytes, "state")
        self._launch("mua_muon_write", stream, (values, state),
                     (values.data_ptr(), vt, state.data_ptr()))

    def orthogonalize(self, x, out, workspace, *, eps=1e-7, stream=None):
        """Newton-Schulz orthogonalisation of the matrices ``x`` ([count, rows,
        cols], fp32 or bf16, any matrix and row strides) into ``out`` (bf16,
        likewise; it may be ``x``)."""
        import torch
        xt = self._type(x, "x")
        xs, xr = self._stack(x, "x")
        os_, orow = self._stack(out, "out")
        if out.dtype != torch.bfloat16:
            raise ValueError(f"out: bfloat16, not {out.dtype}")
        self._buffer(workspace, self.workspace_bytes, "workspace")
        self._launch("mua_muon_orthogonalize", stream, (x, out, workspace),
                     (x.data_ptr(), xt, xs, xr, out.data_ptr(), os_, orow, workspace.data_ptr(),
                      eps))

    def step(self, params, grads, state, workspace, *, lr, beta=0.95, eps=1e-7, wd=0.0,
             scale=None, nesterov=True, t, seed, stream=None):
        """One full step ``t``: momentum, orthogonalisation, update of
        ``params`` (fp32 or bf16) by lr * scale, with decoupled weight decay.
        ``scale`` defaults to sqrt(max(1, rows / cols))."""
        if scale is None:
            scale = math.sqrt(max(1.0, self.rows / self.cols))
        pt, gt = self._values(params, "params"), self._values(grads, "grads")
        self._buffer(state, self.state_bytes, "state")
        self._buffer(workspace, self.workspace_bytes, "workspace")
        self._launch("mua_muon_step", stream, (params, grads, state, workspace),
                     (params.data_ptr(), pt, grads.data_ptr(), gt, state.data_ptr(),
                      workspace.data_ptr(), lr, scale, beta, nesterov, eps, wd, t, seed),
                     params=params)

    def set_wait_limit_ns(self, ns: int):
        """Bound on a wait inside the matrix-product kernels (<= 0: give up at once)."""
        _check(library().mua_muon_set_wait_limit_ns(self._h, int(ns)),
               "mua_muon_set_wait_limit_ns")

    def status(self, buffer, stream=None) -> int:
        """Status bits of a state (``step``, ``momentum``) or of a workspace
        (``orthogonalize``)."""
        self._buffer(buffer, 256, "buffer")
        import torch
        if stream is None:
            stream = torch.cuda.current_stream(buffer.device)
        out = ctypes.c_int32()
        with torch.cuda.device(buffer.device):
            _check(library().mua_muon_get_status(self._h, buffer.data_ptr(), stream.cuda_stream,
                                                 ctypes.byref(out)), "mua_muon_get_status")
        return int(out.value)
