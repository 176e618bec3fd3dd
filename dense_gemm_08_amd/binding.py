"""ctypes binding of ``libdense_gemm.so`` (the C ABI in include/dense_gemm.h).

Argument marshalling only: every step of the product runs in the library's
HIP kernels.  Tensors are passed as raw device pointers with their leading
dimensions, on the caller's current HIP stream (``torch.cuda`` is HIP on
ROCm builds of PyTorch).  There is no fallback: if the library is missing or a
call fails, a :class:`DenseGemmError` is raised.
"""
from __future__ import annotations

import ctypes
import enum
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIBNAME = "libdense_gemm.so"


class Status(enum.IntEnum):
    OK = 0
    INVALID_DIM = 1
    NULL_PTR = 2
    BAD_LD = 3
    MISALIGNED = 4
    TOO_LARGE = 5
    LAUNCH_FAILED = 6
    NO_DEVICE = 7
    BAD_ARG = 8
    NO_MEMORY = 9
    WORKSPACE_TOO_SMALL = 10
    SCRATCH_TOO_SMALL = 11


# dense_gemm_op: the type and layout pairings of dense_gemm_ex
OPS = {("nt", "f16"): 0, ("nn", "bf16"): 1, ("nt", "bf16"): 2, ("nn", "f16"): 3}


class Options(ctypes.Structure):
    """dense_gemm_options: split_k (0 = the library's choice, 1 = none,
    n = n parts) and tile_n (0 = the library's choice, 128 or 256)."""
    _fields_ = [("split_k", ctypes.c_int32), ("tile_n", ctypes.c_int32)]


# dense_gemm_act: the activations of the layer products
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class Epilogue(ctypes.Structure):
    """dense_gemm_epilogue: bias, residual and pre-activation (device pointers
    with strides in elements), activation and form of dense_gemm_layer."""
    _fields_ = [("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("preact", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("act", ctypes.c_int32), ("grad", ctypes.c_int32)]


class Groups(ctypes.Structure):
    """dense_gemm_groups: int32 group ends on the device, their number, and
    the elements between the groups' matrices."""
    _fields_ = [("ends", ctypes.c_void_p), ("count", ctypes.c_int64), ("stride", ctypes.c_int64)]


class DenseGemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = Status(status) if status in Status._value2member_map_ else status
        super().__init__("%s failed: %s (%d)" % (where, _status_string(status), int(status)))


_lib = None

# Every symbol the header declares, with its ctypes signature.
_i64 = ctypes.c_int64
_i32 = ctypes.c_int
_vp = ctypes.c_void_p
_GEMM_ARGS = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
SIGNATURES = {
    "gemm_nt_f16": (_GEMM_ARGS, _i32),
    "gemm_nn_bf16": (_GEMM_ARGS, _i32),
    "gemm_nt_bf16": (_GEMM_ARGS, _i32),
    "gemm_nn_f16": (_GEMM_ARGS, _i32),
    "gemm_nt_f16_ladder": ([_i32] + _GEMM_ARGS, _i32),
    "gemm_nt_e4m3_mx": ([_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                         _vp], _i32),
    "dense_gemm_status_string": ([_i32], ctypes.c_char_p),
    "dense_gemm_validate": ([_i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64], _i32),
    "dense_gemm_tile_of_task": ([_i64, _i64, _i64, _i64, ctypes.POINTER(_i64),
                                 ctypes.POINTER(_i64)], _i32),
    "dense_gemm_xcd_slot": ([_i64, _i64, _i64], _i64),
    "dense_gemm_plan": ([_i32, _i64, _i64, _i64, _i64, ctypes.POINTER(_i64)], _i32),
    "dense_gemm_workspace_size": ([_i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64,
                                   ctypes.POINTER(Options), ctypes.POINTER(ctypes.c_size_t)], _i32),
    "dense_gemm_ex": ([_i32] + _GEMM_ARGS[:-1] + [ctypes.POINTER(Options), _vp, ctypes.c_size_t,
                                                 _vp], _i32),
    "gemm_nt_f16_noalloc": (_GEMM_ARGS, _i32),
    "gemm_nt_e4m3_mx_workspace_size": ([_i64, _i64, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)],
                                       _i32),
    "gemm_nt_e4m3_mx_plan": ([_i64, _i64, _i64, _i64, ctypes.POINTER(_i64)], _i32),
    "dense_gemm_layer": ([_i32] + _GEMM_ARGS[:-1] + [ctypes.POINTER(Epilogue),
                                                    ctypes.POINTER(Groups), _vp, ctypes.c_size_t,
                                                    _vp], _i32),
    "dense_gemm_layer_workspace_size": ([_i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64,
                                         ctypes.POINTER(Groups), _i64,
                                         ctypes.POINTER(ctypes.c_size_t)], _i32),
    "dense_gemm_tn": ([_i32] + _GEMM_ARGS[:-1] + [_vp, ctypes.POINTER(Groups), _vp,
                                                 ctypes.c_size_t, _vp], _i32),
    "dense_gemm_tn_workspace_size": ([_i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32,
                                      ctypes.POINTER(Groups), _i64,
                                      ctypes.POINTER(ctypes.c_size_t)], _i32),
    "gemm_nt_e4m3_mx_ex": ([_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp,
                            _i64, _vp, ctypes.c_size_t, _vp], _i32),
}


def library_path() -> str:
    return os.environ.get("DENSE_GEMM_LIB", os.path.join(_HERE, _LIBNAME))


def load_library():
    """Load the HIP library once; raise if it has not been built.

    PyTorch is imported first when it is installed: it carries its own copy
    of the HIP runtime (and of the HSA runtime below it) under the same
    soname the library links against (libamdhip64.so.7), so with torch
    loaded the dynamic linker binds the library to that copy, and tensors,
    streams and the library's launches share one runtime.  Loaded the other
    way round, the process would map two HIP runtimes, and the library's
    calls would not see the device state torch set up (measured: the first
    call then fails with DENSE_GEMM_NO_DEVICE)."""
    global _lib
    if _lib is not None:
        return _lib
    try:
        import torch  # noqa: F401  (the runtime the library must bind to)
    except ImportError:
        pass
    path = library_path()
    if not os.path.exists(path):
        raise FileNotFoundError(
            "HIP library %s is not built; run `python -c 'import __graft_entry__ as g; g.build()'`"
            % path)
    lib = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return load_library().dense_gemm_status_string(int(status)).decode()
    except Exception:  # library unavailable: fall back to the enum name
        try:
            return Status(status).name
        except ValueError:
            return "unknown status"


def _stream_handle(stream, device) -> int:
    """The HIP stream handle: ``stream`` itself, or the current stream of
    ``device`` when it is None."""
    if stream is None:
        import torch
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _stream_object(stream, device):
    """The torch stream object of a launch stream given as a torch stream or
    a raw HIP stream handle."""
    import torch
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=device)
    return stream


def _used_by(t, stream, device):
    """Mark a tensor from torch's caching allocator as in use by the launch
    stream when that is not the current stream (an explicit ``stream``):
    torch ties each block to the stream it was allocated on, so without the
    mark a block dropped (or freed by the caller) while the call's kernels
    still run on the other stream could be handed to a new allocation on
    the current stream and overwritten under them."""
    if stream is not None:
        t.record_stream(_stream_object(stream, device))
    return t


def _ld(t) -> int:
    """Leading dimension (elements between rows) of a 2-D tensor with unit
    column stride.  A single row may carry any row stride (a transposed
    column, an expanded view): its leading dimension is then its width."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _same_device(*ts):
    dev = ts[0].device
    for t in ts[1:]:
        if t.device != dev:
            raise ValueError("operands on different devices: %s and %s" % (dev, t.device))
    return dev


def _check_tensor(t, dtype_name: str, what: str):
    import torch
    want = torch.float16 if dtype_name == "f16" else torch.bfloat16
    if t.dtype != want:
        raise TypeError("%s must be %s, got %s" % (what, want, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % what)
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("%s must be 2-D with unit column stride" % what)


def workspace_size(layout: str, fmt: str, M: int, N: int, K: int, A_ptr: int, lda: int,
                   B_ptr: int, ldb: int, options: Options | None = None, num_cus: int = 0) -> int:
    """Bytes of workspace dense_gemm_ex needs (dense_gemm_workspace_size)."""
    lib = load_library()
    out = ctypes.c_size_t()
    st = lib.dense_gemm_workspace_size(OPS[(layout, fmt)], M, N, K, A_ptr, lda, B_ptr, ldb,
                                       num_cus, ctypes.byref(options) if options else None,
                                       ctypes.byref(out))
    if st != Status.OK:
        raise DenseGemmError(st, "dense_gemm_workspace_size")
    return out.value


def _call(name: str, layout: str, fmt: str, A, B, D=None, stream=None, workspace=None):
    """D = A @ B.T (layout "nt", B is N x K) or D = A @ B ("nn", B is K x N).
    With ``workspace`` (a device tensor, or True to take one from torch's
    allocator), the call goes through dense_gemm_ex with that workspace.
    The call is asynchronous on ``stream`` (None: the current stream).  A
    workspace or D passed in stays the caller's to keep alive until the
    call's kernels finish; the ones this function allocates are marked as in
    use by ``stream``."""
    import torch
    lib = load_library()
    _check_tensor(A, fmt, "A")
    _check_tensor(B, fmt, "B")
    M, K = A.shape
    if layout == "nt":
        N, Kb = B.shape
    else:
        Kb, N = B.shape
    if Kb != K:
        raise ValueError("inner dimensions differ: A is %s, B is %s" % (tuple(A.shape), tuple(B.shape)))
    own_d = D is None
    if own_d:
        D = torch.empty((M, N), dtype=A.dtype, device=A.device)
    else:
        _check_tensor(D, fmt, "D")
        if D.shape[0] != M or D.shape[1] != N:
            raise ValueError("D has shape %s, expected (%d, %d)" % (tuple(D.shape), M, N))
    dev = _same_device(A, B, D)
    if own_d:
        _used_by(D, stream, dev)
    # the library launches on the current device
    with torch.cuda.device(dev):
        if workspace is None:
            st = getattr(lib, name)(M, N, K, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B),
                                    D.data_ptr(), _ld(D), _stream_handle(stream, dev))
        else:
            if workspace is True:
                need = workspace_size(layout, fmt, M, N, K, A.data_ptr(), _ld(A), B.data_ptr(),
                                      _ld(B))
                workspace = _used_by(torch.empty(max(need, 1), dtype=torch.uint8, device=dev),
                                     stream, dev)
            if not workspace.is_cuda or workspace.device != dev:
                raise ValueError("workspace must be a device tensor on %s" % dev)
            st = lib.dense_gemm_ex(OPS[(layout, fmt)], M, N, K, A.data_ptr(), _ld(A),
                                   B.data_ptr(), _ld(B), D.data_ptr(), _ld(D), None,
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream_handle(stream, dev))
            name = "dense_gemm_ex"
    if st != Status.OK:
        raise DenseGemmError(st, name)
    return D


def gemm_nt_f16(A, B, D=None, stream=None, workspace=None):
    """D = A @ B.T in FP16 (FP32 accumulation); A is M x K, B is N x K.
    ``workspace``: see :func:`_call`."""
    return _call("gemm_nt_f16", "nt", "f16", A, B, D, stream, workspace)


def gemm_nn_bf16(A, B, D=None, stream=None, workspace=None):
    """D = A @ B in BF16 (FP32 accumulation); A is M x K, B is K x N.
    ``workspace``: see :func:`_call`."""
    return _call("gemm_nn_bf16", "nn", "bf16", A, B, D, stream, workspace)


def gemm_nt_bf16(A, B, D=None, stream=None, workspace=None):
    """D = A @ B.T in BF16 (FP32 accumulation); A is M x K, B is N x K.
    ``workspace``: see :func:`_call`."""
    return _call("gemm_nt_bf16", "nt", "bf16", A, B, D, stream, workspace)


def gemm_nn_f16(A, B, D=None, stream=None, workspace=None):
    """D = A @ B in FP16 (FP32 accumulation); A is M x K, B is K x N.
    ``workspace``: see :func:`_call`."""
    return _call("gemm_nn_f16", "nn", "f16", A, B, D, stream, workspace)


def raw(name: str):
    """The raw ctypes function ``name`` (for calls with explicit pointers)."""
    return getattr(load_library(), name)


def mx_workspace_size(M: int, N: int, K: int, num_cus: int = 0) -> int:
    """Bytes of workspace gemm_nt_e4m3_mx_ex needs (gemm_nt_e4m3_mx_workspace_size;
    num_cus 0: the current device's)."""
    out = ctypes.c_size_t()
    st = load_library().gemm_nt_e4m3_mx_workspace_size(M, N, K, num_cus, ctypes.byref(out))
    if st != Status.OK:
        raise DenseGemmError(st, "gemm_nt_e4m3_mx_workspace_size")
    return out.value


def gemm_nt_e4m3_mx(A, SA, B, SB, D=None, stream=None, workspace=None):
    """D = A @ B.T with E4M3 A (M x K), B (N x K) and E8M0 block scales SA
    (M x K/32), SB (N x K/32), FP32 accumulation, BF16 out.  A and B are
    uint8 or float8_e4m3fn device tensors, SA and SB uint8 device tensors,
    all 2-D with unit column stride.  With ``workspace`` (a device tensor, or
    True to take one from torch's allocator), the call goes through
    gemm_nt_e4m3_mx_ex with that workspace."""
    import torch
    lib = load_library()
    for t, what in ((A, "A"), (SA, "SA"), (B, "B"), (SB, "SB")):
        if t.element_size() != 1 or not t.is_cuda or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
            raise ValueError("%s must be a 2-D byte device tensor with unit column stride" % what)
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(SA.shape) != (M, K // 32) or tuple(SB.shape) != (N, K // 32):
        raise ValueError("inconsistent shapes: A %s, SA %s, B %s, SB %s"
                         % (tuple(A.shape), tuple(SA.shape), tuple(B.shape), tuple(SB.shape)))
    own_d = D is None
    if own_d:
        D = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    else:
        _check_tensor(D, "bf16", "D")
        if D.shape[0] != M or D.shape[1] != N:
            raise ValueError("D has shape %s, expected (%d, %d)" % (tuple(D.shape), M, N))
    dev = _same_device(A, SA, B, SB, D)
    if own_d:
        _used_by(D, stream, dev)
    name = "gemm_nt_e4m3_mx"
    with torch.cuda.device(dev):
        args = (M, N, K, A.data_ptr(), _ld(A), SA.data_ptr(), _ld(SA), B.data_ptr(), _ld(B),
                SB.data_ptr(), _ld(SB), D.data_ptr(), _ld(D))
        if workspace is None:
            st = lib.gemm_nt_e4m3_mx(*args, _stream_handle(stream, dev))
        else:
            if workspace is True:
                workspace = _used_by(torch.empty(max(mx_workspace_size(M, N, K), 1),
                                                 dtype=torch.uint8, device=dev), stream, dev)
            if not workspace.is_cuda or workspace.device != dev:
                raise ValueError("workspace must be a device tensor on %s" % dev)
            st = lib.gemm_nt_e4m3_mx_ex(*args, workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(),
                                        _stream_handle(stream, dev))
            name = "gemm_nt_e4m3_mx_ex"
    if st != Status.OK:
        raise DenseGemmError(st, name)
    return D


# ---- the products of a layer ------------------------------------------------
#
# A call for one token takes about 6 us on the GPU, so what these functions do
# before the launch counts: they look each property up once, and enter a
# device context only where the operands are not on the current device.

_FMTS = None   # torch dtype -> (name, dense_gemm_fmt); set by _torch()
_raw_stream = None


def _torch():
    global _FMTS, _raw_stream
    import torch
    if _FMTS is None:
        # (the current stream's handle without building a Stream object,
        # where this torch has it: 0.1 against 2 us)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        # (last, and whole: another thread's call may come in between)
        _FMTS = {torch.bfloat16: ("bf16", 1), torch.float16: ("f16", 0)}
    return torch


def _check_like(t, dtype, dev: int, dims: int, what: str, shape=None):
    """A tensor of this type on device number ``dev``, with ``dims``
    dimensions, a unit last stride and (where given) this shape."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s like A, got %s" % (what, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("operands on different devices: A on cuda:%d, %s on %s"
                         % (dev, what, t.device))
    if t.dim() != dims or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError("%s must be %d-D with unit stride in its last dimension" % (what, dims))
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), shape))


def _check_first(A):
    """A's format, as (name, dense_gemm_fmt), type and device number."""
    dtype = A.dtype
    fmt = _FMTS.get(dtype)
    if fmt is None:
        raise TypeError("A must be float16 or bfloat16, got %s" % dtype)
    if not A.is_cuda:
        raise ValueError("A must be a device tensor")
    if A.dim() != 2 or (A.stride(1) != 1 and A.shape[1] > 1):
        raise ValueError("A must be 2-D with unit column stride")
    return fmt, dtype, A.get_device()


def _check_ends(ends, dev, torch):
    if ends.dtype is not torch.int32:
        raise TypeError("ends must be int32, got %s" % ends.dtype)
    if ends.get_device() != dev:
        raise ValueError("operands on different devices: A on cuda:%d, ends on %s"
                         % (dev, ends.device))
    if ends.dim() != 1 or (ends.shape[0] > 1 and ends.stride(0) != 1):
        raise ValueError("ends must be 1-D and contiguous")


def _stack(t):
    """(elements between the matrices, leading dimension) of a 3-D tensor with
    unit last stride."""
    ld = t.stride(1) if t.shape[1] > 1 else max(t.shape[2], 1)
    return (t.stride(0) if t.shape[0] > 1 else 0), ld


def _launch(name, args, size_of, workspace, stream, dev, torch):
    """Calls ``name(*args, workspace, bytes, stream)`` on device number
    ``dev``.  Without a workspace of the caller's, one is taken from torch's
    allocator if the call turns out to need it (``size_of``: its size query
    and that query's arguments)."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _launch(name, args, size_of, workspace, stream, dev, torch)
    fn = getattr(_lib, name)
    if stream is None and _raw_stream is not None:
        sh = _raw_stream(dev)
    else:
        sh = _stream_handle(stream, dev)
    if workspace is None or workspace is True:
        st = fn(*args, None, 0, sh)
        if st == 10:  # WORKSPACE_TOO_SMALL
            need = ctypes.c_size_t()
            st = getattr(_lib, size_of[0])(*size_of[1:], ctypes.byref(need))
            if st == 0:
                ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
                if stream is not None:
                    _used_by(ws, stream, ws.device)
                st = fn(*args, ws.data_ptr(), need.value, sh)
    else:
        if workspace.get_device() != dev:
            raise ValueError("workspace must be a device tensor on cuda:%d" % dev)
        if not workspace.is_contiguous():  # (its bytes are not its elements')
            raise ValueError("workspace must be contiguous")
        st = fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), sh)
    if st != 0:
        raise DenseGemmError(st, name)


def _layer(layout, A, B, ends, bias, act, residual, preact, grad, D, stream, workspace):
    if _lib is None:
        load_library()
    torch = _torch()
    fmt, dtype, dev = _check_first(A)
    code = ACTS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTS), act))
    M, K = A.shape
    _check_like(B, dtype, dev, 2 if ends is None else 3, "B")
    if layout == "nt":
        N, Kb = B.shape[-2:]
    else:
        Kb, N = B.shape[-2:]
    if Kb != K:
        raise ValueError("inner dimensions differ: A is %s, B is %s"
                         % (tuple(A.shape), tuple(B.shape)))
    groups, G = None, ()
    if ends is None:
        ldb = _ld(B)
    else:
        _check_ends(ends, dev, torch)
        G = (B.shape[0],)
        if ends.shape[0] != G[0]:
            raise ValueError("%d group ends for %d matrices B" % (ends.shape[0], G[0]))
        stride, ldb = _stack(B)
        groups = Groups(ends.data_ptr(), G[0], stride)
    epi = None
    if grad or code or bias is not None or residual is not None or preact is not None:
        epi = Epilogue(act=code, grad=grad)
        if bias is not None:
            _check_like(bias, dtype, dev, 1 + len(G), "bias", G + (N,))
            epi.bias = bias.data_ptr()
            if G and G[0] > 1:
                epi.bias_stride = bias.stride(0)
        if residual is not None:
            _check_like(residual, dtype, dev, 2, "residual", (M, N))
            epi.residual, epi.ldr = residual.data_ptr(), _ld(residual)
        if preact is not None:
            _check_like(preact, dtype, dev, 2, "preact", (M, N))
            epi.preact, epi.ldz = preact.data_ptr(), _ld(preact)
    if D is None:
        D = torch.empty((M, N), dtype=dtype, device=A.device)
        if stream is not None:
            _used_by(D, stream, A.device)
    else:
        _check_like(D, dtype, dev, 2, "D", (M, N))
    args = (OPS[(layout, fmt[0])], M, N, K, A.data_ptr(), _ld(A), B.data_ptr(), ldb)
    _launch("dense_gemm_layer", args + (D.data_ptr(), _ld(D), epi, groups),
            ("dense_gemm_layer_workspace_size",) + args + (groups, 0), workspace, stream, dev, torch)
    return D


def gemm_nt_fused(A, B, bias=None, act="none", residual=None, preact=None, D=None, stream=None,
                  workspace=None):
    """D = act(Z) + residual with Z = A @ B.T + bias, FP16 or BF16 with FP32
    accumulation and one rounding; A is M x K, B is N x K, bias has N values,
    residual is M x N and may be D itself.  ``act``: "none", "relu", "gelu",
    "gelu_tanh" or "silu".  ``preact``: an M x N tensor that receives Z (for
    :func:`gemm_nn_dact`); it must overlap no other.  ``workspace``: a device
    tensor (256-byte aligned, dense_gemm_layer_workspace_size bytes), or None
    to take one from torch's allocator where the call needs it.  The call is
    asynchronous on ``stream`` (None: the current stream)."""
    return _layer("nt", A, B, None, bias, act, residual, preact, 0, D, stream, workspace)


def gemm_nn_fused(A, B, bias=None, act="none", residual=None, preact=None, D=None, stream=None,
                  workspace=None):
    """:func:`gemm_nt_fused` with B K x N: Z = A @ B + bias."""
    return _layer("nn", A, B, None, bias, act, residual, preact, 0, D, stream, workspace)


def gemm_nt_dact(A, B, preact, act, D=None, stream=None, workspace=None):
    """D = (A @ B.T) * act'(preact): the gradient of a layer's input carried
    through the activation that produced it.  A is M x K, B is N x K, preact
    (M x N, may be D itself) is what the forward call stored; ``act`` as
    there, but not "none".  Other arguments as for :func:`gemm_nt_fused`."""
    return _layer("nt", A, B, None, None, act, None, preact, 1, D, stream, workspace)


def gemm_nn_dact(A, B, preact, act, D=None, stream=None, workspace=None):
    """:func:`gemm_nt_dact` with B K x N: D = (A @ B) * act'(preact)."""
    return _layer("nn", A, B, None, None, act, None, preact, 1, D, stream, workspace)


def gemm_nt_grouped(A, B, ends, bias=None, act="none", residual=None, preact=None, D=None,
                    stream=None, workspace=None):
    """:func:`gemm_nt_fused` for rows sorted into G groups (the experts of a
    layer): rows ends[g - 1] .. ends[g] - 1 of A (M x K) are multiplied with
    B[g] (G x N x K) and take bias[g] (G x N).  ``ends``: G int32 values on
    the device, not decreasing; the host never reads them.  Rows at or past
    the last end are not written (with D None they hold whatever the
    allocator returned), and what the operands hold there changes nothing."""
    return _layer("nt", A, B, ends, bias, act, residual, preact, 0, D, stream, workspace)


def gemm_nn_grouped(A, B, ends, bias=None, act="none", residual=None, preact=None, D=None,
                    stream=None, workspace=None):
    """:func:`gemm_nt_grouped` with B G x K x N."""
    return _layer("nn", A, B, ends, bias, act, residual, preact, 0, D, stream, workspace)


def gemm_nt_grouped_dact(A, B, ends, preact, act, D=None, stream=None, workspace=None):
    """:func:`gemm_nt_dact` for rows sorted into groups, with B G x N x K."""
    return _layer("nt", A, B, ends, None, act, None, preact, 1, D, stream, workspace)


def gemm_nn_grouped_dact(A, B, ends, preact, act, D=None, stream=None, workspace=None):
    """:func:`gemm_nn_dact` for rows sorted into groups, with B G x K x N."""
    return _layer("nn", A, B, ends, None, act, None, preact, 1, D, stream, workspace)


def _tn(A, B, ends, D, colsum, stream, workspace):
    if _lib is None:
        load_library()
    torch = _torch()
    fmt, dtype, dev = _check_first(A)
    K, M = A.shape
    _check_like(B, dtype, dev, 2, "B")
    N = B.shape[1]
    if B.shape[0] != K:
        raise ValueError("row counts differ: A is %s, B is %s" % (tuple(A.shape), tuple(B.shape)))
    G = ()
    if ends is not None:
        _check_ends(ends, dev, torch)
        G = (ends.shape[0],)
    own = []
    if D is None:
        D = torch.empty(G + (M, N), dtype=dtype, device=A.device)
        own.append(D)
    else:
        _check_like(D, dtype, dev, 2 + len(G), "D", G + (M, N))
    sums = None
    if colsum is True:
        sums = torch.empty(G + (M,), dtype=dtype, device=A.device)
        own.append(sums)
    elif colsum is not None and colsum is not False:
        sums = colsum
        _check_like(sums, dtype, dev, 1 + len(G), "colsum", G + (M,))
        if not sums.is_contiguous():
            raise ValueError("colsum must be contiguous")
    if stream is not None:
        for t in own:
            _used_by(t, stream, A.device)
    groups = None
    if ends is None:
        ldd = _ld(D)
    else:
        stride, ldd = _stack(D)
        groups = Groups(ends.data_ptr(), G[0], stride)
    args = (M, N, K, A.data_ptr(), _ld(A), B.data_ptr(), _ld(B))
    _launch("dense_gemm_tn",
            (fmt[1],) + args + (D.data_ptr(), ldd, None if sums is None else sums.data_ptr(), groups),
            ("dense_gemm_tn_workspace_size",) + args + (sums is not None, groups, 0), workspace,
            stream, dev, torch)
    return D if sums is None else (D, sums)


def gemm_tn(A, B, D=None, colsum=None, stream=None, workspace=None):
    """D = A.T @ B (M x N, FP16 or BF16, FP32 accumulation): a layer's weight
    gradient from the gradient of its output, A (K x M, a row per token), and
    its input, B (K x N).  ``colsum``: True, or a tensor of M values, for the
    sums of A's columns too (the bias gradient): returns (D, colsum).
    ``workspace`` (dense_gemm_tn_workspace_size bytes) and ``stream`` as for
    :func:`gemm_nt_fused`."""
    return _tn(A, B, None, D, colsum, stream, workspace)


def gemm_tn_grouped(A, B, ends, D=None, colsum=None, stream=None, workspace=None):
    """:func:`gemm_tn` for rows sorted into G groups (``ends`` as for
    :func:`gemm_nt_grouped`): D is G x M x N and colsum G x M, each group's
    sums over its own rows, zero for an empty group."""
    return _tn(A, B, ends, D, colsum, stream, workspace)
