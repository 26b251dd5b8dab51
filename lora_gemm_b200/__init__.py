"""Thin Python binding of the lora_gemm C ABI (include/lora_gemm.h).

Every function here only marshals arguments -- checks dtypes, shapes,
devices and contiguity of torch tensors, allocates outputs with torch when
the caller does not pass them, and hands raw device pointers plus the current
CUDA stream to liblora_gemm.so.  All arithmetic runs in the library's CUDA
kernels; there is no CPU path.  Importing this package fails with ImportError
when the compiled library is missing (build it with
``python lora_gemm_b200/build.py``).
"""

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblora_gemm.so")

LG_OK = 0
LG_ERR_INVALID_ARG = 1
LG_ERR_UNSUPPORTED_SHAPE = 2
LG_ERR_MISALIGNED = 3
LG_ERR_WORKSPACE = 4
LG_ERR_CUDA = 5
LG_ERR_DEVICE_TIMEOUT = 6
LG_ERR_NOT_SM100 = 7

# Size of the built-in scratch array of lg_lora_linear_noalloc (the header's
# LG_NOALLOC_SCRATCH_BYTES).
LG_NOALLOC_SCRATCH_BYTES = 48 << 20

# Norm kinds, stream types and code formats of the block norms (the header's LG_NORM_*, LG_STREAM_*, LG_CODES_*).
_NORM = {None: 0, "rms": 1, "layer": 2}
_STREAM = {torch.bfloat16: 0, torch.float32: 1}
_CODES = {None: 0, "mxfp8": 1, "mxfp4": 2}

# Exported C symbols and their ctypes signatures (the header's declarations).
_c_void_p = ctypes.c_void_p


class BlockNormArgs(ctypes.Structure):
    """lg_block_norm_args."""

    _fields_ = [(f, _c_void_p) for f in ("h", "b", "gate", "scale", "shift", "h_out", "n", "codes", "scales")] + [
        ("M", ctypes.c_int64), ("segment_tokens", ctypes.c_int64), ("D", ctypes.c_int),
        ("stream_type", ctypes.c_int), ("post", ctypes.c_int), ("pre", ctypes.c_int), ("codes_format", ctypes.c_int),
        ("alpha", ctypes.c_float), ("eps", ctypes.c_float)]


class BlockNormBackwardArgs(ctypes.Structure):
    """lg_block_norm_backward_args."""

    _fields_ = [(f, _c_void_p) for f in ("dn", "dh_out", "h_out", "b", "gate", "scale", "dh", "db", "dgate", "dscale",
                                         "dshift")] + [
        ("M", ctypes.c_int64), ("segment_tokens", ctypes.c_int64), ("D", ctypes.c_int),
        ("stream_type", ctypes.c_int), ("post", ctypes.c_int), ("pre", ctypes.c_int), ("alpha", ctypes.c_float),
        ("eps", ctypes.c_float)]


_SIGNATURES = {
    "lg_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "lg_version": (ctypes.c_int, []),
    "lg_launch_count": (ctypes.c_uint64, []),
    "lg_get_last_device_error": (ctypes.c_int, [_c_void_p]),
    "lg_set_wait_limit_ns": (None, [ctypes.c_uint64]),
    "lg_set_cluster_size": (ctypes.c_int, [ctypes.c_int]),
    "lg_set_kernel_variant": (ctypes.c_int, [ctypes.c_int]),
    "lg_lora_merge": (
        ctypes.c_int,
        [ctypes.c_int, ctypes.POINTER(_c_void_p), ctypes.POINTER(_c_void_p), ctypes.POINTER(ctypes.c_int),
         ctypes.POINTER(ctypes.c_float), ctypes.c_int, ctypes.c_int, _c_void_p, _c_void_p, _c_void_p],
    ),
    "lg_lora_linear_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "lg_lora_linear": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
         ctypes.c_int, _c_void_p, ctypes.c_size_t, _c_void_p],
    ),
    "lg_lora_linear_mxfp8": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64,
         ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t, _c_void_p],
    ),
    "lg_lora_linear_swiglu_mxfp8": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
         ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t, _c_void_p],
    ),
    "lg_lora_linear_euler_workspace_size": (
        ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    ),
    "lg_lora_linear_euler": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64, ctypes.c_int,
         ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_float, _c_void_p, ctypes.c_size_t,
         _c_void_p],
    ),
    "lg_lora_linear_noalloc": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
         ctypes.c_int, _c_void_p],
    ),
    "lg_mx_scale_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int]),
    "lg_mx_quantize": (ctypes.c_int, [_c_void_p, ctypes.c_int64, ctypes.c_int, _c_void_p, _c_void_p, _c_void_p]),
    "lg_mxfp4_quantize": (ctypes.c_int, [_c_void_p, ctypes.c_int64, ctypes.c_int, _c_void_p, _c_void_p, _c_void_p]),
    "lg_mxfp4_dequantize": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int64, ctypes.c_int, _c_void_p, _c_void_p]),
    "lg_lora_linear_mxfp4_workspace_size": (
        ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    ),
    "lg_lora_linear_mxfp4": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, ctypes.c_int64,
         ctypes.c_int, ctypes.c_int, ctypes.c_int, _c_void_p, ctypes.c_size_t, _c_void_p],
    ),
    "lg_block_norm": (ctypes.c_int, [ctypes.POINTER(BlockNormArgs), _c_void_p]),
    "lg_block_norm_backward_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]),
    "lg_block_norm_backward": (
        ctypes.c_int, [ctypes.POINTER(BlockNormBackwardArgs), _c_void_p, ctypes.c_size_t, _c_void_p]
    ),
    "lg_renoise": (
        ctypes.c_int,
        [_c_void_p, _c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64, _c_void_p],
    ),
    "lg_euler_step": (
        ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_float, _c_void_p]
    ),
    "lg_shift_ladder": (
        ctypes.c_int,
        [ctypes.c_float, ctypes.c_int, ctypes.c_double, ctypes.POINTER(ctypes.c_float), ctypes.c_int,
         ctypes.POINTER(ctypes.c_int)],
    ),
    "lg_philox_u32": (ctypes.c_int, [_c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint64, _c_void_p]),
    "lg_philox_normal": (ctypes.c_int, [_c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_uint64, _c_void_p]),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"lora_gemm CUDA library not found at {LIB_PATH}; build it with `python lora_gemm_b200/build.py`"
        )
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class LoraGemmError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib.lg_status_string(status).decode()
        super().__init__(f"{where}: status {status} ({msg})")


def _check(status, where):
    if status != LG_OK:
        raise LoraGemmError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _at_least(t, nbytes, name):
    _need(t, torch.uint8, name)
    if t.numel() < nbytes:
        raise ValueError(f"{name} holds {t.numel()} bytes, needs {nbytes}")


def _same_device(ref, *tensors):
    """Every tensor given (None skipped) on ref's device: the kernels run there."""
    for t in tensors:
        if t is not None and t.device != ref.device:
            raise ValueError(f"all tensors must be on {ref.device}, got one on {t.device}")


def _addr(t):
    """A tensor's address as ctypes takes it for a pointer argument (None for null)."""
    return None if t is None else t.data_ptr()


def _launch(device, fn, *args):
    """fn(*args, current stream of device), with device current."""
    index = device.index
    if index == torch.cuda.current_device():
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(device):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def _scales(pair, rows, K, what):
    codes, sc = pair
    _need(codes, torch.uint8, f"{what} codes", 2)
    _shape(codes, (rows, K), f"{what} codes")
    _at_least(sc, mx_scale_bytes(rows, K), f"{what} scales")
    return codes, sc


def status_string(status):
    return lib.lg_status_string(int(status)).decode()


def version():
    return lib.lg_version()


def launch_count():
    """Kernels launched by the library so far in this process."""
    return int(lib.lg_launch_count())


def set_wait_limit_ns(limit_ns):
    """Bound on each wait inside lora_linear's pipeline; 0 restores the default."""
    lib.lg_set_wait_limit_ns(int(limit_ns))


def set_cluster_size(g):
    """SMs sharing one token panel in lora_linear (1, 2, 4, 8; 0 = chosen per shape)."""
    _check(lib.lg_set_cluster_size(int(g)), "lg_set_cluster_size")


def set_kernel_variant(v):
    """lora_linear MMA variant: 1 single-SM, 2 SM pair, 0 chosen per shape."""
    _check(lib.lg_set_kernel_variant(int(v)), "lg_set_kernel_variant")


def get_last_device_error(device=None):
    """Synchronize the current stream and read/clear the device error word (a status code)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        return lib.lg_get_last_device_error(_stream(device))


def lora_merge(As, Bs, scales, A_cat=None, B_cat=None):
    """A_cat = [s_i A_i] stacked along the rank axis, B_cat = [B_i] side by side (FP32)."""
    n = len(As)
    if n != len(Bs) or n != len(scales):
        raise ValueError("As, Bs and scales must have equal length")
    for i, (A, B) in enumerate(zip(As, Bs)):
        _need(A, torch.float32, f"A[{i}]", 2)
        _need(B, torch.float32, f"B[{i}]", 2)
    d_in = As[0].shape[1]
    d_out = Bs[0].shape[0]
    ranks = [A.shape[0] for A in As]
    for A, B in zip(As, Bs):
        if A.shape[1] != d_in or B.shape[0] != d_out or B.shape[1] != A.shape[0]:
            raise ValueError("adapter factor shapes disagree")
    R = sum(ranks)
    dev = As[0].device
    if A_cat is None:
        A_cat = torch.empty((R, d_in), dtype=torch.float32, device=dev)
    if B_cat is None:
        B_cat = torch.empty((d_out, R), dtype=torch.float32, device=dev)
    _need(A_cat, torch.float32, "A_cat", 2)
    _need(B_cat, torch.float32, "B_cat", 2)
    _shape(A_cat, (R, d_in), "A_cat")
    _shape(B_cat, (d_out, R), "B_cat")
    _same_device(A_cat, B_cat, *As, *Bs)
    a_ptrs = (ctypes.c_void_p * n)(*[A.data_ptr() for A in As])
    b_ptrs = (ctypes.c_void_p * n)(*[B.data_ptr() for B in Bs])
    r_arr = (ctypes.c_int * n)(*ranks)
    s_arr = (ctypes.c_float * n)(*[float(s) for s in scales])
    with torch.cuda.device(dev):
        st = lib.lg_lora_merge(n, a_ptrs, b_ptrs, r_arr, s_arr, d_in, d_out, _ptr(A_cat), _ptr(B_cat), _stream(dev))
    _check(st, "lg_lora_merge")
    return A_cat, B_cat


def lora_linear_workspace_size(M, K, N, R):
    return int(lib.lg_lora_linear_workspace_size(int(M), int(K), int(N), int(R)))


def lora_linear(x, W, A_cat, B_cat, y=None, workspace=None):
    """y = x W^T + (x A_cat^T) B_cat^T; bf16 x [M, K], W [N, K]; FP32 A_cat [R, K], B_cat [N, R]."""
    _need(x, torch.bfloat16, "x", 2)
    _need(W, torch.bfloat16, "W", 2)
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be [N, K]")
    R = 0
    if A_cat is not None and A_cat.numel() > 0:
        _need(A_cat, torch.float32, "A_cat", 2)
        _need(B_cat, torch.float32, "B_cat", 2)
        R = A_cat.shape[0]
        if A_cat.shape[1] != K or tuple(B_cat.shape) != (N, R):
            raise ValueError("A_cat must be [R, K] and B_cat [N, R]")
    else:
        A_cat = B_cat = None
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, torch.bfloat16, "y", 2)
    _shape(y, (M, N), "y")
    need = lora_linear_workspace_size(M, K, N, R)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _same_device(x, W, A_cat, B_cat, y, workspace)
    with torch.cuda.device(x.device):
        st = lib.lg_lora_linear(_ptr(x), _ptr(W), _ptr(A_cat), _ptr(B_cat), _ptr(y), M, K, N, R,
                                _ptr(workspace), ws_bytes, _stream(x.device))
    _check(st, "lg_lora_linear")
    return y


def mx_scale_bytes(rows, K):
    """Bytes of E8M0 scales lg_mx_quantize writes for [rows, K] (0 for an unsupported shape)."""
    return int(lib.lg_mx_scale_bytes(int(rows), int(K)))


def mx_quantize(x, codes=None, scales=None):
    """MXFP8 of bf16 rows x [rows, K] along K: (E4M3 codes uint8 [rows, K],
    E8M0 scales uint8 in the blocked layout of include/lora_gemm.h)."""
    _need(x, torch.bfloat16, "x", 2)
    rows, K = x.shape
    if codes is None:
        codes = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(max(mx_scale_bytes(rows, K), 1), dtype=torch.uint8, device=x.device)
    _need(codes, torch.uint8, "codes", 2)
    _shape(codes, (rows, K), "codes")
    _at_least(scales, mx_scale_bytes(rows, K), "scales")
    _same_device(x, codes, scales)
    with torch.cuda.device(x.device):
        st = lib.lg_mx_quantize(_ptr(x), rows, K, _ptr(codes), _ptr(scales), _stream(x.device))
    _check(st, "lg_mx_quantize")
    return codes, scales


def lora_linear_mxfp8(x, x_mx, W_mx, A_cat, B_cat, y=None, workspace=None):
    """lora_linear with the base term as MXFP8 GEMMs: x_mx = mx_quantize(x),
    W_mx = mx_quantize(W) (pairs of codes and scales); the LoRA term from the
    bf16 x.  K must be a multiple of 128."""
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    _need(W_mx[0], torch.uint8, "W codes", 2)
    N = W_mx[0].shape[0]
    xq, xsf = _scales(x_mx, M, K, "x")
    wq, wsf = _scales(W_mx, N, K, "W")
    R = 0
    if A_cat is not None and A_cat.numel() > 0:
        _need(A_cat, torch.float32, "A_cat", 2)
        _need(B_cat, torch.float32, "B_cat", 2)
        R = A_cat.shape[0]
        if A_cat.shape[1] != K or tuple(B_cat.shape) != (N, R):
            raise ValueError("A_cat must be [R, K] and B_cat [N, R]")
    else:
        A_cat = B_cat = None
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _need(y, torch.bfloat16, "y", 2)
    _shape(y, (M, N), "y")
    need = lora_linear_workspace_size(M, K, N, R)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _same_device(x, xq, xsf, wq, wsf, A_cat, B_cat, y, workspace)
    with torch.cuda.device(x.device):
        st = lib.lg_lora_linear_mxfp8(_ptr(x), _ptr(xq), _ptr(xsf), _ptr(wq), _ptr(wsf), _ptr(A_cat), _ptr(B_cat),
                                      _ptr(y), M, K, N, R, _ptr(workspace), ws_bytes, _stream(x.device))
    _check(st, "lg_lora_linear_mxfp8")
    return y


def lora_linear_swiglu_mxfp8(x, x_mx, W2_mx, A_cat, B_cat, out=None, workspace=None):
    """MLP input projection with SwiGLU and the MXFP8 quantizer fused: W2 [2F, K]
    (gate rows, then up rows) as mx_quantize(W2); returns (codes [M, F], scales)
    of silu(z[:, :F]) * z[:, F:] with z = x W2^T + LoRA."""
    _need(x, torch.bfloat16, "x", 2)
    M, K = x.shape
    _need(W2_mx[0], torch.uint8, "W2 codes", 2)
    N2 = W2_mx[0].shape[0]
    if N2 % 2:
        raise ValueError("W2 must have 2F rows (gate rows, then up rows)")
    F = N2 // 2
    xq, xsf = _scales(x_mx, M, K, "x")
    wq, wsf = _scales(W2_mx, N2, K, "W2")
    R = 0
    if A_cat is not None and A_cat.numel() > 0:
        _need(A_cat, torch.float32, "A_cat", 2)
        _need(B_cat, torch.float32, "B_cat", 2)
        R = A_cat.shape[0]
        if A_cat.shape[1] != K or tuple(B_cat.shape) != (N2, R):
            raise ValueError("A_cat must be [R, K] and B_cat [2F, R]")
    else:
        A_cat = B_cat = None
    if out is None:
        out = (torch.empty((M, F), dtype=torch.uint8, device=x.device),
               torch.empty(max(mx_scale_bytes(M, F), 1), dtype=torch.uint8, device=x.device))
    _need(out[0], torch.uint8, "output codes", 2)
    _shape(out[0], (M, F), "output codes")
    _at_least(out[1], mx_scale_bytes(M, F), "output scales")
    need = lora_linear_workspace_size(M, K, N2, R)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _same_device(x, xq, xsf, wq, wsf, A_cat, B_cat, out[0], out[1], workspace)
    with torch.cuda.device(x.device):
        st = lib.lg_lora_linear_swiglu_mxfp8(_ptr(x), _ptr(xq), _ptr(xsf), _ptr(wq), _ptr(wsf), _ptr(A_cat),
                                             _ptr(B_cat), _ptr(out[0]), _ptr(out[1]), M, K, F, R, _ptr(workspace),
                                             ws_bytes, _stream(x.device))
    _check(st, "lg_lora_linear_swiglu_mxfp8")
    return out


def lora_linear_euler_workspace_size(M, K, N, R):
    return int(lib.lg_lora_linear_euler_workspace_size(int(M), int(K), int(N), int(R)))


def lora_linear_euler(x, W, A_cat, B_cat, z, sigma, sigma_next, frame_tokens, z_bf16=None, workspace=None):
    """The step's last projection with the Euler update fused: v = x W^T +
    (x A_cat^T) B_cat^T (W [C, K]) updates the FP32 latent z [frames, C,
    frame_tokens] in place, z += (sigma_next - sigma) v (token m = cell
    m mod frame_tokens of frame m // frame_tokens); z_bf16 (same shape, or
    None) receives bf16(z).  Returns z."""
    _need(x, torch.bfloat16, "x", 2)
    _need(W, torch.bfloat16, "W", 2)
    _need(z, torch.float32, "z")
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be [N, K]")
    if z.numel() != M * N:
        raise ValueError("z must hold M * N elements")
    if z_bf16 is not None:
        _need(z_bf16, torch.bfloat16, "z_bf16")
        if z_bf16.numel() != z.numel():
            raise ValueError("z_bf16 must have as many elements as z")
    R = 0
    if A_cat is not None and A_cat.numel() > 0:
        _need(A_cat, torch.float32, "A_cat", 2)
        _need(B_cat, torch.float32, "B_cat", 2)
        R = A_cat.shape[0]
        if A_cat.shape[1] != K or tuple(B_cat.shape) != (N, R):
            raise ValueError("A_cat must be [R, K] and B_cat [N, R]")
    else:
        A_cat = B_cat = None
    need = lora_linear_euler_workspace_size(M, K, N, R)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _same_device(x, W, A_cat, B_cat, z, z_bf16, workspace)
    with torch.cuda.device(x.device):
        st = lib.lg_lora_linear_euler(_ptr(x), _ptr(W), _ptr(A_cat), _ptr(B_cat), _ptr(z), _ptr(z_bf16), M, K, N, R,
                                      int(frame_tokens), float(sigma), float(sigma_next), _ptr(workspace), ws_bytes,
                                      _stream(x.device))
    _check(st, "lg_lora_linear_euler")
    return z


def lora_linear_noalloc(x, W, A_cat, B_cat, y):
    """lora_linear without a workspace, for callers that cannot allocate device
    memory at call time: the factor copies go to the library's built-in scratch
    array (see lg_lora_linear_noalloc in include/lora_gemm.h).  y must be given."""
    _need(x, torch.bfloat16, "x", 2)
    _need(W, torch.bfloat16, "W", 2)
    _need(y, torch.bfloat16, "y", 2)
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be [N, K]")
    _shape(y, (M, N), "y")
    R = 0
    if A_cat is not None and A_cat.numel() > 0:
        _need(A_cat, torch.float32, "A_cat", 2)
        _need(B_cat, torch.float32, "B_cat", 2)
        R = A_cat.shape[0]
        if A_cat.shape[1] != K or tuple(B_cat.shape) != (N, R):
            raise ValueError("A_cat must be [R, K] and B_cat [N, R]")
    else:
        A_cat = B_cat = None
    _same_device(x, W, A_cat, B_cat, y)
    with torch.cuda.device(x.device):
        st = lib.lg_lora_linear_noalloc(_ptr(x), _ptr(W), _ptr(A_cat), _ptr(B_cat), _ptr(y), M, K, N, R,
                                        _stream(x.device))
    _check(st, "lg_lora_linear_noalloc")
    return y


# The library's size functions, remembered: each is pure host arithmetic, and a
# foreign call costs more than a short call's other checks together.
_scale_bytes = functools.lru_cache(4096)(mx_scale_bytes)


def mxfp4_quantize(x, codes=None, scales=None):
    """MXFP4 of bf16 rows x [rows, K] along K: (E2M1 codes uint8 [rows, K / 2],
    two per byte, E8M0 scales uint8 in mx_quantize's blocked layout)."""
    _need(x, torch.bfloat16, "x", 2)
    rows, K = x.shape
    nscales = _scale_bytes(rows, K)
    if codes is None:
        codes = x.new_empty((rows, K // 2), dtype=torch.uint8)
    else:
        _need(codes, torch.uint8, "codes", 2)
        _shape(codes, (rows, K // 2), "codes")
    if scales is None:
        scales = x.new_empty(nscales, dtype=torch.uint8)
    else:
        _at_least(scales, nscales, "scales")
    _same_device(x, codes, scales)
    _check(_launch(x.device, lib.lg_mxfp4_quantize, _addr(x), rows, K, _addr(codes), _addr(scales)), "lg_mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, out=None):
    """The bf16 values [rows, K] that MXFP4 codes [rows, K / 2] and scales stand for (exact)."""
    _need(codes, torch.uint8, "codes", 2)
    rows, K = codes.shape[0], 2 * codes.shape[1]
    _at_least(scales, _scale_bytes(rows, K), "scales")
    if out is None:
        out = codes.new_empty((rows, K), dtype=torch.bfloat16)
    else:
        _need(out, torch.bfloat16, "out", 2)
        _shape(out, (rows, K), "out")
    _same_device(codes, scales, out)
    _check(_launch(codes.device, lib.lg_mxfp4_dequantize, _addr(codes), _addr(scales), rows, K, _addr(out)),
           "lg_mxfp4_dequantize")
    return out


def lora_linear_mxfp4_workspace_size(M, K, N, R):
    return int(lib.lg_lora_linear_mxfp4_workspace_size(int(M), int(K), int(N), int(R)))


_linear_mxfp4_bytes = functools.lru_cache(4096)(lora_linear_mxfp4_workspace_size)


def lora_linear_mxfp4(x, x_mx, W_mx, A_cat, B_cat, y=None, workspace=None):
    """lora_linear with the base term as MXFP4 products: x_mx = mxfp4_quantize(x)
    (or the codes block_norm wrote with it), W_mx = mxfp4_quantize(W) (pairs of
    codes and scales); the LoRA term from the bf16 x, which may be None without
    adapters.  K must be a multiple of 128."""
    xq, xsf = x_mx
    wq, wsf = W_mx
    _need(xq, torch.uint8, "x codes", 2)
    _need(wq, torch.uint8, "W codes", 2)
    M, K, N = xq.shape[0], 2 * xq.shape[1], wq.shape[0]
    if wq.shape[1] != xq.shape[1]:
        raise ValueError(f"W codes must have shape {(N, K // 2)}, got {tuple(wq.shape)}")
    _at_least(xsf, _scale_bytes(M, K), "x scales")
    _at_least(wsf, _scale_bytes(N, K), "W scales")
    R = 0
    if A_cat is not None and A_cat.numel() > 0:
        _need(A_cat, torch.float32, "A_cat", 2)
        _need(B_cat, torch.float32, "B_cat", 2)
        R = A_cat.shape[0]
        if A_cat.shape[1] != K or tuple(B_cat.shape) != (N, R):
            raise ValueError("A_cat must be [R, K] and B_cat [N, R]")
    else:
        A_cat = B_cat = None
    if x is not None or R > 0:
        _need(x, torch.bfloat16, "x", 2)
        _shape(x, (M, K), "x")
    if y is None:
        y = xq.new_empty((M, N), dtype=torch.bfloat16)
    else:
        _need(y, torch.bfloat16, "y", 2)
        _shape(y, (M, N), "y")
    need = _linear_mxfp4_bytes(M, K, N, R)
    if workspace is None and need > 0:
        workspace = xq.new_empty(need)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _same_device(xq, x, xsf, wq, wsf, A_cat, B_cat, y, workspace)
    if M == 0:
        return y
    st = _launch(xq.device, lib.lg_lora_linear_mxfp4, _addr(x), _addr(xq), _addr(xsf), _addr(wq), _addr(wsf), _addr(A_cat),
                 _addr(B_cat), _addr(y), M, K, N, R, _addr(workspace), ws_bytes)
    _check(st, "lg_lora_linear_mxfp4")
    return y


def _norm_args(h, post, pre, segment_tokens):
    """(M, D, segment_tokens, S) of a block-norm call, its kinds checked."""
    if not isinstance(h, torch.Tensor) or h.dtype not in _STREAM:
        raise TypeError("the stream must be a bfloat16 or float32 torch.Tensor")
    _need(h, h.dtype, "the stream", 2)
    for kind, name in ((post, "post"), (pre, "pre")):
        if kind not in _NORM:
            raise ValueError(f"{name} must be None, 'rms' or 'layer', got {kind!r}")
    M, D = h.shape
    seg = max(M, 1) if segment_tokens is None else int(segment_tokens)
    if seg < 1:
        raise ValueError("segment_tokens must be at least 1")
    return M, D, seg, -(-M // seg)


def _modulation(t, S, D, name):
    if t is not None:
        _need(t, torch.float32, name, 2)
        _shape(t, (S, D), name)


def block_norm(h, b=None, gate=None, scale=None, shift=None, alpha=1.0, eps=1e-6, post="rms", pre="rms",
               segment_tokens=None, quant=None, h_out=None, n=None, q=None):
    """The norms between two blocks, with the gate and the scaled residual:

        h' = alpha h + gate * N_post(b),   n = N_pre(h') (1 + scale) + shift

    h [M, D] is the residual stream (bf16 or FP32), b [M, D] bf16 the block's
    output; gate, scale, shift FP32 [S, D] hold one row per segment of
    segment_tokens rows (default: one segment).  post and pre are "rms",
    "layer" or None; without b (the norm that opens a network) there is nothing
    to norm after the block: post "rms", the default, counts as None then, and
    "layer" is refused.
    quant "mxfp8" or "mxfp4" also quantizes n, as mx_quantize(n) or
    mxfp4_quantize(n) would.  Returns (h', n, (codes, scales)); h' is h itself
    without b, n is None without pre, the pair is None without quant.  Outputs
    may be passed in: h_out (h itself updates in place), n, q."""
    if b is None and post == "rms":
        post = None  # the default kind has nothing to norm
    M, D, seg, S = _norm_args(h, post, pre, segment_tokens)
    if quant not in _CODES:
        raise ValueError(f"quant must be None, 'mxfp8' or 'mxfp4', got {quant!r}")
    _modulation(gate, S, D, "gate")
    _modulation(scale, S, D, "scale")
    _modulation(shift, S, D, "shift")
    dev = h.device
    if b is not None:
        _need(b, torch.bfloat16, "b", 2)
        _shape(b, (M, D), "b")
        if h_out is None:
            h_out = torch.empty_like(h)
        else:
            _need(h_out, h.dtype, "h_out", 2)
            _shape(h_out, (M, D), "h_out")
    elif h_out is not None:
        raise ValueError("h_out needs b: without a block's output the stream stays as it is")
    if pre is not None and n is None:
        n = h.new_empty((M, D), dtype=torch.bfloat16)
    elif n is not None:
        _need(n, torch.bfloat16, "n", 2)
        _shape(n, (M, D), "n")
    codes = scales = None
    if quant is not None:
        width = D if quant == "mxfp8" else D // 2
        nscales = _scale_bytes(M, D)
        if q is None:
            q = (h.new_empty((M, width), dtype=torch.uint8),
                 h.new_empty(nscales, dtype=torch.uint8))
        codes, scales = q
        _need(codes, torch.uint8, "codes", 2)
        _shape(codes, (M, width), "codes")
        _at_least(scales, nscales, "scales")
    elif q is not None:
        raise ValueError("q needs quant")
    _same_device(h, b, gate, scale, shift, h_out, n, codes, scales)
    if M > 0:
        args = BlockNormArgs(_addr(h), _addr(b), _addr(gate), _addr(scale), _addr(shift), _addr(h_out), _addr(n),
                             _addr(codes), _addr(scales), M, seg, D, _STREAM[h.dtype], _NORM[post], _NORM[pre],
                             _CODES[quant], float(alpha), float(eps))
        _check(_launch(dev, lib.lg_block_norm, ctypes.byref(args)), "lg_block_norm")
    return (h if b is None else h_out), n, (q if quant is not None else None)


def block_norm_backward_workspace_size(M, D, segment_tokens):
    return int(lib.lg_block_norm_backward_workspace_size(int(M), int(D), int(segment_tokens)))


_backward_bytes = functools.lru_cache(4096)(block_norm_backward_workspace_size)


def block_norm_backward(dn, dh_out, h_out, b=None, gate=None, scale=None, alpha=1.0, eps=1e-6, post="rms", pre="rms",
                        segment_tokens=None, dh=None, db=None, workspace=None):
    """Gradients of block_norm: dn and dh_out are those of n (bf16; None without
    pre) and of h' (the stream's type; None for zero), h_out the h' that
    block_norm returned, the rest its arguments.  Returns (dh, db, dgate,
    dscale, dshift), the last three FP32 [S, D]; db and dgate are None without
    b, dscale and dshift without pre.  Without b post counts as in block_norm.
    dh may be dh_out itself."""
    if b is None and post == "rms":
        post = None
    M, D, seg, S = _norm_args(h_out, post, pre, segment_tokens)
    _modulation(gate, S, D, "gate")
    _modulation(scale, S, D, "scale")
    dev = h_out.device
    if (dn is None) != (pre is None):
        raise ValueError("dn is given exactly when there is a pre-norm")
    if dn is not None:
        _need(dn, torch.bfloat16, "dn", 2)
        _shape(dn, (M, D), "dn")
    if dh_out is not None:
        _need(dh_out, h_out.dtype, "dh_out", 2)
        _shape(dh_out, (M, D), "dh_out")
    if dh is None:
        dh = torch.empty_like(h_out)
    else:
        _need(dh, h_out.dtype, "dh", 2)
        _shape(dh, (M, D), "dh")
    dgate = dscale = dshift = None
    if b is not None:
        _need(b, torch.bfloat16, "b", 2)
        _shape(b, (M, D), "b")
        if db is None:
            db = torch.empty_like(b)
        else:
            _need(db, torch.bfloat16, "db", 2)
            _shape(db, (M, D), "db")
        dgate = h_out.new_empty((S, D), dtype=torch.float32)
    elif db is not None:
        raise ValueError("db needs b")
    if dn is not None:
        dscale = h_out.new_empty((S, D), dtype=torch.float32)
        dshift = h_out.new_empty((S, D), dtype=torch.float32)
    need = _backward_bytes(M, D, seg)
    if workspace is None and need > 0:
        workspace = h_out.new_empty(need, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _same_device(h_out, dn, dh_out, b, gate, scale, dh, db, workspace)
    if M > 0:
        args = BlockNormBackwardArgs(_addr(dn), _addr(dh_out), _addr(h_out), _addr(b), _addr(gate), _addr(scale),
                                     _addr(dh), _addr(db), _addr(dgate), _addr(dscale), _addr(dshift), M, seg, D,
                                     _STREAM[h_out.dtype], _NORM[post], _NORM[pre], float(alpha), float(eps))
        _check(_launch(dev, lib.lg_block_norm_backward, ctypes.byref(args), _addr(workspace), ws_bytes),
               "lg_block_norm_backward")
    return dh, db, dgate, dscale, dshift


def renoise(up, sigma, seed, offset=0, out=None):
    """x = (1 - sigma) up + sigma eps(seed, offset + i); FP32."""
    _need(up, torch.float32, "up")
    if out is None:
        out = torch.empty_like(up)
    _need(out, torch.float32, "out")
    if out.numel() != up.numel():
        raise ValueError("out must have as many elements as up")
    _same_device(up, out)
    with torch.cuda.device(up.device):
        st = lib.lg_renoise(_ptr(up), _ptr(out), up.numel(), float(sigma), int(seed), int(offset), _stream(up.device))
    _check(st, "lg_renoise")
    return out


def euler_step(x, v, sigma, sigma_next):
    """In place: x += (sigma_next - sigma) v; FP32."""
    _need(x, torch.float32, "x")
    _need(v, torch.float32, "v")
    if x.numel() != v.numel():
        raise ValueError("x and v must have the same number of elements")
    _same_device(x, v)
    with torch.cuda.device(x.device):
        st = lib.lg_euler_step(_ptr(x), _ptr(v), x.numel(), float(sigma), float(sigma_next), _stream(x.device))
    _check(st, "lg_euler_step")
    return x


# Routes of the IC sampler: printed start sigma on HyperFlow's eight-step,
# shift-12 table (page "Open-H3-Regenerate-2K-IC", section
# "三步接着放大的草稿画，八步从噪声重画").
IC_ROUTES = {"up3": 0.835, "up4": 0.923, "hf8": 1.0}


def shift_ladder(sigma0, n_steps=8, shift=12.0):
    """The FP32 sigmas a route visits: sigma0, then every point of the
    shift-`shift`, `n_steps`-step table below it (host computation)."""
    buf = (ctypes.c_float * (int(n_steps) + 2))()
    n = ctypes.c_int(0)
    st = lib.lg_shift_ladder(float(sigma0), int(n_steps), float(shift), buf, len(buf), ctypes.byref(n))
    _check(st, "lg_shift_ladder")
    return [float(buf[i]) for i in range(n.value)]


def philox_u32(n_blocks, seed, block_offset=0, out=None, device=None):
    """Raw Philox4x32-10 words, 4 per block, as an int32 tensor holding the uint32 bits."""
    if out is None:
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        out = torch.empty(4 * int(n_blocks), dtype=torch.int32, device=device)
    _need(out, torch.int32, "out")
    if out.numel() < 4 * n_blocks:
        raise ValueError("out too small")
    with torch.cuda.device(out.device):
        st = lib.lg_philox_u32(_ptr(out), int(n_blocks), int(seed), int(block_offset), _stream(out.device))
    _check(st, "lg_philox_u32")
    return out


def philox_normal(n, seed, offset=0, out=None, device=None):
    """eps[i] = element offset + i of the Box-Muller normal stream (FP32)."""
    if out is None:
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        out = torch.empty(int(n), dtype=torch.float32, device=device)
    _need(out, torch.float32, "out")
    if out.numel() < n:
        raise ValueError("out too small")
    with torch.cuda.device(out.device):
        st = lib.lg_philox_normal(_ptr(out), int(n), int(seed), int(offset), _stream(out.device))
    _check(st, "lg_philox_normal")
    return out
