"""Thin Python binding of the C ABI in include/w4a16.h (ctypes; argument marshalling only).

Each function has the name of the C entry point it calls. Tensors are torch CUDA tensors: the
binding passes their data pointers and the current CUDA stream and checks the returned status.
Every step of the layer runs in the CUDA library; there is no fallback of any kind: if
libw4a16.so is missing the first call raises.
"""
import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libw4a16.so")

OK = 0
EINVAL = -1
EALIGN = -2
EUNSUPPORTED = -3
ENONFINITE = -4
EWORKSPACE = -5
ECUDA = -6
ETIMEOUT = -7

F16 = 0
BF16 = 1
LAYOUT_PLAIN = 0
LAYOUT_TILED = 1
KERNEL_AUTO = 0
KERNEL_GEMV = 1
KERNEL_TC = 2

_DTYPES = {torch.float16: F16, torch.bfloat16: BF16}
_TORCH_DTYPES = {F16: torch.float16, BF16: torch.bfloat16}

_lib = None


class W4A16Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_str(status)} ({status})")


def lib():
    """The loaded ctypes library, with the argument types of include/w4a16.h."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"the W4A16 CUDA library is not built ({LIB_PATH} is missing); "
                           "run `python -m weight_only_int4_07_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.w4a16_quantize.argtypes = [P, I, I, I, I, P, P, P, P, P]
    L.w4a16_quantize.restype = I
    L.w4a16_dequantize.argtypes = [P, P, P, I, I, I, I, I, P, P]
    L.w4a16_dequantize.restype = I
    L.w4a16_gptq_workspace_bytes.argtypes = [I, I]
    L.w4a16_gptq_workspace_bytes.restype = S
    L.w4a16_gptq_quantize.argtypes = [P, P, I, I, I, I, I, I, ctypes.c_double, P, P, P, P, S, P, P]
    L.w4a16_gptq_quantize.restype = I
    L.w4a16_awq_workspace_bytes.argtypes = [I, I, I]
    L.w4a16_awq_workspace_bytes.restype = S
    L.w4a16_awq_quantize.argtypes = [P, P, I, I, I, I, I, I, P, P, P, P, P, S, P, P]
    L.w4a16_awq_quantize.restype = I
    L.w4a16_fp8_quantize_weights.argtypes = [P, I, I, P, P, P]
    L.w4a16_fp8_quantize_weights.restype = I
    L.w4a16_fp8_quantize_acts.argtypes = [P, I, I, I, P, P, P]
    L.w4a16_fp8_quantize_acts.restype = I
    L.w4a16_fp8_gemm.argtypes = [P, P, I, I, P, P, I, P, I, P, P]
    L.w4a16_fp8_gemm.restype = I
    L.w4a16_repack_bytes.argtypes = [I, I, I, I]
    L.w4a16_repack_bytes.restype = S
    L.w4a16_repack.argtypes = [P, P, P, I, I, I, I, P, P]
    L.w4a16_repack.restype = I
    L.w4a16_workspace_bytes.argtypes = [I, I, I, I]
    L.w4a16_workspace_bytes.restype = S
    L.w4a16_select_kernel.argtypes = [I, I, I, I]
    L.w4a16_select_kernel.restype = I
    L.w4a16_gemm.argtypes = [P, I, I, I, P, I, P, P, I, I, I, P, P, S, I, P, P]
    L.w4a16_gemm.restype = I
    L.w4a16_moe_sort_workspace_bytes.argtypes = [I, I, I]
    L.w4a16_moe_sort_workspace_bytes.restype = S
    L.w4a16_moe_sort.argtypes = [P, I, I, I, P, I, P, P, P, P, P, S, P]
    L.w4a16_moe_sort.restype = I
    L.w4a16_moe_sort_grad.argtypes = [P, I, I, I, I, P, P, P]
    L.w4a16_moe_sort_grad.restype = I
    L.w4a16_moe_combine.argtypes = [P, I, I, I, I, P, P, P, P]
    L.w4a16_moe_combine.restype = I
    L.w4a16_moe_combine_grad.argtypes = [P, P, I, I, I, I, P, P, P, P, P]
    L.w4a16_moe_combine_grad.restype = I
    L.w4a16_moe_workspace_bytes.argtypes = [I, I, I, I, I]
    L.w4a16_moe_workspace_bytes.restype = S
    L.w4a16_moe_gemm.argtypes = [P, I, I, I, P, I, P, I, I, I, P, P, S, I, P, P]
    L.w4a16_moe_gemm.restype = I
    L.w4a16_lora_workspace_bytes.argtypes = [I, I, I, I, I, I]
    L.w4a16_lora_workspace_bytes.restype = S
    L.w4a16_lora_gemm.argtypes = [P, I, I, I, P, I, I, I, P, P, P, I, I, P, P, P, S, P, P]
    L.w4a16_lora_gemm.restype = I
    L.w4a16_status_str.argtypes = [I]
    L.w4a16_status_str.restype = ctypes.c_char_p
    L.w4a16_version.argtypes = []
    L.w4a16_version.restype = I
    L.w4a16_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.w4a16_set_wait_limit_ns.restype = ctypes.c_uint64
    _lib = L
    return L


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(fn, status):
    if status != OK:
        raise W4A16Error(fn, status)


def status_str(status: int) -> str:
    return lib().w4a16_status_str(int(status)).decode()


w4a16_status_str = status_str


def w4a16_version() -> int:
    return int(lib().w4a16_version())


def w4a16_set_wait_limit_ns(ns: int) -> int:
    """Limit of every bounded device wait for later launches (0 = the 2 s default); returns the
    previous limit."""
    return int(lib().w4a16_set_wait_limit_ns(int(ns)))


def w4a16_quantize(W, group, sym, codes=None, scales=None, zeros=None, dev_status=None):
    """RTN group quantization of fp16 W [K, N] on the GPU -> (codes, scales, zeros)."""
    K, N = W.shape
    dev = W.device
    if codes is None:
        codes = torch.empty((K // 8, N), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((K // group, N), dtype=torch.float16, device=dev)
    if zeros is None and not sym:
        zeros = torch.empty((K // group, N // 8), dtype=torch.int32, device=dev)
    st = lib().w4a16_quantize(_ptr(W), K, N, group, int(sym), _ptr(codes), _ptr(scales),
                              _ptr(zeros), _ptr(dev_status), _stream())
    _check("w4a16_quantize", st)
    return codes, scales, (None if sym else zeros)


def w4a16_gptq_workspace_bytes(K, N) -> int:
    return int(lib().w4a16_gptq_workspace_bytes(K, N))


def w4a16_gptq_quantize(W, X, group, sym, damp=0.01, codes=None, scales=None, zeros=None,
                        workspace=None, dev_status=None):
    """GPTQ of fp16 W [K, N] with 16-bit calibration inputs X [S, K] on the GPU -> (codes,
    scales, zeros) in the plain packed format."""
    K, N = W.shape
    S = X.shape[0]
    dev = W.device
    if codes is None:
        codes = torch.empty((K // 8, N), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((K // group, N), dtype=torch.float16, device=dev)
    if zeros is None and not sym:
        zeros = torch.empty((K // group, N // 8), dtype=torch.int32, device=dev)
    nbytes = w4a16_gptq_workspace_bytes(K, N)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = lib().w4a16_gptq_quantize(_ptr(W), _ptr(X), _DTYPES[X.dtype], S, K, N, group, int(sym),
                                   float(damp), _ptr(codes), _ptr(scales), _ptr(zeros),
                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _ptr(dev_status), _stream())
    _check("w4a16_gptq_quantize", st)
    return codes, scales, (None if sym else zeros)


def w4a16_awq_workspace_bytes(K, N, S) -> int:
    return int(lib().w4a16_awq_workspace_bytes(K, N, S))


def w4a16_awq_quantize(W, X, group, sym, codes=None, scales=None, zeros=None, s_in=None,
                       workspace=None, dev_status=None):
    """AWQ of fp16 W [K, N] with 16-bit calibration inputs X [S, K] on the GPU -> (codes, scales,
    zeros, s_in): the packed S W and the fp16 factors that divide the layer's input."""
    K, N = W.shape
    S = X.shape[0]
    dev = W.device
    if codes is None:
        codes = torch.empty((K // 8, N), dtype=torch.int32, device=dev)
    if scales is None:
        scales = torch.empty((K // group, N), dtype=torch.float16, device=dev)
    if zeros is None and not sym:
        zeros = torch.empty((K // group, N // 8), dtype=torch.int32, device=dev)
    if s_in is None:
        s_in = torch.empty(K, dtype=torch.float16, device=dev)
    nbytes = w4a16_awq_workspace_bytes(K, N, S)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    st = lib().w4a16_awq_quantize(_ptr(W), _ptr(X), _DTYPES[X.dtype], S, K, N, group, int(sym),
                                  _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(s_in), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                  _stream())
    _check("w4a16_awq_quantize", st)
    return codes, scales, (None if sym else zeros), s_in


def w4a16_fp8_quantize_weights(W):
    """fp16 W [K, N] -> (Wq uint8 [N, K] E4M3 codes, w_scales float32 [N]) on the GPU."""
    K, N = W.shape
    Wq = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    sw = torch.empty(N, dtype=torch.float32, device=W.device)
    _check("w4a16_fp8_quantize_weights",
           lib().w4a16_fp8_quantize_weights(_ptr(W), K, N, _ptr(Wq), _ptr(sw), _stream()))
    return Wq, sw


def w4a16_fp8_quantize_acts(A, Aq=None, sa=None):
    """16-bit A [M, K] -> (Aq uint8 [M, K] E4M3 codes, a_scales float32 [M]) on the GPU."""
    M, K = A.shape
    if Aq is None:
        Aq = torch.empty((M, K), dtype=torch.uint8, device=A.device)
    if sa is None:
        sa = torch.empty(M, dtype=torch.float32, device=A.device)
    _check("w4a16_fp8_quantize_acts",
           lib().w4a16_fp8_quantize_acts(_ptr(A), _DTYPES[A.dtype], M, K, _ptr(Aq), _ptr(sa), _stream()))
    return Aq, sa


def w4a16_fp8_gemm(Aq, sa, Wq, sw, dtype=None, C=None, dev_status=None):
    """C[M, N] = (Aq . Wq^T) * sa[m] * sw[n], FP32 accumulation, C in `dtype` (fp16 default)."""
    M, K = Aq.shape
    N = Wq.shape[0]
    if C is None:
        C = torch.empty((M, N), dtype=torch.float16 if dtype is None else dtype, device=Aq.device)
    _check("w4a16_fp8_gemm", lib().w4a16_fp8_gemm(_ptr(Aq), _ptr(sa), M, K, _ptr(Wq), _ptr(sw), N, _ptr(C),
                                                  _DTYPES[C.dtype], _ptr(dev_status), _stream()))
    return C


def w4a16_dequantize(codes, scales, zeros, K, N, group, sym, dtype=None, out=None):
    """The packed weight as a 16-bit [K, N] matrix, (q - z) * s rounded once (the naive path)."""
    dtype = torch.float16 if dtype is None else dtype
    if out is None:
        out = torch.empty((K, N), dtype=dtype, device=codes.device)
    st = lib().w4a16_dequantize(_ptr(codes), _ptr(scales), _ptr(zeros), K, N, group, int(sym),
                                _DTYPES[out.dtype], _ptr(out), _stream())
    _check("w4a16_dequantize", st)
    return out


def w4a16_repack_bytes(K, N, group, sym) -> int:
    return int(lib().w4a16_repack_bytes(K, N, group, int(sym)))


def w4a16_repack(codes, scales, zeros, K, N, group, sym, out=None):
    """Plain packed weight -> one tiled uint8 buffer (see the header for the layout)."""
    nbytes = w4a16_repack_bytes(K, N, group, sym)
    if nbytes == 0:
        _check("w4a16_repack", EUNSUPPORTED)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    st = lib().w4a16_repack(_ptr(codes), _ptr(scales), _ptr(zeros), K, N, group, int(sym),
                            _ptr(out), _stream())
    _check("w4a16_repack", st)
    return out


def w4a16_workspace_bytes(M, N, K, group) -> int:
    return int(lib().w4a16_workspace_bytes(M, N, K, group))


def w4a16_select_kernel(M, N, K, group) -> int:
    return int(lib().w4a16_select_kernel(M, N, K, group))


def w4a16_gemm(A, wq, scales, zeros, N, group, sym, layout=LAYOUT_PLAIN, C=None, workspace=None,
               kernel=KERNEL_AUTO, dev_status=None):
    """C[M, N] = A[M, K] . dequant(W) with FP32 accumulation; C in the dtype of A."""
    M, K = A.shape
    a_dtype = _DTYPES[A.dtype]
    if C is None:
        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    need = w4a16_workspace_bytes(M, N, K, group)
    if workspace is None and need > 0:
        # the tile counters at the front of a workspace must start at zero
        workspace = torch.zeros(need, dtype=torch.uint8, device=A.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().w4a16_gemm(_ptr(A), a_dtype, M, K, _ptr(wq), int(layout), _ptr(scales), _ptr(zeros),
                          N, group, int(sym), _ptr(C), _ptr(workspace), ws_bytes, int(kernel),
                          _ptr(dev_status), _stream())
    _check("w4a16_gemm", st)
    return C


_noalloc_ready = False


def w4a16_gemm_noalloc(A, codes, scales, zeros, N, group, sym, C=None):
    """C[M, N] = A[M, K] . dequant(W) for callers that cannot allocate device memory: the split-K
    partial sums live in the library's static scratch (see include/w4a16.h for its limit and
    for why calls that overlap on the GPU race)."""
    global _noalloc_ready
    L = lib()
    if not _noalloc_ready:
        P, I = ctypes.c_void_p, ctypes.c_int
        L.w4a16_gemm_noalloc.argtypes = [P, I, I, I, P, P, P, I, I, I, P, P]
        L.w4a16_gemm_noalloc.restype = I
        _noalloc_ready = True
    M, K = A.shape
    if C is None:
        C = torch.empty((M, N), dtype=A.dtype, device=A.device)
    st = L.w4a16_gemm_noalloc(_ptr(A), _DTYPES[A.dtype], M, K, _ptr(codes), _ptr(scales), _ptr(zeros),
                              N, group, int(sym), _ptr(C), _stream())
    _check("w4a16_gemm_noalloc", st)
    return C


# ----------------------------------------------------------------------------- routed layers
_calls = {}


def _need(fn, ok):
    if not ok:
        raise W4A16Error(fn, EINVAL)


def _arg(fn, t, dtype, shape, dev):
    """The address of a contiguous CUDA tensor of this type and shape on device `dev` (its index)."""
    _need(fn, t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev)
    return t.data_ptr()


def _out(fn, t, dtype, shape, dev):
    """`t`, checked, or a new tensor of this type and shape."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    _arg(fn, t, dtype, shape, dev)
    return t


def _room(fn, t, nbytes, dev, zeroed=False):
    """A caller's workspace, checked, or a new one."""
    if t is None:
        make = torch.zeros if zeroed else torch.empty
        return make(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
    _need(fn, t.is_contiguous() and t.get_device() == dev)
    return t


def _call(name, dev, *args):
    """One entry point on the current stream of device `dev`, with that device current. (The stream and
    the device come from the functions below torch.cuda's own: building a Python stream object is 3 us
    of a small call.)"""
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(lib(), name)
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        st = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, stream)
    if st != OK:
        raise W4A16Error(name, st)


def _status_arg(fn, t, dev):
    return None if t is None else _arg(fn, t, torch.int32, t.shape, dev)


def _dev(fn, t):
    _need(fn, t.is_cuda)
    return t.get_device()


def w4a16_moe_sort_workspace_bytes(T, k, n_experts) -> int:
    return int(lib().w4a16_moe_sort_workspace_bytes(T, k, n_experts))


def w4a16_moe_sort(ids, n_experts, X=None, offsets=None, rows=None, slots=None, Xs=None, workspace=None):
    """Tokens sorted by expert: ids int32 [T, k] (and the tokens' 16-bit rows X [T, H]) ->
    (offsets [E + 1], rows [T k], slots [T, k], Xs [T k, H] or None). Entries of `rows` and rows of
    `Xs` at or past offsets[E] are left as they were."""
    fn = "w4a16_moe_sort"
    dev = _dev(fn, ids)
    _need(fn, ids.dim() == 2)
    T, k = ids.shape
    _need(fn, T > 0 and k > 0 and n_experts > 0 and (X is not None or Xs is None))
    i32 = torch.int32
    p = _arg(fn, ids, i32, (T, k), dev)
    offsets = _out(fn, offsets, i32, (n_experts + 1,), dev)
    rows = _out(fn, rows, i32, (T * k,), dev)
    slots = _out(fn, slots, i32, (T, k), dev)
    H = 0
    if X is not None:
        _need(fn, X.dim() == 2 and X.dtype in _DTYPES)
        H = X.shape[1]
        px = _arg(fn, X, X.dtype, (T, H), dev)
        Xs = _out(fn, Xs, X.dtype, (T * k, H), dev)
    need = w4a16_moe_sort_workspace_bytes(T, k, n_experts)
    pw, nb = None, 0
    if need > 0:
        workspace = _room(fn, workspace, need, dev)
        pw, nb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(fn, dev, p, T, k, n_experts, px if H else None, H, offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(),
          Xs.data_ptr() if H else None, pw, nb)
    return offsets, rows, slots, Xs


def _sum_rows(fn, Ys, slots, weights, Y):
    dev = _dev(fn, Ys)
    _need(fn, slots.dim() == 2 and Ys.dim() == 2 and Ys.dtype in _DTYPES)
    (T, k), H, t = slots.shape, Ys.shape[1], Ys.dtype
    ps = _arg(fn, slots, torch.int32, (T, k), dev)
    py = _arg(fn, Ys, t, (T * k, H), dev)
    Y = _out(fn, Y, t, (T, H), dev)
    if fn == "w4a16_moe_sort_grad":
        _call(fn, dev, py, _DTYPES[t], T, k, H, ps, Y.data_ptr())
    else:
        pw = None if weights is None else _arg(fn, weights, torch.float32, (T, k), dev)
        _call(fn, dev, py, _DTYPES[t], T, k, H, ps, pw, Y.data_ptr())
    return Y


def w4a16_moe_combine(Ys, slots, weights=None, Y=None):
    """Y[t] = sum_j weights[t, j] Ys[slots[t, j]] for 16-bit sorted rows Ys [T k, H], slots int32
    [T, k] and fp32 weights [T, k] (None: all 1); FP32 sums, Y [T, H] in the type of Ys."""
    return _sum_rows("w4a16_moe_combine", Ys, slots, weights, Y)


def w4a16_moe_sort_grad(dXs, slots, dX=None):
    """The gradient of w4a16_moe_sort's gather: dX[t] = sum_j dXs[slots[t, j]]."""
    return _sum_rows("w4a16_moe_sort_grad", dXs, slots, None, dX)


def w4a16_moe_combine_grad(dY, Ys, slots, weights=None, dYs=None, dweights=None):
    """The gradient of w4a16_moe_combine -> (dYs [T k, H], dweights fp32 [T, k]); Ys None: dYs
    alone (dweights None). Rows of dYs without a choice are left as they were."""
    fn = "w4a16_moe_combine_grad"
    dev = _dev(fn, dY)
    _need(fn, slots.dim() == 2 and dY.dim() == 2 and dY.dtype in _DTYPES and (Ys is not None or dweights is None))
    (T, k), H, t = slots.shape, dY.shape[1], dY.dtype
    ps = _arg(fn, slots, torch.int32, (T, k), dev)
    pg = _arg(fn, dY, t, (T, H), dev)
    pw = None if weights is None else _arg(fn, weights, torch.float32, (T, k), dev)
    dYs = _out(fn, dYs, t, (T * k, H), dev)
    py = None
    if Ys is not None:
        py = _arg(fn, Ys, t, (T * k, H), dev)
        dweights = _out(fn, dweights, torch.float32, (T, k), dev)
    _call(fn, dev, pg, py, _DTYPES[t], T, k, H, ps, pw, dYs.data_ptr(),
          None if dweights is None else dweights.data_ptr())
    return dYs, dweights


def w4a16_moe_workspace_bytes(R, n_experts, N, K, group) -> int:
    return int(lib().w4a16_moe_workspace_bytes(R, n_experts, N, K, group))


def w4a16_moe_gemm(A, offsets, tiled, N, group, sym, C=None, workspace=None, kernel=KERNEL_AUTO, dev_status=None):
    """C[i] = A[i] . dequant(W_e), offsets[e] <= i < offsets[e + 1], for 16-bit sorted rows A [R, K],
    int32 offsets [E + 1] and uint8 tiled [E, w4a16_repack_bytes(K, N, group, sym)]. Rows of C outside
    every run are left as they were. A workspace may be kept: zeros at first, one per stream."""
    fn = "w4a16_moe_gemm"
    dev = _dev(fn, A)
    _need(fn, A.dim() == 2 and A.dtype in _DTYPES and offsets.dim() == 1)
    (R, K), E, t = A.shape, offsets.shape[0] - 1, A.dtype
    pa = _arg(fn, A, t, (R, K), dev)
    po = _arg(fn, offsets, torch.int32, (E + 1,), dev)
    pw = _arg(fn, tiled, torch.uint8, (E, w4a16_repack_bytes(K, N, group, sym)), dev)
    C = _out(fn, C, t, (R, N), dev)
    if workspace is None:
        with torch.cuda.device(dev):   # (the size goes by the device)
            workspace = _room(fn, None, w4a16_moe_workspace_bytes(R, E, N, K, group), dev, zeroed=True)
    _call(fn, dev, pa, _DTYPES[t], R, K, pw, E, po, N, group, int(sym), C.data_ptr(),
          _room(fn, workspace, 0, dev).data_ptr(), workspace.numel() * workspace.element_size(), int(kernel),
          _status_arg(fn, dev_status, dev))
    return C


def w4a16_lora_workspace_bytes(M, N, K, group, rank, adapters) -> int:
    return int(lib().w4a16_lora_workspace_bytes(M, N, K, group, rank, adapters))


def w4a16_lora_gemm(A, tiled, N, group, sym, lora_a, lora_b, lora_scale, row_adapter, C=None, workspace=None,
                    dev_status=None):
    """C[m] = A[m] . dequant(W) + lora_scale[a] (A[m] . lora_a[a]^T) . lora_b[a]^T, a = row_adapter[m]
    (outside [0, L): the first term alone). 16-bit A [M, K], lora_a [L, r, K], lora_b [L, N, r] of one
    type, tiled uint8 (w4a16_repack), lora_scale fp32 [L], row_adapter int32 [M]; FP32 sums, rounded once.
    A workspace may be kept: zeros at first, one per stream."""
    fn = "w4a16_lora_gemm"
    dev = _dev(fn, A)
    _need(fn, A.dim() == 2 and A.dtype in _DTYPES and lora_a.dim() == 3)
    (M, K), (L, r, _), t = A.shape, lora_a.shape, A.dtype
    pa = _arg(fn, A, t, (M, K), dev)
    pw = _arg(fn, tiled, torch.uint8, (w4a16_repack_bytes(K, N, group, sym),), dev)
    pla = _arg(fn, lora_a, t, (L, r, K), dev)
    plb = _arg(fn, lora_b, t, (L, N, r), dev)
    ps = _arg(fn, lora_scale, torch.float32, (L,), dev)
    pr = _arg(fn, row_adapter, torch.int32, (M,), dev)
    C = _out(fn, C, t, (M, N), dev)
    if workspace is None:
        with torch.cuda.device(dev):   # (the size goes by the device)
            workspace = _room(fn, None, w4a16_lora_workspace_bytes(M, N, K, group, r, L), dev, zeroed=True)
    _call(fn, dev, pa, _DTYPES[t], M, K, pw, N, group, int(sym), pla, plb, ps, L, r, pr, C.data_ptr(),
          _room(fn, workspace, 0, dev).data_ptr(), workspace.numel() * workspace.element_size(),
          _status_arg(fn, dev_status, dev))
    return C
