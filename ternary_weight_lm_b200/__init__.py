"""Python binding of libmmf.so, the B200 FusedBitLinear library.

Argument marshalling only: every step of the projection runs in the library's CUDA kernels.
PyTorch supplies device memory (``tensor.data_ptr()``) and streams
(``torch.cuda.current_stream().cuda_stream``).  There is no CPU path: if the library or a GPU
is missing, calls raise.

The functions named ``mmf_*`` mirror the C ABI in ``include/mmf.h`` one to one and take
tensors that the caller owns.  ``quantize_weights``, ``bitlinear_forward``,
``bitlinear_glu_forward``, ``mlgru_forward``, ``bitlinear_backward``, ``quantize_weights_int8``,
``int8_matmul``, ``int8_linear_forward``, ``linattn_forward``, ``linattn_step`` and
``linattn_backward`` are conveniences that allocate the outputs and the workspace with torch and
then call the same entry points.
"""
import ctypes
import os

__all__ = [
    "MMFError", "lib", "lib_path",
    "mmf_quantize_weights_workspace_bytes", "mmf_quantize_weights", "mmf_ternary_encode",
    "mmf_forward_workspace_bytes", "mmf_bitlinear_forward", "mmf_bitlinear_glu_forward",
    "mmf_quantize_activations", "mmf_quantized_workspace_bytes",
    "mmf_bitlinear_forward_quantized",
    "mmf_ternary_accumulate_i32", "mmf_bitlinear_forward_noalloc", "mmf_get_device_status",
    "mmf_debug_wait_timeout_probe", "mmf_status_string", "mmf_version",
    "mmf_program_workspace_bytes", "mmf_program_init", "mmf_program_run", "Projection",
    "Program", "quantize_weights", "bitlinear_forward", "bitlinear_glu_forward", "workspace",
    "mmf_mlgru_workspace_bytes", "mmf_mlgru_forward", "mmf_mlgru_forward_quantized",
    "mlgru_forward", "mmf_backward_workspace_bytes", "mmf_bitlinear_backward",
    "bitlinear_backward", "mmf_int8_quantize_weights", "mmf_int8_forward_quantized",
    "mmf_int8_workspace_bytes", "mmf_int8_forward", "quantize_weights_int8", "int8_matmul",
    "int8_linear_forward", "LinattnDesc", "mmf_linattn_workspace_bytes",
    "mmf_linattn_backward_workspace_bytes", "mmf_linattn_forward", "mmf_linattn_backward",
    "mmf_linattn_step", "linattn_forward", "linattn_step", "linattn_backward",
    "MMF_F32", "MMF_F16", "STATUS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libmmf.so")

MMF_F32 = 0
MMF_F16 = 1
STATUS = {
    0: "MMF_OK", 1: "MMF_ERR_INVALID_ARG", 2: "MMF_ERR_UNSUPPORTED_SHAPE",
    3: "MMF_ERR_ALIGNMENT", 4: "MMF_ERR_CUDA", 5: "MMF_ERR_TIMEOUT", 6: "MMF_ERR_WORKSPACE",
    7: "MMF_ERR_RESOURCES", 8: "MMF_ERR_PLAN",
}


class MMFError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")
        self.code = code


class Projection(ctypes.Structure):
    """Mirror of the C struct mmf_projection (one FusedBitLinear of a program)."""
    _fields_ = [("x", ctypes.c_void_p), ("xdt", ctypes.c_int), ("norm_w", ctypes.c_void_p),
                ("Wp", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("K", ctypes.c_int64),
                ("N", ctypes.c_int64), ("glu", ctypes.c_int32), ("level", ctypes.c_int32),
                ("y", ctypes.c_void_p), ("ydt", ctypes.c_int)]


class LinattnDesc(ctypes.Structure):
    """Mirror of the C struct mmf_linattn_desc (sizes and strides of a linear attention call)."""
    _fields_ = [("T", ctypes.c_int64), ("B", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p),
                ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("dt", ctypes.c_int), ("scale", ctypes.c_float), ("clear_outside", ctypes.c_int32),
                ("log_decay", ctypes.c_void_p),
                ("q_t", ctypes.c_int64), ("q_h", ctypes.c_int64), ("k_t", ctypes.c_int64),
                ("k_h", ctypes.c_int64), ("v_t", ctypes.c_int64), ("v_h", ctypes.c_int64),
                ("o_t", ctypes.c_int64), ("o_h", ctypes.c_int64)]


_lib = None


def lib():
    """Load libmmf.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise OSError(f"{lib_path} is missing: run ternary_weight_lm_b200/build.py")
        L = ctypes.CDLL(lib_path)
        P, I64, F, SZ, I = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t,
                            ctypes.c_int)
        sigs = {
            "mmf_quantize_weights_workspace_bytes": ([I64, I64], SZ),
            "mmf_quantize_weights": ([P, I, I64, I64, P, P, P, SZ, P], I),
            "mmf_ternary_encode": ([P, I, I64, I64, P, P, P], I),
            "mmf_forward_workspace_bytes": ([I64, I64, I64], SZ),
            "mmf_bitlinear_forward": ([P, I, I64, I64, P, F, P, P, I64, P, I, P, SZ, P], I),
            "mmf_bitlinear_glu_forward": ([P, I, I64, I64, P, F, P, P, I64, P, I, P, SZ, P], I),
            "mmf_quantize_activations": ([P, I, I64, I64, P, F, P, P, P, P], I),
            "mmf_quantized_workspace_bytes": ([I64, I64, I64], SZ),
            "mmf_bitlinear_forward_quantized": ([P, P, P, I64, I64, P, P, I64, I, P, I, P, SZ, P],
                                                I),
            "mmf_ternary_accumulate_i32": ([P, I64, I64, P, I64, P, P, SZ, P], I),
            "mmf_bitlinear_forward_noalloc": ([P, I, I64, I64, P, F, P, P, I64, P, I, P], I),
            "mmf_backward_workspace_bytes": ([I64, I64, I64], SZ),
            "mmf_bitlinear_backward": ([P, I, I64, I64, P, F, P, P, P, P, I64, P, P, I, P, P, P,
                                        SZ, P], I),
            "mmf_mlgru_workspace_bytes": ([I64, I64], SZ),
            "mmf_mlgru_forward": ([P, P, P, I, I64, I64, P, P, F, P, I, P, P, SZ, P], I),
            "mmf_mlgru_forward_quantized": ([P, P, P, I, I64, I64, P, P, F, P, F, P, P, P, P, P,
                                             SZ, P], I),
            "mmf_int8_quantize_weights": ([P, I, I64, I64, P, P, P], I),
            "mmf_int8_forward_quantized": ([P, P, I64, I64, P, P, I64, P, I, P], I),
            "mmf_int8_workspace_bytes": ([I64, I64], SZ),
            "mmf_int8_forward": ([P, I, I64, I64, P, F, P, P, I64, P, I, P, SZ, P], I),
            "mmf_linattn_workspace_bytes": ([P], SZ),
            "mmf_linattn_backward_workspace_bytes": ([P], SZ),
            "mmf_linattn_forward": ([P, P, P, P, P, P, P, P, SZ, P], I),
            "mmf_linattn_backward": ([P, P, P, P, P, P, P, P, P, P, P, P, SZ, P], I),
            "mmf_linattn_step": ([P, P, P, P, P, P, P, I64, P], I),
            "mmf_program_workspace_bytes": ([P, I, I64], SZ),
            "mmf_program_init": ([P, I, I64, F, P, SZ, P], I),
            "mmf_program_run": ([P, P], I),
            "mmf_get_device_status": ([], I),
            "mmf_debug_wait_timeout_probe": ([ctypes.c_uint64, P], I),
            "mmf_status_string": ([I], ctypes.c_char_p),
            "mmf_version": ([], I),
        }
        for name, (args, res) in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


# ------------------------------------------------------------------------------ marshalling
def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _dt(t):
    import torch
    if t.dtype == torch.float32:
        return MMF_F32
    if t.dtype == torch.float16:
        return MMF_F16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, code):
    if code != 0:
        raise MMFError(fn, code)


def _nbytes(t):
    return t.numel() * t.element_size()


# ------------------------------------------------------------------------------ C ABI mirror
def mmf_quantize_weights_workspace_bytes(N, K):
    return lib().mmf_quantize_weights_workspace_bytes(N, K)


def mmf_quantize_weights(W, Wp, beta, ws, stream=None):
    N, K = W.shape
    _check("mmf_quantize_weights", lib().mmf_quantize_weights(
        _ptr(W), _dt(W), N, K, _ptr(Wp), _ptr(beta), _ptr(ws), _nbytes(ws), _stream(stream)))


def mmf_ternary_encode(W, beta, Wp, stream=None):
    N, K = W.shape
    _check("mmf_ternary_encode", lib().mmf_ternary_encode(
        _ptr(W), _dt(W), N, K, _ptr(beta), _ptr(Wp), _stream(stream)))


def mmf_forward_workspace_bytes(T, K, N):
    return lib().mmf_forward_workspace_bytes(T, K, N)


def mmf_bitlinear_forward(x, norm_w, eps, Wp, beta, N, y, ws, stream=None):
    T, K = x.shape
    _check("mmf_bitlinear_forward", lib().mmf_bitlinear_forward(
        _ptr(x), _dt(x), T, K, _ptr(norm_w), float(eps), _ptr(Wp), _ptr(beta), N, _ptr(y),
        _dt(y), _ptr(ws), _nbytes(ws), _stream(stream)))


def mmf_bitlinear_glu_forward(x, norm_w, eps, Wp, beta, N2, h, ws, stream=None):
    T, K = x.shape
    _check("mmf_bitlinear_glu_forward", lib().mmf_bitlinear_glu_forward(
        _ptr(x), _dt(x), T, K, _ptr(norm_w), float(eps), _ptr(Wp), _ptr(beta), N2, _ptr(h),
        _dt(h), _ptr(ws), _nbytes(ws), _stream(stream)))


def mmf_quantize_activations(x, norm_w, eps, A, gamma, rowsum=None, stream=None):
    T, K = x.shape
    _check("mmf_quantize_activations", lib().mmf_quantize_activations(
        _ptr(x), _dt(x), T, K, _ptr(norm_w), float(eps), _ptr(A), _ptr(gamma), _ptr(rowsum),
        _stream(stream)))


def mmf_quantized_workspace_bytes(T, K, N):
    return lib().mmf_quantized_workspace_bytes(T, K, N)


def mmf_bitlinear_forward_quantized(A, gamma, rowsum, Wp, beta, N, glu, y, ws=None,
                                    stream=None):
    """ws: None (the contraction that needs no workspace) or a tensor of at least
    mmf_quantized_workspace_bytes(T, K, N) bytes."""
    T, K = A.shape
    _check("mmf_bitlinear_forward_quantized", lib().mmf_bitlinear_forward_quantized(
        _ptr(A), _ptr(gamma), _ptr(rowsum), T, K, _ptr(Wp), _ptr(beta), N, 1 if glu else 0,
        _ptr(y), _dt(y), _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def mmf_ternary_accumulate_i32(A, Wp, N, acc, ws, stream=None):
    T, K = A.shape
    _check("mmf_ternary_accumulate_i32", lib().mmf_ternary_accumulate_i32(
        _ptr(A), T, K, _ptr(Wp), N, _ptr(acc), _ptr(ws), _nbytes(ws), _stream(stream)))


def mmf_bitlinear_forward_noalloc(x, norm_w, eps, Wp, beta, N, y, stream=None):
    """Forward without a workspace argument: for callers that cannot allocate device memory.
    Scratch is a fixed 4 MiB device array shared by all calls (see include/mmf.h)."""
    T, K = x.shape
    _check("mmf_bitlinear_forward_noalloc", lib().mmf_bitlinear_forward_noalloc(
        _ptr(x), _dt(x), T, K, _ptr(norm_w), float(eps), _ptr(Wp), _ptr(beta), N, _ptr(y),
        _dt(y), _stream(stream)))


def mmf_backward_workspace_bytes(T, K, N):
    return lib().mmf_backward_workspace_bytes(T, K, N)


def mmf_bitlinear_backward(x, norm_w, eps, A, gamma, Wp, beta, N, dy, dx, dW, dnorm_w, ws,
                           stream=None):
    """Straight-through backward (include/mmf.h).  A/gamma: the forward's codes and scales or
    both None; dx, dW, dnorm_w: outputs or None (dx's dtype selects dxdt)."""
    T, K = x.shape
    _check("mmf_bitlinear_backward", lib().mmf_bitlinear_backward(
        _ptr(x), _dt(x), T, K, _ptr(norm_w), float(eps), _ptr(A), _ptr(gamma), _ptr(Wp),
        _ptr(beta), N, _ptr(dy), _ptr(dx), MMF_F32 if dx is None else _dt(dx), _ptr(dW),
        _ptr(dnorm_w), _ptr(ws), _nbytes(ws), _stream(stream)))


def mmf_mlgru_workspace_bytes(T, H):
    return lib().mmf_mlgru_workspace_bytes(T, H)


def _ws(ws):
    return (None, 0) if ws is None else (_ptr(ws), _nbytes(ws))


def mmf_mlgru_forward(I, F, G, h0, norm_w, eps, o, hT=None, ws=None, stream=None):
    """MLGRU recurrence + swish gate norm (include/mmf.h): o [T, H] from I, F, G [T, H]."""
    T, H = I.shape
    wp, wn = _ws(ws)
    _check("mmf_mlgru_forward", lib().mmf_mlgru_forward(
        _ptr(I), _ptr(F), _ptr(G), _dt(I), T, H, _ptr(h0), _ptr(norm_w), float(eps), _ptr(o),
        _dt(o), _ptr(hT), wp, wn, _stream(stream)))


def mmf_mlgru_forward_quantized(I, F, G, h0, norm_w, eps, oproj_norm_w, oproj_eps, A, gamma,
                                rowsum=None, hT=None, ws=None, stream=None):
    """The same, writing o_proj's int8 codes, gamma and code sums instead of o."""
    T, H = I.shape
    wp, wn = _ws(ws)
    _check("mmf_mlgru_forward_quantized", lib().mmf_mlgru_forward_quantized(
        _ptr(I), _ptr(F), _ptr(G), _dt(I), T, H, _ptr(h0), _ptr(norm_w), float(eps),
        _ptr(oproj_norm_w), float(oproj_eps), _ptr(A), _ptr(gamma), _ptr(rowsum), _ptr(hT), wp,
        wn, _stream(stream)))


def mmf_int8_quantize_weights(W, W8, wscale, stream=None):
    """W [N, K] -> int8 codes W8 [N, K] and one scale for each row (include/mmf.h)."""
    N, K = W.shape
    _check("mmf_int8_quantize_weights", lib().mmf_int8_quantize_weights(
        _ptr(W), _dt(W), N, K, _ptr(W8), _ptr(wscale), _stream(stream)))


def mmf_int8_forward_quantized(A, gamma, W8, wscale, y, stream=None):
    """y [T, N] from activation codes A [T, K], gamma [T] and 8-bit weights."""
    T, K = A.shape
    _check("mmf_int8_forward_quantized", lib().mmf_int8_forward_quantized(
        _ptr(A), _ptr(gamma), T, K, _ptr(W8), _ptr(wscale), W8.shape[0], _ptr(y), _dt(y),
        _stream(stream)))


def mmf_int8_workspace_bytes(T, K):
    return lib().mmf_int8_workspace_bytes(T, K)


def mmf_int8_forward(x, norm_w, eps, W8, wscale, y, ws, stream=None):
    T, K = x.shape
    _check("mmf_int8_forward", lib().mmf_int8_forward(
        _ptr(x), _dt(x), T, K, _ptr(norm_w), float(eps), _ptr(W8), _ptr(wscale), W8.shape[0],
        _ptr(y), _dt(y), _ptr(ws), _nbytes(ws), _stream(stream)))


def mmf_linattn_workspace_bytes(desc):
    return lib().mmf_linattn_workspace_bytes(ctypes.byref(desc))


def mmf_linattn_backward_workspace_bytes(desc):
    return lib().mmf_linattn_backward_workspace_bytes(ctypes.byref(desc))


def mmf_linattn_forward(desc, q, k, v, h0, o, hT=None, ws=None, stream=None):
    """Linear attention over whole prompts (include/mmf.h); desc: a LinattnDesc."""
    wp, wn = _ws(ws)
    _check("mmf_linattn_forward", lib().mmf_linattn_forward(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(h0), _ptr(o), _ptr(hT), wp, wn,
        _stream(stream)))


def mmf_linattn_backward(desc, q, k, v, dout, h0, dhT, dq, dk, dv, dh0=None, ws=None,
                         stream=None):
    wp, wn = _ws(ws)
    _check("mmf_linattn_backward", lib().mmf_linattn_backward(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(h0), _ptr(dhT), _ptr(dq),
        _ptr(dk), _ptr(dv), _ptr(dh0), wp, wn, _stream(stream)))


def mmf_linattn_step(desc, q, k, v, o, state, slots=None, stream=None):
    """One token of each sequence; state is updated in place."""
    n = 0 if slots is None else state.shape[0]
    _check("mmf_linattn_step", lib().mmf_linattn_step(
        ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(state), _ptr(slots), n,
        _stream(stream)))


def _proj_array(projs):
    arr = (Projection * len(projs))()
    for i, p in enumerate(projs):
        x, norm_w, Wp, beta, y, glu, level = (p["x"], p.get("norm_w"), p["Wp"], p["beta"], p["y"],
                                              p.get("glu", False), p.get("level", 0))
        arr[i] = Projection(_ptr(x), _dt(x), _ptr(norm_w), _ptr(Wp), _ptr(beta), x.shape[1],
                            Wp.shape[0], 1 if glu else 0, level, _ptr(y), _dt(y))
    return arr


def mmf_program_workspace_bytes(projs, T):
    arr = _proj_array(projs)
    return lib().mmf_program_workspace_bytes(arr, len(projs), T)


def mmf_program_init(projs, T, eps, ws, stream=None):
    arr = _proj_array(projs)
    _check("mmf_program_init", lib().mmf_program_init(arr, len(projs), T, float(eps), _ptr(ws),
                                                      _nbytes(ws), _stream(stream)))


def mmf_program_run(ws, stream=None):
    _check("mmf_program_run", lib().mmf_program_run(_ptr(ws), _stream(stream)))


class Program:
    """A planned list of projections run as one launch (see mmf_program_init).

    ``projs`` is a list of dicts with keys x, Wp, beta, y and optionally norm_w, glu, level;
    the tensors must stay alive and in place for as long as the program is run."""

    def __init__(self, projs, T, eps=1e-8, stream=None):
        n = mmf_program_workspace_bytes(projs, T)
        if n == 0:
            raise MMFError("mmf_program_workspace_bytes", 2)
        self.projs = list(projs)
        self.ws = workspace(n, projs[0]["x"].device)
        mmf_program_init(self.projs, T, eps, self.ws, stream)

    def run(self, stream=None):
        mmf_program_run(self.ws, stream)


def mmf_get_device_status():
    """Status code (int) of the device status word; reading clears it."""
    return lib().mmf_get_device_status()


def mmf_debug_wait_timeout_probe(limit_ns, stream=None):
    _check("mmf_debug_wait_timeout_probe",
           lib().mmf_debug_wait_timeout_probe(int(limit_ns), _stream(stream)))


def mmf_status_string(code):
    return lib().mmf_status_string(code).decode()


def mmf_version():
    return lib().mmf_version()


# ------------------------------------------------------------------------------ conveniences
def workspace(nbytes, device="cuda"):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def quantize_weights(W, stream=None):
    """W [N,K] (fp32/fp16, CUDA) -> (Wp uint8 [N, K/4], beta float32 [1])."""
    import torch
    N, K = W.shape
    Wp = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    beta = torch.empty(1, dtype=torch.float32, device=W.device)
    ws = workspace(mmf_quantize_weights_workspace_bytes(N, K), W.device)
    mmf_quantize_weights(W, Wp, beta, ws, stream)
    return Wp, beta


def bitlinear_forward(x, Wp, beta, norm_w=None, eps=1e-8, out_dtype=None, ws=None,
                      stream=None):
    import torch
    T, K = x.shape
    N = Wp.shape[0]
    y = torch.empty((T, N), dtype=out_dtype or x.dtype, device=x.device)
    if ws is None:
        ws = workspace(mmf_forward_workspace_bytes(T, K, N), x.device)
    mmf_bitlinear_forward(x, norm_w, eps, Wp, beta, N, y, ws, stream)
    return y


def mlgru_forward(I, F, G, h0=None, norm_w=None, eps=1e-8, out_dtype=None, hT=None, ws=None,
                  stream=None):
    """o [T, H] of the MLGRU recurrence and swish gate norm; hT (optional [H] fp32) receives
    the state after the last token."""
    import torch
    T, H = I.shape
    o = torch.empty((T, H), dtype=out_dtype or I.dtype, device=I.device)
    need = mmf_mlgru_workspace_bytes(T, H)
    if ws is None and need > 0:
        ws = workspace(need, I.device)
    mmf_mlgru_forward(I, F, G, h0, norm_w, eps, o, hT, ws, stream)
    return o


def bitlinear_glu_forward(x, Wp, beta, norm_w=None, eps=1e-8, out_dtype=None, ws=None,
                          stream=None):
    import torch
    T, K = x.shape
    N2 = Wp.shape[0]
    h = torch.empty((T, N2 // 2), dtype=out_dtype or x.dtype, device=x.device)
    if ws is None:
        ws = workspace(mmf_forward_workspace_bytes(T, K, N2), x.device)
    mmf_bitlinear_glu_forward(x, norm_w, eps, Wp, beta, N2, h, ws, stream)
    return h


def bitlinear_backward(x, Wp, beta, dy, norm_w=None, eps=1e-8, A=None, gamma=None,
                       dx_dtype=None, want_dx=True, want_dW=True, want_dnorm_w=False, ws=None,
                       stream=None):
    """Straight-through backward of bitlinear_forward: returns ``(dx, dW, dnorm_w)`` (None for
    what was not asked).  dy: fp16 [T, N]; dW and dnorm_w are fp32."""
    import torch
    T, K = x.shape
    N = Wp.shape[0]
    dev = x.device
    dx = torch.empty((T, K), dtype=dx_dtype or x.dtype, device=dev) if want_dx else None
    dW = torch.empty((N, K), dtype=torch.float32, device=dev) if want_dW else None
    dg = torch.empty(K, dtype=torch.float32, device=dev) if want_dnorm_w else None
    if ws is None:
        ws = workspace(mmf_backward_workspace_bytes(T, K, N), dev)
    mmf_bitlinear_backward(x, norm_w, eps, A, gamma, Wp, beta, N, dy, dx, dW, dg, ws, stream)
    return dx, dW, dg


# ------------------------------------------------------------- 8-bit projection, linear attention
def _tensor(name, t, shape, dtypes, device, contiguous=True):
    """Refuses a tensor that the call would misread: dtypes a tuple, shape with None for any, or the
    number of dimensions."""
    got = t.shape
    if (len(got) == shape if shape.__class__ is int else got == shape) and t.dtype in dtypes and \
            t.device == device and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    want = (None,) * shape if isinstance(shape, int) else shape
    if len(got) != len(want) or any(s is not None and s != n for s, n in zip(want, got)):
        raise ValueError(f"{name}: shape {tuple(got)}, expected {want}")
    if t.is_contiguous():
        return
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    if got[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


_current = None


def _current_calls():
    """torch's calls for the current device and for a device's current stream as a handle: without
    their checks (1.3 us a call) where this release has them so, else the public ones."""
    global _current
    if _current is None:
        import torch
        device = getattr(torch._C, "_cuda_getDevice", None)
        handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current = (device or torch.cuda.current_device,
                    handle or (lambda at: torch.cuda.current_stream(at).cuda_stream))
    return _current


def _on(t, stream, call):
    """``call(handle)`` with the tensor's device and the call's stream current, so that what the
    call allocates belongs to the stream that uses it; the handle is the stream's."""
    import torch
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a GPU, got {t.device}")
    at = t.get_device()
    if stream is None:
        device, handle = _current or _current_calls()
        if at == device():
            return call(handle(at))
        with torch.cuda.device(at):
            return call(handle(at))
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=t.device)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
    with torch.cuda.device(at), torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def quantize_weights_int8(W, stream=None):
    """W [N, K] (fp32/fp16, CUDA, contiguous) -> (W8 int8 [N, K], wscale float32 [N])."""
    import torch
    dev = W.device
    _tensor("W", W, 2, (torch.float32, torch.float16), dev)

    def call(handle):
        W8 = torch.empty(W.shape, dtype=torch.int8, device=dev)
        wscale = torch.empty(W.shape[0], dtype=torch.float32, device=dev)
        mmf_int8_quantize_weights(W, W8, wscale, handle)
        return W8, wscale

    return _on(W, stream, call)


def int8_matmul(A, gamma, W8, wscale, out_dtype=None, out=None, stream=None):
    """y [T, N] of activation codes A [T, K] with scales gamma [T] (mmf_quantize_activations) and
    weights from quantize_weights_int8; fp16 unless out_dtype or out says otherwise."""
    import torch
    dev = A.device
    _tensor("A", A, 2, (torch.int8,), dev)
    T, K = A.shape
    N = W8.shape[0]
    _tensor("W8", W8, (N, K), (torch.int8,), dev)
    _tensor("gamma", gamma, (T,), (torch.float32,), dev)
    _tensor("wscale", wscale, (N,), (torch.float32,), dev)
    if out is not None:
        _tensor("out", out, (T, N), (torch.float32, torch.float16), dev)

    def call(handle):
        y = out
        if y is None:
            y = torch.empty((T, N), dtype=out_dtype or torch.float16, device=dev)
        mmf_int8_forward_quantized(A, gamma, W8, wscale, y, handle)
        return y

    return _on(A, stream, call)


def int8_linear_forward(x, W8, wscale, norm_w=None, eps=1e-8, out_dtype=None, ws=None,
                        stream=None):
    """RMSNorm, activation quantisation and 8-bit product of x [T, K]: y [T, N]."""
    import torch
    dev = x.device
    _tensor("x", x, 2, (torch.float32, torch.float16), dev)
    T, K = x.shape
    N = W8.shape[0]
    _tensor("W8", W8, (N, K), (torch.int8,), dev)
    _tensor("wscale", wscale, (N,), (torch.float32,), dev)
    if norm_w is not None:
        _tensor("norm_w", norm_w, (K,), (torch.float32,), dev)

    def call(handle):
        y = torch.empty((T, N), dtype=out_dtype or x.dtype, device=dev)
        scratch = _scratch(ws, max(mmf_int8_workspace_bytes(T, K), 256), dev)
        mmf_int8_forward(x, norm_w, eps, W8, wscale, y, scratch, handle)
        return y

    return _on(x, stream, call)


def _linattn(q, k, v, log_decay, o, scale, cu_seqlens, batch, clear=False):
    """Checks a call's tensors and describes them; clear: zeros for tokens outside the sequences."""
    import torch
    dev, f = q.device, (torch.float32, torch.float16)
    _tensor("q", q, 3, f, dev, contiguous=False)
    T, H, dk = q.shape
    _tensor("k", k, (T, H, dk), (q.dtype,), dev, contiguous=False)
    dv = v.shape[-1]
    _tensor("v", v, (T, H, dv), (q.dtype,), dev, contiguous=False)
    _tensor("log_decay", log_decay, (H,), (torch.float32,), dev)
    if o is not None:
        _tensor("out", o, (T, H, dv), (q.dtype,), dev, contiguous=False)
    if cu_seqlens is not None:
        _tensor("cu_seqlens", cu_seqlens, 1, (torch.int32,), dev)
        if batch is not None and batch != cu_seqlens.numel() - 1:
            raise ValueError(f"batch {batch}, but cu_seqlens has {cu_seqlens.numel() - 1} sequences")
        batch = cu_seqlens.numel() - 1
    return LinattnDesc(
        T, 1 if batch is None else batch, _ptr(cu_seqlens), H, dk, dv, _dt(q),
        dk ** -0.5 if scale is None else scale, clear, _ptr(log_decay), *q.stride()[:2],
        *k.stride()[:2], *v.stride()[:2], *((H * dv, dv) if o is None else o.stride()[:2]))


def _scratch(ws, need, device):
    """The workspace of a call: the caller's, if it is one, or a new one of `need` bytes."""
    if ws is None:
        return workspace(need, device) if need > 0 else None
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws


def _linattn_states(d, device, **states):
    import torch
    for name, t in states.items():
        if t is not None:
            _tensor(name, t, (d.B, d.H, d.dk, d.dv), (torch.float32,), device)


def linattn_forward(q, k, v, log_decay, scale=None, cu_seqlens=None, batch=None, h0=None, hT=None,
                    out=None, ws=None, stream=None):
    """Linear attention with a decay for each head over packed prompts: o [T, H, dv].

    q, k [T, H, dk], v [T, H, dv] of one dtype (fp16 or fp32), views with any token and head
    strides of whole 16 bytes; log_decay [H] fp32, at most 0; scale: dk ** -0.5 unless given.
    cu_seqlens [B + 1] int32 (device), or batch equal sequences (1 unless given).  h0, hT
    [B, H, dk, dv] fp32: states before (zero unless given) and after (written if given; may be
    h0).  Rows of tokens outside the sequences are zero, or left as they were in a given out."""
    import torch
    dev = q.device
    d = _linattn(q, k, v, log_decay, out, scale, cu_seqlens, batch, out is None)
    _linattn_states(d, dev, h0=h0, hT=hT)

    def call(handle):
        o = out
        if o is None:
            o = torch.empty((d.T, d.H, d.dv), dtype=q.dtype, device=dev)
        scratch = _scratch(ws, mmf_linattn_workspace_bytes(d), dev)
        mmf_linattn_forward(d, q, k, v, h0, o, hT, scratch, handle)
        return o

    return _on(q, stream, call)


def linattn_step(q, k, v, log_decay, state, scale=None, slots=None, out=None, stream=None):
    """One new token of each of B sequences: o [B, H, dv]; q, k [B, H, dk], v [B, H, dv].

    state [B, H, dk, dv] fp32 is updated in place; with slots [B] int32 (device) it is a pool
    [n, H, dk, dv] and slots names each row's state (negative: padding, zeros out)."""
    import torch
    dev = q.device
    d = _linattn(q, k, v, log_decay, out, scale, None, q.shape[0])
    _tensor("state", state, (None if slots is not None else d.B, d.H, d.dk, d.dv),
            (torch.float32,), dev)
    if slots is not None:
        _tensor("slots", slots, (d.B,), (torch.int32,), dev)

    def call(handle):
        o = out
        if o is None:
            o = torch.empty((d.B, d.H, d.dv), dtype=q.dtype, device=dev)
        mmf_linattn_step(d, q, k, v, o, state, slots, handle)
        return o

    return _on(q, stream, call)


def linattn_backward(q, k, v, log_decay, dout, scale=None, cu_seqlens=None, batch=None, h0=None,
                     dhT=None, want_dh0=False, ws=None, stream=None):
    """Gradients of linattn_forward: ``(dq, dk, dv, dh0)`` (dh0 None unless asked for).

    dout [T, H, dv]: the gradient of o; dhT: that of hT (none unless given).  Rows of tokens
    outside the sequences are zero."""
    import torch
    dev = q.device
    d = _linattn(q, k, v, log_decay, dout, scale, cu_seqlens, batch, True)
    _linattn_states(d, dev, h0=h0, dhT=dhT)

    def call(handle):
        dq, dk = (torch.empty((d.T, d.H, d.dk), dtype=q.dtype, device=dev) for _ in range(2))
        dv = torch.empty((d.T, d.H, d.dv), dtype=q.dtype, device=dev)
        dh0 = None
        if want_dh0:
            dh0 = torch.empty((d.B, d.H, d.dk, d.dv), dtype=torch.float32, device=dev)
        scratch = _scratch(ws, mmf_linattn_backward_workspace_bytes(d), dev)
        mmf_linattn_backward(d, q, k, v, dout, h0, dhT, dq, dk, dv, dh0, scratch, handle)
        return dq, dk, dv, dh0

    return _on(q, stream, call)
