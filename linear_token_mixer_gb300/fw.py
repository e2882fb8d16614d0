"""Thin ctypes binding of libfw.so (include/fw.h) over torch CUDA tensors.

Argument marshalling only: every step of the recurrence runs in the library's
CUDA kernels.  There is no CPU path; if libfw.so is missing or fails to load,
every call raises.  torch supplies device memory and streams.

stream= (of every call; None: the current stream of the tensors' device): the kernels run there.  The
caller has that stream wait for whatever makes the inputs, and waits for it before the outputs are read
elsewhere; tensors may be given back at once, since the call marks their memory as in use by the stream.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfw.so")

FW_F32, FW_BF16 = 0, 1
MODES = {"falcon1": 0, "linattn": 1, "falcon1a": 2, "falcon2": 3, "falcon2a": 4,
         "falcon3": 5, "falcon3a": 6}
WINDOW_MAX = 8
FLAG_RBW, FLAG_SAME_PAIR, FLAG_ZERO_REST, FLAG_SILU, FLAG_SOFTPLUS = 1, 2, 4, 8, 16
PHIS = {"identity": 0, "elu1": 1}
ALGOS = {"auto": 0, "recurrent": 1, "chunked": 2}
DTYPES = {torch.float32: FW_F32, torch.bfloat16: FW_BF16}

FW_OK = 0
STATUS = {0: "FW_OK", -1: "FW_ERR_NULL", -2: "FW_ERR_SHAPE", -3: "FW_ERR_DTYPE",
          -4: "FW_ERR_ALIGN", -5: "FW_ERR_MODE", -6: "FW_ERR_CUDA", -7: "FW_ERR_TIMEOUT",
          -8: "FW_ERR_UNSUPPORTED", -9: "FW_ERR_ARG", -10: "FW_ERR_DEVICE", -11: "FW_ERR_SCRATCH"}


class FwError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = lib().fw_status_string(status).decode()
        if status == -6:
            msg += " (cudaError %d)" % lib().fw_last_cuda_error()
        super().__init__("%s: %s" % (where, msg))


class fw_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("H", ctypes.c_int64), ("T", ctypes.c_int64),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32)]


class fw_window(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("n", ctypes.c_void_p)]


class fw_norm(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("eps", ctypes.c_float)]


class fw_gates(ctypes.Structure):
    _fields_ = [("dt", ctypes.c_void_p), ("dt_type", ctypes.c_int), ("log_decay", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("skip", ctypes.c_void_p), ("groups", ctypes.c_int64)]


class fw_gated(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int64),
                ("inner", ctypes.c_int64), ("eps", ctypes.c_float), ("rms", ctypes.c_int),
                ("gate_after", ctypes.c_int)]


EXPORTS = ("fw_prefill", "fw_prefill_ex", "fw_prefill_noalloc", "fw_step", "fw_step_ex", "fw_window_prefill",
           "fw_window_step", "fw_decay_workspace", "fw_decay_prefill", "fw_decay_backward",
           "fw_decay_step", "fw_select_workspace", "fw_select_prefill", "fw_select_step", "fw_conv_prefill",
           "fw_conv_workspace", "fw_conv_backward", "fw_conv_step", "fw_gated_norm", "fw_gated_norm_workspace",
           "fw_gated_norm_backward", "fw_layer_norm", "fw_layer_norm_workspace", "fw_layer_norm_backward",
           "fw_check",
           "fw_status_string", "fw_version", "fw_last_cuda_error", "fw_set_wait_limit_us",
           "fw_debug_force_timeout", "fw_debug_segment_split")

_lib = None


def lib():
    """Load libfw.so (building it first is the caller's job: see build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfw.so is not built (run linear_token_mixer_gb300/build.py); "
                               "there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        SP = ctypes.POINTER(fw_shape)
        L.fw_prefill.argtypes = [P, P, P, P, P, P, P, P, SP, I, I, I, F, P]
        U = ctypes.c_uint
        L.fw_prefill_ex.argtypes = [P, P, P, P, P, P, P, P, P, SP, I, I, I, F, U, I, P]
        L.fw_prefill_noalloc.argtypes = L.fw_prefill_ex.argtypes
        L.fw_step.argtypes = [P, P, P, P, P, P, P, SP, I, I, I, F, P]
        L.fw_step_ex.argtypes = [P, P, P, P, P, P, P, SP, I, I, I, F, U, P]
        WP = ctypes.POINTER(fw_window)
        L.fw_window_prefill.argtypes = [P, P, P, P, P, P, P, WP, P, P, WP, SP, I, I, I, I, F, U,
                                        P]
        L.fw_window_step.argtypes = [P, P, P, P, P, P, WP, P, WP, SP, I, I, I, I, F, U, P]
        N, I64 = ctypes.POINTER(fw_norm), ctypes.c_int64
        L.fw_decay_workspace.argtypes = [SP, I, I]
        L.fw_decay_prefill.argtypes = [P, P, P, P, P, P, N, P, P, SP, I, F, U, P, I64, P]
        L.fw_decay_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, SP, I, F, U, P, I64, P]
        L.fw_decay_step.argtypes = [P, P, P, P, P, N, P, SP, I, F, P]
        L.fw_layer_norm.argtypes = [P, P, P, P, P, P, I64, I64, I, F, P]
        L.fw_layer_norm_workspace.argtypes = [I64, I64]
        L.fw_layer_norm_backward.argtypes = [P, P, P, P, P, P, P, P, I64, I64, I, P, I64, P]
        G, GN = ctypes.POINTER(fw_gates), ctypes.POINTER(fw_gated)
        L.fw_select_workspace.argtypes = [SP, I]
        L.fw_select_prefill.argtypes = [P, P, P, G, P, P, P, P, SP, I, F, U, P, I64, P]
        L.fw_select_step.argtypes = [P, P, P, G, P, P, SP, I, F, U, P]
        L.fw_conv_prefill.argtypes = [P, P, P, P, P, P, P, SP, I, I, U, P]
        L.fw_conv_workspace.argtypes = [SP, I]
        L.fw_conv_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, P, SP, I, I, U, P, I64, P]
        L.fw_conv_step.argtypes = [P, P, P, P, P, SP, I, I, U, P]
        L.fw_gated_norm.argtypes = [P, GN, P, P, P, P, I64, I64, I, P]
        L.fw_gated_norm_workspace.argtypes = [I64, I64, I64, I]
        L.fw_gated_norm_backward.argtypes = [P, P, P, GN, P, P, P, P, P, P, P, P, I64, I64, I, P, I64, P]
        for f in (L.fw_select_workspace, L.fw_conv_workspace, L.fw_gated_norm_workspace):
            f.restype = I64
        L.fw_decay_workspace.restype = L.fw_layer_norm_workspace.restype = I64
        L.fw_check.argtypes = [P]
        L.fw_status_string.argtypes = [I]
        L.fw_status_string.restype = ctypes.c_char_p
        L.fw_version.argtypes = []
        L.fw_last_cuda_error.argtypes = []
        L.fw_set_wait_limit_us.argtypes = [ctypes.c_longlong]
        L.fw_set_wait_limit_us.restype = None
        L.fw_debug_force_timeout.argtypes = [I]
        L.fw_debug_force_timeout.restype = None
        L.fw_debug_segment_split.argtypes = [I]
        L.fw_debug_segment_split.restype = None
        for f in (L.fw_prefill, L.fw_prefill_ex, L.fw_prefill_noalloc, L.fw_step, L.fw_step_ex,
                  L.fw_window_prefill,
                  L.fw_window_step, L.fw_decay_prefill, L.fw_decay_backward, L.fw_decay_step,
                  L.fw_select_prefill, L.fw_select_step, L.fw_conv_prefill, L.fw_conv_backward, L.fw_conv_step,
                  L.fw_gated_norm, L.fw_gated_norm_backward,
                  L.fw_layer_norm, L.fw_layer_norm_backward, L.fw_check, L.fw_version, L.fw_last_cuda_error):
            f.restype = I
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fw: tensors must live on a CUDA device (no CPU path)")
    if not t.is_contiguous():
        raise ValueError("fw: tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _used(stream, *tensors):
    """Work on `stream` uses these tensors: memory of theirs that the caller gives back, as that of a
    temporary, is not handed out again before the work is done.  (The current stream, None, needs none
    of this.)"""
    if stream is None or stream == torch.cuda.current_stream(stream.device):
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _flags(rbw, same_pair):
    return (FLAG_RBW if rbw else 0) | (FLAG_SAME_PAIR if same_pair else 0)


def prefill(q, k, v, beta=None, lam=None, S0=None, *, mode="falcon1", phi="identity",
            eps=1e-6, k_init=None, algo="auto", o=None, S_T=None, stream=None, rbw=False,
            same_pair=False, noalloc=False, norm=None, norm_eps=1e-5):
    """Run the recurrence over q, k, v [B, H, T, d] (fp32 or bf16).

    mode: "falcon1", "falcon1a", "falcon2", "falcon2a" or "linattn"; rbw reads
    before the write, same_pair pairs each key with its own value.  Returns
    (o [B,H,T,d] in q's dtype, S_T [B,H,d,d] fp32).  beta, lam [B,H,T] fp32 are
    required in the falcon modes (beta [B,H,T,d] for falcon2 / falcon2a).  S0
    [B,H,d,d] fp32 or None.  noalloc: call fw_prefill_noalloc (the library's
    workspace from its static buffer; pass o and S_T to allocate nothing here
    either).  norm: (weight [d], bias [d]) fp32, either None: layer norm of every
    row of o, in place (bf16 rows are rounded before it and after it; the decayed
    calls norm the fp32 row)."""
    B, H, T, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if S_T is None:
        S_T = torch.empty((B, H, d, d), device=q.device, dtype=torch.float32)
    shp = fw_shape(B, H, T, d, v.shape[-1])
    _norm_ready(norm, norm_eps, q, o, stream, S_T)
    fn = lib().fw_prefill_noalloc if noalloc else lib().fw_prefill_ex
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0), _ptr(k_init), _ptr(o),
            _ptr(S_T), ctypes.byref(shp), DTYPES.get(q.dtype, -1), MODES[mode], PHIS[phi],
            float(eps), _flags(rbw, same_pair), ALGOS[algo], _stream(stream))
    if st != FW_OK:
        raise FwError(st, "fw_prefill_noalloc" if noalloc else "fw_prefill")
    _used(stream, q, k, v, beta, lam, S0, k_init, o, S_T, *(norm or ()))
    return _with_norm(o, norm, norm_eps, stream), S_T


def step(q, k_prev, v, beta, lam, S, *, mode="falcon1", phi="identity", eps=1e-6, o=None,
         stream=None, rbw=False, norm=None, norm_eps=1e-5):
    """One decode step for q, k_prev, v [B, H, d]; S [B, H, d, d] fp32 is
    updated in place (rbw: o = S_old^T q); norm as in prefill.  Returns o [B, H, d] in q's dtype."""
    B, H, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    shp = fw_shape(B, H, 1, d, v.shape[-1])
    _norm_ready(norm, norm_eps, q, o, stream, S)
    st = lib().fw_step_ex(_ptr(q), _ptr(k_prev), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S),
                          _ptr(o), ctypes.byref(shp), DTYPES.get(q.dtype, -1), MODES[mode],
                          PHIS[phi], float(eps), _flags(rbw, False), _stream(stream))
    if st != FW_OK:
        raise FwError(st, "fw_step")
    _used(stream, q, k_prev, v, beta, lam, S, o, *(norm or ()))
    return _with_norm(o, norm, norm_eps, stream)


def new_window(B, H, d, window, device="cuda"):
    """An empty carried window (x, y, n) for `window` pairs: x, y
    [B, H, window-1, d] fp32, n [B, H] int32, all zero."""
    return (torch.zeros((B, H, window - 1, d), device=device, dtype=torch.float32),
            torch.zeros((B, H, window - 1, d), device=device, dtype=torch.float32),
            torch.zeros((B, H), device=device, dtype=torch.int32))


def _window(w):
    if w is None:
        return None
    x, y, n = w
    if n.dtype != torch.int32 or x.dtype != torch.float32 or y.dtype != torch.float32:
        raise ValueError("fw: a window is (x fp32, y fp32, n int32)")
    return ctypes.byref(fw_window(_ptr(x), _ptr(y), _ptr(n)))


def window_prefill(q, k, v, beta, lam, window, S0=None, *, mode="falcon3", phi="identity",
                   eps=1e-6, k_init=None, win_in=None, win_out=None, o=None, S_T=None,
                   stream=None, rbw=False, same_pair=False, norm=None, norm_eps=1e-5):
    """Falcon-3 ("falcon3") or 3A ("falcon3a") over q, k, v [B, H, T, d] with a
    window of `window` pairs.  win_in: the window carried from an earlier call
    (as returned here), or None; win_out: tensors to receive the window after
    the last token (allocated when None); norm as in prefill.  Returns
    (o, S_T, win_out)."""
    B, H, T, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if S_T is None:
        S_T = torch.empty((B, H, d, d), device=q.device, dtype=torch.float32)
    if win_out is None:
        win_out = new_window(B, H, d, window, q.device)
    shp = fw_shape(B, H, T, d, v.shape[-1])
    _norm_ready(norm, norm_eps, q, o, stream, S_T, *win_out)
    st = lib().fw_window_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S0),
                                 _ptr(k_init), _window(win_in), _ptr(o), _ptr(S_T),
                                 _window(win_out), ctypes.byref(shp), int(window),
                                 DTYPES.get(q.dtype, -1), MODES[mode], PHIS[phi], float(eps),
                                 _flags(rbw, same_pair), _stream(stream))
    if st != FW_OK:
        raise FwError(st, "fw_window_prefill")
    _used(stream, q, k, v, beta, lam, S0, k_init, o, S_T, *(win_in or ()), *win_out, *(norm or ()))
    return _with_norm(o, norm, norm_eps, stream), S_T, win_out


def window_step(q, k_prev, v, beta, lam, S, window, win_in=None, win_out=None, *,
                mode="falcon3", phi="identity", eps=1e-6, o=None, stream=None, rbw=False,
                norm=None, norm_eps=1e-5):
    """One Falcon-3 / 3A decode step for q, k_prev, v [B, H, d]; S [B, H, d, d]
    fp32 is updated in place; the window moves from win_in (None: empty) to
    win_out (allocated when None; must not be win_in); norm as in prefill.  Returns
    (o, win_out)."""
    B, H, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if win_out is None:
        win_out = new_window(B, H, d, window, q.device)
    shp = fw_shape(B, H, 1, d, v.shape[-1])
    _norm_ready(norm, norm_eps, q, o, stream, S, *win_out)
    st = lib().fw_window_step(_ptr(q), _ptr(k_prev), _ptr(v), _ptr(beta), _ptr(lam), _ptr(S),
                              _window(win_in), _ptr(o), _window(win_out), ctypes.byref(shp),
                              int(window), DTYPES.get(q.dtype, -1), MODES[mode], PHIS[phi],
                              float(eps), _flags(rbw, False), _stream(stream))
    if st != FW_OK:
        raise FwError(st, "fw_window_step")
    _used(stream, q, k_prev, v, beta, lam, S, o, *(win_in or ()), *win_out, *(norm or ()))
    return _with_norm(o, norm, norm_eps, stream), win_out


def _bad(t, shape, dtype, name, like):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        return ValueError("fw: %s must be %s of %s, not %s of %s" % (
            name, tuple(shape), dtype, tuple(t.shape), t.dtype))
    if t.get_device() != like.get_device():
        return ValueError("fw: %s is on %s, the call's tensors are on %s" % (name, t.device,
                                                                            like.device))
    return ValueError("fw: tensors must be contiguous (%s is not)" % name)


def _arg(t, shape, dtype, name, like):
    """The address of a tensor argument (None: NULL) of the given shape and dtype on like's
    device (_On refuses one that is not a GPU).  These calls serve single tokens, so the checks
    cost as little as they can."""
    if t is None:
        return None
    if (t.shape != shape or t.dtype is not dtype or t.get_device() != like.get_device()
            or not t.is_contiguous()):
        raise _bad(t, shape, dtype, name, like)
    return t.data_ptr()


class _On:
    """The stream of a call and where its new tensors come from: that stream's pool, so that a
    workspace freed at return is reused behind the kernels that read it; outputs are also known
    to the caller's current stream.  A call on the current stream (stream None) allocates as
    torch does."""
    __slots__ = ("like", "index", "handle", "stream", "current")

    def __init__(self, like, stream):
        if not like.is_cuda:
            raise ValueError("fw: tensors must live on a CUDA device (no CPU path)")
        self.like, self.index, self.stream = like, like.get_device(), None
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(self.index)
            return
        if stream.device != like.device:
            raise ValueError("fw: the stream is on %s, the tensors are on %s" % (stream.device,
                                                                              like.device))
        self.handle = stream.cuda_stream
        self.current = torch.cuda.current_stream(like.device)
        if stream != self.current:
            self.stream = stream

    def new(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.like.device)
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device=self.like.device)
        t.record_stream(self.current)
        return t

    def same(self, t):
        """A new tensor of t's shape and type."""
        return torch.empty_like(t) if self.stream is None else self.new(t.shape, t.dtype)

    def workspace(self, given, need, where):
        """(tensor to keep alive, address, bytes) of a workspace of `need` bytes."""
        if need < 0:
            raise FwError(int(need), where)
        if given is None:
            if need == 0:
                return None, None, 0
            given = self.new((need,), torch.uint8)
        elif not given.is_cuda or given.get_device() != self.index or not given.is_contiguous():
            raise ValueError("fw: the workspace must be contiguous and on %s" % self.like.device)
        return given, given.data_ptr(), given.numel() * given.element_size()

    def call(self, fn, where, tensors, *args):
        """fn(*args, stream) on the tensors' device."""
        if torch._C._cuda_getDevice() == self.index:
            st = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.index):
                st = fn(*args, self.handle)
        if st != FW_OK:
            raise FwError(st, where)
        if self.stream is not None:
            _used(self.stream, *tensors)


def _norm(norm, eps, width, like):
    if norm is None:
        return None
    weight, bias = norm
    if not 0.0 <= ctypes.c_float(eps).value < float("inf"):
        raise ValueError("fw: norm_eps must be finite and not negative")
    return ctypes.byref(fw_norm(_arg(weight, (width,), torch.float32, "norm weight", like),
                                _arg(bias, (width,), torch.float32, "norm bias", like), eps))


@functools.lru_cache(maxsize=4096)
def _decay_need(B, H, T, d, dtype, backward):
    return lib().fw_decay_workspace(ctypes.byref(fw_shape(B, H, T, d, d)), dtype, backward)


@functools.lru_cache(maxsize=4096)
def _layer_norm_need(rows, width):
    return lib().fw_layer_norm_workspace(rows, width)


def _axes(q, n):
    if q.dim() != n:
        raise ValueError("fw: q must have %d axes, not %d" % (n, q.dim()))
    return q.shape


def _fresh(on, t, shape, dtype, zero):
    if t is None:
        t = on.new(shape, dtype)
        if zero:
            with torch.cuda.stream(on.stream or torch.cuda.current_stream(t.device)):
                t.zero_()
    return t


def decay_workspace(B, H, T, d, dtype=torch.bfloat16, *, backward=False):
    """Bytes of workspace of decay_prefill (or decay_backward) for this shape."""
    n = _decay_need(B, H, T, d, DTYPES.get(dtype, -1), int(backward))
    if n < 0:
        raise FwError(int(n), "fw_decay_workspace")
    return n


def decay_prefill(q, k, v, log_decay, S0=None, *, scale=1.0, lens=None, norm=None, norm_eps=1e-5,
                  o=None, S_T=None, workspace=None, stream=None):
    """Linear attention with a decay g_h = exp(log_decay[h]) for each head over
    q, k, v [B, H, T, d] (fp32 or bf16): S_t = g_h S_{t-1} + k_t v_t^T,
    o_t = scale S_t^T q_t.

    log_decay [H] fp32; S0 [B, H, d, d] fp32 or None; lens [B] int32 or None
    (tokens of each row of a padded batch; rows of o behind them are left as
    they were with o given, zero without); norm (weight [d], bias [d]) fp32,
    either None: layer norm of every output row; workspace: a tensor of at least
    decay_workspace() bytes (allocated when None).  Returns (o, S_T)."""
    shape = B, H, T, d = _axes(q, 4)
    state, dt, f32 = (B, H, d, d), q.dtype, torch.float32
    args = (_arg(q, shape, dt, "q", q), _arg(k, shape, dt, "k", q), _arg(v, shape, dt, "v", q),
            _arg(log_decay, (H,), f32, "log_decay", q), _arg(S0, state, f32, "S0", q),
            _arg(lens, (B,), torch.int32, "lens", q), _norm(norm, norm_eps, d, q))
    on = _On(q, stream)
    flags = FLAG_ZERO_REST if o is None and lens is not None else 0
    if o is None:
        o = on.new(shape, dt)
    if S_T is None:
        S_T = on.new(state, f32)
    code = DTYPES.get(dt, -1)
    _keep, ws, nws = on.workspace(workspace, _decay_need(B, H, T, d, code, 0), "fw_decay_prefill")
    on.call(lib().fw_decay_prefill, "fw_decay_prefill",
            (q, k, v, log_decay, S0, lens, o, S_T, workspace, *(norm or ())), *args,
            _arg(o, shape, dt, "o", q), _arg(S_T, state, f32, "S_T", q),
            ctypes.byref(fw_shape(B, H, T, d, d)), code, scale, flags, ws, nws)
    return o, S_T


def decay_backward(q, k, v, log_decay, do, S0=None, dS_T=None, *, scale=1.0, lens=None, dq=None,
                   dk=None, dv=None, dS0=None, workspace=None, stream=None):
    """Gradients of decay_prefill (without norm) given do [B, H, T, d], the
    gradient of o, and dS_T [B, H, d, d] fp32 or None, that of S_T.  Returns
    (dq, dk, dv, dS0) in q's dtype and fp32; dS0 is None unless S0 or dS0 is
    given.  Rows behind lens are left as they were in a tensor that is given, and
    zero in one that is allocated here."""
    shape = B, H, T, d = _axes(q, 4)
    state, dt, f32 = (B, H, d, d), q.dtype, torch.float32
    args = (_arg(q, shape, dt, "q", q), _arg(k, shape, dt, "k", q), _arg(v, shape, dt, "v", q),
            _arg(log_decay, (H,), f32, "log_decay", q), _arg(S0, state, f32, "S0", q),
            _arg(lens, (B,), torch.int32, "lens", q), _arg(do, shape, dt, "do", q),
            _arg(dS_T, state, f32, "dS_T", q))
    on = _On(q, stream)
    fresh = dq is None and dk is None and dv is None
    flags = FLAG_ZERO_REST if fresh and lens is not None else 0
    dq, dk, dv = (_fresh(on, t, shape, dt, lens is not None and not fresh) for t in (dq, dk, dv))
    if dS0 is None and S0 is not None:
        dS0 = on.new(state, f32)
    code = DTYPES.get(dt, -1)
    _keep, ws, nws = on.workspace(workspace, _decay_need(B, H, T, d, code, 1), "fw_decay_backward")
    on.call(lib().fw_decay_backward, "fw_decay_backward",
            (q, k, v, log_decay, do, S0, dS_T, lens, dq, dk, dv, dS0, workspace), *args,
            _arg(dq, shape, dt, "dq", q), _arg(dk, shape, dt, "dk", q), _arg(dv, shape, dt, "dv", q),
            _arg(dS0, state, f32, "dS0", q), ctypes.byref(fw_shape(B, H, T, d, d)), code, scale,
            flags, ws, nws)
    return dq, dk, dv, dS0


def decay_step(q, k, v, log_decay, S, *, scale=1.0, norm=None, norm_eps=1e-5, o=None, stream=None):
    """One token of decay_prefill's recurrence for q, k, v [B, H, d]; S
    [B, H, d, d] fp32 is updated in place.  Returns o [B, H, d] in q's dtype."""
    shape = B, H, d = _axes(q, 3)
    dt, f32 = q.dtype, torch.float32
    args = (_arg(q, shape, dt, "q", q), _arg(k, shape, dt, "k", q), _arg(v, shape, dt, "v", q),
            _arg(log_decay, (H,), f32, "log_decay", q), _arg(S, (B, H, d, d), f32, "S", q),
            _norm(norm, norm_eps, d, q))
    on = _On(q, stream)
    if o is None:
        o = on.new(shape, dt)
    on.call(lib().fw_decay_step, "fw_decay_step", (q, k, v, log_decay, S, o, *(norm or ())), *args,
            _arg(o, shape, dt, "o", q), ctypes.byref(fw_shape(B, H, 1, d, d)), DTYPES.get(dt, -1),
            scale)
    return o


@functools.lru_cache(maxsize=4096)
def _select_need(B, H, T, d, dtype):
    return lib().fw_select_workspace(ctypes.byref(fw_shape(B, H, T, d, d)), dtype)


@functools.lru_cache(maxsize=4096)
def _conv_need(B, H, T, d, width):
    return lib().fw_conv_workspace(ctypes.byref(fw_shape(B, H, T, d, d)), width)


@functools.lru_cache(maxsize=4096)
def _gated_need(rows, width, groups, dtype):
    return lib().fw_gated_norm_workspace(rows, width, groups, dtype)


def _gates(dt, log_decay, dt_bias, skip, shape, groups, like):
    """fw_gates of a selective call; shape: that of dt."""
    H, f32 = (shape[1],), torch.float32
    if dt is None or log_decay is None:
        raise ValueError("fw: dt and log_decay are required")
    kind = f32 if dt.dtype is f32 else like.dtype
    return ctypes.byref(fw_gates(
        _arg(dt, shape, kind, "dt", like), DTYPES.get(kind, -1), _arg(log_decay, H, f32, "log_decay", like),
        _arg(dt_bias, H, f32, "dt_bias", like), _arg(skip, H, f32, "skip", like), groups))


def select_workspace(B, H, T, d, dtype=torch.bfloat16):
    """Bytes of workspace of select_prefill for this shape."""
    n = _select_need(B, H, T, d, DTYPES.get(dtype, -1))
    if n < 0:
        raise FwError(int(n), "fw_select_workspace")
    return n


def select_prefill(q, k, v, dt, log_decay, S0=None, *, dt_bias=None, softplus=False, skip=None, scale=1.0,
                   lens=None, o=None, S_T=None, workspace=None, stream=None):
    """Selective scan over v [B, H, T, d] with queries and keys q, k [B, G, T, d] (fp32 or bf16), each
    shared by H / G neighbouring heads: S_t = exp(log_decay[h] dt_t) S_{t-1} + dt_t k_t v_t^T,
    o_t = scale S_t^T q_t + skip[h] v_t, with the steps dt [B, H, T] (fp32, or q's dtype), dt + dt_bias[h],
    or softplus(dt + dt_bias[h]).

    log_decay, dt_bias, skip [H] fp32, the last two or None; S0, lens, o, S_T and workspace
    (of select_workspace() bytes) as in decay_prefill.  Returns (o, S_T)."""
    shape = B, H, T, d = _axes(v, 4)
    G = _axes(q, 4)[1]
    few, state, kind, f32 = (B, G, T, d), (B, H, d, d), q.dtype, torch.float32
    args = (_arg(q, few, kind, "q", q), _arg(k, few, kind, "k", q), _arg(v, shape, kind, "v", q),
            _gates(dt, log_decay, dt_bias, skip, (B, H, T), G, q), _arg(S0, state, f32, "S0", q),
            _arg(lens, (B,), torch.int32, "lens", q))
    on = _On(q, stream)
    flags = FLAG_ZERO_REST if o is None and lens is not None else 0
    if softplus:
        flags |= FLAG_SOFTPLUS
    if o is None:
        o = on.same(v)
    if S_T is None:
        S_T = on.new(state, f32)
    code = DTYPES.get(kind, -1)
    _keep, ws, nws = on.workspace(workspace, _select_need(B, H, T, d, code), "fw_select_prefill")
    on.call(lib().fw_select_prefill, "fw_select_prefill",
            (q, k, v, dt, log_decay, dt_bias, skip, S0, lens, o, S_T, workspace), *args,
            _arg(o, shape, kind, "o", q), _arg(S_T, state, f32, "S_T", q),
            ctypes.byref(fw_shape(B, H, T, d, d)), code, scale, flags, ws, nws)
    return o, S_T


def select_step(q, k, v, dt, log_decay, S, *, dt_bias=None, softplus=False, skip=None, scale=1.0, o=None,
                stream=None):
    """One token of select_prefill's recurrence for q, k [B, G, d], v [B, H, d], dt [B, H]; S
    [B, H, d, d] fp32 is updated in place.  Returns o [B, H, d] in q's dtype."""
    shape = B, H, d = _axes(v, 3)
    G = _axes(q, 3)[1]
    few, kind = (B, G, d), q.dtype
    args = (_arg(q, few, kind, "q", q), _arg(k, few, kind, "k", q), _arg(v, shape, kind, "v", q),
            _gates(dt, log_decay, dt_bias, skip, (B, H), G, q), _arg(S, (B, H, d, d), torch.float32, "S", q))
    on = _On(q, stream)
    if o is None:
        o = on.same(v)
    on.call(lib().fw_select_step, "fw_select_step", (q, k, v, dt, log_decay, dt_bias, skip, S, o), *args,
            _arg(o, shape, kind, "o", q), ctypes.byref(fw_shape(B, H, 1, d, d)), DTYPES.get(kind, -1), scale,
            FLAG_SOFTPLUS if softplus else 0)
    return o


def conv_prefill(x, weight, bias=None, state=None, *, silu=True, lens=None, y=None, state_out=None,
                 stream=None):
    """Short causal convolution of every channel of x [B, H, T, d] (fp32 or bf16, d up to 2^24):
    y_t = act(bias + sum_w weight[w] x_{t-W+1+w}), act silu or none.

    weight [H, d, W] fp32, W = 2 .. 8, the last tap on the row itself; bias [H, d] fp32 or None;
    state [B, H, W-1, d] in x's dtype: the rows before the first, oldest first (None: zeros);
    state_out: a tensor for those behind the last (allocated when None; may be state); lens [B]
    int32 or None, and rows of y behind them, as in decay_prefill.  Returns (y, state_out)."""
    shape = B, H, T, d = _axes(x, 4)
    W, kind, f32 = _taps(weight), x.dtype, torch.float32
    past = (B, H, W - 1, d)
    args = (_arg(x, shape, kind, "x", x), _arg(weight, (H, d, W), f32, "weight", x),
            _arg(bias, (H, d), f32, "bias", x), _arg(state, past, kind, "state", x),
            _arg(lens, (B,), torch.int32, "lens", x))
    on = _On(x, stream)
    flags = (FLAG_SILU if silu else 0) | (FLAG_ZERO_REST if y is None and lens is not None else 0)
    if y is None:
        y = on.same(x)
    if state_out is None:
        state_out = on.new(past, kind)
    on.call(lib().fw_conv_prefill, "fw_conv_prefill", (x, weight, bias, state, lens, y, state_out), *args,
            _arg(y, shape, kind, "y", x), _arg(state_out, past, kind, "state_out", x),
            ctypes.byref(fw_shape(B, H, T, d, d)), W, DTYPES.get(kind, -1), flags)
    return y, state_out


def conv_backward(dy, x, weight, bias=None, state=None, dstate_out=None, *, silu=True, lens=None, dx=None,
                  dweight=None, dbias=None, dstate=None, workspace=None, stream=None):
    """Gradients of conv_prefill given dy (x's shape and dtype) and dstate_out, that of the returned
    state, or None.  Returns (dx, dweight, dbias, dstate): dweight, dbias fp32; dstate in x's dtype, None
    unless state or dstate is given.  Rows of dx behind lens as in decay_backward.  H ceil(d / 32) up to 65535."""
    shape = B, H, T, d = _axes(x, 4)
    W, kind, f32 = _taps(weight), x.dtype, torch.float32
    past = (B, H, W - 1, d)
    args = (_arg(dy, shape, kind, "dy", x), _arg(x, shape, kind, "x", x), _arg(weight, (H, d, W), f32, "weight", x),
            _arg(bias, (H, d), f32, "bias", x), _arg(state, past, kind, "state", x),
            _arg(lens, (B,), torch.int32, "lens", x), _arg(dstate_out, past, kind, "dstate_out", x))
    on = _On(x, stream)
    flags = (FLAG_SILU if silu else 0) | (FLAG_ZERO_REST if dx is None and lens is not None else 0)
    if dx is None:
        dx = on.same(x)
    if dweight is None:
        dweight = on.new((H, d, W), f32)
    if dbias is None:
        dbias = on.new((H, d), f32)
    if dstate is None and state is not None:
        dstate = on.new(past, kind)
    _keep, ws, nws = on.workspace(workspace, _conv_need(B, H, T, d, W), "fw_conv_backward")
    on.call(lib().fw_conv_backward, "fw_conv_backward",
            (dy, x, weight, bias, state, lens, dstate_out, dx, dweight, dbias, dstate, workspace), *args,
            _arg(dx, shape, kind, "dx", x), _arg(dweight, (H, d, W), f32, "dweight", x),
            _arg(dbias, (H, d), f32, "dbias", x), _arg(dstate, past, kind, "dstate", x),
            ctypes.byref(fw_shape(B, H, T, d, d)), W, DTYPES.get(kind, -1), flags, ws, nws)
    return dx, dweight, dbias, dstate


def conv_step(x, weight, bias, state, *, silu=True, y=None, stream=None):
    """One token of conv_prefill for x [B, H, d]; state [B, H, W-1, d] moves on by one row in place.
    Returns y [B, H, d]."""
    shape = B, H, d = _axes(x, 3)
    W, kind = _taps(weight), x.dtype
    args = (_arg(x, shape, kind, "x", x), _arg(weight, (H, d, W), torch.float32, "weight", x),
            _arg(bias, (H, d), torch.float32, "bias", x), _arg(state, (B, H, W - 1, d), kind, "state", x))
    on = _On(x, stream)
    if y is None:
        y = on.same(x)
    on.call(lib().fw_conv_step, "fw_conv_step", (x, weight, bias, state, y), *args, _arg(y, shape, kind, "y", x),
            ctypes.byref(fw_shape(B, H, 1, d, d)), W, DTYPES.get(kind, -1), FLAG_SILU if silu else 0)
    return y


def _taps(weight):
    if weight.dim() != 3:
        raise ValueError("fw: weight must be [H, d, W]")
    return weight.shape[2]


def _gated_shape(x, params):
    """(leading shape, rows, width, groups, inner, shape of a parameter): parameters [width], or
    [H, width] with x [.., H, T, width]."""
    if x.dim() < 1:
        raise ValueError("fw: gated_norm needs at least one axis")
    shape = x.shape
    lead, width = shape[:-1], shape[-1]
    rows = lead.numel()
    for p in params:
        if p is not None and p.dim() == 2:
            if x.dim() < 3:
                raise ValueError("fw: parameters [H, width] go with x [.., H, T, width]")
            return lead, rows, width, shape[-3], shape[-2], (shape[-3], width)
    return lead, rows, width, 1, rows, (width,)


def gated_norm(x, weight=None, bias=None, *, gate=None, residual=None, scale=None, rms=False, gate_after=False,
               eps=1e-5, y=None, total=None, mean=None, rstd=None, stats=True, stream=None):
    """The norm before a block with its scaled residual sum, and the norm behind a mixer with its gate,
    over the last axis of x (fp32 or bf16, width 1 .. 8192), with u = x + scale residual:
    y = norm(u silu(gate)) weight + bias, or with gate_after (norm(u) weight + bias) silu(gate).
    norm: layer norm, or with rms the row over its root mean square.

    gate, residual: x's shape and dtype, or None; scale (with a residual), weight, bias: fp32
    [width], or all of them [H, width] for x [.., H, T, width], or None.  y and total may each be x, gate or
    residual.  Returns (y, total, mean, rstd): total is u as stored, None without a residual;
    the statistics fp32 of x's leading shape (None with stats=False; mean None with rms)."""
    lead, rows, width, groups, inner, par = _gated_shape(x, (weight, bias, scale))
    shape, kind, f32 = x.shape, x.dtype, torch.float32
    x_ = _arg(x, shape, kind, "x", x)
    _finite_eps(eps)
    args = fw_gated(_arg(gate, shape, kind, "gate", x), _arg(residual, shape, kind, "residual", x),
                    _arg(scale, par, f32, "scale", x), _arg(weight, par, f32, "weight", x),
                    _arg(bias, par, f32, "bias", x), groups, inner, eps, int(rms), int(gate_after))
    on = _On(x, stream)
    if y is None:
        y = on.same(x)
    if total is None and residual is not None:
        total = on.same(x)
    if not stats:
        mean = rstd = None
    else:
        mean = None if rms else on.new(lead, f32) if mean is None else mean
        if rstd is None:
            rstd = on.new(lead, f32)
    on.call(lib().fw_gated_norm, "fw_gated_norm", (x, gate, residual, scale, weight, bias, y, total, mean, rstd),
            x_, ctypes.byref(args), _arg(y, shape, kind, "y", x), _arg(total, shape, kind, "total", x),
            _arg(mean, lead, f32, "mean", x), _arg(rstd, lead, f32, "rstd", x), rows, width, DTYPES.get(kind, -1))
    return y, total, mean, rstd


def gated_norm_backward(dy, x, weight, bias, mean, rstd, *, gate=None, residual=None, scale=None, rms=False,
                        gate_after=False, dtotal=None, dx=None, dgate=None, dresidual=None, dweight=None,
                        dbias=None, dscale=None, workspace=None, stream=None):
    """Gradients of gated_norm from its inputs and statistics, given dy and dtotal (or None), those of
    y and total.  Returns (dx, dweight, dbias, dgate, dresidual, dscale): dgate None without a
    gate, dresidual and dscale None without a residual, dresidual dx itself without a scale.  dx, dgate and dresidual
    may each be dy, dtotal, x, gate or residual."""
    lead, rows, width, groups, inner, par = _gated_shape(x, (weight, bias, scale, dweight, dbias, dscale))
    shape, kind, f32 = x.shape, x.dtype, torch.float32
    grads = (_arg(dy, shape, kind, "dy", x), _arg(dtotal, shape, kind, "dtotal", x), _arg(x, shape, kind, "x", x))
    args = fw_gated(_arg(gate, shape, kind, "gate", x), _arg(residual, shape, kind, "residual", x),
                    _arg(scale, par, f32, "scale", x), _arg(weight, par, f32, "weight", x),
                    _arg(bias, par, f32, "bias", x), groups, inner, 0.0, int(rms), int(gate_after))
    stats = (_arg(None if rms else mean, lead, f32, "mean", x), _arg(rstd, lead, f32, "rstd", x))
    on = _On(x, stream)
    if dx is None:
        dx = on.same(x)
    if dgate is None and gate is not None:
        dgate = on.same(x)
    if residual is not None and scale is not None:
        if dresidual is None:
            dresidual = on.same(x)
        if dscale is None:
            dscale = on.new(par, f32)
    if dweight is None:
        dweight = on.new(par, f32)
    if dbias is None:
        dbias = on.new(par, f32)
    _keep, ws, nws = on.workspace(workspace, _gated_need(rows, width, groups, DTYPES.get(kind, -1)),
                                  "fw_gated_norm_backward")
    on.call(lib().fw_gated_norm_backward, "fw_gated_norm_backward",
            (dy, dtotal, x, gate, residual, scale, weight, bias, mean, rstd, dx, dgate, dresidual, dweight, dbias,
             dscale, workspace),
            *grads, ctypes.byref(args), *stats, _arg(dx, shape, kind, "dx", x), _arg(dgate, shape, kind, "dgate", x),
            _arg(dresidual, shape, kind, "dresidual", x), _arg(dweight, par, f32, "dweight", x),
            _arg(dbias, par, f32, "dbias", x), _arg(dscale, par, f32, "dscale", x), rows, width,
            DTYPES.get(kind, -1), ws, nws)
    return dx, dweight, dbias, dgate, dx if residual is not None and dresidual is None else dresidual, dscale


def _finite_eps(eps):
    if not 0.0 <= ctypes.c_float(eps).value < float("inf"):
        raise ValueError("fw: eps must be finite and not negative")


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, y=None, mean=None, rstd=None, stats=True,
               stream=None):
    """Layer norm over the last axis of x (fp32 or bf16, contiguous); weight,
    bias [width] fp32 or None; y may be x.  Returns (y, mean, rstd), the
    statistics fp32 of x's leading shape (None with stats=False)."""
    if x.dim() < 1:
        raise ValueError("fw: layer_norm needs at least one axis")
    shape, dt, f32 = x.shape, x.dtype, torch.float32
    lead, width = shape[:-1], shape[-1]
    args = (_arg(x, shape, dt, "x", x), _arg(weight, (width,), f32, "weight", x),
            _arg(bias, (width,), f32, "bias", x))
    on = _On(x, stream)
    if y is None:
        y = on.new(shape, dt)
    if not stats:
        mean = rstd = None
    else:
        if mean is None:
            mean = on.new(lead, f32)
        if rstd is None:
            rstd = on.new(lead, f32)
    on.call(lib().fw_layer_norm, "fw_layer_norm", (x, weight, bias, y, mean, rstd), *args,
            _arg(y, shape, dt, "y", x), _arg(mean, lead, f32, "mean", x), _arg(rstd, lead, f32, "rstd", x),
            lead.numel(), width, DTYPES.get(dt, -1), eps)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, *, dx=None, dweight=None, dbias=None,
                        workspace=None, stream=None):
    """Gradients of layer_norm given dy (x's shape and dtype) and the forward
    pass's mean and rstd; weight None: ones.  dx may be dy or x.  Returns
    (dx, dweight, dbias), the last two fp32 [width]."""
    if x.dim() < 1:
        raise ValueError("fw: layer_norm needs at least one axis")
    shape, dt, f32 = x.shape, x.dtype, torch.float32
    lead, width = shape[:-1], shape[-1]
    rows = lead.numel()
    args = (_arg(dy, shape, dt, "dy", x), _arg(x, shape, dt, "x", x),
            _arg(weight, (width,), f32, "weight", x), _arg(mean, lead, f32, "mean", x),
            _arg(rstd, lead, f32, "rstd", x))
    on = _On(x, stream)
    if dx is None:
        dx = on.new(shape, dt)
    if dweight is None:
        dweight = on.new((width,), f32)
    if dbias is None:
        dbias = on.new((width,), f32)
    _keep, ws, nws = on.workspace(workspace, _layer_norm_need(rows, width), "fw_layer_norm_backward")
    on.call(lib().fw_layer_norm_backward, "fw_layer_norm_backward",
            (dy, x, weight, mean, rstd, dx, dweight, dbias, workspace), *args,
            _arg(dx, shape, dt, "dx", x), _arg(dweight, (width,), f32, "dweight", x),
            _arg(dbias, (width,), f32, "dbias", x), rows, width, DTYPES.get(dt, -1), ws, nws)
    return dx, dweight, dbias


def _overlap(a, b):
    x, y = a.data_ptr(), b.data_ptr()
    return x < y + b.numel() * b.element_size() and y < x + a.numel() * a.element_size()


def _norm_ready(norm, eps, q, o, stream, *written):
    """Refuse an output norm that _with_norm could not apply to the rows of o (written: what else the
    call writes).  Called before any state moves, so that a refused call has done nothing."""
    if norm is None:
        return
    _norm(norm, eps, q.shape[-1], q)
    _arg(o, q.shape, q.dtype, "o", q)
    _On(q, stream)
    for t in norm:
        if t is not None and t.data_ptr() % 16:
            raise FwError(-4, "fw_layer_norm")
        if t is not None and any(_overlap(t, z) for z in (o, *written)):
            raise FwError(-9, "fw_layer_norm")


def _with_norm(o, norm, norm_eps, stream):
    """The output norm of the other paths: in place over the rows of o."""
    if norm is not None:
        weight, bias = norm
        layer_norm(o, weight, bias, eps=norm_eps, y=o, stats=False, stream=stream)
    return o


def check(stream=None):
    """Synchronise the stream and raise if a bounded device wait ran out."""
    st = lib().fw_check(_stream(stream))
    if st != FW_OK:
        raise FwError(st, "fw_check")
