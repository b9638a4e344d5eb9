"""Python binding of libswinwattn.so: argument marshalling only.

Same names as the C ABI in include/swin_wattn.h and include/swin_seqattn.h. Every step of the
computation runs in the library's CUDA kernels; this module checks tensor
devices, dtypes and contiguity, passes raw pointers and the current CUDA
stream, and turns negative status codes into exceptions. torch is used for
device memory and streams only. There is no fallback: if the library is
missing, the first call raises.
"""
import contextlib
import ctypes
import os

import torch

from .workloads import Workload

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libswinwattn.so")

SWIN_OK = 0
SWIN_ERR_TIMEOUT = -5
SWIN_DTYPE_F32 = 0
SWIN_DTYPE_BF16 = 1
SWIN_FLAG_FORCE_GENERIC = 1
SWIN_FLAG_TEST_TIMEOUT = 2
SWIN_FLAG_FORCE_TILED = 4
SWIN_FLAG_DBIAS_SUMS = 8
SWIN_FLAG_KV_WEIGHTS = 256

EXPORTED = ("swin_wattn_path", "swin_wattn_workspace_size", "swin_wattn_fwd", "swin_wattn_bwd",
            "swin_wattn_bwd_noalloc", "swin_wattn_index_map", "swin_wattn_layout_map",
            "swin_wattn_dbias_sums", "swin_wattn_dbias_finish", "swin_wattn_fwd_band",
            "swin_wattn_bwd_band", "swin_wattn_poll_status",
            "swin_wattn_strerror", "swin_wattn_launch_count",
            "swin_seqattn_path", "swin_seqattn_workspace_size", "swin_seqattn_fwd",
            "swin_seqattn_bwd", "swin_kvcache_workspace_size", "swin_kvcache_append",
            "swin_kvcache_decode", "swin_kvcache_evict")
SWIN_NOALLOC_SCRATCH_BYTES = 1 << 20   # include/swin_wattn.h


class SwinWattnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "H", "W", "win_h", "win_w", "shift_h", "shift_w", "heads", "head_dim",
                 "dtype", "flags", "valid_h", "valid_w")]


class SwinWattnHalo(ctypes.Structure):
    """Halo rows of a row band (include/swin_wattn.h): inputs below the band
    and the outputs that belong to the next band."""
    _fields_ = [("interior", ctypes.c_int32), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("dout", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
                ("dv", ctypes.c_void_p)]


class SwinSeqattnDesc(ctypes.Structure):
    """Attention along a token sequence (include/swin_seqattn.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "S", "heads", "kv_heads", "head_dim", "window", "sinks", "dtype", "flags",
                 "q_stride", "kv_stride")]


class SwinKvcacheDesc(ctypes.Structure):
    """Paged key-value cache (include/swin_seqattn.h)."""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "heads", "kv_heads", "head_dim", "page_size", "num_pages", "max_pages",
                 "window", "sinks", "recent", "budget", "dtype", "flags", "q_stride",
                 "kv_stride")]


class SwinWattnError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: status %d (%s)" % (what, status, swin_wattn_strerror(status)))


_lib = None


def lib():
    """Load libswinwattn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libswinwattn.so not built: run __graft_entry__.build() "
                              "(or python shifted_window_attention_pad_b200/build.py)")
        L = ctypes.CDLL(LIB_PATH)
        D = ctypes.POINTER(SwinWattnDesc)
        P = ctypes.c_void_p
        L.swin_wattn_path.argtypes = [D]
        L.swin_wattn_workspace_size.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
        L.swin_wattn_fwd.argtypes = [D, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.swin_wattn_bwd.argtypes = [D, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.swin_wattn_bwd_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P, P]
        L.swin_wattn_index_map.argtypes = [D, P, P]
        L.swin_wattn_layout_map.argtypes = [D, P, P, P, P]
        L.swin_wattn_dbias_sums.argtypes = [D, ctypes.POINTER(ctypes.c_size_t),
                                            ctypes.POINTER(ctypes.c_size_t)]
        L.swin_wattn_dbias_finish.argtypes = [D, P, P, P]
        HP = ctypes.POINTER(SwinWattnHalo)
        L.swin_wattn_fwd_band.argtypes = [D, HP, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.swin_wattn_bwd_band.argtypes = [D, HP, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.swin_wattn_poll_status.argtypes = [P, ctypes.POINTER(ctypes.c_int), P]
        L.swin_wattn_strerror.argtypes = [ctypes.c_int]
        L.swin_wattn_strerror.restype = ctypes.c_char_p
        L.swin_wattn_launch_count.argtypes = []
        L.swin_wattn_launch_count.restype = ctypes.c_uint64
        for f in ("swin_wattn_path", "swin_wattn_workspace_size", "swin_wattn_fwd",
                  "swin_wattn_bwd", "swin_wattn_bwd_noalloc", "swin_wattn_index_map",
                  "swin_wattn_layout_map", "swin_wattn_dbias_sums", "swin_wattn_dbias_finish",
                  "swin_wattn_fwd_band", "swin_wattn_bwd_band", "swin_wattn_poll_status"):
            getattr(L, f).restype = ctypes.c_int
        Q, C, Z = ctypes.POINTER(SwinSeqattnDesc), ctypes.POINTER(SwinKvcacheDesc), ctypes.c_size_t
        for f, a in (("swin_seqattn_path", [Q]),
                     ("swin_seqattn_workspace_size", [Q, ctypes.POINTER(Z)]),
                     ("swin_seqattn_fwd", [Q] + [P] * 7 + [Z, P]),
                     ("swin_seqattn_bwd", [Q] + [P] * 11 + [Z, P]),
                     ("swin_kvcache_workspace_size", [C, ctypes.POINTER(Z)]),
                     ("swin_kvcache_append", [C, ctypes.c_int32] + [P] * 8 + [Z, P]),
                     ("swin_kvcache_decode", [C] + [P] * 12 + [Z, P]),
                     ("swin_kvcache_evict", [C] + [P] * 10 + [Z, P])):
            getattr(L, f).argtypes = a
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def make_desc(B, H, W, win, shift, heads, head_dim, dtype, flags=0, valid=None):
    """`valid` = (valid_h, valid_w), the extent of tokens that carry field data
    (None: the whole grid)."""
    wh, ww = (win, win) if isinstance(win, int) else win
    sh, sw = (shift, shift) if isinstance(shift, int) else shift
    dt = SWIN_DTYPE_BF16 if dtype in ("bf16", torch.bfloat16, SWIN_DTYPE_BF16) else SWIN_DTYPE_F32
    vh, vw = valid if valid is not None else (0, 0)
    return SwinWattnDesc(B, H, W, wh, ww, sh, sw, heads, head_dim, dt, flags, vh, vw)


def field_valid_extent(field_h, field_w, patch):
    """Valid token extent of a field of field_h x field_w real pixels cut into
    patch x patch tokens: a token is real when its patch holds a real pixel."""
    return -(-field_h // patch), -(-field_w // patch)


def desc_for(wl: Workload, flags=0):
    return make_desc(wl.B, wl.H, wl.W, wl.win, wl.shift, wl.heads, wl.head_dim, wl.dtype, flags,
                     wl.valid)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def _check(rc, what):
    if rc != SWIN_OK:
        raise SwinWattnError(rc, what)


def _elem(desc):
    return torch.bfloat16 if desc.dtype == SWIN_DTYPE_BF16 else torch.float32


def swin_wattn_strerror(status):
    return lib().swin_wattn_strerror(status).decode()


def swin_wattn_path(desc):
    rc = lib().swin_wattn_path(ctypes.byref(desc))
    if rc < 0:
        raise SwinWattnError(rc, "swin_wattn_path")
    return rc


def swin_wattn_workspace_size(desc):
    n = ctypes.c_size_t(0)
    _check(lib().swin_wattn_workspace_size(ctypes.byref(desc), ctypes.byref(n)),
           "swin_wattn_workspace_size")
    return n.value


def new_workspace(desc, device="cuda"):
    """Caller-owned workspace of the size the library asks for (zeroed once)."""
    return torch.zeros(swin_wattn_workspace_size(desc), dtype=torch.uint8, device=device)


def swin_wattn_fwd(desc, q, k, v, bias_table, out, lse=None, workspace=None, stream=None):
    el = _elem(desc)
    if workspace is None:
        workspace = new_workspace(desc, q.device)
    rc = lib().swin_wattn_fwd(ctypes.byref(desc), _ptr(q, el, "q"), _ptr(k, el, "k"),
                              _ptr(v, el, "v"), _ptr(bias_table, torch.float32, "bias_table"),
                              _ptr(out, el, "out"), _ptr(lse, torch.float32, "lse"),
                              _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                              _stream(stream))
    _check(rc, "swin_wattn_fwd")
    return out


def swin_wattn_bwd(desc, q, k, v, bias_table, dout, dq, dk, dv, dbias_table, workspace=None,
                   stream=None):
    el = _elem(desc)
    if workspace is None:
        workspace = new_workspace(desc, q.device)
    rc = lib().swin_wattn_bwd(ctypes.byref(desc), _ptr(q, el, "q"), _ptr(k, el, "k"),
                              _ptr(v, el, "v"), _ptr(bias_table, torch.float32, "bias_table"),
                              _ptr(dout, el, "dout"), _ptr(dq, el, "dq"), _ptr(dk, el, "dk"),
                              _ptr(dv, el, "dv"), _ptr(dbias_table, torch.float32, "dbias_table"),
                              _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                              _stream(stream))
    _check(rc, "swin_wattn_bwd")
    return dq, dk, dv, dbias_table


def make_halo(interior, q=None, k=None, v=None, dout=None, out=None, lse=None, dq=None, dk=None,
              dv=None):
    """SwinWattnHalo from device tensors ([B, shift_h, W, heads, head_dim])."""
    p = lambda t, n: _ptr(t, None, n) if t is not None else None
    return SwinWattnHalo(int(interior), p(q, "halo q"), p(k, "halo k"), p(v, "halo v"),
                         p(dout, "halo dout"), p(out, "halo out"), p(lse, "halo lse"),
                         p(dq, "halo dq"), p(dk, "halo dk"), p(dv, "halo dv"))


def swin_wattn_fwd_band(desc, halo, q, k, v, bias_table, out, lse=None, workspace=None,
                        stream=None):
    el = _elem(desc)
    if workspace is None:
        workspace = new_workspace(desc, q.device)
    rc = lib().swin_wattn_fwd_band(ctypes.byref(desc), ctypes.byref(halo), _ptr(q, el, "q"),
                                   _ptr(k, el, "k"), _ptr(v, el, "v"),
                                   _ptr(bias_table, torch.float32, "bias_table"),
                                   _ptr(out, el, "out"), _ptr(lse, torch.float32, "lse"),
                                   _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                   _stream(stream))
    _check(rc, "swin_wattn_fwd_band")
    return out


def swin_wattn_bwd_band(desc, halo, q, k, v, bias_table, dout, dq, dk, dv, dbias_table,
                        workspace=None, stream=None):
    el = _elem(desc)
    if workspace is None:
        workspace = new_workspace(desc, q.device)
    rc = lib().swin_wattn_bwd_band(ctypes.byref(desc), ctypes.byref(halo), _ptr(q, el, "q"),
                                   _ptr(k, el, "k"), _ptr(v, el, "v"),
                                   _ptr(bias_table, torch.float32, "bias_table"),
                                   _ptr(dout, el, "dout"), _ptr(dq, el, "dq"), _ptr(dk, el, "dk"),
                                   _ptr(dv, el, "dv"),
                                   _ptr(dbias_table, torch.float32, "dbias_table"),
                                   _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                   _stream(stream))
    _check(rc, "swin_wattn_bwd_band")
    return dq, dk, dv, dbias_table


def swin_wattn_bwd_noalloc(desc, q, k, v, bias_table, dout, dq, dk, dv, dbias_table,
                           stream=None):
    """swin_wattn_bwd with the library's static scratch instead of a workspace
    (for callers that cannot allocate; see include/swin_wattn.h)."""
    el = _elem(desc)
    rc = lib().swin_wattn_bwd_noalloc(ctypes.byref(desc), _ptr(q, el, "q"), _ptr(k, el, "k"),
                                      _ptr(v, el, "v"),
                                      _ptr(bias_table, torch.float32, "bias_table"),
                                      _ptr(dout, el, "dout"), _ptr(dq, el, "dq"),
                                      _ptr(dk, el, "dk"), _ptr(dv, el, "dv"),
                                      _ptr(dbias_table, torch.float32, "dbias_table"),
                                      _stream(stream))
    _check(rc, "swin_wattn_bwd_noalloc")
    return dq, dk, dv, dbias_table


def swin_wattn_index_map(desc, out=None, stream=None):
    if out is None:
        Hp = -(-desc.H // desc.win_h) * desc.win_h
        Wp = -(-desc.W // desc.win_w) * desc.win_w
        out = torch.empty((desc.B, Hp // desc.win_h, Wp // desc.win_w, desc.win_h * desc.win_w),
                          dtype=torch.int32, device="cuda")
    _check(lib().swin_wattn_index_map(ctypes.byref(desc), _ptr(out, torch.int32, "map"),
                                      _stream(stream)), "swin_wattn_index_map")
    return out


def swin_wattn_dbias_sums(desc):
    """(offset, bytes) of the exact bias-gradient sums in the workspace."""
    off, n = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().swin_wattn_dbias_sums(ctypes.byref(desc), ctypes.byref(off), ctypes.byref(n)),
           "swin_wattn_dbias_sums")
    return off.value, n.value


def dbias_sums_view(desc, workspace):
    """The exact sums inside `workspace` as an int64 tensor (a view, no copy)."""
    off, n = swin_wattn_dbias_sums(desc)
    return workspace[off:off + n].view(torch.int64)


def swin_wattn_dbias_finish(desc, workspace, dbias_table, stream=None):
    _check(lib().swin_wattn_dbias_finish(ctypes.byref(desc),
                                         _ptr(workspace, torch.uint8, "workspace"),
                                         _ptr(dbias_table, torch.float32, "dbias_table"),
                                         _stream(stream)), "swin_wattn_dbias_finish")
    return dbias_table


def swin_wattn_layout_map(desc, stream=None):
    """(map, labels) of the tcgen05 kernels' own layout stage, both int32
    [B, H^/win_h, W^/win_w, win_h*win_w] on the device."""
    Hp = -(-desc.H // desc.win_h) * desc.win_h
    Wp = -(-desc.W // desc.win_w) * desc.win_w
    shape = (desc.B, Hp // desc.win_h, Wp // desc.win_w, desc.win_h * desc.win_w)
    ids = torch.empty(desc.B * desc.H * desc.W * desc.heads * desc.head_dim, dtype=torch.bfloat16,
                      device="cuda")
    m = torch.empty(shape, dtype=torch.int32, device="cuda")
    lab = torch.empty(shape, dtype=torch.int32, device="cuda")
    _check(lib().swin_wattn_layout_map(ctypes.byref(desc), _ptr(ids, torch.bfloat16, "ids"),
                                       _ptr(m, torch.int32, "map"), _ptr(lab, torch.int32, "labels"),
                                       _stream(stream)), "swin_wattn_layout_map")
    return m, lab


def swin_wattn_poll_status(workspace, stream=None):
    st = ctypes.c_int(0)
    _check(lib().swin_wattn_poll_status(_ptr(workspace, torch.uint8, "workspace"),
                                        ctypes.byref(st), _stream(stream)),
           "swin_wattn_poll_status")
    return st.value


def swin_wattn_launch_count():
    return int(lib().swin_wattn_launch_count())


# ---- convenience wrappers (allocate outputs with torch, then call the ABI) -------
def forward(desc, q, k, v, bias_table, want_lse=False, workspace=None):
    out = torch.empty_like(q)
    lse = (torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if want_lse else None)
    swin_wattn_fwd(desc, q, k, v, bias_table, out, lse, workspace)
    return (out, lse) if want_lse else out


def backward(desc, q, k, v, bias_table, dout, workspace=None):
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dT = torch.empty_like(bias_table)
    swin_wattn_bwd(desc, q, k, v, bias_table, dout, dq, dk, dv, dT, workspace)
    return dq, dk, dv, dT


# ---- attention along a token sequence and its paged cache (include/swin_seqattn.h) ----
# These calls run on the device their tensors are on (all on one), whatever the
# current device is, and on `stream` or that device's current stream.
def _dtype_code(dtype):
    if dtype in ("bf16", torch.bfloat16, SWIN_DTYPE_BF16):
        return SWIN_DTYPE_BF16
    if dtype in ("f32", torch.float32, SWIN_DTYPE_F32):
        return SWIN_DTYPE_F32
    raise ValueError("dtype must be bf16 or f32, got %r" % (dtype,))


def make_seq_desc(B, S, heads, head_dim, window, dtype, kv_heads=None, sinks=0, flags=0,
                  q_stride=0, kv_stride=0):
    """window 0: every earlier token is visible; kv_heads None: one per query
    head; strides in elements between tokens, 0: contiguous."""
    return SwinSeqattnDesc(B, S, heads, heads if kv_heads is None else kv_heads, head_dim, window,
                           sinks, _dtype_code(dtype), flags, q_stride, kv_stride)


def _token_stride(t):
    """Elements from token to token of [B, S, heads, hd], 0 if contiguous."""
    n = t.shape[2] * t.shape[3]
    s = t.stride(1) if t.shape[1] > 1 else (t.stride(0) if t.shape[0] > 1 else n)
    return 0 if s == n else s


def seq_desc_for(q, k, window, sinks=0, flags=0):
    """Description of tensors q [B, S, heads, hd] and k (or v)
    [B, S, kv_heads, hd], parts of a wider projection included."""
    return make_seq_desc(q.shape[0], q.shape[1], q.shape[2], q.shape[3], window, q.dtype,
                         k.shape[2], sinks, flags, _token_stride(q), _token_stride(k))


def _refuse(t, name, dtype, shape, dev):
    if t is None:
        raise ValueError("%s is missing" % name)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, the other tensors on cuda:%d"
                         % (name, t.get_device(), dev))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _device_of(t, name):
    """Device of a call's first tensor, which the others have to share."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.get_device()


def _dense(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this type and shape."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.is_contiguous() and t.get_device() == dev):
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev)


def _maybe(t, name, dtype, shape, dev):
    return None if t is None else _dense(t, name, dtype, shape, dev)


def _tokens(t, name, dtype, shape, stride, dev):
    """Address of [B, T, heads, hd] or [B, heads, hd] with tokens `stride` elements
    apart (0: contiguous)."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.get_device() == dev):
        _refuse(t, name, dtype, shape, dev)
    if not stride:
        if t.is_contiguous():
            return t.data_ptr()
        raise ValueError("%s has strides %s, the description says contiguous" % (name, t.stride()))
    want = ((shape[1] * stride, stride) if len(shape) == 4 else (stride,)) + (shape[-1], 1)
    have = t.stride()
    if have != want:   # a dimension of one entry has no stride
        for n, x, y in zip(shape, have, want):
            if n > 1 and x != y:
                raise ValueError("%s has strides %s, the description says %d between tokens"
                                 % (name, have, stride))
    return t.data_ptr()


def _run(name, fn, dev, workspace, stream, *args):
    """The call on device `dev` and its current stream (or `stream`)."""
    if (not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8
            or workspace.get_device() != dev or not workspace.is_contiguous()):
        _refuse(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)   # current_stream(dev).cuda_stream
    elif stream.device.index != dev:
        raise ValueError("the stream is on %s, the tensors on cuda:%d" % (stream.device, dev))
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, workspace.data_ptr(), workspace.numel(), handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, workspace.data_ptr(), workspace.numel(), handle)
    if rc != SWIN_OK:
        raise SwinWattnError(rc, name)


def swin_seqattn_path(desc):
    rc = lib().swin_seqattn_path(ctypes.byref(desc))
    if rc < 0:
        raise SwinWattnError(rc, "swin_seqattn_path")
    return rc


def _workspace_size(name, desc):
    n = ctypes.c_size_t(0)
    _check(getattr(lib(), name)(ctypes.byref(desc), ctypes.byref(n)), name)
    return n.value


def swin_seqattn_workspace_size(desc):
    return _workspace_size("swin_seqattn_workspace_size", desc)


def swin_kvcache_workspace_size(desc):
    return _workspace_size("swin_kvcache_workspace_size", desc)


def _new_ws(size, device, stream=None):
    """Only the header (the device status word) has to start as zeros. With a
    stream: allocated and zeroed on it, so that the memory is not handed on
    while the stream still works in it."""
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        ws[:256].zero_()
    return ws


def new_seq_workspace(desc, device="cuda"):
    """Caller-owned workspace of the size the library asks for."""
    return _new_ws(swin_seqattn_workspace_size(desc), device)


def new_cache_workspace(desc, device="cuda"):
    """Caller-owned workspace of the size the library asks for."""
    return _new_ws(swin_kvcache_workspace_size(desc), device)


def _seq_shapes(d):
    B, S, H, hd = d.B, d.S, d.heads, d.head_dim
    return (B, S, H, hd), (B, S, d.kv_heads, hd), (B, S, H)


def swin_seqattn_fwd(desc, q, k, v, lengths, out, lse=None, workspace=None, stream=None):
    el, dev = _elem(desc), _device_of(q, "q")
    sq, sk, sl = _seq_shapes(desc)
    qs, ks = desc.q_stride, desc.kv_stride
    args = (_tokens(q, "q", el, sq, qs, dev), _tokens(k, "k", el, sk, ks, dev),
            _tokens(v, "v", el, sk, ks, dev),
            _maybe(lengths, "lengths", torch.int32, (desc.B,), dev),
            _dense(out, "out", el, sq, dev), _maybe(lse, "lse", torch.float32, sl, dev))
    if workspace is None:
        workspace = _new_ws(swin_seqattn_workspace_size(desc), q.device, stream)
    _run("swin_seqattn_fwd", lib().swin_seqattn_fwd, dev, workspace, stream, desc, *args)
    return out


def swin_seqattn_bwd(desc, q, k, v, lengths, out, lse, dout, dq, dk, dv, workspace=None,
                     stream=None):
    el, dev = _elem(desc), _device_of(q, "q")
    sq, sk, sl = _seq_shapes(desc)
    qs, ks = desc.q_stride, desc.kv_stride
    args = (_tokens(q, "q", el, sq, qs, dev), _tokens(k, "k", el, sk, ks, dev),
            _tokens(v, "v", el, sk, ks, dev),
            _maybe(lengths, "lengths", torch.int32, (desc.B,), dev),
            _dense(out, "out", el, sq, dev), _dense(lse, "lse", torch.float32, sl, dev),
            _dense(dout, "dout", el, sq, dev), _tokens(dq, "dq", el, sq, qs, dev),
            _tokens(dk, "dk", el, sk, ks, dev), _tokens(dv, "dv", el, sk, ks, dev))
    if workspace is None:
        workspace = _new_ws(swin_seqattn_workspace_size(desc), q.device, stream)
    _run("swin_seqattn_bwd", lib().swin_seqattn_bwd, dev, workspace, stream, desc, *args)
    return dq, dk, dv


def seq_forward(desc, q, k, v, lengths=None, want_lse=False, workspace=None):
    sq, _, sl = _seq_shapes(desc)
    out = q.new_empty(sq) if desc.q_stride else torch.empty_like(q)
    lse = q.new_empty(sl, dtype=torch.float32) if want_lse else None
    swin_seqattn_fwd(desc, q, k, v, lengths, out, lse, workspace)
    return (out, lse) if want_lse else out


def seq_backward(desc, q, k, v, out, lse, dout, lengths=None, workspace=None):
    """dq, dk, dv, laid out as the description lays out q, k and v: parts of one
    [B, S, heads + 2 kv_heads, hd] buffer when its strides are that buffer's."""
    B, S, H, K, hd = desc.B, desc.S, desc.heads, desc.kv_heads, desc.head_dim
    if desc.q_stride and desc.q_stride == desc.kv_stride == (H + 2 * K) * hd:
        both = q.new_empty((B, S, H + 2 * K, hd))
        dq, dk, dv = both[:, :, :H], both[:, :, H:H + K], both[:, :, H + K:]
    else:
        wide = lambda t, n, s: (torch.empty_like(t) if not s else
                                q.new_empty((B, S, s))[:, :, :n * hd].unflatten(2, (n, hd)))
        dq = wide(q, H, desc.q_stride)
        dk, dv = wide(k, K, desc.kv_stride), wide(v, K, desc.kv_stride)
    return swin_seqattn_bwd(desc, q, k, v, lengths, out, lse, dout, dq, dk, dv, workspace)


def make_cache_desc(B, heads, head_dim, page_size, num_pages, max_pages, dtype, kv_heads=None,
                    window=0, sinks=0, recent=0, budget=0, weights=False, q_stride=0,
                    kv_stride=0):
    """weights: cache_decode will accumulate attention weights."""
    return SwinKvcacheDesc(B, heads, heads if kv_heads is None else kv_heads, head_dim, page_size,
                           num_pages, max_pages, window, sinks, recent, budget,
                           _dtype_code(dtype), SWIN_FLAG_KV_WEIGHTS if weights else 0, q_stride,
                           kv_stride)


def _cache_args(d, el, dev, lengths, page_table, k_cache, v_cache):
    cache = (d.num_pages, d.kv_heads, d.page_size, d.head_dim)
    return (_dense(lengths, "lengths", torch.int32, (d.B,), dev),
            _dense(page_table, "page_table", torch.int32, (d.B, d.max_pages), dev),
            _dense(k_cache, "k_cache", el, cache, dev), _dense(v_cache, "v_cache", el, cache, dev))


def swin_kvcache_append(desc, k, v, counts, lengths, page_table, k_cache, v_cache,
                        workspace=None, stream=None):
    """k, v: [B, T, kv_heads, head_dim]."""
    d, el, dev = desc, _elem(desc), _device_of(k, "k")
    T = k.shape[1] if k.dim() == 4 else 0
    shape, ks = (d.B, T, d.kv_heads, d.head_dim), d.kv_stride
    args = (T, _tokens(k, "k", el, shape, ks, dev), _tokens(v, "v", el, shape, ks, dev),
            _maybe(counts, "counts", torch.int32, (d.B,), dev),
            *_cache_args(d, el, dev, lengths, page_table, k_cache, v_cache))
    if workspace is None:
        workspace = _new_ws(256, k.device, stream)
    _run("swin_kvcache_append", lib().swin_kvcache_append, dev, workspace, stream, d, *args)


def swin_kvcache_decode(desc, q, k_new, v_new, lengths, page_table, k_cache, v_cache, weights,
                        new_weights, out, lse=None, workspace=None, stream=None):
    d, el, dev = desc, _elem(desc), _device_of(q, "q")
    B, H = d.B, d.heads
    so, sk, ks = (B, H, d.head_dim), (B, d.kv_heads, d.head_dim), d.kv_stride
    sw = (B, d.kv_heads, d.max_pages * d.page_size)
    args = (_tokens(q, "q", el, so, d.q_stride, dev),
            None if k_new is None else _tokens(k_new, "k_new", el, sk, ks, dev),
            None if v_new is None else _tokens(v_new, "v_new", el, sk, ks, dev),
            *_cache_args(d, el, dev, lengths, page_table, k_cache, v_cache),
            _maybe(weights, "weights", torch.float32, sw, dev),
            _maybe(new_weights, "new_weights", torch.float32, sw, dev),
            _dense(out, "out", el, so, dev), _maybe(lse, "lse", torch.float32, (B, H), dev))
    if workspace is None:
        workspace = _new_ws(swin_kvcache_workspace_size(d), q.device, stream)
    _run("swin_kvcache_decode", lib().swin_kvcache_decode, dev, workspace, stream, d, *args)
    return out


def swin_kvcache_evict(desc, weights, lengths, page_table, dst_page_table, k_cache, v_cache,
                       new_weights, new_lengths, kept=None, workspace=None, stream=None):
    d, el, dev = desc, _elem(desc), _device_of(weights, "weights")
    sw = (d.B, d.kv_heads, d.max_pages * d.page_size)
    n, t, kc, vc = _cache_args(d, el, dev, lengths, page_table, k_cache, v_cache)
    args = (_dense(weights, "weights", torch.float32, sw, dev), n, t,
            _dense(dst_page_table, "dst_page_table", torch.int32, (d.B, d.max_pages), dev), kc, vc,
            _dense(new_weights, "new_weights", torch.float32, sw, dev),
            _dense(new_lengths, "new_lengths", torch.int32, (d.B,), dev),
            _maybe(kept, "kept", torch.int32, (d.B, d.kv_heads, d.budget), dev))
    if workspace is None:
        workspace = _new_ws(swin_kvcache_workspace_size(d), weights.device, stream)
    _run("swin_kvcache_evict", lib().swin_kvcache_evict, dev, workspace, stream, d, *args)
    return new_weights, new_lengths


def cache_append(desc, k, v, lengths, page_table, k_cache, v_cache, counts=None, workspace=None):
    """Writes tokens k, v [B, T, kv_heads, hd] to the cache's last positions;
    `lengths` already counts them."""
    swin_kvcache_append(desc, k, v, counts, lengths, page_table, k_cache, v_cache, workspace)


def cache_decode(desc, q, lengths, page_table, k_cache, v_cache, k_new=None, v_new=None,
                 weights=None, new_weights=None, want_lse=False, workspace=None):
    """Attention of one token per sequence, q [B, heads, hd], over the cache.
    With `weights` and no new_weights the step's weights are added in place."""
    out = (q.new_empty((desc.B, desc.heads, desc.head_dim)) if desc.q_stride
           else torch.empty_like(q))
    lse = q.new_empty((desc.B, desc.heads), dtype=torch.float32) if want_lse else None
    if weights is not None and new_weights is None:
        new_weights = weights
    swin_kvcache_decode(desc, q, k_new, v_new, lengths, page_table, k_cache, v_cache, weights,
                        new_weights, out, lse, workspace)
    return (out, lse) if want_lse else out


def cache_evict(desc, weights, lengths, page_table, dst_page_table, k_cache, v_cache,
                new_weights=None, new_lengths=None, kept=None, workspace=None):
    """Copies the positions that stay to dst_page_table's pages; returns
    (new_weights, new_lengths)."""
    if new_weights is None:
        new_weights = torch.empty_like(weights)
    if new_lengths is None:
        new_lengths = torch.empty_like(lengths)
    return swin_kvcache_evict(desc, weights, lengths, page_table, dst_page_table, k_cache, v_cache,
                              new_weights, new_lengths, kept, workspace)
