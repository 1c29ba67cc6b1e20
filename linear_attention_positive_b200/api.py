"""ctypes binding of libfavor.so (C ABI in include/favor.h): argument marshalling only.

Every computation runs in the library's kernels; PyTorch provides device memory and streams.
The library is loaded on first use; if it is missing this raises ``FavorError`` (there is no CPU
fallback).
"""

import ctypes
import functools
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfavor.so")

FAVOR_OK = 0
FAVOR_ERR_INVALID_ARG = 1
FAVOR_ERR_UNSUPPORTED = 2
FAVOR_ERR_CUDA = 3
FAVOR_ERR_TIMEOUT = 4
FAVOR_ERR_WORKSPACE = 5
FAVOR_F32 = 0
FAVOR_BF16 = 1

# Exported entry points, in the order include/favor.h declares them.
EXPORTS = (
    "favor_draw_features",
    "favor_workspace_size",
    "favor_ctx_size",
    "favor_fwd",
    "favor_bwd",
    "favor_sync_status",
    "favor_status_string",
    "favor_sp_state_size",
    "favor_sp_workspace_size",
    "favor_sp_state",
    "favor_sp_output",
    "favor_decode_state_size",
    "favor_decode_step",
    "favor_decode_tree",
    "favor_decode_extend_workspace_size",
    "favor_decode_extend",
    "favor_decode_verify",
    "favor_selftest_bounded_wait",
    "favor_fwd_static_scratch",
)


class FavorError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        msg = status_string(status) if _LIB is not None else f"status {status}"
        super().__init__(f"{what}: {msg}" if what else msg)


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int), ("d", ctypes.c_int),
                ("m", ctypes.c_int), ("dtype", ctypes.c_int)]


class VerifyShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("V", ctypes.c_int), ("dtype", ctypes.c_int)]


FAVOR_MAX_STAGES = 24
FAVOR_TREE_MAX_NODES = 128


FAVOR_MAP_POSITIVE = 0
FAVOR_MAP_RELU = 1
FAVOR_MAP_TRIG = 2


class Opts(ctypes.Structure):
    _fields_ = [("split_tiles", ctypes.c_int), ("exp_poly_pct", ctypes.c_int), ("feature_map", ctypes.c_int),
                ("reserved", ctypes.c_int * 5), ("stage_events", ctypes.POINTER(ctypes.c_void_p))]


_LIB = None


def library():
    """The loaded libfavor.so (ctypes.CDLL) with argument types declared."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise FavorError(FAVOR_ERR_CUDA, f"{LIB_PATH} is not built (run linear_attention_positive_b200.build)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
    SP, OP = ctypes.POINTER(Shape), ctypes.POINTER(Opts)
    lib.favor_draw_features.argtypes = [U64, I, I, ctypes.POINTER(ctypes.c_double)]
    lib.favor_draw_features.restype = I
    lib.favor_workspace_size.argtypes = [SP, I, I, OP]
    lib.favor_workspace_size.restype = Z
    lib.favor_ctx_size.argtypes = [SP, I]
    lib.favor_ctx_size.restype = Z
    lib.favor_fwd.argtypes = [SP, P, P, P, P, I, P, P, P, Z, OP, P]
    lib.favor_fwd.restype = I
    lib.favor_bwd.argtypes = [SP, P, P, P, P, P, P, P, I, P, P, P, P, Z, OP, P]
    lib.favor_bwd.restype = I
    lib.favor_sync_status.argtypes = [P]
    lib.favor_sync_status.restype = I
    lib.favor_status_string.argtypes = [I]
    lib.favor_status_string.restype = ctypes.c_char_p
    lib.favor_sp_state_size.argtypes = [SP]
    lib.favor_sp_state_size.restype = Z
    lib.favor_sp_workspace_size.argtypes = [SP]
    lib.favor_sp_workspace_size.restype = Z
    lib.favor_sp_state.argtypes = [SP, P, P, P, P, P, Z, P]
    lib.favor_sp_state.restype = I
    lib.favor_sp_output.argtypes = [SP, P, P, P, P, P, Z, P]
    lib.favor_sp_output.restype = I
    lib.favor_decode_state_size.argtypes = [SP]
    lib.favor_decode_state_size.restype = Z
    lib.favor_decode_step.argtypes = [SP, P, P, P, P, P, P, P]
    lib.favor_decode_step.restype = I
    lib.favor_decode_tree.argtypes = [SP, P, P, P, P, P, P, P, P, P]
    lib.favor_decode_tree.restype = I
    lib.favor_decode_extend_workspace_size.argtypes = [SP, I]
    lib.favor_decode_extend_workspace_size.restype = Z
    lib.favor_decode_extend.argtypes = [SP, P, P, P, P, I, P, P, P, Z, P]
    lib.favor_decode_extend.restype = I
    lib.favor_decode_verify.argtypes = [ctypes.POINTER(VerifyShape), P, P, P, P, P, P, P, P, P, P, P]
    lib.favor_decode_verify.restype = I
    lib.favor_selftest_bounded_wait.argtypes = [ctypes.c_uint, P]
    lib.favor_selftest_bounded_wait.restype = I
    lib.favor_fwd_static_scratch.argtypes = [SP, P, P, P, P, P, P]
    lib.favor_fwd_static_scratch.restype = I
    _LIB = lib
    return lib


def status_string(status):
    return library().favor_status_string(int(status)).decode()


def _check(status, what):
    if status != FAVOR_OK:
        raise FavorError(status, what)


def make_shape(B, H, L, d, m, dtype):
    return Shape(B, H, L, d, m, dtype)


def make_opts(split_tiles=0, exp_poly_pct=0, stage_events=None, feature_map=FAVOR_MAP_POSITIVE):
    """Options struct. ``stage_events``: optional list of 2*FAVOR_MAX_STAGES torch.cuda.Event
    (enable_timing=True, already recorded once so their handles exist) or None entries."""
    o = Opts(split_tiles, exp_poly_pct, feature_map, (ctypes.c_int * 5)(), None)
    if stage_events is not None:
        arr = (ctypes.c_void_p * (2 * FAVOR_MAX_STAGES))()
        for i, ev in enumerate(stage_events[: 2 * FAVOR_MAX_STAGES]):
            arr[i] = ev.cuda_event if ev is not None else None
        o._events_keepalive = arr
        o.stage_events = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
    return o


def draw_features(seed, m, d):
    """Block-orthogonal random features W (m x d, float64), drawn on the host by the library."""
    out = np.empty((m, d), dtype=np.float64)
    st = library().favor_draw_features(ctypes.c_uint64(seed & (2**64 - 1)), int(m), int(d),
                                       out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)))
    _check(st, "favor_draw_features")
    return out


def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return FAVOR_BF16
    if t.dtype == torch.float32:
        return FAVOR_F32
    raise FavorError(FAVOR_ERR_INVALID_ARG, f"unsupported dtype {t.dtype}")


def _shape_of(Q, W):
    B, H, L, d = Q.shape
    return make_shape(B, H, L, d, W.shape[0], _dtype_code(Q))


def workspace_size(shape, causal=False, backward=False, opts=None):
    return library().favor_workspace_size(ctypes.byref(shape), int(causal), int(backward),
                                          ctypes.byref(opts) if opts is not None else None)


def ctx_size(shape, causal=False):
    return library().favor_ctx_size(ctypes.byref(shape), int(causal))


def _stream_ptr(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _empty(size, dtype, device, stream, returned=True):
    """A tensor for a call on ``stream`` (None: the current one). It comes from that stream's memory: a block
    just freed on another may still be in use there, by work this stream does not wait for. One that is
    returned is used on the current stream next, so it must not be handed out before that is done with it."""
    torch = _torch()
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    if stream.device != device:
        raise FavorError(FAVOR_ERR_INVALID_ARG, f"stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        t = torch.empty(size, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _alloc_bytes(n, device, stream=None):
    return _empty(max(int(n), 256), _torch().uint8, device, stream, returned=False)


def _workspace_bytes(workspace, device):
    """Bytes of a caller's workspace, which must be contiguous memory of the tensors' device."""
    if workspace.device != device or not workspace.is_contiguous():
        raise FavorError(FAVOR_ERR_INVALID_ARG, f"workspace must be a contiguous tensor on {device}")
    return workspace.numel() * workspace.element_size()


def _check_inputs(tensors, dtype_like):
    for t in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise FavorError(FAVOR_ERR_INVALID_ARG, "tensors must be contiguous CUDA tensors")
        if t.dtype != dtype_like.dtype:
            raise FavorError(FAVOR_ERR_INVALID_ARG, "Q, K, V, W (and dout) must share one dtype")


def fwd(Q, K, V, W, causal=False, out=None, ctx=None, workspace=None, opts=None, stream=None):
    """FAVOR+ forward through favor_fwd. Q, K, V: [B,H,L,d] bf16 or fp32 CUDA tensors; W: [m,d] in
    the same dtype. Returns the fp32 output (and fills ``ctx`` when given)."""
    torch = _torch()
    _check_inputs((Q, K, V, W), Q)
    shape = _shape_of(Q, W)
    if out is None:
        out = _empty(Q.shape, torch.float32, Q.device, stream)
    if workspace is None:
        ws_n = workspace_size(shape, causal, False, opts)
        if ws_n == 0:
            raise FavorError(FAVOR_ERR_UNSUPPORTED, "favor_workspace_size")
        workspace = _alloc_bytes(ws_n, Q.device, stream)
    st = library().favor_fwd(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(W), int(causal), _ptr(out),
                             _ptr(ctx), _ptr(workspace), _workspace_bytes(workspace, Q.device),
                             ctypes.byref(opts) if opts is not None else None, _stream_ptr(stream))
    _check(st, "favor_fwd")
    return out


def bwd(Q, K, V, W, out, dout, ctx=None, causal=False, workspace=None, opts=None, stream=None):
    """Gradients (dQ, dK, dV) (fp32) of sum(dout * out) through favor_bwd, W fixed."""
    torch = _torch()
    _check_inputs((Q, K, V, W, dout), Q)
    shape = _shape_of(Q, W)
    dQ, dK, dV = (_empty(Q.shape, torch.float32, Q.device, stream) for _ in range(3))
    if workspace is None:
        ws_n = workspace_size(shape, causal, True, opts)
        if ws_n == 0:
            raise FavorError(FAVOR_ERR_UNSUPPORTED, "favor_workspace_size")
        workspace = _alloc_bytes(ws_n, Q.device, stream)
    st = library().favor_bwd(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(W), _ptr(out), _ptr(dout),
                             _ptr(ctx), int(causal), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace),
                             _workspace_bytes(workspace, Q.device), ctypes.byref(opts) if opts is not None else None,
                             _stream_ptr(stream))
    _check(st, "favor_bwd")
    return dQ, dK, dV


def bwd_into(Q, K, V, W, out, dout, dQ, dK, dV, ctx=None, causal=False, workspace=None, opts=None, stream=None):
    """favor_bwd writing into caller-provided fp32 gradient tensors (no allocation when a workspace
    is given)."""
    _check_inputs((Q, K, V, W, dout), Q)
    shape = _shape_of(Q, W)
    if workspace is None:
        ws_n = workspace_size(shape, causal, True, opts)
        if ws_n == 0:
            raise FavorError(FAVOR_ERR_UNSUPPORTED, "favor_workspace_size")
        workspace = _alloc_bytes(ws_n, Q.device, stream)
    st = library().favor_bwd(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(W), _ptr(out), _ptr(dout),
                             _ptr(ctx), int(causal), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace),
                             _workspace_bytes(workspace, Q.device), ctypes.byref(opts) if opts is not None else None,
                             _stream_ptr(stream))
    _check(st, "favor_bwd")
    return dQ, dK, dV


def sync_status(stream=None):
    """Synchronise the stream and return (and clear) the device status word."""
    return library().favor_sync_status(_stream_ptr(stream))


def sp_state(K, V, W, state=None, workspace=None, stream=None):
    """Partial state [B*H, m, d+64] (fp32) of this run of keys through favor_sp_state."""
    torch = _torch()
    _check_inputs((K, V, W), K)
    shape = _shape_of(K, W)
    lib = library()
    if state is None:
        state = _empty(lib.favor_sp_state_size(ctypes.byref(shape)) // 4, torch.float32, K.device, stream)
    if workspace is None:
        workspace = _alloc_bytes(lib.favor_sp_workspace_size(ctypes.byref(shape)), K.device, stream)
    st = lib.favor_sp_state(ctypes.byref(shape), _ptr(K), _ptr(V), _ptr(W), _ptr(state), _ptr(workspace),
                            _workspace_bytes(workspace, K.device), _stream_ptr(stream))
    _check(st, "favor_sp_state")
    return state


def sp_output(Q, W, state, out=None, workspace=None, stream=None):
    """Outputs of this run of queries against a total state, through favor_sp_output."""
    torch = _torch()
    _check_inputs((Q, W), Q)
    shape = _shape_of(Q, W)
    lib = library()
    if out is None:
        out = _empty(Q.shape, torch.float32, Q.device, stream)
    if workspace is None:
        workspace = _alloc_bytes(lib.favor_sp_workspace_size(ctypes.byref(shape)), Q.device, stream)
    st = lib.favor_sp_output(ctypes.byref(shape), _ptr(Q), _ptr(W), _ptr(state), _ptr(out), _ptr(workspace),
                             _workspace_bytes(workspace, Q.device), _stream_ptr(stream))
    _check(st, "favor_sp_output")
    return out


def sp_forward(Q, K, V, W, group=None, state_fn=None, output_fn=None):
    """Sequence-parallel bidirectional forward: this rank holds a contiguous run of every head's
    tokens; its partial key state is summed over the ranks of ``group`` (one all-reduce) and its
    queries are answered from the total. ``state_fn`` / ``output_fn`` default to sp_state /
    sp_output (tests substitute host stand-ins to exercise the exchange without a GPU)."""
    import torch.distributed as dist

    state = (state_fn or sp_state)(K, V, W)
    if dist.is_available() and dist.is_initialized() and dist.get_world_size(group) > 1:
        dist.all_reduce(state, op=dist.ReduceOp.SUM, group=group)
    return (output_fn or sp_output)(Q, W, state)


def decode_state(B, H, d, m, device):
    """A zero (empty) carried state for favor_decode_step."""
    torch = _torch()
    n = library().favor_decode_state_size(ctypes.byref(make_shape(B, H, 1, d, m, FAVOR_F32)))
    if n == 0:
        raise FavorError(FAVOR_ERR_UNSUPPORTED, "favor_decode_state_size")
    return torch.zeros(n // 4, dtype=torch.float32, device=device)


def decode_step(q, k, v, W, state, out=None, stream=None):
    """One token per head through favor_decode_step. q, k, v: [B,H,d] (bf16 or fp32); state from
    decode_state(), updated in place. Returns the fp32 output [B,H,d]."""
    torch = _torch()
    _check_inputs((q, k, v, W), q)
    B, H, d = q.shape
    shape = make_shape(B, H, 1, d, W.shape[0], _dtype_code(q))
    if out is None:
        out = _empty(q.shape, torch.float32, q.device, stream)
    st = library().favor_decode_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(W), _ptr(state),
                                     _ptr(out), _stream_ptr(stream))
    _check(st, "favor_decode_step")
    return out


# The calls of a decoding round take a few microseconds on the device, so their checks are written to
# cost little on the host: one pass over each tensor's attributes, shape structs reused by value, no
# wrapper objects around pointers, and the device switched only where it is another than the current one.

@functools.lru_cache(maxsize=256)
def _shape_ref(cls, *dims):
    """A reference to a shape struct of these values (structs are never written to)."""
    return ctypes.byref(cls(*dims))


def _fits(name, t, shape, dtype, device):
    """Refuses an argument that is not contiguous or not of this shape, type and device."""
    if t.dtype is not dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise FavorError(FAVOR_ERR_INVALID_ARG,
                         f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _opt_ptr(name, t, shape, dtype, device):
    """The address of an argument that may be None, checked."""
    if t is None:
        return None
    _fits(name, t, shape, dtype, device)
    return t.data_ptr()


def _tokens(first, rest, W, state):
    """Checks token tensors [B,H,L,d] of one shape, W [m,d] and a carried state on one CUDA device.
    Returns (B, H, L, d, m, dtype code) and the device."""
    if not first.is_cuda or first.dim() != 4 or W.dim() != 2:
        raise FavorError(FAVOR_ERR_INVALID_ARG, "tokens must be contiguous CUDA tensors [B,H,L,d] and W [m,d]")
    size, dtype, device = first.shape, first.dtype, first.device
    B, H, L, d = size
    m = W.shape[0]
    _fits("tokens", first, size, dtype, device)
    for t in rest:
        _fits("tokens", t, size, dtype, device)
    _fits("W", W, (m, d), dtype, device)
    if state.dtype is not _torch().float32 or state.device != device or state.numel() != B * H * (d + 2) * m or \
            not state.is_contiguous():
        raise FavorError(FAVOR_ERR_INVALID_ARG, "state must come from decode_state() for these B, H, d, m and device")
    return (B, H, L, d, m, _dtype_code(first)), device


def _launch(what, f, device, stream, *args):
    """Calls an entry point whose last argument is the stream (default: the current one of the tensors'
    device) with that device current."""
    torch = _torch()
    raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        st = f(*args, raw)
    else:
        with torch.cuda.device(device):
            st = f(*args, raw)
    if st != FAVOR_OK:
        raise FavorError(st, what)


def decode_tree(q, k, v, W, state, parents, n_nodes=None, out=None, stream=None):
    """Attention of a tree of drafted tokens over the carried state, through favor_decode_tree. q, k, v:
    [B,H,T,d] (bf16 or fp32), T up to FAVOR_TREE_MAX_NODES nodes in topological order; state from
    decode_state(), read only; parents: int32 [B,T], -1 for a root; n_nodes: int32 [B] or None. Returns
    the fp32 output [B,H,T,d]; its rows from n_nodes[b] on are left as they were in ``out`` (undefined
    when ``out`` is None)."""
    torch = _torch()
    dims, device = _tokens(q, (k, v), W, state)
    i32 = torch.int32
    _fits("parents", parents, (dims[0], dims[2]), i32, device)
    nodes = _opt_ptr("n_nodes", n_nodes, (dims[0],), i32, device)
    if out is None:
        out = _empty(q.shape, torch.float32, device, stream)
    else:
        _fits("out", out, q.shape, torch.float32, device)
    _launch("favor_decode_tree", library().favor_decode_tree, device, stream, _shape_ref(Shape, *dims), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), W.data_ptr(), state.data_ptr(), parents.data_ptr(), nodes, out.data_ptr())
    return out


@functools.lru_cache(maxsize=256)
def _extend_workspace(device_index, n_index, *dims):
    """favor_decode_extend_workspace_size of a shape on a device (it depends on the SM count)."""
    with _torch().cuda.device(device_index):
        return library().favor_decode_extend_workspace_size(_shape_ref(Shape, *dims), n_index)


def decode_extend(k, v, W, state, index=None, counts=None, workspace=None, stream=None):
    """Tokens added to the carried state, through favor_decode_extend. k, v: [B,H,L,d] (bf16 or fp32);
    state from decode_state(), updated in place and returned; index: int32 [B,N] positions of the tokens
    to add (such as the path decode_verify returns) or None for all in order; counts: int32 [B] how many
    of them, or None."""
    torch = _torch()
    dims, device = _tokens(k, (v,), W, state)
    i32, n_index, index_ptr = torch.int32, 0, None
    if index is not None:
        if index.dim() != 2 or index.shape[1] == 0:
            raise FavorError(FAVOR_ERR_INVALID_ARG, "index must be [B,N], N >= 1")
        n_index = index.shape[1]
        _fits("index", index, (dims[0], n_index), i32, device)
        index_ptr = index.data_ptr()
    n_tok = _opt_ptr("counts", counts, (dims[0],), i32, device)
    if workspace is None:
        ws_n = _extend_workspace(device.index, n_index, *dims)
        if ws_n == 0:
            raise FavorError(FAVOR_ERR_UNSUPPORTED, "favor_decode_extend_workspace_size")
        workspace = _empty(ws_n, torch.uint8, device, stream, returned=False)
    _launch("favor_decode_extend", library().favor_decode_extend, device, stream, _shape_ref(Shape, *dims),
            k.data_ptr(), v.data_ptr(), W.data_ptr(), index_ptr, n_index, n_tok, state.data_ptr(),
            workspace.data_ptr(), _workspace_bytes(workspace, device))
    return state


def decode_verify(parents, tokens, p, u, r, q=None, n_nodes=None, stream=None):
    """Verification of a drafted tree through favor_decode_verify. parents, tokens: int32 [B,T]; p, q:
    [B,T,V] bf16 or fp32 probabilities of the target and the draft (q None: a deterministic draft); u:
    fp32 [B,T], r: fp32 [B] uniform numbers in [0, 1). Returns (path [B,T], n_path [B], next_token [B]),
    int32: path and n_path go to decode_extend as index and counts."""
    torch = _torch()
    if not p.is_cuda or p.dim() != 3:
        raise FavorError(FAVOR_ERR_INVALID_ARG, "p must be a contiguous CUDA tensor [B,T,V]")
    size, device, i32, f32 = p.shape, p.device, torch.int32, torch.float32
    B, T, V = size
    nodes, row = (B, T), (B,)
    _fits("p", p, size, p.dtype, device)
    draft = _opt_ptr("q", q, size, p.dtype, device)
    _fits("parents", parents, nodes, i32, device)
    _fits("tokens", tokens, nodes, i32, device)
    used = _opt_ptr("n_nodes", n_nodes, row, i32, device)
    _fits("u", u, nodes, f32, device)
    _fits("r", r, row, f32, device)
    if stream is None:
        path, n_path, token = parents.new_empty(nodes), parents.new_empty(row), parents.new_empty(row)
    else:
        path, n_path, token = (_empty(size, i32, device, stream) for size in (nodes, row, row))
    _launch("favor_decode_verify", library().favor_decode_verify, device, stream,
            _shape_ref(VerifyShape, B, T, V, _dtype_code(p)), parents.data_ptr(), tokens.data_ptr(), used, p.data_ptr(),
            draft, u.data_ptr(), r.data_ptr(), path.data_ptr(), n_path.data_ptr(), token.data_ptr())
    return path, n_path, token


def selftest_bounded_wait(limit_us, stream=None):
    """Launches the library's bounded-wait self-test (a wait that nothing ends, given up after
    limit_us); the next sync_status() reports FAVOR_ERR_TIMEOUT."""
    _check(library().favor_selftest_bounded_wait(int(limit_us), _stream_ptr(stream)), "favor_selftest_bounded_wait")


STATIC_SCRATCH_BYTES = 32 << 20


def fwd_static_scratch(Q, K, V, W, out=None, stream=None):
    """Bidirectional bf16 forward through favor_fwd_static_scratch: no workspace is passed, the
    library uses its own fixed device array (for callers that cannot allocate device memory)."""
    torch = _torch()
    _check_inputs((Q, K, V, W), Q)
    shape = _shape_of(Q, W)
    if out is None:
        out = _empty(Q.shape, torch.float32, Q.device, stream)
    st = library().favor_fwd_static_scratch(ctypes.byref(shape), _ptr(Q), _ptr(K), _ptr(V), _ptr(W), _ptr(out),
                                            _stream_ptr(stream))
    _check(st, "favor_fwd_static_scratch")
    return out
