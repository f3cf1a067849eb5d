"""ctypes binding of the C ABI in ``include/mamba3_ssm.h``.

Argument marshalling only: every step of the computation runs in the gfx950
kernels of ``libmamba3_ssm.so``.  PyTorch supplies device memory (tensors are
passed by ``data_ptr()``) and the stream (``torch.cuda.current_stream()``).
If the library is missing this module raises; there is no fallback.

Entry points keep the ABI's names:
  mamba3_ssm_chunked_fwd, mamba3_ssm_chunked_bwd, mamba3_ssm_decode_step,
  mamba3_rope_bc, mamba3_bc_prologue,
  mamba3_layer_norm_fwd, mamba3_layer_norm_bwd, mamba3_linear_fwd,
  mamba3_linear_bwd, mamba3_gated_ffn_fwd, mamba3_gated_ffn_bwd,
  mamba3_qk_norm_rope_fwd, mamba3_qk_norm_rope_bwd, mamba3_window_attn_fwd,
  mamba3_window_attn_bwd, mamba3_window_attn_decode
(and the friendlier aliases without the prefix: chunked_fwd, chunked_bwd,
decode_step, rope_bc, bc_prologue, layer_norm_fwd, ...), plus the workspace
size queries.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# M3_LIBRARY names another build of the same library (e.g. one whose host
# code is compiled with sanitizers, for the host-side tests)
LIB_PATH = os.environ.get("M3_LIBRARY") or os.path.join(HERE, "libmamba3_ssm.so")

M3_OK, M3_ERR_NULL, M3_ERR_SHAPE, M3_ERR_UNSUPPORTED, M3_ERR_ALIGN, M3_ERR_WORKSPACE, M3_ERR_HIP = range(7)
M3_F32, M3_BF16 = 0, 1
M3_FLAG_CHUNK_WALK = 0x10000   # chunked_fwd: walk chunks even for short sequences
M3_FLAG_TOKEN_PATH = 0x20000   # chunked_fwd: token by token (at most M3_TOKEN_PATH_MAX_L tokens)
M3_TOKEN_PATH_MAX_L = 16       # longest call the token path takes
M3_TOKEN_PATH_SUBWALK_L = 8    # ... chosen by default when the sub-chunk walker covers the sizes
M3_NOALLOC_SCRATCH_BYTES = 48 << 20  # the fixed workspace of mamba3_ssm_chunked_fwd_noalloc, per GPU
ABI_SYMBOLS = ("mamba3_ssm_chunked_fwd", "mamba3_ssm_chunked_fwd_workspace_size", "mamba3_ssm_chunked_fwd_noalloc",
               "mamba3_ssm_chunked_bwd",
               "mamba3_ssm_chunked_bwd_workspace_size", "mamba3_ssm_decode_step",
               "mamba3_rope_bc", "mamba3_rope_bc_workspace_size", "mamba3_bc_prologue",
               "mamba3_bc_prologue_workspace_size", "mamba3_layer_norm_fwd", "mamba3_layer_norm_bwd",
               "mamba3_layer_norm_bwd_workspace_size", "mamba3_linear_fwd", "mamba3_linear_fwd_workspace_size",
               "mamba3_linear_bwd", "mamba3_linear_bwd_workspace_size", "mamba3_gated_ffn_fwd",
               "mamba3_gated_ffn_fwd_workspace_size", "mamba3_gated_ffn_bwd", "mamba3_gated_ffn_bwd_workspace_size",
               "mamba3_qk_norm_rope_fwd", "mamba3_qk_norm_rope_bwd", "mamba3_qk_norm_rope_bwd_workspace_size",
               "mamba3_window_attn_fwd", "mamba3_window_attn_bwd", "mamba3_window_attn_bwd_workspace_size",
               "mamba3_window_attn_decode", "mamba3_window_attn_decode_workspace_size",
               "mamba3_status_string", "mamba3_abi_version")
M3_FLAG_UNALIGNED = 0x40000    # linear, gated_ffn: operands off 16 bytes are copied first
M3_FLAG_ROPE_HALVES = 0x80000  # qk_norm_rope: pairs half of rope_dim apart
M3_FLAG_PACKED = 0x100000      # window_attn: sequences of any lengths, given by starts
M3_DECODE_MAX_TOKENS = 16      # new tokens of a sequence that window_attn_decode takes
# activations of linear and gated_ffn
M3_ACT_NONE, M3_ACT_RELU, M3_ACT_SILU, M3_ACT_GELU, M3_ACT_GELU_TANH, M3_ACT_SIGMOID = range(6)


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("rank", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("skip_stride", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class LinearDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class NormRopeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("rows", "seqlen", "q_heads", "k_heads", "head_dim", "rope_dim", "q_stride", "k_stride",
                 "q_out_stride", "k_out_stride", "dq_stride", "dk_stride")] + \
               [("io_dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class AttnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "q_len", "kv_len", "rows", "kv_rows", "q_heads", "kv_heads", "head_dim", "window", "sinks",
                 "q_stride", "k_stride", "v_stride", "o_stride", "do_stride", "dq_stride", "dk_stride",
                 "dv_stride")] + \
               [("scale", ctypes.c_float), ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class AttnDecodeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("batch", "tokens", "capacity", "q_heads", "kv_heads", "head_dim", "window", "sinks", "q_stride",
                 "k_stride", "v_stride", "o_stride", "k_cache_stride", "v_cache_stride")] + \
               [("scale", ctypes.c_float), ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Mamba3Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmamba3_ssm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with state_space_sequence_03_amd/build.py "
                               "(or __graft_entry__.build()); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p
        dp = ctypes.POINTER(Dims)
        L.mamba3_ssm_chunked_fwd.argtypes = [dp] + [vp] * 12 + [vp, sz, vp]
        L.mamba3_ssm_chunked_fwd.restype = ctypes.c_int
        L.mamba3_ssm_chunked_fwd_noalloc.argtypes = [dp] + [vp] * 12 + [vp]
        L.mamba3_ssm_chunked_fwd_noalloc.restype = ctypes.c_int
        L.mamba3_ssm_chunked_fwd_workspace_size.argtypes = [dp]
        L.mamba3_ssm_chunked_fwd_workspace_size.restype = sz
        L.mamba3_ssm_chunked_bwd.argtypes = [dp] + [vp] * 22 + [vp, sz, vp]
        L.mamba3_ssm_chunked_bwd.restype = ctypes.c_int
        L.mamba3_ssm_chunked_bwd_workspace_size.argtypes = [dp]
        L.mamba3_ssm_chunked_bwd_workspace_size.restype = sz
        L.mamba3_ssm_decode_step.argtypes = [dp] + [vp] * 11 + [vp]
        L.mamba3_ssm_decode_step.restype = ctypes.c_int
        L.mamba3_rope_bc.argtypes = [dp] + [vp] * 8 + [vp, sz, vp]
        L.mamba3_rope_bc.restype = ctypes.c_int
        L.mamba3_rope_bc_workspace_size.argtypes = [dp]
        L.mamba3_rope_bc_workspace_size.restype = sz
        L.mamba3_bc_prologue.argtypes = [dp, ctypes.c_int64, vp, vp, vp, vp, ctypes.c_float] + [vp] * 6 + [vp, sz, vp]
        L.mamba3_bc_prologue.restype = ctypes.c_int
        L.mamba3_bc_prologue_workspace_size.argtypes = [dp]
        L.mamba3_bc_prologue_workspace_size.restype = sz
        nd, ld = ctypes.POINTER(NormDims), ctypes.POINTER(LinearDims)
        L.mamba3_layer_norm_fwd.argtypes = [nd, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp]
        L.mamba3_layer_norm_bwd.argtypes = [nd] + [vp] * 9 + [vp, sz, vp]
        L.mamba3_linear_fwd.argtypes = [ld] + [vp] * 6 + [vp, sz, vp]
        L.mamba3_linear_bwd.argtypes = [ld] + [vp] * 7 + [vp, sz, vp]
        L.mamba3_gated_ffn_fwd.argtypes = [ld] + [vp] * 5 + [vp, sz, vp]
        L.mamba3_gated_ffn_bwd.argtypes = [ld] + [vp] * 7 + [vp, sz, vp]
        rd, ad, cd = ctypes.POINTER(NormRopeDims), ctypes.POINTER(AttnDims), ctypes.POINTER(AttnDecodeDims)
        L.mamba3_qk_norm_rope_fwd.argtypes = [rd] + [vp] * 4 + [ctypes.c_float] + [vp] * 5
        L.mamba3_qk_norm_rope_bwd.argtypes = [rd] + [vp] * 6 + [ctypes.c_float] + [vp] * 6 + [vp, sz, vp]
        L.mamba3_window_attn_fwd.argtypes = [ad] + [vp] * 7
        L.mamba3_window_attn_bwd.argtypes = [ad] + [vp] * 10 + [vp, sz, vp]
        L.mamba3_window_attn_decode.argtypes = [cd] + [vp] * 7 + [vp, sz, vp]
        for name, dims in (("qk_norm_rope_bwd", rd), ("window_attn_bwd", ad), ("window_attn_decode", cd),
                           ("layer_norm_bwd", nd), ("linear_fwd", ld), ("linear_bwd", ld), ("gated_ffn_fwd", ld),
                           ("gated_ffn_bwd", ld)):
            query = getattr(L, f"mamba3_{name}_workspace_size")
            query.argtypes = [dims]
            query.restype = sz
        L.mamba3_status_string.argtypes = [ctypes.c_int]
        L.mamba3_status_string.restype = ctypes.c_char_p
        L.mamba3_abi_version.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().mamba3_status_string(int(status)).decode()
    except Exception:  # library missing: still describe the code
        return "unknown"


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _io_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return M3_BF16
    if t.dtype == torch.float32:
        return M3_F32
    raise TypeError(f"io dtype must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _expect(name, t, shape, dtype, device):
    """Shape, dtype and device of an operand (None: absent).  The C ABI takes
    raw pointers and cannot see shapes, so the binding checks them before any
    call: a wrong shape would otherwise be read or written out of bounds."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_stream(stream, x, call, *args, **kw):
    """The call made under torch.cuda.stream(stream): what it allocates belongs
    to that stream, so that the allocator neither hands a workspace dropped at
    return to another stream's work while the kernels still use it, nor takes
    for it memory that such work still writes.  Outputs are recorded for the
    caller's stream too, which reads them next."""
    torch = _torch()
    if stream.device != x.device:
        raise ValueError(f"stream: on {stream.device}, expected {x.device}")
    here = torch.cuda.current_stream(x.device)
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(here)
    return out


def _check(status: int, what: str):
    if status != M3_OK:
        raise Mamba3Error(status, what)


def make_dims(batch, seqlen, nheads, headdim, dstate, rank, chunk, io_dtype, flags=0) -> Dims:
    return Dims(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate), int(rank), int(chunk),
                int(io_dtype), int(flags))


def chunked_fwd_workspace_size(dims: Dims) -> int:
    return int(lib().mamba3_ssm_chunked_fwd_workspace_size(ctypes.byref(dims)))


def rope_bc_workspace_size(dims: Dims) -> int:
    return int(lib().mamba3_rope_bc_workspace_size(ctypes.byref(dims)))


def _core_operands(torch, x, B, C, dt, A, lam, theta, h0, prev_B, prev_x):
    b, L, H, R, P = x.shape
    N = B.shape[-1]
    io, f32, dev = x.dtype, torch.float32, x.device
    for name, t in (("B", B), ("C", C)):
        _expect(name, t, (b, L, H, R, N), io, dev)
    for name, t in (("dt", dt), ("A", A), ("lam", lam)):
        _expect(name, t, (b, L, H), f32, dev)
    _expect("theta", theta, (b, L, H, N // 2), f32, dev)
    _expect("h0", h0, (b, H, N, P), f32, dev)
    _expect("prev_B", prev_B, (b, H, R, N), io, dev)
    _expect("prev_x", prev_x, (b, H, R, P), io, dev)


def mamba3_ssm_chunked_fwd(x, B, C, dt, A, lam, theta, h0=None, prev_B=None, prev_x=None, *, chunk=64,
                           segments=0, chunk_walk=False, token_path=False, y=None, h_final=None, want_final=True,
                           workspace=None, stream=None):
    """Whole-sequence forward.  Returns (y, h_final) (h_final None if not wanted).
    chunk_walk / token_path force one of the two paths for short calls (the
    library picks one by default)."""
    if stream is not None:
        return _on_stream(stream, x, mamba3_ssm_chunked_fwd, x, B, C, dt, A, lam, theta, h0, prev_B, prev_x,
                          chunk=chunk, segments=segments, chunk_walk=chunk_walk, token_path=token_path, y=y,
                          h_final=h_final, want_final=want_final, workspace=workspace)
    torch = _torch()
    b, L, H, R, P = x.shape
    N = B.shape[-1]
    _core_operands(torch, x, B, C, dt, A, lam, theta, h0, prev_B, prev_x)
    _expect("y", y, x.shape, x.dtype, x.device)
    _expect("h_final", h_final, (b, H, N, P), torch.float32, x.device)
    flags = segments | (M3_FLAG_CHUNK_WALK if chunk_walk else 0) | (M3_FLAG_TOKEN_PATH if token_path else 0)
    dims = make_dims(b, L, H, P, N, R, chunk, _io_code(x), flags=flags)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None and want_final:
        h_final = torch.empty((b, H, N, P), device=x.device, dtype=torch.float32)
    ws_bytes = chunked_fwd_workspace_size(dims)
    if ws_bytes > 0 and workspace is None:
        workspace = torch.empty(ws_bytes, device=x.device, dtype=torch.uint8)
    st = lib().mamba3_ssm_chunked_fwd(ctypes.byref(dims), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A),
                                      _ptr(lam), _ptr(theta), _ptr(h0), _ptr(prev_B), _ptr(prev_x), _ptr(y),
                                      _ptr(h_final), _ptr(workspace),
                                      ctypes.c_size_t(workspace.numel() if workspace is not None else 0),
                                      _stream(stream))
    _check(st, "mamba3_ssm_chunked_fwd")
    return y, h_final


def mamba3_ssm_chunked_fwd_noalloc(x, B, C, dt, A, lam, theta, h0=None, prev_B=None, prev_x=None, *, y, h_final,
                                   chunk=64, segments=0, stream=None):
    """mamba3_ssm_chunked_fwd with the workspace taken from the library's fixed
    per-GPU array: the caller passes every output (y, h_final may be None) and
    the call allocates nothing.  Calls that overlap on one GPU race on that
    array."""
    torch = _torch()
    b, L, H, R, P = x.shape
    N = B.shape[-1]
    _core_operands(torch, x, B, C, dt, A, lam, theta, h0, prev_B, prev_x)
    if y is None:
        raise ValueError("y is required (this entry point allocates nothing)")
    _expect("y", y, x.shape, x.dtype, x.device)
    _expect("h_final", h_final, (b, H, N, P), torch.float32, x.device)
    dims = make_dims(b, L, H, P, N, R, chunk, _io_code(x), flags=segments)
    st = lib().mamba3_ssm_chunked_fwd_noalloc(ctypes.byref(dims), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A),
                                              _ptr(lam), _ptr(theta), _ptr(h0), _ptr(prev_B), _ptr(prev_x), _ptr(y),
                                              _ptr(h_final), _stream(stream))
    _check(st, "mamba3_ssm_chunked_fwd_noalloc")
    return y, h_final


def chunked_bwd_workspace_size(dims: Dims) -> int:
    return int(lib().mamba3_ssm_chunked_bwd_workspace_size(ctypes.byref(dims)))


def mamba3_ssm_chunked_bwd(x, B, C, dt, A, lam, theta, dy, h0=None, prev_B=None, prev_x=None, dh_final=None, *,
                           chunk=64, segments=0, want_dh0=True, workspace=None, out=None, stream=None):
    """Backward of the chunked forward.  Returns a dict with dx, dB, dC (io dtype),
    ddt, dA, dlam, dtheta (fp32), dh0 (fp32, if wanted) and, when prev is given,
    dprev_B and dprev_x (io dtype).  segments: 0 = the library's choice, else
    the number of sequence segments walked in parallel (flags' low 16 bits).
    out: optional dict of preallocated outputs (any of the keys above)."""
    if stream is not None:
        return _on_stream(stream, x, mamba3_ssm_chunked_bwd, x, B, C, dt, A, lam, theta, dy, h0, prev_B, prev_x,
                          dh_final, chunk=chunk, segments=segments, want_dh0=want_dh0, workspace=workspace, out=out)
    torch = _torch()
    b, L, H, R, P = x.shape
    N = B.shape[-1]
    _core_operands(torch, x, B, C, dt, A, lam, theta, h0, prev_B, prev_x)
    _expect("dy", dy, x.shape, x.dtype, x.device)
    _expect("dh_final", dh_final, (b, H, N, P), torch.float32, x.device)
    dims = make_dims(b, L, H, P, N, R, chunk, _io_code(x), flags=segments)
    given = dict(out or {})
    out = {"dx": torch.empty_like(x), "dB": torch.empty_like(B), "dC": torch.empty_like(C),
           "ddt": torch.empty_like(dt), "dA": torch.empty_like(A), "dlam": torch.empty_like(lam),
           "dtheta": torch.empty_like(theta)}
    if want_dh0:
        out["dh0"] = torch.empty((b, H, N, P), device=x.device, dtype=torch.float32)
    if prev_B is not None:
        out["dprev_B"] = torch.empty_like(prev_B)
        out["dprev_x"] = torch.empty_like(prev_x)
    for k, t in given.items():
        if k not in out:
            raise ValueError(f"out: unexpected or unwanted output {k!r}")
        _expect(k, t, out[k].shape, out[k].dtype, x.device)
        out[k] = t
    ws_bytes = chunked_bwd_workspace_size(dims)
    if ws_bytes > 0 and workspace is None:
        workspace = torch.empty(ws_bytes, device=x.device, dtype=torch.uint8)
    st = lib().mamba3_ssm_chunked_bwd(ctypes.byref(dims), _ptr(x), _ptr(B), _ptr(C), _ptr(dt), _ptr(A), _ptr(lam),
                                      _ptr(theta), _ptr(h0), _ptr(prev_B), _ptr(prev_x), _ptr(dy), _ptr(dh_final),
                                      _ptr(out["dx"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["ddt"]),
                                      _ptr(out["dA"]), _ptr(out["dlam"]), _ptr(out["dtheta"]), _ptr(out.get("dh0")),
                                      _ptr(out.get("dprev_B")), _ptr(out.get("dprev_x")), _ptr(workspace),
                                      ctypes.c_size_t(workspace.numel() if workspace is not None else 0),
                                      _stream(stream))
    _check(st, "mamba3_ssm_chunked_bwd")
    return out


def mamba3_ssm_decode_step(state, x, B, C, dt, A, lam, theta, prev_B=None, prev_x=None, *, y=None, stream=None):
    """One token, state updated in place.  Shapes: state (b,H,N,P) fp32, x (b,H,R,P),
    B/C (b,H,R,N), dt/A/lam (b,H), theta (b,H,N/2).  Returns y (b,H,R,P)."""
    if stream is not None:
        return _on_stream(stream, x, mamba3_ssm_decode_step, state, x, B, C, dt, A, lam, theta, prev_B, prev_x, y=y)
    torch = _torch()
    b, H, R, P = x.shape
    N = B.shape[-1]
    io, f32, dev = x.dtype, torch.float32, x.device
    _expect("state", state, (b, H, N, P), f32, dev)
    for name, t in (("B", B), ("C", C), ("prev_B", prev_B)):
        _expect(name, t, (b, H, R, N), io, dev)
    _expect("prev_x", prev_x, (b, H, R, P), io, dev)
    for name, t in (("dt", dt), ("A", A), ("lam", lam)):
        _expect(name, t, (b, H), f32, dev)
    _expect("theta", theta, (b, H, N // 2), f32, dev)
    _expect("y", y, x.shape, io, dev)
    dims = make_dims(b, 1, H, P, N, R, 16, _io_code(x))
    if y is None:
        y = torch.empty_like(x)
    st = lib().mamba3_ssm_decode_step(ctypes.byref(dims), _ptr(state), _ptr(x), _ptr(B), _ptr(C), _ptr(dt),
                                      _ptr(A), _ptr(lam), _ptr(theta), _ptr(prev_B), _ptr(prev_x), _ptr(y),
                                      _stream(stream))
    _check(st, "mamba3_ssm_decode_step")
    return y


def mamba3_rope_bc(B, C, dt, theta, angle0=None, *, B_rot=None, C_rot=None, angle_final=None,
                   want_final=True, workspace=None, stream=None):
    """Cumulative-angle rotation.  Returns (B_rot, C_rot, angle_final)."""
    if stream is not None:
        return _on_stream(stream, B, mamba3_rope_bc, B, C, dt, theta, angle0, B_rot=B_rot, C_rot=C_rot,
                          angle_final=angle_final, want_final=want_final, workspace=workspace)
    torch = _torch()
    b, L, H, R, N = B.shape
    io, f32, dev = B.dtype, torch.float32, B.device
    for name, t in (("C", C), ("B_rot", B_rot), ("C_rot", C_rot)):
        _expect(name, t, B.shape, io, dev)
    _expect("dt", dt, (b, L, H), f32, dev)
    _expect("theta", theta, (b, L, H, N // 2), f32, dev)
    _expect("angle0", angle0, (b, H, N // 2), f32, dev)
    _expect("angle_final", angle_final, (b, H, N // 2), f32, dev)
    dims = make_dims(b, L, H, 16, N, R, 16, _io_code(B))
    if B_rot is None:
        B_rot = torch.empty_like(B)
    if C_rot is None:
        C_rot = torch.empty_like(C)
    if angle_final is None and want_final:
        angle_final = torch.empty((b, H, N // 2), device=B.device, dtype=torch.float32)
    ws_bytes = rope_bc_workspace_size(dims)
    if ws_bytes > 0 and workspace is None:
        workspace = torch.empty(ws_bytes, device=B.device, dtype=torch.uint8)
    st = lib().mamba3_rope_bc(ctypes.byref(dims), _ptr(B), _ptr(C), _ptr(dt), _ptr(theta), _ptr(angle0),
                              _ptr(B_rot), _ptr(C_rot), _ptr(angle_final), _ptr(workspace),
                              ctypes.c_size_t(workspace.numel() if workspace is not None else 0),
                              _stream(stream))
    _check(st, "mamba3_rope_bc")
    return B_rot, C_rot, angle_final


def bc_prologue_workspace_size(dims: Dims) -> int:
    return int(lib().mamba3_bc_prologue_workspace_size(ctypes.byref(dims)))


def mamba3_bc_prologue(u, W, dt, theta, nheads, rank, dstate, gain=None, bias=None, eps=1e-5, angle0=None, *,
                       B_rot=None, C_rot=None, angle_final=None, want_final=True, workspace=None, stream=None):
    """Projection of u (B, L, D) by W (2*H*R*N, D) to B and C, RMS-normalised
    per (token, head, rank) vector with gain and bias, and rotated by the
    cumulative angle.  Returns (B_rot, C_rot, angle_final)."""
    if stream is not None:
        return _on_stream(stream, u, mamba3_bc_prologue, u, W, dt, theta, nheads, rank, dstate, gain, bias, eps, angle0,
                          B_rot=B_rot, C_rot=C_rot, angle_final=angle_final, want_final=want_final,
                          workspace=workspace)
    torch = _torch()
    b, L, D = u.shape
    H, R, N = nheads, rank, dstate
    io, f32, dev = u.dtype, torch.float32, u.device
    _expect("W", W, (2 * H * R * N, D), io, dev)
    _expect("dt", dt, (b, L, H), f32, dev)
    _expect("theta", theta, (b, L, H, N // 2), f32, dev)
    for name, t in (("gain", gain), ("bias", bias)):
        _expect(name, t, (2, H, R, N), f32, dev)
    for name, t in (("B_rot", B_rot), ("C_rot", C_rot)):
        _expect(name, t, (b, L, H, R, N), io, dev)
    for name, t in (("angle0", angle0), ("angle_final", angle_final)):
        _expect(name, t, (b, H, N // 2), f32, dev)
    dims = make_dims(b, L, H, 16, N, R, 16, _io_code(u))
    if B_rot is None:
        B_rot = torch.empty((b, L, H, R, N), device=u.device, dtype=u.dtype)
    if C_rot is None:
        C_rot = torch.empty((b, L, H, R, N), device=u.device, dtype=u.dtype)
    if angle_final is None and want_final:
        angle_final = torch.empty((b, H, N // 2), device=u.device, dtype=torch.float32)
    ws_bytes = bc_prologue_workspace_size(dims)
    if ws_bytes > 0 and workspace is None:
        workspace = torch.empty(ws_bytes, device=u.device, dtype=torch.uint8)
    st = lib().mamba3_bc_prologue(ctypes.byref(dims), ctypes.c_int64(D), _ptr(u), _ptr(W), _ptr(gain), _ptr(bias),
                                  ctypes.c_float(eps), _ptr(dt), _ptr(theta), _ptr(angle0), _ptr(B_rot), _ptr(C_rot),
                                  _ptr(angle_final), _ptr(workspace),
                                  ctypes.c_size_t(workspace.numel() if workspace is not None else 0), _stream(stream))
    _check(st, "mamba3_bc_prologue")
    return B_rot, C_rot, angle_final


# ---------------------------------------------------------------------------
# the residual block around the core: layer norm, linear, gated feed-forward
# ---------------------------------------------------------------------------
# (a call of a few rows is bound by its host side: the checks' passing path is
# kept short, and the error is worked out only when one fails)
def _rows(name, t, width, rows, dtype, device):
    """(pointer, row stride in elements; 0: contiguous) of a matrix of rows:
    (..., width) contiguous, or (rows, width) with rows further apart."""
    if t.dtype is dtype and t.device == device and t.numel() == rows * width and t.shape[-1] == width:
        if t.is_contiguous():
            return t.data_ptr(), 0
        if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= width:
            return t.data_ptr(), t.stride(0)
        raise ValueError(f"{name}: must be contiguous, or 2-d with contiguous rows")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {rows} rows of {width}")


def _vec(name, t, shape, dtype, device):
    """Pointer of a contiguous operand of the given shape (None: absent)."""
    if t is None:
        return None
    if t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _expect(name, t, shape, dtype, device)
    raise ValueError(f"{name}: must be contiguous")


def _raw_stream(device):
    """Handle of the device's current stream."""
    torch = _torch()
    current = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object
    if current is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return current(device.index)


def _rows_of(x):
    """rows, width, type code of x (..., width)."""
    shape = x.shape
    if not shape or shape[-1] == 0:
        raise ValueError(f"x: shape {tuple(shape)}, expected (..., width) with a width from 1")
    return x.numel() // shape[-1], shape[-1], _io_code(x)


def mamba3_layer_norm_fwd(x, gain=None, bias=None, eps=1e-5, *, y=None, mean=None, rstd=None, want_stats=False,
                          stream=None):
    """Layer norm of the rows of x (..., D).  Returns (y, mean, rstd); the
    statistics ((rows) fp32, for the backward) are None unless wanted or given."""
    if stream is not None:
        return _on_stream(stream, x, mamba3_layer_norm_fwd, x, gain, bias, eps, y=y, mean=mean, rstd=rstd,
                          want_stats=want_stats)
    torch = _torch()
    rows, D, code = _rows_of(x)
    io, dev, f32 = x.dtype, x.device, torch.float32
    px, sx = _rows("x", x, D, rows, io, dev)
    if y is None:
        y = torch.empty_like(x) if sx == 0 else x.new_empty(x.shape)
        py, sy = y.data_ptr(), 0
    else:
        py, sy = _rows("y", y, D, rows, io, dev)
    if want_stats or mean is not None or rstd is not None:
        mean = torch.empty(rows, dtype=f32, device=dev) if mean is None else mean
        rstd = torch.empty_like(mean) if rstd is None else rstd
    st = lib().mamba3_layer_norm_fwd(NormDims(rows, D, sx, sy, 0, code, 0), px, _vec("gain", gain, (D,), f32, dev),
                                     _vec("bias", bias, (D,), f32, dev), eps, py,
                                     _vec("mean", mean, (rows,), f32, dev), _vec("rstd", rstd, (rows,), f32, dev),
                                     _raw_stream(dev))
    _check(st, "mamba3_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd_workspace_size(dims: NormDims) -> int:
    return int(lib().mamba3_layer_norm_bwd_workspace_size(ctypes.byref(dims)))


def mamba3_layer_norm_bwd(x, mean, rstd, dy, gain=None, dskip=None, *, want_dx=True, want_dgain=True,
                          want_dbias=True, dx=None, dgain=None, dbias=None, workspace=None, stream=None):
    """Backward of layer_norm_fwd.  dskip: a gradient that reaches x past the
    norm, added to dx.  Returns a dict with dx (io dtype), dgain and dbias (fp32),
    as wanted.  dskip and dx have the same row stride: a dx made here has x's
    shape, and dskip's row stride where dskip is a column slice."""
    if stream is not None:
        return _on_stream(stream, x, mamba3_layer_norm_bwd, x, mean, rstd, dy, gain, dskip, want_dx=want_dx,
                          want_dgain=want_dgain, want_dbias=want_dbias, dx=dx, dgain=dgain, dbias=dbias,
                          workspace=workspace)
    torch = _torch()
    rows, D, code = _rows_of(x)
    io, dev, f32 = x.dtype, x.device, torch.float32
    px, sx = _rows("x", x, D, rows, io, dev)
    pdy, sdy = _rows("dy", dy, D, rows, io, dev)
    psk, ssk = (None, 0) if dskip is None else _rows("dskip", dskip, D, rows, io, dev)
    out = {}
    pdx = pg = pb = pws = None
    nws = 0
    if want_dx or dx is not None:
        if dx is None:
            if ssk:
                dx = torch.empty_strided((rows, D), (ssk, 1), dtype=io, device=dev).view(x.shape)
            else:
                dx = torch.empty_like(x) if sx == 0 else x.new_empty(x.shape)
            pdx = dx.data_ptr()
        else:
            pdx, sdx = _rows("dx", dx, D, rows, io, dev)
            if dskip is not None and (sdx or D) != (ssk or D):
                raise ValueError("dx and dskip must have the same row stride")
            ssk = sdx
        out["dx"] = dx
    if dgain is not None:
        out["dgain"], pg = dgain, _vec("dgain", dgain, (D,), f32, dev)
    elif want_dgain:
        out["dgain"] = dgain = torch.empty(D, dtype=f32, device=dev)
        pg = dgain.data_ptr()
    if dbias is not None:
        out["dbias"], pb = dbias, _vec("dbias", dbias, (D,), f32, dev)
    elif want_dbias:
        out["dbias"] = dbias = torch.empty(D, dtype=f32, device=dev)
        pb = dbias.data_ptr()
    dims = NormDims(rows, D, sx, sdy, ssk, code, 0)
    L = lib()
    if pg or pb:
        workspace, pws, nws = _workspace(L.mamba3_layer_norm_bwd_workspace_size, dims, workspace, dev)
    st = L.mamba3_layer_norm_bwd(dims, px, _vec("gain", gain, (D,), f32, dev), _vec("mean", mean, (rows,), f32, dev),
                                 _vec("rstd", rstd, (rows,), f32, dev), pdy, psk, pdx, pg, pb, pws, nws,
                                 _raw_stream(dev))
    _check(st, "mamba3_layer_norm_bwd")
    return out


def linear_fwd_workspace_size(dims: LinearDims) -> int:
    return int(lib().mamba3_linear_fwd_workspace_size(ctypes.byref(dims)))


def linear_bwd_workspace_size(dims: LinearDims) -> int:
    return int(lib().mamba3_linear_bwd_workspace_size(ctypes.byref(dims)))


def gated_ffn_fwd_workspace_size(dims: LinearDims) -> int:
    return int(lib().mamba3_gated_ffn_fwd_workspace_size(ctypes.byref(dims)))


def gated_ffn_bwd_workspace_size(dims: LinearDims) -> int:
    return int(lib().mamba3_gated_ffn_bwd_workspace_size(ctypes.byref(dims)))


def _workspace(query, dims, workspace, device):
    """(tensor, pointer, bytes) of the workspace a call needs (None, None, 0: none)."""
    need = query(dims)
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _torch().empty(need, device=device, dtype=_torch().uint8)
        return workspace, workspace.data_ptr(), need
    if workspace.device != device:
        raise ValueError(f"workspace: on {workspace.device}, expected {device}")
    if not workspace.is_contiguous():  # its bytes are counted from its entries
        raise ValueError("workspace: must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _weight_rows(W, gated):
    """Rows of W and the width of the operator's result."""
    if W.dim() != 2:
        raise ValueError(f"W: shape {tuple(W.shape)}, expected (rows of W, d_in)")
    n = W.shape[0]
    if not gated:
        return n, n
    if n % 2:
        raise ValueError(f"W: {n} rows, expected the gate's and as many more")
    return n, n // 2


def _product_fwd(name, gated, x, W, bias, residual, act, y, pre, want_pre, workspace, stream):
    if stream is not None:
        return _on_stream(stream, x, _product_fwd, name, gated, x, W, bias, residual, act, y, pre, want_pre,
                          workspace, None)
    torch = _torch()
    rows, K, code = _rows_of(x)
    wrows, N = _weight_rows(W, gated)
    io, dev, L = x.dtype, x.device, lib()
    px, sx = _rows("x", x, K, rows, io, dev)
    if y is None:
        y = x.new_empty(x.shape[:-1] + (N,))
        py, sy = y.data_ptr(), 0
    else:
        py, sy = _rows("y", y, N, rows, io, dev)
    pr, sr = (None, 0) if residual is None else _rows("residual", residual, N, rows, io, dev)
    ppre = None
    if pre is not None:
        ppre = _vec("pre", pre, x.shape[:-1] + (wrows,), io, dev)
    elif want_pre:
        pre = x.new_empty(x.shape[:-1] + (wrows,))
        ppre = pre.data_ptr()
    pW = _vec("W", W, (wrows, K), io, dev)
    pb = _vec("bias", bias, (wrows,), torch.float32, dev)
    dims = LinearDims(rows, K, N, sx, sy, sr, code, act, M3_FLAG_UNALIGNED if (px | pW) & 15 else 0, 0)
    s = _raw_stream(dev)
    if gated:
        workspace, pws, nws = _workspace(L.mamba3_gated_ffn_fwd_workspace_size, dims, workspace, dev)
        st = L.mamba3_gated_ffn_fwd(dims, px, pW, pb, py, ppre, pws, nws, s)
    else:
        workspace, pws, nws = _workspace(L.mamba3_linear_fwd_workspace_size, dims, workspace, dev)
        st = L.mamba3_linear_fwd(dims, px, pW, pb, pr, py, ppre, pws, nws, s)
    _check(st, name)
    return y, pre


def _product_bwd(name, gated, x, W, dy, pre, act, want_dx, want_dW, want_dbias, dx, dW, dbias, workspace, stream):
    if stream is not None:
        return _on_stream(stream, x, _product_bwd, name, gated, x, W, dy, pre, act, want_dx, want_dW, want_dbias,
                          dx, dW, dbias, workspace, None)
    torch = _torch()
    rows, K, code = _rows_of(x)
    wrows, N = _weight_rows(W, gated)
    io, dev, L = x.dtype, x.device, lib()
    px, sx = _rows("x", x, K, rows, io, dev)
    pdy, sdy = _rows("dy", dy, N, rows, io, dev)
    ppre = None
    if pre is not None:
        ppre, spre = _rows("pre", pre, wrows, rows, io, dev)
        if spre:
            raise ValueError("pre: must be contiguous")
    elif gated or act != M3_ACT_NONE:
        raise ValueError("pre is required (the forward's want_pre)")
    pW = _vec("W", W, (wrows, K), io, dev)
    out = {}
    pdx = pdW = pb = None
    if dx is not None:
        out["dx"], pdx = dx, _vec("dx", dx, x.shape, io, dev)
    elif want_dx:
        out["dx"] = dx = torch.empty_like(x) if sx == 0 else x.new_empty(x.shape)
        pdx = dx.data_ptr()
    if dW is not None:
        out["dW"], pdW = dW, _vec("dW", dW, (wrows, K), io, dev)
    elif want_dW:
        out["dW"] = dW = torch.empty_like(W)
        pdW = dW.data_ptr()
    if dbias is not None:
        out["dbias"], pb = dbias, _vec("dbias", dbias, (wrows,), torch.float32, dev)
    elif want_dbias:
        out["dbias"] = dbias = torch.empty(wrows, dtype=torch.float32, device=dev)
        pb = dbias.data_ptr()
    dims = LinearDims(rows, K, N, sx, sdy, 0, code, act, M3_FLAG_UNALIGNED if (px | pW | pdy) & 15 else 0, 0)
    query, call = ((L.mamba3_gated_ffn_bwd_workspace_size, L.mamba3_gated_ffn_bwd) if gated else
                   (L.mamba3_linear_bwd_workspace_size, L.mamba3_linear_bwd))
    workspace, pws, nws = _workspace(query, dims, workspace, dev)
    st = call(dims, px, pW, ppre, pdy, pdx, pdW, pb, pws, nws, _raw_stream(dev))
    _check(st, name)
    return out


def mamba3_linear_fwd(x, W, bias=None, residual=None, *, act=M3_ACT_NONE, y=None, pre=None, want_pre=False,
                      workspace=None, stream=None):
    """act(x W^T + bias) + residual for x (..., d_in), W (d_out, d_in).  Returns
    (y, pre); pre = x W^T + bias (for the backward) is None unless wanted or given."""
    return _product_fwd("mamba3_linear_fwd", False, x, W, bias, residual, act, y, pre, want_pre, workspace, stream)


def mamba3_linear_bwd(x, W, dy, pre=None, *, act=M3_ACT_NONE, want_dx=True, want_dW=True, want_dbias=True, dx=None,
                      dW=None, dbias=None, workspace=None, stream=None):
    """Backward of linear_fwd.  Returns a dict with dx, dW (io dtype) and dbias
    (fp32), as wanted.  pre is required unless act is M3_ACT_NONE."""
    return _product_bwd("mamba3_linear_bwd", False, x, W, dy, pre, act, want_dx, want_dW, want_dbias, dx, dW, dbias,
                        workspace, stream)


def mamba3_gated_ffn_fwd(x, W, bias=None, *, act=M3_ACT_SILU, h=None, pre=None, want_pre=False, workspace=None,
                         stream=None):
    """act(g) u with [g u] = x W^T + bias for x (..., d_in), W (2F, d_in): the
    gate's rows, then the other F.  Returns (h, pre); pre (..., 2F) (for the
    backward) is None unless wanted or given."""
    return _product_fwd("mamba3_gated_ffn_fwd", True, x, W, bias, None, act, h, pre, want_pre, workspace, stream)


def mamba3_gated_ffn_bwd(x, W, dh, pre, *, act=M3_ACT_SILU, want_dx=True, want_dW=True, want_dbias=True, dx=None,
                         dW=None, dbias=None, workspace=None, stream=None):
    """Backward of gated_ffn_fwd.  Returns a dict with dx, dW (io dtype) and
    dbias (2F, fp32), as wanted."""
    return _product_bwd("mamba3_gated_ffn_bwd", True, x, W, dh, pre, act, want_dx, want_dW, want_dbias, dx, dW, dbias,
                        workspace, stream)


# ---------------------------------------------------------------------------
# the attention layer beside the core: norms of queries and keys with their
# rotation, windowed attention with sinks, the same over a cache
# ---------------------------------------------------------------------------
def _empty(t):
    """A contiguous tensor like t."""
    torch = _torch()
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _tokens(name, t, shape, dtype, device):
    """(pointer, elements from token to token; 0: contiguous) of an operand of
    the given shape (..., heads, dim): contiguous, or with heads side by side
    and tokens evenly further apart (a slice of the heads of a wider tensor)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _expect(name, t, shape, dtype, device)
    return _spacing(name, t, shape)


def _spacing(name, t, shape):
    """_tokens of an operand whose shape, type and device are known to be right."""
    if t.is_contiguous():
        return t.data_ptr(), 0
    st = t.stride()
    heads, dim = shape[-2], shape[-1]
    if (dim == 1 or st[-1] == 1) and (heads == 1 or st[-2] == dim):
        step = None  # elements between tokens; dimensions of one entry say nothing
        inner = 1    # tokens that the dimensions looked at so far hold
        for i in range(len(shape) - 3, -1, -1):
            n = shape[i]
            if n != 1:
                if step is None:
                    step = st[i]
                elif st[i] != inner * step:
                    break
                inner *= n
        else:
            if step is None:
                return t.data_ptr(), 0
            if step >= heads * dim:
                return t.data_ptr(), step
    raise ValueError(f"{name}: must be contiguous, or with heads side by side and evenly spaced tokens")


def _heads_of(name, shape, least):
    if len(shape) < least or shape[-1] == 0:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected (..., heads, head_dim)")
    return shape[:-2], shape[-2], shape[-1]


def _norm_rope_dims(q, k, gain_q, gain_k, theta, pos, halves):
    """What both directions check of the operands they share: dims (the strides
    of what is not shared left 0), shapes of q and k, pointers of q, k, the
    gains, theta and pos, type, device."""
    torch = _torch()
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is required")
    io, dev, f32, shape = x.dtype, x.device, torch.float32, x.shape
    lead, Hq, D = _heads_of("q" if q is not None else "k", shape, 3)
    qs = ks = pq = pk = None
    sq = sk = Hk = 0
    if q is not None:
        qs = shape
        pq, sq = _spacing("q", q, qs)
    else:
        Hq = 0
    if k is not None:
        ks = k.shape
        if ks[:-2] != lead or ks[-1] != D:
            raise ValueError(f"k: shape {tuple(ks)}, expected {tuple(lead)} tokens of heads of {D}")
        if k.dtype is not io or k.device != dev:
            _expect("k", k, ks, io, dev)
        Hk = ks[-2]
        pk, sk = _spacing("k", k, ks)
    rope = 0
    if theta is not None:
        ts = theta.shape
        rope = 2 * ts[0] if len(ts) == 1 else -1
        if not 0 <= rope <= D:
            raise ValueError(f"theta: shape {tuple(theta.shape)}, expected at most (head_dim / 2,) = ({D // 2},)")
        theta = _vec("theta", theta, (rope // 2,), f32, dev)
    if pos is not None:
        pos = _vec("pos", pos, lead, torch.int64, dev)
    rows = 1
    for n in lead:
        rows *= n
    if gain_q is not None:
        gain_q = _vec("gain_q", gain_q, (D,), f32, dev)
    if gain_k is not None:
        gain_k = _vec("gain_k", gain_k, (D,), f32, dev)
    dims = NormRopeDims(rows, lead[-1], Hq, Hk, D, rope, sq, sk, 0, 0, 0, 0, _io_code(x),
                        M3_FLAG_ROPE_HALVES if halves else 0)
    return dims, qs, ks, (pq, pk, gain_q, gain_k, theta, pos), io, dev


def mamba3_qk_norm_rope_fwd(q, k, gain_q=None, gain_k=None, eps=1e-5, *, theta=None, pos=None, halves=False,
                            q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q (..., L, q_heads, D) and k (..., L, k_heads, D),
    gains (D) fp32, and the rotation of the first 2 * len(theta) entries by
    pos theta (theta fp32; None: no rotation).  pos: (..., L) int64, or None: a
    token's index along L.  halves: pairs are (j, j + len(theta)), else (2j, 2j + 1).
    q and k may be slices of one projection's heads; either may be None.
    Returns (q_out, k_out), which may be given (q and k themselves, too)."""
    if stream is not None:
        return _on_stream(stream, q if q is not None else k, mamba3_qk_norm_rope_fwd, q, k, gain_q, gain_k, eps,
                          theta=theta, pos=pos, halves=halves, q_out=q_out, k_out=k_out)
    dims, qs, ks, (pq, pk, pgq, pgk, pt, pp), io, dev = _norm_rope_dims(q, k, gain_q, gain_k, theta, pos, halves)
    pqo = pko = None
    if qs is None:
        q_out = None
    elif q_out is None:
        q_out = _empty(q)
        pqo = q_out.data_ptr()
    else:
        pqo, dims.q_out_stride = _tokens("q_out", q_out, qs, io, dev)
    if ks is None:
        k_out = None
    elif k_out is None:
        k_out = _empty(k)
        pko = k_out.data_ptr()
    else:
        pko, dims.k_out_stride = _tokens("k_out", k_out, ks, io, dev)
    st = lib().mamba3_qk_norm_rope_fwd(dims, pq, pk, pgq, pgk, eps, pt, pp, pqo, pko, _raw_stream(dev))
    _check(st, "mamba3_qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_bwd_workspace_size(dims: NormRopeDims) -> int:
    return int(lib().mamba3_qk_norm_rope_bwd_workspace_size(ctypes.byref(dims)))


def mamba3_qk_norm_rope_bwd(q, k, dq_out, dk_out, gain_q=None, gain_k=None, eps=1e-5, *, theta=None, pos=None,
                            halves=False, want_dgain=True, dq=None, dk=None, dgain_q=None, dgain_k=None,
                            workspace=None, stream=None):
    """Backward of qk_norm_rope_fwd from its inputs and the gradients of its
    results.  Returns a dict with dq, dk (io dtype; those of q and k that are
    given) and, as wanted or given, dgain_q, dgain_k (fp32).  dq and dk may be
    dq_out and dk_out themselves."""
    if stream is not None:
        return _on_stream(stream, q if q is not None else k, mamba3_qk_norm_rope_bwd, q, k, dq_out, dk_out, gain_q,
                          gain_k, eps, theta=theta, pos=pos, halves=halves, want_dgain=want_dgain, dq=dq, dk=dk,
                          dgain_q=dgain_q, dgain_k=dgain_k, workspace=workspace)
    dims, qs, ks, (pq, pk, pgq, pgk, pt, pp), io, dev = _norm_rope_dims(q, k, gain_q, gain_k, theta, pos, halves)
    f32, D, out = _torch().float32, dims.head_dim, {}
    pdqo = pdko = pdq = pdk = pnq = pnk = pws = None
    nws = 0
    if qs is not None:
        if dq_out is None:
            raise ValueError("dq_out is required with q")
        pdqo, dims.q_out_stride = _tokens("dq_out", dq_out, qs, io, dev)
        if dq is None:
            dq = _empty(q)
            pdq = dq.data_ptr()
        else:
            pdq, dims.dq_stride = _tokens("dq", dq, qs, io, dev)
        out["dq"] = dq
        if dgain_q is not None or want_dgain:
            if dgain_q is None:
                dgain_q = q.new_empty(D, dtype=f32)
            out["dgain_q"], pnq = dgain_q, _vec("dgain_q", dgain_q, (D,), f32, dev)
    if ks is not None:
        if dk_out is None:
            raise ValueError("dk_out is required with k")
        pdko, dims.k_out_stride = _tokens("dk_out", dk_out, ks, io, dev)
        if dk is None:
            dk = _empty(k)
            pdk = dk.data_ptr()
        else:
            pdk, dims.dk_stride = _tokens("dk", dk, ks, io, dev)
        out["dk"] = dk
        if dgain_k is not None or want_dgain:
            if dgain_k is None:
                dgain_k = k.new_empty(D, dtype=f32)
            out["dgain_k"], pnk = dgain_k, _vec("dgain_k", dgain_k, (D,), f32, dev)
    L = lib()
    if pnq or pnk:
        workspace, pws, nws = _workspace(L.mamba3_qk_norm_rope_bwd_workspace_size, dims, workspace, dev)
    st = L.mamba3_qk_norm_rope_bwd(dims, pq, pk, pdqo, pdko, pgq, pgk, eps, pt, pp, pdq, pdk, pnq, pnk, pws, nws,
                                   _raw_stream(dev))
    _check(st, "mamba3_qk_norm_rope_bwd")
    return out


def _attn_dims(q, k, v, starts, window, sinks, scale, grads=False):
    """Dims of a windowed attention (strides of q, k, v set), pointers of q, k, v
    and starts, shapes of q and k, type, device."""
    io, dev, ps, rows, kv_rows, flags = q.dtype, q.device, None, 0, 0, 0
    qs, ks = q.shape, k.shape
    lead, Hq, D = _heads_of("q", qs, 3)
    pq, sq = _spacing("q", q, qs)
    if starts is None:
        if len(qs) != 4 or len(ks) != 4 or ks[0] != qs[0] or ks[3] != D:
            raise ValueError("q is (batch, q_len, heads, head_dim), k and v (batch, kv_len, heads, head_dim)")
        batch, q_len, kv_len = qs[0], qs[1], ks[1]
        (pk, sk, kv_rows), (pv, sv, rv) = _sequences("k", k, ks, io, dev), _sequences("v", v, ks, io, dev)
        if kv_len == 1 and (grads or kv_rows != rv) and k.stride(0) <= 1 << 20 and v.stride(0) <= 1 << 20:
            # single tokens may be anything evenly spaced
            (pk, sk), (pv, sv), kv_rows, rv = _tokens("k", k, ks, io, dev), _tokens("v", v, ks, io, dev), 0, 0
        if kv_rows != rv:
            raise ValueError("k and v must have as many rows from sequence to sequence")
    else:
        if len(qs) != 3 or len(ks) != 3 or ks[0] != qs[0] or ks[2] != D:
            raise ValueError("with starts, q, k and v are (tokens, heads, head_dim) of the same tokens")
        if starts.dim() != 1 or starts.shape[0] < 1:
            raise ValueError(f"starts: shape {tuple(starts.shape)}, expected (sequences + 1,)")
        ps = _vec("starts", starts, starts.shape, _torch().int64, dev)
        batch, q_len, kv_len, rows, flags = starts.shape[0] - 1, 0, 0, qs[0], M3_FLAG_PACKED
        (pk, sk), (pv, sv) = _tokens("k", k, ks, io, dev), _tokens("v", v, ks, io, dev)
    dims = AttnDims(batch, q_len, kv_len, rows, kv_rows, Hq, ks[-2], D, window, sinks, sq, sk, sv, 0, 0, 0, 0, 0,
                    D ** -0.5 if scale is None else scale, _io_code(q), flags, 0)
    return dims, (pq, pk, pv, ps), qs, ks, io, dev


def _sequences(name, t, shape, dtype, device):
    """(pointer, elements from token to token, tokens from sequence to sequence;
    0: the length) of keys (batch, length, heads, dim), which may be the first
    tokens of longer sequences (a cache's)."""
    if not t.is_contiguous() and t.shape == shape and shape[0] > 1 and shape[1] > 0:
        row, between = shape[2] * shape[3], t.stride(0)
        step = t.stride(1) if t.stride(1) >= row else row if shape[1] == 1 else 0
        if step > 0 and between % step == 0 and between // step > shape[1]:
            p, s = _tokens(name, t[0], shape[1:], dtype, device)
            # a single token says nothing about the rows it is one of: its own width, or else what divides the distance
            unit = s or (row if between % row == 0 else step)
            return p, 0 if unit == row else unit, between // unit
    return _tokens(name, t, shape, dtype, device) + (0,)


def mamba3_window_attn_fwd(q, k, v, *, window=0, sinks=0, scale=None, starts=None, o=None, lse=None, want_lse=False,
                           stream=None):
    """Causal attention of q (batch, q_len, q_heads, D) over k, v (batch, kv_len,
    kv_heads, D): the queries are the last q_len of kv_len positions and see the
    `window` last keys up to their own (0: all) and the first `sinks`.  starts
    (sequences + 1, int64): packed sequences, q, k, v (tokens, heads, D).  scale:
    of the scores, D^-1/2 by default.  k and v may be the first tokens of a
    longer cache.  Returns (o, lse); lse (tokens, q_heads) fp32 with q's leading
    shape (for the backward) is None unless wanted or given."""
    if stream is not None:
        return _on_stream(stream, q, mamba3_window_attn_fwd, q, k, v, window=window, sinks=sinks, scale=scale,
                          starts=starts, o=o, lse=lse, want_lse=want_lse)
    dims, (pq, pk, pv, ps), qs, _, io, dev = _attn_dims(q, k, v, starts, window, sinks, scale)
    if o is None:
        o = _empty(q)
        po = o.data_ptr()
    else:
        po, dims.o_stride = _tokens("o", o, qs, io, dev)
    pl = None
    if lse is not None:
        pl = _vec("lse", lse, qs[:-1], _torch().float32, dev)
    elif want_lse:
        lse = q.new_empty(qs[:-1], dtype=_torch().float32)
        pl = lse.data_ptr()
    st = lib().mamba3_window_attn_fwd(dims, pq, pk, pv, ps, po, pl, _raw_stream(dev))
    _check(st, "mamba3_window_attn_fwd")
    return o, lse


def window_attn_bwd_workspace_size(dims: AttnDims) -> int:
    return int(lib().mamba3_window_attn_bwd_workspace_size(ctypes.byref(dims)))


def mamba3_window_attn_bwd(q, k, v, o, lse, do, *, window=0, sinks=0, scale=None, starts=None, want_dq=True,
                           want_dk=True, want_dv=True, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of window_attn_fwd (the same q, k, v, window, sinks, scale,
    starts; its o and lse).  Returns a dict with dq, dk, dv (io dtype), as
    wanted.  With starts, gradients that the call makes itself hold nothing in
    the rows of no sequence."""
    if stream is not None:
        return _on_stream(stream, q, mamba3_window_attn_bwd, q, k, v, o, lse, do, window=window, sinks=sinks,
                          scale=scale, starts=starts, want_dq=want_dq, want_dk=want_dk, want_dv=want_dv, dq=dq, dk=dk,
                          dv=dv, workspace=workspace)
    dims, (pq, pk, pv, ps), qs, ks, io, dev = _attn_dims(q, k, v, starts, window, sinks, scale, True)
    po, dims.o_stride = _tokens("o", o, qs, io, dev)
    pdo, dims.do_stride = _tokens("do", do, qs, io, dev)
    pl = _vec("lse", lse, qs[:-1], _torch().float32, dev)
    if pl is None:
        raise ValueError("lse is required (the forward's want_lse)")
    out, pdq, pdk, pdv = {}, None, None, None
    if dq is not None:
        out["dq"], (pdq, dims.dq_stride) = dq, _tokens("dq", dq, qs, io, dev)
    elif want_dq:
        out["dq"] = dq = _empty(q)
        pdq = dq.data_ptr()
    if dk is not None:
        out["dk"], (pdk, dims.dk_stride) = dk, _tokens("dk", dk, ks, io, dev)
    elif want_dk:
        out["dk"] = dk = _empty(k)
        pdk = dk.data_ptr()
    if dv is not None:
        out["dv"], (pdv, dims.dv_stride) = dv, _tokens("dv", dv, ks, io, dev)
    elif want_dv:
        out["dv"] = dv = _empty(v)
        pdv = dv.data_ptr()
    if dims.kv_rows and (dk is not None or dv is not None):
        raise ValueError("gradients of keys that are part of a longer cache: pass k and v as contiguous sequences")
    L = lib()
    workspace, pws, nws = _workspace(L.mamba3_window_attn_bwd_workspace_size, dims, workspace, dev)
    st = L.mamba3_window_attn_bwd(dims, pq, pk, pv, po, pl, pdo, ps, pdq, pdk, pdv, pws, nws, _raw_stream(dev))
    _check(st, "mamba3_window_attn_bwd")
    return out


def window_attn_decode_workspace_size(dims: AttnDecodeDims) -> int:
    return int(lib().mamba3_window_attn_decode_workspace_size(ctypes.byref(dims)))


def mamba3_window_attn_decode(q, k, v, k_cache, v_cache, lens, *, window=0, sinks=0, scale=None, o=None,
                              workspace=None, stream=None):
    """The T new tokens (M3_DECODE_MAX_TOKENS at most) q (batch, T, q_heads, D),
    k, v (batch, T, kv_heads, D), written to the caches (batch, capacity, kv_heads,
    D) in place and attending over them.  lens (batch, int64): tokens in each cache
    before the call (negative: an idle sequence; fewer than the last call left
    drops its last tokens, with a window or before the cache wraps).  Position p
    lies in slot p below `sinks`, else in slot sinks + (p - sinks) mod (capacity -
    sinks) (window_cache_slots).
    Returns o (batch, T, q_heads, D)."""
    if stream is not None:
        return _on_stream(stream, q, mamba3_window_attn_decode, q, k, v, k_cache, v_cache, lens, window=window,
                          sinks=sinks, scale=scale, o=o, workspace=workspace)
    io, dev, qs, ks, cs = q.dtype, q.device, q.shape, k.shape, k_cache.shape
    if len(qs) != 4 or len(ks) != 4 or len(cs) != 4 or ks[:2] != qs[:2] or cs[0] != qs[0] or cs[2:] != ks[2:]:
        raise ValueError("q, k, v are (batch, tokens, heads, head_dim), "
                         "the caches (batch, capacity, heads of k, head_dim)")
    _, Hq, D = _heads_of("q", qs, 4)
    pq, sq = _spacing("q", q, qs)
    if ks[3] != D:
        raise ValueError(f"k: head_dim {ks[3]}, expected {D}")
    pk, sk = _tokens("k", k, ks, io, dev)
    pv, sv = _tokens("v", v, ks, io, dev)
    pkc, skc = _tokens("k_cache", k_cache, cs, io, dev)
    pvc, svc = _tokens("v_cache", v_cache, cs, io, dev)
    so = 0
    if o is None:
        o = _empty(q)
        po = o.data_ptr()
    else:
        po, so = _tokens("o", o, qs, io, dev)
    dims = AttnDecodeDims(qs[0], qs[1], cs[1], Hq, ks[2], D, window, sinks, sq, sk, sv, so, skc, svc,
                          D ** -0.5 if scale is None else scale, _io_code(q), 0, 0)
    L = lib()
    workspace, pws, nws = _workspace(L.mamba3_window_attn_decode_workspace_size, dims, workspace, dev)
    st = L.mamba3_window_attn_decode(dims, pq, pk, pv, pkc, pvc, _vec("lens", lens, qs[:1], _torch().int64, dev), po,
                                     pws, nws, _raw_stream(dev))
    _check(st, "mamba3_window_attn_decode")
    return o


def window_cache_slots(pos, sinks, capacity):
    """Slots of a cache of `capacity` slots where window_attn_decode keeps the
    tokens at positions pos (an integer tensor): for filling one after a prefill."""
    if not 0 <= sinks < capacity:
        raise ValueError(f"a cache of {capacity} slots has no ring behind {sinks} sinks")
    return _torch().where(pos < sinks, pos, sinks + (pos - sinks) % (capacity - sinks))


chunked_fwd = mamba3_ssm_chunked_fwd
chunked_fwd_noalloc = mamba3_ssm_chunked_fwd_noalloc
chunked_bwd = mamba3_ssm_chunked_bwd
decode_step = mamba3_ssm_decode_step
rope_bc = mamba3_rope_bc
bc_prologue = mamba3_bc_prologue
layer_norm_fwd = mamba3_layer_norm_fwd
layer_norm_bwd = mamba3_layer_norm_bwd
linear_fwd = mamba3_linear_fwd
linear_bwd = mamba3_linear_bwd
gated_ffn_fwd = mamba3_gated_ffn_fwd
gated_ffn_bwd = mamba3_gated_ffn_bwd
qk_norm_rope_fwd = mamba3_qk_norm_rope_fwd
qk_norm_rope_bwd = mamba3_qk_norm_rope_bwd
window_attn_fwd = mamba3_window_attn_fwd
window_attn_bwd = mamba3_window_attn_bwd
window_attn_decode = mamba3_window_attn_decode
