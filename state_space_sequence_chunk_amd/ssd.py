"""Python binding of the C ABI in include/ssd.h (argument marshalling only).

Every function here forwards device pointers of torch tensors and the current HIP
stream to the shared library built from ``csrc/``; all computation happens in the HIP
kernels. When the library is missing or cannot be loaded, calls raise -- there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libssd_mi355x.so")

SSD_F32, SSD_BF16 = 0, 1
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_DTYPE",
          4: "SSD_ERR_UNSUPPORTED", 5: "SSD_ERR_WORKSPACE", 6: "SSD_ERR_ALIGN", 7: "SSD_ERR_HIP",
          8: "SSD_ERR_TOO_LARGE"}
# Bytes of the scratch array behind ssd_forward_noalloc (SSD_NOALLOC_SCRATCH_BYTES in ssd.h).
NOALLOC_SCRATCH_BYTES = 256 << 20

# Entry points declared in include/ssd.h.
EXPORTS = ("ssd_status_string", "ssd_validate_shape", "ssd_forward_workspace_bytes",
           "ssd_state_pass_workspace_bytes", "ssd_chunk_cumsum", "ssd_state_pass",
           "ssd_state_scan", "ssd_chunk_out", "ssd_forward", "ssd_decode_step", "ssd_backward_workspace_bytes",
           "ssd_backward", "ssd_state_pass_segmented_workspace_bytes", "ssd_state_pass_segmented",
           "ssd_chunk_out_segmented", "ssd_segment_plan", "ssd_forward_noalloc",
           "ssd_chunk_out_plan", "ssd_delta_forward_workspace_bytes", "ssd_delta_forward",
           "ssd_delta_decode_step", "ssd_delta_backward_workspace_bytes", "ssd_delta_backward",
           "ssd_delta_forward_plan", "ssd_delta_backward_plan",
           "ssd_group_norm", "ssd_group_norm_backward_workspace_bytes", "ssd_group_norm_backward")
# Activations of the group norm (ssd_act in ssd.h).
ACTS = {"none": 0, "silu": 1, "gate_pre": 2, "gate_post": 3}
# HBM stream probes declared in include/ssd_probe.h (measurement only).
PROBE_EXPORTS = ("ssd_probe_read", "ssd_probe_write", "ssd_probe_copy", "ssd_probe_mix")


class SSDError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(code, code)} ({msg})")
        self.code = code


class ssd_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("chunk", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("states_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ssd_norm_shape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("z_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("center", ctypes.c_int32), ("eps", ctypes.c_float)]


_lib = None


def load_library():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"HIP library not built: {LIB_PATH} is missing. Build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` or "
            "`python state_space_sequence_chunk_amd/build.py`.")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    sp = ctypes.POINTER(ssd_shape)
    lib.ssd_status_string.argtypes = [i32]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_validate_shape.argtypes = [sp]
    lib.ssd_forward_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.ssd_state_pass_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.ssd_chunk_cumsum.argtypes = [sp, vp, vp, vp, vp, vp]
    lib.ssd_state_pass.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ssd_state_scan.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.ssd_chunk_out.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.ssd_forward.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ssd_forward_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.ssd_decode_step.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.ssd_backward_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.ssd_backward.argtypes = [sp] + [vp] * 17 + [sz, vp]
    lib.ssd_state_pass_segmented_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.ssd_state_pass_segmented.argtypes = [sp] + [vp] * 9 + [sz, vp]
    lib.ssd_chunk_out_segmented.argtypes = [sp] + [vp] * 9 + [sz, vp]
    i32p = ctypes.POINTER(ctypes.c_int32)
    lib.ssd_segment_plan.argtypes = [sp, i32p, i32p, i32p]
    lib.ssd_chunk_out_plan.argtypes = [sp, i32p, i32p, ctypes.POINTER(ctypes.c_double)]
    f32 = ctypes.c_float
    lib.ssd_delta_forward_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.ssd_delta_forward.argtypes = [sp] + [vp] * 6 + [f32] + [vp] * 3 + [sz, vp]
    lib.ssd_delta_decode_step.argtypes = [sp] + [vp] * 6 + [f32] + [vp] * 3
    lib.ssd_delta_backward_workspace_bytes.argtypes = [sp, ctypes.POINTER(sz)]
    lib.ssd_delta_backward.argtypes = [sp] + [vp] * 8 + [f32] + [vp] * 7 + [sz, vp]
    lib.ssd_delta_forward_plan.argtypes = [sp] + [i32p] * 4
    lib.ssd_delta_backward_plan.argtypes = [sp] + [i32p] * 3
    np_ = ctypes.POINTER(ssd_norm_shape)
    lib.ssd_group_norm.argtypes = [np_] + [vp] * 6
    lib.ssd_group_norm_backward_workspace_bytes.argtypes = [np_, ctypes.POINTER(sz)]
    lib.ssd_group_norm_backward.argtypes = [np_] + [vp] * 10 + [sz, vp]
    lib.ssd_probe_read.argtypes = [vp, sz, vp, i32, i32, vp]
    lib.ssd_probe_write.argtypes = [vp, sz, i32, i32, vp]
    lib.ssd_probe_copy.argtypes = [vp, vp, sz, i32, i32, vp]
    lib.ssd_probe_mix.argtypes = [vp, sz, vp, sz, i32, i32, vp]
    for name in EXPORTS[1:] + PROBE_EXPORTS:
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def _check(code: int, where: str):
    if code != 0:
        msg = load_library().ssd_status_string(code).decode()
        raise SSDError(code, where, msg)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return SSD_BF16
    if dt == torch.float32:
        return SSD_F32
    raise ValueError(f"unsupported dtype {dt}")


def _code(dt):
    return dt if isinstance(dt, int) else dtype_code(dt)


def make_shape(batch, seqlen, nheads, headdim, dstate, ngroups, chunk, in_dtype,
               states_dtype=None, out_dtype=None) -> ssd_shape:
    """Shape struct; states default to the input dtype, y to fp32."""
    ind = _code(in_dtype)
    std = ind if states_dtype is None else _code(states_dtype)
    outd = SSD_F32 if out_dtype is None else _code(out_dtype)
    return ssd_shape(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate),
                     int(ngroups), int(chunk), ind, std, outd, 0)


def shape_of(x: torch.Tensor, B: torch.Tensor, chunk: int, states_dtype=None,
             out_dtype=None) -> ssd_shape:
    """Shape struct from x [b, L, h, P] and B [b, L, g, S]."""
    b, L, H, P = x.shape
    G, S = B.shape[2], B.shape[3]
    return make_shape(b, L, H, P, S, G, chunk, x.dtype, states_dtype, out_dtype)


def _p(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the SSD library must be contiguous")
    if not t.is_cuda and not t.is_pinned():  # (a kernel reads pinned host memory, other host memory faults it)
        raise ValueError("tensors passed to the SSD library must be on a GPU")
    return t.data_ptr()  # (argtypes says that it is a pointer)


def _stream(stream):
    if stream is None:  # the handle alone: a Stream object costs as much as a small launch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def validate_shape(shape: ssd_shape) -> int:
    return int(load_library().ssd_validate_shape(ctypes.byref(shape)))


def forward_workspace_bytes(shape: ssd_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_forward_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssd_forward_workspace_bytes")
    return int(n.value)


def state_pass_workspace_bytes(shape: ssd_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_state_pass_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssd_state_pass_workspace_bytes")
    return int(n.value)


def ssd_chunk_cumsum(shape, dt, A, G, dt_t=None, stream=None):
    _check(load_library().ssd_chunk_cumsum(ctypes.byref(shape), _p(dt), _p(A), _p(G), _p(dt_t),
                                           _stream(stream)), "ssd_chunk_cumsum")


def ssd_state_pass(shape, x, A, B, G, dt_t, h0, states, final_state, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_state_pass(ctypes.byref(shape), _p(x), _p(A), _p(B), _p(G), _p(dt_t),
                                         _p(h0), _p(states), _p(final_state), _p(workspace),
                                         nbytes, _stream(stream)), "ssd_state_pass")


def ssd_state_scan(shape, x, A, B, dt_t, h0, states, final_state, stream=None):
    _check(load_library().ssd_state_scan(ctypes.byref(shape), _p(x), _p(A), _p(B), _p(dt_t),
                                         _p(h0), _p(states), _p(final_state), _stream(stream)),
           "ssd_state_scan")


def ssd_chunk_out(shape, x, B, C, G, dt_t, states, D, y, stream=None):
    _check(load_library().ssd_chunk_out(ctypes.byref(shape), _p(x), _p(B), _p(C), _p(G),
                                        _p(dt_t), _p(states), _p(D), _p(y), _stream(stream)),
           "ssd_chunk_out")


def state_pass_segmented_workspace_bytes(shape: ssd_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_state_pass_segmented_workspace_bytes(ctypes.byref(shape),
                                                                   ctypes.byref(n)),
           "ssd_state_pass_segmented_workspace_bytes")
    return int(n.value)


def segment_plan(shape: ssd_shape):
    """(heads per workgroup, chunks per segment, segments) of the segmented state pass;
    raises SSDError (SSD_ERR_UNSUPPORTED) for shapes without a plan."""
    h, k, n = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().ssd_segment_plan(ctypes.byref(shape), ctypes.byref(h),
                                           ctypes.byref(k), ctypes.byref(n)),
           "ssd_segment_plan")
    return int(h.value), int(k.value), int(n.value)


def chunk_out_plan(shape: ssd_shape):
    """(heads per workgroup, interaction tiles shared, executed matrix-core flops per launch)
    of the output kernel ssd_forward launches for the shape."""
    h, sh, fl = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_double(0.0)
    _check(load_library().ssd_chunk_out_plan(ctypes.byref(shape), ctypes.byref(h),
                                             ctypes.byref(sh), ctypes.byref(fl)),
           "ssd_chunk_out_plan")
    return int(h.value), bool(sh.value), float(fl.value)


def ssd_state_pass_segmented(shape, x, A, B, G, dt_t, h0, seg_relative_states, final_state,
                             workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_state_pass_segmented(
        ctypes.byref(shape), _p(x), _p(A), _p(B), _p(G), _p(dt_t), _p(h0),
        _p(seg_relative_states), _p(final_state), _p(workspace), nbytes, _stream(stream)),
        "ssd_state_pass_segmented")


def ssd_chunk_out_segmented(shape, x, B, C, G, dt_t, D, seg_relative_states, y, workspace,
                            stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_chunk_out_segmented(
        ctypes.byref(shape), _p(x), _p(B), _p(C), _p(G), _p(dt_t), _p(D),
        _p(seg_relative_states), _p(y), _p(workspace), nbytes, _stream(stream)),
        "ssd_chunk_out_segmented")


def ssd_forward(shape, x, dt, A, B, C, D, h0, y, final_state, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_forward(ctypes.byref(shape), _p(x), _p(dt), _p(A), _p(B), _p(C),
                                      _p(D), _p(h0), _p(y), _p(final_state), _p(workspace),
                                      nbytes, _stream(stream)), "ssd_forward")


def ssd_forward_noalloc(shape, x, dt, A, B, C, D, h0, y, final_state, stream=None):
    """ssd_forward without a workspace: the library's own per-device scratch array holds
    the intermediates (no allocation; calls that overlap on one GPU race)."""
    _check(load_library().ssd_forward_noalloc(ctypes.byref(shape), _p(x), _p(dt), _p(A), _p(B),
                                              _p(C), _p(D), _p(h0), _p(y), _p(final_state),
                                              _stream(stream)), "ssd_forward_noalloc")


def ssd_decode_step(shape, x, dt, A, B, C, D, state, y, stream=None):
    _check(load_library().ssd_decode_step(ctypes.byref(shape), _p(x), _p(dt), _p(A), _p(B),
                                          _p(C), _p(D), _p(state), _p(y), _stream(stream)),
           "ssd_decode_step")


def probe_read(src, sink, *, mode=0, workgroups=0, stream=None):
    """Stream `src` (a contiguous device tensor) through a read-only kernel."""
    _check(load_library().ssd_probe_read(_p(src), src.numel() * src.element_size(), _p(sink),
                                         mode, workgroups, _stream(stream)), "ssd_probe_read")


def probe_write(dst, *, mode=0, workgroups=0, stream=None):
    _check(load_library().ssd_probe_write(_p(dst), dst.numel() * dst.element_size(), mode,
                                          workgroups, _stream(stream)), "ssd_probe_write")


def probe_copy(src, dst, *, mode=0, workgroups=0, stream=None):
    if src.numel() * src.element_size() != dst.numel() * dst.element_size():
        raise ValueError("probe_copy: src and dst sizes differ")
    _check(load_library().ssd_probe_copy(_p(src), _p(dst), src.numel() * src.element_size(),
                                         mode, workgroups, _stream(stream)), "ssd_probe_copy")


def probe_mix(src, read_bytes, dst, write_bytes, *, mode=0, workgroups=0, stream=None):
    """Read read_bytes of src and write write_bytes of dst in one pass (see ssd_probe.h)."""
    if read_bytes > src.numel() * src.element_size() or write_bytes > dst.numel() * dst.element_size():
        raise ValueError("probe_mix: sizes exceed the buffers")
    _check(load_library().ssd_probe_mix(_p(src), read_bytes, _p(dst), write_bytes, mode,
                                        workgroups, _stream(stream)), "ssd_probe_mix")


def decode_step(x, dt, A, B, C, D, state, *, stream=None):
    """One token for every (batch, head): x [b, h, P], dt [b, h], B/C [b, g, S]; `state`
    (fp32 [b, h, P, S], e.g. ssd_forward's final state) is updated in place. Returns y
    (fp32 [b, h, P])."""
    b, H, P = x.shape
    sh = make_shape(b, 1, H, P, B.shape[2], B.shape[1], 1, x.dtype, torch.float32)
    y = torch.empty((b, H, P), dtype=torch.float32, device=x.device)
    ssd_decode_step(sh, x, dt, A, B, C, D, state, y, stream)
    return y


def backward_workspace_bytes(shape: ssd_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_backward_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssd_backward_workspace_bytes")
    return int(n.value)


def ssd_backward(shape, x, dt, A, B, C, D, h0, dy, dfinal, dx, ddt, dA, dB, dC, dD, dh0,
                 workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_backward(ctypes.byref(shape), _p(x), _p(dt), _p(A), _p(B), _p(C),
                                       _p(D), _p(h0), _p(dy), _p(dfinal), _p(dx), _p(ddt),
                                       _p(dA), _p(dB), _p(dC), _p(dD), _p(dh0), _p(workspace),
                                       nbytes, _stream(stream)), "ssd_backward")


def backward(x, dt, A, B, C, D, h0, dy, dfinal=None, *, chunk, stream=None):
    """Gradients of sum(dy * y) + sum(dfinal * final) (fp32 tensors, input layouts):
    returns dict dx, ddt, dA, dB, dC, dD, dh0."""
    sh = shape_of(x, B, chunk)
    b, L, H, P = x.shape
    S = B.shape[3]
    f32 = dict(dtype=torch.float32, device=x.device)
    out = {"dx": torch.empty(x.shape, **f32), "ddt": torch.empty(dt.shape, **f32),
           "dA": torch.empty(A.shape, **f32), "dB": torch.empty(B.shape, **f32),
           "dC": torch.empty(C.shape, **f32), "dD": torch.empty((H,), **f32),
           "dh0": torch.empty((b, H, P, S), **f32)}
    ws = torch.empty(backward_workspace_bytes(sh), dtype=torch.uint8, device=x.device)
    ssd_backward(sh, x, dt, A, B, C, D, h0, dy, dfinal, out["dx"], out["ddt"], out["dA"],
                 out["dB"], out["dC"], out["dD"], out["dh0"], ws, stream)
    return out


class Forward:
    """Holds the output and workspace buffers of one problem size and runs ssd_forward.

    torch supplies the device memory; the call itself is one C-ABI invocation.
    """

    def __init__(self, x, B, chunk, states_dtype=None, device=None, out_dtype=None):
        self.shape = shape_of(x, B, chunk, states_dtype, out_dtype)
        dev = device or x.device
        b, L, H, P = x.shape
        S = B.shape[3]
        ydt = torch.bfloat16 if self.shape.out_dtype == SSD_BF16 else torch.float32
        self.y = torch.empty((b, L, H, P), dtype=ydt, device=dev)
        self.final = torch.empty((b, H, P, S), dtype=torch.float32, device=dev)
        self.workspace = torch.empty(forward_workspace_bytes(self.shape), dtype=torch.uint8,
                                     device=dev)

    def __call__(self, x, dt, A, B, C, D=None, h0=None, stream=None):
        ssd_forward(self.shape, x, dt, A, B, C, D, h0, self.y, self.final, self.workspace,
                    stream)
        return self.y, self.final


class ForwardGraph:
    """ssd_forward on fixed input buffers, recorded once in a HIP graph (through
    torch.cuda.CUDAGraph) and replayed: a replay is one graph launch instead of one launch
    per kernel, which is most of the time of a small problem. Every replay reads the input
    tensors given here (update them in place between replays) and writes the same y and
    final tensors. The forward pass records no memset and allocates nothing, so the graph
    holds only its kernels."""

    def __init__(self, x, dt, A, B, C, D=None, h0=None, *, chunk, states_dtype=None,
                 out_dtype=None):
        self.fwd = Forward(x, B, chunk, states_dtype, out_dtype=out_dtype)
        self.args = (x, dt, A, B, C, D, h0)
        # one call outside the capture (kernel attributes are set on first use)
        self.fwd(*self.args)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.fwd(*self.args, stream=torch.cuda.current_stream())

    @property
    def y(self):
        return self.fwd.y

    @property
    def final(self):
        return self.fwd.final

    def replay(self):
        self.graph.replay()
        return self.fwd.y, self.fwd.final


def forward(x, dt, A, B, C, D=None, h0=None, *, chunk, states_dtype=None, out_dtype=None,
            stream=None):
    """One-shot forward pass; returns (y [b, L, h, P] in out_dtype (fp32 by default),
    final state fp32 [b, h, P, S])."""
    f = Forward(x, B, chunk, states_dtype, out_dtype=out_dtype)
    return f(x, dt, A, B, C, D, h0, stream)


def delta_shape_of(v: torch.Tensor, k: torch.Tensor, out_dtype=None) -> ssd_shape:
    """Shape struct of the gated delta rule from v [b, L, h, P] and k [b, L, g, S]."""
    return shape_of(v, k, 64, torch.float32, out_dtype)


def _check_delta(v, g, beta, k, q, states=(), rows=()):
    """The checks the C ABI cannot make: types, layouts and devices of the tensors. `states` and
    `rows` are (name, tensor or None) pairs of the state's and v's shape, fp32."""
    vs, ks = v.shape, k.shape
    n = len(vs)
    if n < 3 or len(ks) != n:
        raise ValueError("v is [b, L, h, P] and k [b, L, g, S] (without L for a decode step)")
    if ks[:n - 2] != vs[:n - 2] or q.shape != ks:
        raise ValueError(f"k and q are {tuple(vs[:n - 2])} + (groups, dstate): got {tuple(ks)}, "
                         f"{tuple(q.shape)}")
    if g.shape != vs[:n - 1] or beta.shape != vs[:n - 1]:
        raise ValueError(f"g and beta are {tuple(vs[:n - 1])}: got {tuple(g.shape)}, {tuple(beta.shape)}")
    dt, dev, f32 = v.dtype, v.device, torch.float32
    if k.dtype != dt or q.dtype != dt or beta.dtype != dt:
        raise ValueError("v, beta, k and q have one dtype")
    if g.dtype != f32:
        raise ValueError("g is float32")
    if g.device != dev or beta.device != dev or k.device != dev or q.device != dev:
        raise ValueError("all tensors are on one device")
    if states:
        want = (vs[0], vs[n - 2], vs[n - 1], ks[n - 1])
    for name, t in states:
        if t is not None and (t.shape != want or t.dtype != f32 or t.device != dev):
            raise ValueError(f"{name} is float32 {want} on {dev}: got {t.dtype} {tuple(t.shape)} on {t.device}")
    for name, t in rows:
        if t is not None and (t.shape != vs or t.dtype != f32 or t.device != dev):
            raise ValueError(f"{name} is float32 {tuple(vs)} on {dev}: got {t.dtype} {tuple(t.shape)} on {t.device}")


def _run(call, stream, tensors):
    """call() with the tensors' device current. On a stream other than the current one, what the
    call allocates belongs to that stream, its inputs are not reused before the stream is done with
    them, and its outputs are handed back to the caller's stream."""
    t = tensors[0]
    if stream is not None and t.is_cuda and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
    if not t.is_cuda or (stream is None and t.device.index == torch.cuda.current_device()):
        return call()
    with torch.cuda.device(t.device):
        here = torch.cuda.current_stream()
        if stream is None or stream == here:
            return call()
        with torch.cuda.stream(stream):
            for x in tensors:
                if x is not None:
                    x.record_stream(stream)
            out = call()
            for x in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
                if x is not None:
                    x.record_stream(here)
            return out


def delta_forward_workspace_bytes(shape: ssd_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_delta_forward_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssd_delta_forward_workspace_bytes")
    return int(n.value)


def delta_backward_workspace_bytes(shape: ssd_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_delta_backward_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssd_delta_backward_workspace_bytes")
    return int(n.value)


def delta_forward_plan(shape: ssd_shape):
    """(segments, waves a workgroup, waves a workgroup of the first walk over segments, heads a wave
    prepares) of the delta rule's forward pass; zeros where no chunked kernel runs."""
    n = [ctypes.c_int32(0) for _ in range(4)]
    _check(load_library().ssd_delta_forward_plan(ctypes.byref(shape), *map(ctypes.byref, n)), "ssd_delta_forward_plan")
    return tuple(int(x.value) for x in n)


def delta_backward_plan(shape: ssd_shape):
    """(waves a workgroup of the walks, heads a wave prepares, heads a workgroup takes the gradients of)
    of the delta rule's backward pass; zeros for an empty sequence."""
    n = [ctypes.c_int32(0) for _ in range(3)]
    _check(load_library().ssd_delta_backward_plan(ctypes.byref(shape), *map(ctypes.byref, n)), "ssd_delta_backward_plan")
    return tuple(int(x.value) for x in n)


def ssd_delta_forward(shape, v, g, beta, k, q, h0, scale, y, final_state, workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_delta_forward(
        ctypes.byref(shape), _p(v), _p(g), _p(beta), _p(k), _p(q), _p(h0), scale, _p(y),
        _p(final_state), _p(workspace), nbytes, _stream(stream)), "ssd_delta_forward")


def ssd_delta_decode_step(shape, v, g, beta, k, q, state, scale, state_out, y, stream=None):
    _check(load_library().ssd_delta_decode_step(
        ctypes.byref(shape), _p(v), _p(g), _p(beta), _p(k), _p(q), _p(state), scale,
        _p(state_out), _p(y), _stream(stream)), "ssd_delta_decode_step")


def ssd_delta_backward(shape, v, g, beta, k, q, h0, dy, dfinal, scale, dv, dg, dbeta, dk, dq, dh0,
                       workspace, stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_delta_backward(
        ctypes.byref(shape), _p(v), _p(g), _p(beta), _p(k), _p(q), _p(h0), _p(dy), _p(dfinal),
        scale, _p(dv), _p(dg), _p(dbeta), _p(dk), _p(dq), _p(dh0), _p(workspace), nbytes,
        _stream(stream)), "ssd_delta_backward")


def delta_forward(v, g, beta, k, q, h0=None, *, scale=1.0, out_dtype=None, stream=None):
    """Gated delta rule over whole sequences: v [b, L, h, P], g (fp32 log decays) and beta
    [b, L, h], k and q [b, L, groups, S], optional state h0 (fp32 [b, h, P, S]). Returns
    (y [b, L, h, P] in out_dtype (fp32 by default), final state fp32 [b, h, P, S]). With bf16 inputs
    products keep 16 bits of fp32 values; fp32 inputs keep all 24."""
    if v.dim() != 4:
        raise ValueError("v is [b, L, h, P]")
    _check_delta(v, g, beta, k, q, (("h0", h0),))
    sh = delta_shape_of(v, k, out_dtype)
    b, L, H, P = v.shape

    def call():
        y = torch.empty(v.shape, dtype=out_dtype or torch.float32, device=v.device)
        final = torch.empty((b, H, P, k.shape[3]), dtype=torch.float32, device=v.device)
        ws = torch.empty(delta_forward_workspace_bytes(sh), dtype=torch.uint8, device=v.device)
        ssd_delta_forward(sh, v, g, beta, k, q, h0, scale, y, final, ws, stream)
        return y, final

    return _run(call, stream, (v, g, beta, k, q, h0))


def delta_decode_step(v, g, beta, k, q, state, *, scale=1.0, state_out=None, stream=None):
    """One token of the gated delta rule: v [b, h, P], g and beta [b, h], k and q [b, groups, S].
    The state (fp32 [b, h, P, S], e.g. delta_forward's final state) is updated in place, or,
    with state_out, left as it is and the new one written there. Returns y (fp32 [b, h, P])."""
    if v.dim() != 3:
        raise ValueError("v is [b, h, P]")
    out = state if state_out is None else state_out
    _check_delta(v, g, beta, k, q, (("state", state), ("state_out", state_out)))
    if out is not state and out.data_ptr() != state.data_ptr() and _overlap(out, state):
        raise ValueError("state_out is the state itself or does not overlap it")
    b, H, P = v.shape
    sh = ssd_shape(b, 1, H, P, k.shape[2], k.shape[1], 64, dtype_code(v.dtype), SSD_F32, SSD_F32, 0)

    def call():
        y = torch.empty((b, H, P), dtype=torch.float32, device=v.device)
        ssd_delta_decode_step(sh, v, g, beta, k, q, state, scale, out, y, stream)
        return y

    return _run(call, stream, (v, g, beta, k, q, state, state_out))


def _overlap(a, b):
    lo = max(a.data_ptr(), b.data_ptr())
    hi = min(a.data_ptr() + a.numel() * a.element_size(), b.data_ptr() + b.numel() * b.element_size())
    return lo < hi


def delta_backward(v, g, beta, k, q, h0, dy, dfinal=None, *, scale=1.0, stream=None):
    """Gradients of sum(dy * y) + sum(dfinal * final) of delta_forward (fp32 tensors, input
    layouts): returns dict dv, dg, dbeta, dk, dq, dh0."""
    if v.dim() != 4:
        raise ValueError("v is [b, L, h, P]")
    _check_delta(v, g, beta, k, q, (("h0", h0), ("dfinal", dfinal)), (("dy", dy),))
    sh = delta_shape_of(v, k)

    def call():
        f32 = dict(dtype=torch.float32, device=v.device)
        out = {"dv": torch.empty(v.shape, **f32), "dg": torch.empty(g.shape, **f32),
               "dbeta": torch.empty(g.shape, **f32), "dk": torch.empty(k.shape, **f32),
               "dq": torch.empty(k.shape, **f32),
               "dh0": torch.empty((v.shape[0],) + v.shape[2:] + (k.shape[3],), **f32)}
        ws = torch.empty(delta_backward_workspace_bytes(sh), dtype=torch.uint8, device=v.device)
        ssd_delta_backward(sh, v, g, beta, k, q, h0, dy, dfinal, scale, out["dv"], out["dg"],
                           out["dbeta"], out["dk"], out["dq"], out["dh0"], ws, stream)
        return out

    return _run(call, stream, (v, g, beta, k, q, h0, dy, dfinal))


def make_norm_shape(tokens, channels, groups, x_dtype, z_dtype=None, out_dtype=None, *, act="none",
                    center=False, eps=1e-5) -> ssd_norm_shape:
    """Shape struct of the group norm; out defaults to fp32."""
    if act not in ACTS:
        raise ValueError(f"unknown activation {act!r}")
    zd = SSD_F32 if z_dtype is None else _code(z_dtype)
    od = SSD_F32 if out_dtype is None else _code(out_dtype)
    return ssd_norm_shape(int(tokens), int(channels), int(groups), _code(x_dtype), zd, od, ACTS[act],
                          int(center), eps)


def group_norm_backward_workspace_bytes(shape: ssd_norm_shape) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_group_norm_backward_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)),
           "ssd_group_norm_backward_workspace_bytes")
    return int(n.value)


def ssd_group_norm(shape, x, z, weight, bias, out, stream=None):
    _check(load_library().ssd_group_norm(ctypes.byref(shape), _p(x), _p(z), _p(weight), _p(bias),
                                         _p(out), _stream(stream)), "ssd_group_norm")


def ssd_group_norm_backward(shape, x, z, weight, bias, dy, dx, dz, dweight, dbias, workspace,
                            stream=None):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().ssd_group_norm_backward(
        ctypes.byref(shape), _p(x), _p(z), _p(weight), _p(bias), _p(dy), _p(dx), _p(dz),
        _p(dweight), _p(dbias), _p(workspace), nbytes, _stream(stream)), "ssd_group_norm_backward")


def _norm_shape_of(x, weight, bias, z, dy, groups, eps, center, act, out_dtype):
    """Shape struct of a call on x [..., channels], with the checks of its tensors."""
    if x.dim() < 1:
        raise ValueError("x is [..., channels]")
    C, dev, f32 = x.shape[-1], x.device, torch.float32
    if (z is not None) != (act in ("gate_pre", "gate_post")):
        raise ValueError("z goes with a gate, and a gate needs z")
    if z is not None and (z.shape != x.shape or z.device != dev):
        raise ValueError(f"z has x's shape {tuple(x.shape)} and device: got {tuple(z.shape)}")
    if dy is not None and (dy.shape != x.shape or dy.dtype != f32 or dy.device != dev):
        raise ValueError(f"dy is float32 {tuple(x.shape)} on {dev}: got {dy.dtype} {tuple(dy.shape)}")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and (t.shape != (C,) or t.dtype != f32 or t.device != dev):
            raise ValueError(f"{name} is float32 [{C}] on {dev}")
    return make_norm_shape(x.numel() // C if C else 0, C, groups, x.dtype, None if z is None else z.dtype,
                           out_dtype, act=act, center=center, eps=eps)


def group_norm(x, weight=None, bias=None, *, z=None, groups=1, eps=1e-5, center=False, act="none",
               out_dtype=None, stream=None):
    """Group norm of each token's channels with an activation. The statistics are each token's own, as a
    causal layer needs (torch.nn.GroupNorm takes them over a sequence too). x [..., channels] (bf16 or fp32),
    act "none", "silu", "gate_pre" (norm of x * silu(z)) or "gate_post" (norm times silu(z)), the
    mean subtracted where center is true. weight and bias are fp32 [channels] or None. Returns the
    output in out_dtype (fp32 by default)."""
    sh = _norm_shape_of(x, weight, bias, z, None, groups, eps, center, act, out_dtype)

    def call():
        out = torch.empty(x.shape, dtype=out_dtype or torch.float32, device=x.device)
        ssd_group_norm(sh, x, z, weight, bias, out, stream)
        return out

    return _run(call, stream, (x, weight, bias, z))


def group_norm_backward(x, weight, bias, dy, *, z=None, groups=1, eps=1e-5, center=False, act="none",
                        stream=None):
    """Gradients of sum(dy * group_norm(x, ...)), fp32: returns dict dx, dz, dw, db (dz, dw and db
    None where there is no z, weight or bias)."""
    sh = _norm_shape_of(x, weight, bias, z, dy, groups, eps, center, act, None)

    def call():
        f32 = dict(dtype=torch.float32, device=x.device)
        C = x.shape[-1]
        out = {"dx": torch.empty(x.shape, **f32), "dz": None if z is None else torch.empty(x.shape, **f32),
               "dw": None if weight is None else torch.empty(C, **f32),
               "db": None if bias is None else torch.empty(C, **f32)}
        ws = torch.empty(group_norm_backward_workspace_bytes(sh), dtype=torch.uint8, device=x.device)
        ssd_group_norm_backward(sh, x, z, weight, bias, dy, out["dx"], out["dz"], out["dw"], out["db"],
                                ws, stream)
        return out

    return _run(call, stream, (x, weight, bias, dy, z))
