"""Python binding of libssm: the C-ABI calls, same names, torch tensors in.

Argument marshalling only: shapes are read off the tensors, outputs and the
workspace are allocated with torch (device memory), and the call is queued
on the current torch stream.  Every step of the scan runs in the library's
CUDA kernels; if ``libssm.so`` is missing these functions raise.

Host tensors are accepted too: they are copied to the GPU on the current
stream, the call runs there, the outputs are copied back into host tensors
(pinned when the inputs were pinned) and the stream is synchronised before
returning.  This is the end-to-end path a caller with host buffers uses; for
ssm_scan_fwd it is the library's own ssm_scan_fwd_host, which overlaps the
copies in both directions with each other and with the scan.
"""
import contextlib
import ctypes

import torch

from . import _lib as L

SOFTPLUS = L.SSM_DT_SOFTPLUS
RMS_BC = L.SSM_RMSNORM_BC
RMS_DT = L.SSM_RMSNORM_DT
BETA_SIGMOID = L.GDR_BETA_SIGMOID
QK_L2NORM = L.GDR_QK_L2NORM

_IO = {torch.float32: L.SSM_F32, torch.bfloat16: L.SSM_BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return getattr(stream, "cuda_stream", stream)


class _Staging:
    """Moves host inputs to the device and device outputs back, on one stream."""

    def __init__(self, tensors):
        firsts = [t for t in tensors if t is not None]
        self.host = firsts[0].device.type == "cpu"
        self.pinned = self.host and firsts[0].is_pinned()
        self.device = torch.device("cuda", torch.cuda.current_device()) if self.host \
            else firsts[0].device

    def dev(self, t):
        if t is None:
            return None
        if self.host:
            return t.contiguous().to(self.device, non_blocking=self.pinned)
        return t.contiguous()

    def back(self, outs):
        if not self.host:
            return outs
        res = []
        for t in outs:
            if t is None:
                res.append(None)
                continue
            h = torch.empty(t.shape, dtype=t.dtype, pin_memory=self.pinned)
            h.copy_(t, non_blocking=self.pinned)
            res.append(h)
        torch.cuda.current_stream(self.device).synchronize()
        return tuple(res)


def _io_of(x):
    if x.dtype not in _IO:
        raise TypeError("io dtype must be float32 or bfloat16, got %s" % x.dtype)
    return _IO[x.dtype]


_CHECK_ALL = False


def check_every_call(on=True):
    """Make every scan call synchronise and check its status word (as if
    check=True were passed), e.g. for a test session."""
    global _CHECK_ALL
    _CHECK_ALL = bool(on)


def _check_status(ws, stream, where):
    """Synchronise ``stream`` and raise SsmError(SSM_ERR_TIMEOUT) if the call
    that used workspace ``ws`` recorded an expired device wait."""
    L.check(L.lib().ssm_workspace_status(ws.data_ptr(), stream), where)


def _workspace(nbytes, workspace, device):
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace


def ssm_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *,
                 flags=SOFTPLUS, rms_eps=1e-6, want_states=False, y=None, h_last=None,
                 workspace=None, check=False, stream=None, _write=None):
    """Mamba-1 selective scan (include/ssm.h, ssm_scan_fwd).

    x, dt, z: [b, L, C]; B, C: [b, L, G, N]; A: [C, N] f32; D, dt_bias: [C] f32;
    h0: [b, C, N] f32.  Returns (y [b, L, C], h_last [b, C, N] f32,
    states [b, L, C, N] f32 or None).  With check=True (always for host
    tensors) the stream is synchronised and an expired device wait raises."""
    sg = _Staging([x, dt, A, B, C, D, z, dt_bias, h0])
    if sg.host and _write is None:
        return _scan_host(x, dt, A, B, C, D, z, dt_bias, h0, flags, rms_eps, want_states,
                          y, h_last, workspace, sg, stream)
    x, dt, A, B, C, D, z, dt_bias, h0 = map(sg.dev, (x, dt, A, B, C, D, z, dt_bias, h0))
    if _write is not None:
        _write = (_write[0], sg.dev(_write[1]))
    b, Lq, Cn = x.shape
    G, N = B.shape[2], B.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if h_last is None:
        h_last = torch.empty((b, Cn, N), dtype=torch.float32, device=x.device)
    states = (torch.empty((b, Lq, Cn, N), dtype=torch.float32, device=x.device)
              if want_states else None)
    a = L.ScanArgs(batch=b, seqlen=Lq, channels=Cn, state=N, groups=G, io=_io_of(x),
                   flags=flags, rms_eps=rms_eps, x=_ptr(x), dt=_ptr(dt), z=_ptr(z),
                   B=_ptr(B), C=_ptr(C), A=_ptr(A), D=_ptr(D), dt_bias=_ptr(dt_bias),
                   h0=_ptr(h0), y=_ptr(y), h_last=_ptr(h_last), states=_ptr(states))
    lib = L.lib()
    nbytes = ctypes.c_size_t(0)
    L.check(lib.ssm_scan_workspace(ctypes.byref(a), ctypes.byref(nbytes)), "ssm_scan_workspace")
    ws = _workspace(nbytes.value, workspace, x.device)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    st = _stream(stream, x.device)
    if _write is None:
        L.check(lib.ssm_scan_fwd(ctypes.byref(a), st), "ssm_scan_fwd")
    else:
        L.check(lib.ssm_scan_fwd_write(ctypes.byref(a), int(_write[0]), _ptr(_write[1]), st),
                "ssm_scan_fwd_write")
    if check or sg.host or _CHECK_ALL:
        _check_status(ws, st, "ssm_scan_fwd")
    return sg.back((y, h_last, states))


def _scan_host(x, dt, A, B, C, D, z, dt_bias, h0, flags, rms_eps, want_states, y, h_last,
               workspace, sg, stream):
    """ssm_scan_fwd on host tensors through ssm_scan_fwd_host: outputs are host
    tensors (the given ones, else new ones, pinned when the inputs are), the
    workspace device memory; the stream is synchronised and the status word
    checked before returning."""
    x, dt, A, B, C, D, z, dt_bias, h0 = (None if t is None else t.contiguous()
                                         for t in (x, dt, A, B, C, D, z, dt_bias, h0))
    b, Lq, Cn = x.shape
    G, N = B.shape[2], B.shape[3]
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, pin_memory=sg.pinned)
    if h_last is None:
        h_last = torch.empty((b, Cn, N), dtype=torch.float32, pin_memory=sg.pinned)
    states = (torch.empty((b, Lq, Cn, N), dtype=torch.float32, pin_memory=sg.pinned)
              if want_states else None)
    a = L.ScanArgs(batch=b, seqlen=Lq, channels=Cn, state=N, groups=G, io=_io_of(x),
                   flags=flags, rms_eps=rms_eps, x=_ptr(x), dt=_ptr(dt), z=_ptr(z),
                   B=_ptr(B), C=_ptr(C), A=_ptr(A), D=_ptr(D), dt_bias=_ptr(dt_bias),
                   h0=_ptr(h0), y=_ptr(y), h_last=_ptr(h_last), states=_ptr(states))
    lib = L.lib()
    nbytes = ctypes.c_size_t(0)
    L.check(lib.ssm_scan_host_workspace(ctypes.byref(a), ctypes.byref(nbytes)),
            "ssm_scan_host_workspace")
    ws = _workspace(nbytes.value, workspace, sg.device)
    a.workspace, a.workspace_bytes = ws.data_ptr(), nbytes.value
    st = _stream(stream, sg.device)
    L.check(lib.ssm_scan_fwd_host(ctypes.byref(a), st), "ssm_scan_fwd_host")
    _check_status(ws, st, "ssm_scan_fwd_host")
    return y, h_last, states


def ssm_scan_fwd_write(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, t, state,
                       flags=SOFTPLUS, rms_eps=1e-6, want_states=False, y=None, h_last=None,
                       check=False, stream=None):
    """Mamba-1 scan with the state written at token t (include/ssm.h,
    ssm_scan_fwd_write): h_t is replaced by ``state`` [b, C, N] float32, y_t
    reads it and tokens t+1.. continue from it.  Arguments and results as
    ssm_scan_fwd."""
    if state.dtype != torch.float32:
        raise TypeError("state must be float32")
    return ssm_scan_fwd(x, dt, A, B, C, D, z, dt_bias, h0, flags=flags, rms_eps=rms_eps,
                        want_states=want_states, y=y, h_last=h_last, check=check,
                        stream=stream, _write=(t, state))


def ssd_workspace_bytes(**shape):
    a = L.SsdArgs(**shape)
    n = ctypes.c_size_t(0)
    L.check(L.lib().ssd_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(n)),
            "ssd_chunk_scan_workspace")
    return n.value


def ssd_conv_workspace_bytes(**shape):
    a = L.SsdConvArgs(**shape)
    n = ctypes.c_size_t(0)
    L.check(L.lib().ssd_conv_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(n)),
            "ssd_conv_chunk_scan_workspace")
    return n.value


def ssd_chunk_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *,
                       chunk=256, flags=SOFTPLUS, want_states=False, y=None, h_last=None,
                       workspace=None, check=False, stream=None):
    """Mamba-2 SSD scan (include/ssm.h, ssd_chunk_scan_fwd).

    x, z: [b, L, H, P]; dt: [b, L, H]; B, C: [b, L, G, N]; A, D, dt_bias: [H] f32;
    h0: [b, H, N, P] f32.  Returns (y, h_last [b, H, N, P], states or None).
    With check=True (always for host tensors) the stream is synchronised and
    an expired device wait raises."""
    sg = _Staging([x, dt, A, B, C, D, z, dt_bias, h0])
    x, dt, A, B, C, D, z, dt_bias, h0 = map(sg.dev, (x, dt, A, B, C, D, z, dt_bias, h0))
    b, Lq, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if y is None:
        y = torch.empty_like(x)
    if h_last is None:
        h_last = torch.empty((b, H, N, P), dtype=torch.float32, device=x.device)
    states = (torch.empty((b, Lq, H, N, P), dtype=torch.float32, device=x.device)
              if want_states else None)
    a = L.SsdArgs(batch=b, seqlen=Lq, heads=H, head_dim=P, state=N, groups=G, chunk=chunk,
                  io=_io_of(x), flags=flags, x=_ptr(x), z=_ptr(z), dt=_ptr(dt), B=_ptr(B),
                  C=_ptr(C), A=_ptr(A), D=_ptr(D), dt_bias=_ptr(dt_bias), h0=_ptr(h0),
                  y=_ptr(y), h_last=_ptr(h_last), states=_ptr(states))
    lib = L.lib()
    nbytes = ctypes.c_size_t(0)
    L.check(lib.ssd_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(nbytes)),
            "ssd_chunk_scan_workspace")
    if nbytes.value:
        workspace = _workspace(nbytes.value, workspace, x.device)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), nbytes.value
    st = _stream(stream, x.device)
    L.check(lib.ssd_chunk_scan_fwd(ctypes.byref(a), st), "ssd_chunk_scan_fwd")
    if nbytes.value and (check or sg.host or _CHECK_ALL):
        _check_status(workspace, st, "ssd_chunk_scan_fwd")
    return sg.back((y, h_last, states))


def ssd_conv_chunk_scan_fwd(xBC, conv_w, dt, A, *, heads, state, groups=1, conv_bias=None,
                            conv_state_in=None, want_conv_state=False, D=None, z=None,
                            dt_bias=None, h0=None, chunk=256, flags=SOFTPLUS, y=None,
                            h_last=None, conv_state_out=None, workspace=None, check=False,
                            stream=None):
    """The Mamba-2 mixer's causal convolution fused in front of the SSD scan
    (include/ssm.h, ssd_conv_chunk_scan_fwd).

    xBC: [b, L, heads*64 + 2*groups*state] bf16, before the convolution;
    conv_w: [channels, 4] f32; conv_bias: [channels]; conv_state_in:
    [b, channels, 3] f32; dt: [b, L, H]; z: [b, L, H, 64]; A, D, dt_bias: [H];
    h0: [b, H, N, 64].  Returns (y, h_last, conv_state_out or None)."""
    sg = _Staging([xBC, conv_w, dt, A, conv_bias, conv_state_in, D, z, dt_bias, h0])
    xBC, conv_w, dt, A, conv_bias, conv_state_in, D, z, dt_bias, h0 = map(
        sg.dev, (xBC, conv_w, dt, A, conv_bias, conv_state_in, D, z, dt_bias, h0))
    b, Lq, ctot = xBC.shape
    P = (ctot - 2 * groups * state) // heads
    if y is None:
        y = torch.empty((b, Lq, heads, P), dtype=xBC.dtype, device=xBC.device)
    if h_last is None:
        h_last = torch.empty((b, heads, state, P), dtype=torch.float32, device=xBC.device)
    if conv_state_out is None and want_conv_state:
        conv_state_out = torch.empty((b, ctot, 3), dtype=torch.float32, device=xBC.device)
    a = L.SsdConvArgs(batch=b, seqlen=Lq, heads=heads, head_dim=P, state=state, groups=groups,
                      chunk=chunk, io=_io_of(xBC), flags=flags, xBC=_ptr(xBC),
                      conv_w=_ptr(conv_w), conv_bias=_ptr(conv_bias),
                      conv_state_in=_ptr(conv_state_in), conv_state_out=_ptr(conv_state_out),
                      z=_ptr(z), dt=_ptr(dt), A=_ptr(A), D=_ptr(D), dt_bias=_ptr(dt_bias),
                      h0=_ptr(h0), y=_ptr(y), h_last=_ptr(h_last))
    lib = L.lib()
    nbytes = ctypes.c_size_t(0)
    L.check(lib.ssd_conv_chunk_scan_workspace(ctypes.byref(a), ctypes.byref(nbytes)),
            "ssd_conv_chunk_scan_workspace")
    workspace = _workspace(nbytes.value, workspace, xBC.device)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), nbytes.value
    st = _stream(stream, xBC.device)
    L.check(lib.ssd_conv_chunk_scan_fwd(ctypes.byref(a), st), "ssd_conv_chunk_scan_fwd")
    if Lq and (check or sg.host or _CHECK_ALL):
        _check_status(workspace, st, "ssd_conv_chunk_scan_fwd")
    return sg.back((y, h_last, conv_state_out))


def ssm_scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, *, flags=SOFTPLUS,
                  rms_eps=1e-6, y=None, stream=None):
    """One decode token (include/ssm.h, ssm_scan_step); ``state`` is updated in place.

    Mamba-1: state [b, C, N], x/dt/z [b, C], B/C [b, G, N], A [C, N].
    Mamba-2: state [b, H, N, P], x/z [b, H, P], dt [b, H], B/C [b, G, N], A [H].
    Returns y (and, for host tensors, the updated state copied back)."""
    if state.dim() == 3:
        kind, (b, U, N), P = L.SSM_STEP_MAMBA1, state.shape, 1
    elif state.dim() == 4:
        kind, (b, U, N, P) = L.SSM_STEP_MAMBA2, state.shape
    else:
        raise ValueError("state must be [b, C, N] or [b, H, N, P]")
    sg = _Staging([state, x, dt, A, B, C, D, z, dt_bias])
    host_state = state
    state = state if not sg.host else state.contiguous().to(sg.device, non_blocking=sg.pinned)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous (it is updated in place)")
    x, dt, A, B, C, D, z, dt_bias = map(sg.dev, (x, dt, A, B, C, D, z, dt_bias))
    G = B.shape[1]
    if y is None:
        y = torch.empty_like(x)
    a = L.StepArgs(kind=kind, io=_io_of(x), flags=flags, rms_eps=rms_eps, batch=b, units=U,
                   head_dim=P, state=N, groups=G, x=_ptr(x), dt=_ptr(dt), z=_ptr(z),
                   B=_ptr(B), C=_ptr(C), A=_ptr(A), D=_ptr(D), dt_bias=_ptr(dt_bias),
                   state_io=_ptr(state), y=_ptr(y))
    L.check(L.lib().ssm_scan_step(ctypes.byref(a), _stream(stream, x.device)), "ssm_scan_step")
    if sg.host:
        y_h, st_h = sg.back((y, state))
        host_state.copy_(st_h)
        return y_h
    return y


def ssm_conv1d_fwd(x, w, bias=None, state=None, *, silu=True, u=None, state_out=None,
                   in_place=False, stream=None):
    """The mixers' causal depthwise convolution, then silu (include/ssm.h,
    ssm_conv1d_fwd).

    x: [b, L, C] (float32 or bfloat16); w: [C, W] float32 (W <= 4); bias: [C]
    float32; state: [b, C, W - 1] float32, the inputs before the sequence
    (oldest first) or None for a sequence start.  Returns (u, state_out):
    u [b, L, C] in x's dtype and the last W - 1 inputs.  With in_place=True
    the state tensor itself is updated (the decode form, one token)."""
    sg = _Staging([x, w, bias, state])
    host_state = state
    x, w, bias = map(sg.dev, (x, w, bias))
    if state is not None:
        state = sg.dev(state)
    b, Lq, C = x.shape
    W = w.shape[1]
    if u is None:
        u = torch.empty_like(x)
    if in_place:
        if state is None:
            raise ValueError("in_place needs a state tensor")
        state_out = state
    elif state_out is None:
        state_out = torch.empty((b, C, max(W - 1, 0)), dtype=torch.float32, device=x.device)
    a = L.ConvArgs(batch=b, seqlen=Lq, channels=C, width=W, io=_io_of(x),
                   flags=L.SSM_CONV_SILU if silu else 0, x=_ptr(x), w=_ptr(w),
                   bias=_ptr(bias), state_in=_ptr(state), u=_ptr(u),
                   state_out=_ptr(state_out) if W > 1 else None)
    L.check(L.lib().ssm_conv1d_fwd(ctypes.byref(a), _stream(stream, x.device)),
            "ssm_conv1d_fwd")
    if sg.host:
        u_h, so_h = sg.back((u, state_out))
        if in_place:
            host_state.copy_(so_h)
        return u_h, so_h
    return u, state_out


def ssm_gated_rmsnorm_fwd(y, z=None, weight=None, eps=1e-5, *, out=None, stream=None):
    """The Mamba-2 mixer's gated norm (include/ssm.h, ssm_gated_rmsnorm_fwd):
    y * silu(z), RMS-normalised over the last axis (the mixer's whole width,
    heads x head_dim), times weight.  y, z: [..., width] (float32 or
    bfloat16); weight: [width] float32.  out may be y (in place)."""
    sg = _Staging([y, z, weight])
    y, z, weight = map(sg.dev, (y, z, weight))
    width = y.shape[-1]
    rows = y.numel() // width if width else 0
    if out is None:
        out = torch.empty_like(y)
    a = L.GatedNormArgs(rows=rows, width=width, io=_io_of(y), flags=0, eps=eps, y=_ptr(y),
                        z=_ptr(z), weight=_ptr(weight), out=_ptr(out))
    L.check(L.lib().ssm_gated_rmsnorm_fwd(ctypes.byref(a), _stream(stream, y.device)),
            "ssm_gated_rmsnorm_fwd")
    if sg.host:
        return sg.back((out,))[0]
    return out


def ssd_attention_fwd(dt, A, B, C, dt_bias=None, *, flags=SOFTPLUS, alpha=None,
                      workspace=None, stream=None):
    """The hidden attention of the SSD map (include/ssm.h, ssd_attention_fwd):
    alpha [b, H, L, L] float32 (query t, key s), causal, with
    y_t = sum_s alpha[t, s] x_s + D x_t from a zero state.
    dt [b, L, H] and B, C [b, L, G, N] (float32 or bfloat16); A, dt_bias [H]."""
    sg = _Staging([dt, A, B, C, dt_bias])
    dt, A, B, C, dt_bias = map(sg.dev, (dt, A, B, C, dt_bias))
    b, Lq, H = dt.shape
    G, N = B.shape[2], B.shape[3]
    if alpha is None:
        alpha = torch.empty((b, H, Lq, Lq), dtype=torch.float32, device=dt.device)
    a = L.AttnArgs(batch=b, seqlen=Lq, heads=H, state=N, groups=G, io=_io_of(dt), flags=flags,
                   dt=_ptr(dt), B=_ptr(B), C=_ptr(C), A=_ptr(A), dt_bias=_ptr(dt_bias),
                   alpha=_ptr(alpha))
    lib = L.lib()
    nbytes = ctypes.c_size_t(0)
    L.check(lib.ssd_attention_workspace(ctypes.byref(a), ctypes.byref(nbytes)),
            "ssd_attention_workspace")
    if nbytes.value:
        if workspace is None or workspace.numel() * workspace.element_size() < nbytes.value:
            workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=dt.device)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), nbytes.value
    L.check(lib.ssd_attention_fwd(ctypes.byref(a), _stream(stream, dt.device)),
            "ssd_attention_fwd")
    if sg.host:
        return sg.back((alpha,))[0]
    return alpha


# ------------------------------------------------------------ gated delta rule

_ANY_ROW = (1 << 31) - 1  # rows of a cache that is not there: only negative slots are out of range
_GDR_FLAGS = SOFTPLUS | BETA_SIGMOID | QK_L2NORM


@contextlib.contextmanager
def _scope(t, stream):
    """The device of ``t`` and ``stream`` (a torch stream or a raw handle)
    current, so that copies, outputs and workspaces belong to the stream that
    uses them."""
    device = t.device if t.is_cuda else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream) or 0, device)
        with torch.cuda.stream(stream):
            yield


def _elsewhere(t, stream):
    """Whether a call on ``t`` needs _scope."""
    return stream is not None or (t.is_cuda and t.get_device() != torch._C._cuda_getDevice())


def _at(t):
    return 0 if t is None else t.data_ptr()


def _raw_stream(t):
    """Handle of the current stream of ``t``'s device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _rows(t, inner, align):
    """``t`` [lead.., inner..] as the kernels take it: rows of dense inner
    values at one stride.  Returns (t, stride), stride 0 for a dense tensor; a
    tensor laid out otherwise, or off ``align`` bytes, is copied."""
    aligned = t.data_ptr() % align == 0
    if t.is_contiguous():
        return (t if aligned else t.clone()), 0
    shape, strides, lead = t.shape, t.stride(), t.dim() - inner
    if aligned and inner == 2 and lead == 1:  # [b, heads, dim], the usual slice
        row, want = strides[0], shape[1] * shape[2]
        if strides[2] == 1 and strides[1] == shape[2] and row >= want:
            return t, row
    elif aligned and inner == 1 and lead == 1 and strides[1] == 1 and strides[0] >= shape[1]:
        return t, strides[0]
    want, row = 1, 0
    for i in range(t.dim() - 1, -1, -1):
        if shape[i] == 1:
            continue
        if i < lead and not row:  # the innermost axis of tokens sets the stride
            row = strides[i]
            aligned = aligned and row >= want
            want = row
        aligned = aligned and strides[i] == want
        want *= shape[i]
    return (t, row) if aligned else (t.contiguous(), 0)


def _expect(name, t, dtype, shape, at):
    """``at``: index of the device the other tensors are on (-1: the host)."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == at):
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != shape:
        raise ValueError("%s must be %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != at:
        raise ValueError("%s is on %s, the other tensors on %s" % (
            name, t.device, "the host" if at < 0 else "cuda:%d" % at))


def _own(name, t):
    """An output or cache tensor: written where it lies, so it must be dense."""
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (it is written in place)" % name)
    return t


def _gdr_inputs(q, k, v, dt, A, beta, dt_bias):
    """Checks the tensors a scan and a step share; returns their sizes."""
    shape, key, io, dev = v.shape, q.shape, v.dtype, v.get_device()
    gate, h, V, hk, K = shape[:-1], shape[-2], shape[-1], key[-2], key[-1]
    # what holds in an ordinary call first, in one line: a small call's host time counts
    if not (q.dtype is io and k.dtype is io and beta.dtype is io and k.shape == key
            and key[:-2] == shape[:-2] and beta.shape == gate and q.get_device() == dev
            and k.get_device() == dev and beta.get_device() == dev):
        lead = tuple(shape[:-2])
        _expect("q", q, io, lead + (hk, K), dev)
        _expect("k", k, io, lead + (hk, K), dev)
        _expect("beta", beta, io, lead + (h,), dev)
    if dt is not None:
        _expect("dt", dt, io, gate, dev)
        _expect("A", A, torch.float32, (h,), dev)
        _expect("dt_bias", dt_bias, torch.float32, (h,), dev)
    return hk, K, h, V


def gdr_chunk_scan_fwd(q, k, v, dt, A, beta, dt_bias=None, h0=None, *, scale=None,
                       flags=_GDR_FLAGS, l2_eps=1e-6, cu_seqlens=None, slots=None, y=None,
                       h_last=None, workspace=None, check=False, stream=None):
    """The gated delta rule over prompts (include/ssm.h, gdr_chunk_scan_fwd).

    q, k: [b, L, Hk, K]; v: [b, L, H, V]; dt, beta: [b, L, H] (dt None: no
    decay); A, dt_bias: [H] f32; h0: [b, H, K, V] f32; scale: K ** -0.5 unless
    given.  Returns (y [b, L, H, V], h_last [b, H, K, V] f32).

    With cu_seqlens [n + 1] int32, b is 1 and the sequences lie one behind the
    other; h0 and h_last then have a row per sequence or, with slots [n] int32,
    are caches of any number of rows, sequence i's state in row slots[i] (a
    sequence whose slot is out of range is skipped; h_last must be given, and
    may be h0).  Slices of wider tensors (dense heads, one stride between
    tokens) are read where they lie.  With check=True (always for host
    tensors) the stream is synchronised and an expired device wait raises."""
    if _elsewhere(v, stream):
        with _scope(v, stream):
            return gdr_chunk_scan_fwd(q, k, v, dt, A, beta, dt_bias, h0, scale=scale, flags=flags,
                                      l2_eps=l2_eps, cu_seqlens=cu_seqlens, slots=slots, y=y,
                                      h_last=h_last, workspace=workspace, check=check)
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("q, k and v must be [b, L, heads, dim]")
    hk, K, h, V = _gdr_inputs(q, k, v, dt, A, beta, dt_bias)
    b, Lq = v.shape[:2]
    dev = v.get_device()
    n = b
    if cu_seqlens is not None:
        n = cu_seqlens.numel() - 1
        if b != 1 or n < 0:
            raise ValueError("cu_seqlens needs batch 1 and n + 1 entries")
        _expect("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), dev)
    rows = n
    if slots is not None:
        _expect("slots", slots, torch.int32, (n,), dev)
        if h_last is None:
            raise ValueError("slots needs h_last, the cache the states go to")
        rows = h_last.shape[0]
    _expect("h0", h0, torch.float32, (rows, h, K, V), dev)
    _expect("h_last", h_last, torch.float32, (rows, h, K, V), dev)
    _expect("y", y, v.dtype, (b, Lq, h, V), dev)
    if workspace is not None:  # (device memory for host tensors too)
        if not workspace.is_cuda or workspace.get_device() != (
                dev if dev >= 0 else torch.cuda.current_device()):
            raise ValueError("workspace is on %s, the call runs on %s" % (
                workspace.device, "cuda:%d" % dev if dev >= 0 else "the current CUDA device"))
        _own("workspace", workspace)
    host_y, host_h = y, h_last
    sg = None
    if not v.is_cuda:
        sg = _Staging([v])
        same = h0 is not None and h_last is not None and h0.data_ptr() == h_last.data_ptr()
        q, k, v, dt, A, beta, dt_bias, h0, cu_seqlens, slots, y = map(
            sg.dev, (q, k, v, dt, A, beta, dt_bias, h0, cu_seqlens, slots, y))
        h_last = h0 if same else sg.dev(h_last)
    q, q_row = _rows(q, 2, 16)
    k, k_row = _rows(k, 2, 16)
    v, v_row = _rows(v, 2, 16)
    dt, dt_row = (None, 0) if dt is None else _rows(dt, 1, dt.element_size())
    beta, beta_row = _rows(beta, 1, beta.element_size())
    if h0 is not None and h0 is not h_last:
        h0 = h0.contiguous()
    y = v.new_empty((b, Lq, h, V)) if y is None else _own("y", y)
    h_last = (v.new_empty((n, h, K, V), dtype=torch.float32) if h_last is None
              else _own("h_last", h_last))
    A, dt_bias = _dense(A), _dense(dt_bias)
    cu_seqlens, slots = _dense(cu_seqlens), _dense(slots)
    fields = (b, Lq, h, hk, K, V, n, rows, q_row, k_row, v_row, dt_row, beta_row, _io_of(v), flags,
              K ** -0.5 if scale is None else scale, l2_eps, q.data_ptr(), k.data_ptr(),
              v.data_ptr(), _at(dt), beta.data_ptr(), _at(A), _at(dt_bias), _at(h0),
              _at(cu_seqlens), _at(slots), y.data_ptr(), h_last.data_ptr())
    nbytes = ctypes.c_size_t(0)
    L.check(L.packed("gdr_chunk_scan_workspace")(L.GDR_SCAN(*fields, 0, 0), ctypes.addressof(nbytes)),
            "gdr_chunk_scan_workspace")
    if nbytes.value and (workspace is None
                         or workspace.numel() * workspace.element_size() < nbytes.value):
        workspace = v.new_empty(nbytes.value, dtype=torch.uint8)
    st = _raw_stream(y)
    L.check(L.packed("gdr_chunk_scan_fwd")(
        L.GDR_SCAN(*fields, workspace.data_ptr() if nbytes.value else 0, nbytes.value), st),
        "gdr_chunk_scan_fwd")
    if nbytes.value and n and (check or sg or _CHECK_ALL):
        _check_status(workspace, st, "gdr_chunk_scan_fwd")
    if sg is None:
        return y, h_last
    return _home(sg, (host_y, host_h), (y, h_last))


def _dense(t):
    return None if t is None else t.contiguous()


def _home(sg, given, outs):
    """Device outputs back in host memory: into the caller's own tensors where
    there are some."""
    outs = sg.back(outs)
    return tuple(o if g is None else g.copy_(o) for g, o in zip(given, outs))


def gdr_scan_step(state, q, k, v, dt, A, beta, dt_bias=None, *, scale=None, flags=_GDR_FLAGS,
                  l2_eps=1e-6, slots=None, y=None, stream=None):
    """One decode token of the gated delta rule per sequence (include/ssm.h,
    gdr_scan_step); ``state`` is updated in place.

    q, k: [b, Hk, K]; v: [b, H, V]; dt, beta: [b, H]; state: [b, H, K, V] f32
    or, with slots [b] int32, a cache of any number of rows (a row whose slot
    is out of range is skipped, its y left as it was).  Returns y [b, H, V]."""
    if _elsewhere(v, stream):
        with _scope(v, stream):
            return gdr_scan_step(state, q, k, v, dt, A, beta, dt_bias, scale=scale, flags=flags,
                                 l2_eps=l2_eps, slots=slots, y=y)
    if v.dim() != 3 or q.dim() != 3:
        raise ValueError("q, k and v must be [b, heads, dim]")
    hk, K, h, V = _gdr_inputs(q, k, v, dt, A, beta, dt_bias)
    b, dev = v.shape[0], v.get_device()
    rows = state.shape[0] if slots is not None else b
    _expect("slots", slots, torch.int32, (b,), dev)
    _expect("state", _own("state", state), torch.float32, (rows, h, K, V), dev)
    _expect("y", y, v.dtype, (b, h, V), dev)
    host_y, host_state, sg = y, state, None
    if not v.is_cuda:
        sg = _Staging([v])
        q, k, v, dt, A, beta, dt_bias, state, slots, y = map(
            sg.dev, (q, k, v, dt, A, beta, dt_bias, state, slots, y))
    q, q_row = _rows(q, 2, 16)
    k, k_row = _rows(k, 2, 16)
    v, v_row = _rows(v, 2, 16)
    dt, dt_row = (None, 0) if dt is None else _rows(dt, 1, dt.element_size())
    beta, beta_row = _rows(beta, 1, beta.element_size())
    y = v.new_empty((b, h, V)) if y is None else _own("y", y)
    A, dt_bias, slots = _dense(A), _dense(dt_bias), _dense(slots)
    L.check(L.packed("gdr_scan_step")(
        L.GDR_STEP(b, h, hk, K, V, rows, q_row, k_row, v_row, dt_row, beta_row, _io_of(v), flags,
                   K ** -0.5 if scale is None else scale, l2_eps, q.data_ptr(), k.data_ptr(),
                   v.data_ptr(), _at(dt), beta.data_ptr(), _at(A), _at(dt_bias), _at(slots),
                   state.data_ptr(), y.data_ptr()), _raw_stream(y)), "gdr_scan_step")
    if sg is None:
        return y
    return _home(sg, (host_y, host_state), (y, state))[0]


def gdr_gated_rmsnorm_fwd(x, z=None, weight=None, eps=1e-5, *, out=None, stream=None):
    """The gated delta rule's norm (include/ssm.h, gdr_gated_rmsnorm_fwd): x
    [.., H, W] RMS-normalised over its last axis, times weight [W] f32, times
    silu(z).  z: x's shape, or None; a slice of a wider tensor (dense heads,
    one stride between tokens) is read where it lies.  out may be x."""
    if _elsewhere(x, stream):
        with _scope(x, stream):
            return gdr_gated_rmsnorm_fwd(x, z, weight, eps, out=out)
    if x.dim() < 2:
        raise ValueError("x must be [.., heads, width]")
    shape, dev = x.shape, x.get_device()
    h, W = shape[-2], shape[-1]
    _expect("z", z, x.dtype, shape, dev)
    _expect("weight", weight, torch.float32, (W,), dev)
    _expect("out", out, x.dtype, shape, dev)
    host_out, sg = out, None
    if not x.is_cuda:
        sg = _Staging([x])
        same = out is x
        x, z, weight, out = map(sg.dev, (x, z, weight, out))
        out = x if same else out
    z, z_row = (None, 0) if z is None else _rows(z if z.dim() > 2 else z[None], 2, 16)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    x = _own("out", out) if x is out else x.contiguous()
    tokens = x.numel() // (h * W) if h * W else 0
    weight = _dense(weight)
    L.check(L.packed("gdr_gated_rmsnorm_fwd")(
        L.GDR_NORM(tokens, h, W, z_row, _io_of(x), 0, eps, x.data_ptr(), _at(z), _at(weight),
                   _own("out", out).data_ptr()), _raw_stream(out)), "gdr_gated_rmsnorm_fwd")
    return out if sg is None else _home(sg, (host_out,), (out,))[0]


def ssm_conv1d_packed_fwd(x, w, bias=None, state=None, *, cu_seqlens, slots=None, silu=True,
                          u=None, stream=None):
    """The mixers' causal depthwise convolution, then silu, over packed
    sequences (include/ssm.h, ssm_conv1d_packed_fwd).

    x: [T, C]; w: [C, W] f32 (W <= 4); bias: [C] f32; cu_seqlens: [n + 1]
    int32; state: [n, C, W - 1] f32, updated in place, or with slots [n] int32
    a cache of any number of rows, or None (zeros before every sequence).
    Returns (u [T, C], state); rows of no sequence are left as they were."""
    if _elsewhere(x, stream):
        with _scope(x, stream):
            return ssm_conv1d_packed_fwd(x, w, bias, state, cu_seqlens=cu_seqlens, slots=slots,
                                         silu=silu, u=u)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [T, C] and w [C, W]")
    T, C = x.shape
    W, n, dev = w.shape[1], cu_seqlens.numel() - 1, x.get_device()
    if n < 0:
        raise ValueError("cu_seqlens must have n + 1 entries")
    _expect("w", w, torch.float32, (C, W), dev)
    _expect("bias", bias, torch.float32, (C,), dev)
    _expect("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), dev)
    _expect("slots", slots, torch.int32, (n,), dev)
    rows = n if slots is None else _ANY_ROW if state is None else state.shape[0]
    if state is not None:
        _expect("state", _own("state", state), torch.float32, (rows, C, W - 1), dev)
    _expect("u", u, x.dtype, (T, C), dev)
    host_u, host_state, sg = u, state, None
    if not x.is_cuda:
        sg = _Staging([x])
        x, w, bias, state, cu_seqlens, slots, u = map(
            sg.dev, (x, w, bias, state, cu_seqlens, slots, u))
    x, x_row = _rows(x, 1, 16)
    u = x.new_empty((T, C)) if u is None else _own("u", u)
    w, bias, cu_seqlens, slots = _dense(w), _dense(bias), _dense(cu_seqlens), _dense(slots)
    L.check(L.packed("ssm_conv1d_packed_fwd")(
        L.CONV_PACKED(T, C, W, n, rows, x_row, _io_of(x), L.SSM_CONV_SILU if silu else 0,
                      x.data_ptr(), w.data_ptr(), _at(bias), _at(state), cu_seqlens.data_ptr(),
                      _at(slots), u.data_ptr()), _raw_stream(u)), "ssm_conv1d_packed_fwd")
    if sg is None:
        return u, state
    if state is None:
        return _home(sg, (host_u,), (u,))[0], None
    return _home(sg, (host_u, host_state), (u, state))
