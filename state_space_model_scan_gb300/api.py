"""Torch-facing wrappers around the C ABI.

They allocate outputs and workspace with torch, marshal pointers/strides/stream
into the ABI structs and raise on a non-OK status.  All arithmetic runs in
libssd.so.
"""
import functools
import inspect

import torch

from . import _lib


def _on_stream(f):
    """f with a ``stream`` argument and a tensor first.  The tensor's GPU is the current one meanwhile (the library launches
    there, and a stream of None is that GPU's current one).  What f allocates comes from the given stream's memory (a block that
    the caller's stream has freed may still be in use there), and the caller's stream, which will read the outputs, is noted for them."""
    params = list(inspect.signature(f).parameters)
    first, at = params[0], params.index("stream")

    @functools.wraps(f)
    def call(*args, **kw):
        dev = (args[0] if args else kw[first]).device
        if dev.type == "cuda" and dev.index != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return call(*args, **kw)
        stream = kw.get("stream") if len(args) <= at else args[at]
        if stream is None:
            return f(*args, **kw)
        caller = torch.cuda.current_stream(stream.device)
        with torch.cuda.stream(stream):
            out = f(*args, **kw)
        for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
            if t is not None and t.numel() > 0:
                t.record_stream(caller)
        return out
    return call


class Workspace:
    """A reusable device workspace: grows to the largest size requested."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None

    def get(self, nbytes):
        nbytes = max(int(nbytes), 256)
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device or "cuda")
        self.buf.record_stream(torch.cuda.current_stream(self.buf.device))   # it may be another than when it was allocated
        return self.buf


def _nseqs(x, cu_seqlens):
    return (cu_seqlens.numel() - 1) if cu_seqlens is not None else x.shape[0]


@_on_stream
def ssd_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_states=None, cu_seqlens=None,
                chunk_size=128, return_final_states=True, algo="auto", seg_chunks=0, workspace=None,
                y=None, final_states=None, stream=None, keep_chunk_states=False, chunk_states=None,
                state_dtype=None):
    """y, final_states = SSD scan (see include/ssd.h for the definition and layouts).

    x, z: [B, L, H, P]; dt: [B, L, H] fp32; A, D, dt_bias: [H] fp32; B, C: [B, L, G, N];
    initial_states: [S, H, P, N] fp32 or bf16; cu_seqlens: int32 [S+1] (batch 1).
    state_dtype: storage dtype of the returned final states (default: that of initial_states,
    else fp32); the scan itself carries its state in fp32 either way.
    keep_chunk_states: also return the carried chunk states (a uint8 device buffer, tensor-core
    path only; raises SSDError(SSD_ERR_UNSUPPORTED) otherwise) for ssd_backward(chunk_states=...),
    which then skips their recompute.  chunk_states: a caller-owned buffer to fill instead.
    """
    Bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    S = _nseqs(x, cu_seqlens)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if final_states is None and return_final_states:
        sdt = state_dtype or (initial_states.dtype if initial_states is not None else torch.float32)
        final_states = torch.empty(S, H, P, N, dtype=sdt, device=x.device)
    prob = _lib.problem(Bsz, L, H, P, G, N, chunk_size, S if cu_seqlens is not None else 0, algo, seg_chunks)
    args = _lib.fwd_args(x, dt, A, B, C, y, D=D, z=z, dt_bias=dt_bias, initial_states=initial_states,
                         final_states=final_states, cu_seqlens=cu_seqlens)
    if keep_chunk_states or chunk_states is not None:
        need = _lib.chunk_states_size(prob, args)
        if chunk_states is None:
            chunk_states = torch.empty(need, dtype=torch.uint8, device=x.device)
        if chunk_states.numel() * chunk_states.element_size() < need:
            raise ValueError("chunk_states holds %d bytes, %d needed" % (chunk_states.numel() * chunk_states.element_size(), need))
        args.chunk_states = chunk_states.data_ptr()
    nbytes = _lib.fwd_workspace_size(prob, args)
    ws = workspace.get(nbytes) if workspace is not None else torch.empty(max(nbytes, 256), dtype=torch.uint8,
                                                                          device=x.device)
    _lib.check(_lib.ssd_fwd(prob, args, ws, stream), "ssd_fwd")
    if keep_chunk_states:
        return y, final_states, chunk_states
    return y, final_states


@_on_stream
def ssd_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, initial_states=None, dfinal_states=None,
                 cu_seqlens=None, chunk_size=128, algo="auto", seg_chunks=0, bwd_heads=0, workspace=None,
                 stream=None, chunk_states=None):
    """Gradients of sum(dy*y) + sum(dfinal_states*final_states).  Returns a dict with
    dx, ddt, dA, dB, dC and, when the matching input is given, dD, dz, ddt_bias, dinitial_states.
    bwd_heads: heads per CTA of the tensor-core gradient kernel (0 = library choice).
    chunk_states: the buffer ssd_forward(keep_chunk_states=True) returned for the same inputs."""
    Bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    S = _nseqs(x, cu_seqlens)
    dev = x.device
    g = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=dev),
             ddt=torch.empty(dt.shape, dtype=torch.float32, device=dev),
             dA=torch.empty(H, dtype=torch.float32, device=dev),
             dB=torch.empty(B.shape, dtype=B.dtype, device=dev),
             dC=torch.empty(C.shape, dtype=C.dtype, device=dev))
    if D is not None:
        g["dD"] = torch.empty(H, dtype=torch.float32, device=dev)
    if z is not None:
        g["dz"] = torch.empty(z.shape, dtype=z.dtype, device=dev)
    if dt_bias is not None:
        g["ddt_bias"] = torch.empty(H, dtype=torch.float32, device=dev)
    if initial_states is not None:   # in the initial states' storage dtype
        g["dinitial_states"] = torch.empty(S, H, P, N, dtype=initial_states.dtype, device=dev)
    prob = _lib.problem(Bsz, L, H, P, G, N, chunk_size, S if cu_seqlens is not None else 0, algo, seg_chunks,
                        bwd_heads)
    fa = _lib.fwd_args(x, dt, A, B, C, None, D=D, z=z, dt_bias=dt_bias, initial_states=initial_states,
                       cu_seqlens=cu_seqlens, chunk_states=chunk_states)
    ba = _lib.bwd_args(fa, dy, g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], dD=g.get("dD"), dz=g.get("dz"),
                       ddt_bias=g.get("ddt_bias"), dinitial_states=g.get("dinitial_states"),
                       dfinal_states=dfinal_states)
    nbytes = _lib.bwd_workspace_size(prob, ba)
    ws = workspace.get(nbytes) if workspace is not None else torch.empty(max(nbytes, 256), dtype=torch.uint8,
                                                                          device=dev)
    _lib.check(_lib.ssd_bwd(prob, ba, ws, stream), "ssd_bwd")
    return g


def _rows(t, width):
    """[..., width] (features contiguous, rows at a common stride) as a 2-D [rows, width] view."""
    return t.reshape(-1, width)


@_on_stream
def gated_norm_forward(y, weight, group_size, z=None, eps=1e-5, layer_norm=False, gate_after=False, stream=None):
    """out, rstd = the gated normalisation of y over groups of `group_size` features (see
    include/ssd.h, ssd_gated_norm_fwd): RMS (default) or LayerNorm (layer_norm=True, no bias)
    of u = y silu(z), times weight; with gate_after=True, of u = y, times weight and silu(z).
    y, z: [..., width]."""
    width = y.shape[-1]
    y2 = _rows(y, width)
    z2 = _rows(z, width) if z is not None else None
    out = torch.empty_like(y2)
    rstd = torch.empty(y2.shape[0], width // group_size, dtype=torch.float32, device=y.device)
    prob = _lib.norm_problem(y2.shape[0], width, group_size, eps, y.dtype, layer_norm, gate_after)
    _lib.check(_lib.gated_norm_fwd(prob, y2, z2, weight, out, rstd, stream), "ssd_gated_norm_fwd")
    return out.reshape(y.shape), rstd


@_on_stream
def gated_norm_backward(y, weight, rstd, dout, group_size, z=None, eps=1e-5, layer_norm=False, gate_after=False,
                        stream=None):
    """dy, dz (None without z), dweight: gradients of sum(dout * out) (same options as the forward)."""
    width = y.shape[-1]
    y2, d2 = _rows(y, width), _rows(dout, width)
    z2 = _rows(z, width) if z is not None else None
    dy = torch.empty_like(y2)
    dz = torch.empty_like(z2) if z is not None else None
    dw = torch.empty(width, dtype=torch.float32, device=y.device)
    prob = _lib.norm_problem(y2.shape[0], width, group_size, eps, y.dtype, layer_norm, gate_after)
    ws = torch.empty(max(_lib.gated_norm_bwd_workspace_size(prob), 16), dtype=torch.uint8, device=y.device)
    _lib.check(_lib.gated_norm_bwd(prob, y2, z2, weight, rstd, d2, dy, dz, dw, ws, stream), "ssd_gated_norm_bwd")
    return dy.reshape(y.shape), (dz.reshape(z.shape) if dz is not None else None), dw


@_on_stream
def conv1d_forward(xbc, weight, bias=None, cu_seqlens=None, silu=True, stream=None):
    """Causal depthwise conv1d (+ SiLU) over the sequence axis of xbc [batch, seqlen, channels]
    (see include/ssd.h, ssd_conv1d_fwd); packed sequences (cu_seqlens, batch 1) never mix."""
    Bsz, L, Cn = xbc.shape
    out = torch.empty(Bsz, L, Cn, dtype=xbc.dtype, device=xbc.device)
    prob = _lib.conv_problem(Bsz, L, Cn, weight.shape[1], 0 if cu_seqlens is None else cu_seqlens.numel() - 1,
                             xbc.dtype, silu)
    _lib.check(_lib.conv1d_fwd(prob, xbc, weight, bias, cu_seqlens, out, stream), "ssd_conv1d_fwd")
    return out


@_on_stream
def conv1d_backward(xbc, weight, dout, bias=None, cu_seqlens=None, silu=True, stream=None):
    """dxbc, dweight, dbias (None without bias): gradients of sum(dout * conv1d_forward(...))."""
    Bsz, L, Cn = xbc.shape
    du = torch.empty(Bsz, L, Cn, dtype=xbc.dtype, device=xbc.device)
    dw = torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    prob = _lib.conv_problem(Bsz, L, Cn, weight.shape[1], 0 if cu_seqlens is None else cu_seqlens.numel() - 1,
                             xbc.dtype, silu)
    ws = torch.empty(max(_lib.conv1d_bwd_workspace_size(prob), 16), dtype=torch.uint8, device=xbc.device)
    _lib.check(_lib.conv1d_bwd(prob, xbc, weight, bias, cu_seqlens, dout, du, dw, db, ws, stream), "ssd_conv1d_bwd")
    return du, dw, db


def split_xbc(xbc, nheads, headdim, ngroups, dstate):
    """x [B, L, H, P], B and C [B, L, G, N] as views of the packed xbc [B, L, H P + 2 G N] (no copy);
    the scan takes them as they are (strided tensors)."""
    Bsz, L, Cn = xbc.shape
    hp, gn = nheads * headdim, ngroups * dstate
    assert Cn == hp + 2 * gn
    x = xbc[..., :hp].unflatten(-1, (nheads, headdim))
    Bm = xbc[..., hp:hp + gn].unflatten(-1, (ngroups, dstate))
    Cm = xbc[..., hp + gn:].unflatten(-1, (ngroups, dstate))
    return x, Bm, Cm


class SSDFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run in libssd.so.  On the tensor-core
    path the forward keeps its carried chunk states for the backward."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens, chunk_size):
        kw = dict(D=D, z=z, dt_bias=dt_bias, initial_states=initial_states, cu_seqlens=cu_seqlens,
                  chunk_size=chunk_size)
        try:
            y, fin, cs = ssd_forward(x, dt, A, B, C, keep_chunk_states=True, **kw)
        except _lib.SSDError as e:   # the SIMT path recomputes its states
            if e.code != 2:
                raise
            y, fin = ssd_forward(x, dt, A, B, C, **kw)
            cs = None
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens)
        ctx.chunk_states = cs
        ctx.chunk_size = chunk_size
        return y, fin

    @staticmethod
    def backward(ctx, dy, dfin):
        x, dt, A, B, C, D, z, dt_bias, init, cu = ctx.saved_tensors
        g = ssd_backward(x, dt, A, B, C, dy.contiguous(), D=D, z=z, dt_bias=dt_bias, initial_states=init,
                         dfinal_states=None if dfin is None else dfin.contiguous(), cu_seqlens=cu,
                         chunk_size=ctx.chunk_size, chunk_states=ctx.chunk_states)
        return (g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g.get("dD"), g.get("dz"), g.get("ddt_bias"),
                g.get("dinitial_states"), None, None)


@_on_stream
def complex_ssd_forward(x, A, B, C, dt, initial_states=None, chunk_size=64, return_imag=False,
                        return_final=False, stream=None):
    """Complex-A SSD scan (Mamba-3-Lite): h_t = exp(softplus(dt_t) A) h_{t-1} + x_t (outer) B_t,
    y_t = sum_n C_t[n] h_t[:, n].  x [batch, seqlen, nheads, headdim], B/C [batch, seqlen, nheads,
    dstate] and A [nheads] complex64; dt [batch, seqlen, nheads] float32; initial_states
    [batch, nheads, headdim, dstate] complex64.  Returns Re y (float32), then Im y and the final
    state when asked for."""
    Bt, T, H, Dh = x.shape
    N = B.shape[-1]
    dev = x.device
    for t in (x, B, C, A) + ((initial_states,) if initial_states is not None else ()):
        if t.dtype != torch.complex64 or not t.is_contiguous():
            raise ValueError("complex tensors must be contiguous complex64")
    if dt.dtype != torch.float32 or not dt.is_contiguous():
        raise ValueError("dt must be contiguous float32")
    prob = _lib.ComplexProblem(Bt, T, H, Dh, N, chunk_size)
    y_re = torch.empty(Bt, T, H, Dh, dtype=torch.float32, device=dev)
    y_im = torch.empty_like(y_re) if return_imag else None
    final = torch.empty(Bt, H, Dh, N, dtype=torch.complex64, device=dev) if return_final else None
    ws = torch.empty(_lib.complex_fwd_workspace_size(prob), dtype=torch.uint8, device=dev)
    _lib.check(_lib.complex_fwd(prob, x, dt, A, B, C, initial_states, y_re, y_im, final, ws, stream),
               "ssd_complex_fwd")
    out = (y_re,)
    if return_imag:
        out += (y_im,)
    if return_final:
        out += (final,)
    return out[0] if len(out) == 1 else out


# ---------------------------------------------------------------------------------------------
# The selective scan, the convolution with a carried window, single-token steps and 8-bit
# snapshots of states.  Checks, allocation and the call are the compiled binding's
# (csrc/binding.cpp): ValueError for tensors that do not fit together, SSDError for what the
# library refuses.  stream: launch there instead of on the current stream; the caller orders the two around the call.
# The outputs are then that stream's memory, and may be freed while the caller's current stream still reads them.
# Outputs carry no gradient (SelectiveScanFunction's do); what a call updates in place counts as changed for autograd.
def _handle(stream):
    return None if stream is None else stream.cuda_stream


def selective_scan_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_states=None, cu_seqlens=None,
                           return_final_states=True, state_dtype=None, keep_chunk_states=False, stream=None):
    """y, final_states = the selective scan: a decay rate per channel and state (see include/ssd.h,
    ssd_selective_fwd): h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t, y_t = (C_t . h_t + D x_t) silu(z_t) with
    dt = softplus(dt + dt_bias).

    x, z: [batch, seqlen, channels]; dt: the same in float32 or x's type; B, C: [batch, seqlen, ngroups,
    dstate]; A: [channels, dstate], D, dt_bias: [channels] float32; initial_states: [S, channels, dstate]
    float32 or bfloat16; cu_seqlens: int32 [S + 1] (batch 1).  state_dtype: of the final states (default:
    that of initial_states, else float32).  keep_chunk_states: also return the buffer that
    selective_scan_backward(chunk_states=...) starts from."""
    if state_dtype not in (None, torch.float32, torch.bfloat16):
        raise ValueError("state_dtype is float32 or bfloat16")
    sd = -1 if state_dtype is None else _lib.SSD_BF16 if state_dtype == torch.bfloat16 else _lib.SSD_F32
    return _lib.fast().selective_fwd(x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens, bool(return_final_states),
                                     sd, bool(keep_chunk_states), _handle(stream))


def selective_scan_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, initial_states=None, dfinal_states=None,
                            cu_seqlens=None, chunk_states=None, workspace=None, stream=None):
    """Gradients of sum(dy * y) + sum(dfinal_states * final_states): a dict with dx, ddt, dA, dB, dC and, when
    the matching input is given, dD, dz, ddt_bias, dinitial_states.  chunk_states: the buffer that
    selective_scan_forward(keep_chunk_states=True) returned for the same inputs (without it the
    forward's states are computed again)."""
    return _lib.fast().selective_bwd(x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens, dy, dfinal_states, chunk_states,
                                     workspace, _handle(stream))


class SelectiveScanFunction(torch.autograd.Function):
    """Autograd wrapper of the selective scan.  Where gradients are asked for, the forward keeps its chunk states for the backward
    (4 bytes a token, channel and dstate / 16, dstate padded as in ssd_selective_chunk_states_size; with keep_chunk_states=False the
    backward computes them again).  An output that nothing was computed from costs no gradient of zeros.  A second
    differentiation is refused."""

    @classmethod
    def apply(cls, x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_states=None, cu_seqlens=None, keep_chunk_states=True):
        inputs = (x, dt, A, B, C, D, z, dt_bias, initial_states)
        keep = keep_chunk_states and torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)
        return super().apply(*inputs, cu_seqlens, keep)

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens, keep):
        y, fin, *kept = selective_scan_forward(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, initial_states=initial_states,
                                               cu_seqlens=cu_seqlens, keep_chunk_states=keep)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, initial_states, cu_seqlens, kept[0] if keep else None)
        ctx.set_materialize_grads(False)
        return y, fin

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dfin):
        x, dt, A, B, C, D, z, dt_bias, init, cu, kept = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else dy
        g = selective_scan_backward(x, dt, A, B, C, dy.contiguous(), D=D, z=z, dt_bias=dt_bias, initial_states=init,
                                    dfinal_states=None if dfin is None else dfin.contiguous(), cu_seqlens=cu,
                                    chunk_states=kept)
        return (g["dx"], g["ddt"], g["dA"], g["dB"], g["dC"], g.get("dD"), g.get("dz"), g.get("ddt_bias"),
                g.get("dinitial_states"), None, None)


def ssd_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, state_indices=None, stream=None):
    """y = one token of ssd_forward's recurrence for each request (see include/ssd.h, ssd_step); `state`
    [nslots, nheads, headdim, dstate] float32 or bfloat16 is updated in place at state_indices (int32 [batch];
    default: slot i for request i).  x, z, y: [batch, nheads, headdim]; dt: [batch, nheads] float32; A, D,
    dt_bias: [nheads] float32; B, C: [batch, ngroups, dstate].  A request whose slot is out of range is
    padding: its y is zero.  The slots of one call must differ."""
    return _lib.fast().step(False, state, x, dt, A, B, C, D, z, dt_bias, state_indices, _handle(stream))


def selective_scan_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, state_indices=None, stream=None):
    """y = one token of selective_scan_forward's recurrence for each request; `state` [nslots, channels, dstate] is
    updated in place.  x, z, y: [batch, channels]; dt: the same in float32 or x's type; A: [channels, dstate],
    D, dt_bias: [channels] float32; B, C: [batch, ngroups, dstate].  Slots as in ssd_step."""
    return _lib.fast().step(True, state, x, dt, A, B, C, D, z, dt_bias, state_indices, _handle(stream))


def conv1d_prompt(xbc, weight, bias, conv_states, cu_seqlens=None, state_indices=None, has_initial=None, silu=True,
                  stream=None):
    """conv1d_forward whose sequences go on from carried windows (see include/ssd.h, ssd_conv1d_prompt): `conv_states`
    [nslots, width - 1, channels] of xbc's type holds the inputs before each sequence's first token and
    is left holding its last ones.  xbc: [batch, seqlen, channels]; state_indices: int32, one slot per
    sequence (default: slot i); has_initial: uint8 or bool per sequence, 0 where it starts from zeros."""
    return _lib.fast().conv1d_prompt(xbc, weight, bias, conv_states, cu_seqlens, state_indices, has_initial, bool(silu),
                                     _handle(stream))


def conv1d_step(xbc, weight, bias, conv_states, state_indices=None, silu=True, stream=None):
    """The convolution of one token per request: xbc [batch, channels]; conv_states and state_indices as in
    conv1d_prompt (a request whose slot is out of range sees a window of zeros and leaves none)."""
    return _lib.fast().conv1d_step(xbc, weight, bias, conv_states, state_indices, bool(silu), _handle(stream))


def snapshot_store(states, snapshots, scales, state_indices=None, slots=None, stream=None):
    """Puts states aside in 8 bits (see include/ssd.h, ssd_snapshot_store): state state_indices[i] of the pool `states`
    [nslots, ..., dstate] (float32 or bfloat16) goes to snapshots[slots[i]] (int8, the same inner shape)
    and scales[slots[i]] (float32, one per row of dstate values).  Indices are int32 and default to i."""
    _lib.fast().snapshot(True, states, snapshots, scales, state_indices, slots, _handle(stream))


def snapshot_load(snapshots, scales, states, slots=None, state_indices=None, stream=None):
    """Takes states up again: snapshot slots[i] is read back into state state_indices[i] of the pool `states`."""
    _lib.fast().snapshot(False, states, snapshots, scales, state_indices, slots, _handle(stream))


# ---------------------------------------------------------------------------------------------
# The gated delta rule (chunked, with every gradient, and one token at a time) and the norm of queries and keys with the
# rotation by position that precedes it, or an attention.  Streams, outputs and errors as above.
def _state_code(state_dtype):
    if state_dtype not in (None, torch.float32, torch.bfloat16):
        raise ValueError("state_dtype is float32 or bfloat16")
    return -1 if state_dtype is None else _lib.SSD_BF16 if state_dtype == torch.bfloat16 else _lib.SSD_F32


def gated_delta_forward(q, k, v, g, beta, scale=None, initial_states=None, cu_seqlens=None, return_final_states=True, state_dtype=None,
                        keep_chunk_states=False, stream=None):
    """o, final_states = the gated delta rule (see include/ssd.h, ssd_delta_fwd): per value head a state S [headdim, dstate],
    S <- exp(g_t) S, u = beta_t (v_t - S k_t), S <- S + u k_t^T, o_t = scale S q_t.

    q, k: [batch, seqlen, ngroups, dstate]; v, o: [batch, seqlen, nheads, headdim], q's type; head h reads group
    h // (nheads // ngroups); g (log decay, at most 0), beta: [batch, seqlen, nheads] float32 or v's type; scale: dstate ** -0.5
    by default; initial_states: [S, nheads, headdim, dstate] float32 or bfloat16; cu_seqlens: int32 [S + 1] (batch 1), tokens before the
    first sequence and behind the last are padding: never read, and zeros in the outputs and gradients (padding inside a row of a batch
    holds finite values: one that is not reaches every token of its chunk of 64).  Keys are expected
    at unit length (qk_norm_forward(mode="l2")).  state_dtype: of the final states (default: that of
    initial_states, else float32).  keep_chunk_states: also return the buffer that gated_delta_backward(chunk_states=...)
    starts from."""
    return _lib.fast().delta_fwd(q, k, v, g, beta, initial_states, cu_seqlens, scale, bool(return_final_states), _state_code(state_dtype),
                                 bool(keep_chunk_states), _handle(stream))


def gated_delta_backward(q, k, v, g, beta, do, scale=None, initial_states=None, dfinal_states=None, cu_seqlens=None, chunk_states=None,
                         workspace=None, stream=None):
    """Gradients of sum(do * o) + sum(dfinal_states * final_states): a dict with dq, dk, dv, dg, dbeta and, with initial_states,
    dinitial_states, each of its input's type.  chunk_states: the buffer that gated_delta_forward(keep_chunk_states=True)
    returned for the same inputs (without it the forward runs again)."""
    return _lib.fast().delta_bwd(q, k, v, g, beta, initial_states, cu_seqlens, scale, do, dfinal_states, chunk_states, workspace,
                                 _handle(stream))


class GatedDeltaFunction:
    """The gated delta rule in an autograd graph: o, final_states = GatedDeltaFunction.apply(...).  Where gradients are asked for, the
    forward keeps what the backward starts from (ssd_delta_chunk_states_size: on tensor cores 90 KB per 64 tokens and value head;
    with keep_chunk_states=False the backward computes it again).  Gradients go to q, k, v, g, beta and initial_states; an unused
    final state costs no gradient of zeros.  A second differentiation is refused, and so is a forward-mode one."""

    @staticmethod
    def apply(q, k, v, g, beta, initial_states=None, cu_seqlens=None, scale=None, keep_chunk_states=True):
        return _lib.fast().delta_apply(q, k, v, g, beta, initial_states, cu_seqlens, scale, bool(keep_chunk_states))


def gated_delta_step(state, q, k, v, g, beta, scale=None, state_indices=None, stream=None):
    """o = one token of gated_delta_forward's recurrence for each request; `state` [nslots, nheads, headdim, dstate] float32 or
    bfloat16 is updated in place at state_indices.  q, k: [batch, ngroups, dstate]; v, o: [batch, nheads, headdim]; g, beta:
    [batch, nheads] float32 or v's type.  Slots as in ssd_step."""
    return _lib.fast().delta_step(state, q, k, v, g, beta, scale, state_indices, _handle(stream))


_QK_MODES = {"rms": _lib.SSD_QK_RMS, "l2": _lib.SSD_QK_L2}


def _qk_mode(mode):
    if mode not in _QK_MODES:
        raise ValueError("mode is 'rms' or 'l2'")
    return _QK_MODES[mode]


def qk_norm_forward(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, mode="rms", interleaved=False, eps=1e-6,
                    stream=None):
    """q_out, k_out = queries and keys normalised per head (mode "rms": x / sqrt(mean x^2 + eps), "l2": x / sqrt(sum x^2 + eps)), times
    the weights, and rotated by their tokens' positions (see include/ssd.h, ssd_qk_norm_fwd) in one pass.

    q: [batch, seqlen, q_heads, dim], k: [batch, seqlen, k_heads, dim] of the same type, or None; weights: float32 [dim];
    cos, sin: float32 [rows, rotary / 2], without them nothing is rotated; positions: int32 [batch, seqlen] (default: a token's
    place in its row), a token with one outside the table is padding: its outputs are zero.  interleaved: features (2i, 2i + 1)
    are a pair, else (i, i + rotary / 2)."""
    return _lib.fast().qk_fwd(q, k, q_weight, k_weight, cos, sin, positions, _qk_mode(mode), bool(interleaved), eps, _handle(stream))


def qk_norm_backward(q, k, dq, dk, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, mode="rms", interleaved=False,
                     eps=1e-6, workspace=None, stream=None):
    """Gradients of sum(dq * q_out) + sum(dk * k_out): a dict with dq, dk (when k is given) and, with the weights, dq_weight, dk_weight
    (float32).  Nothing but the inputs is needed from the forward."""
    return _lib.fast().qk_bwd(q, k, q_weight, k_weight, cos, sin, positions, _qk_mode(mode), bool(interleaved), eps, dq, dk, workspace,
                              _handle(stream))


class QKNormFunction:
    """The norm and rotation of queries and keys in an autograd graph: q_out, k_out = QKNormFunction.apply(...).  It keeps its inputs
    alone; gradients go to q, k and the weights.  A second differentiation is refused, and so is a forward-mode one."""

    @staticmethod
    def apply(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, mode="rms", interleaved=False, eps=1e-6):
        return _lib.fast().qk_apply(q, k, q_weight, k_weight, cos, sin, positions, _qk_mode(mode), bool(interleaved), eps)
