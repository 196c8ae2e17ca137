"""Language-model operators of liblitela: head norms with rotation, the gated delta rule.

Like the rest of the binding this module only marshals arguments to the C ABI (include/litela.h
has the formulas, the layouts and the rules); outputs and workspaces come from torch, so every call
can be captured into a CUDA graph and two calls share nothing.  A call with `stream` runs on that
stream, which the caller has made wait for the inputs (and for which it keeps them), and takes its
buffers from that stream's memory.  Buffers that a caller gives to be written count as modified for
autograd.  To capture a training step, capture the _fwd_save and _bwd calls or torch.autograd.grad:
torch's .backward() may not accumulate, inside a capture, into leaves that a graph of eager calls still
holds.  The functions are reached through the
package:

    from linear_attention_diffusion_litela_b200 import lite_la_qk_norm_rope, lite_la_gated_delta
"""
from __future__ import annotations

import functools
import struct

from . import _check, lib
from . import _torch as _import_torch

_torch = functools.cache(_import_torch)

# The argument structs of include/litela.h, packed in one go: a ctypes.Structure filled field by field
# took longer than the kernel of a one-token call.  A view is (pointer, batch, token, head stride).
_VIEW = "Pqqq"
_DELTA_ARGS = struct.Struct("@" + 4 * _VIEW + "PPqqqqPPPiiiiifiPN")    # lite_la_delta_args
_DELTA_GRADS = struct.Struct("@" + 4 * _VIEW + "PPPP")                 # lite_la_delta_grads
_NO_VIEW = (0, 0, 0, 0)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


@functools.cache
def _current_stream():
    """device -> handle of torch's current stream there (without making a Stream object: 1.2 us of a call
    of 15, where this torch can)"""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(fn, dev, stream, *args):
    """fn(*args, stream) on device `dev`; stream None: torch's current one there."""
    cuda = _torch().cuda
    handle = _current_stream()(dev) if stream is None else stream.cuda_stream
    if cuda.current_device() == dev:
        _check(fn(*args, handle))
    else:
        with cuda.device(dev):
            _check(fn(*args, handle))


def _on(stream, make, *args, returned=True, **kw):
    """make(*args, **kw): a buffer of a call with `stream`, from that stream's memory.  A block of the
    current stream's may have been freed under work that is still queued there, which a caller's wait
    before the call need not cover.  The current stream may go on to use what is returned."""
    cuda = _torch().cuda
    with cuda.stream(stream):
        t = make(*args, **kw)
    if returned:
        t.record_stream(cuda.current_stream(t.device))
    return t


@functools.cache
def _wrote():
    """f(t): the caller's buffer t has been written; a backward that needs what was in it must not take this"""
    return _torch().autograd.graph.increment_version


# ---------------------------------------------------------------------------------------
# head norms with rotation


def _rows(t, name, shape, dev):
    if t.dtype is not _torch().bfloat16 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise TypeError("%s must be a contiguous bf16 tensor of qkv's shape on qkv's device" % name)
    return t.data_ptr()


def _norm_args(qkv, Hq, Hk, d, q_weight, k_weight, cos, sin, positions, eps, interleaved):
    """Checks; returns (device, (cos, sin, positions, .. eps) as the C calls take them)."""
    torch = _torch()
    if not isinstance(qkv, torch.Tensor) or not qkv.is_cuda or qkv.dtype is not torch.bfloat16 or qkv.dim() != 3 \
            or not qkv.is_contiguous():
        raise TypeError("qkv must be a contiguous bf16 CUDA tensor [B, N, (Hq + Hk + Hv)*d]")
    B, N, W = qkv.shape
    dev = qkv.get_device()
    if d <= 0 or W % d != 0 or W // d < Hq + Hk or Hq < 0 or Hk < 0:
        raise ValueError("qkv last dim %d is not (Hq + Hk + Hv)*d with Hq = %d, Hk = %d, d = %d" % (W, Hq, Hk, d))
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not torch.float32 or w.shape != (d,) or not w.is_contiguous()
                              or w.get_device() != dev):
            raise TypeError("q_weight and k_weight must be contiguous fp32 tensors [d] on qkv's device")
    if (cos is None) != (sin is None):
        raise TypeError("cos and sin come together")
    rot = table = pos_bytes = 0
    if cos is not None:
        shape = cos.shape
        for t in (cos, sin):
            if t.dtype is not torch.float32 or len(shape) != 2 or t.shape != shape or not t.is_contiguous() \
                    or t.get_device() != dev:
                raise TypeError("cos and sin must be contiguous fp32 tensors [positions, rot/2] on qkv's device")
        table, rot = shape[0], 2 * shape[1]
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or positions.shape != (B, N) \
                or not positions.is_contiguous() or positions.get_device() != dev:
            raise TypeError("positions must be a contiguous int32 or int64 tensor [B, N] on qkv's device")
        pos_bytes = positions.element_size()
    return dev, (_ptr(cos), _ptr(sin), _ptr(positions), pos_bytes, B, N, Hq, Hk, W // d - Hq - Hk, d, rot, table,
                 int(interleaved), eps)


def lite_la_qk_norm_rope_fwd(qkv, Hq: int, Hk: int, d: int = 32, q_weight=None, k_weight=None, cos=None, sin=None,
                             positions=None, eps: float = 1e-6, interleaved: bool = False, out=None, stream=None):
    """RMS norm of every q and k head of packed rows (bf16 [B, N, (Hq + Hk + Hv)*d]) and rotation
    by position; returns out in qkv's layout (v copied).  out=qkv works in place.  A row at a
    negative position is padding: left alone in place, zeros otherwise."""
    dev, args = _norm_args(qkv, Hq, Hk, d, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    given = out is not None
    if not given:
        like = _torch().empty_like
        out = like(qkv) if stream is None else _on(stream, like, qkv)
    o = _rows(out, "out", qkv.shape, dev)
    _call(lib().lite_la_qk_norm_rope_fwd, dev, stream, qkv.data_ptr(), o, _ptr(q_weight), _ptr(k_weight), *args)
    if given:
        _wrote()(out)
    return out


def lite_la_qk_norm_rope_bwd(qkv, dout, Hq: int, Hk: int, d: int = 32, q_weight=None, k_weight=None, cos=None,
                             sin=None, positions=None, eps: float = 1e-6, interleaved: bool = False, dqkv=None,
                             stream=None):
    """Gradient of sum(dout * out): returns (dqkv bf16, dq_weight, dk_weight fp32; None for a
    weight that is None).  dqkv=dout works in place."""
    return _norm_bwd(qkv, dout, Hq, Hk, d, q_weight, k_weight, cos, sin, positions, eps, interleaved, dqkv, stream,
                     q_weight is not None, k_weight is not None)


def _norm_bwd(qkv, dout, Hq, Hk, d, q_weight, k_weight, cos, sin, positions, eps, interleaved, dqkv, stream, want_q, want_k):
    """... with the weights' gradients that are wanted"""
    torch = _torch()
    dev, args = _norm_args(qkv, Hq, Hk, d, q_weight, k_weight, cos, sin, positions, eps, interleaved)
    like, given = torch.empty_like, dqkv is not None
    if not given:
        dqkv = like(qkv) if stream is None else _on(stream, like, qkv)
    do, dx = _rows(dout, "dout", qkv.shape, dev), _rows(dqkv, "dqkv", qkv.shape, dev)
    dwq, dwk = (None if not want else like(w) if stream is None else _on(stream, like, w)
                for want, w in ((want_q, q_weight), (want_k, k_weight)))
    size, ws = 0, None
    if want_q or want_k:
        size = lib().lite_la_qk_norm_rope_workspace_bytes(d)
        kw = dict(dtype=torch.uint8, device=qkv.device)
        ws = torch.empty(size, **kw) if stream is None else _on(stream, torch.empty, size, returned=False, **kw)
    _call(lib().lite_la_qk_norm_rope_bwd, dev, stream, qkv.data_ptr(), do, dx, _ptr(q_weight), _ptr(k_weight),
          _ptr(dwq), _ptr(dwk), *args, _ptr(ws), size)
    if given:
        _wrote()(dqkv)
    return dqkv, dwq, dwk


_FUNCTIONS = {}


def _dense(t):
    """A gradient as autograd hands it, contiguous and aligned as the calls want it."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _norm_function():
    if "norm" not in _FUNCTIONS:
        torch = _torch()

        from torch.autograd.function import once_differentiable

        class QKNormRope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, qkv, q_weight, k_weight, cos, sin, positions, kw):
                ctx.save_for_backward(qkv, q_weight, k_weight, cos, sin, positions)
                ctx.kw = kw
                return lite_la_qk_norm_rope_fwd(qkv, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin,
                                                positions=positions, **kw)

            @staticmethod
            @once_differentiable
            def backward(ctx, grad):
                qkv, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
                grad = _dense(grad.to(torch.bfloat16))
                _, want_q, want_k = ctx.needs_input_grad[:3]     # (frozen weights cost nothing)
                dqkv, dwq, dwk = _norm_bwd(qkv, grad, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin,
                                           positions=positions, dqkv=None, stream=None, want_q=want_q, want_k=want_k,
                                           **ctx.kw)
                return dqkv, dwq, dwk, None, None, None, None

        _FUNCTIONS["norm"] = QKNormRope
    return _FUNCTIONS["norm"]


def lite_la_qk_norm_rope(qkv, Hq: int, Hk: int, d: int = 32, q_weight=None, k_weight=None, cos=None, sin=None,
                         positions=None, eps: float = 1e-6, interleaved: bool = False):
    """lite_la_qk_norm_rope_fwd that torch autograd can differentiate (qkv and the weights)."""
    return _norm_function().apply(qkv, q_weight, k_weight, cos, sin, positions,
                                  dict(Hq=Hq, Hk=Hk, d=d, eps=eps, interleaved=interleaved))


# ---------------------------------------------------------------------------------------
# the gated delta rule


def _view(t, name, shape, dev):
    """A bf16 tensor [B, N, heads, d] with adjacent channels as (pointer, strides)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev:
        raise TypeError("%s must be a bf16 CUDA tensor %s on q's device" % (name, list(shape)))
    sb, st, sh, sc = t.stride()
    if sc != 1 and t.numel() > 0:
        raise TypeError("%s: the channels of a head must be adjacent" % name)
    B, N, H, _ = shape   # a dimension of one has no stride
    return t.data_ptr(), 0 if B == 1 else sb, 0 if N == 1 else st, 0 if H == 1 else sh


def _token_view(t, name, shape, dev):
    """... [B, heads, d]: one token"""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != dev:
        raise TypeError("%s must be a bf16 CUDA tensor %s on q's device" % (name, list(shape)))
    sb, sh, sc = t.stride()
    if sc != 1 and t.numel() > 0:
        raise TypeError("%s: the channels of a head must be adjacent" % name)
    return t.data_ptr(), 0 if shape[0] == 1 else sb, 0, 0 if shape[1] == 1 else sh


def _gate(t, name, shape, dev):
    """An fp32 tensor [B, (N,) Hv] as (pointer, batch, token stride)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != shape or t.get_device() != dev \
            or (t.stride(-1) != 1 and shape[-1] > 1 and t.numel() > 0):
        raise TypeError("%s must be an fp32 tensor %s on q's device with adjacent heads" % (name, list(shape)))
    return t.data_ptr(), 0 if shape[0] == 1 else t.stride(0), 0 if len(shape) == 2 or shape[1] == 1 else t.stride(1)


def _states(t, name, shape, dev):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != shape or t.get_device() != dev \
            or not t.is_contiguous():
        raise TypeError("%s must be a contiguous fp32 tensor %s on q's device" % (name, list(shape)))
    return t.data_ptr()


class _Delta:
    """The checked arguments of a call over whole sequences."""

    def __init__(self, q, k, v, g, beta, scale, cu_seqlens):
        torch = _torch()
        if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 4:
            raise TypeError("q must be a bf16 CUDA tensor [B, N, Hk, d]")
        if not isinstance(v, torch.Tensor) or v.dim() != 4:
            raise TypeError("v must be a bf16 CUDA tensor [B, N, Hv, d]")
        B, N, Hk, d = q.shape
        Hv, dev = v.shape[2], q.get_device()
        self.device, self.dev, self.qshape, self.vshape = q.device, dev, (B, N, Hk, d), (B, N, Hv, d)
        self.views = (*_view(q, "q", self.qshape, dev), *_view(k, "k", self.qshape, dev),
                      *_view(v, "v", self.vshape, dev))
        gp, g_sb, g_st = _gate(g, "g", (B, N, Hv), dev)
        bp, b_sb, b_st = _gate(beta, "beta", (B, N, Hv), dev)
        self.gates = (gp, bp, g_sb, g_st, b_sb, b_st)
        self.scale = float(d) ** -0.5 if scale is None and d > 0 else float(scale or 0.0)
        self.cu, self.S = 0, B
        if cu_seqlens is not None:
            if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype is not torch.int32 \
                    or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or cu_seqlens.get_device() != dev \
                    or cu_seqlens.numel() < 1:
                raise TypeError("cu_seqlens must be a contiguous int32 tensor [sequences + 1] on q's device")
            if B != 1:
                raise ValueError("packed sequences come in one buffer: B must be 1, not %d" % B)
            self.cu, self.S = cu_seqlens.data_ptr(), cu_seqlens.numel() - 1
        self.sizes = (self.S, N, Hk, Hv, d)
        self.states = (self.S, Hv, d, d)

    def bytes(self, fn):
        return fn(*self.sizes, int(self.cu != 0))

    def pack(self, out, state_in, state_out, zero_tail, ws, ws_bytes):
        return _DELTA_ARGS.pack(*self.views, *out, *self.gates, state_in, state_out, self.cu, *self.sizes, self.scale,
                                zero_tail, ws, ws_bytes)


def _delta_forward(q, k, v, g, beta, state_in, state_out, cu_seqlens, scale, out, stream, save):
    torch = _torch()
    a = _Delta(q, k, v, g, beta, scale, cu_seqlens)
    si = 0 if state_in is None else _states(state_in, "state_in", a.states, a.dev)
    given = [x for x in (state_out, out) if x is not None]
    if state_out is None:
        kw = dict(dtype=torch.float32, device=a.device)
        if stream is not None:
            state_out = _on(stream, torch.empty, a.states, **kw)
        else:
            state_out = torch.empty_like(state_in) if si else torch.empty(a.states, **kw)
    so = _states(state_out, "state_out", a.states, a.dev)
    zero_tail = int(out is None)
    if out is None:
        kw = dict(memory_format=torch.contiguous_format)
        out = torch.empty_like(v, **kw) if stream is None else _on(stream, torch.empty_like, v, **kw)
    o = _view(out, "out", a.vshape, a.dev)
    L = lib()
    size = a.bytes(L.lite_la_gated_delta_saved_bytes if save else L.lite_la_gated_delta_workspace_bytes)
    buf = None
    if size or save:
        kw = dict(dtype=torch.uint8, device=a.device)
        buf = torch.empty(size, **kw) if stream is None else _on(stream, torch.empty, size, returned=save, **kw)
    if save:
        _call(L.lite_la_gated_delta_fwd_save, a.dev, stream, a.pack(o, si, so, zero_tail, 0, 0), buf.data_ptr(), size)
    else:
        _call(L.lite_la_gated_delta_fwd, a.dev, stream, a.pack(o, si, so, zero_tail, _ptr(buf), size))
    for x in given:
        _wrote()(x)
    return out, state_out, buf


def lite_la_gated_delta_fwd(q, k, v, g, beta, state_in=None, state_out=None, cu_seqlens=None, scale=None, out=None,
                            stream=None):
    """The gated delta rule over whole sequences.  q, k: bf16 [B, N, Hk, d], v: bf16 [B, N, Hv, d]
    (any strides with adjacent channels, so views of packed rows do); g (log decay), beta: fp32
    [B, N, Hv].  state_in: fp32 [sequences, Hv, d, d] or None (zeros); state_out is allocated when
    None and may be state_in.  cu_seqlens (int32 [sequences + 1], on the device) packs sequences
    of different lengths into one buffer (B = 1).  scale defaults to d ** -0.5.  Returns (out bf16
    [B, N, Hv, d], state_out); rows behind the last packed sequence are left as they are in `out`
    (zeros when it is allocated here)."""
    return _delta_forward(q, k, v, g, beta, state_in, state_out, cu_seqlens, scale, out, stream, False)[:2]


def lite_la_gated_delta_fwd_save(q, k, v, g, beta, state_in=None, state_out=None, cu_seqlens=None, scale=None,
                                 out=None, stream=None):
    """lite_la_gated_delta_fwd that also returns what lite_la_gated_delta_bwd needs: (out, state_out,
    saved)."""
    return _delta_forward(q, k, v, g, beta, state_in, state_out, cu_seqlens, scale, out, stream, True)


def lite_la_gated_delta_bwd(q, k, v, g, beta, dout, saved, dstate_out=None, state_in=None, cu_seqlens=None,
                            scale=None, stream=None):
    """Gradients of sum(dout * out) + sum(dstate_out * state_out) for the forward that left `saved`
    (lite_la_gated_delta_fwd_save with the same arguments): (dq, dk, dv bf16, dg, dbeta fp32,
    dstate_in fp32 or None without state_in)."""
    torch = _torch()
    a = _Delta(q, k, v, g, beta, scale, cu_seqlens)
    do = _view(dout, "dout", a.vshape, a.dev)
    if not isinstance(saved, torch.Tensor) or saved.dtype is not torch.uint8 or not saved.is_contiguous() \
            or saved.get_device() != a.dev:
        raise TypeError("saved must be what lite_la_gated_delta_fwd_save returned")
    def new(shape, dtype, returned=True):
        kw = dict(dtype=dtype, device=a.device)
        return torch.empty(shape, **kw) if stream is None else _on(stream, torch.empty, shape, returned=returned, **kw)

    si = dstate_in = None
    if state_in is not None:
        si, dstate_in = _states(state_in, "state_in", a.states, a.dev), new(a.states, torch.float32)
    dso = 0 if dstate_out is None else _states(dstate_out, "dstate_out", a.states, a.dev)
    dq, dk, dv = (new(shape, torch.bfloat16) for shape in (a.qshape, a.qshape, a.vshape))
    dg, dbeta = (new(a.vshape[:3], torch.float32) for _ in range(2))
    size = a.bytes(lib().lite_la_gated_delta_bwd_workspace_bytes)
    ws = new(size, torch.uint8, False)
    grads = _DELTA_GRADS.pack(*do, *_view(dq, "dq", a.qshape, a.dev), *_view(dk, "dk", a.qshape, a.dev),
                              *_view(dv, "dv", a.vshape, a.dev), dg.data_ptr(), dbeta.data_ptr(), dso,
                              _ptr(dstate_in))
    _call(lib().lite_la_gated_delta_bwd, a.dev, stream, a.pack(_NO_VIEW, si or 0, 0, 0, ws.data_ptr(), size), grads,
          saved.data_ptr(), saved.numel())
    return dq, dk, dv, dg, dbeta, dstate_in


def _delta_function():
    if "delta" not in _FUNCTIONS:
        torch = _torch()
        from torch.autograd.function import once_differentiable

        class GatedDelta(torch.autograd.Function):
            @staticmethod
            def forward(ctx, q, k, v, g, beta, state_in, cu_seqlens, scale):
                ctx.set_materialize_grads(False)
                out, state_out, saved = lite_la_gated_delta_fwd_save(q, k, v, g, beta, state_in=state_in,
                                                                     cu_seqlens=cu_seqlens, scale=scale)
                ctx.save_for_backward(q, k, v, g, beta, state_in, cu_seqlens, saved)
                ctx.scale = scale
                return out, state_out

            @staticmethod
            @once_differentiable
            def backward(ctx, dout, dstate):
                q, k, v, g, beta, state_in, cu_seqlens, saved = ctx.saved_tensors
                if dout is None:
                    dout = torch.zeros_like(v, memory_format=torch.contiguous_format)
                dout = dout.to(torch.bfloat16)
                if dout.stride(-1) != 1 or dout.data_ptr() % 16 != 0 or any(x % 8 for x in dout.stride()[:3]):
                    dout = _dense(dout)
                if dstate is not None:
                    dstate = _dense(dstate.float())
                grads = lite_la_gated_delta_bwd(q, k, v, g, beta, dout, saved, dstate_out=dstate, state_in=state_in,
                                                cu_seqlens=cu_seqlens, scale=ctx.scale)
                return (*grads, None, None)

        _FUNCTIONS["delta"] = GatedDelta
    return _FUNCTIONS["delta"]


def lite_la_gated_delta(q, k, v, g, beta, state_in=None, cu_seqlens=None, scale=None):
    """lite_la_gated_delta_fwd that torch autograd can differentiate: returns (out, state_out) with
    gradients for q, k, v, g, beta and state_in.  The forward keeps its states (one per 64 tokens) for
    the backward; where no gradient is wanted it does not."""
    torch = _torch()
    given = [t for t in (q, k, v, g, beta, state_in) if isinstance(t, torch.Tensor)]
    # (a tangent of forward-mode differentiation goes to the function, which refuses it)
    if not (torch.is_grad_enabled() and any(t.requires_grad for t in given)) \
            and all(torch.autograd.forward_ad.unpack_dual(t).tangent is None for t in given):
        return lite_la_gated_delta_fwd(q, k, v, g, beta, state_in=state_in, cu_seqlens=cu_seqlens, scale=scale)
    return _delta_function().apply(q, k, v, g, beta, state_in, cu_seqlens, scale)


def lite_la_gated_delta_step(q, k, v, g, beta, states, state_indices=None, scale=None, out=None, stream=None):
    """One token of each of B sequences: q, k bf16 [B, Hk, d], v bf16 [B, Hv, d], g, beta fp32
    [B, Hv]; states fp32 [pool, Hv, d, d] is updated in place, row b's state being
    states[state_indices[b]] (int32 [B] on the device; None: states[b]).  A row with an index
    outside the pool, or with one that an earlier row has, touches no state and gets zeros.
    Returns out bf16 [B, Hv, d]."""
    torch = _torch()
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3 or not isinstance(v, torch.Tensor) \
            or v.dim() != 3 or not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise TypeError("q, k must be [B, Hk, d], v [B, Hv, d] and states [pool, Hv, d, d] CUDA tensors")
    B, Hk, d = q.shape
    Hv, pool, dev = v.shape[1], states.shape[0], q.get_device()
    shape = (B, Hv, d)
    gp, g_sb, _ = _gate(g, "g", (B, Hv), dev)
    bp, b_sb, _ = _gate(beta, "beta", (B, Hv), dev)
    st = _states(states, "states", (pool, Hv, d, d), dev)
    if state_indices is not None and (state_indices.dtype is not torch.int32 or state_indices.shape != (B,)
                                      or not state_indices.is_contiguous() or state_indices.get_device() != dev):
        raise TypeError("state_indices must be a contiguous int32 tensor [B] on q's device")
    given = out is not None
    if not given:
        kw = dict(memory_format=torch.contiguous_format)
        out = torch.empty_like(v, **kw) if stream is None else _on(stream, torch.empty_like, v, **kw)
    args = _DELTA_ARGS.pack(*_token_view(q, "q", (B, Hk, d), dev), *_token_view(k, "k", (B, Hk, d), dev),
                            *_token_view(v, "v", shape, dev), *_token_view(out, "out", shape, dev), gp, bp, g_sb, 0,
                            b_sb, 0, st, st, 0, B, 1, Hk, Hv, d,
                            float(d) ** -0.5 if scale is None and d > 0 else float(scale or 0.0), 0, 0, 0)
    _call(lib().lite_la_gated_delta_step, dev, stream, args, _ptr(state_indices), pool)
    _wrote()(states)
    if given:
        _wrote()(out)
    return out
