"""Language-model operators of liblitela: head norms with rotation, the gated delta rule.

Like the rest of the binding this module only marshals arguments to the C ABI (include/litela.h
has the formulas, the layouts and the rules); outputs and workspaces come from torch, so every call
can be captured into a CUDA graph and two calls share nothing.  The functions are reached through
the package:

    from linear_attention_diffusion_litela_b200 import lite_la_qk_norm_rope, lite_la_gated_delta
"""
from __future__ import annotations

import ctypes

from . import _check, _stream_handle, _torch, lib

_vp, _c_int, _c_float, _c_size, _c_ll = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                                         ctypes.c_longlong)


class View(ctypes.Structure):
    """lite_la_view"""
    _fields_ = [("data", _vp), ("batch_stride", _c_ll), ("token_stride", _c_ll), ("head_stride", _c_ll)]


class DeltaArgs(ctypes.Structure):
    """lite_la_delta_args"""
    _fields_ = [("q", View), ("k", View), ("v", View), ("out", View), ("g", _vp), ("beta", _vp),
                ("g_batch_stride", _c_ll), ("g_token_stride", _c_ll), ("beta_batch_stride", _c_ll),
                ("beta_token_stride", _c_ll), ("state_in", _vp), ("state_out", _vp), ("cu_seqlens", _vp),
                ("B", _c_int), ("N", _c_int), ("Hk", _c_int), ("Hv", _c_int), ("d", _c_int), ("scale", _c_float),
                ("zero_tail", _c_int), ("workspace", _vp), ("workspace_bytes", _c_size)]


class DeltaGrads(ctypes.Structure):
    """lite_la_delta_grads"""
    _fields_ = [("dout", View), ("dq", View), ("dk", View), ("dv", View), ("dg", _vp), ("dbeta", _vp),
                ("dstate_out", _vp), ("state_out", _vp), ("dstate_in", _vp)]


def _ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------------------------------
# head norms with rotation


def _norm_args(qkv, Hq, Hk, d, q_weight, k_weight, cos, sin, positions):
    """Checks; returns (B, N, Hv, rot, table_len, position_bytes)."""
    torch = _torch()
    if not isinstance(qkv, torch.Tensor) or not qkv.is_cuda or qkv.dtype != torch.bfloat16 or qkv.dim() != 3 \
            or not qkv.is_contiguous():
        raise TypeError("qkv must be a contiguous bf16 CUDA tensor [B, N, (Hq + Hk + Hv)*d]")
    B, N, W = qkv.shape
    if d <= 0 or W % d != 0 or W // d < Hq + Hk or Hq < 0 or Hk < 0:
        raise ValueError("qkv last dim %d is not (Hq + Hk + Hv)*d with Hq = %d, Hk = %d, d = %d" % (W, Hq, Hk, d))
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (d,) or not w.is_contiguous()
                              or w.device != qkv.device):
            raise TypeError("%s must be a contiguous fp32 tensor [d] on qkv's device" % name)
    if (cos is None) != (sin is None):
        raise TypeError("cos and sin come together")
    rot = table = 0
    if cos is not None:
        for t in (cos, sin):
            if t.dtype != torch.float32 or t.dim() != 2 or not t.is_contiguous() or t.device != qkv.device \
                    or t.shape != cos.shape:
                raise TypeError("cos and sin must be contiguous fp32 tensors [positions, rot/2] on qkv's device")
        table, rot = int(cos.shape[0]), 2 * int(cos.shape[1])
    bytes_ = 0
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or tuple(positions.shape) != (B, N) \
                or not positions.is_contiguous() or positions.device != qkv.device:
            raise TypeError("positions must be a contiguous int32 or int64 tensor [B, N] on qkv's device")
        bytes_ = positions.element_size()
    return B, N, W // d - Hq - Hk, rot, table, bytes_


def lite_la_qk_norm_rope_fwd(qkv, Hq: int, Hk: int, d: int = 32, q_weight=None, k_weight=None, cos=None, sin=None,
                             positions=None, eps: float = 1e-6, interleaved: bool = False, out=None, stream=None):
    """RMS norm of every q and k head of packed rows (bf16 [B, N, (Hq + Hk + Hv)*d]) and rotation
    by position; returns out in qkv's layout (v copied).  out=qkv works in place.  A row at a
    negative position is padding: left alone in place, zeros otherwise."""
    torch = _torch()
    B, N, Hv, rot, table, pb = _norm_args(qkv, Hq, Hk, d, q_weight, k_weight, cos, sin, positions)
    if out is None:
        out = torch.empty_like(qkv)
    elif out.dtype != torch.bfloat16 or out.shape != qkv.shape or not out.is_contiguous() or out.device != qkv.device:
        raise TypeError("out must be a contiguous bf16 tensor of qkv's shape on qkv's device")
    with torch.cuda.device(qkv.device):
        _check(lib().lite_la_qk_norm_rope_fwd(
            qkv.data_ptr(), out.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(positions), pb,
            B, N, Hq, Hk, Hv, d, rot, table, int(interleaved), eps, _stream_handle(stream, qkv.device)))
    return out


def lite_la_qk_norm_rope_bwd(qkv, dout, Hq: int, Hk: int, d: int = 32, q_weight=None, k_weight=None, cos=None,
                             sin=None, positions=None, eps: float = 1e-6, interleaved: bool = False, dqkv=None,
                             stream=None):
    """Gradient of sum(dout * out): returns (dqkv bf16, dq_weight, dk_weight fp32; None for a
    weight that is None).  dqkv=dout works in place."""
    torch = _torch()
    B, N, Hv, rot, table, pb = _norm_args(qkv, Hq, Hk, d, q_weight, k_weight, cos, sin, positions)
    for t, name in ((dout, "dout"), (dqkv, "dqkv")):
        if t is not None and (t.dtype != torch.bfloat16 or t.shape != qkv.shape or not t.is_contiguous()
                              or t.device != qkv.device):
            raise TypeError("%s must be a contiguous bf16 tensor of qkv's shape on qkv's device" % name)
    if dqkv is None:
        dqkv = torch.empty_like(qkv)
    dwq = None if q_weight is None else torch.empty_like(q_weight)
    dwk = None if k_weight is None else torch.empty_like(k_weight)
    ws = None
    if dwq is not None or dwk is not None:
        ws = torch.empty(int(lib().lite_la_qk_norm_rope_workspace_bytes(d)), dtype=torch.uint8, device=qkv.device)
        _on_stream(ws, stream)
    with torch.cuda.device(qkv.device):
        _check(lib().lite_la_qk_norm_rope_bwd(
            qkv.data_ptr(), dout.data_ptr(), dqkv.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(dwq), _ptr(dwk),
            _ptr(cos), _ptr(sin), _ptr(positions), pb, B, N, Hq, Hk, Hv, d, rot, table, int(interleaved), eps,
            _ptr(ws), 0 if ws is None else ws.numel(), _stream_handle(stream, qkv.device)))
    return dqkv, dwq, dwk


def _on_stream(t, stream):
    """A workspace that torch made on the current stream is used on `stream`: torch must not hand
    its memory on before that stream is done with it."""
    if stream is not None:
        t.record_stream(stream)


_FUNCTIONS = {}


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
                if grad.dtype != torch.bfloat16 or not grad.is_contiguous():
                    grad = grad.to(torch.bfloat16).contiguous()
                dqkv, dwq, dwk = lite_la_qk_norm_rope_bwd(qkv, grad, q_weight=q_weight, k_weight=k_weight, cos=cos,
                                                          sin=sin, positions=positions, **ctx.kw)
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


def _view(t, name, shape, device):
    """lite_la_view of a bf16 [B, N, heads, d] tensor with adjacent channels."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16 or tuple(t.shape) != shape \
            or t.device != device:
        raise TypeError("%s must be a bf16 CUDA tensor %s on q's device" % (name, list(shape)))
    if t.stride(-1) != 1 and t.numel() > 0:
        raise TypeError("%s: the channels of a head must be adjacent" % name)
    # a dimension of one has no stride
    return View(t.data_ptr(), *(0 if n == 1 else s for n, s in zip(t.shape[:3], t.stride()[:3])))


def _gate(t, name, shape, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape or t.device != device \
            or (t.stride(-1) != 1 and shape[-1] > 1 and t.numel() > 0):
        raise TypeError("%s must be an fp32 tensor %s on q's device with adjacent heads" % (name, list(shape)))
    return t.data_ptr(), 0 if shape[0] == 1 else t.stride(0), 0 if shape[1] == 1 else t.stride(1)


def _states(t, name, shape, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or tuple(t.shape) != shape \
            or not t.is_contiguous() or t.device != device:
        raise TypeError("%s must be a contiguous fp32 tensor %s on q's device" % (name, list(shape)))
    return t.data_ptr()


def _delta_args(q, k, v, g, beta, scale, cu_seqlens):
    """The fields that every call has; returns (args, sequences)."""
    torch = _torch()
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 4:
        raise TypeError("q must be a bf16 CUDA tensor [B, N, Hk, d]")
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise TypeError("v must be a bf16 CUDA tensor [B, N, Hv, d]")
    B, N, Hk, d = q.shape
    Hv, device = int(v.shape[2]), q.device
    a = DeltaArgs()
    a.q, a.k = _view(q, "q", (B, N, Hk, d), device), _view(k, "k", (B, N, Hk, d), device)
    a.v = _view(v, "v", (B, N, Hv, d), device)
    a.g, a.g_batch_stride, a.g_token_stride = _gate(g, "g", (B, N, Hv), device)
    a.beta, a.beta_batch_stride, a.beta_token_stride = _gate(beta, "beta", (B, N, Hv), device)
    a.scale = float(d) ** -0.5 if scale is None and d > 0 else float(scale or 0.0)
    a.B, a.N, a.Hk, a.Hv, a.d = B, N, Hk, Hv, d
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 \
                or not cu_seqlens.is_contiguous() or cu_seqlens.device != device or cu_seqlens.numel() < 1:
            raise TypeError("cu_seqlens must be a contiguous int32 tensor [sequences + 1] on q's device")
        if B != 1:
            raise ValueError("packed sequences come in one buffer: B must be 1, not %d" % B)
        a.cu_seqlens, a.B = cu_seqlens.data_ptr(), cu_seqlens.numel() - 1
    return a, int(a.B)


def _delta_forward(q, k, v, g, beta, state_in, state_out, cu_seqlens, scale, out, stream, save):
    torch = _torch()
    a, S = _delta_args(q, k, v, g, beta, scale, cu_seqlens)
    d, Hv, device = int(a.d), int(a.Hv), q.device
    if state_in is not None:
        a.state_in = _states(state_in, "state_in", (S, Hv, d, d), device)
    if state_out is None:
        state_out = torch.empty((S, Hv, d, d), dtype=torch.float32, device=device)
    a.state_out = _states(state_out, "state_out", (S, Hv, d, d), device)
    if out is None:
        out = torch.empty(v.shape, dtype=torch.bfloat16, device=device)
        a.zero_tail = 1
    a.out = _view(out, "out", tuple(v.shape), device)
    size = lib().lite_la_gated_delta_saved_bytes if save else lib().lite_la_gated_delta_workspace_bytes
    buf = torch.empty(int(size(a.B, a.N, a.Hk, Hv, d, int(cu_seqlens is not None))), dtype=torch.uint8, device=device)
    _on_stream(buf, stream)
    with torch.cuda.device(device):
        if save:
            _check(lib().lite_la_gated_delta_fwd_save(ctypes.byref(a), buf.data_ptr(), buf.numel(),
                                                      _stream_handle(stream, device)))
        else:
            a.workspace, a.workspace_bytes = buf.data_ptr(), buf.numel()
            _check(lib().lite_la_gated_delta_fwd(ctypes.byref(a), _stream_handle(stream, device)))
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


def lite_la_gated_delta_bwd(q, k, v, g, beta, dout, saved, state_out=None, dstate_out=None, state_in=None,
                            cu_seqlens=None, scale=None, stream=None):
    """Gradients of sum(dout * out) + sum(dstate_out * state_out) for the forward that left `saved`
    (lite_la_gated_delta_fwd_save with the same arguments) and wrote state_out: (dq, dk, dv bf16, dg,
    dbeta fp32, dstate_in fp32 or None without state_in)."""
    torch = _torch()
    a, S = _delta_args(q, k, v, g, beta, scale, cu_seqlens)
    d, Hv, device = int(a.d), int(a.Hv), q.device
    gr = DeltaGrads()
    gr.dout = _view(dout, "dout", tuple(v.shape), device)
    if not isinstance(saved, torch.Tensor) or saved.dtype != torch.uint8 or not saved.is_contiguous() \
            or saved.device != device:
        raise TypeError("saved must be what lite_la_gated_delta_fwd_save returned")
    shape = (S, Hv, d, d)
    dstate_in = None
    if state_in is not None:
        a.state_in = _states(state_in, "state_in", shape, device)
        dstate_in = torch.empty(shape, dtype=torch.float32, device=device)
        gr.dstate_in = dstate_in.data_ptr()
    if dstate_out is not None:
        gr.dstate_out = _states(dstate_out, "dstate_out", shape, device)
        gr.state_out = _states(state_out, "state_out", shape, device)
    dq, dk, dv = (torch.empty(t.shape, dtype=torch.bfloat16, device=device) for t in (q, k, v))
    dg, dbeta = (torch.empty(g.shape, dtype=torch.float32, device=device) for _ in range(2))
    gr.dq, gr.dk = _view(dq, "dq", tuple(q.shape), device), _view(dk, "dk", tuple(q.shape), device)
    gr.dv = _view(dv, "dv", tuple(v.shape), device)
    gr.dg, gr.dbeta = dg.data_ptr(), dbeta.data_ptr()
    ws = torch.empty(int(lib().lite_la_gated_delta_bwd_workspace_bytes(a.B, a.N, a.Hk, Hv, d,
                                                                       int(cu_seqlens is not None))),
                     dtype=torch.uint8, device=device)
    _on_stream(ws, stream)
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
    with torch.cuda.device(device):
        _check(lib().lite_la_gated_delta_bwd(ctypes.byref(a), ctypes.byref(gr), saved.data_ptr(), saved.numel(),
                                             _stream_handle(stream, device)))
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
                ctx.save_for_backward(q, k, v, g, beta, state_in, cu_seqlens, state_out, saved)
                ctx.scale = scale
                return out, state_out

            @staticmethod
            @once_differentiable
            def backward(ctx, dout, dstate):
                q, k, v, g, beta, state_in, cu_seqlens, state_out, saved = ctx.saved_tensors
                if dout is None:
                    dout = torch.zeros_like(v, memory_format=torch.contiguous_format)
                dout = dout.to(torch.bfloat16)
                try:
                    _view(dout, "dout", tuple(v.shape), q.device)
                    strides_ok = dout.data_ptr() % 16 == 0 and all(x % 8 == 0 for x in dout.stride()[:3])
                except TypeError:
                    strides_ok = False
                if not strides_ok:
                    dout = dout.contiguous()
                if dstate is not None:
                    dstate = dstate.float().contiguous()
                grads = lite_la_gated_delta_bwd(q, k, v, g, beta, dout, saved, state_out=state_out, dstate_out=dstate,
                                                state_in=state_in, cu_seqlens=cu_seqlens, scale=ctx.scale)
                return (*grads, None, None)

        _FUNCTIONS["delta"] = GatedDelta
    return _FUNCTIONS["delta"]


def lite_la_gated_delta(q, k, v, g, beta, state_in=None, cu_seqlens=None, scale=None):
    """lite_la_gated_delta_fwd that torch autograd can differentiate: returns (out, state_out) with
    gradients for q, k, v, g, beta and state_in.  The forward keeps its states (one per 64 tokens) for
    the backward; where no gradient is wanted it does not."""
    torch = _torch()
    if not torch.is_grad_enabled() or not any(isinstance(t, torch.Tensor) and t.requires_grad
                                              for t in (q, k, v, g, beta, state_in)):
        return lite_la_gated_delta_fwd(q, k, v, g, beta, state_in=state_in, cu_seqlens=cu_seqlens, scale=scale)
    return _delta_function().apply(q, k, v, g, beta, state_in, cu_seqlens, scale)


def lite_la_gated_delta_step(q, k, v, g, beta, states, state_indices=None, scale=None, out=None, stream=None):
    """One token of each of B sequences: q, k bf16 [B, Hk, d], v bf16 [B, Hv, d], g, beta fp32
    [B, Hv]; states fp32 [pool, Hv, d, d] is updated in place, row b's state being
    states[state_indices[b]] (int32 [B] on the device; None: states[b]).  A row with an index
    outside the pool, or with one that an earlier row has, touches no state and gets zeros.
    Returns out bf16 [B, Hv, d]."""
    torch = _torch()
    if not all(isinstance(t, torch.Tensor) and t.dim() == 3 for t in (q, k, v)) \
            or not all(isinstance(t, torch.Tensor) and t.dim() == 2 for t in (g, beta)):
        raise TypeError("q, k must be [B, Hk, d], v [B, Hv, d], g and beta [B, Hv]")
    a, B = _delta_args(*(t.unsqueeze(1) for t in (q, k, v, g, beta)), scale, None)
    d, Hv, device = int(a.d), int(a.Hv), q.device
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise TypeError("states must be a contiguous fp32 tensor [pool, Hv, d, d]")
    a.state_in = a.state_out = _states(states, "states", (int(states.shape[0]), Hv, d, d), device)
    if state_indices is not None and (state_indices.dtype != torch.int32 or tuple(state_indices.shape) != (B,)
                                      or not state_indices.is_contiguous() or state_indices.device != device):
        raise TypeError("state_indices must be a contiguous int32 tensor [B] on q's device")
    if out is None:
        out = torch.empty((B, Hv, d), dtype=torch.bfloat16, device=device)
    elif not isinstance(out, torch.Tensor) or tuple(out.shape) != (B, Hv, d):
        raise TypeError("out must be a bf16 CUDA tensor [B, Hv, d]")
    a.out = _view(out.unsqueeze(1), "out", (B, 1, Hv, d), device)
    with torch.cuda.device(device):
        _check(lib().lite_la_gated_delta_step(ctypes.byref(a), _ptr(state_indices), int(states.shape[0]),
                                              _stream_handle(stream, device)))
    return out
