"""Calls at the edges of the gated delta rule's and the head norms' entry points: no tokens, streams,
frozen weights, gradients as autograd hands them, rows far apart."""
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from linear_attention_diffusion_litela_b200 import seq
from tests.test_gpu_delta import autograd, fwd, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


@pytest.mark.parametrize("lens,packed", [([0, 0, 0], True), ([0], True), ([0, 0], False)])
@pytest.mark.parametrize("d,carry", [(32, True), (128, True), (64, False)])
def test_a_training_step_without_tokens(lens, packed, d, carry):
    """The states pass through, and so do their gradients"""
    t = make(lens, packed, 1, 2, d, carry, seed=d)
    for n in ("q", "k", "v", "g", "beta"):
        t[n].requires_grad_()
    out, state, grads = autograd(t)
    assert out.shape == t["v"].shape and all(grads[n].shape == t[n].shape for n in grads)
    assert torch.equal(state, t["state_in"] if carry else torch.zeros_like(t["dstate"]))
    if carry:
        assert torch.equal(grads["state_in"], t["dstate"])


def test_buffers_of_a_call_on_another_stream(monkeypatch):
    """They come from that stream's memory, not from blocks that the current stream may still have in use"""
    t = make([300, 80], True, 1, 2, 64, True)
    qkv = torch.randn(2, 600, 6 * 64, device="cuda").bfloat16()
    w = torch.ones(64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    # memory that the current stream could give
    spare = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (1 << 9, 1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24) for _ in range(3)]
    del spare
    buffers = []
    call = seq._call

    def spy(fn, dev, stream, *args):
        for x in args:
            if isinstance(x, bytes) and len(x) == seq._DELTA_ARGS.size:
                buffers.append(seq._DELTA_ARGS.unpack(x)[-2])
        if fn is ll.lib().lite_la_qk_norm_rope_bwd:
            buffers.append(args[-2])
        call(fn, dev, stream, *args)

    monkeypatch.setattr(seq, "_call", spy)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    kw = dict(state_in=t["state_in"], cu_seqlens=t["cu"], stream=s)
    made = list(ll.lite_la_gated_delta_fwd(*args, **kw))
    made += ll.lite_la_gated_delta_fwd_save(*args, **kw)
    made += ll.lite_la_gated_delta_bwd(*args, t["dout"], made[-1], dstate_out=t["dstate"], **kw)
    made.append(ll.lite_la_gated_delta_step(*(x[0, :2] for x in args), t["state_in"].clone(), stream=s))
    made.append(ll.lite_la_qk_norm_rope_fwd(qkv, 2, 2, d=64, q_weight=w, stream=s))
    made += [x for x in ll.lite_la_qk_norm_rope_bwd(qkv, qkv.clone(), 2, 2, d=64, q_weight=w, k_weight=w, stream=s)]
    torch.cuda.synchronize()
    at = [x.data_ptr() for x in made] + [p for p in buffers if p]
    assert len(at) == len(made) + 3     # the forward's and both backwards' workspaces
    segments = torch.cuda.memory_snapshot()
    for p in at:
        own = [g for g in segments if g["address"] <= p < g["address"] + g["total_size"]]
        assert len(own) == 1 and own[0]["stream"] == s.cuda_stream


def test_a_captured_call_on_another_stream():
    t = make([150, 70], True, 1, 2, 64, True)
    want = fwd(t)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = fwd(t, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tangents_are_refused_not_lost():
    """Forward-mode differentiation is not offered: refused whether or not a gradient is wanted as well"""
    import torch.autograd.forward_ad as forward_ad
    t = make([40, 40], False, 1, 1, 32, False)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    with forward_ad.dual_level():
        for i in range(5):
            dual = list(args)
            dual[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises((RuntimeError, NotImplementedError)):
                ll.lite_la_gated_delta(*dual)
        plain = ll.lite_la_gated_delta(*args)     # no tangent, none lost
    assert all(torch.equal(a, b) for a, b in zip(plain, fwd(t)))
    with forward_ad.dual_level():
        state = forward_ad.make_dual(torch.zeros(2, 1, 32, 32, device="cuda"), torch.ones(2, 1, 32, 32, device="cuda"))
        with pytest.raises((RuntimeError, NotImplementedError)):
            ll.lite_la_gated_delta(*args, state_in=state)
        with pytest.raises((RuntimeError, NotImplementedError)):
            ll.lite_la_qk_norm_rope(forward_ad.make_dual(t["q"].flatten(2), torch.ones_like(t["q"].flatten(2))), 1, 0)


@pytest.mark.parametrize("wanted", [(), (0,), (1,), (2,), (0, 2), (0, 1, 2)])
def test_frozen_weights_of_the_head_norms(monkeypatch, wanted):
    """Only the weights' gradients that autograd wants are computed; they are those of the full call"""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    leaves = [r(2, 50, 6 * 64).bfloat16(), 1 + 0.2 * r(64), 1 + 0.2 * r(64)]
    dout = r(2, 50, 6 * 64).bfloat16()
    want = ll.lite_la_qk_norm_rope_bwd(leaves[0], dout, 3, 2, d=64, q_weight=leaves[1], k_weight=leaves[2])
    for i in wanted:
        leaves[i].requires_grad_()
    out = ll.lite_la_qk_norm_rope(leaves[0], 3, 2, d=64, q_weight=leaves[1], k_weight=leaves[2])
    assert out.requires_grad == bool(wanted)
    asked = []
    call = seq._call
    monkeypatch.setattr(seq, "_call", lambda fn, dev, stream, *args: (asked.append(args), call(fn, dev, stream, *args)))
    if wanted:
        got = torch.autograd.grad(out, [leaves[i] for i in wanted], dout)
        assert all(torch.equal(a, want[i]) for a, i in zip(got, wanted))
        (args,) = asked
        assert [bool(args[5]), bool(args[6])] == [1 in wanted, 2 in wanted]      # dq_weight, dk_weight
        assert bool(args[-2]) == (1 in wanted or 2 in wanted)                    # the workspace


def odd(x):
    """x's values, contiguous, 4 bytes from a 16-byte boundary: as a gradient may be a part of something"""
    pad = 4 // x.element_size()
    y = torch.empty(x.numel() + pad, dtype=x.dtype, device=x.device)[pad:].view(x.shape).copy_(x)
    assert y.is_contiguous() and y.data_ptr() % 16 == 4
    return y


def test_incoming_gradients_off_the_alignment():
    t = make([90, 50], True, 1, 2, 64, True)
    want = autograd(t)[2]
    got = autograd(dict(t, dout=odd(t["dout"]), dstate=odd(t["dstate"])))[2]
    assert all(torch.equal(got[n], want[n]) for n in want)
    x = torch.randn(2, 50, 6 * 64, device="cuda").bfloat16().requires_grad_()
    dout = torch.randn(2, 50, 6 * 64, device="cuda").bfloat16()
    grads = [torch.autograd.grad(ll.lite_la_qk_norm_rope(x, 3, 2, d=64), x, g)[0] for g in (dout, odd(dout))]
    assert torch.equal(*grads)


def test_gradient_of_sequences_without_tokens():
    """Rows, but none of them a sequence's: the state's gradient passes through, the rows' are zero"""
    t = make([0, 0], True, 1, 2, 64, True)
    for n in ("q", "k", "v", "g", "beta", "dout"):
        t[n] = torch.ones((1, 200) + t[n].shape[2:], dtype=t[n].dtype, device="cuda")
    _, state, grads = autograd(t)
    assert torch.equal(state, t["state_in"]) and torch.equal(grads["state_in"], t["dstate"])
    assert not any(grads[n].any() for n in ("q", "k", "v", "g", "beta"))


def wide(N, stride, heads, d, at=0, buffer=None):
    """[1, N, heads, d] with its rows `stride` elements apart, from element `at` on of a buffer"""
    buffer = torch.empty(N * stride, dtype=torch.bfloat16, device="cuda") if buffer is None else buffer
    return buffer.as_strided((1, N, heads, d), (0, stride, d, 1), at), buffer


@pytest.mark.parametrize("N,stride", [(30, 2 ** 27), (200, 2 ** 24)])     # the recurrence; chunks
def test_outputs_beyond_2_31_elements(N, stride):
    t = make([N], False, 1, 2, 32, True, seed=4)
    want, want_s = fwd(t)
    out, _ = wide(N, stride, 2, 32)
    _, state = fwd(t, out=out)
    assert torch.equal(out, want) and torch.equal(state, want_s)


def test_one_token_outputs_beyond_2_31_elements():
    B, stride = 20, 2 ** 27
    t = make([1] * B, False, 1, 2, 32, True, seed=6)
    one = [t[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    states = [t["state_in"].clone() for _ in range(2)]
    want = ll.lite_la_gated_delta_step(*one, states[0])
    v, _ = wide(B, stride, 2, 32)
    out, _ = wide(B, stride, 2, 32)
    v.copy_(t["v"].transpose(0, 1))
    one[2] = v[0]
    ll.lite_la_gated_delta_step(*one, states[1], out=out[0])
    assert torch.equal(out[0], want) and torch.equal(*states)


def test_gradients_beyond_2_31_elements():
    """dq, dk and dv in one buffer, each between the others' rows, dout far apart too (the C call takes views)"""
    N, stride, d = 200, 2 ** 24, 32
    t = make([N], False, 1, 2, d, True, seed=4)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    _, _, saved = ll.lite_la_gated_delta_fwd_save(*args, state_in=t["state_in"])
    want = ll.lite_la_gated_delta_bwd(*args, t["dout"], saved, dstate_out=t["dstate"], state_in=t["state_in"])
    a = seq._Delta(*args, None, None)
    dout, _ = wide(N, stride, 2, d)
    dout.copy_(t["dout"])
    dq, buffer = wide(N, stride, 1, d)
    dk, dv = wide(N, stride, 1, d, 64, buffer)[0], wide(N, stride, 2, d, 128, buffer)[0]
    dg, dbeta, dstate = (torch.empty_like(x) for x in want[3:])
    size = a.bytes(ll.lib().lite_la_gated_delta_bwd_workspace_bytes)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    views = [seq._view(x, "", x.shape, a.dev) for x in (dout, dq, dk, dv)]
    grads = seq._DELTA_GRADS.pack(*sum(views, ()), dg.data_ptr(), dbeta.data_ptr(), t["dstate"].data_ptr(), dstate.data_ptr())
    seq._call(ll.lib().lite_la_gated_delta_bwd, a.dev, None,
              a.pack(seq._NO_VIEW, t["state_in"].data_ptr(), 0, 0, ws.data_ptr(), size), grads, saved.data_ptr(), saved.numel())
    assert all(torch.equal(x, y) for x, y in zip((dq, dk, dv, dg, dbeta, dstate), want))


def test_buffers_written_in_place_are_known_to_autograd():
    """A backward that needs what a later call has written over says so, as torch's own in-place operations make it"""
    t = make([70, 70], False, 1, 2, 64, True)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    weight = torch.ones((), device="cuda", requires_grad=True)

    def lost(y):   # `y` is needed for weight's gradient
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            torch.autograd.grad(y.sum(), weight)

    qkv = torch.randn(2, 50, 6 * 64, device="cuda").bfloat16()
    for write in (lambda x: ll.lite_la_qk_norm_rope_fwd(x, 3, 2, d=64, out=x),
                  lambda x: ll.lite_la_qk_norm_rope_bwd(qkv, x, 3, 2, d=64, dqkv=x)):
        x = qkv.clone()
        y = x * weight
        write(x)
        lost(y)
    for write in (lambda x: ll.lite_la_gated_delta_fwd(*args, state_in=x, state_out=x),
                  lambda x: ll.lite_la_gated_delta_fwd_save(*args, state_in=t["state_in"], state_out=x),
                  lambda x: ll.lite_la_gated_delta_step(*(a[:, 0] for a in args), x)):
        x = t["state_in"].clone()
        y = x * weight
        write(x)
        lost(y)
    x = torch.zeros_like(t["v"])
    y = x * weight
    ll.lite_la_gated_delta_fwd(*args, out=x)
    lost(y)
    x = torch.zeros_like(t["v"][:, 0])
    y = x * weight
    ll.lite_la_gated_delta_step(*(a[:, 0] for a in args), t["state_in"].clone(), out=x)
    lost(y)
    # nothing given, nothing written: the gradient is there
    y = qkv * weight
    ll.lite_la_qk_norm_rope_fwd(qkv, 3, 2, d=64)
    assert torch.isfinite(torch.autograd.grad(y.sum(), weight)[0])
    # and a saved state that a later token is put into
    q = t["q"].clone().requires_grad_()
    S = t["state_in"].clone()
    out, _ = ll.lite_la_gated_delta(q, *args[1:], state_in=S)
    ll.lite_la_gated_delta_step(*(a[:, 0] for a in args), S)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out.float().sum(), q)
    with torch.inference_mode():
        ll.lite_la_gated_delta_step(*(a[:, 0] for a in args), t["state_in"].clone())
