"""The gated delta rule against the fp64 oracle (one token after another).

Tolerances.  out and the gradients of q, k and v are rounded to bf16 once: half a step, 2^-8 of the
value.  Before that every sum is fp32 and every operand of a matrix product is a bf16 value or an
fp32 value held as a bf16 pair (off by at most 2^-17 of itself; the product of two low halves that
is left out adds 2^-16).  At most 8 such products follow one another inside a chunk, the carried
state decays, and a sum of n <= 128 signed terms is about sqrt(n) <= 12 times smaller than its
absolute terms: 8 * 12 * 2^-17 < 2^-10 of a typical value if every error had its largest size and
the same sign; errors of random sign leave under 2^-14 of the largest value of a head, which is what
states and fp32 gradients are held to (2^-13 where two such sums are subtracted)."""
import numpy as np
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from oracle.seq_oracle import gated_delta

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


HALF = 2.0 ** -8
F32 = 2.0 ** -14


def make(lens, packed, Hk, Hv, d, carry, seed=0, rate=1.0):
    """Inputs as such layers make them: unit keys, decays of e^-1e-3 .. e^-2 a token, strengths in (0, 1)"""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    B, N = (1, sum(lens)) if packed else (len(lens), lens[0])
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    t = dict(q=unit(r(B, N, Hk, d)), k=unit(r(B, N, Hk, d)), v=r(B, N, Hv, d).bfloat16())
    t["g"] = -rate * torch.exp(r(B, N, Hv) * 1.5 - 3)
    t["beta"] = torch.sigmoid(r(B, N, Hv))
    t["state_in"] = r(len(lens), Hv, d, d) if carry else None
    t["cu"] = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda") if packed else None
    t["lens"], t["dout"], t["dstate"] = lens, r(B, N, Hv, d).bfloat16(), r(len(lens), Hv, d, d)
    return t


def sequences(t):
    """(entry, token slice) of each sequence"""
    if t["cu"] is None:
        return [(i, slice(0, n)) for i, n in enumerate(t["lens"])]
    at = np.cumsum([0] + list(t["lens"]))
    return [(0, slice(int(a), int(b))) for a, b in zip(at[:-1], at[1:])]


def np64(x):
    return x.detach().double().cpu().numpy()


def ref(t, grads=False, scale=None):
    d = t["q"].shape[-1]
    for i, (e, sl) in enumerate(sequences(t)):
        args = [np64(t[n][e, sl]) for n in ("q", "k", "v", "g", "beta")]
        S0 = None if t["state_in"] is None else np64(t["state_in"][i])
        yield i, e, sl, gated_delta(*args, d ** -0.5 if scale is None else scale, S0,
                                    (np64(t["dout"][e, sl]), np64(t["dstate"][i])) if grads else None)


def close16(got, want):
    """bf16 [N, H, d] against 64 bits: per head"""
    got = np64(got)
    top = np.abs(want).max(axis=(0, 2), keepdims=True, initial=0.0)
    return (np.abs(got - want) <= HALF * np.abs(want) + 4 * F32 * top + 1e-30).all()


def close32(got, want, k=1):
    """fp32 [H, ...] against 64 bits: per head"""
    got = np64(got)
    top = np.abs(want).max(axis=tuple(range(1, want.ndim)), keepdims=True, initial=0.0)
    return (np.abs(got - want) <= k * F32 * top + 1e-30).all()


def fwd(t, **kw):
    return ll.lite_la_gated_delta_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], state_in=t["state_in"],
                                      cu_seqlens=t["cu"], **kw)


def check_fwd(t, out, state, scale=None):
    ll.lite_la_device_status()
    for i, e, sl, (o, S) in ref(t, scale=scale):
        assert close16(out[e, sl], o), "out of sequence %d" % i
        assert close32(state[i], S), "state of sequence %d" % i


SHAPES = [
    # lens, packed, Hk, Hv, d, carry
    ([1], False, 1, 1, 32, False), ([1], False, 2, 4, 128, True), ([2, 2], False, 1, 2, 64, True),
    ([5, 0, 1, 9], True, 2, 2, 32, True), ([33, 33, 33], False, 3, 3, 128, False),
    ([64], False, 1, 1, 128, False), ([65], False, 1, 2, 64, True), ([63, 1, 64, 128, 0, 130], True, 1, 2, 128, True),
    ([200, 7, 311], True, 2, 4, 64, False), ([127, 300], True, 1, 1, 32, True), ([257, 257], False, 2, 6, 32, True),
    ([700], False, 1, 1, 128, True), ([1, 1, 1, 500], True, 1, 1, 64, True), ([0, 0, 3], True, 1, 1, 128, True),
    ([1025], False, 1, 1, 32, False),
]


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", SHAPES)
def test_forward(lens, packed, Hk, Hv, d, carry):
    t = make(lens, packed, Hk, Hv, d, carry, seed=sum(lens) + d)
    out, state = fwd(t)
    check_fwd(t, out, state)


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", [([70, 20], True, 1, 2, 64, True), ([300], False, 1, 1, 128, True)])
@pytest.mark.parametrize("case", ["strong decay", "resets", "no decay", "no write", "full write", "equal keys"])
def test_forward_at_the_ends_of_the_gates(lens, packed, Hk, Hv, d, carry, case):
    t = make(lens, packed, Hk, Hv, d, carry, seed=5)
    if case == "strong decay":
        t["g"] = t["g"] - 30
    elif case == "resets":
        t["g"][:, ::7] = -float("inf")
        t["g"][:, 3::31] = -1e30
    elif case == "no decay":
        t["g"] = torch.zeros_like(t["g"])
    elif case == "no write":
        t["beta"] = torch.zeros_like(t["beta"])
    elif case == "full write":
        t["beta"] = torch.ones_like(t["beta"])
    else:
        t["k"] = t["k"][:, :1].expand_as(t["k"])     # token stride 0
        t["beta"] = torch.ones_like(t["beta"])
    out, state = fwd(t)
    with np.errstate(under="ignore"):
        check_fwd(t, out, state)


def test_packed_views_and_strides():
    """q, k and v as views of packed rows, heads before tokens, gates inside a wider tensor."""
    B, N, Hk, Hv, d = 2, 150, 2, 4, 64
    t = make([N] * B, False, Hk, Hv, d, True)
    want, want_s = fwd(t)
    row = torch.cat([t[n].flatten(2) for n in ("q", "k", "v")], -1)
    q, k, v = row.split([Hk * d, Hk * d, Hv * d], -1)
    gb = torch.cat([t["g"], t["beta"]], -1)
    out = torch.full((B, N, Hv + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    o, s = ll.lite_la_gated_delta_fwd(q.view(B, N, Hk, d), k.view(B, N, Hk, d), v.view(B, N, Hv, d), gb[..., :Hv],
                                      gb[..., Hv:], state_in=t["state_in"], out=out[:, :, 1:Hv + 1])
    assert torch.equal(o, want) and torch.equal(s, want_s)
    assert (out[:, :, 0] == 7).all() and (out[:, :, Hv + 1:] == 7).all()
    by_head = [t[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v")]
    o, s = ll.lite_la_gated_delta_fwd(*by_head, t["g"], t["beta"], state_in=t["state_in"])
    assert torch.equal(o, want) and torch.equal(s, want_s)


def test_state_in_place_and_in_two_parts():
    t = make([190, 190], False, 1, 2, 64, True)
    out, state = fwd(t)
    S = t["state_in"].clone()
    fwd(t, state_out=S)                 # another buffer than state_in: the same result
    assert torch.equal(S, state)
    S = t["state_in"].clone()
    parts = []
    for sl in (slice(0, 77), slice(77, 190)):
        o, _ = ll.lite_la_gated_delta_fwd(*(t[n][:, sl] for n in ("q", "k", "v", "g", "beta")), state_in=S, state_out=S)
        parts.append(o)
    check_fwd(t, torch.cat(parts, 1), S)


def test_rows_of_no_sequence():
    """Rows behind the last sequence (and what stands in them) touch nothing and are left alone."""
    t = make([90, 41], True, 1, 2, 64, True)
    want, want_s = fwd(t)
    pad = {n: torch.cat([t[n], torch.full_like(t[n][:, :40], float("nan"))], 1) for n in ("q", "k", "v", "g", "beta")}
    out = torch.full((1, 171, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    o, s = ll.lite_la_gated_delta_fwd(*pad.values(), state_in=t["state_in"], cu_seqlens=t["cu"], out=out)
    assert torch.equal(o[:, :131], want) and torch.equal(s, want_s) and (o[:, 131:] == 3).all()
    o, s = ll.lite_la_gated_delta_fwd(*pad.values(), state_in=t["state_in"], cu_seqlens=t["cu"])
    assert torch.equal(o[:, :131], want) and torch.equal(s, want_s) and not o[:, 131:].any()


def test_nan_stays_in_its_sequence():
    t = make([100, 70, 64], True, 1, 1, 64, False)
    want, want_s = fwd(t)
    t["v"][0, 120] = float("nan")
    t["k"][0, 121] = float("inf")
    out, s = fwd(t)
    assert torch.equal(out[:, :100], want[:, :100]) and torch.equal(out[:, 170:], want[:, 170:])
    assert torch.equal(s[[0, 2]], want_s[[0, 2]]) and torch.equal(out[:, 100:120], want[:, 100:120])
    assert torch.isnan(out[:, 120:170]).all()


def test_bad_offsets_stay_inside_the_buffers():
    """Offsets that point outside are cut; the call comes back and other rows are right."""
    t = make([64, 64], True, 1, 1, 32, False)
    want, _ = fwd(t)
    t["cu"] = torch.tensor([0, 64, 2 ** 30], dtype=torch.int32, device="cuda")
    out, _ = fwd(t)
    ll.lite_la_device_status()
    assert torch.equal(out, want)
    t["cu"] = torch.tensor([-5, 64, 128], dtype=torch.int32, device="cuda")
    out, _ = fwd(t)
    assert torch.equal(out, want)


@pytest.mark.parametrize("B,pool,Hk,Hv,d", [(1, 1, 1, 1, 32), (3, 5, 2, 4, 128), (17, 20, 1, 3, 64), (200, 200, 1, 1, 32)])
def test_step(B, pool, Hk, Hv, d):
    t = make([1] * B, False, Hk, Hv, d, False, seed=B)
    g = torch.Generator(device="cuda").manual_seed(1)
    states = torch.randn((pool, Hv, d, d), generator=g, device="cuda")
    slots = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32)
    before = states.clone()
    t["state_in"] = states[slots.long()].clone()
    one = [t[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    out = ll.lite_la_gated_delta_step(*one, states, state_indices=slots)
    check_fwd(t, out[:, None], states[slots.long()])
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert torch.equal(states[rest], before[rest])
    if B == pool:
        again = before.clone()
        order = torch.argsort(slots)
        out2 = ll.lite_la_gated_delta_step(*(x[order] for x in one), again)
        assert torch.equal(out2, out[order]) and torch.equal(again, states)


def test_step_padded_and_repeated_rows():
    t = make([1] * 6, False, 1, 2, 64, False)
    one = [t[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    states = torch.randn(4, 2, 64, 64, device="cuda")
    before = states.clone()
    slots = torch.tensor([2, -1, 0, 2, 4, 0], dtype=torch.int32, device="cuda")
    out = ll.lite_la_gated_delta_step(*one, states, state_indices=slots)
    assert not out[[1, 3, 4, 5]].any()
    want = before.clone()
    o = ll.lite_la_gated_delta_step(*(x[[0, 2]] for x in one), want, state_indices=slots[[0, 2]])
    assert torch.equal(out[[0, 2]], o) and torch.equal(states, want) and torch.equal(states[[1, 3]], before[[1, 3]])


def test_step_follows_the_sequence_form():
    """A prompt, then its next tokens one at a time: as the whole sequence at once."""
    t = make([100, 100], False, 2, 4, 128, True)
    out, state = fwd(t)
    part = [t[n][:, :93] for n in ("q", "k", "v", "g", "beta")]
    o, S = ll.lite_la_gated_delta_fwd(*part, state_in=t["state_in"])
    outs = [o] + [ll.lite_la_gated_delta_step(*(t[n][:, i] for n in ("q", "k", "v", "g", "beta")), S)[:, None]
                  for i in range(93, 100)]
    check_fwd(t, torch.cat(outs, 1), S)


def test_norm_then_delta_on_packed_rows():
    """The run as a layer has it: packed rows, head norms with rotation, the delta rule on views."""
    from oracle.seq_oracle import qk_norm_rope
    B, N, Hk, Hv, d = 2, 140, 2, 4, 64
    t = make([N] * B, False, Hk, Hv, d, False)
    qkv = torch.randn(B, N, (2 * Hk + Hv) * d, device="cuda").bfloat16()
    w = torch.full((d,), d ** -0.5, device="cuda")     # with this weight the norm is the unit norm
    ang = torch.arange(N, device="cuda")[:, None] * 0.1 ** torch.arange(16, device="cuda")[None]
    y = ll.lite_la_qk_norm_rope_fwd(qkv, Hk, Hk, d=d, q_weight=w, k_weight=w, cos=ang.cos(), sin=ang.sin())
    heads = y.view(B, N, -1, d)
    t["q"], t["k"], t["v"] = heads[:, :, :Hk], heads[:, :, Hk:2 * Hk], heads[:, :, 2 * Hk:]
    want = qk_norm_rope(np64(qkv).reshape(B, N, -1, d), Hk, Hk, np64(w), np64(w), np64(ang.cos()), np64(ang.sin()),
                        np.tile(np.arange(N), (B, 1)), 1e-6, False)
    assert (np.abs(np64(heads) - want) <= HALF * np.abs(want) + 2.0 ** -18).all()
    out, state = fwd(t)
    check_fwd(t, out, state)


def test_streams_and_graphs():
    t = make([150, 70], True, 1, 2, 64, True)
    want, want_s = fwd(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, st = fwd(t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and torch.equal(st, want_s)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fwd(t))
        graphs.append(graph)
    # two graphs at once, on two streams
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o[0].zero_()
            o[1].zero_()
        torch.cuda.synchronize()
        for st, graph in ((a, graphs[0]), (b, graphs[1])):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[0], want) and torch.equal(o[1], want_s) for o in outs)
    # the one-token form, replayed with other slots
    states = torch.randn(8, 2, 64, 64, device="cuda")
    one = [t[n][0, :4] for n in ("q", "k", "v", "g", "beta")]
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ll.lite_la_gated_delta_step(*one, states, state_indices=slots)
    for new in ([0, 1, 2, 3], [7, 5, -1, 1]):
        slots.copy_(torch.tensor(new, dtype=torch.int32))
        copy = states.clone()
        graph.replay()
        assert torch.equal(out, ll.lite_la_gated_delta_step(*one, copy, state_indices=slots)) and torch.equal(states, copy)


def test_equal_calls_give_equal_bits():
    t = make([400, 3, 129], True, 2, 4, 128, True)
    a, b = fwd(t), fwd(t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_empty():
    t = make([0, 0], True, 1, 2, 32, True)
    out, state = fwd(t)
    assert out.shape == (1, 0, 2, 32) and torch.equal(state, t["state_in"])
    e = [x[:0] for x in (t["q"], t["k"], t["v"], t["g"], t["beta"])]
    out, state = ll.lite_la_gated_delta_fwd(*e)
    assert out.shape[0] == 0 and state.shape[0] == 0


# ---------------------------------------------------------------------------------------
# gradients


def leaves(t):
    names = ["q", "k", "v", "g", "beta"] + (["state_in"] if t["state_in"] is not None else [])
    return names, [t[n].detach().clone().requires_grad_() for n in names]


def autograd(t, with_state=True):
    names, x = leaves(t)
    kw = dict(zip(names, x))
    out, state = ll.lite_la_gated_delta(*(kw[n] for n in ("q", "k", "v", "g", "beta")), state_in=kw.get("state_in"),
                                        cu_seqlens=t["cu"])
    if with_state:
        grads = torch.autograd.grad((out, state), x, (t["dout"], t["dstate"]))
    else:
        grads = torch.autograd.grad(out, x, t["dout"])
    return out, state, dict(zip(names, grads))


def check_grads(t, out, state, grads, with_state=True):
    ll.lite_la_device_status()
    if not with_state:
        t = dict(t, dstate=torch.zeros_like(t["dstate"]))
    for i, e, sl, (o, S, (dq, dk, dv, dg, db, dS)) in ref(t, grads=True):
        assert close16(out[e, sl], o) and close32(state[i], S), "forward of sequence %d" % i
        for n, want in (("q", dq), ("k", dk), ("v", dv)):
            assert close16(grads[n][e, sl], want), "d%s of sequence %d" % (n, i)
        # dg_t = <S, G> at the chunk's end + the sum from t on of (q . dq - v . dv): where the true value
        # is small (0 for a first token without a state) these sums cancel.  Each of their terms is off by
        # at most F32 of the sum of its absolute products, and so is the difference: the largest such sum of
        # a head is the measure, not dg.
        terms = [np.abs(np64(t["v"][e, sl]) * dv).sum(-1),
                 np.abs(np.repeat(np64(t["q"][e, sl]) * dq, dv.shape[1] // dq.shape[1], 1)).sum(-1)]
        bound = 4 * F32 * (np.maximum(*terms).max(0, initial=0.0) + np.abs(dg).max(0, initial=0.0)) + 1e-30
        assert (np.abs(np64(grads["g"][e, sl]) - dg) <= bound).all(), "dg of sequence %d" % i
        assert close32(grads["beta"][e, sl].T, db.T, 2), "dbeta of sequence %d" % i
        if "state_in" in grads:
            assert close32(grads["state_in"][i], dS, 2), "dstate of sequence %d" % i


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", SHAPES)
def test_gradients(lens, packed, Hk, Hv, d, carry):
    t = make(lens, packed, Hk, Hv, d, carry, seed=sum(lens) + d)
    check_grads(t, *autograd(t))
    check_grads(t, *autograd(t, False), with_state=False)


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", [([70, 20], True, 1, 2, 64, True), ([150], False, 1, 1, 128, True)])
@pytest.mark.parametrize("case", ["strong decay", "resets", "no decay", "no write", "full write"])
def test_gradients_at_the_ends_of_the_gates(lens, packed, Hk, Hv, d, carry, case):
    t = make(lens, packed, Hk, Hv, d, carry, seed=5)
    if case == "strong decay":
        t["g"] = t["g"] - 30
    elif case == "resets":
        t["g"][:, ::7] = -float("inf")
    elif case == "no decay":
        t["g"] = torch.zeros_like(t["g"])
    elif case == "no write":
        t["beta"] = torch.zeros_like(t["beta"])
    else:
        t["beta"] = torch.ones_like(t["beta"])
    with np.errstate(under="ignore"):
        check_grads(t, *autograd(t))


def test_gradient_against_differences():
    """Central differences of the kernels' own forward in the gates and the values: out and state are
    linear in v exactly; in g and beta the step leaves a relative 1e-3."""
    t = make([130], False, 1, 2, 64, True, seed=3)
    _, _, grads = autograd(t)

    def loss(**kw):
        u = dict(t, **kw)
        out, state = fwd(u)
        # out's bf16 rounding is random: its share of the loss averages over 16640 values
        return (out.double() * t["dout"].double()).sum() + (state.double() * t["dstate"].double()).sum()

    rng = torch.Generator(device="cuda").manual_seed(9)
    for n, step in (("g", 0.05), ("beta", 0.05), ("state_in", 0.5)):
        dirn = torch.randn(t[n].shape, generator=rng, device="cuda")
        num = (loss(**{n: t[n] + step * dirn}) - loss(**{n: t[n] - step * dirn})) / (2 * step)
        ana = (grads[n].double() * dirn.double()).sum()
        # rounding of out: 2^-9 typical, |out dout| summed as random signs, over the step
        out = fwd(t)[0].double()
        noise = 2.0 ** -9 * float((out * t["dout"].double()).norm()) / step
        curve = 0.01 * float((grads[n].double() * dirn.double()).norm())
        assert abs(float(num - ana)) <= 6 * noise + 5 * curve + 0.01 * abs(float(ana)), (n, float(num), float(ana))


def test_gradient_of_shared_and_strided_inputs():
    """Packed rows as the leaf: views of it go in, one gradient comes back; broadcast keys too."""
    B, N, Hk, Hv, d = 2, 100, 2, 4, 64
    t = make([N] * B, False, Hk, Hv, d, False)
    want = autograd(t)[2]
    row = torch.cat([t[n].flatten(2) for n in ("q", "k", "v")], -1).requires_grad_()
    h = row.view(B, N, -1, d)
    out, state = ll.lite_la_gated_delta(h[:, :, :Hk], h[:, :, Hk:2 * Hk], h[:, :, 2 * Hk:], t["g"], t["beta"])
    got, = torch.autograd.grad((out, state), row, (t["dout"], t["dstate"]))
    assert torch.equal(got, torch.cat([want[n].flatten(2) for n in ("q", "k", "v")], -1))
    # one key head expanded over two
    k1 = t["k"][:, :, :1].clone().requires_grad_()
    u = dict(t, k=k1.detach().expand(B, N, Hk, d).contiguous())
    out, state = ll.lite_la_gated_delta(t["q"], k1.expand(B, N, Hk, d), t["v"], t["g"], t["beta"])
    got, = torch.autograd.grad((out, state), k1, (t["dout"], t["dstate"]))
    assert torch.equal(got, autograd(u)[2]["k"].sum(2, keepdim=True))
    # an incoming gradient with heads before tokens, and one of fp32
    out, state = ll.lite_la_gated_delta(*(x.requires_grad_() for x in (t["q"], t["k"], t["v"])), t["g"], t["beta"])
    by_head = t["dout"].transpose(1, 2).contiguous().transpose(1, 2)
    got = torch.autograd.grad((out, state), t["q"], (by_head, t["dstate"]))[0]
    assert torch.equal(got, want["q"])


def test_gradient_rows_of_no_sequence():
    t = make([90, 41], True, 1, 2, 64, True)
    want = autograd(t)[2]
    for n in ("q", "k", "v", "g", "beta", "dout"):
        t[n] = torch.cat([t[n], torch.full_like(t[n][:, :40], float("nan"))], 1)
    got = autograd(t)[2]
    for n in want:
        if n != "state_in":
            assert torch.equal(got[n][:, :131], want[n]) and not got[n][:, 131:].any(), n
        else:
            assert torch.equal(got[n], want[n])


def test_gradient_streams_graphs_and_equal_bits():
    t = make([150, 70], True, 1, 2, 64, True)
    _, _, want = autograd(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = autograd(t)[2]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(got[n], want[n]) for n in want)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    out, state, saved = ll.lite_la_gated_delta_fwd_save(*args, state_in=t["state_in"], cu_seqlens=t["cu"], stream=s)
    got = ll.lite_la_gated_delta_bwd(*args, t["dout"], saved, dstate_out=t["dstate"],
                                     state_in=t["state_in"], cu_seqlens=t["cu"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, want[n]) for a, n in zip(got, ("q", "k", "v", "g", "beta", "state_in")))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, state, saved = ll.lite_la_gated_delta_fwd_save(*args, state_in=t["state_in"], cu_seqlens=t["cu"])
        got = ll.lite_la_gated_delta_bwd(*args, t["dout"], saved, dstate_out=t["dstate"],
                                         state_in=t["state_in"], cu_seqlens=t["cu"])
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        assert all(torch.equal(a, want[n]) for a, n in zip(got, ("q", "k", "v", "g", "beta", "state_in")))


def test_no_gradient_wanted():
    t = make([100], False, 1, 1, 32, False)
    want, want_s = fwd(t)
    x = [t[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    with torch.no_grad():
        out, s = ll.lite_la_gated_delta(*x)
    assert torch.equal(out, want) and not out.requires_grad
    out, s = ll.lite_la_gated_delta(*x)
    assert torch.equal(out, want) and torch.equal(s, want_s) and out.requires_grad
    g = torch.autograd.grad(s, x[1], torch.ones_like(s))[0]     # the state alone is used
    assert torch.isfinite(g).all() and g.any()
    with pytest.raises(RuntimeError):
        y = torch.autograd.grad(out.float().sum(), x[0], create_graph=True)[0]
        torch.autograd.grad(y.float().sum(), x[1])
