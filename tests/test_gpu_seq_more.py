"""More of the language-model operators on the GPU: packed calls of few tokens each, the edges of the
rule that picks the recurrence, offsets beyond 2^31 elements, several calls at once.

Tolerances are those of test_gpu_delta.py and test_gpu_norm.py: half a step of bf16 (2^-8) on outputs in
bf16, 2^-14 of a head's largest value on fp32 states (bf16 pairs as factors of fp32 sums)."""
import numpy as np
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from oracle.seq_oracle import gated_delta, qk_norm_rope
from tests.test_gpu_delta import close16, close32, fwd, make, np64, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


def check(t, out, state):
    for i, e, sl, (want, S) in ref(t):
        assert close16(out[e, sl], want) and close32(state[i], S), t["lens"]


SHORT = [[1] * 40, [0] * 30 + [120] + [3] * 20, [8] * 64, [8] * 63 + [9], [2, 0, 9, 30, 1, 4], [0, 0, 0, 33, 0], [7] * 5 + [0] * 60,
         [512] + [0] * 63, [513] + [0] * 63]


@pytest.mark.parametrize("lens", SHORT, ids=lambda x: "%d in %d" % (sum(x), len(x)))
@pytest.mark.parametrize("Hk,Hv,d,carry", [(1, 2, 32, True), (2, 2, 64, False), (1, 1, 128, True)])
def test_packed_calls_of_few_tokens(lens, Hk, Hv, d, carry):
    t = make(lens, True, Hk, Hv, d, carry, seed=len(lens))
    check(t, *fwd(t))


@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
def test_lengths_around_the_steps(N):
    t = make([N, N], False, 1, 3, 64, True, seed=N)
    check(t, *fwd(t))


def test_short_packed_call_keeps_to_its_rows_and_sequences():
    """Rows of no sequence: left alone in a given buffer, zeros in a new one; a NaN stays in its sequence."""
    lens = [3, 1, 6, 2]
    t = make(lens, True, 1, 2, 64, True, seed=5)
    pad = lambda x: torch.nn.functional.pad(x, (0,) * (2 * (x.dim() - 2)) + (2, 5))  # noqa: E731
    args = [pad(t[n]) for n in ("q", "k", "v", "g", "beta")]
    cu = t["cu"] + 2
    want, want_s = fwd(t)
    out, s = ll.lite_la_gated_delta_fwd(*args, state_in=t["state_in"], cu_seqlens=cu)
    assert torch.equal(out[:, 2:14], want) and torch.equal(s, want_s)
    assert not out[:, :2].any() and not out[:, 14:].any()
    given = torch.full_like(args[2], 7.0)
    ll.lite_la_gated_delta_fwd(*args, state_in=t["state_in"], cu_seqlens=cu, out=given)
    assert torch.equal(given[:, 2:14], want) and (given[:, :2] == 7).all() and (given[:, 14:] == 7).all()
    args[1][0, 2 + 3 + 1 + 2, 0, 5] = float("nan")     # token 2 of sequence 2
    out, s = ll.lite_la_gated_delta_fwd(*args, state_in=t["state_in"], cu_seqlens=cu)
    assert torch.equal(out[:, 2:8], want[:, :6]) and torch.isnan(out[:, 8:12]).all() and torch.equal(out[:, 12:14], want[:, 10:])
    assert torch.equal(s[[0, 1, 3]], want_s[[0, 1, 3]]) and torch.isnan(s[2]).all()


def test_state_beyond_2_31_elements():
    """A pool of 2^31 + 2^24 state elements: the last entry's offsets do not fit in 32 bits."""
    Hv, d = 16, 128
    pool = (2 ** 31 + 2 ** 24) // (Hv * d * d)
    states = torch.empty(pool, Hv, d, d, device="cuda")
    t = make([1, 1], False, 4, Hv, d, True, seed=3)
    slots = torch.tensor([pool - 1, 0], dtype=torch.int32, device="cuda")
    states[slots.long()] = t["state_in"]
    out = ll.lite_la_gated_delta_step(*(t[n][:, 0] for n in ("q", "k", "v", "g", "beta")), states, state_indices=slots)
    check(t, out[:, None], states[slots.long()])


@pytest.mark.parametrize("N", [20, 200])
def test_views_beyond_2_31_elements(N):
    """v's and out's rows 2^24 elements apart: the last ones' offsets do not fit in 32 bits (N = 200)."""
    t = make([N], False, 1, 2, 32, True, seed=4)
    big = torch.empty(N * 2 ** 24, dtype=torch.bfloat16, device="cuda")
    v = big.as_strided((1, N, 2, 32), (0, 2 ** 24, 32, 1))
    out = big.as_strided((1, N, 2, 32), (0, 2 ** 24, 32, 1), 64)
    v.copy_(t["v"])
    with pytest.raises(ll.LiteLAError):     # the spans of v and out interleave: refused, whatever the rows
        ll.lite_la_gated_delta_fwd(t["q"], t["k"], v, t["g"], t["beta"], out=out)
    check(t, *ll.lite_la_gated_delta_fwd(t["q"], t["k"], v, t["g"], t["beta"], state_in=t["state_in"]))


def test_norm_rows_beyond_2_31_elements():
    Hq, Hk, Hv, d = 24, 4, 4, 128
    W = (Hq + Hk + Hv) * d
    N = 2 ** 31 // W + 40
    x = torch.zeros(1, N, W, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(1, 30, W, generator=g, device="cuda").bfloat16()
    x[:, -30:] = tail
    ang = torch.randn(50, d // 2, generator=g, device="cuda")
    pos = torch.full((1, N), -1, dtype=torch.int32, device="cuda")
    pos[:, -30:] = torch.arange(30, dtype=torch.int32, device="cuda")
    ll.lite_la_qk_norm_rope_fwd(x, Hq, Hk, d=d, cos=ang.cos(), sin=ang.sin(), positions=pos, out=x)
    want = qk_norm_rope(np64(tail).reshape(1, 30, -1, d), Hq, Hk, None, None, np64(ang.cos()), np64(ang.sin()), np.arange(30)[None],
                        1e-6, False)
    got = np64(x[:, -30:]).reshape(want.shape)
    top = np.abs(want).max(-1, keepdims=True)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * top).all()
    assert not x[:, -60:-30].any()


@pytest.mark.parametrize("Hq,Hk,Hv", [(3, 0, 2), (0, 2, 0), (5, 1, 0), (1, 7, 9), (0, 0, 3)])
@pytest.mark.parametrize("d,il", [(32, True), (128, False)])
def test_norm_parts_of_a_row_and_padding(Hq, Hk, Hv, d, il):
    """q, k and v of uneven widths, in place and out of place, with padded rows; the gradient too."""
    B, N = 2, 37
    W = (Hq + Hk + Hv) * d
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy, ang = r(B, N, W).bfloat16(), r(B, N, W).bfloat16(), r(40, d // 2)
    wq, wk = 1 + 0.2 * r(d), 1 + 0.2 * r(d)
    pos = torch.arange(N, device="cuda").repeat(B, 1)
    pos[1, ::3] = -1
    kw = dict(d=d, q_weight=wq, k_weight=wk, cos=ang.cos(), sin=ang.sin(), positions=pos, interleaved=il)
    heads = lambda t: np64(t).reshape(B, N, -1, d)  # noqa: E731
    want = qk_norm_rope(heads(x), Hq, Hk, np64(wq), np64(wk), np64(ang.cos()), np64(ang.sin()), pos.cpu().numpy(), 1e-6, il)
    out = ll.lite_la_qk_norm_rope_fwd(x, Hq, Hk, **kw)
    top = np.abs(want).max(-1, keepdims=True)
    assert (np.abs(heads(out) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * top).all()
    there = x.clone()
    ll.lite_la_qk_norm_rope_fwd(there, Hq, Hk, out=there, **kw)
    real = pos >= 0
    assert torch.equal(there[real], out[real]) and torch.equal(there[~real], x[~real])
    dx, dwq, dwk = ll.lite_la_qk_norm_rope_bwd(x, dy, Hq, Hk, **kw)
    grad = dy.clone()
    again = ll.lite_la_qk_norm_rope_bwd(x, grad, Hq, Hk, dqkv=grad, **kw)
    assert torch.equal(dx, again[0]) and torch.equal(dwq, again[1]) and torch.equal(dwk, again[2])
    assert not dx[~real].any()
    _, ref_q, ref_k = qk_norm_rope(heads(x), Hq, Hk, np64(wq), np64(wk), np64(ang.cos()), np64(ang.sin()), pos.cpu().numpy(), 1e-6,
                                   il, dout=heads(dy))
    for got, want_w, n in ((dwq, ref_q, Hq), (dwk, ref_k, Hk)):
        # |t| <= sqrt(2) max |dy|, |x| r up to 5: terms below 30, B N n of them, 2^-17 of their sum
        assert np.abs(np64(got) - want_w).max() <= 2.0 ** -17 * 30 * B * N * n + 1e-30


def test_calls_at_once():
    """Three calls on streams of their own, and a graph of a call on a fourth, share nothing."""
    a, b = make([700, 30, 0, 64], True, 2, 4, 128, True, seed=1), make([9, 3, 5], True, 2, 4, 64, True, seed=2)
    c = make([130, 130], False, 1, 2, 32, False, seed=3)
    want = [fwd(t) for t in (a, b, c)]
    call = lambda t, **kw: ll.lite_la_gated_delta_fwd(*(t[n] for n in ("q", "k", "v", "g", "beta")),  # noqa: E731
                                                      state_in=t["state_in"], cu_seqlens=t["cu"], **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call(a)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(streams[3]):
            graph.replay()
        got.append([call(t, stream=st) for t, st in zip((a, b, c), streams)])
    torch.cuda.synchronize()
    for results in got:
        for x, w in zip(results, want):
            assert torch.equal(x[0], w[0]) and torch.equal(x[1], w[1])
    assert torch.equal(captured[0], want[0][0]) and torch.equal(captured[1], want[0][1])
    ll.lite_la_device_status()


def test_decay_gradient_where_decays_are_strong():
    """dg_n = <G_n, A_n>, the state that decays and its gradient, is small there beside the sums of q . dq
    and dv . v that differ by it from token to token.  States and their gradients come from fp32 sums of
    products with factors of bf16 pairs (2^-17 each, two of them): 2^-16 of their norms, so dg is off by at
    most 2^-15 |G_n| |A_n|.  Its terms are summed over a chunk of 64 tokens in fp32, each rounding 2^-24 of a sum
    that is at most the chunk's largest |G| |A|: 64 of them, 2^-18 of that."""
    N, H, d = 150, 2, 64
    t = make([N], False, H, H, d, True, seed=8, rate=40.0)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    out, state, saved = ll.lite_la_gated_delta_fwd_save(*args, state_in=t["state_in"])
    got = ll.lite_la_gated_delta_bwd(*args, t["dout"], saved, dstate_out=t["dstate"], state_in=t["state_in"])
    q, k, v, g, beta, do = (np64(x[0]) for x in (*args, t["dout"]))
    want = gated_delta(q, k, v, g, beta, d ** -0.5, np64(t["state_in"][0]), (do, np64(t["dstate"][0])))[2]
    S, G, decayed = np64(t["state_in"][0]), np64(t["dstate"][0]), []
    for n in range(N):
        decayed.append(np.exp(g[n])[:, None, None] * S)
        u = beta[n][:, None] * (v[n] - np.einsum("hij,hi->hj", decayed[n], k[n]))
        S = decayed[n] + k[n][:, :, None] * u[:, None, :]
    norm = lambda x: np.sqrt((x * x).sum((-1, -2)))  # noqa: E731
    size, off = np.zeros((N, H)), np.zeros((N, H))
    for n in reversed(range(N)):
        G = G + d ** -0.5 * q[n][:, :, None] * do[n][:, None, :]
        G = G - k[n][:, :, None] * want[2][n][:, None, :]
        size[n], off[n] = norm(G) * norm(decayed[n]), np.abs(np64(got[3][0, n]) - want[3][n])
        G = np.exp(g[n])[:, None, None] * G
    for c in range(0, N, 64):
        s = size[c:c + 64]
        assert (off[c:c + 64] <= 2.0 ** -15 * s + 2.0 ** -18 * s.max(0)).all(), c
