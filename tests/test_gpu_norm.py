"""Head norms with rotation against the fp64 oracle.

Tolerances.  The result is rounded to bf16 once (half a step: 2^-8 of the value).  Before that come
fp32 sums of d <= 128 terms in 8 sequential and log2 tree additions (under 16 roundings of 2^-24
each), one rsqrt and four products: under 2^-19 of the head's largest value; twice that is
allowed.  The weights' gradients are fp32 sums whose longest chain is below 64 additions at these
sizes: 2^-18 of the sum of absolute terms, doubled for the terms' own error."""
import numpy as np
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from oracle.seq_oracle import qk_norm_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


HALF = 2.0 ** -8


def make(B, N, Hq, Hk, Hv, d, rot, P, seed=0, weights=True, far=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    W = (Hq + Hk + Hv) * d
    t = dict(qkv=r(B, N, W).bfloat16(), dout=r(B, N, W).bfloat16())
    t["wq"], t["wk"] = (1 + 0.3 * r(d), 1 + 0.3 * r(d)) if weights else (None, None)
    ang = r(P, rot // 2) * 3 if rot else None
    t["cos"], t["sin"] = (ang.cos(), ang.sin()) if rot else (None, None)
    t["pos"] = torch.randint(0, P, (B, N), generator=g, device="cuda") if rot else None
    return t


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def kw(t, d, il=False):
    return dict(d=d, q_weight=t["wq"], k_weight=t["wk"], cos=t["cos"], sin=t["sin"], positions=t["pos"], eps=1e-6,
                interleaved=il)


def ref(t, Hq, Hk, d, il, dout=None):
    B, N, W = t["qkv"].shape
    pos = np.zeros((B, N), int) if t["pos"] is None else t["pos"].cpu().numpy()
    return qk_norm_rope(np64(t["qkv"]).reshape(B, N, -1, d), Hq, Hk, np64(t["wq"]), np64(t["wk"]), np64(t["cos"]),
                        np64(t["sin"]), pos, 1e-6, il, dout=None if dout is None else np64(dout).reshape(B, N, -1, d))


def check_out(got, want):
    got = np64(got).reshape(want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    top = np.nan_to_num(np.abs(want)).max(-1, keepdims=True)
    err = np.nan_to_num(np.abs(got - want))
    assert (err <= HALF * np.nan_to_num(np.abs(want)) + 2.0 ** -18 * top).all(), err.max()


def check_grads(t, got, Hq, Hk, d, il):
    B, N, W = t["qkv"].shape
    dx, dwq, dwk = ref(t, Hq, Hk, d, il, t["dout"])
    x, g = (np64(t[n]).reshape(B, N, -1, d) for n in ("qkv", "dout"))
    h = Hq + Hk
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    w = 1.0 if t["wq"] is None else max(np.abs(np64(t["wq"])).max(), np.abs(np64(t["wk"])).max())
    # dx = r (t - xn mean(t xn)): terms up to r |t| (1 + |xn|), |t| up to sqrt(2) max |dout| w
    mag = r * 1.5 * w * np.abs(g).max(-1, keepdims=True) * (1 + np.abs(x * r).max(-1, keepdims=True))
    got_dx = np64(got[0]).reshape(dx.shape)
    err = np.abs(got_dx - dx)[:, :, :h]
    assert (err <= HALF * np.abs(dx[:, :, :h]) + 2.0 ** -18 * mag[:, :, :h]).all()
    keep = np.ones((B, N)) if t["pos"] is None else (t["pos"].cpu().numpy() >= 0)
    assert np.array_equal(got_dx[:, :, h:], g[:, :, h:] * keep[:, :, None, None])
    tot = np.abs(g * x * r)[:, :, :h] * 1.5
    for have, want, part in ((got[1], dwq, slice(0, Hq)), (got[2], dwk, slice(Hq, h))):
        if have is None:
            continue
        # a channel's terms take the rotation partner's too: the head's largest sum bounds them
        bound = 2.0 ** -17 * tot[:, :, part].sum((0, 1, 2)).max(initial=0.0) + 1e-30
        assert np.abs(np64(have) - want).max() <= bound


SHAPES = [
    # B, N, Hq, Hk, Hv, d, rot, interleaved
    (1, 1, 1, 1, 1, 32, 32, False), (1, 1, 32, 8, 8, 128, 128, False), (2, 37, 3, 1, 2, 32, 16, True),
    (3, 65, 5, 5, 5, 64, 64, False), (1, 129, 2, 2, 0, 128, 64, True), (2, 300, 70, 70, 70, 32, 32, False),
    (1, 1000, 4, 2, 2, 64, 32, False), (1, 7, 0, 3, 1, 128, 128, True), (2, 33, 9, 3, 3, 128, 0, False),
    (1, 70, 1, 0, 0, 32, 0, False), (1, 513, 16, 4, 4, 128, 112, False),
]


@pytest.mark.parametrize("B,N,Hq,Hk,Hv,d,rot,il", SHAPES)
def test_forward_and_gradient(B, N, Hq, Hk, Hv, d, rot, il):
    t = make(B, N, Hq, Hk, Hv, d, rot, 50, seed=N)
    out = ll.lite_la_qk_norm_rope_fwd(t["qkv"], Hq, Hk, **kw(t, d, il))
    check_out(out, ref(t, Hq, Hk, d, il))
    check_grads(t, ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], Hq, Hk, **kw(t, d, il)), Hq, Hk, d, il)


def test_in_place_equals_out_of_place():
    t = make(2, 45, 6, 2, 2, 64, 64, 50)
    out = ll.lite_la_qk_norm_rope_fwd(t["qkv"], 6, 2, **kw(t, 64))
    x = t["qkv"].clone()
    assert ll.lite_la_qk_norm_rope_fwd(x, 6, 2, out=x, **kw(t, 64)) is x
    assert torch.equal(x, out)
    a = ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], 6, 2, **kw(t, 64))
    y = t["dout"].clone()
    b = ll.lite_la_qk_norm_rope_bwd(t["qkv"], y, 6, 2, dqkv=y, **kw(t, 64))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_weights_token_positions_and_int32():
    t = make(2, 40, 4, 4, 4, 32, 32, 64, weights=False)
    t["pos"] = None
    out = ll.lite_la_qk_norm_rope_fwd(t["qkv"], 4, 4, **kw(t, 32))
    dx, dwq, dwk = ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], 4, 4, **kw(t, 32))
    assert dwq is None and dwk is None
    for dtype in (torch.int32, torch.int64):
        t["pos"] = torch.arange(40, device="cuda", dtype=dtype).repeat(2, 1)
        check_out(out, ref(t, 4, 4, 32, False))
        assert torch.equal(out, ll.lite_la_qk_norm_rope_fwd(t["qkv"], 4, 4, **kw(t, 32)))
        check_grads(t, (dx, None, None), 4, 4, 32, False)


def test_padded_rows_and_positions_behind_the_table():
    t = make(2, 20, 2, 1, 1, 64, 32, 30)
    t["pos"][0, 3:] = -1
    t["pos"][1, 7] = 30
    t["pos"][1, 9] = 2 ** 40
    t["qkv"][0, 3:] = float("nan")       # what a padded row holds does not matter
    out = ll.lite_la_qk_norm_rope_fwd(t["qkv"], 2, 1, **kw(t, 64))
    q = t["qkv"].clone()
    t["qkv"][0, 3:] = 0
    want = ref(t, 2, 1, 64, False)
    check_out(out, want)
    assert not np64(out)[0, 3:].any()
    x = q.clone()
    ll.lite_la_qk_norm_rope_fwd(x, 2, 1, out=x, **kw(t, 64))
    assert torch.isnan(x[0, 3:]).all()   # left alone in place
    t["pos"][1, 7] = t["pos"][1, 9] = 1
    t["qkv"] = q
    got = ll.lite_la_qk_norm_rope_bwd(q, t["dout"], 2, 1, **kw(t, 64))
    assert not np64(got[0])[0, 3:].any() and torch.isfinite(got[1]).all() and torch.isfinite(got[2]).all()
    t["qkv"] = torch.nan_to_num(q)
    check_grads(t, got, 2, 1, 64, False)


def test_zero_rows_and_large_values():
    t = make(1, 6, 2, 2, 0, 32, 32, 50)
    t["qkv"][0, 0] = 0
    t["qkv"][0, 1] *= 1e18
    t["qkv"][0, 2] *= 1e-18
    check_out(ll.lite_la_qk_norm_rope_fwd(t["qkv"], 2, 2, **kw(t, 32)), ref(t, 2, 2, 32, False))


def test_autograd_and_equal_bits():
    t = make(2, 130, 8, 2, 2, 128, 128, 500)
    leaves = [t[n].detach().clone().requires_grad_() for n in ("qkv", "wq", "wk")]
    args = dict(d=128, cos=t["cos"], sin=t["sin"], positions=t["pos"], eps=1e-6)
    for _ in range(2):
        out = ll.lite_la_qk_norm_rope(leaves[0], 8, 2, q_weight=leaves[1], k_weight=leaves[2], **args)
        grads = torch.autograd.grad(out, leaves, t["dout"])
        want = ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], 8, 2, **kw(t, 128))
        assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # a gradient that is not contiguous
    out = ll.lite_la_qk_norm_rope(leaves[0], 8, 2, q_weight=leaves[1], k_weight=leaves[2], **args)
    g = torch.autograd.grad(out, leaves, t["dout"].transpose(0, 1).contiguous().transpose(0, 1))
    assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_other_stream_and_graph():
    t = make(2, 65, 4, 2, 2, 64, 64, 500)
    want = ll.lite_la_qk_norm_rope_fwd(t["qkv"], 4, 2, **kw(t, 64))
    want_g = ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], 4, 2, **kw(t, 64))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = ll.lite_la_qk_norm_rope_fwd(t["qkv"], 4, 2, stream=s, **kw(t, 64))
    got = ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], 4, 2, stream=s, **kw(t, 64))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got, want_g))
    graph = torch.cuda.CUDAGraph()
    x = t["qkv"].clone()
    with torch.cuda.graph(graph):
        out = ll.lite_la_qk_norm_rope_fwd(x, 4, 2, **kw(t, 64))
        got = ll.lite_la_qk_norm_rope_bwd(x, t["dout"], 4, 2, **kw(t, 64))
    for k in range(3):
        x.copy_(t["qkv"] * (1 if k < 2 else 0))
        graph.replay()
        if k < 2:
            assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got, want_g))
    assert not out[..., :6 * 64].any()


def test_empty():
    x = torch.empty(0, 5, 6 * 32, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(32, device="cuda")
    assert ll.lite_la_qk_norm_rope_fwd(x, 2, 2, q_weight=w).shape == x.shape
    dx, dwq, dwk = ll.lite_la_qk_norm_rope_bwd(x, x.clone(), 2, 2, q_weight=w, k_weight=w)
    assert not dwq.any() and not dwk.any()


def test_many_rows():
    """More rows than the gradient's grid has warps, and a row of an odd number of steps."""
    B, N, Hq, Hk, Hv, d = 1, 30011, 3, 2, 1, 64
    t = make(B, N, Hq, Hk, Hv, d, 64, 100)
    out = ll.lite_la_qk_norm_rope_fwd(t["qkv"], Hq, Hk, **kw(t, d))
    check_out(out, ref(t, Hq, Hk, d, False))
    check_grads(t, ll.lite_la_qk_norm_rope_bwd(t["qkv"], t["dout"], Hq, Hk, **kw(t, d)), Hq, Hk, d, False)
