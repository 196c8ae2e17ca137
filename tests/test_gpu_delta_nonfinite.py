"""A NaN or an infinity in a token's inputs leaves the outputs of earlier tokens as they are, bit for bit,
and reaches all later ones and the state: at every place of a chunk, in both forms of the gated delta rule
(up to 32 tokens the recurrence, more in chunks of 64).  Sequence i of a call has its bad token at place
first + i; the others' values are those of a call without any."""
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from tests.test_gpu_delta import fwd, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


NAN, INF = float("nan"), float("inf")
SIZES = [(32, 0, 32), (64, 0, 64), (150, 0, 64), (150, 64, 64), (150, 128, 22)]   # tokens, first place, places


def check(name, value, d, N, first, count, channel=None):
    """`channel`: only this one of the token's is bad, and only its outputs have to show it"""
    t = make([N] * count, False, 1, 2, d, True, seed=N + first + d)
    want, _ = fwd(t)
    t[name] = t[name].clone()
    for i in range(count):
        if channel is None:
            t[name][i, first + i] = value
        else:
            t[name][i, first + i, :, channel] = value
    out, state = fwd(t)
    ll.lite_la_device_status()
    seen = slice(None) if channel is None or name == "k" else channel
    before = torch.arange(N, device="cuda")[None] < first + torch.arange(count, device="cuda")[:, None]
    same = (out == want).flatten(2).all(-1)
    wrong = (before & ~same).nonzero().tolist()
    assert not wrong, "earlier tokens of (sequence, token) %s differ" % wrong[:8]
    assert not torch.isfinite(out[..., seen]).flatten(2).any(-1)[~before].any()
    assert not torch.isfinite(state[..., seen]).any()


@pytest.mark.parametrize("N,first,count", SIZES)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("name,value,channel", [("k", NAN, None), ("k", INF, 3), ("v", NAN, None), ("v", -INF, 17)])
def test_keys_and_values(name, value, channel, d, N, first, count):
    check(name, value, d, N, first, count, channel)


@pytest.mark.parametrize("N,first,count", SIZES)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_write_strengths(value, d, N, first, count):
    check("beta", value, d, N, first, count)


@pytest.mark.parametrize("N,first,count", SIZES)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("value", [NAN, INF])
def test_decays(value, d, N, first, count):
    check("g", value, d, N, first, count)


@pytest.mark.parametrize("N,first,count", SIZES)
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("value", [NAN, INF])
def test_queries(value, d, N, first, count):
    """A bad query shows in its own token's outputs at least, and in no earlier ones"""
    t = make([N] * count, False, 1, 2, d, True, seed=N + first + d)
    want, _ = fwd(t)
    t["q"] = t["q"].clone()
    at = first + torch.arange(count, device="cuda")
    t["q"][torch.arange(count, device="cuda"), at, :, 5] = value
    out, _ = fwd(t)
    before = torch.arange(N, device="cuda")[None] < at[:, None]
    assert (out == want).flatten(2).all(-1)[before].all()
    assert not torch.isfinite(out[torch.arange(count, device="cuda"), at]).any()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("N", [20, 150])
def test_a_state_before_the_sequence(N, d):
    """A bad element of state_in: its value channel in all tokens, and no other sequence"""
    t = make([N] * 3, False, 1, 2, d, True, seed=N + d)
    want, want_s = fwd(t)
    t["state_in"][1, 1, 4, 9] = NAN
    out, state = fwd(t)
    assert torch.equal(out[[0, 2]], want[[0, 2]]) and torch.equal(state[[0, 2]], want_s[[0, 2]])
    assert torch.equal(out[1, :, 0], want[1, :, 0]) and torch.equal(state[1, 0], want_s[1, 0])
    assert not torch.isfinite(out[1, :, 1, 9]).any() and not torch.isfinite(state[1, 1, :, 9]).any()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("name,value", [("k", NAN), ("v", INF), ("g", NAN), ("beta", INF), ("q", NAN)])
def test_the_forward_of_a_training_step(name, value, d):
    """It keeps to the same: the same bits as the forward alone, bad tokens and all"""
    t = make([150] * 64, False, 1, 2, d, True, seed=d)
    at = torch.arange(64, device="cuda")
    t[name][at, 64 + at] = value
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    out, state, _ = ll.lite_la_gated_delta_fwd_save(*args, state_in=t["state_in"])
    want, want_s = fwd(t)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.equal(state.isnan(), want_s.isnan()) and torch.equal(state.nan_to_num(), want_s.nan_to_num())


@pytest.mark.parametrize("name", ["k", "v", "g", "beta", "q", "dout"])
def test_gradients_of_other_sequences(name):
    """A bad token leaves the gradients of all other sequences as they are, bit for bit"""
    t = make([100, 70, 64], True, 2, 4, 64, True, seed=3)

    def grads():
        args = [t[n] for n in ("q", "k", "v", "g", "beta")]
        kw = dict(state_in=t["state_in"], cu_seqlens=t["cu"])
        _, _, saved = ll.lite_la_gated_delta_fwd_save(*args, **kw)
        got = ll.lite_la_gated_delta_bwd(*args, t["dout"], saved, dstate_out=t["dstate"], **kw)
        ll.lite_la_device_status()
        return got

    want = grads()
    t[name][0, 120] = NAN
    got = grads()
    for a, b in zip(got[:5], want[:5]):
        assert torch.equal(a[:, :100], b[:, :100]) and torch.equal(a[:, 170:], b[:, 170:])
    assert torch.equal(got[5][[0, 2]], want[5][[0, 2]])
