"""How exact the fp32 results of the gated delta rule are: as exact as plain fp32 operations would be, so that
no operand is left in two bf16 terms (2^-17).

Tolerances.  2-norms of the difference to 64 bits over the result's.  An fp32 operand of a product enters in
terms that leave 2^-25 of it, both operands together 2^-24; the products are added in fp32 up to 128 at a
time, in blocks of 16, so 8 roundings (or cuts, 2^-23) of a partial sum that is at most the sum's own size on
the average: sqrt(8) 2^-23 < 2^-21.5 if each lost its most, and half of that (2^-22.5) as they fall.  Three
products follow one another in a chunk, and one operand (X) is a result of up to three small ones: errors add
up as squares, sqrt(6) 2^-22.5 < 2^-21.2.  What a chunk hands on decays and is overwritten, so that a state's
error stays the size of its newest parts': 2^-21 in all.  Two terms leave 2^-18 of an operand at random, 2^-20
and more of a result."""
import numpy as np
import pytest
import torch

import linear_attention_diffusion_litela_b200 as ll
from tests.test_gpu_delta import fwd, make, np64, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_diffusion_litela_b200.build import build
    build()


STATE = 2.0 ** -21
CASES = [  # lens, packed, Hk, Hv, d, carry
    ([208, 208], False, 2, 4, 32, False), ([600], False, 4, 8, 32, True), ([64, 90, 33, 200], True, 2, 4, 64, True),
    ([333], False, 2, 4, 64, False), ([150, 64], True, 2, 4, 128, False), ([400], False, 1, 4, 128, True),
]


def off(got, want):
    return np.linalg.norm(np64(got) - want) / max(np.linalg.norm(want), 1e-30)


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", CASES)
@pytest.mark.parametrize("rate", [1.0, 0.1])
def test_states(lens, packed, Hk, Hv, d, carry, rate):
    t = make(lens, packed, Hk, Hv, d, carry, seed=sum(lens) + d, rate=rate)
    _, state = fwd(t)
    ll.lite_la_device_status()
    far = [off(state[i], S) for i, _, _, (_, S) in ref(t)]
    assert max(far) <= STATE, far


# dbeta_i = w_i . W_i: the gradient of what a token writes and what the state before it got wrong, each a result
# of three products like a state's: sqrt(2) 2^-21, and of a dot product of signed terms again 2^-21 of their norms
DBETA = 2.0 ** -20


def gradients(t):
    """dstate_in, dbeta and dg of every sequence as (how far off, over the result's norm)"""
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    kw = dict(state_in=t["state_in"], cu_seqlens=t["cu"])
    _, _, saved = ll.lite_la_gated_delta_fwd_save(*args, **kw)
    got = ll.lite_la_gated_delta_bwd(*args, t["dout"], saved, dstate_out=t["dstate"], **kw)
    ll.lite_la_device_status()
    far = dict(dstate=[], dbeta=[], dg=[])
    for i, e, sl, (_, _, (_, _, _, dg, db, dS)) in ref(t, grads=True):
        if t["state_in"] is not None:
            far["dstate"].append(off(got[5][i], dS))
        far["dbeta"].append(off(got[4][e, sl], db))
        far["dg"].append(off(got[3][e, sl], dg))
    return far


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", CASES)
@pytest.mark.parametrize("rate", [1.0, 0.1])
def test_gradients_of_states_and_write_strengths(lens, packed, Hk, Hv, d, carry, rate):
    far = gradients(make(lens, packed, Hk, Hv, d, carry, seed=sum(lens) + d, rate=rate))
    assert max(far["dstate"], default=0.0) <= STATE and max(far["dbeta"]) <= DBETA, far


# dg_t = <G, A>, the state that decays and its gradient, each 2^-21 off at random: sqrt(2) 2^-21 of it.  It comes
# from sums over the 64 tokens of a chunk of terms that are up to a few times dg: 64 roundings of 2^-24 of them
# add up to 8 2^-24 times three, 2^-19.4 if all were at their most, a quarter of that as they fall: 2^-20.2 together
DG = 2.0 ** -20


@pytest.mark.parametrize("lens,packed,Hk,Hv,d,carry", CASES)
@pytest.mark.parametrize("rate", [1.0, 0.1])
def test_gradients_of_decays(lens, packed, Hk, Hv, d, carry, rate):
    far = gradients(make(lens, packed, Hk, Hv, d, carry, seed=sum(lens) + d + 1, rate=rate))
    assert max(far["dg"]) <= DG, far
