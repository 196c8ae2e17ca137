"""What the timing of the language-model operators runs: cases, inputs, plain forms, exact forms.

Operators (see include/litela.h for the definitions):

  norm_fwd   RMS norm of every query and key head and rotation by position, on packed q|k|v rows
  norm_bwd   its gradient (dq | dk | dv and the two weights' gradients)
  delta_fwd  the gated delta rule over whole sequences, padded batch or packed, with states
  delta_step the gated delta rule's one-token form on a pool of states
  delta_train  the gated delta rule's forward and backward, as a training step calls it

`own` False: elementary torch operations in 32 bits (64 where 32 lose what matters).
`own` True: the library's calls.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64       # tokens per chunk of the plain form
DEV = "cuda"
NORM_EPS = 1e-6


# ---------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # the 4096px call's q|k|v before its linear attention: 32768 rows of 3 x 70 heads of 32
        dict(name="norm_4096px", op="norm_fwd", B=2, N=16384, Hq=70, Hk=70, Hv=70, d=32, rot=32, interleaved=False,
             far=0),
        # one new token for each of 64 sequences at far positions, grouped heads
        dict(name="norm_token_64", op="norm_fwd", B=64, N=1, Hq=32, Hk=8, Hv=8, d=128, rot=128, interleaved=False,
             far=100000),
        # a training batch of an odd length, grouped heads, all of a head rotated
        dict(name="norm_bwd_4099", op="norm_bwd", B=2, N=4099, Hq=32, Hk=8, Hv=8, d=128, rot=128, interleaved=False,
             far=0),
        # a small step with half of each head rotated in neighbouring pairs
        dict(name="norm_bwd_small", op="norm_bwd", B=1, N=517, Hq=16, Hk=16, Hv=16, d=64, rot=32, interleaved=True,
             far=0),
        # one long prompt
        dict(name="delta_long_16384", op="delta_fwd", lens="16384", packed=False, Hk=16, Hv=32, d=128, carry=False),
        # prompts of different lengths in one packed call, continued from states
        dict(name="delta_ragged_8192", op="delta_fwd", lens="4097,1,2048,777,64,1205", packed=True, Hk=8, Hv=16, d=128,
             carry=True),
        # the 1024px token count with this library's 70 heads of 32, causal
        dict(name="delta_70x32", op="delta_fwd", lens="1024,1024", packed=False, Hk=70, Hv=70, d=32, carry=False),
        # a few tokens (a short question, or drafted tokens) for each of 16 sequences
        dict(name="delta_short_16", op="delta_fwd", lens="9,3,5,17,1,8,2,30,4,7,11,6,3,1,13,5", packed=True, Hk=4,
             Hv=8, d=64, carry=True),
        # one token of one sequence: latency
        dict(name="step_1", op="delta_step", B=1, pool=4, Hk=16, Hv=32, d=128),
        # one token of each of 96 sequences: the states' bytes
        dict(name="step_96", op="delta_step", B=96, pool=100, Hk=16, Hv=32, d=128),
        # a training step, equal lengths
        dict(name="train_2x2048", op="delta_train", lens="2048,2048", packed=False, Hk=8, Hv=16, d=128, carry=False),
        # a training step, packed documents, shared key heads, half-size heads
        dict(name="train_ragged_d64", op="delta_train", lens="1500,333,64,2003,100,96", packed=True, Hk=4, Hv=16, d=64,
             carry=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total, count):
    cuts = sorted(rng.randint(0, total) for _ in range(count - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "delta_fwd", "delta_fwd", "delta_step", "delta_train"])
    d = rng.choice([32, 64, 128])
    if op in ("norm_fwd", "norm_bwd"):
        Hk = rng.choice([1, 2, 4, 8, 16, 70 if d == 32 else 12])
        Hq = Hk * rng.choice([1, 2, 4])
        rows = _log_int(rng, 1, min(32768, 2 * 10 ** 8 // ((Hq + 2 * Hk) * d)))
        B = rng.choice([1, 2, 3])
        return dict(op=op, B=B, N=max(1, rows // B), Hq=Hq, Hk=Hk, Hv=Hk, d=d,
                    rot=rng.choice([d, d // 2]), interleaved=rng.random() < 0.5, far=rng.choice([0, 0, 30000]))
    Hk = rng.choice([1, 2, 4, 8])
    Hv = Hk * rng.choice([1, 2, 4])
    if op == "delta_step":
        B = _log_int(rng, 1, 96)
        return dict(op=op, B=B, pool=B + rng.randint(0, 9), Hk=Hk, Hv=Hv, d=d)
    top = min(16384 if op == "delta_fwd" else 4096, 2 ** 19 // Hv)
    total = _log_int(rng, 16, top)
    packed = rng.random() < 0.7
    if packed:
        lens = _lens(rng, total, rng.randint(1, 9))
    else:
        B = rng.choice([1, 2, 3])
        lens = [max(1, total // B)] * B
    return dict(op=op, lens=",".join(map(str, lens)), packed=packed, Hk=Hk, Hv=Hv, d=d, carry=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _gates(g, *shape):
    """log decay of a head with its own rate, and the write strength, as such a layer's
    softplus and sigmoid give them"""
    rate = torch.rand(shape[-1:], generator=g, device=DEV) * 15 + 1
    dt = torch.exp(torch.rand(shape[-1:], generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
    bias = dt + torch.log(-torch.expm1(-dt))
    gate = -rate * torch.nn.functional.softplus(0.5 * _randn(g, *shape) + bias)
    return gate, torch.sigmoid(_randn(g, *shape))


def prepare(case, seed):
    g = _gen(seed)
    op, d = case["op"], case["d"]
    s = dict(case=case)
    if op in ("norm_fwd", "norm_bwd"):
        B, N, Hq, Hk, Hv = (case[k] for k in ("B", "N", "Hq", "Hk", "Hv"))
        heads = Hq + Hk + Hv
        s["qkv"] = _randn(g, B, N, heads * d).to(torch.bfloat16)
        s["wq"] = 1 + 0.2 * _randn(g, d)
        s["wk"] = 1 + 0.2 * _randn(g, d)
        start = int(torch.randint(0, case["far"] + 1, (1,), generator=g, device=DEV)) if case["far"] else 0
        P = start + N + 5 + B
        inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
        ang = torch.arange(P, dtype=torch.float64, device=DEV)[:, None] * inv[None]
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["pos"] = start + (torch.arange(N, device=DEV)[None] + torch.arange(B, device=DEV)[:, None])
        if op == "norm_bwd":
            s["dout"] = _randn(g, B, N, heads * d).to(torch.bfloat16)
        return s
    Hk, Hv = case["Hk"], case["Hv"]
    if op == "delta_step":
        B = case["B"]
        s["q"] = _unit(_randn(g, B, Hk, d)).to(torch.bfloat16)
        s["k"] = _unit(_randn(g, B, Hk, d)).to(torch.bfloat16)
        s["v"] = _randn(g, B, Hv, d).to(torch.bfloat16)
        s["g"], s["beta"] = _gates(g, B, Hv)
        s["states"] = 0.3 * _randn(g, case["pool"], Hv, d, d)
        s["slots"] = torch.randperm(case["pool"], generator=g, device=DEV)[:B].to(torch.int32)
        return s
    lens = [int(x) for x in case["lens"].split(",")]
    if case["packed"]:
        B, N = 1, sum(lens)
        s["cu"] = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device=DEV)
    else:
        B, N = len(lens), lens[0]
        s["cu"] = None
    s["lens"] = lens
    s["q"] = _unit(_randn(g, B, N, Hk, d)).to(torch.bfloat16)
    s["k"] = _unit(_randn(g, B, N, Hk, d)).to(torch.bfloat16)
    s["v"] = _randn(g, B, N, Hv, d).to(torch.bfloat16)
    s["g"], s["beta"] = _gates(g, B, N, Hv)
    s["state_in"] = 0.3 * _randn(g, len(lens), Hv, d, d) if case["carry"] else None
    if op == "delta_train":
        s["dout"] = _randn(g, B, N, Hv, d).to(torch.bfloat16)
        s["leaves"] = [s[n].requires_grad_() for n in ("q", "k", "v", "g", "beta")]
        if case["carry"]:
            s["leaves"].append(s["state_in"].requires_grad_())
        s["dstate"] = 0.3 * _randn(g, len(lens), Hv, d, d) if case["carry"] else None
    return s


# ---------------------------------------------------------------------------------------
# plain forms


def _rotate(x, cos, sin, rot, interleaved, back=False):
    """x [..., d] with its first `rot` channels rotated by the angles of cos, sin [..., rot / 2]"""
    if back:
        sin = -sin
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, b * cos + a * sin
    ab = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((ab, x[..., rot:]), dim=-1)


def _plain_norm(s, grad):
    c = s["case"]
    B, N, Hq, Hk, Hv, d, rot, il = (c[k] for k in ("B", "N", "Hq", "Hk", "Hv", "d", "rot", "interleaved"))
    x = s["qkv"].view(B, N, Hq + Hk + Hv, d)
    cos, sin = s["cos"][s["pos"]][:, :, None], s["sin"][s["pos"]][:, :, None]
    w = torch.cat((s["wq"].expand(Hq, d), s["wk"].expand(Hk, d)))
    qk = x[:, :, :Hq + Hk].float()
    r = torch.rsqrt((qk * qk).mean(-1, keepdim=True) + NORM_EPS)
    if not grad:
        y = _rotate(qk * r * w, cos, sin, rot, il).to(torch.bfloat16)
        return torch.cat((y, x[:, :, Hq + Hk:]), dim=2).view(B, N, -1)
    dy = s["dout"].view(B, N, Hq + Hk + Hv, d)
    t = _rotate(dy[:, :, :Hq + Hk].float(), cos, sin, rot, il, back=True)
    xn = qk * r
    dw = (t * xn).sum((0, 1), dtype=torch.float64)
    t = t * w
    dx = r * (t - xn * (t * xn).mean(-1, keepdim=True))
    dqkv = torch.cat((dx.to(torch.bfloat16), dy[:, :, Hq + Hk:]), dim=2).view(B, N, -1)
    return dqkv, dw[:Hq].sum(0).float(), dw[Hq:].sum(0).float()


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular A [..., n, n], n a power of two: inverses of the
    diagonal blocks of 1, 2, 4, ... rows, [[X, 0], [Y, Z]]^-1 = [[X', 0], [-Z' Y X', Z']]"""
    n = A.shape[-1]
    inv = torch.ones(A.shape[:-2] + (n, 1, 1), dtype=A.dtype, device=A.device)
    size = 1
    while size < n:
        m = n // (2 * size)
        blocks = A.unflatten(-1, (m, 2 * size)).unflatten(-3, (m, 2 * size))       # [.., m, 2s, m, 2s]
        i = torch.arange(m, device=A.device)
        low = blocks.movedim(-2, -3)[..., i, i, size:, :size]                        # [.., m, s, s]
        x, z = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        y = -(z @ low @ x)
        inv = torch.cat((torch.cat((x, torch.zeros_like(y)), -1), torch.cat((y, z), -1)), -2)
        size *= 2
    return inv[..., 0, :, :]


def _padded(s):
    """index [S, L] of each sequence's tokens in the flattened rows, and the truth of being one"""
    lens = s["lens"]
    L = max(1, -(-max(lens) // CHUNK)) * CHUNK
    n = torch.tensor(lens, device=DEV)[:, None]
    at = torch.arange(L, device=DEV)[None]
    first = torch.tensor(np.cumsum([0] + lens[:-1]), device=DEV)[:, None]
    real = at < n
    return torch.where(real, first + at, 0), real


def _plain_delta(s, q, k, v, g, beta, state):
    """out in v's layout, and the last states"""
    c = s["case"]
    Hk, Hv, d = c["Hk"], c["Hv"], c["d"]
    index, real = _padded(s)
    S, L = index.shape
    nc = L // CHUNK
    keep = real[:, :, None]

    def rows(x):   # [S, L, H, ...], zero behind a sequence's end
        y = x.flatten(0, 1)[index]
        return torch.where(keep if y.dim() == 3 else keep[..., None], y, torch.zeros((), dtype=y.dtype, device=DEV))

    def chunks(x):   # [S, H, nc, CHUNK, ...]
        return x.unflatten(1, (nc, CHUNK)).movedim(3, 1)

    Q, K = (chunks(rows(x.float()).repeat_interleave(Hv // Hk, dim=2)) for x in (q, k))
    V, G, Bt = (chunks(rows(x.float())) for x in (v, g, beta))
    G = G.double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    to_end, G = torch.exp(G[..., -1:] - G).float(), torch.exp(G).float()
    A = (Bt[..., None] * (K @ K.transpose(-1, -2)) * D).tril(-1)
    P = (Q @ K.transpose(-1, -2)) * D * d ** -0.5
    T = _unit_lower_inverse(A)
    U0, W = T @ (Bt[..., None] * V), T @ ((Bt * G)[..., None] * K)
    Qs, Ke = Q * (G * d ** -0.5)[..., None], K * to_end[..., None]
    state = torch.zeros(S, Hv, d, d, device=DEV) if state is None else state
    outs = []
    for i in range(nc):
        u = U0[:, :, i] - W[:, :, i] @ state
        outs.append(Qs[:, :, i] @ state + P[:, :, i] @ u)
        state = G[:, :, i, -1, None, None] * state + Ke[:, :, i].transpose(-1, -2) @ u
    out = torch.stack(outs, 2).movedim(1, 3).flatten(1, 2)    # [S, L, Hv, d]
    return out[real].to(torch.bfloat16).view(v.shape), state


def _plain_step(s):
    c = s["case"]
    group = c["Hv"] // c["Hk"]
    q, k = (s[n].float().repeat_interleave(group, dim=1) for n in ("q", "k"))
    slots = s["slots"].long()
    state = s["states"][slots] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (state * k[..., None]).sum(-2))
    state = state + k[..., None] * u[..., None, :]
    out = (state * q[..., None]).sum(-2) * c["d"] ** -0.5
    s["states"][slots] = state
    return out.to(torch.bfloat16), s["states"]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _own(s)
    if op in ("norm_fwd", "norm_bwd"):
        return _plain_norm(s, op == "norm_bwd")
    if op == "delta_step":
        return _plain_step(s)
    out, state = _plain_delta(s, s["q"], s["k"], s["v"], s["g"], s["beta"], s["state_in"])
    if op == "delta_fwd":
        return out, state
    return _grads(s, out, state)


def _grads(s, out, state):
    if s["dstate"] is None:
        grads = torch.autograd.grad(out, s["leaves"], s["dout"])
    else:
        grads = torch.autograd.grad((out, state), s["leaves"], (s["dout"], s["dstate"]))
    return (out.detach(), state.detach()) + tuple(grads)


# ---------------------------------------------------------------------------------------
# the library's calls


def _own(s):
    import linear_attention_diffusion_litela_b200 as ll
    c = s["case"]
    op = c["op"]
    if op in ("norm_fwd", "norm_bwd"):
        args = dict(d=c["d"], q_weight=s["wq"], k_weight=s["wk"], cos=s["cos"], sin=s["sin"], positions=s["pos"],
                    eps=NORM_EPS, interleaved=c["interleaved"])
        if op == "norm_fwd":
            return ll.lite_la_qk_norm_rope_fwd(s["qkv"], c["Hq"], c["Hk"], **args)
        return ll.lite_la_qk_norm_rope_bwd(s["qkv"], s["dout"], c["Hq"], c["Hk"], **args)
    if op == "delta_step":
        out = ll.lite_la_gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["states"],
                                          state_indices=s["slots"])
        return out, s["states"]
    if op == "delta_fwd":
        return ll.lite_la_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], state_in=s["state_in"],
                                          cu_seqlens=s["cu"])
    out, state = ll.lite_la_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], state_in=s["state_in"],
                                        cu_seqlens=s["cu"])
    return _grads(s, out, state)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c, d = case, case["d"]
    if c["op"] in ("norm_fwd", "norm_bwd"):
        rows, qk, v = c["B"] * c["N"], (c["Hq"] + c["Hk"]) * d, c["Hv"] * d
        table = rows * (c["rot"] * 4 + 8)
        if c["op"] == "norm_fwd":
            return dict(bytes=rows * 2 * (qk + v) * 2 + table + 8 * d, flops=rows * qk * 8)
        return dict(bytes=rows * 2 * (3 * qk + 2 * v) + table + 16 * d, flops=rows * qk * 18)
    Hk, Hv = c["Hk"], c["Hv"]
    token = 2 * d * (2 * Hk + 2 * Hv) + 8 * Hv      # q, k, v, out; g, beta
    state = Hv * d * d * 4
    if c["op"] == "delta_step":
        return dict(bytes=c["B"] * (token + 2 * state + 4), flops=c["B"] * Hv * 7 * d * d)
    lens = [int(x) for x in c["lens"].split(",")]
    n = sum(lens)
    carried = 2 if c["carry"] else 1
    if c["op"] == "delta_fwd":
        return dict(bytes=n * token + len(lens) * state * carried, flops=n * Hv * 6 * d * d)
    # forward as above; backward: q, k, v, dout, g, beta in, their gradients out
    back = n * (2 * d * (2 * Hk + 2 * Hv) + 8 * Hv + 2 * d * (2 * Hk + Hv) + 8 * Hv)
    return dict(bytes=n * token + back + len(lens) * state * (2 * carried), flops=n * Hv * 20 * d * d)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, token by token


def _exact_norm(s, grad):
    c = s["case"]
    B, N, Hq, Hk, Hv, d, rot, il = (c[k] for k in ("B", "N", "Hq", "Hk", "Hv", "d", "rot", "interleaved"))
    heads = Hq + Hk
    x = s["qkv"].double().view(B, N, -1, d)
    lo = torch.arange(0, rot, 2, device=DEV) if il else torch.arange(rot // 2, device=DEV)
    hi = lo + 1 if il else lo + rot // 2
    turn = torch.complex(s["cos"][s["pos"]].double(), s["sin"][s["pos"]].double())[:, :, None]
    w = [s["wq"].double()] * Hq + [s["wk"].double()] * Hk
    w = torch.stack(w)
    a = x[:, :, :heads]
    mean = a.pow(2).sum(-1, keepdim=True) / d + NORM_EPS
    if not grad:
        y = a / mean.sqrt() * w
        z = torch.complex(y[..., lo], y[..., hi]) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        return torch.cat((y, x[:, :, heads:]), 2).view(B, N, -1)
    dy = s["dout"].double().view(B, N, -1, d)
    t = dy[:, :, :heads].clone()
    z = torch.complex(t[..., lo], t[..., hi]) * turn.conj()
    t[..., lo], t[..., hi] = z.real, z.imag
    dwh = (t * a / mean.sqrt()).sum((0, 1))
    t = t * w
    dx = t / mean.sqrt() - a * (t * a).sum(-1, keepdim=True) / (d * mean.pow(1.5))
    return torch.cat((dx, dy[:, :, heads:]), 2).view(B, N, -1), dwh[:Hq].sum(0), dwh[Hq:].sum(0)


def _exact_delta(s, grad):
    """The recurrence S <- e^g S + k (beta (v - e^g S^T k))^T, out = S^T q / sqrt(d), and its
    derivative by the chain rule, one token after another for all sequences and heads."""
    c = s["case"]
    Hk, Hv, d = c["Hk"], c["Hv"], c["d"]
    group, lens = Hv // Hk, s["lens"]
    S, L = len(lens), max(lens)
    scale = 1.0 / math.sqrt(d)

    def by_time(x):   # [L, S, H, ...] in 64 bits; zeros behind a sequence's end
        flat = x.detach().double().flatten(0, 1)
        y = torch.zeros((L, S) + flat.shape[1:], dtype=torch.float64, device=DEV)
        at = 0
        for i, n in enumerate(lens):
            y[:n, i] = flat[at:at + n]
            at += n
        return y

    def back(y, like):
        return torch.cat([y[:n, i] for i, n in enumerate(lens)]).view(like.shape)

    q, k = (by_time(s[n]).repeat_interleave(group, 2) for n in ("q", "k"))
    v, g, beta = (by_time(s[n]) for n in ("v", "g", "beta"))
    alpha = g.exp()
    state = torch.zeros(S, Hv, d, d, dtype=torch.float64, device=DEV) if s["state_in"] is None \
        else s["state_in"].detach().double()
    out = torch.empty_like(v)
    errs, before = torch.empty_like(v), []
    for t in range(L):
        if grad:
            before.append(state)
        decayed = alpha[t][..., None, None] * state
        err = v[t] - torch.einsum("shij,shi->shj", decayed, k[t])
        errs[t] = err
        state = decayed + torch.einsum("shi,shj->shij", k[t], beta[t][..., None] * err)
        out[t] = scale * torch.einsum("shij,shi->shj", state, q[t])
    if not grad:
        return back(out, s["v"]), state
    last = state
    do = by_time(s["dout"])
    G = torch.zeros_like(last) if s["dstate"] is None else s["dstate"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    for t in reversed(range(L)):
        now = before[t + 1] if t + 1 < L else last
        dq[t] = scale * torch.einsum("shij,shj->shi", now, do[t])
        G = G + scale * torch.einsum("shi,shj->shij", q[t], do[t])
        u = beta[t][..., None] * errs[t]
        du = torch.einsum("shij,shi->shj", G, k[t])
        dk[t] = torch.einsum("shij,shj->shi", G, u)
        db[t] = (du * errs[t]).sum(-1)
        de = beta[t][..., None] * du
        dv[t] = de
        decayed = alpha[t][..., None, None] * before[t]
        dk[t] -= torch.einsum("shij,shj->shi", decayed, de)
        G = G - torch.einsum("shi,shj->shij", k[t], de)
        dg[t] = (G * decayed).sum((-1, -2))
        G = alpha[t][..., None, None] * G
    share = lambda x: x.unflatten(2, (Hk, group)).sum(3)  # noqa: E731
    grads = [back(share(dq), s["q"]), back(share(dk), s["k"]), back(dv, s["v"]), back(dg, s["g"]),
             back(db, s["beta"])]
    if c["carry"]:
        grads.append(G)
    return (back(out, s["v"]), last) + tuple(grads)


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        op = case["op"]
        if op in ("norm_fwd", "norm_bwd"):
            return _exact_norm(s, op == "norm_bwd")
        if op == "delta_step":
            group = case["Hv"] // case["Hk"]
            q, k = (s[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
            states = s["states"].double()
            slots = s["slots"].long()
            old = states[slots] * s["g"].double().exp()[..., None, None]
            u = s["beta"].double()[..., None] * (s["v"].double() - torch.einsum("bhij,bhi->bhj", old, k))
            new = old + torch.einsum("bhi,bhj->bhij", k, u)
            states[slots] = new
            return torch.einsum("bhij,bhi->bhj", new, q) / math.sqrt(case["d"]), states
        return _exact_delta(s, op == "delta_train")
