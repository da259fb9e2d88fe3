"""GPU parity of the routing's balance loss, per-expert counts and logit gradients (moe_balance,
moe_route_backward) through the C ABI, against the float64 oracle.

Tolerances, in roundings of u = 2^-24.  Counts and tokens are equal.  A probability's exponent x (l - m, or
l itself where the row's largest logit lies in [-16, 16]) is off by the difference, its product with
log2 e and that constant: 2.3 u |x| of p, 92 u for |x| <= 40, and the exponential, the sum and the reciprocal
add under 32 u: 2^-17 of p; what lies further down is under 1e-17 of the row (e^-40).  A loss adds, in any
chain, the tokens of a lane (a chunk's, at most max(64, T / 512), over at least 16 groups: 9), 6 + 16 over
lanes and waves, at most 512 / 16 + 1 pieces, 16 + 6 and the sequences' few dozen: under 110 u beside p's
128: 2^-16 for T <= 70000.  (test_long_batch: chunks grow from 32768 tokens on, so that there are at most
512.)  z = m + log(sum): 17 u for the sum and 4 u (|m| + |z|): under 2^-21 (|m| + |z| + 1) + 9 u each, the
latter within the loss's 2^-16 z^2.  A gradient's terms carry 2^-17 from p three times and under 64
roundings: 2^-15 of their magnitudes, then the output's own rounding.
"""
import numpy as np
import pytest
import torch

import oracle.block_oracle as O
from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def make(T, E, k, seq, seed=0, lost=0.05, masked=0.05, spread=1.5):
    """logits (bf16), ids with unrouted slots, gates, dgates; some experts masked for some tokens, some
    tokens with a NaN (unrouted) or without any logit."""
    r = np.random.default_rng(np.random.SeedSequence(30, spawn_key=(T, E, k, seed)))
    l = r.normal(size=(T, E)) * spread + r.normal(size=E)
    l[r.random((T, E)) < masked] = -np.inf
    lb = torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16)
    l = lb.float().numpy().astype(np.float64)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    ids[r.random((T, k)) < lost] = -1
    ids[r.random((T, k)) < lost / 4] = E + 3
    for t in range(T):
        if r.random() < lost:
            l[t, r.integers(E)] = np.nan
            ids[t] = -1
        elif r.random() < lost / 2:
            l[t] = -np.inf
    gates = r.random((T, k)).astype(np.float32)
    gates /= gates.sum(1, keepdims=True)
    gates[(ids < 0) | (ids >= E)] = 0.0
    dgates = r.normal(size=(T, k)).astype(np.float32)
    dgates[(ids < 0) | (ids >= E)] = np.nan        # whatever stands there
    return dict(T=T, E=E, k=k, l=l, ids=ids, gates=gates, dgates=dgates,
                seq=np.asarray(seq if seq is not None else [0, T], np.int32), given=seq is not None,
                logits=torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16).cuda())


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run_balance(c):
    S = len(c["seq"]) - 1
    counts = torch.full((S, c["E"]), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((S + 2,), -7, dtype=torch.int32, device="cuda")
    losses = torch.full((2,), float("nan"), device="cuda")
    ws = torch.full((B.moe_balance_workspace_size(c["T"], c["E"], S),), 255, dtype=torch.uint8, device="cuda")
    B.moe_balance(c["logits"], cuda(c["ids"]), c["T"], c["E"], c["k"], counts, tokens, losses,
                  seq_offsets=cuda(c["seq"]) if c["given"] else None, S=S, workspace=ws)
    return counts, tokens, losses


def z_bound(c):
    live = [t for t, s in enumerate(O.counted(c["l"], c["ids"], c["seq"])) if s is not None]
    if not live:
        return 0.0
    z = np.array([O.softmax(c["l"][t])[1] for t in live])
    m = np.array([np.abs(c["l"][t].max()) for t in live])
    return float(np.mean(2 * np.abs(z) * 2.0 ** -21 * (m + np.abs(z) + 1)) + 2.0 ** -16 * np.mean(z * z))


def check_balance(c):
    counts, tokens, losses = run_balance(c)
    wc, wt, wl = O.balance(c["l"], c["ids"], c["seq"])
    np.testing.assert_array_equal(counts.cpu().numpy(), wc)
    np.testing.assert_array_equal(tokens.cpu().numpy(), wt)
    g = losses.double().cpu().numpy()
    assert abs(g[0] - wl[0]) <= 2.0 ** -16 * wl[0], (g, wl)
    assert abs(g[1] - wl[1]) <= z_bound(c), (g, wl, z_bound(c))
    return counts, tokens, losses


# T, E, k, sequences (None: the whole batch)
CASES = [
    (1, 1, 1, None), (1, 32, 4, None), (5, 7, 3, None), (64, 32, 4, None), (65, 32, 4, [0, 65]), (300, 8, 8, None),
    (129, 9, 2, [0, 0, 64, 64, 65, 129]),        # empty sequences, borders on and behind a 64-token chunk
    (200, 33, 5, [3, 50, 51, 190]),              # padding in front and behind
    (97, 64, 6, None), (70, 65, 6, [0, 70]), (150, 100, 32, [0, 10, 150]), (90, 128, 8, [0, 30, 60, 90]),
    (80, 200, 4, None), (130, 256, 8, [0, 128, 130]), (70, 500, 8, [0, 1, 2, 3, 70]), (140, 512, 8, [0, 140]),
    (140, 511, 3, [5, 5, 5]),                    # nothing in any sequence
    (256, 2, 1, list(range(257))),               # one token each
    (3000, 32, 4, [0, 1000, 1000, 2900]),
]


@pytest.mark.parametrize("T,E,k,seq", CASES)
def test_balance(T, E, k, seq):
    _announce(f"balance T={T} E={E} k={k} S={1 if seq is None else len(seq) - 1}")
    check_balance(make(T, E, k, seq))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gates,losses", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("T,E,k,seq", CASES)
def test_route_backward(T, E, k, seq, gates, losses, dtype):
    _announce(f"route_backward T={T} E={E} k={k} gates={gates} losses={losses} {dtype}")
    c = make(T, E, k, seq, seed=1)
    S = len(c["seq"]) - 1
    dl = np.array([0.7 * T, 0.2 * T], np.float32) if losses else None
    dlogits = torch.full((T, E), float("nan"), dtype=dtype, device="cuda")
    more = {}
    if losses:
        counts, tokens, _ = run_balance(c)
        more = dict(seq_offsets=cuda(c["seq"]) if c["given"] else None, S=S, counts=counts, tokens=tokens,
                    dlosses=cuda(dl))
    B.moe_route_backward(c["logits"] if losses else None, cuda(c["ids"]), cuda(c["gates"]) if gates else None,
                         cuda(c["dgates"]) if gates else None, T, E, k, dlogits, **more)
    want, mag = O.route_backward(c["l"], c["ids"], c["gates"], c["dgates"] if gates else None, c["seq"], dl)
    g = dlogits.double().cpu().numpy()
    bound = HALF[dtype] * np.abs(want) * 1.01 + 2.0 ** -15 * mag + 1e-15
    bad = np.argwhere(~(np.abs(g - want) <= bound))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), float(np.nanmax(np.abs(g - want) / bound)))


def test_lowest_value_masks():
    """Experts masked with the type's lowest value: no probability, no gradient; a token whose every
    logit is the lowest value keeps even probabilities."""
    _announce("lowest-value masks")
    low = float(torch.finfo(torch.bfloat16).min)
    T, E, k = 70, 32, 4
    c = make(T, E, k, None, seed=2, lost=0.0, masked=0.0)
    c["l"][:, 20:] = low
    c["l"][3] = low
    c["logits"] = torch.from_numpy(c["l"].astype(np.float32)).to(torch.bfloat16).cuda()
    c["ids"] = np.argsort(-c["l"], axis=1, kind="stable")[:, :k].astype(np.int32)
    counts, tokens, losses = run_balance(c)
    wc, _, wl = O.balance(c["l"], c["ids"], c["seq"])
    np.testing.assert_array_equal(counts.cpu().numpy(), wc)
    assert abs(float(losses[0]) - wl[0]) <= 2.0 ** -16 * wl[0]
    assert float(losses[1]) == float("inf")       # the square of the lowest value passes fp32's range
    d = torch.full((T, E), float("nan"), device="cuda")
    dl = np.array([float(T), 0.0], np.float32)
    B.moe_route_backward(c["logits"], cuda(c["ids"]), None, None, T, E, k, d, counts=counts, tokens=tokens,
                         dlosses=cuda(dl))
    want, mag = O.route_backward(c["l"], c["ids"], None, None, c["seq"], dl)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= 2.0 ** -15 * mag + 1e-15)


def test_even_load_has_no_balance_gradient():
    """Each expert chosen equally often: the counts' differences from their mean are exactly 0."""
    _announce("even load")
    T, E, k = 64, 8, 2
    c = make(T, E, k, None, seed=3, lost=0.0, masked=0.0)
    c["ids"] = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)], np.int32)
    counts, tokens, _ = check_balance(c)
    d = torch.full((T, E), float("nan"), device="cuda")
    B.moe_route_backward(c["logits"], cuda(c["ids"]), None, None, T, E, k, d, counts=counts, tokens=tokens,
                         dlosses=cuda(np.array([100.0, 0.0], np.float32)))
    assert not d.any()


def test_repeated_expert_in_a_token():
    _announce("the same expert twice")
    T, E, k = 20, 16, 3
    c = make(T, E, k, None, seed=4, lost=0.0)
    c["ids"][:, 2] = c["ids"][:, 0]
    check_balance(c)
    d = torch.full((T, E), float("nan"), device="cuda")
    B.moe_route_backward(None, cuda(c["ids"]), cuda(c["gates"]), cuda(c["dgates"]), T, E, k, d)
    want, mag = O.route_backward(c["l"], c["ids"], c["gates"], c["dgates"], None, None)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= 2.0 ** -16 * mag + 1e-30)


def test_no_tokens():
    _announce("no tokens")
    c = dict(T=0, E=32, k=4, l=np.zeros((0, 32)), ids=np.zeros((0, 4), np.int32), seq=np.array([0, 0, 0], np.int32),
             given=True, logits=torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"))
    counts, tokens, losses = run_balance(c)
    assert not counts.any() and not tokens.any() and not losses.any()


def test_offsets_outside_are_clamped():
    """Sequence borders before 0 and behind T: as if clamped."""
    _announce("offsets outside")
    c = make(100, 32, 4, [-5, 40, 1 << 30], seed=5)
    counts, tokens, losses = run_balance(c)
    wc, wt, wl = O.balance(c["l"], c["ids"], [0, 40, 100])
    np.testing.assert_array_equal(counts.cpu().numpy(), wc)
    np.testing.assert_array_equal(tokens.cpu().numpy(), wt)
    assert abs(float(losses[0]) - wl[0]) <= 2.0 ** -16 * wl[0]


def test_long_batch():
    """More than 1024 chunks of 64 tokens: chunks grow with the batch."""
    _announce("balance, 70000 tokens")
    T, E, k = 70000, 8, 2
    c = make(T, E, k, [0, 30000, 69999], seed=6)
    counts, tokens, _ = check_balance(c)
    d = torch.full((T, E), float("nan"), device="cuda")
    dl = np.array([0.7 * T, 0.2 * T], np.float32)
    B.moe_route_backward(c["logits"], cuda(c["ids"]), cuda(c["gates"]), cuda(c["dgates"]), T, E, k, d,
                         seq_offsets=cuda(c["seq"]), S=2, counts=counts, tokens=tokens, dlosses=cuda(dl))
    want, mag = O.route_backward(c["l"], c["ids"], c["gates"], c["dgates"], c["seq"], dl)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= 2.0 ** -23 * np.abs(want) + 2.0 ** -15 * mag + 1e-15)


def test_binding_checks():
    _announce("balance binding checks")
    l = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="tokens holds"):
        B.moe_balance(l, i(4, 2), 4, 8, 2, i(1, 8), i(2), f(2), workspace=ws)
    with pytest.raises(ValueError, match="seq_offsets holds"):
        B.moe_balance(l, i(4, 2), 4, 8, 2, i(2, 8), i(4), f(2), seq_offsets=i(2), S=2, workspace=ws)
    with pytest.raises(TypeError):
        B.moe_balance(l.float(), i(4, 2), 4, 8, 2, i(1, 8), i(3), f(2), workspace=ws)
    with pytest.raises(B.MXFP4Error, match="workspace"):
        B.moe_balance(l, i(4, 2), 4, 8, 2, i(1, 8), i(3), f(2))
    with pytest.raises(TypeError):
        B.moe_route_backward(None, i(4, 2), f(4, 2), f(4, 2), 4, 8, 2, l.half())
    torch.cuda.synchronize()
