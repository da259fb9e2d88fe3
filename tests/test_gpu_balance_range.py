"""The routing's balance and the logits' gradient over the whole range that their arguments may have:
logits of any finite size, and what tokens beside a counted one hold.  Against the float64 oracle, or
bit for bit.

Tolerances, from the kernels' arithmetic (u = 2^-24, half a step of fp32).  A probability is
exp2(x log2 e) / sum with x = l - m and m the row's maximum, or x = l while the maximum is small (at
most 16 in size).  Its exponent is off by the roundings of l - m, of the product and of the constant: at
most 2.3 u |x| of p, and |x| <= 87 where p has not vanished: 2^-16.2 of p; exp2, the sum over at most
512 experts in chains of 8 + 6 and the reciprocal add under 20 u.  So p is within 2^-16.
 - loss: p's error, and roundings of sums of one sign: at most 64 tokens in a lane's chain, 6 + 16 over
   the lanes and waves, 32 + 16 + 6 and the sequences' in the later launches, under 200 u in all:
   2^-15.2 of the loss, stated as 2^-15;
 - z = m + ln(sum): 2^-17 for the sum's own error, and 4 u (|m| + |z|);
 - a gradient: p once (2^-16), sums of p (within 2^-19 of their magnitudes, since far logits hardly
   weigh), under 40 more roundings, and z's error times 2 dz / n: 2^-15 of the magnitudes, plus the
   latter; then the output's own rounding.  fp32's least normal number is 2^-126: an exponential
   below it may come out as 0.  The sum is at least 1 with x = l - m and at least e^-16 with x = l, so
   p loses less than 2^-126 e^16 < 2^-102, and the gradient that times p's factor.
"""
import numpy as np
import pytest
import torch

import oracle.block_oracle as O
from mxfp4_mixture_experts_amd import binding as B
from test_gpu_balance import _announce, cuda, make, run_balance

pytestmark = pytest.mark.gpu

MOST = float(torch.finfo(torch.bfloat16).max)
EXPERTS = [8, 32, 100, 512]        # 1, 4, 16 and 64 lanes a token


def with_logits(c, l):
    """The case c with the logits l (rounded to bf16) and the routing that follows from them."""
    c["logits"] = torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16).cuda()
    c["l"] = c["logits"].float().cpu().numpy().astype(np.float64)
    order = np.argsort(-c["l"], axis=1, kind="stable")[:, :c["k"]].astype(np.int32)
    c["ids"] = np.where(c["ids"] == -1, -1, order).astype(np.int32)
    return c


def z_error(z, m):
    return 2.0 ** -17 + 2.0 ** -22 * (np.abs(z) + np.abs(m))


def check_losses(c):
    counts, tokens, losses = run_balance(c)
    wc, wt, wl = O.balance(c["l"], c["ids"], c["seq"])
    np.testing.assert_array_equal(counts.cpu().numpy(), wc)
    np.testing.assert_array_equal(tokens.cpu().numpy(), wt)
    got = losses.double().cpu().numpy()
    assert abs(got[0] - wl[0]) <= 2.0 ** -15 * wl[0], (got, wl)
    live = [t for t, s in enumerate(O.counted(c["l"], c["ids"], c["seq"])) if s is not None]
    z = np.array([O.softmax(c["l"][t])[1] for t in live])
    if np.max(np.abs(z)) >= 2.0 ** 63:                    # its square may pass fp32's range
        assert got[1] > 2.0 ** 100
    else:
        m = c["l"][live].max(1)
        off = np.mean(2 * np.abs(z) * z_error(z, m) + z_error(z, m) ** 2) + 2.0 ** -16 * np.mean(z * z)
        assert abs(got[1] - wl[1]) <= off, (got, wl, off)
    return counts, tokens


def logit_gradient(c, counts, tokens, dlosses, gates=True, dtype=torch.float32):
    d = torch.full((c["T"], c["E"]), float("nan"), dtype=dtype, device="cuda")
    B.moe_route_backward(c["logits"], cuda(c["ids"]), cuda(c["gates"]) if gates else None,
                         cuda(c["dgates"]) if gates else None, c["T"], c["E"], c["k"], d,
                         seq_offsets=cuda(c["seq"]) if c["given"] else None, S=len(c["seq"]) - 1, counts=counts,
                         tokens=tokens, dlosses=cuda(np.asarray(dlosses, np.float32)))
    return d


def check_gradient(c, counts, tokens, dlosses, gates=True):
    d = logit_gradient(c, counts, tokens, dlosses, gates).double().cpu().numpy()
    want, mag = O.route_backward(c["l"], c["ids"], c["gates"], c["dgates"] if gates else None, c["seq"],
                                 np.asarray(dlosses, np.float32).astype(np.float64))
    load, toks, _ = O.balance(c["l"], c["ids"], c["seq"])
    b = abs(dlosses[1]) * 2.0 / max(int(toks[-2]), 1)
    bound = 2.0 ** -23 * np.abs(want) + 2.0 ** -15 * mag + 2.0 ** -126
    for t, s in enumerate(O.counted(c["l"], c["ids"], c["seq"])):
        if s is not None:
            p, z = O.softmax(c["l"][t])
            per_count = c["E"] * abs(dlosses[0]) / (c["k"] * float(toks[s]) ** 2 * float(toks[-1]))
            factor = per_count * 2 * np.max(np.abs(load[s] - load[s].mean())) + b * abs(z)
            bound[t] += p * b * z_error(z, c["l"][t].max()) + 2.0 ** -102 * factor
    bad = np.argwhere(~(np.abs(d - want) <= bound))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), d[tuple(bad[0])], want[tuple(bad[0])])
    return d


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("top", [1e5, -1e5, 3e9, 1e10, -1e10, 1e30, -1e30, 2.4e38, MOST, -1e38, -MOST])
def test_large_finite_logits(top, E):
    """A row whose largest logit is far from 0, some experts sharing it and some at the lowest
    value, among ordinary tokens."""
    _announce(f"logits up to {top:g}, E={E}")
    T, k = 70, 4
    c = make(T, E, k, None, seed=20, lost=0.0, masked=0.0)
    l = c["l"].copy()
    for t in (0, 3, 37, 69):
        l[t] = top
        l[t, 1::3] = -MOST
        l[t, 2::3] = top * (1.25 if top < 0 else 0.5) if abs(top) < 2e38 else -MOST
    with_logits(c, l)
    counts, tokens = check_losses(c)
    check_gradient(c, counts, tokens, [0.7 * T, 0.0], gates=False)
    if abs(top) < 1e30:
        check_gradient(c, counts, tokens, [0.7 * T, 0.2 * T])


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("spread", [20.0, 60.0, 300.0])
def test_wide_logits(spread, E):
    """Logits on both sides of 64, so that neighbouring tokens take either form of the exponential."""
    _announce(f"logits spread over {spread}, E={E}")
    T = 150
    c = make(T, E, 4, [0, 40, 40, 149], seed=21, spread=spread)
    counts, tokens = check_losses(c)
    check_gradient(c, counts, tokens, [0.7 * T, 0.2 * T])


@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("top,low", [(-60.0, -100.0), (-17.0, -95.0), (-16.0, -80.0), (-3.0, -85.0), (16.0, -60.0),
                                     (60.0, -20.0), (64.0, -20.0)])
def test_small_probabilities(top, low, E):
    """Experts far below a token's largest logit keep their probability, and their gradient, down to
    e^-71, wherever the largest lies."""
    _announce(f"logits {top} and {low}, E={E}")
    T = 70
    c = make(T, E, 2, None, seed=24, lost=0.0, masked=0.0)
    l = np.full((T, E), low)
    l[np.arange(T), np.arange(T) % 3] = top
    l[np.arange(T), 3 + np.arange(T) % 4] = 0.5 * (top + low)
    with_logits(c, l)
    counts, tokens = check_losses(c)
    d = check_gradient(c, counts, tokens, [0.7 * T, 0.2 * T], gates=False)
    assert np.all(d[np.arange(T), 3 + np.arange(T) % 4] != 0) and np.all(d[:, 7] != 0)


@pytest.mark.parametrize("E", EXPERTS)
def test_other_tokens_leave_the_bits(E):
    """What unrouted tokens and padding hold -- logits of any size, NaN, infinities -- changes no bit of
    the losses or of a counted token's gradient."""
    _announce(f"what other tokens hold, E={E}")
    T = 151
    r = np.random.default_rng(E)
    c = make(T, E, 4, [5, 60, 60, 140], seed=22, lost=0.0, masked=0.0)
    other = np.zeros(T, bool)
    other[r.choice(T, 40, replace=False)] = True
    c["ids"][other] = -1
    other[:5] = other[140:] = True                        # padding, routed or not
    seen = []
    for held in (None, 0.0, 65.0, -300.0, 1e30, -np.inf, np.inf, np.nan):
        l = c["l"].copy()
        if held is not None:
            l[other] = held
            l[other, 1] = -2.0
        d = dict(c, logits=torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16).cuda())
        counts, tokens, losses = run_balance(d)
        grads = [logit_gradient(d, counts, tokens, [0.7 * T, 0.2 * T], gates) for gates in (True, False)]
        seen.append([counts, tokens, losses, *grads])
        assert int(tokens[-2]) == int((~other).sum())
        for got, want in zip(seen[-1], seen[0]):
            assert torch.equal(got, want), held


def test_a_row_does_not_depend_on_its_place():
    """One token's gradient through the z loss: the same bits beside small and beside large logits, at
    any place of a wave."""
    _announce("one row at several places")
    for E in EXPERTS:
        r = np.random.default_rng(E + 1)
        row = r.normal(size=E) * 3
        T, k = 70, 2
        rows = []
        for place, around in ((0, 1.0), (17, 1.0), (17, 200.0), (69, 200.0)):
            c = make(T, E, k, None, seed=23, lost=0.0, masked=0.0)
            l = r.normal(size=(T, E)) * around
            l[place] = row
            with_logits(c, l)
            counts, tokens, _ = run_balance(c)
            assert int(tokens[-2]) == T
            rows.append(logit_gradient(c, counts, tokens, [0.0, 0.2 * T], gates=False)[place])
        assert all(torch.equal(x, rows[0]) for x in rows)


def _packed(T, E, k, seq, seed):
    """A case on the device without masked experts, and buffers for its calls."""
    c = make(T, E, k, seq, seed=seed, lost=0.0, masked=0.0)
    S = len(seq) - 1
    buf = dict(counts=torch.empty((S, E), dtype=torch.int32, device="cuda"),
               tokens=torch.empty((S + 2,), dtype=torch.int32, device="cuda"), losses=torch.empty(2, device="cuda"),
               ws=torch.empty((B.moe_balance_workspace_size(T, E, S),), dtype=torch.uint8, device="cuda"),
               ids=cuda(c["ids"]), seq=cuda(c["seq"]), dl=cuda(np.array([0.7 * T, 0.2 * T], np.float32)),
               dlogits=torch.full((T, E), float("nan"), device="cuda"))

    def balance():
        B.moe_balance(c["logits"], buf["ids"], T, E, k, buf["counts"], buf["tokens"], buf["losses"],
                      seq_offsets=buf["seq"], S=S, workspace=buf["ws"])

    def gradient():
        B.moe_route_backward(c["logits"], buf["ids"], None, None, T, E, k, buf["dlogits"], seq_offsets=buf["seq"],
                             S=S, counts=buf["counts"], tokens=buf["tokens"], dlosses=buf["dl"])
    return c, buf, balance, gradient


def _least_ms(call, times=5):
    best = float("inf")
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("E", [8, 32, 512])
@pytest.mark.parametrize("T,used", [(300, [0, 20, 150, 290]), (300, [0, 300]), (40, [0, 1, 2, 3, 30])])
def test_runs_of_empty_sequences(T, used, E):
    """Thousands of equal offsets in front of, inside and behind a chunk of tokens: the values of the
    used sequences alone."""
    _announce(f"runs of empty sequences, T={T} E={E} {used}")
    k, run = 2, 3000
    seq, at = [], []
    for i, o in enumerate(used):
        seq += [o] * (run if i < len(used) - 1 else 1 + run)
        at.append(len(seq) - 1)
    c, buf, balance, gradient = _packed(T, E, k, seq, 25)
    balance()
    gradient()
    dense = dict(c, seq=np.asarray(used, np.int32))
    wc, wt, wl = O.balance(c["l"], c["ids"], dense["seq"])
    S = len(used) - 1
    np.testing.assert_array_equal(buf["counts"][at[:-1]].cpu().numpy(), wc)
    assert int(buf["counts"].sum()) == int(wc.sum())
    np.testing.assert_array_equal(buf["tokens"][at[:-1]].cpu().numpy(), wt[:S])
    assert buf["tokens"][-2:].tolist() == wt[-2:].tolist()
    got = buf["losses"].double().cpu().numpy()
    assert abs(got[0] - wl[0]) <= 2.0 ** -15 * wl[0] and abs(got[1] - wl[1]) <= 2.0 ** -15 * wl[1] + 2.0 ** -16
    tokens = torch.cat([buf["tokens"][at[:-1]], buf["tokens"][-2:]]).contiguous()
    counts = buf["counts"][at[:-1]].contiguous()
    assert torch.equal(logit_gradient(dense, counts, tokens, buf["dl"].cpu().numpy(), gates=False), buf["dlogits"])
    check_gradient(dense, counts, tokens, buf["dl"].cpu().numpy().astype(np.float64), gates=False)


def test_runs_of_empty_sequences_cost_no_walk():
    """65535 empty sequences in the middle of the tokens take about the time that they take behind
    them, where no token passes them (looking at them one by one: over 20 times that)."""
    _announce("time of empty sequences")
    T, E, k, run = 64, 8, 2, 65535
    inside = [0] + [33] * (run + 1) + [T]
    behind = [0, 33] + [T] * (run + 1)
    times = []
    for seq in (inside, behind):
        _, _, balance, gradient = _packed(T, E, k, seq, 26)
        balance()
        times.append((_least_ms(balance), _least_ms(gradient)))
    print(f"[case] ms inside {times[0]}, behind {times[1]}", flush=True)
    assert times[0][0] < 4 * times[1][0] and times[0][1] < 4 * times[1][1] + 0.1, times


@pytest.mark.parametrize("E", [8, 512])
def test_most_sequences(E):
    """MOE_MAX_SEQUENCES of them, all but a few empty."""
    _announce(f"2^20 sequences, E={E}")
    T, k, S = 300, 2, B.MOE_MAX_SEQUENCES
    seq = np.zeros(S + 1, np.int32)
    used = [0, 5, 170, 290]
    at = [3, S // 2, S - 9]                     # the used sequences
    for i, s in enumerate(at):
        seq[s + 1:] = used[i + 1]
    c, buf, balance, gradient = _packed(T, E, k, seq, 27)
    balance()
    gradient()
    wc, wt, wl = O.balance(c["l"], c["ids"], np.asarray(used))
    np.testing.assert_array_equal(buf["counts"][at].cpu().numpy(), wc)
    assert int(buf["counts"].sum(dtype=torch.int64)) == int(wc.sum())
    assert buf["tokens"][at].tolist() == wt[:3].tolist() and buf["tokens"][-2:].tolist() == wt[-2:].tolist()
    got = buf["losses"].double().cpu().numpy()
    assert abs(got[0] - wl[0]) <= 2.0 ** -15 * wl[0] and abs(got[1] - wl[1]) <= 2.0 ** -15 * wl[1] + 2.0 ** -16
    dense = dict(c, seq=np.asarray(used, np.int32))
    tokens = torch.cat([buf["tokens"][at], buf["tokens"][-2:]]).contiguous()
    assert torch.equal(logit_gradient(dense, buf["counts"][at].contiguous(), tokens, buf["dl"].cpu().numpy(),
                                      gates=False), buf["dlogits"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [5, 8, 33, 64, 512])
def test_tensors_off_16_bytes(E, dtype):
    """Tensors that begin between 16-byte borders: the bits of aligned ones, and nothing before or
    behind the outputs is written."""
    _announce(f"balance, storage offsets, E={E} {dtype}")
    T, k = 77, 3
    c = make(T, E, k, [2, 30, 30, 75], seed=28)
    dl = cuda(np.array([0.7 * T, 0.2 * T], np.float32))
    args = [c["logits"], cuda(c["ids"]), cuda(c["gates"]), cuda(c["dgates"]), cuda(c["seq"]), dl]

    def shifted(t, by):
        flat = torch.full((t.numel() + 16,), 7, dtype=t.dtype, device="cuda")
        flat[by:by + t.numel()] = t.reshape(-1)
        return flat, flat[by:by + t.numel()].view(t.shape)

    def run(by):
        logits, ids, gates, dgates, seq, dlosses = (shifted(t, by)[1] for t in args)
        outs = [shifted(torch.zeros(shape, dtype=d, device="cuda"), by)
                for shape, d in (((3, E), torch.int32), ((5,), torch.int32), ((2,), torch.float32), ((T, E), dtype))]
        (_, counts), (_, tokens), (_, losses), (_, dlogits) = outs
        B.moe_balance(logits, ids, T, E, k, counts, tokens, losses, seq_offsets=seq, S=3,
                      workspace=torch.full((B.moe_balance_workspace_size(T, E, 3),), 255, dtype=torch.uint8, device="cuda"))
        B.moe_route_backward(logits, ids, gates, dgates, T, E, k, dlogits, seq_offsets=seq, S=3, counts=counts,
                             tokens=tokens, dlosses=dlosses)
        for flat, view in outs:
            assert bool((flat[:by] == 7).all()) and bool((flat[by + view.numel():] == 7).all())
        return [view for _, view in outs]

    want = run(0)
    for by in (1, 2, 3):
        for got, w in zip(run(by), want):
            assert torch.equal(got, w), by


def test_two_graphs_share_a_workspace():
    """Two captured balances of different sizes on one workspace, replayed in turn: each replay gives the
    eager result."""
    _announce("two graphs, one workspace")
    sizes = [(700, 32, [0, 100, 100, 650]), (5000, 512, list(range(0, 5001, 25))), (64, 8, [0, 64])]
    ws = torch.full((max(B.moe_balance_workspace_size(T, E, len(seq) - 1) for T, E, seq in sizes),), 255,
                    dtype=torch.uint8, device="cuda")
    graphs = []
    for i, (T, E, seq) in enumerate(sizes):
        c, buf, _, _ = _packed(T, E, 2, seq, 30 + i)
        outs = [buf["counts"], buf["tokens"], buf["losses"]]

        def call(c=c, buf=buf, T=T, E=E, S=len(seq) - 1):
            B.moe_balance(c["logits"], buf["ids"], T, E, 2, buf["counts"], buf["tokens"], buf["losses"],
                          seq_offsets=buf["seq"], S=S, workspace=ws)
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append((g, outs, want, (c, buf)))     # a graph reads its inputs where they were captured
    for turn in (0, 1, 2, 1, 0, 2, 0):
        g, outs, want, _ = graphs[turn]
        for o in outs:
            o.fill_(-7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want)), turn
