"""The operators around the expert block together, as they are used: a block's forward pass from the
residual stream to the next block's input, its router's gradients, captured graphs, other streams
and offsets past 32 bits.  Values against the float64 oracles stage by stage (tolerances as in
test_gpu_block_norm.py and test_gpu_balance.py), otherwise bit for bit against the separate calls.

The balance past 32-bit offsets: a workgroup's chunk of 16385 tokens runs 16 at a time, so a lane adds
1024 or 1025 values; with even logits over 512 experts these are 1 / 512 each and every sum is exact."""
import numpy as np
import pytest
import torch

import oracle.block_oracle as O
import oracle.moe_oracle as M
from mxfp4_mixture_experts_amd import binding as B
from mxfp4_mixture_experts_amd import synthetic as S
from mxfp4_mixture_experts_amd.runner import DeviceProblem
from test_gpu_block_norm import EPS, HALF, TINY, close, dev, f64, nan_like, routing, stream_rows, weights, workspace
from test_gpu_graph import _replay_matches

pytestmark = pytest.mark.gpu


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def _dev_bits(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


class Block:
    """One MoE block on the device: norm, router, routing, balance, experts, output, next norm."""

    def __init__(self, T, H, inner, E, k, dtype, tag):
        self.T, self.H, self.E, self.k = T, H, E, k
        r = np.random.default_rng(np.random.SeedSequence(40, spawn_key=(T, H, tag)))
        self.x = stream_rows(r, T, H, dtype)
        self.w_in, self.w_post, self.w_next = weights(r, H), weights(r, H), weights(r, H)
        router = S.make_router(T, H, E, tag=tag)
        self.rw, self.rb = _dev_bits(router.w), _dev_bits(router.bias)
        gu = S.make_custom(E=E, N=2 * inner, K=H, T=T, k=k, route="logits", tag=tag + 1, combine=False)
        dn = S.make_custom(E=E, N=H, K=inner, T=T, k=k, x_per_slot=True, route="logits", tag=tag + 2, combine=True)
        self.up, self.down = DeviceProblem(gu), DeviceProblem(dn)
        d, u = self.down, self.up
        d.x, d.topk_ids, d.gates, d.offsets, d.sorted_rows = u.act, u.topk_ids, u.gates, u.offsets, u.sorted_rows
        self.logits = u.logits
        self.xn = u.x
        self.x_out = nan_like((T, H), dtype)
        self.xn_next = nan_like((T, H), torch.bfloat16)
        self.counts = torch.zeros((1, E), dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros((3,), dtype=torch.int32, device="cuda")
        self.losses = nan_like((2,), torch.float32)
        self.ws = workspace(B.moe_balance_workspace_size(T, E, 1))

    def forward(self, stream=None):
        T, H, E, k = self.T, self.H, self.E, self.k
        B.moe_norm(self.x, self.w_in, T, H, self.xn, eps=EPS, stream=stream)
        B.mxfp4_moe_router(self.xn, self.rw, self.rb, T, H, E, self.logits, stream)
        self.up.route_group(stream)
        B.moe_balance(self.logits, self.up.topk_ids, T, E, k, self.counts, self.tokens, self.losses, workspace=self.ws,
                      stream=stream)
        self.up.expert_proj_swiglu(stream)
        self.down.expert_proj(stream)
        B.moe_combine_norm(self.down.out, self.up.gates, T, k, H, self.x, self.x_out, w_post=self.w_post, scale=0.5,
                           w_next=self.w_next, xn=self.xn_next, eps=EPS, stream=stream)

    def outputs(self):
        return [self.xn, self.logits, self.up.topk_ids, self.counts, self.tokens, self.losses, self.up.act,
                self.down.out, self.x_out, self.xn_next]


# T, H, inner, E, k
CASES = {"one_token": (1, 2880, 512, 32, 4), "decode_batch": (5, 256, 128, 8, 2), "prompt": (150, 320, 96, 16, 4)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", sorted(CASES))
def test_block_forward(case, dtype):
    T, H, inner, E, k = CASES[case]
    _announce(f"block forward {case} {dtype}")
    b = Block(T, H, inner, E, k, dtype, tag=500 + 10 * sorted(CASES).index(case))
    b.forward()
    want = O.norm(f64(b.x), f64(b.w_in), EPS)
    close(b.xn, want, (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + TINY, "xn")
    l, ids = f64(b.logits), b.up.topk_ids.cpu().numpy()
    counts, tokens, losses = O.balance(l, ids, [0, T])
    np.testing.assert_array_equal(b.counts.cpu().numpy(), counts)
    np.testing.assert_array_equal(b.tokens.cpu().numpy(), tokens)
    assert int(b.counts.sum()) == T * k
    # the counts are the grouping's
    np.testing.assert_array_equal(np.diff(b.up.offsets.cpu().numpy()), counts[0])
    assert abs(float(b.losses[0]) - losses[0]) <= 2.0 ** -16 * losses[0]
    assert abs(float(b.losses[1]) - losses[1]) <= 2.0 ** -15 * losses[1] + 2.0 ** -18
    # the output: the combine's bits, then the norms
    y = nan_like((T, H), torch.float32)
    B.moe_combine(b.down.out, b.up.gates, T, k, H, y)
    fused = nan_like((T, H), dtype)
    B.moe_combine_norm(y.view(T, 1, H), None, T, 1, H, b.x, fused, w_post=b.w_post, scale=0.5, eps=EPS)
    assert torch.equal(fused, b.x_out), "combine then output norm is not the fused output"
    nxt = nan_like((T, H), torch.bfloat16)
    B.moe_norm(b.x_out, b.w_next, T, H, nxt, eps=EPS)
    assert torch.equal(nxt, b.xn_next)
    u = O.norm(f64(y), f64(b.w_post), EPS)
    want = f64(b.x) + 0.5 * u
    close(b.x_out, want, HALF[dtype] * np.abs(want) * 1.01 + 2.0 ** -19 * (np.abs(f64(b.x)) + np.abs(u)) + TINY, "x_out")


def test_one_token_output_after_the_fused_projection():
    """One token: mxfp4_expert_proj_combine's y through moe_combine_norm (k = 1, no gates) equals the
    projection's slots through it, bit for bit."""
    _announce("one token, fused projection then output norm")
    b = Block(1, 2880, 512, 32, 4, torch.bfloat16, tag=560)
    b.forward()
    d = b.down
    y = nan_like((1, 2880), torch.float32)
    B.mxfp4_expert_proj_combine(d.blocks, d.scales, d.bias, 32, 2880, 512, b.up.act, True, 4, b.up.topk_ids,
                                b.up.gates, y)
    x_out, xn = nan_like((1, 2880), torch.bfloat16), nan_like((1, 2880), torch.bfloat16)
    B.moe_combine_norm(y.view(1, 1, 2880), None, 1, 1, 2880, b.x, x_out, w_post=b.w_post, scale=0.5, w_next=b.w_next,
                       xn=xn, eps=EPS)
    assert torch.equal(x_out, b.x_out) and torch.equal(xn, b.xn_next)


def test_router_gradient_through_the_block():
    """The router's training step: the block output's gradients, then the logits' through the gates
    and the losses; end to end against the oracle on the GPU's own forward values."""
    T, H, inner, E, k = 90, 320, 96, 16, 4
    _announce("router gradient")
    b = Block(T, H, inner, E, k, torch.float32, tag=570)
    b.forward()
    r = np.random.default_rng(571)
    dx_out, dxn = dev(r.normal(size=(T, H))), dev(r.normal(size=(T, H)), torch.bfloat16)
    dx, dproj, dgates = nan_like((T, H), torch.float32), nan_like((T, k, H), torch.float32), nan_like((T, k), torch.float32)
    dw_post, dw_next = nan_like((H,), torch.float32), nan_like((H,), torch.float32)
    B.moe_combine_norm_backward(dx_out, b.down.out, b.up.gates, T, k, H, dx=dx, dproj=dproj, dgates=dgates,
                                w_post=b.w_post, dw_post=dw_post, scale=0.5, dxn=dxn, x_out=b.x_out, w_next=b.w_next,
                                dw_next=dw_next, eps=EPS,
                                workspace=workspace(B.moe_combine_norm_backward_workspace_size(T, H)))
    dl = dev([0.01 * T, 0.001 * T])
    dlogits = nan_like((T, E), torch.float32)
    B.moe_route_backward(b.logits, b.up.topk_ids, b.up.gates, dgates, T, E, k, dlogits, counts=b.counts,
                         tokens=b.tokens, dlosses=dl)
    w = O.combine_norm_backward(f64(dx_out), f64(dxn), f64(b.x_out), f64(b.w_next), f64(b.down.out), f64(b.up.gates),
                                f64(b.w_post), 0.5, EPS)
    close(dgates, w["dgates"], (2.0 ** -16 + 2.0 ** -18) * w["mag_dgates"], "dgates")
    close(dproj, w["dproj"], 2.0 ** -16 * w["mag_dproj"] + TINY, "dproj")
    ids = b.up.topk_ids.cpu().numpy()
    want, mag = O.route_backward(f64(b.logits), ids, f64(b.up.gates), f64(dgates), [0, T], f64(dl))
    close(dlogits, want, 2.0 ** -15 * mag + 1e-15, "dlogits")
    # the gates' part sums to 0 over the experts, the losses' too but for z
    total = f64(dlogits).sum(1)
    z = np.array([O.softmax(row)[1] for row in f64(b.logits)])
    assert np.all(np.abs(total - float(f64(dl)[1]) * 2.0 / T * z) <= 2.0 ** -15 * mag.sum(1))
    # the router's input gradient: x's, through the first norm
    dxr, dw = nan_like((T, H), torch.float32), nan_like((H,), torch.float32)
    din = torch.matmul(dlogits, b.rw.float()).to(torch.bfloat16)
    B.moe_norm_backward(din, b.x, b.w_in, T, H, dxr, dw, dres=dx, eps=EPS,
                        workspace=workspace(B.moe_norm_backward_workspace_size(T, H)))
    want, want_w, mag, mag_w = O.norm_backward(f64(din), f64(b.x), f64(b.w_in), EPS)
    close(dxr, want + f64(dx), 2.0 ** -24 * np.abs(want + f64(dx)) + 2.0 ** -17 * (mag + np.abs(f64(dx))), "dx")
    close(dw, want_w, (2.0 ** -18 + 64 * 2.0 ** -24) * mag_w, "dw")


@pytest.mark.parametrize("case", sorted(CASES))
def test_graph_block_forward(case):
    T, H, inner, E, k = CASES[case]
    _announce(f"graph: block forward {case}")
    b = Block(T, H, inner, E, k, torch.bfloat16, tag=600 + 10 * sorted(CASES).index(case))
    _replay_matches(b.forward, b.outputs())


def test_graph_backward():
    _announce("graph: the gradients")
    T, H, E, k = 700, 520, 32, 4
    r = np.random.default_rng(611)
    x, w1, w2 = stream_rows(r, T, H, torch.bfloat16), weights(r, H), weights(r, H)
    gates, proj = dev(routing(r, T, k)), dev(r.normal(size=(T, k, H)))
    dxo, dxn = dev(r.normal(size=(T, H)), torch.bfloat16), dev(r.normal(size=(T, H)), torch.bfloat16)
    logits = dev(r.normal(size=(T, E)), torch.bfloat16)
    ids = torch.topk(logits.float(), k).indices.to(torch.int32).contiguous()
    seq = torch.tensor([0, 100, 100, 650], dtype=torch.int32, device="cuda")
    o = dict(dx=nan_like((T, H), torch.bfloat16), dproj=nan_like((T, k, H), torch.float32),
             dgates=nan_like((T, k), torch.float32), dw_post=nan_like((H,), torch.float32),
             dw_next=nan_like((H,), torch.float32))
    dx2, dw2 = nan_like((T, H), torch.bfloat16), nan_like((H,), torch.float32)
    counts = torch.zeros((3, E), dtype=torch.int32, device="cuda")
    tokens = torch.zeros(5, dtype=torch.int32, device="cuda")
    losses, dlogits, dl = nan_like((2,), torch.float32), nan_like((T, E), torch.float32), dev([5.0, 0.5])
    # one workspace for calls in order on one stream
    ws = workspace(max(B.moe_combine_norm_backward_workspace_size(T, H), B.moe_norm_backward_workspace_size(T, H),
                       B.moe_balance_workspace_size(T, E, 3)))

    def step():
        B.moe_balance(logits, ids, T, E, k, counts, tokens, losses, seq_offsets=seq, S=3, workspace=ws)
        B.moe_combine_norm_backward(dxo, proj, gates, T, k, H, **o, w_post=w1, scale=0.5, dxn=dxn, x_out=x, w_next=w2,
                                    eps=EPS, workspace=ws)
        B.moe_route_backward(logits, ids, gates, o["dgates"], T, E, k, dlogits, seq_offsets=seq, S=3, counts=counts,
                             tokens=tokens, dlosses=dl)
        B.moe_norm_backward(dxn, x, w1, T, H, dx2, dw2, dres=o["dx"], eps=EPS, workspace=ws)
    _replay_matches(step, [*o.values(), counts, tokens, losses, dlogits, dx2, dw2])


def test_other_streams():
    """Two blocks on two streams at once, each with its own workspace, by argument and by torch's
    current stream: the bits of the default stream."""
    _announce("two streams")
    T, H, inner, E, k = CASES["prompt"]
    blocks = [Block(T, H, inner, E, k, torch.bfloat16, tag=640 + 10 * i) for i in range(2)]
    want = []
    for b in blocks:
        b.forward()
        want.append([o.clone() for o in b.outputs()])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for b in blocks:
        for o in (b.x_out, b.xn_next, b.losses):
            o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        blocks[0].forward(s[0])
        with torch.cuda.stream(s[1]):
            blocks[1].forward()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert all(torch.equal(o, v) for o, v in zip(b.outputs(), w))


def _norm64(x, w):
    x = x.double()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()


def test_norm_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are computed, from their own values."""
    _announce("norm: 2.46e9 elements")
    T, N = 300000, 8192
    x = torch.ones((T, N), dtype=torch.bfloat16, device="cuda")
    w = weights(np.random.default_rng(1), N)
    tail = stream_rows(np.random.default_rng(2), 5, N, torch.bfloat16)
    x[-5:] = tail
    xn = torch.empty_like(x)
    B.moe_norm(x, w, T, N, xn, eps=EPS)
    for rows in (slice(0, 2), slice(262143, 262146), slice(T - 5, T)):
        want = _norm64(x[rows], w)
        assert bool(((xn[rows].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs()).all())
    del xn
    dx = torch.empty_like(x)
    B.moe_norm_backward(x, x, w, T, N, dx, None, eps=EPS)
    got = dx[-5:].double().cpu().numpy()
    want, _, mag, _ = O.norm_backward(f64(tail), f64(tail), f64(w), EPS)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * mag)


def test_combine_norm_past_32_bit_offsets():
    _announce("combine_norm: 2.3e9 elements")
    T, k, N = 70000, 4, 8192
    proj = torch.ones((T, k, N), dtype=torch.bfloat16, device="cuda")
    r = np.random.default_rng(3)
    tail = dev(r.normal(size=(3, k, N)), torch.bfloat16)
    proj[-3:] = tail
    gates = dev(routing(r, T, k, lost=0.0))
    x = torch.zeros((T, N), dtype=torch.float32, device="cuda")
    x_out = torch.empty_like(x)
    B.moe_combine_norm(proj, gates, T, k, N, x, x_out)
    h, mag = O.combine(f64(tail), f64(gates[-3:]))
    close(x_out[-3:], h, (2.0 ** -24 + k * 2.0 ** -24) * mag, "x_out")
    del x, x_out
    dproj = torch.empty_like(proj)
    dx_out = torch.ones((T, N), dtype=torch.bfloat16, device="cuda")
    dgates = nan_like((T, k), torch.float32)
    B.moe_combine_norm_backward(dx_out, proj, gates, T, k, N, dproj=dproj, dgates=dgates)
    want = f64(gates[-3:])[:, :, None] * np.ones(N)
    close(dproj[-3:], want, 2.0 ** -8 * want, "dproj")
    want = f64(tail).sum(2)
    close(dgates[-3:], want, 2.0 ** -18 * np.abs(f64(tail)).sum(2), "dgates")


def test_balance_past_32_bit_offsets():
    _announce("balance: 4.3e9 logits")
    T, E, k = (1 << 23) + 5, 512, 1
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    logits[-5:, 500] = 4.0
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    ids[-5:] = 500
    seq = torch.tensor([0, T - 5, T], dtype=torch.int32, device="cuda")
    counts = torch.zeros((2, E), dtype=torch.int32, device="cuda")
    tokens, losses = torch.zeros(4, dtype=torch.int32, device="cuda"), nan_like((2,), torch.float32)
    B.moe_balance(logits, ids, T, E, k, counts, tokens, losses, seq_offsets=seq, S=2,
                  workspace=workspace(B.moe_balance_workspace_size(T, E, 2)))
    assert tokens.tolist() == [T - 5, 5, T, 2]
    assert int(counts[0, 0]) == T - 5 and int(counts[1, 500]) == 5 and int(counts.sum()) == T
    p500 = np.exp(4.0) / (np.exp(4.0) + 511)
    want = 0.5 * (1.0 + E * p500)
    # a workgroup adds 16384 tokens 1024 at a time, 16 in a lane's chain
    assert abs(float(losses[0]) - want) <= 2.0 ** -16 * want
    d = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
    B.moe_route_backward(logits, ids, None, None, T, E, k, d, seq_offsets=seq, S=2, counts=counts, tokens=tokens,
                         dlosses=dev([1.0, 0.0]))
    got = d[-5:].double().cpu().numpy()
    a = E / (2 * 25.0)
    p = np.full(E, (1 - p500) / 511)
    p[500] = p500
    c = np.zeros(E)
    c[500] = 5
    want = a * p * (c - p @ c)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * a * p * (c + p @ c + 2 * c.mean()) + 1e-15)


def test_more_rows_than_one_launch():
    """A forward pass of more rows than one launch's grid takes."""
    _announce("norm: 4194309 rows")
    T, N, k = (1 << 22) + 5, 8, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16)
    w = weights(np.random.default_rng(4), N)
    xn = nan_like((T, N), torch.bfloat16)
    B.moe_norm(x, w, T, N, xn, eps=EPS)
    want = _norm64(x, w)
    assert bool(((xn.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs()).all())
    proj = torch.randn((T, k, N), generator=g, device="cuda")
    gates = torch.rand((T, k), generator=g, device="cuda")
    x_out, xn2 = nan_like((T, N), torch.bfloat16), nan_like((T, N), torch.bfloat16)
    B.moe_combine_norm(proj, gates, T, k, N, x, x_out, scale=0.5, w_next=w, xn=xn2, eps=EPS)
    terms = gates.double()[:, :, None] * proj.double()
    want = x.double() + 0.5 * terms.sum(1)
    slack = 2.0 ** -22 * (x.double().abs() + terms.abs().sum(1))
    assert bool(((x_out.double() - want).abs() <= 2.0 ** -8 * want.abs() * 1.01 + slack).all())
    want = _norm64(x_out, w)
    assert bool(((xn2.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want.abs()).all())


def test_padding_holds_anything():
    """NaN logits, ids and gates behind the last sequence reach no output."""
    _announce("padding")
    T, E, k = 100, 32, 4
    r = np.random.default_rng(8)
    l = r.normal(size=(T, E))
    ids = np.argsort(-l, axis=1)[:, :k].astype(np.int32)
    l[60:] = np.nan
    l[70] = np.inf
    gates = routing(r, T, k, lost=0.0)
    gates[60:] = np.nan
    logits, idt = dev(l, torch.bfloat16), torch.from_numpy(ids).cuda()
    seq = torch.tensor([0, 25, 60], dtype=torch.int32, device="cuda")
    counts = torch.zeros((2, E), dtype=torch.int32, device="cuda")
    tokens, losses = torch.zeros(4, dtype=torch.int32, device="cuda"), nan_like((2,), torch.float32)
    B.moe_balance(logits, idt, T, E, k, counts, tokens, losses, seq_offsets=seq, S=2,
                  workspace=workspace(B.moe_balance_workspace_size(T, E, 2)))
    wc, wt, wl = O.balance(f64(logits), ids, [0, 25, 60])
    np.testing.assert_array_equal(counts.cpu().numpy(), wc)
    assert tokens.tolist() == [25, 35, 60, 2] and abs(float(losses[0]) - wl[0]) <= 2.0 ** -16 * wl[0]
    d = nan_like((T, E), torch.float32)
    dg = dev(np.where(np.isnan(gates), np.nan, 1.0))
    B.moe_route_backward(logits, idt, dev(gates), dg, T, E, k, d, seq_offsets=seq, S=2, counts=counts, tokens=tokens,
                         dlosses=dev([3.0, 1.0]))
    assert bool(torch.isfinite(d).all()) and not d[60:].any() and bool((d[:60] != 0).any(1).all())


def test_smallest_and_largest_teams_share_one_norm():
    """The norm of a row does not depend on how many rows there are or where it lies."""
    _announce("row independence")
    for N in (8, 100, 511, 520, 1500, 2881, 8200):
        r = np.random.default_rng(N)
        x, w = stream_rows(r, 37, N, torch.bfloat16), weights(r, N)
        all_rows, one = nan_like((37, N), torch.bfloat16), nan_like((1, N), torch.bfloat16)
        B.moe_norm(x, w, 37, N, all_rows, eps=EPS)
        for t in (0, 17, 36):
            B.moe_norm(x[t:t + 1].contiguous(), w, 1, N, one, eps=EPS)
            assert torch.equal(one[0], all_rows[t]), (N, t)
