"""The whole expert layer of a few tokens on the GPU against the float64 oracle.

Tolerance: intervals carried through the layer.  Where a rounding to bf16 lies between two steps, a
value known to +-e before it lies between the roundings of its ends, so a rounding that both sides make
alike costs nothing and one near a border its whole step.
  xn      before its rounding off by (H / 64 + 20) 2^-24 of itself: a lane's H / 64 squares summed in
          fp32 one after the other, the wave's sum, the root, the division and two products.
  sums    an MFMA adds the products of 32 elements to its accumulator; taken as a sum aligned to its
          largest term and cut there, 32 2^-23 of the terms' magnitudes over all steps, and each step's
          sum is rounded (2^-23 with cutting), K / 32 times, then 12 waves' partial sums and the bias:
          (2^-18 + (K / 32 + 16) 2^-23) of the magnitudes.  The router's sums, a lane's products of pairs
          (H / 128 and 4 at least, 2^-23 each) and the wave's, are within it.
  gates   the logits' error dl moves a softmax by the factor exp(2 dl) at most; the exponential, the sum
          and the quotient by (k + 8) 2^-23.
  act     the projection's box through the activation (the oracle's swiglu_range), 4e-6 relative and 2e-5
          for its own arithmetic, as for the library's other gated projections, then its rounding.
  y       each wave's k products and sums, 12 waves' sums, the biases and the residual, (2 k + 14) 2^-23 of
          the terms' magnitudes, and its rounding.
The kernel's ids are held to the logits: each within 2 dl of what the oracle takes at its place, equal
where the oracle's margins are wider; the oracle then follows the kernel's ids.
"""
import numpy as np
import pytest
import torch

import oracle.moe_oracle as M
import oracle.mx_oracle as O
from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def sums(mag, K):
    return (2.0 ** -18 + (K / 32 + 16) * 2.0 ** -23) * mag


def rounded(v, e):
    """bf16(v) and how far bf16 of a value within e of v can lie from it."""
    r = O.bf16(v)
    return r, np.maximum(np.abs(O.bf16(v + e) - r), np.abs(O.bf16(v - e) - r))


class Layer:
    def __init__(self, T, E, k, H, F, x="bf16", norm=True, residual=True, y="bf16", biases=True, seed=0, lo=117,
                 hi=124):
        r = np.random.default_rng([seed, T, E, k, H, F])
        self.s = (T, H, E, k, F)
        self.norm, self.residual = norm, residual
        xv = r.normal(size=(T, H)) * np.exp(r.normal(size=(T, 1)))
        self.x = O.bf16(xv) if x == "bf16" else xv.astype(np.float32).astype(np.float64)
        self.dx = cuda(self.x).to(torch.bfloat16 if x == "bf16" else torch.float32)
        bf = lambda a: (O.bf16(a), cuda(O.bf16(a)).to(torch.bfloat16))
        self.w_norm, self.dw_norm = bf(1 + 0.1 * r.normal(size=H)) if norm else (None, None)
        self.rw, self.drw = bf(r.normal(size=(E, H)) / np.sqrt(H) * 2)
        self.rb, self.drb = bf(r.normal(size=E) * 0.1) if biases else (None, None)
        self.gu = (r.integers(0, 256, (E, 2 * F, H // 32, 16)).astype(np.uint8),
                   r.integers(lo, hi, (E, 2 * F, H // 32)).astype(np.uint8))
        self.down = (r.integers(0, 256, (E, H, F // 32, 16)).astype(np.uint8),
                     r.integers(lo, hi, (E, H, F // 32)).astype(np.uint8))
        self.bgu, self.dbgu = bf(r.normal(size=(E, 2 * F)) * 0.3) if biases else (None, None)
        self.bd, self.dbd = bf(r.normal(size=(E, H)) * 0.3) if biases else (None, None)
        self.dgu, self.ddown = tuple(map(cuda, self.gu)), tuple(map(cuda, self.down))
        self.y = torch.full((T, H), float("nan"), dtype=torch.bfloat16 if y == "bf16" else torch.float32,
                            device="cuda")
        self.ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        self.gates = torch.full((T, k), float("nan"), dtype=torch.float32, device="cuda")
        self.ws = torch.full((B.mxfp4_moe_layer_workspace_size(T, H, E, k, F),), 0xFF, dtype=torch.uint8,
                             device="cuda")

    def call(self, outs=True, stream=None, y=None):
        B.mxfp4_moe_layer(self.dx, *self.s, self.drw, self.drb, *self.dgu, self.dbgu, *self.ddown, self.dbd,
                          self.y if y is None else y, w_norm=self.dw_norm, eps=EPS, residual=self.residual,
                          topk_ids=self.ids if outs else None, gates=self.gates if outs else None,
                          workspace=self.ws, stream=stream)

    def check(self):
        T, H, E, k, F = self.s
        w_gu, w_down = O.decode(*self.gu), O.decode(*self.down)
        x = self.x
        if self.norm:
            v = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS) * self.w_norm
            xn, exn = rounded(v, np.abs(v) * (H / 64 + 20) * 2.0 ** -24)
        else:
            xn, exn = x, np.zeros_like(x)
        assert np.array_equal(xn, O.layer_route(x, self.w_norm, EPS, self.rw, self.rb, k)[0])
        logits, mag = O.matmul(xn, self.rw, self.rb)
        dl = exn @ np.abs(self.rw).T + sums(mag, H)
        d = dl.max(1)
        # the kernel's routing
        ids, gates = self.ids.cpu().numpy(), self.gates.cpu().numpy().astype(np.float64)
        want = np.argsort(-logits, axis=1, kind="stable")
        assert ((ids >= 0) & (ids < E)).all() and all(len(set(row)) == k for row in ids.tolist())
        got_l = np.take_along_axis(logits, ids, 1)
        want_l = np.take_along_axis(logits, want, 1)
        assert (np.abs(got_l - want_l[:, :k]) <= 2 * d[:, None]).all(), "ids"
        g = np.exp(got_l - got_l.max(1, keepdims=True))
        g /= g.sum(1, keepdims=True)
        eg = g * (np.expm1(2 * d)[:, None] + (k + 8) * 2.0 ** -23)
        assert (np.abs(gates - g) <= eg).all(), "gates"
        # through the experts
        p, mag = O.expert_matmul(w_gu, self.bgu, xn, False, ids)
        ep, _ = O.expert_matmul(np.abs(w_gu), None, exn, False, ids)
        ep = ep + sums(mag, H)
        f = M.swiglu(p)
        lo, hi = M.swiglu_range(p - ep, p + ep)
        ef = np.maximum(hi - f, f - lo)
        act, ea = rounded(f, ef + 4e-6 * (np.abs(f) + ef) + 2e-5)
        o, mag_o = O.expert_matmul(w_down, self.bd, act, True, ids)
        eo, _ = O.expert_matmul(np.abs(w_down), None, ea, True, ids)
        eo = eo + sums(mag_o, F)
        h = (g[..., None] * o).sum(1)
        size = (g[..., None] * mag_o).sum(1)
        eh = (g[..., None] * eo + eg[..., None] * (np.abs(o) + eo)).sum(1)
        assert np.allclose(h, O.layer(xn, ids, g, w_gu, self.bgu, w_down, self.bd)[0], rtol=1e-12, atol=1e-12)
        if self.residual:
            h, size = h + x, size + np.abs(x)
        eh = eh + (2 * k + 14) * 2.0 ** -23 * (size + eh)
        half = 2.0 ** -8 if self.y.dtype == torch.bfloat16 else 2.0 ** -24
        bound = eh + half * (np.abs(h) + eh)
        got = self.y.float().cpu().numpy().astype(np.float64)
        err = np.abs(got - h)
        assert (err <= bound).all(), (f"y: {int((~(err <= bound)).sum())} of {err.size} outside, worst "
                                      f"{float(np.nanmax(err / bound)):.3g}")
        return h


def run(*a, **kw):
    _announce(f"layer {a} {kw}")
    layer = Layer(*a, **kw)
    layer.call()
    layer.check()
    return layer


SIZES = [  # T, E, k, H, F
    (1, 1, 1, 32, 32), (1, 4, 2, 64, 96), (2, 8, 8, 32, 512), (3, 5, 3, 288, 160), (1, 32, 4, 2880, 2880),
    (8, 32, 4, 512, 544), (16, 64, 16, 96, 64), (5, 7, 3, 1056, 32), (4, 13, 4, 2048, 768), (7, 64, 1, 160, 2880),
    (16, 3, 2, 320, 1024), (16, 2, 2, 4096, 96), (2, 3, 2, 3104, 96), (2, 3, 2, 96, 3136), (8, 2, 1, 96, 8192),
    (1, 2, 2, 8192, 64), (8, 32, 4, 160, 1440), (1, 32, 4, 96, 1088),
    (8, 2, 2, 8192, 32), (15, 4, 2, 4352, 32), (13, 64, 3, 32, 32)]


@pytest.mark.parametrize("T,E,k,H,F", SIZES)
def test_layer(T, E, k, H, F):
    run(T, E, k, H, F, x="f32" if (T + E) % 2 else "bf16", y="f32" if T % 2 else "bf16")


@pytest.mark.parametrize("x,norm,residual,y,biases", [("bf16", False, False, "bf16", True),
                                                      ("bf16", False, True, "f32", False),
                                                      ("f32", True, False, "bf16", False),
                                                      ("f32", True, True, "f32", True),
                                                      ("bf16", True, False, "f32", False)])
def test_forms(x, norm, residual, y, biases):
    run(3, 11, 4, 416, 352, x=x, norm=norm, residual=residual, y=y, biases=biases, seed=1)


@pytest.mark.parametrize("T,E,k,H,F", [(16, 16, 16, 64, 4096), (16, 64, 8, 64, 1024), (16, 16, 16, 32, 1440),
                                       (8, 8, 8, 32, 8192)])
def test_rows_pass_the_lds(T, E, k, H, F):
    """More activations than fit at once: the down projection goes by groups of experts."""
    run(T, E, k, H, F, seed=2)


def test_without_the_optional_outputs_and_in_place():
    a = run(4, 8, 2, 192, 128, seed=3)
    want = a.y.clone()
    a.y.fill_(float("nan"))
    a.call(outs=False)
    assert torch.equal(a.y, want)
    a.call(outs=False, y=a.dx)          # y over x
    assert torch.equal(a.dx, want)


def test_every_call_is_the_same():
    a = run(6, 32, 4, 1024, 768, seed=4)
    want = (a.y.clone(), a.ids.clone(), a.gates.clone())
    for _ in range(5):
        a.ws.fill_(0xFF)
        a.y.fill_(float("nan"))
        a.call()
        assert torch.equal(a.y, want[0]) and torch.equal(a.ids, want[1]) and torch.equal(a.gates, want[2])


@pytest.mark.parametrize("F", [288, 1440, 2080])
def test_a_token_does_not_hear_of_the_others(F):
    """The same token alone and in a batch: bit for bit, as its sums take the same order."""
    a = Layer(8, 16, 4, 512, F, seed=5)
    a.call()
    for t in (0, 3, 7):
        b = Layer(8, 16, 4, 512, F, seed=5)
        y = torch.empty((1, 512), dtype=torch.bfloat16, device="cuda")
        B.mxfp4_moe_layer(b.dx[t:t + 1], 1, 512, 16, 4, F, b.drw, b.drb, *b.dgu, b.dbgu, *b.ddown, b.dbd, y,
                          w_norm=b.dw_norm, eps=EPS, residual=True, workspace=b.ws)
        assert torch.equal(y[0], a.y[t])


def test_ties_take_the_lower_expert():
    a = Layer(3, 16, 5, 64, 64, seed=6)
    a.drw[:] = a.drw[:1].clone()
    a.drb.zero_()
    a.drb[[2, 9]] = 1.0
    a.call()
    assert a.ids.cpu().tolist() == [[2, 9, 0, 1, 3]] * 3


def test_rejected_tokens_keep_the_residual():
    """NaN in a token, a NaN or infinite logit: no expert, the residual alone; the others as before."""
    want = Layer(4, 8, 2, 128, 96, seed=7)
    want.call()
    a = Layer(4, 8, 2, 128, 96, seed=7)
    a.dx[1, 5] = float("nan")
    a.dx[2, 9] = float("inf")
    a.call()
    keep = [0, 3]
    assert torch.equal(a.y[keep], want.y[keep]) and torch.equal(a.ids[keep], want.ids[keep])
    assert (a.ids[[1, 2]] == -1).all() and (a.gates[[1, 2]] == 0).all()
    assert torch.equal(a.y[[1, 2]].view(torch.int16)[:, :5], a.dx[[1, 2]].view(torch.int16)[:, :5])
    assert torch.isnan(a.y[1, 5]) and torch.isinf(a.y[2, 9])
    for bias in (float("nan"), float("inf")):
        b = Layer(4, 8, 2, 128, 96, seed=7)
        b.residual = False
        b.drb[3] = bias
        b.call()
        assert (b.ids == -1).all() and (b.gates == 0).all() and (b.y == 0).all()
    b = Layer(4, 8, 2, 128, 96, seed=7)          # -infinity shuts an expert out
    b.drb[3] = float("-inf")
    b.call()
    assert (b.ids != 3).all() and (b.ids >= 0).all() and torch.isfinite(b.y.float()).all()
    b.drb[:] = float("-inf")
    b.drb[3] = 0.0
    b.call()
    assert b.ids.cpu().tolist() == [[3, 0]] * 4 and b.gates.cpu().tolist() == [[1.0, 0.0]] * 4


def test_captured_on_another_stream():
    a = run(5, 16, 3, 352, 288, seed=8)
    ids, gates = a.ids.clone(), a.gates.clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        a.call()
        a.call(y=a.y)
    for seed in (9, 10, 11):
        b = Layer(5, 16, 3, 352, 288, seed=seed)
        a.dx.copy_(b.dx)
        a.x = b.x
        a.y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        a.check()
    with torch.cuda.stream(stream):
        a.call()
    stream.synchronize()
    a.check()
    assert ids.shape == a.ids.shape and gates.shape == a.gates.shape


def test_two_calls_at_once_with_their_own_workspaces():
    cases = [Layer(8, 32, 4, 768, 512, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cases, streams):
            c.call(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()


def test_the_operators_together():
    """The layer of a few tokens beside the same layer by MXFP4 products: norm, router, routing, both
    projections of quantised rows, combine.  The second rounds its rows to 4 bits, so the two agree as
    far as that rounding lets them: the oracle follows the same quantised rows."""
    T, E, k, H, F = 6, 8, 2, 256, 192
    a = run(T, E, k, H, F, seed=30, residual=False, y="f32")
    xn = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    B.moe_norm(a.dx, a.dw_norm, T, H, xn, eps=EPS)
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    off, order = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32,
                                                                                  device="cuda")
    host = a.ids.cpu().numpy().reshape(-1)
    off.copy_(cuda(np.concatenate([[0], np.cumsum(np.bincount(host, minlength=E))]).astype(np.int32)))
    order.copy_(cuda(np.argsort(host, kind="stable").astype(np.int32)))
    xq = (u8(T, H // 32, 16), u8(T, H // 32))
    B.mxfp4_quantize(xn, *xq)
    act = torch.empty((T, k, F), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_expert_matmul_swiglu(*a.dgu, a.dbgu, E, 2 * F, H, *xq, False, T, k, off, order, act)
    aq = (u8(T, k, F // 32, 16), u8(T, k, F // 32))
    B.mxfp4_quantize(act.view(T * k, F), aq[0].view(T * k, F // 32, 16), aq[1].view(T * k, F // 32))
    out = torch.empty((T, k, H), dtype=torch.float32, device="cuda")
    B.mxfp4_expert_matmul(*a.ddown, a.dbd, E, H, F, *aq, True, T, k, off, order, out)
    y = torch.empty((T, H), dtype=torch.float32, device="cuda")
    B.moe_combine(out, a.gates, T, k, H, y)
    # the oracle on the very codes that the kernels wrote
    ids, g = a.ids.cpu().numpy(), a.gates.cpu().numpy().astype(np.float64)
    codes, byte = O.quantize(xn.float().cpu().numpy())
    assert np.array_equal(O.pack(codes), xq[0].cpu().numpy()) and np.array_equal(byte, xq[1].cpu().numpy())
    act_h = act.float().cpu().numpy().astype(np.float64)
    p, mag = O.expert_matmul(O.decode(*a.gu), a.bgu, O.values(codes, byte), False, ids)
    e = (2.0 ** -16 + (H / 64 + 8) * 2.0 ** -23) * mag
    f = M.swiglu(p)
    lo, hi = M.swiglu_range(p - e, p + e)
    dev = np.maximum(hi - f, f - lo)
    assert (np.abs(act_h - f) <= dev + (2.0 ** -8 + 4e-6) * (np.abs(f) + dev) + 2e-5).all()
    codes, byte = O.quantize(act_h)
    o, mag = O.expert_matmul(O.decode(*a.down), a.bd, O.values(codes, byte), True, ids)
    e = (2.0 ** -16 + (F / 64 + 8) * 2.0 ** -23) * mag + 2.0 ** -24 * np.abs(o)
    bound = (g[..., None] * (e + (k + 1) * 2.0 ** -24 * (np.abs(o) + e))).sum(1)
    assert (np.abs(y.cpu().numpy() - (g[..., None] * o).sum(1)) <= bound + 1e-30).all()
