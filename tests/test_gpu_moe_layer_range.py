"""The expert layer of a few tokens where numbers leave the ordinary range: NaN blocks, every scale byte,
an infinity at a row's end, an eps below fp32's normal numbers.

Tolerances are those of test_gpu_moe_layer (intervals carried through the layer).  Outputs near fp32's
least numbers have 2^-149 for each product and sum besides (their spacing there).
"""
import numpy as np
import pytest
import torch

import oracle.moe_oracle as M
import oracle.mx_oracle as O
from mxfp4_mixture_experts_amd import binding as B
from test_gpu_moe_layer import Layer, cuda, rounded, sums

pytestmark = pytest.mark.gpu

SIZES = [(4, 8, 2, 128, 96), (9, 6, 3, 288, 160), (16, 8, 2, 2880, 96), (3, 5, 2, 4128, 1088)]  # T, E, k, H, F


@pytest.mark.parametrize("T,E,k,H,F", SIZES)
@pytest.mark.parametrize("row", ["gate", "up", "down"])
def test_a_nan_block_reaches_its_tokens_only(T, E, k, H, F, row):
    """Scale byte 255: a gate or up row makes every output of the expert's tokens NaN, a down row one
    output; every other value keeps its bits."""
    a = Layer(T, E, k, H, F, seed=40)
    a.call()
    clean, ids = a.y.clone(), a.ids.clone()
    expert = int(ids[0, k - 1])
    tokens = (ids == expert).any(1).cpu().numpy()
    for block in (0, (F if row == "down" else H) // 32 - 1):
        b = Layer(T, E, k, H, F, seed=40)
        out = 7 % H
        if row == "down":
            b.ddown[1][expert, out, block] = 255
        else:
            b.dgu[1][expert, 2 * (F - 1) + (row == "up"), block] = 255
        b.call()
        assert torch.equal(b.ids, ids)
        want = np.zeros((T, H), bool)
        if row == "down":
            want[tokens, out] = True
        else:
            want[tokens] = True
        got = torch.isnan(b.y).cpu().numpy()
        assert (got == want).all(), (int((got & ~want).sum()), int((want & ~got).sum()))
        keep = torch.from_numpy(~want).cuda()
        assert torch.equal(b.y[keep], clean[keep])


@pytest.mark.parametrize("T,E,k,H,F", [(3, 6, 3, 288, 160), (8, 4, 2, 416, 1088)])
def test_the_least_scales_of_gate_and_up(T, E, k, H, F):
    """Bytes 0..2 under normed rows of 2^126: the projections are ordinary numbers again."""
    a = Layer(T, E, k, H, F, norm=False, residual=False, y="f32", seed=41)
    a.x = O.bf16(np.random.default_rng(41).normal(size=(T, H)) * 2.0 ** 122)
    a.rw = O.bf16(a.rw * 2.0 ** -122)
    r = np.random.default_rng(42)
    a.gu = (a.gu[0], r.integers(0, 3, a.gu[1].shape).astype(np.uint8))
    a.dx, a.drw, a.dgu = cuda(a.x).to(torch.bfloat16), cuda(a.rw).to(torch.bfloat16), tuple(map(cuda, a.gu))
    a.call()
    a.check()


@pytest.mark.parametrize("T,E,k,H,F", [(3, 6, 3, 288, 160), (8, 4, 2, 96, 1088)])
@pytest.mark.parametrize("lo,hi", [(0, 1), (0, 3), (1, 20), (240, 248)])
def test_the_scales_of_the_down_projection(T, E, k, H, F, lo, hi):
    a = Layer(T, E, k, H, F, residual=False, y="f32", biases=False, seed=43)
    r = np.random.default_rng(44)
    a.down = (a.down[0], r.integers(lo, hi, a.down[1].shape).astype(np.uint8))
    a.ddown = tuple(map(cuda, a.down))
    a.call()
    ids, g = a.ids.cpu().numpy(), a.gates.cpu().numpy().astype(np.float64)
    xn, exn = a.x / np.sqrt(np.mean(a.x * a.x, -1, keepdims=True) + 1e-5) * a.w_norm, None
    xn, exn = rounded(xn, np.abs(xn) * (H / 64 + 20) * 2.0 ** -24)
    w_gu, w_down = O.decode(*a.gu), O.decode(*a.down)
    p, mag = O.expert_matmul(w_gu, None, xn, False, ids)
    ep = O.expert_matmul(np.abs(w_gu), None, exn, False, ids)[0] + sums(mag, H)
    f = M.swiglu(p)
    lo_f, hi_f = M.swiglu_range(p - ep, p + ep)
    ef = np.maximum(hi_f - f, f - lo_f)
    act, ea = rounded(f, ef + 4e-6 * (np.abs(f) + ef) + 2e-5)
    o, mag_o = O.expert_matmul(w_down, None, act, True, ids)
    eo = O.expert_matmul(np.abs(w_down), None, ea, True, ids)[0] + sums(mag_o, F)
    h, size = (g[..., None] * o).sum(1), (g[..., None] * mag_o).sum(1)
    bound = (g[..., None] * eo).sum(1) + (2 * k + 20) * 2.0 ** -23 * size * 1.01 + (F + 40) * 2.0 ** -149
    got = a.y.cpu().numpy().astype(np.float64)
    err = np.abs(got - h)
    assert (err <= bound).all(), float(np.nanmax(err / bound))


@pytest.mark.parametrize("H,F", [(288, 160), (2880, 96), (4128, 96), (544, 1088)])
def test_an_infinity_at_the_end_of_a_row(H, F):
    """The last element of a normed row is infinite: every logit is -infinity, so the token's experts are
    the first, and every gate and up sum is +infinity, which the activation brings to its limit."""
    T, E, k = 3, 4, 2
    a = Layer(T, E, k, H, F, norm=False, residual=False, y="f32", seed=45)
    a.drw[:, -1] = -1.0
    a.dx[1, -1] = float("inf")
    codes = a.gu[0].copy()
    codes[..., -1, 15] = (codes[..., -1, 15] & 0x0f) | 0x20      # the last weight of every row: +1
    a.dgu = (cuda(codes), a.dgu[1])
    a.call()
    assert a.ids[1].tolist() == [0, 1] and a.gates[1].tolist() == [0.5, 0.5]
    act = np.full((1, k, F), M.swiglu(np.array([np.inf, np.inf]))[0])
    ids = np.array([[0, 1]])
    o, mag = O.expert_matmul(O.decode(*a.down), a.bd, O.bf16(act), True, ids)
    size = 0.5 * mag.sum(1)
    err = np.abs(a.y[1].cpu().numpy() - 0.5 * o.sum(1)[0])
    assert (err <= 0.5 * sums(mag, F).sum(1)[0] + (2 * k + 15) * 2.0 ** -23 * size[0]).all()


@pytest.mark.parametrize("eps", [1e-42, 1e-39, 2.0 ** -126])
def test_an_eps_below_the_normal_numbers(eps):
    """A row of zeros stays zeros under any eps, as in moe_norm: its experts are the router bias's."""
    a = Layer(4, 8, 2, 288, 160, seed=46)
    a.dx[1:3] = 0.0
    want, ids = None, None
    for e in (1e-5, eps):
        a.y.fill_(float("nan"))
        B.mxfp4_moe_layer(a.dx, *a.s, a.drw, a.drb, *a.dgu, a.dbgu, *a.ddown, a.dbd, a.y, w_norm=a.dw_norm, eps=e,
                          residual=True, topk_ids=a.ids, gates=a.gates, workspace=a.ws)
        if want is None:
            want, ids = a.y[1:3].clone(), a.ids[1:3].clone()
    assert (a.ids >= 0).all()
    assert torch.equal(a.y[1:3], want) and torch.equal(a.ids[1:3], ids)
    assert torch.isfinite(a.y.float()).all()
