"""NaN blocks (scale byte 255) through the routed products and the gated activation: NaN in the outputs
whose row of weights or of activations holds one and in no other; every other output keeps its bits."""
import numpy as np
import pytest
import torch

import oracle.moe_oracle as M
from mxfp4_mixture_experts_amd import binding as B
from test_gpu_mx_matmul import bf16_bias, cuda, operand
from test_gpu_mx_tiles import SPREAD, grouping, kernel_of

pytestmark = pytest.mark.gpu

CASES = [("rows", (2, 2, 1, 1), 66, 288), ("rows", (27, 20, 11, 1, 5) + (0,) * 35, 50, 4128),
         ((64, 128), (60, 0, 70, 96), 200, 96), ((128, 128), SPREAD, 704, 544), ((128, 256), SPREAD, 1154, 288)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("kernel,counts,N,K", CASES)
def test_routed(kernel, counts, N, K, per_slot):
    E, T, k = len(counts), sum(counts) // 2, 2
    print(f"[case] {sum(counts)} rows, {E} experts, {N}x{K} per_slot={per_slot}", flush=True)
    assert kernel_of(T * k, N, K, E, T) == kernel
    r = np.random.default_rng([61, T, N, K])
    w, x = operand(r, (E, N), K), operand(r, (T, k) if per_slot else (T,), K)
    _, db = bf16_bias(r, E, N)
    ids, offsets, order = grouping(r, counts)
    last = K // 32 - 1
    bad_w, bad_x = w[1].copy(), x[1].copy()
    rows_of_w = [(0, 2, 0), (0, N - 1, last), (E - 1 if counts[-1] else 2, 7, last // 2)]   # gate, up, up
    for e, n, block in rows_of_w:
        bad_w[e, n, block] = 255
    flat = bad_x.reshape(-1, K // 32)
    flat[0, last], flat[-1, 0] = 255, 255
    p = np.zeros((T, k, N))
    for e, n, _ in rows_of_w:
        p[ids == e, n] = np.nan
    p.reshape(len(flat), -1)[[0, -1]] = np.nan

    def run(ws, xs):
        args = (cuda(w[0]), cuda(ws), db, E, N, K, cuda(x[0]), cuda(xs), per_slot, T, k, cuda(offsets), cuda(order))
        outs = [torch.zeros((T, k, N), dtype=d, device="cuda") for d in (torch.float32, torch.bfloat16)]
        for out in outs:
            B.mxfp4_expert_matmul(*args, out)
        act = torch.zeros((T, k, N // 2), dtype=torch.bfloat16, device="cuda")
        B.mxfp4_expert_matmul_swiglu(*args, act)
        return (*outs, act)

    for got, clean, want in zip(run(bad_w, bad_x), run(w[1], x[1]), (p, p, M.swiglu(p))):
        nan = np.isnan(want)
        assert not torch.isnan(clean).any()
        seen = torch.isnan(got).cpu().numpy()
        assert (seen == nan).all(), (int((seen & ~nan).sum()), int((nan & ~seen).sum()))
        keep = torch.from_numpy(~nan).cuda()
        assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("M_,N,K", [(1030, 2000, 96), (2060, 2100, 544)])
def test_dense(M_, N, K):
    r = np.random.default_rng([62, M_])
    a, b = operand(r, (M_,), K), operand(r, (N,), K)
    args = lambda: (*map(cuda, a), *map(cuda, b), M_, N, K)
    clean, got = (torch.zeros((M_, N), dtype=torch.float32, device="cuda") for _ in range(2))
    B.mxfp4_matmul(*args(), clean)
    a[1][0, 0] = a[1][M_ - 1, K // 32 - 1] = b[1][3, 1] = b[1][N - 1, K // 32 - 1] = 255
    B.mxfp4_matmul(*args(), got)
    want = torch.zeros((M_, N), dtype=torch.bool, device="cuda")
    want[[0, M_ - 1]], want[:, [3, N - 1]] = True, True
    assert torch.equal(torch.isnan(got), want) and torch.equal(got[~want], clean[~want])


@pytest.mark.parametrize("kernel,T", [("rows", 3), ((64, 128), 200)])
def test_a_nan_of_a_tensor_reaches_the_down_projection(kernel, T):
    """Quantised rows that hold a NaN or an infinity, through the gated activation, quantised again and
    through the down projection: their tokens' outputs are NaN to the end."""
    E, k, H, F = 4, 2, 96, 64
    r = np.random.default_rng([63, T])
    x = torch.from_numpy(r.normal(size=(T, H)).astype(np.float32)).cuda()
    x[0, 5], x[T - 1, H - 1] = float("nan"), float("-inf")
    counts = np.array([T, T, 0, 0])
    _, offsets, order = grouping(r, counts)
    assert kernel_of(T * k, 2 * F, H, E, T) == kernel
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    gu, down = tuple(map(cuda, operand(r, (E, 2 * F), H))), tuple(map(cuda, operand(r, (E, H), F)))
    xq, aq = (u8(T, H // 32, 16), u8(T, H // 32)), (u8(T, k, F // 32, 16), u8(T, k, F // 32))
    act = torch.empty((T, k, F), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((T, k, H), dtype=torch.float32, device="cuda")
    B.mxfp4_quantize(x, *xq)
    B.mxfp4_expert_matmul_swiglu(*gu, None, E, 2 * F, H, *xq, False, T, k, cuda(offsets), cuda(order), act)
    B.mxfp4_quantize(act, *aq)
    B.mxfp4_expert_matmul(*down, None, E, H, F, *aq, True, T, k, cuda(offsets), cuda(order), out)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[0, T - 1]] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
