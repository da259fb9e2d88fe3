"""Products of two MXFP4 operands on the GPU against the float64 oracle on the same codes.

Tolerance.  Products of two E2M1 values and two powers of two are exact.  An MFMA adds the products of
64 or 128 elements to its fp32 accumulator; taken as a sum aligned to its largest term and cut there,
each term may lose 2^-23 of the largest: 128 * 2^-23 of the terms' magnitudes, over all steps at most
that share of their sum; and each step's sum is rounded (2^-23 with cutting), K / 64 times, then a few
more (the waves' partial sums, the bias).  In all (2^-16 + (K / 64 + 8) 2^-23) of the magnitudes' sum,
and the rounding of the output: 2^-8 (bf16) or 2^-24 (fp32) of the value.  Through the activation the
projection's error box is carried exactly (the oracle's swiglu_range), with 2^-8 + 4e-6 relative and 2e-5
for the activation's own arithmetic and rounding, as for the library's other gated projections.
"""
import numpy as np
import pytest
import torch

import oracle.moe_oracle as M
import oracle.mx_oracle as O
from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def sum_bound(mag, K):
    return (2.0 ** -16 + (K / 64 + 8) * 2.0 ** -23) * mag


def out_bound(want, mag, K, dtype):
    e = sum_bound(mag, K)
    return e + HALF[dtype] * (np.abs(want) + e) + 1e-40


def act_bound(p, mag, K):
    e = sum_bound(mag, K)
    f = M.swiglu(p)
    lo, hi = M.swiglu_range(p - e, p + e)
    dev = np.maximum(hi - f, f - lo)
    return dev + (2.0 ** -8 + 4e-6) * (np.abs(f) + dev) + 2e-5


def close(got, want, bound, what):
    g = got.detach().float().cpu().numpy().astype(np.float64)
    err = np.abs(g - want)
    ok = err <= bound
    assert ok.all(), (f"{what}: {int((~ok).sum())} of {ok.size} outside the bound, worst "
                      f"{float(np.nanmax(err / bound)):.3g} times it, first {np.argwhere(~ok)[:3].tolist()}")


def operand(r, shape, K, lo=118, hi=131):
    blocks = r.integers(0, 256, (*shape, K // 32, 16)).astype(np.uint8)
    scales = r.integers(lo, hi, (*shape, K // 32)).astype(np.uint8)
    return blocks, scales


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf16_bias(r, *shape):
    b = O.bf16(r.normal(size=shape))
    return b, torch.from_numpy(b).to(torch.bfloat16).cuda()


def run_matmul(M_, N, K, dtype, bias, seed=0, lo=118, hi=131):
    r = np.random.default_rng([seed, M_, N, K])
    a, b = operand(r, (M_,), K, lo, hi), operand(r, (N,), K, lo, hi)
    hb, db = bf16_bias(r, N) if bias else (None, None)
    out = torch.full((M_, N), float("nan"), dtype=dtype, device="cuda")
    B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), M_, N, K, out, bias=db)
    want, mag = O.matmul(O.decode(*a), O.decode(*b), hb)
    close(out, want, out_bound(want, mag, K, dtype), f"matmul {M_}x{N}x{K}")
    return out


SIZES = [(1, 1, 32), (1, 16, 64), (1, 17, 96), (2, 2880, 2880), (3, 33, 160), (15, 31, 416), (16, 192, 256),
         (17, 5, 32), (17, 193, 288), (33, 64, 64), (64, 191, 1056), (65, 100, 2880), (128, 192, 256), (129, 385, 224),
         (200, 97, 4128), (257, 200, 96), (300, 1023, 512), (513, 576, 2880)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M_,N,K", SIZES)
def test_matmul(M_, N, K, dtype):
    _announce(f"matmul {M_}x{N}x{K} {dtype}")
    run_matmul(M_, N, K, dtype, bias=(M_ + N) % 2 == 0)


@pytest.mark.parametrize("M_,N,K", [(5, 40, 96), (130, 200, 288)])
def test_every_scale_byte(M_, N, K):
    """Scales from the least to the largest whose products stay in range; tiny with tiny."""
    _announce(f"matmul scales {M_}x{N}x{K}")
    r = np.random.default_rng([9, M_])
    for a_range, b_range in (((0, 3), (200, 253)), ((60, 70), (180, 190)), ((250, 255), (0, 5)), ((0, 255), (127, 128))):
        a, b = operand(r, (M_,), K, *a_range), operand(r, (N,), K, *b_range)
        out = torch.empty((M_, N), dtype=torch.float32, device="cuda")
        B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), M_, N, K, out)
        want, mag = O.matmul(O.decode(*a), O.decode(*b))
        keep = mag < 2.0 ** 126
        g = out.cpu().numpy().astype(np.float64)
        assert (np.abs(g - want) <= out_bound(want, mag, K, torch.float32) + 2.0 ** -126)[keep].all()


@pytest.mark.parametrize("M_,N,K", [(4, 50, 96), (16, 30, 2880), (100, 250, 96), (300, 200, 2880)])
def test_nan_blocks(M_, N, K):
    """Byte 255 makes its row's outputs NaN, and no other's."""
    r = np.random.default_rng([11, M_])
    a, b = operand(r, (M_,), K), operand(r, (N,), K)
    rows, cols = [0, M_ - 1], [3, N - 1]
    for i, row in enumerate(rows):
        a[1][row, (K // 32 - 1) if i else 0] = 255
    for i, col in enumerate(cols):
        b[1][col, (K // 32 - 1) if i else 1] = 255
    out = torch.zeros((M_, N), dtype=torch.float32, device="cuda")
    B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), M_, N, K, out)
    got = np.isnan(out.cpu().numpy())
    want = np.zeros((M_, N), bool)
    want[rows], want[:, cols] = True, True
    assert (got == want).all()


def test_rows_behind_the_last_stay():
    for M_ in (3, 40):
        r = np.random.default_rng(12)
        a, b = operand(r, (M_,), 64), operand(r, (100,), 64)
        out = torch.full((M_ + 2, 101), 9.0, dtype=torch.float32, device="cuda")
        B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), M_, 100, 64, out)
        flat = out.view(-1)
        assert (flat[M_ * 100:] == 9.0).all() and not (flat[:M_ * 100] == 9.0).all()


def routing(r, T, E, k, zipf=False, lost=0.0):
    ids = np.empty((T, k), np.int32)
    p = (np.arange(E) + 1.0) ** -1.5 if zipf else np.ones(E)
    for t in range(T):
        ids[t] = r.choice(E, k, replace=False, p=p / p.sum())
    ids[r.random((T, k)) < lost] = -1
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable").astype(np.int32)
    offsets = np.zeros(E + 1, np.int32)
    offsets[1:] = np.cumsum(np.bincount(flat[flat >= 0], minlength=E))
    return ids, offsets, order


EXPERTS = [(1, 4, 2, 32, 32, False), (1, 32, 4, 96, 2880, False), (3, 8, 8, 34, 96, True), (7, 3, 1, 18, 160, False),
           (16, 32, 4, 50, 64, False), (40, 4, 2, 200, 96, True), (64, 32, 4, 194, 288, False),
           (200, 5, 3, 130, 416, True), (300, 70, 2, 66, 96, False), (33, 512, 6, 20, 64, False),
           (700, 2, 2, 386, 512, False), (1000, 8, 4, 100, 1056, True)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("T,E,k,N,K,zipf", EXPERTS)
def test_expert_matmul(T, E, k, N, K, zipf, per_slot):
    _announce(f"expert matmul T={T} E={E} k={k} N={N} K={K} per_slot={per_slot}")
    r = np.random.default_rng([21, T, E, k, N, K])
    w, x = operand(r, (E, N), K), operand(r, (T, k) if per_slot else (T,), K)
    hb, db = bf16_bias(r, E, N)
    ids, offsets, order = routing(r, T, E, k, zipf, lost=0.05)
    want, mag = O.expert_matmul(O.decode(*w), hb, O.decode(*x), per_slot, ids)
    args = (*map(cuda, w), db, E, N, K, *map(cuda, x), per_slot, T, k, cuda(offsets), cuda(order))
    routed = ids >= 0
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((T, k, N), 7.0, dtype=dtype, device="cuda")
        B.mxfp4_expert_matmul(*args, out)
        close(out[torch.from_numpy(routed)], want[routed], out_bound(want[routed], mag[routed], K, dtype), "out")
        assert (out[torch.from_numpy(~routed)] == 7.0).all()
    act = torch.full((T, k, N // 2), 7.0, dtype=torch.bfloat16, device="cuda")
    B.mxfp4_expert_matmul_swiglu(*args, act)
    close(act[torch.from_numpy(routed)], M.swiglu(want[routed]), act_bound(want[routed], mag[routed], K), "act")
    assert (act[torch.from_numpy(~routed)] == 7.0).all()


@pytest.mark.parametrize("T", [6, 300])
def test_no_bias_and_odd_width(T):
    r = np.random.default_rng([22, T])
    E, k, N, K = 4, 2, 71, 96
    w, x = operand(r, (E, N), K), operand(r, (T,), K)
    ids, offsets, order = routing(r, T, E, k)
    want, mag = O.expert_matmul(O.decode(*w), None, O.decode(*x), False, ids)
    out = torch.empty((T, k, N), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_expert_matmul(*map(cuda, w), None, E, N, K, *map(cuda, x), False, T, k, cuda(offsets), cuda(order), out)
    close(out, want, out_bound(want, mag, K, torch.bfloat16), "out")


@pytest.mark.parametrize("T", [4, 200])
def test_bad_groupings_stay_inside(T):
    """Offsets past the rows and rows out of range are clamped or skipped; every other row is right."""
    r = np.random.default_rng([23, T])
    E, k, N, K = 3, 2, 40, 64
    w, x = operand(r, (E, N), K), operand(r, (T,), K)
    ids, offsets, order = routing(r, T, E, k)
    bad_rows = order.copy()
    bad_rows[1], bad_rows[-1] = T * k + 5, -3
    bad_off = offsets.copy()
    bad_off[-1] = 1 << 30
    out = torch.full((T, k, N), 7.0, dtype=torch.float32, device="cuda")
    B.mxfp4_expert_matmul(*map(cuda, w), None, E, N, K, *map(cuda, x), False, T, k, cuda(bad_off), cuda(bad_rows), out)
    want, mag = O.expert_matmul(O.decode(*w), None, O.decode(*x), False, ids)
    want, mag = want.reshape(T * k, N), mag.reshape(T * k, N)
    keep = np.ones(T * k, bool)
    keep[order[1]] = keep[order[-1]] = False
    flat = out.view(T * k, N)
    close(flat[torch.from_numpy(keep)], want[keep], out_bound(want[keep], mag[keep], K, torch.float32), "out")
    assert (flat[torch.from_numpy(~keep)] == 7.0).all()
    empty = torch.full((T, k, N), 7.0, dtype=torch.float32, device="cuda")
    B.mxfp4_expert_matmul(*map(cuda, w), None, E, N, K, *map(cuda, x), False, T, k, cuda(np.zeros(E + 1, np.int32)),
                          cuda(order), empty)
    assert (empty == 7.0).all()


def test_gradients_of_a_linear_layer():
    """Both gradient products of y = x . w^T through the two quantisers, against float64 on what they
    store; and their distance from the unquantised gradients is the format's (2^-2 of a block's
    largest, far above the sum's rounding)."""
    r = np.random.default_rng(31)
    T, N, K = 96, 160, 64
    x, w, dy = (torch.from_numpy(r.normal(size=s).astype(np.float32)).to(torch.bfloat16).cuda()
                for s in ((T, K), (N, K), (T, N)))

    def packed(t, transposed):
        rows, k = (t.shape[1], t.shape[0]) if transposed else t.shape
        q = (torch.empty((rows, k // 32, 16), dtype=torch.uint8, device="cuda"),
             torch.empty((rows, k // 32), dtype=torch.uint8, device="cuda"))
        v = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda")
        (B.mxfp4_quantize_transposed if transposed else B.mxfp4_quantize)(t, *q, values=v)
        return q, v.float().cpu().numpy().astype(np.float64)

    dyq, dyv = packed(dy, False)
    wt, wtv = packed(w, True)
    dyt, dytv = packed(dy, True)
    xt, xtv = packed(x, True)
    dx = torch.empty((T, K), dtype=torch.float32, device="cuda")
    dw = torch.empty((N, K), dtype=torch.float32, device="cuda")
    B.mxfp4_matmul(*dyq, *wt, T, K, N, dx)
    B.mxfp4_matmul(*dyt, *xt, N, K, T, dw)
    for got, a, b, n, full in ((dx, dyv, wtv, N, dy.float() @ w.float()), (dw, dytv, xtv, T, dy.float().t() @ x.float())):
        want, mag = O.matmul(a, b)
        close(got, want, out_bound(want, mag, n, torch.float32), "gradient")
        true = full.cpu().numpy()
        assert np.abs(got.cpu().numpy() - true).std() < 0.3 * true.std()


def test_captured_and_on_another_stream():
    r = np.random.default_rng(41)
    for M_ in (2, 200):
        a, b = operand(r, (M_,), 288), operand(r, (200,), 288)
        da, db_ = tuple(map(cuda, a)), tuple(map(cuda, b))
        out = torch.empty((M_, 200), dtype=torch.float32, device="cuda")
        B.mxfp4_matmul(*da, *db_, M_, 200, 288, out)
        want = out.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            B.mxfp4_matmul(*da, *db_, M_, 200, 288, out)
        for _ in range(3):
            out.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        out2 = torch.empty_like(out)
        B.mxfp4_matmul(*da, *db_, M_, 200, 288, out2, stream=side)
        side.synchronize()
        assert torch.equal(out2, want)
