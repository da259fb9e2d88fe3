"""The kernels of the MXFP4 products that test_gpu_mx_matmul's sizes do not reach: the tiles of 128 rows
(128 x 128 and 128 x 256), dense and routed, with every number of row sub-tiles, tails of K of both
parities, ragged and odd widths; and the second passes of the kernel for few rows.

Which kernel a size takes is computed here as the launch rule has it, and asserted case by case.
Tolerances are those of test_gpu_mx_matmul, derived there for any K.
"""
import numpy as np
import pytest
import torch

import oracle.moe_oracle as M
import oracle.mx_oracle as O
from mxfp4_mixture_experts_amd import binding as B
from test_gpu_mx_matmul import act_bound, bf16_bias, close, cuda, operand, out_bound, run_matmul

pytestmark = pytest.mark.gpu


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def kernel_of(rows, N, K, experts=0, tokens=0):
    """The kernel of a product of so many rows, outputs and inputs (of so many tokens, routed to so many
    experts): "rows" or the tile's rows and outputs."""
    groups = min(experts, rows) if experts else 1
    light = groups * -(-N // 16) <= (1024 if K > 1024 else 512) or (K >= 2560 and K % 256)
    if light and (rows <= 2 * groups and tokens <= 32 if experts else rows <= 16):
        return "rows"

    def tiles(tm, tn):
        return (rows // tm + min(experts, rows) if experts else -(-rows // tm)) * -(-N // tn)

    if tiles(64, 128) <= 256 or (experts and rows <= 32 * groups):
        return 64, 128
    return (128, 128) if tiles(128, 128) <= 256 else (128, 256)


def grouping(r, counts):
    """(ids [rows / 2, 2], offsets, order) of rows spread at random over experts with these counts."""
    order = r.permutation(sum(counts)).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    ids = np.empty(len(order), np.int32)
    for e in range(len(counts)):
        part = order[offsets[e]:offsets[e + 1]]
        part.sort()
        ids[part] = e
    return ids.reshape(-1, 2), offsets, order


# rows % 128 in 1..32, ..64, ..96, ..128; K's stages of 256: one, broken and whole, and last ones of either parity
DENSE = [((128, 128), 1025, 2000, 32), ((128, 128), 1057, 2000, 96), ((128, 128), 1089, 1993, 256),
         ((128, 128), 1121, 2000, 288), ((128, 128), 1152, 1921, 544), ((128, 128), 1030, 1990, 1056),
         ((128, 128), 1088, 2048, 2880), ((128, 128), 1100, 1925, 512),
         ((128, 256), 2049, 2100, 32), ((128, 256), 2081, 2101, 96), ((128, 256), 2113, 2048, 256),
         ((128, 256), 2145, 2060, 288), ((128, 256), 2176, 2305, 544), ((128, 256), 2060, 2100, 1056),
         ((128, 256), 2100, 2304, 2880), ((128, 256), 2112, 2087, 512), ((128, 256), 4097, 1200, 800)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kernel,rows,N,K", DENSE)
def test_dense_tiles(kernel, rows, N, K, dtype):
    _announce(f"matmul {rows}x{N}x{K} {dtype}")
    assert kernel_of(rows, N, K) == kernel
    run_matmul(rows, N, K, dtype, bias=(N + K // 32) % 2 == 0)


SPREAD = (1, 0, 33, 65, 97, 128, 129, 161, 193, 225, 256, 512, 0, 300)   # 2100 rows
ROUTED = [((128, 128), SPREAD, 700, 96), ((128, 128), SPREAD, 704, 288), ((128, 128), SPREAD, 650, 1056),
          ((128, 256), SPREAD, 1150, 96), ((128, 256), SPREAD, 1152, 288), ((128, 256), SPREAD, 1154, 544),
          ((128, 256), (1500, 2, 500, 98), 1670, 1056), ((128, 256), (0, 0, 3000), 1410, 320)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("kernel,counts,N,K", ROUTED)
def test_routed_tiles(kernel, counts, N, K, per_slot):
    _announce(f"expert matmul {sum(counts)} rows, {len(counts)} experts, {N}x{K} per_slot={per_slot}")
    check_routed(kernel, counts, N, K, per_slot)


# 2 rows an expert and fewer on average, all in a few: several groups of 16, and K beyond one pass of 24 steps of 128
FEW = [((27, 20, 11, 1, 5) + (0,) * 35, 50, 96), ((16, 33, 1) + (0,) * 22, 34, 2880), ((2, 2, 1, 1), 66, 4128),
       ((40,) + (0,) * 19, 18, 6240), ((1, 1) + (0,) * 30, 2880, 6176), ((17, 3) + (0,) * 8, 64, 8224)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("counts,N,K", FEW)
def test_few_rows_in_several_passes(counts, N, K, per_slot):
    _announce(f"expert matmul {counts[:5]}.. of {len(counts)} experts, {N}x{K} per_slot={per_slot}")
    check_routed("rows", counts, N, K, per_slot)


# as few rows, where the smallest tiles take them: too many workgroups, aligned rows, too many tokens
TILED = [((1, 2, 0, 1) * 16, 1100, 96), ((2, 1, 0, 1) * 8, 800, 2560), ((1,) * 20 + (0,) * 12, 1700, 1024),
         ((37, 20, 17, 1, 5) + (0,) * 35, 50, 96), ((64, 10) + (0,) * 40, 34, 2880)]


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("counts,N,K", TILED)
def test_few_rows_in_tiles(counts, N, K, per_slot):
    _announce(f"expert matmul {counts[:5]}.. of {len(counts)} experts, {N}x{K} per_slot={per_slot}")
    check_routed((64, 128), counts, N, K, per_slot)


@pytest.mark.parametrize("rows,N,K", [(1, 8200, 96), (16, 8201, 1024), (3, 16390, 2048), (7, 16400, 2560)])
def test_few_dense_rows_in_tiles(rows, N, K):
    _announce(f"matmul {rows}x{N}x{K}")
    assert kernel_of(rows, N, K) == (64, 128)
    run_matmul(rows, N, K, torch.float32, bias=True)


@pytest.mark.parametrize("rows,N,K", [(1, 40, 4128), (16, 33, 6240), (5, 5760, 3136), (9, 17, 9248)])
def test_few_dense_rows_of_a_long_k(rows, N, K):
    _announce(f"matmul {rows}x{N}x{K}")
    assert kernel_of(rows, N, K) == "rows"
    run_matmul(rows, N, K, torch.float32, bias=True)


def check_routed(kernel, counts, N, K, per_slot):
    E, T, k = len(counts), sum(counts) // 2, 2
    assert kernel_of(T * k, N, K, E, T) == kernel
    r = np.random.default_rng([51, T, E, N, K])
    w, x = operand(r, (E, N), K), operand(r, (T, k) if per_slot else (T,), K)
    hb, db = bf16_bias(r, E, N)
    ids, offsets, order = grouping(r, counts)
    want, mag = O.expert_matmul(O.decode(*w), hb, O.decode(*x), per_slot, ids)
    args = (*map(cuda, w), db, E, N, K, *map(cuda, x), per_slot, T, k, cuda(offsets), cuda(order))
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((T, k, N), float("nan"), dtype=dtype, device="cuda")
        B.mxfp4_expert_matmul(*args, out)
        close(out, want, out_bound(want, mag, K, dtype), "out")
    act = torch.full((T, k, N // 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_expert_matmul_swiglu(*args, act)
    close(act, M.swiglu(want), act_bound(want, mag, K), "act")


@pytest.mark.parametrize("kernel,rows,N,K", [((128, 128), 1030, 2000, 96), ((128, 256), 2060, 2100, 288)])
def test_every_scale_byte(kernel, rows, N, K):
    """Scales from the least to the largest whose products stay in range; tiny with tiny."""
    assert kernel_of(rows, N, K) == kernel
    r = np.random.default_rng([52, rows])
    for a_range, b_range in (((0, 3), (200, 253)), ((60, 70), (180, 190)), ((250, 255), (0, 5)), ((0, 255), (127, 128))):
        a, b = operand(r, (rows,), K, *a_range), operand(r, (N,), K, *b_range)
        out = torch.empty((rows, N), dtype=torch.float32, device="cuda")
        B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), rows, N, K, out)
        want, mag = O.matmul(O.decode(*a), O.decode(*b))
        keep = mag < 2.0 ** 126
        err = np.abs(out.cpu().numpy().astype(np.float64) - want)
        assert (err <= out_bound(want, mag, K, torch.float32) + 2.0 ** -126)[keep].all()


@pytest.mark.parametrize("kernel,counts,N", [("rows", (27, 20, 11, 1, 5) + (0,) * 35, 50), ((128, 128), SPREAD, 700),
                                             ((128, 256), SPREAD, 1150)])
def test_bad_groupings_stay_inside(kernel, counts, N):
    """Offsets past the rows and rows out of range are clamped or skipped; every other row is right."""
    E, T, k, K = len(counts), sum(counts) // 2, 2, 64
    assert kernel_of(T * k, N, K, E, T) == kernel
    r = np.random.default_rng([53, T, N])
    w, x = operand(r, (E, N), K), operand(r, (T,), K)
    ids, offsets, order = grouping(r, counts)
    bad_rows, bad_off = order.copy(), offsets.copy()
    lost = [order[1], order[T], order[-1]]
    bad_rows[1], bad_rows[T], bad_rows[-1] = T * k, 1 << 30, -3
    bad_off[0], bad_off[-1] = -5, 1 << 30
    out = torch.full((T, k, N), 7.0, dtype=torch.float32, device="cuda")
    B.mxfp4_expert_matmul(*map(cuda, w), None, E, N, K, *map(cuda, x), False, T, k, cuda(bad_off), cuda(bad_rows), out)
    want, mag = O.expert_matmul(O.decode(*w), None, O.decode(*x), False, ids)
    want, mag = want.reshape(T * k, N), mag.reshape(T * k, N)
    keep = np.ones(T * k, bool)
    keep[lost] = False
    flat = out.view(T * k, N)
    close(flat[torch.from_numpy(keep)], want[keep], out_bound(want[keep], mag[keep], K, torch.float32), "out")
    assert (flat[torch.from_numpy(~keep)] == 7.0).all()


@pytest.mark.parametrize("kernel,rows,N", [((128, 128), 1030, 2000), ((128, 256), 2060, 2100)])
def test_nothing_behind_the_outputs_is_written(kernel, rows, N):
    assert kernel_of(rows, N, 64) == kernel
    r = np.random.default_rng([54, rows])
    a, b = operand(r, (rows,), 64), operand(r, (N,), 64)
    out = torch.full((rows * N + 4096,), 9.0, dtype=torch.float32, device="cuda")
    B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), rows, N, 64, out)
    assert (out[rows * N:] == 9.0).all()
    off = torch.full((rows * N + 4096,), 9.0, dtype=torch.bfloat16, device="cuda")[1:]   # not on a 16-byte border
    B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), rows, N, 64, off)
    assert (off[rows * N:] == 9.0).all()
    assert torch.equal(off[:rows * N], out[:rows * N].bfloat16())


@pytest.mark.parametrize("kernel,rows,N,K", [((128, 128), 1030, 2000, 288), ((128, 256), 2060, 2100, 544)])
def test_captured(kernel, rows, N, K):
    assert kernel_of(rows, N, K) == kernel
    r = np.random.default_rng([55, rows])
    a, b = tuple(map(cuda, operand(r, (rows,), K))), tuple(map(cuda, operand(r, (N,), K)))
    out = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_matmul(*a, *b, rows, N, K, out)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.mxfp4_matmul(*a, *b, rows, N, K, out)
    for _ in range(3):
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
