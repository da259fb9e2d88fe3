"""The MXFP4 products and the expert layer on tensors that stand where their interface allows: scale bytes
from any byte on, biases and outputs on the border of their elements only, inside larger buffers whose
other bytes stay as they are.  The same bits as on tensors of their own."""
import numpy as np
import pytest
import torch

import oracle.mx_oracle as O
from mxfp4_mixture_experts_amd import binding as B
from test_gpu_moe_layer import Layer
from test_gpu_mx_matmul import bf16_bias, close, cuda, operand, out_bound
from test_gpu_mx_tiles import SPREAD, grouping, kernel_of

pytestmark = pytest.mark.gpu


def inside(t, off, fill):
    """A copy of t that starts `off` elements into a buffer filled with `fill`, and the buffer."""
    buf = torch.full((t.numel() + 64,), fill, dtype=t.dtype, device="cuda")
    buf[off:off + t.numel()] = t.reshape(-1)
    return buf[off:off + t.numel()].view(t.shape), buf


@pytest.mark.parametrize("off", [1, 7, 15])
@pytest.mark.parametrize("kernel,rows,N,K", [("rows", 5, 66, 416), ((64, 128), 70, 200, 288), ((128, 128), 1030, 2000, 32),
                                             ((128, 256), 2060, 2100, 1056)])
def test_dense(kernel, rows, N, K, off):
    assert kernel_of(rows, N, K) == kernel
    r = np.random.default_rng([71, rows])
    a, b = operand(r, (rows,), K), operand(r, (N,), K)
    bias = bf16_bias(r, N)[1]
    want = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_matmul(*map(cuda, a), *map(cuda, b), rows, N, K, want, bias=bias)
    sa, sb = inside(cuda(a[1]), off, 255)[0], inside(cuda(b[1]), 16 - off, 255)[0]   # beside them: NaN's byte
    out, buf = inside(torch.zeros_like(want), off, 9.0)
    B.mxfp4_matmul(cuda(a[0]), sa, cuda(b[0]), sb, rows, N, K, out, bias=inside(bias, off, float("nan"))[0])
    assert torch.equal(out, want)
    assert (buf[:off] == 9.0).all() and (buf[off + out.numel():] == 9.0).all()


@pytest.mark.parametrize("off", [1, 9])
@pytest.mark.parametrize("kernel,counts,N,K", [("rows", (5, 0, 2, 1), 66, 416), ((64, 128), (60, 0, 70, 96), 200, 288),
                                               ((128, 128), SPREAD, 704, 96), ((128, 256), SPREAD, 1154, 288)])
def test_routed(kernel, counts, N, K, off):
    E, T, k = len(counts), sum(counts) // 2, 2
    assert kernel_of(T * k, N, K, E, T) == kernel
    r = np.random.default_rng([72, T, N])
    w, x = operand(r, (E, N), K), operand(r, (T,), K)
    bias = bf16_bias(r, E, N)[1]
    _, offsets, order = grouping(r, counts)
    offsets, order = cuda(offsets), cuda(order)
    want = torch.empty((T, k, N // 2), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_expert_matmul_swiglu(*map(cuda, w), bias, E, N, K, *map(cuda, x), False, T, k, offsets, order, want)
    out, buf = inside(torch.zeros_like(want), off, 9.0)
    B.mxfp4_expert_matmul_swiglu(cuda(w[0]), inside(cuda(w[1]), off, 255)[0], inside(bias, off, float("nan"))[0], E, N, K,
                                 cuda(x[0]), inside(cuda(x[1]), 16 - off, 255)[0], False, T, k,
                                 inside(offsets, 1, 1 << 30)[0], inside(order, 3, -1)[0], out)
    assert torch.equal(out, want)
    assert (buf[:off] == 9.0).all() and (buf[off + out.numel():] == 9.0).all()


@pytest.mark.parametrize("T,E,k,H,F", [(1, 4, 2, 288, 160), (9, 6, 3, 2880, 96), (3, 5, 2, 4128, 1088)])
def test_layer(T, E, k, H, F):
    a = Layer(T, E, k, H, F, seed=73, y="f32")
    a.call()
    want = (a.y.clone(), a.ids.clone(), a.gates.clone())
    nan = float("nan")
    a.dgu = (a.dgu[0], inside(a.dgu[1], 3, 255)[0])
    a.ddown = (a.ddown[0], inside(a.ddown[1], 13, 255)[0])
    a.dbgu, a.dbd, a.drb = (inside(t, i, nan)[0] for i, t in enumerate((a.dbgu, a.dbd, a.drb), 1))
    outs = [inside(torch.zeros_like(t), 3, 9) for t in want]
    a.y, a.ids, a.gates = (t for t, _ in outs)
    a.call()
    for (t, buf), w in zip(outs, want):
        assert torch.equal(t, w)
        assert (buf[:3] == 9).all() and (buf[3 + t.numel():] == 9).all()


def test_a_token_that_names_an_expert_twice():
    """Both of its slots get the expert's output."""
    r = np.random.default_rng(74)
    E, T, k, N, K = 3, 4, 2, 40, 96
    w, x = operand(r, (E, N), K), operand(r, (T,), K)
    ids = torch.tensor([[1, 1], [0, 2], [2, 2], [1, 0]], dtype=torch.int32, device="cuda")
    offsets, order = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k))
    B.mxfp4_moe_route_group(None, ids, T, E, k, ids.clone(), None, offsets, order)
    out = torch.zeros((T, k, N), device="cuda")
    B.mxfp4_expert_matmul(*map(cuda, w), None, E, N, K, *map(cuda, x), False, T, k, offsets, order, out)
    assert torch.equal(out[0, 0], out[0, 1]) and torch.equal(out[2, 0], out[2, 1])
    want, mag = O.expert_matmul(O.decode(*w), None, O.decode(*x), False, ids.cpu().numpy())
    close(out, want, out_bound(want, mag, K, torch.float32), "out")
