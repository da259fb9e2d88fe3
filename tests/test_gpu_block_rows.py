"""Gradients of the norms around the block for batches in which a team of threads takes several rows: a
launch has at most 256 workgroups of at most `teams` teams, so a team takes a second row from
T = 256 * teams + 1 on.  Rows fetched ahead, LDS buffers in turn, gates' gradients written one row late
and the weights' gradients added over rows, teams and workgroups, against the float64 oracle; the last
round of rows leaves some teams without one.

Tolerances as in test_gpu_block_norm.py.  A weight's gradient is added over a team's rows
(ceil(T / (256 teams))), the workgroup's teams, then 4 + 2 + 16 partial sums: under T / 128 + 32
roundings of 2^-24 of the magnitudes' sum, beside what a row's own arithmetic is off by.
"""
import numpy as np
import pytest
import torch

import oracle.block_oracle as O
from mxfp4_mixture_experts_amd import binding as B
from test_gpu_block_norm import (DTYPES, EPS, HALF, TINY, _announce, _backward, _rng, close, dev, f64, make_block,
                                 nan_like, stream_rows, weights, workspace)

pytestmark = pytest.mark.gpu

# T, N and the rows of one round of the launch: parts of a wave (under eight elements, 2 and 16 lanes), one
# wave, two waves, the model's width, one chunk's widest row, two and four chunks a thread
NORMS = [(300001, 5, 131072), (150000, 16, 65536), (20001, 96, 8192), (5000, 512, 2048), (4500, 520, 2048),
         (2500, 1023, 2048), (1111, 2880, 512), (1025, 2881, 512), (1400, 4096, 512), (700, 5000, 256),
         (600, 8192, 256), (600, 9000, 256), (513, 16383, 256)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,rows", NORMS)
def test_norm_backward_rows(T, N, rows, dtype):
    _announce(f"norm_backward rows: T={T} N={N} {dtype}")
    assert T > rows and T % rows
    r = _rng(50, T, N)
    x, w = stream_rows(r, T, N, dtype), weights(r, N)
    dxn = dev(r.normal(size=(T, N)), torch.bfloat16)
    for dres in (None, dev(r.normal(size=(T, N)), dtype)):
        dx, dw = nan_like((T, N), dtype), nan_like((N,), torch.float32)
        B.moe_norm_backward(dxn, x, w, T, N, dx, dw, dres=dres, eps=EPS,
                            workspace=workspace(B.moe_norm_backward_workspace_size(T, N)))
        want, want_w, mag, mag_w = O.norm_backward(f64(dxn), f64(x), f64(w), EPS)
        if dres is not None:
            want, mag = want + f64(dres), mag + np.abs(f64(dres))
        close(dx, want, HALF[dtype] * np.abs(want) + 2.0 ** -17 * mag + TINY, "dx")
        close(dw, want_w, (2.0 ** -18 + (T / 128 + 32) * 2.0 ** -24) * mag_w + TINY, "dw")


# T, k, N: up to four slots' rows held, up to eight, none; one, two and four chunks a thread
BLOCKS = [(17001, 2, 40), (9001, 4, 200), (9001, 7, 200), (5000, 4, 512), (3500, 4, 520), (2500, 8, 520), (2100, 11, 520),
          (1111, 1, 2880), (1111, 4, 2880), (1111, 8, 2880), (600, 9, 2880), (700, 3, 4096), (700, 2, 5000),
          (700, 4, 5000), (600, 5, 5000), (520, 3, 8192), (600, 2, 9000), (520, 1, 16383)]
TYPES = [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("xt,pt", TYPES)
@pytest.mark.parametrize("T,k,N", BLOCKS)
def test_combine_norm_backward_rows(T, k, N, xt, pt):
    _announce(f"combine_norm_backward rows: T={T} k={k} N={N} x {xt} proj {pt}")
    _, gates, proj, _, _, _ = make_block(T, k, N, xt, pt, key=50)
    _backward(T, k, N, xt, pt, True, True, gates, proj, key=50, check=True)


@pytest.mark.parametrize("post,nxt", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("T,k,N", [(9001, 4, 200), (1111, 4, 2880), (600, 9, 2880), (700, 2, 5000), (600, 2, 9000)])
def test_combine_norm_backward_rows_without_a_norm(T, k, N, post, nxt):
    """Without either norm the rows share fewer barriers."""
    _announce(f"combine_norm_backward rows: T={T} k={k} N={N} post={post} next={nxt}")
    _, gates, proj, _, _, _ = make_block(T, k, N, torch.bfloat16, torch.float32, key=51)
    _backward(T, k, N, torch.bfloat16, torch.float32, post, nxt, gates, proj, key=51, check=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [5, 200, 2880, 8192, 9000])
def test_rows_whose_squares_pass_the_range(N, dtype):
    """A row whose sum of squares passes fp32's range has r = 0: its norm is 0, and its gradient what
    came past the norm, whatever its products add up to."""
    _announce(f"rows of huge values, N={N} {dtype}")
    T = 4
    r = _rng(52, N)
    x, w = stream_rows(r, T, N, dtype), weights(r, N)
    x[1] = 3e38
    x[2, ::2], x[2, 1::2] = 1e38, -2e38
    dxn, dres = dev(2.0 + r.random((T, N)), torch.bfloat16), dev(r.normal(size=(T, N)), dtype)
    xn, dx, dw = nan_like((T, N), torch.bfloat16), nan_like((T, N), dtype), nan_like((N,), torch.float32)
    B.moe_norm(x, w, T, N, xn, eps=EPS)
    assert not xn[1:3].any()
    B.moe_norm_backward(dxn, x, w, T, N, dx, dw, dres=dres, eps=EPS,
                        workspace=workspace(B.moe_norm_backward_workspace_size(T, N)))
    assert torch.equal(dx[1:3], dres[1:3])
    others = [0, 3]
    want, want_w, mag, mag_w = O.norm_backward(f64(dxn)[others], f64(x)[others], f64(w), EPS)
    want, mag = want + f64(dres)[others], mag + np.abs(f64(dres)[others])
    close(dx[others], want, HALF[dtype] * np.abs(want) + 2.0 ** -17 * mag + TINY, "dx")
    close(dw, want_w, (2.0 ** -18 + 64 * 2.0 ** -24) * mag_w + TINY, "dw")
    # the next norm of the block's output: the same gradient
    got, got_w = nan_like((T, N), dtype), nan_like((N,), torch.float32)
    proj = dev(r.normal(size=(T, 1, N)))
    B.moe_combine_norm_backward(dres, proj, None, T, 1, N, dx=got, dxn=dxn, x_out=x, w_next=w, dw_next=got_w, eps=EPS,
                                workspace=workspace(B.moe_combine_norm_backward_workspace_size(T, N)))
    assert torch.equal(got[1:3], dres[1:3])
    close(got[others], want, HALF[dtype] * np.abs(want) + 2.0 ** -17 * mag + TINY, "dx")
    close(got_w, want_w, (2.0 ** -18 + 64 * 2.0 ** -24) * mag_w + TINY, "dw_next")
