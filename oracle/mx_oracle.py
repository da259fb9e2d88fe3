"""CPU oracle for the MXFP4 quantisation, the products of two MXFP4 operands and
the whole expert layer of a few tokens.

TEST INFRASTRUCTURE ONLY: the tests and the smoke check import it.  The
definitions written out in float64 with numpy; it shares no code with the
library.  Pinned by tests/test_mx_oracle.py to brute force over the 16 codes,
closed forms and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from . import moe_oracle as M

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# borders between neighbouring magnitudes; at a border the even code wins
BORDERS = (GRID[1:] + GRID[:-1]) / 2
EVEN_BELOW = np.array([True, False, True, False, True, False, True])


def quantize(x):
    """(codes [..., K], scale bytes [..., K / 32]) of x along its last axis."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.frexp(amax)[1] - 1 - 2          # floor(log2 amax) - 2
    e = np.where(amax > 0, np.maximum(e, -127), -127)
    a = np.ldexp(np.abs(b), -e[..., None])
    code = np.zeros(b.shape, np.uint8)
    for border, even_below in zip(BORDERS, EVEN_BELOW):
        code += (a > border) if even_below else (a >= border)
    code |= np.signbit(b).astype(np.uint8) << 3
    code = np.where(bad[..., None], 0, code).astype(np.uint8)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(x.shape), byte


def pack(codes):
    """Blocks [..., K / 32, 16] of codes [..., K], the even element in the low nibble."""
    c = codes.reshape(*codes.shape[:-1], -1, 16, 2)
    return (c[..., 0] | (c[..., 1] << 4)).astype(np.uint8)


def values(codes, byte):
    """What codes [..., K] stand for under scale bytes [..., K / 32]; NaN under byte 255."""
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    f = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return (v.reshape(*byte.shape, 32) * f[..., None]).reshape(codes.shape)


def unpack(blocks):
    """Codes [..., K] of blocks [..., K / 32, 16]."""
    c = np.stack([blocks & 15, blocks >> 4], -1)
    return c.reshape(*blocks.shape[:-2], -1)


def decode(blocks, byte):
    return values(unpack(blocks), byte)


def matmul(a, b, bias=None):
    """(a . b^T + bias, sum of |terms|)."""
    out, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        out, mag = out + bias, mag + np.abs(bias)
    return out, mag


def expert_matmul(w, bias, x, x_per_slot, ids):
    """Projections [T, k, N] of each slot through its expert and the sums of |terms|; NaN where the
    id is out of range.  w [E, N, K], x [T, K] or [T, k, K]."""
    T, k = ids.shape
    out = np.full((T, k, w.shape[1]), np.nan)
    mag = np.zeros_like(out)
    for e in range(w.shape[0]):
        t, s = np.nonzero(ids == e)
        if len(t):
            rows = x[t, s] if x_per_slot else x[t]
            out[t, s], mag[t, s] = matmul(rows, w[e], None if bias is None else bias[e])
    return out, mag


def bf16(x):
    """x rounded to bf16, to nearest even (finite x within the range), as float64."""
    m, e = np.frexp(np.asarray(x, np.float64))
    e8 = np.maximum(e, -125)
    return np.ldexp(np.rint(np.ldexp(m, e - e8 + 8)), e8 - 8)


def layer_route(x, w_norm, eps, router_w, router_b, k):
    """(xn, logits, ids, gates): the normed rows rounded to bf16, the float64 logits, the k largest
    (ties to the lower index) and the softmax over them."""
    x = np.asarray(x, np.float64)
    xn = x
    if w_norm is not None:
        xn = bf16(x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w_norm)
    logits = xn @ router_w.T + (0.0 if router_b is None else router_b)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(logits, ids, 1)
    g = np.exp(top - top[:, :1])
    return xn, logits, ids, g / g.sum(1, keepdims=True)


def layer(xn, ids, gates, w_gu, b_gu, w_down, b_down):
    """(h [T, H], bound-carrying magnitudes): the gate-weighted sum of the experts' outputs on the
    normed rows.  Returns also the act before rounding and its projection's magnitudes."""
    p, mag_p = expert_matmul(w_gu, b_gu, xn, False, ids)
    act = M.swiglu(p)
    out, mag_out = expert_matmul(w_down, b_down, bf16(act), True, ids)
    h = (gates[..., None] * out).sum(1)
    return h, (gates[..., None] * mag_out).sum(1), act, p, mag_p
