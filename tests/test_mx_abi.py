"""The MXFP4 quantisation and the products of two MXFP4 operands reject bad arguments with the
documented status before any HIP call; the binding's own checks.  No GPU needed."""
import ctypes
import os

import pytest
import torch

from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.library_path()), reason="library not built")


def p(v=64):
    return ctypes.c_void_p(v) if v else None


def _q(x=64, xt=0, rows=4, K=64, blocks=64, scales=64, values=64):
    return B.load_library().mxfp4_quantize(p(x), xt, rows, K, p(blocks), p(scales), p(values), None)


@pytest.mark.parametrize("kw", [dict(xt=2), dict(xt=-1), dict(rows=-1), dict(K=0), dict(K=16), dict(K=-32), dict(K=33),
                                dict(rows=1 << 45), dict(x=0), dict(blocks=0), dict(scales=0), dict(x=72),
                                dict(blocks=72), dict(values=72)])
def test_quantize_rejects(kw):
    assert _q(**kw) == 1, kw
    assert B.load_library().mxfp4_last_error() != b""


def _qt(x=64, xt=0, R=64, C=7, blocks=64, scales=64, values=64):
    return B.load_library().mxfp4_quantize_transposed(p(x), xt, R, C, p(blocks), p(scales), p(values), None)


@pytest.mark.parametrize("kw", [dict(xt=2), dict(R=-32), dict(R=33), dict(R=(1 << 30) + 32), dict(C=-1),
                                dict(C=(1 << 21) + 1), dict(R=1 << 30, C=1 << 20), dict(x=0), dict(blocks=0),
                                dict(scales=0), dict(x=65), dict(x=66, xt=1), dict(blocks=72), dict(values=72)])
def test_quantize_transposed_rejects(kw):
    assert _qt(**kw) == 1, kw


def _mm(ab=64, as_=64, bb=64, bs=64, bias=64, M=4, N=5, K=64, out=64, ot=1):
    return B.load_library().mxfp4_matmul(p(ab), p(as_), p(bb), p(bs), p(bias), M, N, K, p(out), ot, None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(M=(1 << 30) + 1), dict(N=0), dict(N=(1 << 27) + 1), dict(K=0),
                                dict(K=48), dict(K=1 << 26), dict(M=1 << 24, N=1 << 20), dict(ot=2), dict(ab=0),
                                dict(as_=0), dict(bb=0), dict(bs=0), dict(out=0), dict(ab=72), dict(bb=72),
                                dict(bias=65), dict(out=66), dict(out=65, ot=0)])
def test_matmul_rejects(kw):
    assert _mm(**kw) == 1, kw


def _em(swiglu=False, blocks=64, scales=64, bias=64, E=4, N=6, K=64, xb=64, xs=64, per=0, T=4, k=2, off=64, rows=64,
        out=64, ot=1):
    lib = B.load_library()
    args = (p(blocks), p(scales), p(bias), E, N, K, p(xb), p(xs), per, T, k, p(off), p(rows), p(out))
    return lib.mxfp4_expert_matmul_swiglu(*args, None) if swiglu else lib.mxfp4_expert_matmul(*args, ot, None)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kw", [dict(E=0), dict(E=513), dict(N=0), dict(N=(1 << 27) + 2), dict(K=0), dict(K=40),
                                dict(K=1 << 26), dict(T=-1), dict(k=0), dict(k=5), dict(k=33, E=64),
                                dict(T=1 << 30, k=2), dict(T=1 << 28, N=1 << 20), dict(blocks=0), dict(scales=0),
                                dict(xb=0), dict(xs=0), dict(off=0), dict(rows=0), dict(out=0), dict(blocks=72),
                                dict(xb=72), dict(bias=65), dict(off=66), dict(rows=66), dict(out=65)])
def test_expert_matmul_rejects(kw, swiglu):
    assert _em(swiglu, **kw) == 1, kw


def test_types_of_the_outputs():
    assert _em(ot=2) == 1 and _em(out=66) == 1
    assert _em(True, N=5) == 1          # gate and up rows go in pairs


def test_nothing_to_do():
    assert _q(rows=0, x=0, blocks=0, scales=0) == 0
    assert _qt(R=0, x=0, blocks=0, scales=0) == 0 and _qt(C=0, x=0, blocks=0, scales=0) == 0
    assert _mm(M=0, ab=0, as_=0, out=0) == 0
    assert _em(T=0, xb=0, xs=0, out=0) == 0 and _em(True, T=0, xb=0, out=0) == 0


def test_binding_checks():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):     # host tensors
        B.mxfp4_quantize(x, u8(4, 2, 16), u8(4, 2))
    with pytest.raises(ValueError):
        B.mxfp4_quantize_transposed(x.view(-1), u8(4, 2, 16), u8(4, 2))
    with pytest.raises(ValueError):
        B.mxfp4_matmul(u8(4, 2, 16), u8(4, 2), u8(4, 2, 16), u8(4, 2), 4, 4, 64, torch.zeros(4, 4))
    with pytest.raises(B.MXFP4Error):   # sizes past an int32
        B.mxfp4_matmul(u8(4, 2, 16), u8(4, 2), u8(4, 2, 16), u8(4, 2), 1 << 31, 4, 64, torch.zeros(4, 4))
    with pytest.raises(B.MXFP4Error):
        B.mxfp4_expert_matmul(u8(1), u8(1), None, 1, 4, 64, u8(1), u8(1), False, 1 << 32, 1, u8(1), u8(1),
                              torch.zeros(4))
