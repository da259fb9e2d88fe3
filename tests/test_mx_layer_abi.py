"""The whole expert layer rejects bad arguments with the documented status before any HIP call; the
binding's own checks.  No GPU needed."""
import ctypes
import os

import pytest
import torch

from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.library_path()), reason="library not built")


def p(v):
    return ctypes.c_void_p(v) if v else None


def _layer(x=64, xt=0, T=2, H=64, E=8, k=2, F=32, wn=64, eps=1e-5, rw=64, rb=64, gb=64, gs=64, gx=64, db=64, ds=64,
           dx=64, res=1, y=64, yt=0, ids=64, gates=64, ws=64, nbytes=1 << 20):
    return B.load_library().mxfp4_moe_layer(p(x), xt, T, H, E, k, F, p(wn), eps, p(rw), p(rb), p(gb), p(gs), p(gx),
                                            p(db), p(ds), p(dx), res, p(y), yt, p(ids), p(gates), p(ws), nbytes, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=17), dict(E=0), dict(E=65), dict(k=0), dict(k=9),
                                dict(E=64, k=17), dict(H=0), dict(H=48), dict(H=8224), dict(F=0), dict(F=-32),
                                dict(F=40), dict(F=8224), dict(T=9, H=8192), dict(T=16, F=4128), dict(xt=2),
                                dict(yt=2), dict(xt=1, wn=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(eps=float("inf")), dict(x=0), dict(rw=0), dict(gb=0), dict(gs=0), dict(db=0),
                                dict(ds=0), dict(y=0), dict(x=72), dict(wn=72), dict(rw=72), dict(gb=72), dict(db=72),
                                dict(rb=65), dict(gx=65), dict(dx=65), dict(y=65), dict(y=66, yt=1), dict(ids=66),
                                dict(gates=66)])
def test_layer_rejects(kw):
    assert _layer(**kw) == 1, kw
    assert B.load_library().mxfp4_last_error() != b""


def test_layer_rejects_the_workspace():
    need = B.mxfp4_moe_layer_workspace_size(2, 64, 8, 2, 32)
    bad = {_layer(ws=0), _layer(nbytes=need - 1), _layer(ws=72)}
    assert len(bad) == 1 and bad.pop() not in (0, 1)


def test_workspace_sizes():
    assert B.mxfp4_moe_layer_workspace_size(0, 64, 8, 2, 32) == 0
    assert B.mxfp4_moe_layer_workspace_size(16, 4096, 64, 16, 4096) >= 16 * 16 * 4096 * 2
    for bad in ((17, 64, 8, 2, 32), (1, 63, 8, 2, 32), (1, 64, 65, 2, 32), (1, 64, 8, 9, 32), (1, 64, 8, 2, 0),
                (16, 8192, 8, 2, 32)):
        with pytest.raises(B.MXFP4Error):
            B.mxfp4_moe_layer_workspace_size(*bad)


def test_nothing_to_do():
    assert _layer(T=0, x=0, y=0, rw=0, gb=0, ws=0, nbytes=0) == 0


def test_binding_checks():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    args = (bf(4, 64), None, u8(4, 64, 2, 16), u8(4, 64, 2), None, u8(4, 64, 1, 16), u8(4, 64, 1), None)
    with pytest.raises(ValueError):     # host tensors
        B.mxfp4_moe_layer(bf(1, 64), 1, 64, 4, 2, 32, *args, bf(1, 64))
    with pytest.raises(B.MXFP4Error):   # sizes past an int32
        B.mxfp4_moe_layer(bf(1, 64), 1 << 31, 64, 4, 2, 32, *args, bf(1, 64))
    with pytest.raises(B.MXFP4Error):
        B.mxfp4_moe_layer_workspace_size(1, 64, 4, 2, 1 << 31)
