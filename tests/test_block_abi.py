"""The norms around the block and the routing's balance reject bad arguments with the
documented status before any HIP call; workspace sizes; the binding's own checks.  No GPU needed."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from mxfp4_mixture_experts_amd import binding as B
from test_abi_sanitized import _runtime

pytestmark = pytest.mark.skipif(not os.path.exists(B.library_path()), reason="library not built")

BAD_SIZE = ctypes.c_size_t(-1).value
BIG = ctypes.c_size_t(1 << 40)
NAN, INF = float("nan"), float("inf")


def p(v=64):
    return ctypes.c_void_p(v) if v else None


def _norm(T=4, N=64, eps=1e-5, x=64, xt=0, w=64, xn=64):
    return B.load_library().moe_norm(p(x), xt, p(w), T, N, eps, p(xn), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(N=0), dict(N=16385), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN),
                                dict(eps=INF), dict(xt=2), dict(xt=-1), dict(x=0), dict(w=0), dict(xn=0), dict(x=63),
                                dict(x=66, xt=1), dict(w=65), dict(xn=65)])
def test_norm_rejects(kw):
    assert _norm(**kw) == 1, kw
    assert B.load_library().mxfp4_last_error() != b""


def _norm_bwd(T=4, N=64, eps=1e-5, dxn=64, x=64, xt=0, w=64, dres=0, dx=64, dw=64, ws=64, nbytes=BIG):
    return B.load_library().moe_norm_backward(p(dxn), p(x), xt, p(w), p(dres), T, N, eps, p(dx), p(dw), p(ws), nbytes,
                                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(N=0), 1), (dict(N=16385), 1), (dict(eps=0.0), 1), (dict(xt=3), 1), (dict(dxn=0), 1),
    (dict(x=0), 1), (dict(w=0), 1), (dict(dx=0), 1), (dict(dres=65), 1), (dict(dw=66), 1), (dict(dx=66, xt=1), 1),
    (dict(ws=0), 2), (dict(nbytes=ctypes.c_size_t(4 * 64 * 4 - 1)), 2), (dict(ws=72), 2),
])
def test_norm_backward_rejects(kw, status):
    assert _norm_bwd(**kw) == status, kw


def _comb(T=4, k=4, N=64, eps=1e-5, scale=1.0, proj=64, pt=1, gates=64, w_post=64, x=64, xt=0, x_out=64, w_next=64,
          xn=64):
    return B.load_library().moe_combine_norm(p(proj), pt, p(gates), T, k, N, p(w_post), p(x), xt, scale, eps, p(x_out),
                                             p(w_next), p(xn), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(k=0), dict(k=33), dict(N=0), dict(N=16385), dict(T=1 << 27, k=32), dict(eps=0.0), dict(scale=INF),
    dict(scale=NAN), dict(pt=2), dict(xt=2), dict(proj=0), dict(x=0), dict(x_out=0), dict(w_next=0), dict(xn=0),
    dict(proj=66), dict(gates=66), dict(w_post=65), dict(x=65), dict(x_out=66, xt=1), dict(w_next=65), dict(xn=65),
])
def test_combine_norm_rejects(kw):
    assert _comb(**kw) == 1, kw


def _comb_bwd(T=4, k=4, N=64, eps=1e-5, scale=1.0, dx_out=64, dxn=64, x_out=64, w_next=64, proj=64, pt=1, gates=64,
              w_post=64, xt=0, dx=64, dproj=64, dgates=64, dw_post=64, dw_next=64, ws=64, nbytes=BIG):
    return B.load_library().moe_combine_norm_backward(
        p(dx_out), p(dxn), p(x_out), p(w_next), p(proj), pt, p(gates), T, k, N, p(w_post), xt, scale, eps, p(dx),
        p(dproj), p(dgates), p(dw_post), p(dw_next), p(ws), nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(k=0), 1), (dict(k=33), 1), (dict(N=16385), 1), (dict(eps=NAN), 1), (dict(scale=INF), 1),
    (dict(pt=5), 1), (dict(xt=5), 1), (dict(gates=0), 1), (dict(w_post=0), 1), (dict(dx_out=0, dxn=0, dw_next=0), 1),
    (dict(x_out=0), 1), (dict(w_next=0), 1), (dict(dxn=0), 1), (dict(proj=0), 1), (dict(dproj=66), 1),
    (dict(dgates=66), 1), (dict(dw_post=66), 1), (dict(dw_next=66), 1), (dict(dx=66, xt=1), 1),
    (dict(ws=0), 2), (dict(nbytes=ctypes.c_size_t(2 * 4 * 64 * 4 - 1)), 2), (dict(ws=72), 2),
    (dict(ws=0, dw_post=0), 2),
])
def test_combine_norm_backward_rejects(kw, status):
    assert _comb_bwd(**kw) == status, kw


def _bal(T=8, E=32, k=4, S=1, logits=64, ids=64, seq=0, counts=64, tokens=64, losses=64, ws=64, nbytes=BIG):
    return B.load_library().moe_balance(p(logits), p(ids), T, E, k, p(seq), S, p(counts), p(tokens), p(losses), p(ws),
                                        nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(T=(1 << 30) + 1, k=1), 1), (dict(T=1 << 29, k=8), 1), (dict(E=0), 1), (dict(E=513), 1),
    (dict(k=0), 1), (dict(k=5, E=4), 1), (dict(k=33, E=64), 1), (dict(S=0), 1), (dict(S=2), 1),
    (dict(S=1 << 28, seq=64), 1), (dict(logits=0), 1), (dict(ids=0), 1), (dict(counts=0), 1), (dict(tokens=0), 1),
    (dict(losses=0), 1), (dict(logits=65), 1), (dict(ids=66), 1), (dict(seq=66), 1), (dict(counts=66), 1),
    (dict(tokens=66), 1), (dict(losses=66), 1), (dict(ws=0), 2), (dict(ws=72), 2),
    (dict(nbytes=ctypes.c_size_t(16)), 2), (dict(T=0, ws=0), 2),
])
def test_balance_rejects(kw, status):
    assert _bal(**kw) == status, kw


def _rb(T=8, E=32, k=4, S=1, logits=64, ids=64, gates=64, dgates=64, seq=0, counts=64, tokens=64, dlosses=64,
        dlogits=64, dt=1):
    return B.load_library().moe_route_backward(p(logits), p(ids), p(gates), p(dgates), T, E, k, p(seq), S, p(counts),
                                               p(tokens), p(dlosses), p(dlogits), dt, None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(E=0), dict(E=513), dict(k=0), dict(k=33, E=64), dict(S=0), dict(S=2), dict(dt=2), dict(ids=0),
    dict(dlogits=0), dict(gates=0), dict(dgates=0, dlosses=0), dict(logits=0), dict(counts=0), dict(tokens=0),
    dict(logits=65), dict(ids=66), dict(gates=66), dict(dgates=66), dict(dlosses=66), dict(dlogits=66), dict(seq=66),
])
def test_route_backward_rejects(kw):
    assert _rb(**kw) == 1, kw


def test_no_tokens_is_a_noop():
    assert _norm(T=0, x=0, w=0, xn=0) == 0
    assert _norm_bwd(T=0, dxn=0, x=0, w=0, dx=0, dw=0, ws=0) == 0
    assert _comb(T=0, proj=0, gates=0, x=0, x_out=0) == 0
    assert _comb_bwd(T=0, dx_out=0, dxn=0, proj=0, dw_post=0, dw_next=0, ws=0) == 0
    assert _rb(T=0, logits=0, ids=0, gates=0, dgates=0, dlosses=0, counts=0, tokens=0, dlogits=0) == 0
    # nothing asked for
    assert _comb_bwd(dx=0, dproj=0, dgates=0, dw_post=0, dw_next=0, ws=0) == 0


def test_workspace_sizes():
    lib = B.load_library()
    nb, cb, bal = (lib.moe_norm_backward_workspace_size, lib.moe_combine_norm_backward_workspace_size,
                   lib.moe_balance_workspace_size)
    assert nb(0, 64) == 0 and cb(0, 64) == 0          # no rows, no sums
    assert nb(4096, 2880) > 0 and cb(4096, 2880) == 2 * nb(4096, 2880)
    assert nb(1 << 30, 16384) == nb(1 << 20, 16384) <= 64 << 20      # bounded by the launch, not by the rows
    for args in ((-1, 64), (4, 0), (4, 16385)):
        assert nb(*args) == BAD_SIZE and cb(*args) == BAD_SIZE
    assert bal(0, 32, 1) > 0 and bal(4096, 32, 1) > bal(0, 32, 1)
    assert bal(4096, 32, 9) > bal(4096, 32, 1)
    for args in ((-1, 32, 1), (4, 0, 1), (4, 513, 1), (4, 32, 0), (4, 512, 1 << 23), ((1 << 30) + 1, 32, 1)):
        assert bal(*args) == BAD_SIZE, args
    with pytest.raises(B.MXFP4Error):
        B.moe_balance_workspace_size(4, 0, 1)


def test_binding_rejects_host_tensors():
    x, w, y = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_norm(x, w, 2, 8, x)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_combine_norm(y, None, 2, 1, 8, x, x)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_balance(x, w, 2, 8, 1, w, w, w)


@pytest.mark.skipif(shutil.which("g++") is None or os.environ.get("MXFP4_MOE_LIB") is not None,
                    reason="g++ not available, or already a child of this test")
def test_under_host_sanitizers():
    """The refusals above against the host-sanitizer build of the C-ABI layer."""
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not (asan and ubsan):
        pytest.skip("sanitizer runtimes not installed")
    from mxfp4_mixture_experts_amd import build_lib
    env = dict(os.environ)
    env.update({"MXFP4_MOE_LIB": build_lib.build_host_sanitized(), "LD_PRELOAD": f"{asan} {ubsan}",
                "ASAN_OPTIONS": "detect_leaks=0:abort_on_error=1",
                "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1", "HIP_VISIBLE_DEVICES": ""})
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                         capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    text = res.stdout + res.stderr
    assert res.returncode == 0, text[-4000:]
    assert "AddressSanitizer" not in text and "runtime error" not in text, text[-4000:]
