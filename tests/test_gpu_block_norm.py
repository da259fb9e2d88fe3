"""GPU parity of the norms around the expert block (moe_norm, moe_combine_norm and their
gradients) through the C ABI, against the float64 oracle.

Tolerances.  An output is rounded once to its type: at most 2^-8 (bf16) or 2^-24 (fp32) of the
value.  Before it comes fp32 arithmetic, each operation within 2^-24 of its result:
 - a row's sum of squares adds at most 32 elements in a thread, 6 lane exchanges, 8 waves: under 46
   roundings, all of one sign; half of that reaches r, with 2 for the hardware's reciprocal square
   root and 4 products: under 2^-19 of xn in all;
 - a gradient's terms (G, dh) pass two such row sums and under 64 more operations: 2^-17 of the sum of
   their magnitudes, which the oracle carries along (2^-16 behind the output norm, where the rounding
   of h moves r as well: the oracle's magnitudes hold that factor);
 - the weights' sums add a team's rows (one where T <= 256 times the teams of a workgroup), the
   workgroup's teams (at most T / 256 + 1) and 4 + 2 + 16 sums of workgroups: under T / 512 + 64
   roundings at the sizes here.
"""
import numpy as np
import pytest
import torch

import oracle.block_oracle as O
from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.gpu

EPS = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-36


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def _rng(*key):
    return np.random.default_rng(np.random.SeedSequence(20, spawn_key=key))


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype).contiguous()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def nan_like(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def close(got, want, bound, what):
    g = f64(got)
    assert g.shape == want.shape
    err = np.abs(g - want)
    ok = err <= bound
    assert np.all(ok), (f"{what}: {int((~ok).sum())} of {ok.size} outside the bound, worst "
                        f"{float(np.nanmax(err / (bound + TINY))):.3g} times it, first {np.argwhere(~ok)[:3].tolist()}")


def stream_rows(r, T, N, dtype):
    """Rows of unlike size with a few large channels."""
    x = r.normal(size=(T, N)) * np.exp(0.7 * r.normal(size=(T, 1)))
    x[:, r.random(N) < 0.01] *= 40.0
    return dev(x, dtype)


def weights(r, N):
    return dev(1.0 + 0.3 * r.normal(size=N), torch.bfloat16)


def workspace(nbytes):
    return torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device="cuda")   # NaN patterns


# T, N: one element, one chunk with and without a tail, wave and workgroup borders, odd widths, the
# model's width, the widest rows of one, two and four chunks a thread
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 63), (4, 512), (3, 513), (1, 2880), (7, 2880), (6, 2881), (33, 2879), (2, 4096),
          (3, 4097), (2, 8192), (2, 8193), (3, 16383), (2, 16384), (600, 96), (1500, 520)]
DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N", SHAPES)
def test_norm(T, N, dtype):
    _announce(f"norm T={T} N={N} {dtype}")
    r = _rng(1, T, N)
    x, w = stream_rows(r, T, N, dtype), weights(r, N)
    xn = nan_like((T, N), torch.bfloat16)
    B.moe_norm(x, w, T, N, xn, eps=EPS)
    want = O.norm(f64(x), f64(w), EPS)
    close(xn, want, (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + TINY, "xn")


def test_norm_small_rows_and_eps():
    """eps decides a row of small values; a row of zeros gives zeros."""
    _announce("norm: zero and small rows")
    N = 300
    x = np.zeros((4, N))
    x[1] = 1e-4
    x[2] = -1e-6
    x[3, 5] = 1e-3
    for dtype in DTYPES:
        xd, w = dev(x, dtype), weights(_rng(2), N)
        for eps in (1e-5, 1e-12):
            xn = nan_like((4, N), torch.bfloat16)
            B.moe_norm(xd, w, 4, N, xn, eps=eps)
            want = O.norm(f64(xd), f64(w), np.float64(np.float32(eps)))
            close(xn, want, (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + TINY, f"xn eps={eps}")
            assert not f64(xn)[0].any()


def test_norm_nan_and_inf_stay_in_their_row():
    _announce("norm: NaN and inf rows")
    r = _rng(3)
    x = stream_rows(r, 5, 2880, torch.bfloat16)
    x[1, 17] = float("nan")
    x[3, 2879] = float("inf")
    w = weights(r, 2880)
    xn = nan_like((5, 2880), torch.bfloat16)
    B.moe_norm(x, w, 5, 2880, xn, eps=EPS)
    g = f64(xn)
    assert np.isnan(g[1]).all() and np.isnan(g[3, 2879]) and not np.delete(g[3], 2879).any()
    for t in (0, 2, 4):
        want = O.norm(f64(x)[t:t + 1], f64(w), EPS)[0]
        assert np.all(np.abs(g[t] - want) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_rows_off_16_bytes(offset, dtype):
    """Tensors that begin between 16-byte borders: the same bits as aligned copies, and nothing
    before or behind them is written."""
    _announce(f"norm: storage offset {offset} {dtype}")
    r = _rng(4, offset)
    T, N = 9, 2880
    x, w = stream_rows(r, T, N, dtype), weights(r, N)
    want = nan_like((T, N), torch.bfloat16)
    B.moe_norm(x, w, T, N, want, eps=EPS)

    def shifted(t):
        flat = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device="cuda")
        flat[offset:offset + t.numel()] = t.reshape(-1)
        return flat, flat[offset:offset + t.numel()].view(t.shape)

    _, xs = shifted(x)
    _, ws = shifted(w)
    flat, xn = shifted(want * 0)
    B.moe_norm(xs, ws, T, N, xn, eps=EPS)
    assert torch.equal(xn, want)
    assert bool((flat[:offset] == 7).all()) and bool((flat[offset + T * N:] == 7).all())
    flat, xo = shifted(x * 0)
    _, proj = shifted(dev(r.normal(size=(T, 2, N))))
    gates = dev(r.random((T, 2)))
    want_o = nan_like((T, N), dtype)
    B.moe_combine_norm(proj.clone(), gates, T, 2, N, x, want_o, w_post=w, eps=EPS)
    B.moe_combine_norm(proj, gates, T, 2, N, xs, xo, w_post=ws, eps=EPS)
    assert torch.equal(xo, want_o)
    assert bool((flat[:offset] == 7).all()) and bool((flat[offset + T * N:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N", SHAPES)
def test_norm_backward(T, N, dtype):
    _announce(f"norm_backward T={T} N={N} {dtype}")
    r = _rng(5, T, N)
    x, w = stream_rows(r, T, N, dtype), weights(r, N)
    dxn = dev(r.normal(size=(T, N)), torch.bfloat16)
    dres = dev(r.normal(size=(T, N)), dtype) if T % 2 else None
    dx, dw = nan_like((T, N), dtype), nan_like((N,), torch.float32)
    ws = workspace(B.moe_norm_backward_workspace_size(T, N))
    B.moe_norm_backward(dxn, x, w, T, N, dx, dw, dres=dres, eps=EPS, workspace=ws)
    want, want_w, mag, mag_w = O.norm_backward(f64(dxn), f64(x), f64(w), EPS)
    if dres is not None:
        want, mag = want + f64(dres), mag + np.abs(f64(dres))
    close(dx, want, HALF[dtype] * np.abs(want) + 2.0 ** -17 * mag + TINY, "dx")
    close(dw, want_w, (2.0 ** -18 + (T / 512 + 64) * 2.0 ** -24) * mag_w + TINY, "dw")
    # in place over dres, and without dw
    if dres is not None:
        B.moe_norm_backward(dxn, x, w, T, N, dres, None, dres=dres, eps=EPS)
        assert torch.equal(dres, dx)


def routing(r, T, k, lost=0.2):
    g = r.random((T, k)).astype(np.float32) + 0.05
    g /= g.sum(1, keepdims=True)
    g[r.random((T, k)) < lost] = 0.0
    return g


# T, k, N
BLOCKS = [(1, 1, 1), (3, 2, 7), (1, 4, 2880), (9, 4, 2880), (4, 3, 2881), (5, 8, 96), (5, 9, 520), (2, 32, 130),
          (2, 5, 4097), (3, 2, 8192), (2, 3, 9000), (2, 1, 16384), (2, 4, 16383), (700, 4, 104)]


def make_block(T, k, N, xt, pt, key=0, lost=0.2):
    r = _rng(6, T, k, N, key)
    gates = routing(r, T, k, lost)
    proj = r.normal(size=(T, k, N))
    proj[gates == 0] = np.nan                       # an unrouted slot's row is never written
    return r, dev(gates), dev(proj, pt), stream_rows(r, T, N, xt), weights(r, N), weights(r, N)


def unit_bound(h, mag, k, w):
    """How far the output norm of the combine may be off: the combine's k roundings move h itself
    and, through the sum of squares, r."""
    r = 1.0 / np.sqrt(np.mean(h * h, -1, keepdims=True) + EPS)
    moved = (np.abs(h) * mag).sum(-1, keepdims=True) / np.maximum((h * h).sum(-1, keepdims=True), 1e-300)
    return r * np.abs(w) * (k * 2.0 ** -24 * mag + np.abs(h) * (2.0 ** -19 + k * 2.0 ** -24 * moved))


@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("xt,pt", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,k,N", BLOCKS)
def test_combine_norm(T, k, N, xt, pt, post, nxt):
    _announce(f"combine_norm T={T} k={k} N={N} x {xt} proj {pt} post={post} next={nxt}")
    r, gates, proj, x, w_post, w_next = make_block(T, k, N, xt, pt)
    w_post = w_post if post else None
    scale = 0.37
    x_out = nan_like((T, N), xt)
    xn = nan_like((T, N), torch.bfloat16) if nxt else None
    B.moe_combine_norm(proj, gates, T, k, N, x, x_out, w_post=w_post, scale=scale, w_next=w_next if nxt else None,
                       xn=xn, eps=EPS)
    h, mag = O.combine(f64(proj), f64(gates))
    u = h if w_post is None else O.norm(h, f64(w_post), EPS)
    off = k * 2.0 ** -24 * mag if w_post is None else unit_bound(h, mag, k, f64(w_post))
    s = float(np.float32(scale))
    want = f64(x) + s * u
    close(x_out, want, HALF[xt] * np.abs(want) * 1.01 + s * off * 1.01 + 2.0 ** -23 * (np.abs(f64(x)) + np.abs(s * u))
          + TINY, "x_out")
    if nxt:
        want = O.norm(f64(x_out), f64(w_next), EPS)          # the norm of what was stored
        close(xn, want, (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + TINY, "xn")
        same = nan_like((T, N), torch.bfloat16)
        B.moe_norm(x_out, w_next, T, N, same, eps=EPS)
        assert torch.equal(xn, same), "not the bits of moe_norm"
    # in place over x
    B.moe_combine_norm(proj, gates, T, k, N, x, x, w_post=w_post, scale=scale, eps=EPS)
    assert torch.equal(x, x_out)


def test_combine_norm_is_moe_combine():
    """x = 0, scale 1, no norm: the bits of moe_combine; gates None: a plain sum."""
    _announce("combine_norm against moe_combine")
    for T, k, N in [(5, 4, 2880), (3, 7, 33)]:
        _, gates, proj, _, _, _ = make_block(T, k, N, torch.float32, torch.float32, key=1)
        y, x_out = nan_like((T, N), torch.float32), nan_like((T, N), torch.float32)
        B.moe_combine(proj, gates, T, k, N, y)
        B.moe_combine_norm(proj, gates, T, k, N, torch.zeros_like(y), x_out)
        assert torch.equal(y, x_out)
        one = proj[:, 0].contiguous().nan_to_num()
        B.moe_combine_norm(one, None, T, 1, N, torch.zeros_like(y), x_out)
        assert torch.equal(one, x_out)


def test_unrouted_token_keeps_its_stream():
    _announce("combine_norm: a token without a routed slot")
    T, k, N = 3, 4, 2880
    r, gates, proj, x, w_post, w_next = make_block(T, k, N, torch.bfloat16, torch.float32, key=2)
    gates[1] = 0.0
    proj[1] = float("nan")
    x_out, xn = nan_like((T, N), torch.bfloat16), nan_like((T, N), torch.bfloat16)
    B.moe_combine_norm(proj, gates, T, k, N, x, x_out, w_post=w_post, scale=0.5, w_next=w_next, xn=xn, eps=EPS)
    assert torch.equal(x_out[1], x[1]) and bool(torch.isfinite(xn.float()).all())
    out = _backward(T, k, N, torch.bfloat16, torch.float32, True, True, gates=gates, proj=proj)
    assert not out["dproj"][1].any() and not out["dgates"][1].any()
    assert all(bool(torch.isfinite(v.float()).all()) for v in out.values())


def _backward(T, k, N, xt, pt, post, nxt, gates, proj, key=3, check=False, want_all=True):
    r = _rng(7, T, k, N, key)
    x_out, w_post, w_next = stream_rows(r, T, N, xt), weights(r, N), weights(r, N)
    dx_out = dev(r.normal(size=(T, N)), xt) if (T + k) % 3 or not nxt else None
    dxn = dev(r.normal(size=(T, N)), torch.bfloat16)
    scale = 0.37
    o = {"dx": nan_like((T, N), xt), "dproj": nan_like((T, k, N), pt), "dgates": nan_like((T, k), torch.float32)}
    if post:
        o["dw_post"] = nan_like((N,), torch.float32)
    if nxt:
        o["dw_next"] = nan_like((N,), torch.float32)
    args = dict(w_post=w_post if post else None, scale=scale, eps=EPS,
                workspace=workspace(B.moe_combine_norm_backward_workspace_size(T, N)))
    if nxt:
        args.update(dxn=dxn, x_out=x_out, w_next=w_next)
    B.moe_combine_norm_backward(dx_out, proj, gates, T, k, N, **o, **args)
    if check:
        s = float(np.float32(scale))
        w = O.combine_norm_backward(None if dx_out is None else f64(dx_out), f64(dxn) if nxt else None, f64(x_out),
                                    f64(w_next), f64(proj), f64(gates), f64(w_post) if post else None, s, EPS)
        rows = (T / 512 + 64) * 2.0 ** -24
        close(o["dx"], w["dx"], HALF[xt] * np.abs(w["dx"]) * 1.01 + 2.0 ** -17 * w["mag_dx"] + TINY, "dx")
        close(o["dproj"], w["dproj"], HALF[pt] * np.abs(w["dproj"]) * 1.01 + 2.0 ** -16 * w["mag_dproj"] + TINY, "dproj")
        close(o["dgates"], w["dgates"], (2.0 ** -16 + 2.0 ** -18) * w["mag_dgates"] + TINY, "dgates")
        if post:
            close(o["dw_post"], w["dw_post"], (2.0 ** -16 + rows) * w["mag_post"] + TINY, "dw_post")
        if nxt:
            close(o["dw_next"], w["dw_next"], (2.0 ** -18 + rows) * w["mag_next"] + TINY, "dw_next")
        # one output at a time, each with the bits that it has beside the others
        for name in o:
            one = {name: torch.full_like(o[name], float("nan"))}
            B.moe_combine_norm_backward(dx_out, proj, gates, T, k, N, **one, **args)
            assert torch.equal(one[name], o[name]), name
        if dx_out is not None:
            B.moe_combine_norm_backward(dx_out, proj, gates, T, k, N, dx=dx_out, **args)     # in place
            assert torch.equal(dx_out, o["dx"])
    return o


@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("xt,pt", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,k,N", BLOCKS)
def test_combine_norm_backward(T, k, N, xt, pt, post, nxt):
    _announce(f"combine_norm_backward T={T} k={k} N={N} x {xt} proj {pt} post={post} next={nxt}")
    _, gates, proj, _, _, _ = make_block(T, k, N, xt, pt, key=3)
    _backward(T, k, N, xt, pt, post, nxt, gates, proj, check=True)


def test_unrouted_slot_of_an_infinite_gradient():
    """A gradient that holds an infinity or a NaN still leaves an unrouted slot's dproj and dgate 0."""
    _announce("combine_norm_backward: infinite gradient, unrouted slot")
    for N in (64, 2880):
        T, k = 3, 2
        gates = dev([[0.5, 0.0], [0.0, 0.0], [0.25, 0.75]])
        proj = dev(np.ones((T, k, N)))
        proj[0, 1] = proj[1] = float("nan")
        dx_out = dev(np.ones((T, N)))
        dx_out[0, 3], dx_out[1, 5] = float("inf"), float("nan")
        dproj, dgates = nan_like((T, k, N), torch.float32), nan_like((T, k), torch.float32)
        B.moe_combine_norm_backward(dx_out, proj, gates, T, k, N, dproj=dproj, dgates=dgates)
        assert not dproj[0, 1].any() and not dproj[1].any() and not dgates[0, 1].any() and not dgates[1].any()
        assert float(dproj[0, 0, 3]) == float("inf") and torch.equal(dproj[2, 1], torch.full((N,), 0.75, device="cuda"))
        assert torch.equal(dgates[2], torch.full((k,), float(N), device="cuda"))


def test_combine_norm_backward_dense():
    """k = 1 without gates: a dense block's output."""
    _announce("combine_norm_backward: gates None")
    T, N = 12, 520
    r = _rng(8)
    proj, dx_out, w = dev(r.normal(size=(T, 1, N))), dev(r.normal(size=(T, N))), weights(r, N)
    dproj = nan_like((T, 1, N), torch.float32)
    B.moe_combine_norm_backward(dx_out, proj, None, T, 1, N, dproj=dproj, w_post=w, scale=0.5, eps=EPS)
    w64 = O.combine_norm_backward(f64(dx_out), None, None, None, f64(proj), np.ones((T, 1)), f64(w), 0.5, EPS)
    close(dproj, w64["dproj"], 2.0 ** -16 * w64["mag_dproj"], "dproj")


def test_no_rows_give_zero_weight_gradients():
    _announce("backward of no rows")
    N = 2881
    dw, dw2 = nan_like((N,), torch.float32), nan_like((N,), torch.float32)
    e = torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    B.moe_norm_backward(e, e, w, 0, N, e, dw, eps=EPS)
    assert not dw.any()
    B.moe_combine_norm_backward(e, torch.empty((0, 2, N), device="cuda"), None, 0, 2, N, w_post=w, dw_post=dw.fill_(3),
                                dxn=e, x_out=e, w_next=w, dw_next=dw2, eps=EPS)
    assert not dw.any() and not dw2.any()


def test_binding_checks():
    _announce("binding checks")
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError, match="elements"):
        B.moe_norm(x, w, 5, 64, x)
    with pytest.raises(ValueError, match="elements"):
        B.moe_norm(x, w, 4, 65, x)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_norm(x.t(), w, 4, 64, x)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_norm(x.cpu(), w, 4, 64, x)
    with pytest.raises(TypeError):
        B.moe_norm(x.half(), w, 4, 64, x)
    with pytest.raises(TypeError):
        B.moe_norm(x, w.float(), 4, 64, x)
    with pytest.raises(TypeError):
        B.moe_norm_backward(x, f, w, 4, 64, x)                    # dx of another type than x
    with pytest.raises(B.MXFP4Error, match="workspace"):
        B.moe_norm_backward(x, x, w, 4, 64, torch.empty_like(x), torch.empty(64, device="cuda"))
    with pytest.raises(B.MXFP4Error, match="go together"):
        B.moe_combine_norm(f.view(4, 1, 64), None, 4, 1, 64, x, x, w_next=w)
    torch.cuda.synchronize()


def test_repeatable():
    """The same inputs give the same bits, whatever the workspace held."""
    _announce("repeatable")
    T, k, N = 1111, 4, 2880
    _, gates, proj, _, _, _ = make_block(T, k, N, torch.bfloat16, torch.float32, key=4)
    a = _backward(T, k, N, torch.bfloat16, torch.float32, True, True, gates, proj)
    b = _backward(T, k, N, torch.bfloat16, torch.float32, True, True, gates, proj)
    for name in a:
        assert torch.equal(a[name], b[name]), name
