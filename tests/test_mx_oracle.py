"""The oracle of the MXFP4 quantisation and products against computations independent of it: brute
force over the 16 codes, closed forms, torch's bf16 rounding, and planted mistakes."""
import numpy as np
import pytest
import torch

import oracle.moe_oracle as M
import oracle.mx_oracle as O


def _brute(x):
    """Codes and byte of one block of 32 by trying every code: nearest, then even."""
    amax = max(abs(v) for v in x)
    e = -127 if amax == 0 else max(-127, int(np.floor(np.log2(amax))) - 2)
    table = M.e2m1_table()
    codes = []
    for v in x:
        best = min(range(8), key=lambda c: (abs(abs(v) * 2.0 ** -e - table[c]), c & 1))
        codes.append(best | (8 if np.signbit(v) else 0))
    return codes, e + 127


def test_codes_are_the_nearest():
    r = np.random.default_rng(1)
    for scale in (1.0, 2.0 ** -120, 2.0 ** 100, 1e-3):
        x = r.normal(size=(20, 32)) * np.exp(2 * r.normal(size=(20, 1))) * scale
        codes, byte = O.quantize(x)
        for i in range(20):
            want, wb = _brute(x[i])
            assert codes[i].tolist() == want and byte[i, 0] == wb


def test_borders_go_to_the_even_code():
    x = np.zeros(32)
    x[:8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9]
    x[8:16] = -x[:8]
    codes, byte = O.quantize(x[None])
    assert byte[0, 0] == 127
    assert O.values(codes, byte)[0, :8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    assert (codes[0, 8:16] == (codes[0, :8] | 8)).all()


def test_stored_values_are_fixed_points():
    r = np.random.default_rng(2)
    codes = r.integers(0, 16, (50, 64)).astype(np.uint8)
    codes[:, ::32] = 7                     # a 6 in every block: the exponent is the scale's own
    byte = r.integers(0, 253, (50, 2)).astype(np.uint8)
    again, byte2 = O.quantize(O.values(codes, byte))
    assert (byte2 == byte).all()
    assert (O.values(again, byte2) == O.values(codes, byte)).all()


def test_decode_agrees_with_the_format():
    r = np.random.default_rng(3)
    blocks = r.integers(0, 256, (5, 3, 16)).astype(np.uint8)
    byte = r.integers(100, 140, (5, 3)).astype(np.uint8)
    assert (O.decode(blocks, byte) == M.dequantize_mxfp4(blocks, byte).reshape(5, 96)).all()
    assert (O.pack(O.unpack(blocks)) == blocks).all()


def test_special_blocks():
    x = np.zeros((4, 32))
    x[1, 5], x[2, 6] = np.nan, -np.inf
    x[3, 0] = 2.0 ** -149
    codes, byte = O.quantize(x)
    assert byte[:, 0].tolist() == [0, 255, 255, 0]
    assert (codes == 0).all()
    assert np.isnan(O.values(codes, byte)[1:3]).all()


def test_bf16_rounding_is_torchs():
    r = np.random.default_rng(4)
    x = r.normal(size=4096).astype(np.float32) * np.exp(10 * r.normal(size=4096)).astype(np.float32)
    x[:4] = [0.0, 1.00390625, 1.01171875, -2.0 ** -130]
    want = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    assert (O.bf16(x) == want.astype(np.float64)).all()


def test_products_on_unit_rows():
    r = np.random.default_rng(5)
    w = r.normal(size=(3, 7, 32))
    x = np.eye(32)[:6]
    ids = np.array([[0, 2], [1, 0], [2, 1], [0, 1], [1, 2], [2, 0]])
    out, _ = O.expert_matmul(w, None, x, False, ids)
    for t in range(6):
        for s in range(2):
            assert (out[t, s] == w[ids[t, s], :, t]).all()


def test_layer_with_one_expert_is_a_gated_mlp():
    r = np.random.default_rng(6)
    x = O.bf16(r.normal(size=(3, 32)))
    gu, down = r.normal(size=(1, 64, 32)), r.normal(size=(1, 32, 32))
    xn, _, ids, gates = O.layer_route(x, None, 1e-5, r.normal(size=(1, 32)), None, 1)
    assert (gates == 1).all() and (ids == 0).all()
    h, _, act, _, _ = O.layer(xn, ids, gates, gu, None, down, None)
    p = x @ gu[0].T
    g, u = np.minimum(p[:, ::2], 7.0), np.clip(p[:, 1::2], -7, 7)
    a = (u + 1) * g / (1 + np.exp(-1.702 * g))
    assert np.allclose(act[:, 0], a, rtol=1e-12, atol=0)
    assert np.allclose(h, O.bf16(a) @ down[0].T, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("plant", ["odd_tie", "floor_scale", "no_saturation"])
def test_planted_mistakes_are_seen(plant, monkeypatch):
    x = np.zeros(32)
    x[:3] = [2.5, 7.9, 0.25]
    good = O.quantize(x[None])
    if plant == "odd_tie":
        monkeypatch.setattr(O, "EVEN_BELOW", ~O.EVEN_BELOW)
        assert (O.quantize(x[None])[0] != good[0]).any()
    elif plant == "floor_scale":
        want, wb = _brute(x)
        assert good[1][0, 0] == wb and good[1][0, 0] != wb - 1
    else:
        assert O.values(*good)[0, 1] == 6.0
