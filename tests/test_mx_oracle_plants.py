"""Mistakes planted in the oracle of the MXFP4 quantisation, products and layer: each of its pins
(test_mx_oracle) fails for the mistakes that it is there for, and passes without them."""
import numpy as np
import pytest

import oracle.mx_oracle as O
import test_mx_oracle as pins


class _Numpy:
    """numpy, with some functions of its own."""

    def __init__(self, **own):
        self.__dict__.update(own)

    def __getattr__(self, name):
        return getattr(np, name)


def _exponent(off):
    return lambda m: m.setattr(O, "np", _Numpy(frexp=lambda x: (np.frexp(x)[0], np.frexp(x)[1] + off)))


def _round_exponent(m):
    """The scale by the nearest power of two instead of the one below."""
    def frexp(x):
        f, e = np.frexp(x)
        return f, e + (f > 0.75)
    m.setattr(O, "np", _Numpy(frexp=frexp))


def _no_saturation(m):
    """Magnitudes from 7 on go to a code behind 6's (the sign's)."""
    m.setattr(O, "BORDERS", np.append(O.BORDERS, 7.0))
    m.setattr(O, "EVEN_BELOW", np.append(O.EVEN_BELOW, False))


def _odd_ties(m):
    m.setattr(O, "EVEN_BELOW", ~O.EVEN_BELOW)


def _ties_up(m):
    m.setattr(O, "EVEN_BELOW", np.zeros_like(O.EVEN_BELOW))


def _a_border_moved(m):
    b = O.BORDERS.copy()
    b[5] = 3.25
    m.setattr(O, "BORDERS", b)


def _no_floor(m):
    """Without the least exponent -127 the byte of a tiny block wraps around."""
    m.setattr(O, "np", _Numpy(maximum=lambda a, b: np.asarray(a)))


def _no_nan(m):
    m.setattr(O, "np", _Numpy(isfinite=lambda x: np.ones_like(x, dtype=bool)))


def _high_nibble_first(m):
    def unpack(blocks):
        return np.stack([blocks >> 4, blocks & 15], -1).reshape(*blocks.shape[:-2], -1)
    m.setattr(O, "unpack", unpack)


def _wrong_slot(m):
    def expert_matmul(w, bias, x, x_per_slot, ids):
        return good(w, bias, x, x_per_slot, ids[:, ::-1])
    good = O.expert_matmul
    m.setattr(O, "expert_matmul", expert_matmul)


def _no_rounding(m):
    m.setattr(O, "bf16", lambda x: np.asarray(x, np.float64))


def _gate_rows_first(m):
    """Gate and up rows as two halves instead of in turn."""
    def swiglu(p):
        half = p.shape[-1] // 2
        return good(np.stack([p[..., :half], p[..., half:]], -1).reshape(p.shape))
    good = O.M.swiglu
    m.setattr(O.M, "swiglu", swiglu)


def _clamped_nan(m):
    """The activation's clamps as C's fmin and fmax have them, which drop a NaN."""
    def swiglu(p):
        p = np.asarray(p, np.float64)
        g, u = np.fmin(p[..., 0::2], 7.0), np.fmin(np.fmax(p[..., 1::2], -7.0), 7.0)
        return (u + 1.0) * g / (1.0 + np.exp(-1.702 * g))
    m.setattr(O.M, "swiglu", swiglu)


def nan_reaches_the_outputs():
    """A NaN block of one gate row makes its token's layer output NaN, another token's not."""
    r = np.random.default_rng(7)
    gu, down = r.normal(size=(2, 64, 32)), r.normal(size=(2, 32, 32))
    gu[1, 4] = np.nan
    ids, gates = np.array([[0], [1]]), np.ones((2, 1))
    h = O.layer(O.bf16(r.normal(size=(2, 32))), ids, gates, gu, None, down, None)[0]
    assert np.isfinite(h[0]).all() and np.isnan(h[1]).all()


PLANTS = [(_exponent(1), pins.test_codes_are_the_nearest), (_exponent(-1), pins.test_codes_are_the_nearest),
          (_round_exponent, pins.test_codes_are_the_nearest), (_no_saturation, pins.test_codes_are_the_nearest),
          (_a_border_moved, pins.test_codes_are_the_nearest), (_odd_ties, pins.test_borders_go_to_the_even_code),
          (_ties_up, pins.test_borders_go_to_the_even_code), (_no_saturation, pins.test_borders_go_to_the_even_code),
          (_exponent(1), pins.test_stored_values_are_fixed_points), (_no_floor, pins.test_special_blocks),
          (_no_nan, pins.test_special_blocks), (_high_nibble_first, pins.test_decode_agrees_with_the_format),
          (_wrong_slot, pins.test_products_on_unit_rows),
          (_gate_rows_first, pins.test_layer_with_one_expert_is_a_gated_mlp),
          (_no_rounding, pins.test_bf16_rounding_is_torchs),
          (_clamped_nan, nan_reaches_the_outputs)]


@pytest.mark.parametrize("plant,pin", PLANTS, ids=[f"{i}-{pin.__name__}" for i, (_, pin) in enumerate(PLANTS)])
def test_a_planted_mistake_fails_its_pin(plant, pin, monkeypatch):
    pin()
    plant(monkeypatch)
    with pytest.raises((AssertionError, ValueError, OverflowError, IndexError)):
        pin()
