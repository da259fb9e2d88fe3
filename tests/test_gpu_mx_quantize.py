"""MXFP4 quantisation on the GPU against the oracle: codes, scale bytes and values bit for bit (the
definition leaves nothing to rounding order)."""
import numpy as np
import pytest
import torch

import oracle.mx_oracle as O
from mxfp4_mixture_experts_amd import binding as B

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float32]


def _announce(msg):
    print(f"[case] {msg}", flush=True)


def quantized(x, transposed=False, values=True):
    """The library's (codes [., .], bytes, values) of a device tensor, as numpy; the output buffers hold
    garbage before."""
    R, C = x.shape
    rows, K = (C, R) if transposed else (R, C)
    blocks = torch.full((rows, K // 32, 16), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // 32), 0x5A, dtype=torch.uint8, device="cuda")
    v = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda") if values else None
    (B.mxfp4_quantize_transposed if transposed else B.mxfp4_quantize)(x, blocks, scales, values=v)
    return (O.unpack(blocks.cpu().numpy()), scales.cpu().numpy(),
            None if v is None else v.float().cpu().numpy().astype(np.float64))


def check(x, transposed=False):
    host = x.float().cpu().numpy().astype(np.float64)
    codes, byte = O.quantize(np.ascontiguousarray(host.T) if transposed else host)
    got_c, got_b, got_v = quantized(x, transposed)
    assert (got_b == byte).all()
    assert (got_c == codes).all()
    want = O.values(codes, byte)
    assert ((got_v == want) | (np.isnan(got_v) & np.isnan(want))).all()
    plain_c, plain_b, _ = quantized(x, transposed, values=False)
    assert (plain_b == byte).all() and (plain_c == codes).all()


def activations(seed, rows, K, dtype):
    r = np.random.default_rng(seed)
    x = r.normal(size=(rows, K)) * np.exp(r.normal(size=(rows, 1)))
    x[:, r.random(K) < 0.02] *= 50.0
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype).contiguous()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 2880), (3, 96), (7, 160), (64, 64), (129, 2880), (1000, 288),
                                    (33, 8224)])
def test_rows(rows, K, dtype):
    _announce(f"quantize {rows}x{K} {dtype}")
    check(activations(rows + K, rows, K, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,C", [(32, 1), (32, 64), (64, 7), (96, 129), (256, 2880), (288, 1023), (512, 130),
                                 (2048, 65), (8224, 33)])
def test_transposed(R, C, dtype):
    _announce(f"quantize_transposed {R}x{C} {dtype}")
    check(activations(R + C, R, C, dtype), transposed=True)


def _every_border(dtype):
    """Blocks whose maximum is 4 .. 7.99 at every exponent of the type, filled with the midpoints
    between codes and the type's neighbours of them."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float64)
    rows = []
    for e in range(-133, 126):
        for sign in (1.0, -1.0):
            block = [7.96875 if e % 2 else 4.0]
            for m in mids:
                step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20
                block += [m, m * (1 - step), m * (1 + step), -m]
            block += [6.0, 0.0, -0.0]
            rows.append(np.ldexp(sign * np.array(block), e))
    x = np.array(rows)
    return torch.from_numpy(x).to(torch.float32).to(dtype).cuda().contiguous()


@pytest.mark.parametrize("dtype", DTYPES)
def test_borders_at_every_exponent(dtype):
    x = _every_border(dtype)
    assert x.shape[1] == 32
    check(x)
    check(x.t().contiguous(), transposed=True)


def test_every_bf16_value():
    """Every finite bf16 as a block's maximum and as an element beside a larger one."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v.float())].cuda()
    x = torch.zeros((v.numel(), 32), dtype=torch.bfloat16, device="cuda")
    x[:, 9] = v
    check(x)
    for top in (1.0, 2.0 ** -126, 1.5 * 2.0 ** 100):
        x[:, 30] = top
        check(x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinity_stay_in_their_blocks(dtype):
    x = activations(5, 64, 160, dtype)
    x[3, 40], x[7, 159], x[9, 0], x[9, 33] = float("nan"), float("inf"), -float("inf"), float("nan")
    check(x)
    check(x[:, :].contiguous(), transposed=True)
    largest = torch.full((32, 64), torch.finfo(dtype).max, dtype=dtype, device="cuda")
    check(largest)
    check(torch.zeros((32, 64), dtype=dtype, device="cuda"))
    check(torch.full((32, 64), 2.0 ** -133, dtype=dtype, device="cuda"))


def test_odd_addresses_of_the_transposed_input():
    """bf16 rows that start on no 4-byte border, and scales anywhere."""
    flat = activations(6, 1, 64 * 66 + 1 + 31, torch.bfloat16).view(-1)
    x = flat[1:1 + 64 * 66].view(64, 66)
    assert x.data_ptr() % 4 == 2
    check(x, transposed=True)


def test_round_trip_through_dequantize():
    x = activations(7, 65, 2880, torch.float32)
    blocks = torch.empty((65, 90, 16), dtype=torch.uint8, device="cuda")
    scales = torch.empty((65, 90), dtype=torch.uint8, device="cuda")
    v, back = torch.empty((2, 65, 2880), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_quantize(x, blocks, scales, values=v)
    B.mxfp4_dequantize(blocks, scales, back)
    assert torch.equal(v, back)
    again = torch.empty_like(blocks)
    B.mxfp4_quantize(v, again, scales.clone())
    B.mxfp4_dequantize(again, scales, back)
    assert torch.equal(v, back)


def test_past_32_bits():
    """More than 2^32 bytes of input and of values: the last rows are right."""
    rows, K = 1 << 20, 2080
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    tail = activations(8, 64, K, torch.bfloat16)
    x[-64:] = tail
    blocks = torch.empty((rows, K // 32, 16), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    v = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    B.mxfp4_quantize(x, blocks, scales, values=v)
    codes, byte = O.quantize(tail.float().cpu().numpy())
    assert (O.unpack(blocks[-64:].cpu().numpy()) == codes).all() and (scales[-64:].cpu().numpy() == byte).all()
    assert (v[-64:].float().cpu().numpy() == O.values(codes, byte)).all()
    assert not blocks[:-64].any()
    # the transposed form: the same rows as columns
    xt = x.view(1 << 15, K * 32)
    B.mxfp4_quantize_transposed(xt, blocks.view(K * 32, 1 << 10, 16), scales.view(K * 32, 1 << 10),
                                values=v.view(K * 32, 1 << 15))
    host = xt[-32:].float().cpu().numpy()
    codes, byte = O.quantize(np.ascontiguousarray(host.T))
    got = blocks.view(K * 32, 1 << 10, 16)[:, -1].cpu().numpy()
    assert (got == O.pack(codes)[:, 0]).all()
    assert (scales.view(K * 32, 1 << 10)[:, -1].cpu().numpy() == byte[:, 0]).all()


def test_another_stream():
    x = activations(9, 513, 2880, torch.bfloat16)
    want = quantized(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    blocks = torch.empty((513, 90, 16), dtype=torch.uint8, device="cuda")
    scales = torch.empty((513, 90), dtype=torch.uint8, device="cuda")
    B.mxfp4_quantize(x, blocks, scales, stream=side)
    side.synchronize()
    assert (O.unpack(blocks.cpu().numpy()) == want[0]).all() and (scales.cpu().numpy() == want[1]).all()
