"""Mixture-of-experts layer where its numbers are at their ends: what the pairs of e4m3
values still hold, tokens of very small values, h past fp32."""
import numpy as np
import pytest
import torch

import decode_gemm_e8_b200 as e8
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

H, INNER = 256, 128


@pytest.fixture(scope="module")
def cbk():
    cb = e8.Codebook(0)
    yield cb
    assert e8.e8_sync_status(cb) == e8.E8_OK
    cb.free()


def _picking_layer(cbk, gate_weight, up_weight):
    """One expert: g = gate_weight * x[0] in every row, u_i = up_weight * x[1 + i], Y_i = h_i."""
    gate, up = torch.zeros(1, INNER, H), torch.zeros(1, INNER, H)
    gate[0, :, 0] = gate_weight
    up[0, torch.arange(INNER), 1 + torch.arange(INNER)] = up_weight
    down = torch.zeros(1, H, INNER)
    down[0, torch.arange(INNER), torch.arange(INNER)] = 1
    w13, w2 = e8.e8_mx4_moe_pack(cbk, gate.to(dev()), up.to(dev()), down.to(dev()))
    return torch.zeros(1, H, dtype=torch.bfloat16, device=dev()), w13, w2


def _bf16(shape, low, high, seed):
    """bf16 values between two powers of two, even over the exponents."""
    g = torch.Generator().manual_seed(seed)
    v = torch.exp2(low + (high - low) * torch.rand(shape, generator=g, dtype=torch.float64))
    return v.bfloat16().clamp(2.0 ** low, 2.0 ** high * (1 - 2.0 ** -8))


@pytest.mark.parametrize("T", [1, 7, 40])
def test_tokens_are_exact_down_to_2_13_below_their_largest(cbk, T):
    layer = _picking_layer(cbk, 1.0, 1.0)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 128
    x[:, 1:65] = _bf16((T, 64), -6, 5, 1)      # (h keeps them too: each 64 span less than 2^12)
    x[:, 65:129] = _bf16((T, 64), -4, 7, 2)
    x[:, 3] *= -1
    y = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1).cpu()
    # silu(128) is 128 in fp32 and p is 1
    assert torch.equal(y[:, :INNER], 128 * x[:, 1:129]) and not y[:, INNER:].any()


@pytest.mark.parametrize("T", [1, 40])
def test_smaller_values_are_off_by_2_21_of_the_largest(cbk, T):
    layer = _picking_layer(cbk, 1.0, 1.0)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 128
    x[:, 1:129] = _bf16((T, 128), -13, -6, 3)
    y = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1).cpu().double() / 128
    x = x.double()[:, 1:129]
    # X, then h (2^-9 of it, 2^-21 of the largest at least) and Y (2^-8)
    x_off = 2.0 ** -21 * 128
    h_off = torch.maximum(2.0 ** -9 * (x + x_off), 2.0 ** -21 * torch.full_like(x, 2.0 ** -6 + x_off))
    tol = (x_off + h_off) * (1 + 2.0 ** -8) + 2.0 ** -8 * x
    assert ((y[:, :INNER] - x).abs() <= tol).all()
    assert ((y[:, :INNER] - x).abs() > 2.0 ** -8 * x).any()    # (no longer exact)


@pytest.mark.parametrize("T", [1, 40])
def test_tokens_of_the_smallest_values(cbk, T):
    """Largest 2^-118, below the least scale of a pair: bf16 values, subnormal ones too, are
    held exactly all the same."""
    layer = _picking_layer(cbk, 2.0 ** 122, 2.0 ** 100)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 2.0 ** -118
    x[:, 1:129] = _bf16((T, 128), -131, -119, 4)
    y = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1).cpu().double()
    want = 16 / (1 + np.exp(-16.0)) * 2.0 ** 100 * x.double()[:, 1:129]
    # h 2^-9, Y 2^-8, and the fp32 silu (a few roundings of 2^-24)
    assert ((y[:, :INNER] - want).abs() <= (2.0 ** -9 + 2.0 ** -8 + 2.0 ** -16) * want).all()
    assert (want > 0).all()


def test_h_past_fp32_makes_its_token_nan_and_no_other(cbk):
    layer = _picking_layer(cbk, 1.0, 2.0 ** 60)
    x = torch.zeros(5, H, dtype=torch.bfloat16)
    x[:, 0] = 8
    x[:, 1:129] = 1
    clean = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1)
    assert clean.isfinite().all()
    keep = [0, 1, 3, 4]
    # a token of 2^70 and ones: its scale is 2^63, the ones are 2^-63 of that, less than half
    # of the least step 2^-13, and enter as zeros (2^-70 of the largest: within the 2^-21
    # that values so small are held to); u and h are 0, and so is Y
    x[2, 0] = 2.0 ** 70
    y = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1)
    assert (y[2] == 0).all() and torch.equal(y[keep], clean[keep])
    # u = 2^130 is past fp32 by itself; then u = 2^60 2^30 and h = 2^90 2^70 is
    x[2, :129] = 2.0 ** 70
    y = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1)
    assert y[2].isnan().all() and torch.equal(y[keep], clean[keep])
    x[2, 1:129] = 2.0 ** 60
    layer = _picking_layer(cbk, 1.0, 2.0 ** 30)
    y = e8.e8_mx4_moe(cbk, x.to(dev()), *layer, 1)
    assert y[2].isnan().all() and y[keep].isfinite().all()
