"""Microscaled 4-bit products with the largest sizes that 32 bits hold."""
import pytest
import torch

import decode_gemm_e8_b200 as e8
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def cbk():
    torch.cuda.empty_cache()
    cb = e8.Codebook(0)
    yield cb
    assert e8.e8_sync_status(cb) == e8.E8_OK
    cb.free()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("K", [TOP, TOP - 255, TOP - 256])
def test_longest_sums(cbk, K):
    """All but the last few columns are zeros: the result is the product of those."""
    first = K // 256 * 256 - 512
    x = torch.zeros(1, K, dtype=torch.bfloat16, device=dev())
    w = torch.zeros(2, K, dtype=torch.bfloat16, device=dev())
    x[:, first:] = torch.randn(1, K - first, device=dev()).bfloat16()
    w[:, first:] = torch.randn(2, K - first, device=dev()).bfloat16()
    tail = [e8.e8_mx4_decode_to_bf16(cbk, e8.e8_mx4_encode(cbk, t[:, first:].contiguous())).double() for t in (x, w)]
    m, a = e8.e8_mx4_encode(cbk, w), e8.e8_mx4_encode(cbk, x)
    ref = tail[0] @ tail[1].T
    # half a bf16 step, and fewer than 1024 additions in fp32 of terms whose magnitudes sum to A
    tol = 2.0 ** -8 * ref.abs() + 1024 * 2.0 ** -23 * (tail[0].abs() @ tail[1].abs().T)
    for y in (e8.e8_mx4_gemm(cbk, x, m), e8.e8_mx4_gemm_codes(cbk, a, m)):
        assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("M", [TOP, TOP - 255, TOP - 256])
def test_most_tokens(cbk, M):
    """2^31 tokens of 32 values, all zeros but the first and last hundred, times 8 x 32."""
    N, K = 8, 32
    codes = torch.zeros(M, 16, dtype=torch.uint8, device=dev())
    scales = torch.full(((M + 127) // 128 * 512,), 127, dtype=torch.uint8, device=dev())
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=dev())
    g = torch.Generator(device="cuda").manual_seed(1)
    ends = torch.randint(0, 256, (200, 16), generator=g, device=dev(), dtype=torch.uint8)
    codes[:100], codes[-100:] = ends[:100], ends[100:]
    m = e8.e8_mx4_encode(cbk, torch.randn(N, K, generator=g, device=dev()))
    e8.e8_mx4_gemm_codes(cbk, e8.Mx4Matrix(codes, scales, M, K), m, Y=y)
    few = e8.Mx4Matrix(ends, torch.full((1024,), 127, dtype=torch.uint8, device=dev()), 200, K)
    ref = e8.e8_mx4_decode_to_bf16(cbk, few).double() @ e8.e8_mx4_decode_to_bf16(cbk, m).double().T
    # 32 products, exact as they are, on a common grid of 26 bits at most: half a bf16 step
    # and the fp32 sum
    tol = 2.0 ** -8 * ref.abs() + 32 * 2.0 ** -23 * 32 * 36
    got = torch.cat([y[:100], y[-100:]]).double()
    assert ((got - ref).abs() <= tol).all()
    for part in (y[100:100000], y[M // 2:M // 2 + 100000], y[-100000:-100]):
        assert (part == 0).all()
