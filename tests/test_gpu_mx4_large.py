"""Microscaled 4-bit operators where sizes, counts and offsets are at their ends."""
import pytest
import torch

import decode_gemm_e8_b200 as e8
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cbk():
    cb = e8.Codebook(0)
    yield cb
    assert e8.e8_sync_status(cb) == e8.E8_OK
    cb.free()


def _codes(rows, K, batch=None, seed=0):
    """Random codes with scales of 2^-6 .. 2^1, written down without the encoder."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lead = () if batch is None else (batch,)
    cs, ss = (K + 31) // 32 * 16, (rows + 127) // 128 * ((K + 127) // 128) * 512
    c = torch.empty(lead + (rows, cs), dtype=torch.uint8, device=dev())
    s = torch.empty(lead + (ss,), dtype=torch.uint8, device=dev())
    for part in c.view(-1).split(1 << 30):
        part.copy_(torch.randint(0, 256, part.shape, generator=g, device=dev(), dtype=torch.uint8))
    s.copy_(torch.randint(121, 129, s.shape, generator=g, device=dev(), dtype=torch.uint8))
    return e8.Mx4Matrix(c, s, rows, K, batch)


def _rows(m, first, rows):
    """The matrix of `rows` rows from a multiple of 128 on."""
    tiles = (m.K + 127) // 128 * 512
    return e8.Mx4Matrix(m.codes[first:first + rows].clone(),
                        m.scales[first // 128 * tiles:(first + rows + 127) // 128 * tiles].clone(), rows, m.K)


def test_encode_and_decode_past_2_31_values(cbk):
    rows, K = 33024, 65568
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=dev())
    x[-300:] = torch.randn(300, K, device=dev()).bfloat16()
    m = e8.e8_mx4_encode(cbk, x)
    want = e8.e8_mx4_encode(cbk, x[-256:].contiguous())
    assert torch.equal(m.codes[-256:], want.codes)
    assert torch.equal(m.scales[-want.scales.numel():], want.scales)
    back = e8.e8_mx4_decode_to_bf16(cbk, m)
    assert torch.equal(back[-256:], e8.e8_mx4_decode_to_bf16(cbk, want)) and not back[:-300].any()


@pytest.mark.parametrize("rows,K,batch", [(4300000, 8, None), (4200001, 3, None), (1, 32, 70000), (2, 5, 66000)])
def test_more_row_blocks_and_matrices_than_a_grid_holds(cbk, rows, K, batch):
    shape = (rows, K) if batch is None else (batch, rows, K)
    x = torch.randn(shape, device=dev())
    m = e8.e8_mx4_encode(cbk, x)
    back = e8.e8_mx4_decode_to_bf16(cbk, m)
    last = x[-100:].contiguous()
    assert torch.equal(back[-100:], e8.e8_mx4_decode_to_bf16(cbk, e8.e8_mx4_encode(cbk, last)))
    again = e8.e8_mx4_encode(cbk, back.float())          # the form's own values are kept
    assert torch.equal(e8.e8_mx4_decode_to_bf16(cbk, again), back)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_product_with_codes_past_2_31_bytes(cbk, M):
    N, K = 70016, 65536
    m = _codes(N, K)
    x = torch.randn(M, K, device=dev()).bfloat16()
    y = e8.e8_mx4_gemm(cbk, x, m)
    for first in (0, 69888):
        part = _rows(m, first, 128)
        ref = e8.e8_mx4_decode_to_bf16(cbk, e8.e8_mx4_encode(cbk, x)).double() @ \
            e8.e8_mx4_decode_to_bf16(cbk, part).double().T
        # half a bf16 step, and K additions in fp32 on sums of size sqrt(K)
        err = (y[:, first:first + 128].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * ref.abs().max()).all()
        assert err.norm() <= 2.0 ** -8 * ref.norm()


@pytest.mark.parametrize("M,N,K", [(1, 128, 300000), (5, 3, 100001), (20, 1, 70000), (100000, 16, 32), (70000, 24, 200),
                                   (2, 500000, 64)])
def test_product_of_long_and_flat_shapes(cbk, M, N, K):
    m = _codes(N, K, seed=1)
    x = torch.randn(M, K, device=dev()).bfloat16()
    y = e8.e8_mx4_gemm(cbk, x, m)
    ref = e8.e8_mx4_decode_to_bf16(cbk, e8.e8_mx4_encode(cbk, x)).double() @ \
        e8.e8_mx4_decode_to_bf16(cbk, m).double().T
    assert (y.double() - ref).norm() <= 2.0 ** -8 * ref.norm()


def test_experts_past_2_31_bytes(cbk):
    E, H, inner, T = 40, 8192, 8192, 3
    w13, w2 = _codes(2 * inner, H, E, 2), _codes(H, inner, E, 3)
    router = torch.zeros(E, H, dtype=torch.bfloat16, device=dev())
    router[E - 1] = 1
    x = (torch.rand(T, H, device=dev()) * 2.0 ** -6).bfloat16()
    ids = torch.empty(T, 1, dtype=torch.int32, device=dev())
    y = e8.e8_mx4_moe(cbk, x, router, w13, w2, 1, experts=ids)
    assert (ids == E - 1).all()
    one = [e8.Mx4Matrix(m.codes[-1:].clone(), m.scales[-1:].clone(), m.rows, m.K, 1) for m in (w13, w2)]
    # (the number of experts decides how K is split when they are fewer than the slots)
    y1 = torch.cat([e8.e8_mx4_moe(cbk, x[i:i + 1].clone(), router[-1:].clone(), *one, 1) for i in range(T)])
    ref = y1.double()
    assert ref.isfinite().all() and (ref != 0).any()
    assert (y.double() - ref).norm() <= 2.0 ** -7 * ref.norm()


@pytest.mark.parametrize("T,E,topk,H,inner", [(2, 2, 2, 32768, 128), (3, 2, 1, 128, 65536), (1, 512, 16, 128, 128),
                                              (64, 512, 16, 256, 128), (64, 1, 1, 128, 128), (18, 24, 16, 128, 256),
                                              (19, 511, 3, 384, 128)])
def test_layer_at_the_ends_of_its_ranges(cbk, T, E, topk, H, inner):
    w13, w2 = _codes(2 * inner, H, E, 4), _codes(H, inner, E, 5)
    router = (torch.randn(E, H, device=dev()) * H ** -0.5).bfloat16()
    x = (torch.randn(T, H, device=dev()) * H ** -0.5).bfloat16()
    ids = torch.empty(T, topk, dtype=torch.int32, device=dev())
    p = torch.empty(T, topk, device=dev())
    y = e8.e8_mx4_moe(cbk, x, router, w13, w2, topk, experts=ids, probs=p)
    logits = x.double() @ router.double().T
    assert torch.equal(ids.long(), logits.topk(topk).indices)
    d13, d2 = (e8.e8_mx4_decode_to_bf16(cbk, m).double() for m in (w13, w2))
    ref = torch.zeros(T, H, dtype=torch.float64, device=dev())
    for t in range(T):
        for k in range(topk):
            e = int(ids[t, k])
            u = d13[e] @ x[t].double()
            h = torch.nn.functional.silu(u[0::2]) * u[1::2]
            ref[t] += float(p[t, k]) * (d2[e] @ h)
    # bf16 output 2^-9 in the mean, h with 8 significant bits 2^-9 a term
    assert (y.double() - ref).norm() <= 2.0 ** -8 * ref.norm()
