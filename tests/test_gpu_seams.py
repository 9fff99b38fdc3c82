"""Microscaled 4-bit calls and E8 calls on each other's results, in one stream.

e8_gemm's first kernel reads its tokens before it waits for the kernel in front of it; a
call that writes tokens therefore has to be over when that kernel starts.  Buffers are
filled with NaN first, so that a token read too early cannot pass for a result."""
import pytest
import torch

import decode_gemm_e8_b200 as e8
from decode_gemm_e8_b200 import synth
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

K = 4096


@pytest.fixture(scope="module")
def cbk():
    cb = e8.Codebook(0)
    yield cb
    assert e8.e8_sync_status(cb) == e8.E8_OK
    cb.free()


@pytest.fixture(scope="module")
def e8_weights(cbk):
    W = synth.gaussian_weights(K, K, K ** -0.5, 5)
    s = synth.suggest_scale(W, 4)
    i1, i2 = e8.e8_encode(cbk, gu.to_dev(W), 4, 77, s)
    return i1, i2, K, 77, s


def _mx(cbk, seed, std=K ** -0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return e8.e8_mx4_encode(cbk, torch.randn(K, K, generator=g, device=gu.dev()) * std)


def _tokens(M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, K, generator=g, device=gu.dev()).bfloat16()


def _near(got, want):
    """The partial sums of e8_gemm are added in arrival order: at most a few hundred
    additions, each off by 2^-24 of a partial sum."""
    assert got.isfinite().all()
    assert (got - want).double().norm() <= 2.0 ** -14 * want.double().norm()


@pytest.mark.parametrize("M", [1, 8, 9, 32])
def test_product_then_e8_product_then_product(cbk, e8_weights, M):
    i1, i2, N, seed, s = e8_weights
    a, b = _mx(cbk, 1), _mx(cbk, 2)
    x = _tokens(M, 3)
    y = torch.empty(M, K, dtype=torch.bfloat16, device=gu.dev())
    mid = torch.empty(M, K, device=gu.dev())
    z = torch.empty(M, K, dtype=torch.bfloat16, device=gu.dev())
    ws = [torch.empty(max(16, n), dtype=torch.uint8, device=gu.dev()) for n in (
        e8.load_library().e8_mx4_gemm_workspace_bytes(M, K, K),
        e8.e8_workspace_bytes(e8.E8_GEMM_AUTO, M, K, K, 4))]

    def chain(gap=lambda: None):
        y.fill_(float("nan"))
        gap()
        e8.e8_mx4_gemm(cbk, x, a, Y=y, workspace=ws[0])
        gap()
        e8.e8_gemm(cbk, y, i1, i2, N, K, 4, seed, s, Y=mid, workspace=ws[1])
        gap()
        e8.e8_mx4_gemm(cbk, mid, b, Y=z, workspace=ws[0])
        gap()

    g = torch.cuda.CUDAGraph()
    chain()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(4):
            chain()
    for seed_x in range(4, 10):
        x.copy_(_tokens(M, seed_x))
        chain(torch.cuda.synchronize)
        want_y, want_mid = y.clone(), mid.clone()
        for run in (chain, g.replay):
            for buf in (mid, z):
                buf.fill_(float("nan"))
            run()
            torch.cuda.synchronize()
            assert torch.equal(y, want_y)
            _near(mid, want_mid)
            # (of the sums that this run got: a last bit may choose another 4-bit value)
            assert torch.equal(z, e8.e8_mx4_gemm(cbk, mid.clone(), b))


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("M", [1, 8, 32])
def test_decoded_tokens_into_e8_products(cbk, e8_weights, M, grouped):
    i1, i2, N, seed, s = e8_weights
    tokens = [e8.e8_mx4_encode(cbk, _tokens(M, t)) for t in range(6)]
    m = e8.e8_mx4_encode(cbk, _tokens(M, 99))
    y = torch.empty(M, K, dtype=torch.bfloat16, device=gu.dev())
    out = [torch.empty(M, K, device=gu.dev()) for _ in range(2)]

    def chain(gap=lambda: None):
        y.fill_(float("nan"))
        gap()
        e8.e8_mx4_decode_to_bf16(cbk, m, out=y)
        gap()
        if grouped:
            e8.e8_gemm_grouped(cbk, y, [(i1, i2, N, seed, s, o) for o in out], K, 4)
        else:
            e8.e8_gemm_act_noalloc(cbk, y, i1, i2, N, K, 4, seed, s, out[0])
        gap()

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            chain()
    for t in tokens:
        m.codes.copy_(t.codes)
        m.scales.copy_(t.scales)
        chain(torch.cuda.synchronize)
        want = [o.clone() for o in out[: 2 if grouped else 1]]
        for run in (chain, g.replay):
            for o in out:
                o.fill_(float("nan"))
            run()
            torch.cuda.synchronize()
            for got, w in zip(out, want):
                _near(got, w)


def test_experts_into_an_e8_product(cbk, e8_weights):
    i1, i2, N, seed, s = e8_weights
    E, inner, M = 8, 256, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, up = (torch.randn(E, inner, K, generator=g, device=gu.dev()) * K ** -0.5 for _ in range(2))
    down = torch.randn(E, K, inner, generator=g, device=gu.dev()) * inner ** -0.5
    w13, w2 = e8.e8_mx4_moe_pack(cbk, gate, up, down)
    router = torch.randn(E, K, generator=g, device=gu.dev()).bfloat16()
    x = _tokens(M, 2)
    y = torch.empty(M, K, dtype=torch.bfloat16, device=gu.dev())

    def chain(gap=lambda: None):
        y.fill_(float("nan"))
        e8.e8_mx4_moe(cbk, x, router, w13, w2, 2, Y=y)
        gap()
        return e8.e8_gemm(cbk, y, i1, i2, N, K, 4, seed, s)

    want = chain(torch.cuda.synchronize)
    for _ in range(10):
        _near(chain(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [chain() for _ in range(4)]
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            _near(o, want)
