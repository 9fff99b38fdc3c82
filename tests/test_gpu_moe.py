"""Mixture-of-experts layer with microscaled 4-bit experts against the binary64 oracle."""
import numpy as np
import pytest
import torch

import decode_gemm_e8_b200 as e8
from oracle import mx4_oracle as mx
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cbk():
    cb = e8.Codebook(0)
    yield cb
    cb.free()


def _layer(cbk, E, H, inner, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gate, up = (torch.randn(E, inner, H, generator=g, device=dev()) * H ** -0.5 for _ in range(2))
    down = torch.randn(E, H, inner, generator=g, device=dev()) * inner ** -0.5
    router = (torch.randn(E, H, generator=g, device=dev()) * H ** -0.5).bfloat16()
    w13, w2 = e8.e8_mx4_moe_pack(cbk, gate, up, down)
    return router, w13, w2


def _tokens(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device=dev())
    x = x * torch.exp(torch.randn(T, 1, generator=g, device=dev()))
    x[:, ::37] *= 16
    return x.bfloat16()


def _run(cbk, x, router, w13, w2, topk, renorm=True):
    T = x.shape[0]
    ids = torch.empty(T, topk, dtype=torch.int32, device=dev())
    p = torch.empty(T, topk, device=dev())
    y = e8.e8_mx4_moe(cbk, x, router, w13, w2, topk, renormalize=renorm, experts=ids, probs=p)
    assert e8.e8_sync_status(cbk) == e8.E8_OK
    return y, ids, p


def _check(cbk, x, router, w13, w2, topk, renorm=True):
    y, ids, p = _run(cbk, x, router, w13, w2, topk, renorm)
    d13, d2 = (e8.e8_mx4_decode_to_bf16(cbk, m).cpu().double().numpy() for m in (w13, w2))
    ref, rid, rp, A = mx.moe(x.cpu().double().numpy(), router.cpu().double().numpy(), d13, d2, topk, renorm)
    assert np.array_equal(ids.cpu().numpy(), rid)
    # exp of an fp32 difference (the difference rounds by 2^-24 of up to ~100) and one division
    assert np.allclose(p.cpu().numpy(), rp, rtol=2e-5, atol=1e-30)
    # output rounding 2^-8; h with 8 significant bits: 2^-9 of each term, and as much
    # again for the fp32 sums and probabilities
    err = np.abs(y.cpu().double().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * A + 1e-37).all()
    assert np.linalg.norm(err) <= (2.0 ** -8 + 2.0 ** -9) * np.linalg.norm(ref) + 1e-37
    return y


@pytest.mark.parametrize("T,E,topk,H,inner,renorm", [
    (1, 1, 1, 128, 128, True), (1, 4, 2, 256, 128, True), (2, 3, 3, 128, 256, False),
    (5, 8, 2, 384, 640, True), (16, 16, 4, 512, 256, False), (33, 5, 3, 640, 384, True),
    (64, 4, 4, 256, 384, True), (64, 40, 8, 256, 128, False), (63, 130, 16, 128, 128, True),
    (7, 9, 1, 1152, 128, False), (1, 300, 8, 256, 256, True), (3, 4, 2, 128, 2048, True)])
def test_layer(cbk, T, E, topk, H, inner, renorm):
    router, w13, w2 = _layer(cbk, E, H, inner, T + E)
    _check(cbk, _tokens(T, H, T * 3 + 1), router, w13, w2, topk, renorm)


def test_every_token_to_one_expert(cbk):
    router, w13, w2 = _layer(cbk, 6, 256, 256, 3)
    router.zero_()
    x = _tokens(64, 256, 5).abs()
    router[4] = 1
    y = _check(cbk, x, router, w13, w2, 1)
    ids = _run(cbk, x, router, w13, w2, 1)[1]
    assert (ids == 4).all() and y.isfinite().all()


def test_ties_go_to_the_lowest_expert(cbk):
    router, w13, w2 = _layer(cbk, 12, 256, 128, 4)
    router.copy_(torch.randint(-2, 3, (12, 256), device=dev()))   # sums exact in any order
    router[7] = router[2]
    router[9] = router[2]
    x = torch.randint(-3, 4, (20, 256), device=dev()).bfloat16()
    _check(cbk, x, router, w13, w2, 5)
    x.zero_()                                                      # all logits equal
    ids = _run(cbk, x, router, w13, w2, 5)[1]
    assert (ids.cpu() == torch.arange(5)).all()


def test_near_ties_need_the_64_bit_sum(cbk):
    """Logits that differ by less than fp32 resolves are still ordered."""
    router, w13, w2 = _layer(cbk, 4, 128, 128, 6)
    x = torch.ones(2, 128, device=dev()).bfloat16()
    router.fill_(1.0)
    router[3, 127] = 1.0 + 2.0 ** -7
    router[1, :2] = torch.tensor([2.0 ** 30, -2.0 ** 30])
    router[2, :3] = torch.tensor([2.0 ** 30, -2.0 ** 30, 1.0 + 2.0 ** -6])
    ids = _run(cbk, x, router, w13, w2, 2)[1]
    want = mx.route(x.cpu().double().numpy(), router.cpu().double().numpy(), 2, True)[0]
    assert np.array_equal(ids.cpu().numpy(), want)


def test_nan_token_and_quiet_tokens(cbk):
    router, w13, w2 = _layer(cbk, 8, 256, 256, 7)
    x = _tokens(9, 256, 8)
    clean, cid, _ = _run(cbk, x, router, w13, w2, 2)
    x2 = x.clone()
    x2[4, 17] = float("nan")
    x2[6, 3] = float("inf")
    y, ids, _ = _run(cbk, x2, router, w13, w2, 2)
    keep = [i for i in range(9) if i not in (4, 6)]
    assert y[4].isnan().all()
    assert not y[6].isfinite().any()
    assert torch.equal(ids[keep], cid[keep]) and torch.equal(y[keep], clean[keep])
    assert (ids >= 0).all() and (ids < 8).all()
    # zeros stay zeros, tiny and huge tokens keep their relative accuracy
    x3 = x.clone()
    x3[0] = 0
    x3[1] *= 2.0 ** -60
    x3[2] = x3[2] * 2.0 ** 20
    y = _check(cbk, x3[:2].contiguous(), router, w13, w2, 2)
    assert (y[0] == 0).all()
    _check(cbk, x3[2:3].contiguous(), router, w13, w2, 2)


def test_only_chosen_experts_are_read(cbk):
    """A NaN expert changes nothing for tokens that do not choose it."""
    router, w13, w2 = _layer(cbk, 8, 128, 128, 9)
    x = _tokens(3, 128, 10)
    y, ids, _ = _run(cbk, x, router, w13, w2, 2)
    unused = [e for e in range(8) if e not in set(ids.flatten().tolist())]
    for m in (w13, w2):
        m.scales.view(8, -1)[unused] = 255
    assert torch.equal(_run(cbk, x, router, w13, w2, 2)[0], y)


def test_runs_repeat_graphs_replay_and_streams_do_not_mix(cbk):
    router, w13, w2 = _layer(cbk, 16, 512, 256, 11)
    x = _tokens(24, 512, 12)
    want = [_run(cbk, _tokens(24, 512, s), router, w13, w2, 4)[0] for s in (12, 13, 14)]
    for _ in range(20):
        assert torch.equal(e8.e8_mx4_moe(cbk, x, router, w13, w2, 4), want[0])
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = e8.e8_mx4_moe(cbk, static, router, w13, w2, 4)
    for i, s in enumerate((12, 13, 14)):
        static.copy_(_tokens(24, 512, s))
        g.replay()
        assert torch.equal(y, want[i])
    # two streams at once, each with a workspace of its own
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    xs = [_tokens(24, 512, s) for s in (13, 14)]
    torch.cuda.synchronize()
    for _ in range(5):
        ys = [e8.e8_mx4_moe(cbk, xs[i], router, w13, w2, 4, stream=ss[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want[1]) and torch.equal(ys[1], want[2])


def test_empty_and_refused(cbk):
    router, w13, w2 = _layer(cbk, 4, 128, 128, 15)
    assert e8.e8_mx4_moe(cbk, _tokens(1, 128, 1)[:0], router, w13, w2, 2).shape == (0, 128)
    x = _tokens(3, 128, 1)
    for bad in (lambda: e8.e8_mx4_moe(cbk, x, router, w13, w2, 5), lambda: e8.e8_mx4_moe(cbk, x, router, w13, w2, 0),
                lambda: e8.e8_mx4_moe(cbk, _tokens(65, 128, 1), router, w13, w2, 2),
                lambda: e8.e8_mx4_moe(cbk, x.float(), router, w13, w2, 2),
                lambda: e8.e8_mx4_moe(cbk, x, router[:3], w13, w2, 2),
                lambda: e8.e8_mx4_moe(cbk, x.cpu(), router, w13, w2, 2),
                lambda: e8.e8_mx4_moe(cbk, x, router, w2, w13, 2)):
        with pytest.raises(e8.E8Error):
            bad()


def test_layer_with_the_other_operators(cbk):
    """A decode step's tail: a compressed projection, the layer on its result, and a second
    microscaled product on the layer's output, captured together."""
    T, H = 8, 256
    router, w13, w2 = _layer(cbk, 8, H, 256, 20)
    proj = e8.e8_mx4_encode(cbk, torch.randn(H, H, device=dev()) * H ** -0.5)
    head = e8.e8_mx4_encode(cbk, torch.randn(500, H, device=dev()) * H ** -0.5)
    x = _tokens(T, H, 21)

    def step(v):
        a = e8.e8_mx4_gemm(cbk, v, proj)
        b = e8.e8_mx4_moe(cbk, a, router, w13, w2, 2)
        return a, b, e8.e8_mx4_gemm(cbk, b, head)

    a, b, c = step(x)
    _check(cbk, a, router, w13, w2, 2)
    dec = [mx.roundtrip(v.cpu().double().numpy()) for v in (b,)][0]
    hw = e8.e8_mx4_decode_to_bf16(cbk, head).cpu().double().numpy()
    ref = dec @ hw.T
    assert np.linalg.norm(c.cpu().double().numpy() - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    static = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = step(static)
    static.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, (a, b, c)))


@pytest.mark.parametrize("T,E,topk,H,inner", [(1, 8, 2, 256, 256), (1, 64, 8, 1024, 512), (4, 16, 4, 128, 128),
                                              (40, 32, 4, 512, 384)])
def test_many_runs_of_short_units(cbk, T, E, topk, H, inner):
    """Units so short that a block's weights run a unit ahead of the one that claims them:
    twenty thousand runs end without a wait that gives up, all with the same result."""
    router, w13, w2 = _layer(cbk, E, H, inner, 8)
    x = _tokens(T, H, 9)
    first = _run(cbk, x, router, w13, w2, topk)[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ys = [e8.e8_mx4_moe(cbk, x, router, w13, w2, topk) for _ in range(50)]
    for _ in range(400):
        g.replay()
    assert e8.e8_sync_status(cbk) == e8.E8_OK
    assert all(torch.equal(y, first) for y in ys)


def test_layers_in_a_row(cbk):
    """A layer's output is the next one's input, in one workspace, eagerly and captured."""
    T, E, topk, H, inner = 8, 16, 4, 512, 256
    layers = [_layer(cbk, E, H, inner, s) for s in (1, 2, 3)]
    x = _tokens(T, H, 4)
    size = e8.load_library().e8_mx4_moe_workspace_bytes(T, H, E, topk, inner)
    ws = torch.empty(size, dtype=torch.uint8, device=dev())

    def run(apart):
        y = x
        for layer in layers:
            y = e8.e8_mx4_moe(cbk, y, *layer, topk, workspace=ws)
            if apart:
                torch.cuda.synchronize()
        return y

    want = run(True)
    for _ in range(20):
        assert torch.equal(run(False), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = run(False)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and e8.e8_sync_status(cbk) == e8.E8_OK
