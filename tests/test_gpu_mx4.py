"""Microscaled 4-bit form on the GPU: codes, scales and values bit for bit against the
oracle, products against binary64."""
import numpy as np
import pytest
import torch

import decode_gemm_e8_b200 as e8
from oracle import mx4_oracle as mx
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def cbk():
    cb = e8.Codebook(0)
    yield cb
    cb.free()


def _data(rows, K, dtype, seed, pad=0):
    """[rows, K] slice of a wider device tensor, and its values in binary64."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K + pad, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    if rows > 2:
        x[1] = 0
        x[2, : min(K, 40)] *= 2.0 ** -20
    # halfway points of the grid, so that ties are met
    x[0, : min(K, 8)] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0])[: min(K, 8)]
    x = x.to(DTYPES[dtype]).to(dev())[:, :K]
    return x, x.cpu().double().numpy()


SHAPES = [(1, 1, 0), (1, 32, 0), (1, 4096, 0), (3, 31, 0), (5, 33, 3), (129, 255, 0), (128, 256, 8),
          (37, 257, 0), (200, 1000, 24), (2, 16384, 0), (300, 264, 1)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,K,pad", SHAPES)
def test_encode_and_decode_are_exact(cbk, rows, K, pad, dtype):
    x, v = _data(rows, K, dtype, rows * 7 + K, pad)
    m = e8.e8_mx4_encode(cbk, x)
    c, b = mx.quantise(v)
    p, t = mx.pack(c, b)
    assert np.array_equal(m.codes.cpu().numpy(), p)
    assert np.array_equal(m.scales.cpu().numpy(), t)
    out = e8.e8_mx4_decode_to_bf16(cbk, m)
    assert np.array_equal(out.cpu().double().numpy(), mx.values(c, b, K))


def test_encode_of_a_batch(cbk):
    x = torch.randn(3, 130, 200, device=dev()).bfloat16()
    m = e8.e8_mx4_encode(cbk, x)
    for i in range(3):
        one = e8.e8_mx4_encode(cbk, x[i])
        assert torch.equal(one.codes, m.codes[i]) and torch.equal(one.scales, m.scales[i])
    assert torch.equal(e8.e8_mx4_decode_to_bf16(cbk, m)[2],
                       e8.e8_mx4_decode_to_bf16(cbk, one))
    # matrices of one row that lie further apart
    y = torch.randn(4, 2, 64, device=dev())[:, :1]
    n = e8.e8_mx4_encode(cbk, y)
    assert torch.equal(n.codes[3], e8.e8_mx4_encode(cbk, y[3]).codes)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_extreme_values(cbk, dtype):
    x = torch.zeros(8, 96)
    x[0, 5] = float("inf")
    x[1, 40] = float("nan")
    x[2] = torch.finfo(DTYPES[dtype]).max
    x[3] = torch.finfo(DTYPES[dtype]).smallest_normal
    x[4, :50] = torch.finfo(DTYPES[dtype]).smallest_normal * torch.arange(50) / 16
    x[5] = -0.0
    x[6, 64:] = -float("inf")
    x = x.to(DTYPES[dtype]).to(dev())
    c, b = mx.quantise(x.cpu().double().numpy())
    m = e8.e8_mx4_encode(cbk, x)
    p, t = mx.pack(c, b)
    assert np.array_equal(m.codes.cpu().numpy(), p) and np.array_equal(m.scales.cpu().numpy(), t)
    out = e8.e8_mx4_decode_to_bf16(cbk, m).cpu().double().numpy()
    assert np.array_equal(out, mx.values(c, b, 96), equal_nan=True)


def _check_product(Y, a, w):
    """bf16 rounding of the output: half a step, 2^-8 of the value; fp32 sums of K
    exact products: K additions off by at most 2^-23 of the magnitudes' sum."""
    ref, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    y = Y.cpu().double().numpy()
    K = a.shape[1]
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    fine = ~np.isnan(ref)
    tol = 2.0 ** -8 * np.abs(ref) + K * 2.0 ** -23 * mag + 1e-37
    assert (np.abs(y - ref)[fine] <= tol[fine]).all()
    n = np.linalg.norm(ref[fine])
    assert np.linalg.norm((y - ref)[fine]) <= 2.0 ** -8 * n + 1e-37


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 130, 96), (7, 257, 160), (16, 384, 1024),
            (17, 129, 2080), (33, 512, 4104), (64, 300, 65), (65, 256, 512), (100, 1000, 777),
            (128, 128, 256), (129, 640, 300), (200, 513, 1056), (256, 256, 256), (257, 511, 513),
            (300, 4099, 264), (333, 700, 4104), (512, 1024, 768), (1000, 520, 1000)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(cbk, M, N, K):
    dtype = ("bf16", "f16", "f32")[(M + N + K) % 3]
    x, v = _data(M, K, dtype, M + N, pad=(M % 3) * 5)
    w, wv = _data(N, K, "f32", K)
    m = e8.e8_mx4_encode(cbk, w)
    Y = e8.e8_mx4_gemm(cbk, x, m)
    _check_product(Y, mx.roundtrip(v), mx.roundtrip(wv))
    again = e8.e8_mx4_gemm_codes(cbk, e8.e8_mx4_encode(cbk, x), m)
    assert torch.equal(Y, again)
    assert e8.e8_sync_status(cbk) == e8.E8_OK


def test_products_with_extreme_scales_and_nan(cbk):
    x, _ = _data(40, 320, "f32", 1)
    w, _ = _data(150, 320, "f32", 2)
    x[3] *= 2.0 ** -100
    x[4, 100] = float("nan")
    x[5] *= 2.0 ** 60
    w[7] *= 2.0 ** 50
    w[9, 3] = float("inf")
    w[11] = 0
    Y = e8.e8_mx4_gemm(cbk, x, e8.e8_mx4_encode(cbk, w))
    _check_product(Y, mx.roundtrip(x.cpu().numpy()), mx.roundtrip(w.cpu().numpy()))


def test_rows_and_columns_stay_apart(cbk):
    """A NaN row of X or W touches its own row or column of Y alone, and nothing behind Y
    is written."""
    M, N, K = 70, 200, 416
    x, _ = _data(M, K, "bf16", 3)
    w, _ = _data(N, K, "bf16", 4)
    m = e8.e8_mx4_encode(cbk, w)
    clean = e8.e8_mx4_gemm(cbk, x, m)
    x2 = x.clone()
    x2[11] = float("nan")
    buf = torch.full((M + 4, N), 7.0, dtype=torch.bfloat16, device=dev())
    e8.e8_mx4_gemm(cbk, x2, m, Y=buf[:M])
    keep = torch.arange(M, device=dev()) != 11
    assert torch.equal(buf[:M][keep], clean[keep]) and buf[11].isnan().all()
    assert (buf[M:] == 7).all()


def test_empty_and_refused(cbk):
    w = e8.e8_mx4_encode(cbk, torch.randn(16, 64, device=dev()))
    assert e8.e8_mx4_gemm(cbk, torch.empty(0, 64, device=dev()), w).shape == (0, 16)
    none = e8.e8_mx4_encode(cbk, torch.empty(0, 64, device=dev()))
    assert e8.e8_mx4_gemm(cbk, torch.randn(3, 64, device=dev()), none).shape == (3, 0)
    x = torch.randn(3, 64, device=dev())
    for bad in (lambda: e8.e8_mx4_encode(cbk, x.double()), lambda: e8.e8_mx4_encode(cbk, x.T),
                lambda: e8.e8_mx4_gemm(cbk, x[:, :63], w), lambda: e8.e8_mx4_gemm(cbk, x.cpu(), w),
                lambda: e8.e8_mx4_encode(cbk, x[:1].expand(3, 64)),
                lambda: e8.e8_mx4_gemm(cbk, x, w, Y=torch.empty(3, 16, device=dev())),
                lambda: e8.e8_mx4_gemm(cbk, x, w, workspace=torch.empty(16, dtype=torch.uint8, device=dev()))):
        with pytest.raises(e8.E8Error):
            bad()


def test_streams_and_graph(cbk):
    """Calls on another stream, and a captured call replayed on new inputs."""
    x, _ = _data(20, 512, "bf16", 5)
    w = e8.e8_mx4_encode(cbk, _data(300, 512, "f32", 6)[0])
    want = e8.e8_mx4_gemm(cbk, x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = e8.e8_mx4_gemm(cbk, x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    static = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = e8.e8_mx4_gemm(cbk, static, w)
        z = e8.e8_mx4_decode_to_bf16(cbk, e8.e8_mx4_encode(cbk, y))
    for seed in (8, 9):
        static.copy_(_data(20, 512, "bf16", seed)[0])
        g.replay()
        torch.cuda.synchronize()
        ref = e8.e8_mx4_gemm(cbk, static, w)
        assert torch.equal(y, ref)
        assert torch.equal(z, e8.e8_mx4_decode_to_bf16(cbk, e8.e8_mx4_encode(cbk, ref)))


@pytest.mark.parametrize("M,N,K", [(300, 8000, 100), (512, 5120, 320), (1000, 5000, 1000), (700, 16, 544),
                                   (260, 8, 33), (2049, 768, 130), (9, 2048, 8200), (8, 2050, 4100),
                                   (3, 130, 2049), (256, 1024, 2304)])
def test_product_tiles_and_tails(cbk, M, N, K):
    """Many tiles and few, columns that end inside one, K tails of one to four 64-column steps."""
    x, v = _data(M, K, "bf16", M + N, pad=(M % 2) * 8)
    w, wv = _data(N, K, "bf16", K)
    m = e8.e8_mx4_encode(cbk, w)
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device=dev())
    Y = buf[:M * N].view(M, N)
    e8.e8_mx4_gemm(cbk, x, m, Y=Y)
    _check_product(Y, mx.roundtrip(v), mx.roundtrip(wv))
    assert (buf[M * N:] == 7).all()
    assert torch.equal(Y, e8.e8_mx4_gemm_codes(cbk, e8.e8_mx4_encode(cbk, x), m))
    assert e8.e8_sync_status(cbk) == e8.E8_OK


@pytest.mark.parametrize("M", [1, 5, 8, 9, 40, 300])
def test_nan_and_unaligned_tokens_at_every_size(cbk, M):
    K, N = 1000, 200
    x, _ = _data(M, K + 3, "f16", M)
    x[M - 1, 500] = float("nan")
    w, _ = _data(N, K, "f32", 2)
    w[9, 3] = float("inf")
    part = x[:, 3:]                                   # rows start anywhere
    Y = e8.e8_mx4_gemm(cbk, part, e8.e8_mx4_encode(cbk, w))
    _check_product(Y, mx.roundtrip(part.cpu().double().numpy()), mx.roundtrip(w.cpu().double().numpy()))
    assert Y[M - 1].isnan().all() and Y[:, 9].isnan().all()


def test_products_on_two_streams_and_in_two_graphs(cbk):
    x = [_data(M, 1024, "bf16", M)[0] for M in (4, 50, 400)]
    m = e8.e8_mx4_encode(cbk, _data(1500, 1024, "bf16", 1)[0])
    want = [e8.e8_mx4_gemm(cbk, v, m) for v in x]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            got.append([e8.e8_mx4_gemm(cbk, v, m, stream=s) for v in x])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for ys in got for a, b in zip(ys, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys = [e8.e8_mx4_gemm(cbk, v, m) for v in x]
        graphs.append((g, ys))
    for (g, ys), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            for _ in range(20):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, ys in graphs for a, b in zip(ys, want))
    assert e8.e8_sync_status(cbk) == e8.E8_OK


@pytest.mark.parametrize("rows,K", [(5, 8), (9, 31), (130, 241), (33, 248), (40, 249), (7, 255), (70, 257), (12, 263),
                                    (3, 497), (200, 1000), (600, 1032)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off", [0, 1, 2, 3, 5])
def test_rows_at_any_alignment(cbk, rows, K, dtype, off):
    """Rows that start at every place of a 16-byte word, values there and back, nothing
    written behind the last row."""
    t = dict(bf16=torch.bfloat16, f16=torch.float16, f32=torch.float32)[dtype]
    flat = torch.randn(rows * K + off, device=dev(), generator=torch.Generator(device="cuda").manual_seed(K)).to(t)
    x = flat[off:].view(rows, K)
    m = e8.e8_mx4_encode(cbk, x)
    want = e8.e8_mx4_encode(cbk, torch.cat([x, x.new_zeros(rows, -K % 8)], 1)[:, :K])   # rows on 16 bytes
    assert torch.equal(m.codes, want.codes) and torch.equal(m.scales, want.scales)
    buf = torch.full((rows * K + 64,), 7.0, dtype=torch.bfloat16, device=dev())
    e8.e8_mx4_decode_to_bf16(cbk, m, out=buf[:rows * K].view(rows, K))
    assert np.array_equal(buf[:rows * K].view(rows, K).float().cpu().numpy(),
                          mx.roundtrip(x.cpu().double().numpy()).astype(np.float32))
    assert (buf[rows * K:] == 7).all()


def test_calls_in_a_row_and_between_other_work(cbk):
    """Each kernel may start while the one before it ends: results of calls in a row, after
    copies, fills, other kernels and other streams, eagerly and captured, are those of calls
    apart from each other."""
    w0, w1 = (_data(640, 640, "bf16", s)[0] for s in (1, 2))
    x = {M: _data(M, 640, "bf16", M)[0] for M in (1, 8, 33, 300)}
    m0 = e8.e8_mx4_encode(cbk, w0)
    out = e8.Mx4Matrix(torch.empty_like(m0.codes), torch.empty_like(m0.scales), 640, 640)
    side = torch.cuda.Stream()

    def chain(M, apart):
        gap = torch.cuda.synchronize if apart else (lambda: None)
        a = x[M].clone()
        gap()
        src = torch.empty_like(w0).copy_(w1)                       # a copy before the encoder
        gap()
        e8.e8_mx4_encode(cbk, src, out=out)                        # weights that the next call reads
        gap()
        y = e8.e8_mx4_gemm(cbk, a, out)
        gap()
        z = e8.e8_mx4_gemm(cbk, y, m0)
        gap()
        back = e8.e8_mx4_decode_to_bf16(cbk, out)
        gap()
        e8.e8_mx4_encode(cbk, back + 1, out=out)                   # written again after it was read
        gap()
        src.zero_()
        gap()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            u = e8.e8_mx4_gemm(cbk, z, out)
        torch.cuda.current_stream().wait_stream(side)
        gap()
        v = e8.e8_mx4_gemm(cbk, u, m0)
        u.record_stream(torch.cuda.current_stream())
        e8.e8_mx4_encode(cbk, src, out=out)
        return y, z, back, u, v

    for M in x:
        want = chain(M, True)
        torch.cuda.synchronize()
        for _ in range(10):
            got = chain(M, False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = chain(M, False)
        for _ in range(10):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert e8.e8_sync_status(cbk) == e8.E8_OK


def test_a_captured_call_may_be_the_first_or_follow_a_fill(cbk):
    x = _data(2, 256, "bf16", 1)[0]
    m = e8.e8_mx4_encode(cbk, _data(128, 256, "bf16", 2)[0])
    want = e8.e8_mx4_gemm(cbk, x, m)
    pad = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    for before in (lambda: None, lambda: pad.zero_(), lambda: pad[:1 << 19].copy_(pad[1 << 19:])):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            before()
            y = e8.e8_mx4_gemm(cbk, x, m)
            back = e8.e8_mx4_decode_to_bf16(cbk, m)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(back, e8.e8_mx4_decode_to_bf16(cbk, m))
