"""Host side of the microscaled 4-bit calls and of the mixture-of-experts layer: sizes, and
every refusal before the first CUDA call (this host has no GPU: a CUDA call would answer
E8_ECUDA or E8_EDEVICE).  Handles and addresses are stand-ins that are never read."""
import pytest

import decode_gemm_e8_b200 as e8
from decode_gemm_e8_b200 import build as e8build
from oracle import mx4_oracle as mx

CB, D = 1 << 20, 1 << 24


@pytest.fixture(scope="module")
def lib():
    e8build.build()
    return e8.load_library()


def test_sizes(lib):
    for rows, K in ((1, 1), (1, 32), (128, 128), (129, 129), (4099, 4104), (14336, 4096)):
        assert lib.e8_mx4_code_bytes(rows, K) == mx.code_bytes(rows, K)
        assert lib.e8_mx4_scale_bytes(rows, K) == mx.scale_bytes(rows, K)
    assert lib.e8_mx4_code_bytes(0, 5) == 0 and lib.e8_mx4_scale_bytes(0, 5) == 0
    # past 32 bits
    assert lib.e8_mx4_code_bytes(2 ** 31 - 1, 2 ** 20) == (2 ** 31 - 1) * 2 ** 19
    for bad in ((-1, 32), (1, 0), (2 ** 31, 32), (1, 2 ** 31)):
        assert lib.e8_mx4_code_bytes(*bad) == -1 and lib.e8_mx4_scale_bytes(*bad) == -1
    assert lib.e8_mx4_gemm_workspace_bytes(5, 100, 300) >= mx.code_bytes(5, 300) + mx.scale_bytes(5, 300)
    for bad in ((0, 8, 32), (8, 0, 32), (8, 8, 0), (-1, 8, 32)):
        assert lib.e8_mx4_gemm_workspace_bytes(*bad) == 0
    assert lib.e8_mx4_moe_workspace_bytes(4, 256, 8, 2, 128) > 0
    for bad in ((65, 256, 8, 2, 128), (4, 200, 8, 2, 128), (4, 256, 8, 9, 128), (4, 256, 8, 2, 100),
                (4, 256, 513, 2, 128), (4, 256, 8, 0, 128), (4, 256, 64, 17, 128), (0, 256, 8, 2, 128),
                (4, 65536, 8, 2, 128)):
        assert lib.e8_mx4_moe_workspace_bytes(*bad) == 0


def test_encode_and_decode_refusals(lib):
    def enc(cb=CB, x=D, dt=0, batch=1, rows=4, K=64, ldx=64, c=D, s=D):
        return lib.e8_mx4_encode(cb, x, dt, batch, rows, K, ldx, c, s, None)

    for bad in (dict(cb=None), dict(x=None), dict(x=D + 1), dict(dt=3), dict(dt=-1), dict(batch=-1), dict(rows=-1),
                dict(K=0), dict(ldx=63), dict(c=None), dict(s=None), dict(c=D + 8), dict(s=D + 4),
                dict(dt=2, x=D + 2), dict(ldx=2 ** 31)):
        assert enc(**bad) == e8.E8_EINVAL, bad
    assert enc(rows=0) == e8.E8_OK and enc(batch=0) == e8.E8_OK

    def dec(cb=CB, c=D, s=D, batch=1, rows=4, K=64, o=D):
        return lib.e8_mx4_decode_to_bf16(cb, c, s, batch, rows, K, o, None)

    for bad in (dict(cb=None), dict(c=None), dict(s=None), dict(o=None), dict(o=D + 2), dict(c=D + 4), dict(K=0),
                dict(rows=-2)):
        assert dec(**bad) == e8.E8_EINVAL, bad
    assert dec(rows=0) == e8.E8_OK


def test_product_refusals(lib):
    def mul(cb=CB, x=D, dt=0, M=4, ldx=64, c=D, s=D, N=100, K=64, y=D, ws=D, n=None):
        n = lib.e8_mx4_gemm_workspace_bytes(M, N, K) if n is None else n
        return lib.e8_mx4_gemm(cb, x, dt, M, ldx, c, s, N, K, y, ws, n, None)

    for bad in (dict(cb=None), dict(x=None), dict(dt=7), dict(M=-1), dict(N=-1), dict(K=0), dict(ldx=10), dict(c=None),
                dict(s=D + 8), dict(y=None), dict(y=D + 2), dict(x=D + 1)):
        assert mul(**bad) == e8.E8_EINVAL, bad
    assert mul(ws=None) == e8.E8_EWORKSPACE and mul(ws=D + 4) == e8.E8_EWORKSPACE and mul(n=100) == e8.E8_EWORKSPACE
    assert mul(M=0) == e8.E8_OK and mul(N=0) == e8.E8_OK

    def codes(cb=CB, a=D, b=D, M=4, c=D, s=D, N=100, K=64, y=D, ws=D, n=1 << 40):
        return lib.e8_mx4_gemm_codes(cb, a, b, M, c, s, N, K, y, ws, n, None)

    for bad in (dict(cb=None), dict(a=None), dict(b=None), dict(a=D + 8), dict(c=D + 1), dict(s=None), dict(y=D + 8)):
        assert codes(**bad) == e8.E8_EINVAL, bad
    assert codes(M=0) == e8.E8_OK


def test_moe_refusals(lib):
    def moe(cb=CB, x=D, T=4, H=256, r=D, E=8, k=2, c13=D, s13=D, inner=128, c2=D, s2=D, y=D, ids=None, p=None, ws=D,
            n=1 << 40):
        return lib.e8_mx4_moe(cb, x, T, H, r, E, k, 1, c13, s13, inner, c2, s2, y, ids, p, ws, n, None)

    for bad in (dict(cb=None), dict(x=None), dict(x=D + 8), dict(T=65), dict(T=-1), dict(H=192), dict(H=0), dict(E=0),
                dict(E=513), dict(k=0), dict(k=9), dict(E=64, k=17), dict(inner=130), dict(c13=D + 16), dict(s13=None),
                dict(c2=None), dict(s2=D + 16), dict(r=None), dict(y=None), dict(ids=D + 4), dict(p=D + 4)):
        assert moe(**bad) == e8.E8_EINVAL, bad
    assert moe(ws=None) == e8.E8_EWORKSPACE and moe(n=64) == e8.E8_EWORKSPACE and moe(ws=D + 8) == e8.E8_EWORKSPACE
    assert moe(T=0) == e8.E8_OK
