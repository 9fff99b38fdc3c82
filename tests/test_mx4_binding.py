"""What the Python binding of the microscaled 4-bit calls refuses by itself (no GPU)."""
import pytest
import torch

import decode_gemm_e8_b200 as e8


def _parts(rows=130, K=200, dtype=torch.uint8):
    return torch.zeros(rows, (K + 31) // 32 * 16, dtype=dtype), torch.zeros(2 * 2 * 512, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.int16, torch.int32, torch.float32, torch.int64])
def test_a_matrix_is_made_of_bytes(dtype):
    c, s = _parts()
    wide_c, wide_s = _parts(dtype=dtype)
    for parts in ((wide_c, s), (c, wide_s), (wide_c, wide_s)):
        with pytest.raises(e8.E8Error) as err:
            e8.Mx4Matrix(*parts, 130, 200)
        assert err.value.code == e8.E8_EINVAL
    for one in (torch.uint8, torch.int8, torch.float8_e4m3fn):
        m = e8.Mx4Matrix(c.view(one), s.view(one), 130, 200)
        assert m.codes.shape == (130, 112) and m.batch is None


def test_a_matrix_has_the_bytes_of_its_shape():
    c, s = _parts()
    e8.Mx4Matrix(c, s, 130, 200)
    for bad in ((c, s, 129, 200), (c, s, 130, 225), (c, s[1:], 130, 200), (c[:-1], s, 130, 200), (c, s, -1, 200),
                (c, s, 130, 0), (c, s, 130, 200, 2), (c, s, 130, 200, 0)):
        with pytest.raises(e8.E8Error):
            e8.Mx4Matrix(*bad)
