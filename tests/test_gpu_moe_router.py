"""Choice of experts where an fp32 sum of the logits would choose others."""
import numpy as np
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


def _fp32_logit(row):
    """The router's sum over x = 1 in its own order (8 values a lane and step of 256, lanes
    joined in pairs, then parts), but in fp32."""
    parts = []
    for chunk in np.split(row.astype(np.float32), len(row) // 256):
        lanes = np.zeros(32, np.float32)
        for i in range(8):
            lanes = (lanes + chunk.reshape(32, 8)[:, i]).astype(np.float32)
        while len(lanes) > 1:
            lanes = (lanes[0::2] + lanes[1::2]).astype(np.float32)
        parts.append(lanes[0])
    total = np.float32(0)
    for p in parts:
        total = np.float32(total + p)
    return total


@pytest.mark.parametrize("T", [1, 3, 30])
def test_logits_that_fp32_would_order_otherwise(cbk, T):
    """Large terms that cancel stand in one lane, in two lanes, in two steps and at both ends,
    with small terms between them that an fp32 sum would lose: the choice follows 64 bits."""
    width, E = 1024, 6
    r = np.zeros((E, width))
    for e, (i, j) in enumerate([(None, None), (0, 2), (0, 8), (0, 256), (0, 1023)]):
        r[e, 10:250] = 1
        if i is not None:
            r[e, i], r[e, j] = 2.0 ** 30, -2.0 ** 30
            r[e, 1], r[e, 10 + e] = 1 + 2.0 ** -(7 - e), 0          # 240 + 2^-(7 - e) in all
    logits = r.sum(1)
    assert (np.argsort(-logits, kind="stable") == [4, 3, 2, 1, 0, 5]).all()
    narrow = np.array([_fp32_logit(row) for row in r])
    assert (np.argsort(-narrow, kind="stable") != [4, 3, 2, 1, 0, 5]).any() and narrow.argmax() == 0
    router = torch.tensor(r).bfloat16().to(dev())
    assert (router.double().cpu().numpy() == r).all()
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, up, down = (torch.randn(E, *s, generator=g, device=dev()) for s in ((128, width), (128, width), (width, 128)))
    w13, w2 = e8.e8_mx4_moe_pack(cbk, gate, up, down)
    x = torch.ones(T, width, dtype=torch.bfloat16, device=dev())
    ids = torch.empty(T, 5, dtype=torch.int32, device=dev())
    e8.e8_mx4_moe(cbk, x, router, w13, w2, 5, experts=ids)
    assert (ids.cpu() == torch.tensor([4, 3, 2, 1, 0])).all()
