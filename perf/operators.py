"""Microscaled 4-bit operators: what is measured of them, and their plain forms.

Three operators: quantising to blocks of 32 four-bit floats that share a
power-of-two scale and reading them back, the product of two matrices held in
that form, and a mixture-of-experts layer for a few tokens whose experts are
held in it.

The form: along K, blocks of 32 values; a = max|x| of the block,
E = clamp(floor(log2 a) - 2, -127, 125) (-127 for a block of zeros), and every
value is x / 2^E rounded to nearest even onto {0, .5, 1, 1.5, 2, 3, 4, 6},
saturating at 6.  Codes: uint8 [rows][16 * ceil(K / 32)], value 2i in the low
nibble (sign in bit 3).  Scales: bytes E + 127 in tiles of 128 rows by 4 blocks
of 512 bytes, row r and block b of a tile at
(r % 32) * 16 + (r / 32) * 4 + b, the tiles of a row of tiles one after the other.
"""
import math

import torch

own = False

# sizes of an 8B decoder layer's projections (hidden 4096, MLP 14336), as the
# framework's own benchmark has them, and generic ones around them
_LARGEST_QUANT = 14336 * 4096
_LARGEST_PRODUCT = 4096 * 14336 * 4096
_LARGEST_MOE = 8 * 4096 * 14336


def listed():
    return [
        # one token's hidden state, between two layers of a decode step
        {"name": "quant_token", "op": "quant", "rows": 1, "K": 4096, "dtype": "bf16", "pad": 0},
        # a prompt's activations, cut out of a wider buffer (row stride > K)
        {"name": "quant_prompt_strided", "op": "quant", "rows": 2048, "K": 4096, "dtype": "bf16", "pad": 1024},
        # odd sizes: the last block of every row is short
        {"name": "quant_ragged", "op": "quant", "rows": 1021, "K": 4099, "dtype": "f16", "pad": 0},
        # an MLP up-projection's weights, fp32 as a checkpoint conversion has them
        {"name": "quant_weights", "op": "quant", "rows": 14336, "K": 4096, "dtype": "f32", "pad": 0},
        # single-token decode, a square projection
        {"name": "product_m1_4096", "op": "product", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16"},
        # small-batch decode, MLP up-projection
        {"name": "product_m16_mlp", "op": "product", "M": 16, "N": 14336, "K": 4096, "dtype": "bf16"},
        # a chunk of mixed requests: nothing is a multiple of a tile
        {"name": "product_ragged", "op": "product", "M": 333, "N": 4099, "K": 4104, "dtype": "f16"},
        # prefill of 4096 tokens, MLP up-projection
        {"name": "product_prefill", "op": "product", "M": 4096, "N": 14336, "K": 4096, "dtype": "bf16"},
        # one token, many small experts: latency
        {"name": "moe_token_e64", "op": "moe", "T": 1, "E": 64, "topk": 8, "H": 2048, "I": 1024, "renorm": True},
        # one token, few large experts: weight streaming
        {"name": "moe_token_e8_large", "op": "moe", "T": 1, "E": 8, "topk": 2, "H": 4096, "I": 14336, "renorm": True},
        # odd everything, probabilities over all experts
        {"name": "moe_odd", "op": "moe", "T": 33, "E": 13, "topk": 3, "H": 1152, "I": 640, "renorm": False},
        # a full decode batch: nearly every expert is hit
        {"name": "moe_batch_e128", "op": "moe", "T": 64, "E": 128, "topk": 8, "H": 2048, "I": 768, "renorm": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "moe"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op == "quant":
        K = _log(rng, 32, 16384)
        rows = _log(rng, 1, min(16384, _LARGEST_QUANT // K))
        return {"op": op, "rows": rows, "K": K, "dtype": dtype, "pad": rng.choice([0, 0, 8, 37, 512])}
    if op == "product":
        K, N = _log(rng, 128, 14336), _log(rng, 128, 14336)
        M = _log(rng, 1, min(4096, _LARGEST_PRODUCT // (K * N)))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": dtype}
    E = _log(rng, 2, 128)
    H = 128 * _log(rng, 4, 32)
    inner = 128 * _log(rng, 2, max(2, min(112, _LARGEST_MOE // (128 * E * H))))
    return {"op": op, "T": _log(rng, 1, 64), "E": E, "topk": rng.randint(1, min(8, E)), "H": H, "I": inner,
            "renorm": rng.choice([True, False])}


# ------------------------------------------------------------------ plain ---
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _quantise(x):
    """x [..., rows, K] -> (magnitude codes with sign in bit 3 as int32
    [..., rows, Kp], scale bytes int32 [..., rows, Kp / 32])."""
    x = x.float()
    K = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -K % 32)).unflatten(-1, (-1, 32))
    a = x.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 3, -127).clamp(-127, 125)
    inv = ((127 - e) << 23).view(torch.float32)   # 2^-e
    v = (x * inv).abs()
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    q = (torch.round(v / step) * step).clamp(max=6.0)
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.int32)
    code = code + 8 * torch.signbit(x).to(torch.int32)
    return code.flatten(-2), (e + 127).squeeze(-1)


def _values(code, byte):
    """What codes and scale bytes stand for, fp32 [..., rows, Kp]."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=code.device)
    scale = torch.where(byte == 0, torch.full((), 2.0 ** -127, device=code.device), (byte << 23).view(torch.float32))
    return (table[code].unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def _pack(code, byte):
    """Codes and scale bytes -> (packed uint8 [..., rows, Kp / 2], tiled scale bytes uint8 [..., bytes])."""
    c = code.to(torch.uint8)
    packed = (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()
    rows, kb = byte.shape[-2:]
    s = torch.nn.functional.pad(byte.to(torch.uint8), (0, -kb % 4, 0, -rows % 128))
    s = s.unflatten(-1, (-1, 4)).unflatten(-3, (-1, 4, 32))     # [..., tile, r / 32, r % 32, kq, 4]
    s = s.movedim(-2, -4).movedim(-3, -2).contiguous()          # [..., tile, kq, r % 32, r / 32, 4]
    return packed, s.flatten(-5)


def _unpack(packed, tiled, rows, K):
    code = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).int()
    kq = (K + 127) // 128
    s = tiled.unflatten(-1, (-1, kq, 32, 4, 4)).movedim(-2, -3).movedim(-4, -2)
    s = s.flatten(-2).flatten(-4, -2)
    return code, s[..., :rows, :(K + 31) // 32].int()


def _read(m):
    return _values(*_unpack(m["codes"], m["scales"], m["rows"], m["K"]))


def _plain_moe(s):
    x, k = s["x"], s["topk"]
    logits = x.double() @ s["router"].double().T
    top, which = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, which = top[:, :k], which[:, :k]
    base = top[:, :1]
    num = torch.exp((top - base).float())
    p = num / (num if s["renorm"] else torch.exp((logits - base).float())).sum(-1, keepdim=True)
    share = torch.zeros_like(logits, dtype=torch.float32).scatter_(1, which, p)      # [T, E]
    gu = x.float() @ _read(s["w13"]).transpose(-1, -2)                                # [E, T, 2 I]
    g, u = gu[..., 0::2], gu[..., 1::2]
    h = g / (1 + torch.exp(-g)) * u
    o = h @ _read(s["w2"]).transpose(-1, -2)                                          # [E, T, H]
    return (o * share.T.unsqueeze(-1)).sum(0).bfloat16()


# -------------------------------------------------------------------- run ---
_handle = None


def _matrix(e8, m, batch=None):
    return e8.Mx4Matrix(m["codes"], m["scales"], m["rows"], m["K"], batch=batch)


def run(state):
    if own:
        global _handle
        import decode_gemm_e8_b200 as e8
        if _handle is None:
            _handle = e8.e8_codebook_build(torch.cuda.current_device())
        if state["op"] == "quant":
            return e8.e8_mx4_decode_to_bf16(_handle, e8.e8_mx4_encode(_handle, state["x"]))
        if state["op"] == "product":
            return e8.e8_mx4_gemm(_handle, state["x"], _matrix(e8, state["w"]))
        return e8.e8_mx4_moe(_handle, state["x"], state["router"], _matrix(e8, state["w13"], state["E"]),
                             _matrix(e8, state["w2"], state["E"]), state["topk"], renormalize=state["renorm"])
    if state["op"] == "quant":
        x = state["x"]
        return _values(*_quantise(x))[:, :x.shape[1]].bfloat16()
    if state["op"] == "product":
        return (_values(*_quantise(state["x"])) @ _read(state["w"]).T).bfloat16()
    return _plain_moe(state)


# ---------------------------------------------------------------- prepare ---
def _activations(g, rows, K, dtype, pad=0):
    """Hidden states: unit normal, one column in 64 eight times as large, now
    and then a row of zeros (a padded token), rows of different loudness."""
    x = torch.randn(rows, K + pad, generator=g, device="cuda")
    loud = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    outlier = 1 + 7 * (torch.rand(1, K + pad, generator=g, device="cuda") < 1 / 64)
    keep = torch.rand(rows, 1, generator=g, device="cuda") >= (0.02 if rows > 16 else 0.0)
    return (x * loud * outlier * keep).to(_TYPES[dtype])[:, :K]


def _weights(g, batch, rows, K, std):
    """Normal weights in the packed form; `batch` matrices one after the other."""
    packed, tiled = [], []
    for _ in range(batch):
        p, t = _pack(*_quantise(std * torch.randn(rows, K, generator=g, device="cuda")))
        packed.append(p)
        tiled.append(t)
    return {"codes": torch.stack(packed) if batch > 1 else packed[0].unsqueeze(0),
            "scales": torch.stack(tiled) if batch > 1 else tiled[0].unsqueeze(0), "rows": rows, "K": K}


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "quant":
        return {"op": op, "x": _activations(g, case["rows"], case["K"], case["dtype"], case["pad"])}
    if op == "product":
        w = _weights(g, 1, case["N"], case["K"], 0.02)
        w["codes"], w["scales"] = w["codes"][0], w["scales"][0]
        return {"op": op, "x": _activations(g, case["M"], case["K"], case["dtype"]), "w": w}
    T, E, H, inner = case["T"], case["E"], case["H"], case["I"]
    return {"op": op, "E": E, "topk": case["topk"], "renorm": case["renorm"],
            "x": _activations(g, T, H, "bf16"),
            "router": (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).bfloat16(),
            "w13": _weights(g, E, 2 * inner, H, H ** -0.5), "w2": _weights(g, E, H, inner, inner ** -0.5)}


def prepare(case, seed):
    return _inputs(case, seed)


def work(case):
    packed = 17 / 32   # bytes a value: four bits and its share of a scale byte
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": n * (size + 2 * packed + 2), "flops": 4 * n}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size + N * K * packed + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k, H, inner = case["T"], case["E"], case["topk"], case["H"], case["I"]
    hit = E * (1 - (1 - k / E) ** T)   # experts that some token is sent to, on the average
    return {"bytes": hit * 3 * H * inner * packed + 2 * E * H + 4 * T * H, "flops": 6 * T * k * H * inner + 2 * T * E * H}


# ------------------------------------------------------------------ exact ---
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _two_to(E):
    """2^E exactly (a library power may be off in its last bit)."""
    return ((E.long() + 1023) << 52).view(torch.float64)


def _exact_quantise(x):
    """Nearest grid value by comparison with the midpoints; at a midpoint the
    value of even code."""
    x = x.double()
    K = x.shape[1]
    b = torch.nn.functional.pad(x, (0, -K % 32)).reshape(x.shape[0], -1, 32)
    a = b.abs().amax(2, keepdim=True)
    E = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))) - 2
    E = torch.where(_two_to(E + 3) <= a, E + 1, E)      # log2 may round across a power of two
    E = torch.where(_two_to(E + 2) > a, E - 1, E)
    E = torch.where(a > 0, E, torch.full_like(E, -127)).clamp(-127, 125)
    v = b.abs() / _two_to(E)
    out = torch.zeros_like(v)
    for i in range(1, 8):
        mid = (_GRID[i - 1] + _GRID[i]) / 2
        up = (v > mid) | ((v == mid) if i % 2 == 0 else torch.zeros_like(v, dtype=torch.bool))
        out = torch.where(up, torch.full_like(v, _GRID[i]), out)
    out = out * _two_to(E)
    return torch.where(b < 0, -out, out).reshape(x.shape[0], -1)[:, :K]


def _exact_read(codes, scales, rows, K):
    """Codes and tiled scales of one matrix, read by their addresses."""
    dev = codes.device
    r = torch.arange(rows, device=dev).unsqueeze(1)
    k = torch.arange(K, device=dev).unsqueeze(0)
    nib = (codes[r, k // 2].long() >> (4 * (k % 2))) & 15
    b = k // 32
    at = ((r // 128) * ((K + 127) // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    grid = torch.tensor(_GRID, dtype=torch.float64, device=dev)
    v = grid[nib & 7] * _two_to(scales[at].long() - 127)
    return torch.where(nib > 7, -v, v)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "quant":
        return _exact_quantise(s["x"])
    if case["op"] == "product":
        w = s["w"]
        return _exact_quantise(s["x"]) @ _exact_read(w["codes"], w["scales"], w["rows"], w["K"]).T
    x, E, k = s["x"].double(), case["E"], case["topk"]
    logits = x @ s["router"].double().T
    y = torch.zeros_like(x)
    order = torch.argsort(-logits, dim=1, stable=True)[:, :k]
    full = torch.softmax(logits, 1)
    for e in range(E):
        rows = (order == e).any(1).nonzero()[:, 0]
        if not len(rows):
            continue
        p = full[rows, e]
        if case["renorm"]:
            p = p / full[rows].gather(1, order[rows]).sum(1)
        gu = x[rows] @ _exact_read(s["w13"]["codes"][e], s["w13"]["scales"][e], 2 * case["I"], case["H"]).T
        h = torch.nn.functional.silu(gu[:, 0::2]) * gu[:, 1::2]
        y[rows] += p.unsqueeze(1) * (h @ _exact_read(s["w2"]["codes"][e], s["w2"]["scales"][e], case["H"], case["I"]).T)
    return y
