"""Every output of the persistent kernel, over several rounds of tiles, against the
64-bit form on the GPU; the bounds are those of act8_reference.py, element by
element, in torch."""
import math

import pytest
import torch

from act8_reference import U
from post_weight_quantization_26_b200 import synth

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_26_b200 import build, gptq
    build.build()
    gptq.load_library()
    return gptq


def layer(d_row, d_col, group, seed, scale):
    words, s, z = synth.gen_packed_layer(d_row, d_col, group, seed)
    return words.cuda(), (s * scale).cuda(), z.cuda()


def acts(n, d, xg):
    gen = torch.Generator().manual_seed(n + d)
    codes = torch.randint(-127, 128, (n, d), generator=gen, dtype=I8).cuda()
    return codes, torch.exp(torch.randn(n, -(-d // 128) if xg else 1, generator=gen)).cuda()


def product(L, group, codes, scales):
    """Y and its bound, (m + 16) u sum over runs |sx sw P|."""
    words, s, z = L
    rows, d = words.shape[0], codes.shape[1]
    q = torch.empty(rows, d, dtype=torch.float64, device="cuda")
    for k in range(8):
        q[:, k::8] = (words.view(torch.int32).long() >> (4 * k)) % 16
    run = math.gcd(group, 128) if group else 128
    y = torch.zeros(codes.shape[0], rows, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for k in range(0, d, run):
        e, g = min(d, k + run), k // group if group else 0
        term = codes[:, k:e].double() @ (q[:, k:e] - z[:, g:g + 1].double()).T
        term *= scales[:, (k // 128 if scales.shape[1] > 1 else 0)].double()[:, None]
        term *= s[:, g].double()[None, :]
        y += term
        mag += term.abs()
    return y, (-(-d // run) + 16) * U * mag


def worst(got, ref, tol):
    assert torch.isfinite(got).all()
    over = (got.double() - ref).abs() / (tol + 1e-40)
    assert float(over.max()) <= 1.0, f"worst error over bound {float(over.max()):.3f}"


# rows, columns, weight group, tokens: a tile for every SM and more, two to eight
# rounds of them, the last one partial; runs of 32, 64 and 128 columns and across chunks
@pytest.mark.parametrize("shape", [(130, 160, 0, 50001), (300, 416, 32, 25003), (129, 640, 128, 40010),
                                   (257, 384, 64, 33333), (200, 1024, 256, 45001), (64, 128, 128, 140001)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("xg", [0, 128])
def test_every_token(G, shape, xg):
    rows, cols, group, n = shape
    gate, up = layer(rows, cols, group, 1, 0.02), layer(rows, cols, group, 2, 0.02)
    codes, scales = acts(n, cols, xg)
    cfg = G.make_config(group_size=group)
    y = G.gptq_w4a8_matmul(*gate, cfg, codes, scales, dtype=F32)
    yb = G.gptq_w4a8_matmul(*gate, cfg, codes, scales, dtype=BF)
    hf = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=F32)
    h8, hs = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=I8)
    assert G.gptq_device_status() == 0
    g, dg = product(gate, group, codes, scales)
    worst(y, g, dg)
    worst(yb, g, dg + 2.0 ** -8 * g.abs())
    u, du = product(up, group, codes, scales)
    silu = g / (1.0 + torch.exp(-g))
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 8 * U * h.abs()
    worst(hf, h, dh)
    for b in range(hs.shape[1]):  # a scale's block of 128 rows
        part = slice(128 * b, min(rows, 128 * b + 128))
        s, top = hs[:, b].double(), h[:, part].abs().amax(1)
        assert ((s - top / 127).abs() <= dh[:, part].amax(1) / 127 + 2 * U * top / 127 + 2.0 ** -149).all()
        worst(h8[:, part].double() * s[:, None], h[:, part],
              (0.5 + 127 * 4 * U) * s[:, None] + dh[:, part] + 2.0 ** -149)
