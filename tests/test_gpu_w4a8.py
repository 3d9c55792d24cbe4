"""The products of packed 4-bit layers with 8-bit activations, plain and
gated, against their 64-bit forms; the bounds are derived in act8_reference.py."""
import numpy as np
import pytest
import torch

import act8_reference as R
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


def layer(d_row, d_col, group, seed=0):
    return tuple(t.cuda() for t in synth.gen_packed_layer(d_row, d_col, group, seed))


def acts(n, d, xg, seed=0):
    """Random codes over the whole range and scales that differ widely."""
    gen = torch.Generator().manual_seed(1000 + seed + 3 * n + d)
    codes = torch.empty((n, (d + 15) // 16 * 16), dtype=I8, device="cuda")[:, :d]
    codes.copy_(torch.randint(-127, 128, (n, d), generator=gen, dtype=I8))
    scales = torch.exp(torch.randn(n, -(-d // 128) if xg else 1, generator=gen)).cuda()
    return codes, scales


def np_layer(L):
    return tuple(t.cpu().numpy() for t in L)


def check_matmul(G, L, group, codes, scales, dtype, Y=None, **kw):
    cfg = G.make_config(bits=4, group_size=group, **kw)
    y = G.gptq_w4a8_matmul(*L, cfg, codes, scales, Y=Y, dtype=dtype)
    assert y.dtype == dtype and G.gptq_device_status() == 0
    ref, bound = R.product(*np_layer(L), group, codes.cpu().numpy(), scales.cpu().numpy())
    R.check_float(y.double().cpu().numpy(), ref, bound, bf16=dtype == BF)
    return y


def check_gated(G, gate, up, group, codes, scales, dtype, out=None):
    cfg = G.make_config(bits=4, group_size=group)
    got = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, out=out, dtype=dtype)
    assert G.gptq_device_status() == 0
    ref, bound = R.gated(np_layer(gate), np_layer(up), group, codes.cpu().numpy(),
                         scales.cpu().numpy())
    if dtype == I8:
        R.check_codes(got[0].cpu().numpy(), got[1].cpu().numpy(), ref, bound, 128)
    else:
        R.check_float(got.double().cpu().numpy(), ref, bound, bf16=dtype == BF)
    return got


def small(L):
    """Scales for which silu is neither linear nor saturated."""
    return L[0], L[1] * 0.02, L[2]


# (rows, columns, weight group): single row and column block, odd rows, ragged
# last chunk, every kind of group
SHAPES = [(1, 32, 0), (1, 32, 32), (33, 160, 0), (64, 256, 0), (128, 512, 128), (48, 384, 64),
          (40, 320, 32), (300, 1024, 256), (131, 1152, 128), (257, 2080, 0), (96, 1536, 64),
          (130, 96, 96), (70, 480, 96), (129, 640, 160), (260, 4096, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("n", [1, 3, 8, 9, 17, 40, 64, 65, 129, 300])
@pytest.mark.parametrize("xg", [0, 128])
def test_matmul(G, shape, n, xg):
    rows, cols, group = shape
    kw = {"block": 32} if group and group % 64 else {}
    check_matmul(G, layer(rows, cols, group, seed=n), group, *acts(n, cols, xg),
                 F32 if (n + rows) % 2 else BF, **kw)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2] not in (96, 160)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("n", [1, 3, 8, 9, 17, 40, 64, 65, 129, 300])
@pytest.mark.parametrize("dtype", [F32, BF, I8])
def test_gated(G, shape, n, dtype):
    rows, cols, group = shape
    check_gated(G, small(layer(rows, cols, group, seed=n)), small(layer(rows, cols, group, seed=n + 1)),
                group, *acts(n, cols, 128 * (n % 2)), dtype)


@pytest.mark.parametrize("n", [2, 20, 100, 500])
def test_what_lies_beside_stays(G, n):
    """Outputs inside wider arrays: columns beside them and rows behind the
    last token stay as they were; inputs may be strided too."""
    rows, cols, group = 200, 384, 128
    gate, up = small(layer(rows, cols, group, 1)), small(layer(rows, cols, group, 2))
    codes, scales = acts(n, cols, 128)
    wide = torch.full((n + 1, cols + 32), -128, dtype=I8, device="cuda")
    wide[:n, 16:16 + cols] = codes
    codes = wide[:n, 16:16 + cols]
    for dtype, fill in ((F32, 7.0), (BF, 7.0)):
        big = torch.full((n + 2, rows + 5), fill, dtype=dtype, device="cuda")
        check_matmul(G, gate, group, codes, scales, dtype, Y=big[:n, 2:2 + rows])
        assert (big[n:] == fill).all() and (big[:, :2] == fill).all() and (big[:, 2 + rows:] == fill).all()
        big.fill_(fill)
        check_gated(G, gate, up, group, codes, scales, dtype, out=big[:n, 2:2 + rows])
        assert (big[n:] == fill).all() and (big[:, :2] == fill).all() and (big[:, 2 + rows:] == fill).all()
    big = torch.full((n + 2, rows + 5), 99, dtype=I8, device="cuda")
    hs = torch.full((n + 1, 2), 3.0, device="cuda")
    check_gated(G, gate, up, group, codes, scales, I8, out=(big[:n, 2:2 + rows], hs[:n]))
    assert (big[n:] == 99).all() and (big[:, :2] == 99).all() and (big[:, 2 + rows:] == 99).all()
    assert (hs[n] == 3.0).all()


@pytest.mark.parametrize("n", [1, 8, 30, 200])
def test_extreme_codes(G, n):
    """The largest sums that a run can reach, all of one sign: codes 0 or 15
    with zero points 15 or 0, activations -128 and 127."""
    rows, cols = 140, 2048
    for group in (0, 64, 128):
        ng = cols // group if group else 1
        for word, zero in ((-1, 0), (0, 15)):
            L = (torch.full((rows, cols // 8), word, dtype=torch.int32, device="cuda"),
                 torch.full((rows, ng), 0.5, device="cuda"),
                 torch.full((rows, ng), zero, dtype=torch.uint8, device="cuda"))
            for c in (-128, 127):
                codes = torch.full((n, cols), c, dtype=I8, device="cuda")
                y = G.gptq_w4a8_matmul(*L, G.make_config(group_size=group), codes,
                                       torch.ones(n, 1, device="cuda"))
                assert (y == 0.5 * c * (15 if zero == 0 else -15) * cols).all()


@pytest.mark.parametrize("n", [1, 40, 200])
def test_nan_scale_stays_in_its_token(G, n):
    rows, cols, group = 130, 512, 128
    gate, up = small(layer(rows, cols, group, 1)), small(layer(rows, cols, group, 2))
    cfg = G.make_config(group_size=group)
    codes, scales = acts(n, cols, 128)
    clean = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=I8)
    scales[n - 1, 2] = float("nan")
    codes[n - 1, 256:384] = 0
    y = G.gptq_w4a8_matmul(*gate, cfg, codes, scales)
    assert torch.isnan(y[n - 1]).all() and torch.isfinite(y[:n - 1]).all()
    h = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=I8)
    assert torch.isnan(h[1][n - 1]).all() and (h[0][n - 1] == 0).all()
    assert torch.equal(h[0][:n - 1], clean[0][:n - 1]) and torch.equal(h[1][:n - 1], clean[1][:n - 1])


@pytest.mark.parametrize("n", [2, 40, 200])
def test_saturated_gate(G, n):
    """Gates far on either side: silu is 0 or the gate itself, and no NaN."""
    rows, cols = 64, 256
    gate, up = layer(rows, cols, 0, 1), small(layer(rows, cols, 0, 2))
    gate = (gate[0], gate[1] * 50.0, gate[2])
    codes, scales = acts(n, cols, 0)
    check_gated(G, gate, up, 0, codes, scales, F32)
    check_gated(G, gate, up, 0, codes, scales, I8)
    h, hs = G.gptq_w4a8_gated(gate, up, G.make_config(), torch.zeros_like(codes), scales, dtype=I8)
    assert (h == 0).all() and (hs == 0).all()


def test_no_tokens(G):
    L = layer(64, 256, 0)
    codes, scales = acts(0, 256, 0)
    assert G.gptq_w4a8_matmul(*L, G.make_config(), codes, scales).shape == (0, 64)
    assert G.gptq_w4a8_gated(L, L, G.make_config(), codes, scales, dtype=I8)[1].shape == (0, 1)


@pytest.mark.parametrize("n", [1, 8, 24, 64, 100, 256, 700])
def test_same_layer_twice_and_repeats(G, n):
    """gate and up may be the same layer; calls repeat bit by bit, on another
    stream and from a replayed graph with other inputs too."""
    rows, cols, group = 520, 1024, 128
    L = small(layer(rows, cols, group, 3))
    cfg = G.make_config(group_size=group)
    codes, scales = acts(n, cols, 128)
    check_gated(G, L, L, group, codes, scales, BF)

    def both(codes, stream=None):
        return (G.gptq_w4a8_matmul(*L, cfg, codes, scales, stream=stream),
                *G.gptq_w4a8_gated(L, L, cfg, codes, scales, dtype=I8, stream=stream))

    want = both(codes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(codes, side)
    again = both(codes)  # at the same time on the current stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, again))
    held = codes.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(held)
    for seed in (5, 6):
        held.copy_(acts(n, cols, 128, seed)[0])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, both(held)))


# enough tiles for the persistent kernel (more than one a CTA), odd in every way
@pytest.mark.parametrize("shape", [(130, 160, 0, 40000), (300, 416, 32, 13001), (129, 640, 128, 39000),
                                   (257, 384, 64, 19777), (200, 1024, 256, 25001), (64, 96, 96, 50000)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("xg", [0, 128])
def test_many_tokens(G, shape, xg):
    rows, cols, group, n = shape
    kw = {"block": 32} if group and group % 64 else {}
    gate, up = small(layer(rows, cols, group, 1)), small(layer(rows, cols, group, 2))
    codes, scales = acts(n, cols, xg)
    cfg = G.make_config(bits=4, group_size=group, **kw)
    y = G.gptq_w4a8_matmul(*gate, cfg, codes, scales, dtype=F32)
    h = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=BF)
    h8, hs = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=I8)
    assert G.gptq_device_status() == 0
    # every token of some stretches: the first and last tiles and one between
    tok = np.unique(np.concatenate([np.arange(260), np.arange(n // 2, n // 2 + 130),
                                    np.arange(n - 300, n)]))
    c, s = codes[tok].cpu().numpy(), scales[tok].cpu().numpy()
    R.check_float(y[tok].cpu().numpy(), *R.product(*np_layer(gate), group, c, s))
    ref, bound = R.gated(np_layer(gate), np_layer(up), group, c, s)
    R.check_float(h[tok].double().cpu().numpy(), ref, bound, bf16=True)
    R.check_codes(h8[tok].cpu().numpy(), hs[tok].cpu().numpy(), ref, bound, 128)
    # and all tokens against the same tokens in small batches, within twice the bound
    whole = y.double()
    for a in range(0, n, 9973):
        part = G.gptq_w4a8_matmul(*gate, cfg, codes[a:a + 100], scales[a:a + 100].contiguous())
        top = float(part.abs().max())
        assert float((whole[a:a + 100] - part).abs().max()) <= 1e-5 * top


# layers of the 65B and 7B shapes on sampled rows
@pytest.mark.parametrize("case", [(8192, 22016, 128, 1), (8192, 22016, 128, 16),
                                  (22016, 8192, 128, 4), (4096, 11008, 0, 33),
                                  (11008, 4096, 64, 130), (22016, 8192, 128, 600)],
                         ids=lambda c: "x".join(map(str, c)))
def test_full_size_sampled(G, case):
    rows, cols, group, n = case
    gate, up = layer(rows, cols, group, 1), layer(rows, cols, group, 2)
    codes, scales = acts(n, cols, 128)
    cfg = G.make_config(group_size=group)
    scales = scales / (30.0 * cols ** 0.5)
    y = G.gptq_w4a8_matmul(*gate, cfg, codes, scales)
    h = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=F32)
    h8, hs = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=I8)
    assert G.gptq_device_status() == 0
    rng = np.random.default_rng(n)
    pick = np.unique(np.concatenate([np.arange(128), np.arange(rows - rows % 128 - 128, rows),
                                     rng.choice(rows, 32)]))
    tok = np.unique(np.concatenate([[0, n - 1], rng.choice(n, min(n, 12))]))
    g, u = (tuple(t[pick].cpu().numpy() for t in L) for L in (gate, up))
    c, s = codes[tok].cpu().numpy(), scales[tok].double().cpu().numpy()
    R.check_float(y[tok][:, pick].cpu().numpy(), *R.product(*g, group, c, s))
    ref, bound = R.gated(g, u, group, c, s)
    R.check_float(h[tok][:, pick].cpu().numpy(), ref, bound)
    first = pick < 128
    R.check_codes(h8[tok][:, :128].cpu().numpy(), hs[tok][:, :1].cpu().numpy(), ref[:, first],
                  bound[:, first], 128)


def test_refusals(G):
    L = layer(64, 256, 64)
    cfg = G.make_config(group_size=64)
    codes, scales = acts(4, 256, 128)
    for bad in (dict(codes=codes.float()), dict(codes=codes.T.contiguous().T),
                dict(scales=scales[:3]), dict(scales=scales.double()),
                dict(scales=torch.ones(4, 3, device="cuda")),
                dict(L=(L[0], L[1], L[2][:63])), dict(L=(L[0], L[1].T.contiguous().T, L[2])),
                dict(L=(L[0][:, :16], L[1], L[2])), dict(L=(L[0].cpu(), L[1], L[2])),
                dict(cfg=G.make_config(group_size=128)), dict(Y=torch.empty(4, 63, device="cuda")),
                dict(Y=torch.empty(4, 64, device="cuda", dtype=torch.float16)),
                dict(Y=torch.empty(4, 64, device="cuda", dtype=I8))):
        with pytest.raises(ValueError):
            G.gptq_w4a8_matmul(*bad.get("L", L), bad.get("cfg", cfg), bad.get("codes", codes),
                               bad.get("scales", scales), Y=bad.get("Y"))
    for out in (torch.empty(4, 64, device="cuda", dtype=I8),
                (torch.empty(4, 64, device="cuda"), torch.empty(4, 1, device="cuda")),
                (torch.empty(4, 64, device="cuda", dtype=I8), torch.empty(4, 2, device="cuda"))):
        with pytest.raises(ValueError):
            G.gptq_w4a8_gated(L, L, cfg, codes, scales, out=out)
    with pytest.raises(ValueError):
        G.gptq_w4a8_gated(L, layer(32, 256, 64), cfg, codes, scales)
    wide = torch.zeros(4, 264, dtype=I8, device="cuda")
    for view in (wide[:, :256], wide[:, 8:].contiguous().view(-1)[8:8 + 512].view(2, 256)):
        with pytest.raises(G.GptqError):  # a stride or a start that is no multiple of 16
            G.gptq_w4a8_matmul(*L, cfg, view, scales[:view.shape[0]].contiguous())
    with pytest.raises(G.GptqError):
        G.gptq_w4a8_matmul(L[0], L[1], L[2], G.make_config(bits=3, group_size=64), codes, scales)


def shifted(t):
    """The same values at an address one element further."""
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    room[1:] = t.flatten()
    return room[1:].view(t.shape)


@pytest.mark.parametrize("shape", [(77, 1536, 128), (161, 1024, 64), (45, 1920, 32), (130, 640, 128)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("n", [1, 8, 9, 16, 17, 64, 65, 130])
@pytest.mark.parametrize("xg", [0, 128])
def test_alignment_of_scales(G, shape, n, xg):
    """Scales and zero points at any element's address: another way into the
    kernels, the same order of sums, the same bits."""
    rows, cols, group = shape
    gate, up = small(layer(rows, cols, group, n)), small(layer(rows, cols, group, n + 1))
    codes, scales = acts(n, cols, xg)
    y = check_matmul(G, gate, group, codes, scales, F32)
    h, hs = check_gated(G, gate, up, group, codes, scales, I8)
    cfg = G.make_config(group_size=group)
    moved = [(L[0], shifted(L[1]), shifted(L[2])) for L in (gate, up)]
    for layers, s in ((moved, scales), ((gate, up), shifted(scales)), (moved, shifted(scales)),
                      ((gate, moved[1]), scales)):
        assert torch.equal(G.gptq_w4a8_matmul(*layers[0], cfg, codes, s), y)
        h2, hs2 = G.gptq_w4a8_gated(*layers, cfg, codes, s, dtype=I8)
        assert torch.equal(h2, h) and torch.equal(hs2, hs)
    assert G.gptq_device_status() == 0
