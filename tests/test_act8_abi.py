"""Refusals of the feed-forward block's calls: nothing is launched for bad
arguments, in the C entry points and in the binding, without a GPU."""
import ctypes

import pytest
import torch

from post_weight_quantization_26_b200 import build as B

FAKE = ctypes.c_void_p(0x7F0000000000)  # never dereferenced: validation fails first


def off(k):
    return ctypes.c_void_p(0x7F0000000000 + k)


@pytest.fixture(scope="module")
def G():
    B.build()
    from post_weight_quantization_26_b200 import gptq
    gptq.load_library()
    return gptq


NORM = dict(X=FAKE, x_type=1, ldx=64, res=FAKE, r_type=1, ldr=64, w=FAKE, eps=1e-6, n=4, d=64,
            group=128, out=FAKE, ldo=64, codes=FAKE, ldq=64, scales=FAKE, stream=None)


@pytest.mark.parametrize("bad", [
    dict(X=None), dict(codes=None), dict(scales=None), dict(out=None),
    dict(x_type=2), dict(x_type=-1), dict(r_type=2), dict(ldx=63), dict(ldr=63), dict(ldo=63),
    dict(ldq=63), dict(n=-1), dict(n=1 << 31), dict(d=0), dict(d=65537), dict(group=64),
    dict(group=-128), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(eps=1e300), dict(X=off(1)), dict(X=off(2), x_type=0), dict(res=off(1)),
    dict(out=off(1)), dict(w=off(2)), dict(scales=off(2)),
], ids=str)
def test_norm_refuses(G, bad):
    assert G.load_library().gptq_rmsnorm_quant8(*{**NORM, **bad}.values()) == 1


def test_norm_of_no_tokens(G):
    f = G.load_library().gptq_rmsnorm_quant8
    assert f(*{**NORM, "n": 0, "X": None, "codes": None, "scales": None}.values()) == 0


def _matmul(G, cfg=None, **bad):
    a = dict(qw=FAKE, s=FAKE, z=FAKE, d_row=64, d_col=256, cfg=cfg, codes=FAKE, ldq=256, xs=FAKE,
             xg=128, n=4, Y=FAKE, y_type=0, ldy=64, stream=None)
    a.update(bad)
    return G.load_library().gptq_w4a8_matmul(*a.values())


def _gated(G, cfg=None, **bad):
    a = dict(qg=FAKE, sg=FAKE, zg=FAKE, qw=FAKE, s=FAKE, z=FAKE, d_row=64, d_col=256, cfg=cfg,
             codes=FAKE, ldq=256, xs=FAKE, xg=128, n=4, Y=FAKE, y_type=0, ldy=64, hs=FAKE, ws=FAKE,
             ws_bytes=1 << 20, stream=None)
    a.update(bad)
    return G.load_library().gptq_w4a8_gated(*a.values())


SHARED = [
    dict(qw=None), dict(s=None), dict(z=None), dict(qw=off(4)), dict(s=off(2)), dict(d_row=0),
    dict(d_row=(1 << 24) + 1), dict(d_col=240), dict(d_col=0), dict(d_col=65568, ldq=65568),
    dict(codes=None), dict(codes=off(8)), dict(ldq=240), dict(ldq=264), dict(xs=None),
    dict(xs=off(2)), dict(xg=64), dict(n=-1), dict(n=(1 << 24) + 1), dict(Y=None), dict(Y=off(2)),
    dict(y_type=1, Y=off(1)), dict(y_type=3), dict(y_type=-1), dict(ldy=63),
]


@pytest.mark.parametrize("bad", SHARED + [dict(y_type=2)], ids=str)
def test_matmul_refuses(G, bad):
    assert _matmul(G, ctypes.byref(G.make_config(bits=4, group_size=128)), **bad) == 1


@pytest.mark.parametrize("bad", SHARED + [
    dict(qg=None), dict(sg=None), dict(zg=None), dict(qg=off(4)), dict(sg=off(2)),
    dict(y_type=2, hs=None), dict(y_type=2, hs=off(2))], ids=str)
def test_gated_refuses(G, bad):
    assert _gated(G, ctypes.byref(G.make_config(bits=4, group_size=128)), **bad) == 1


def test_products_refuse_configurations(G):
    for cfg in (G.make_config(bits=3), G.make_config(bits=8), G.make_config(group_size=100),
                G.make_config(group_size=96, block=32), G.make_config(group_size=512)):
        assert _matmul(G, ctypes.byref(cfg)) == 1
        assert _gated(G, ctypes.byref(cfg)) == 1
    assert _matmul(G, None) == 1 and _gated(G, None) == 1


def test_gated_workspace(G):
    """Only an 8-bit output of up to 16 tokens needs one: fp32 rows of whole
    blocks of 128."""
    size = G.load_library().gptq_w4a8_workspace_size
    assert size(1, 64, 2) == 512 and size(16, 129, 2) == 16 * 256 * 4
    for none in ((17, 64, 2), (16, 64, 1), (16, 64, 0), (0, 64, 2), (-1, 64, 2), (4, 0, 2),
                 (4, (1 << 24) + 1, 2)):
        assert size(*none) == 0
    cfg = ctypes.byref(G.make_config(bits=4, group_size=128))
    for bad in (dict(ws=None), dict(ws=off(128)), dict(ws_bytes=2047)):
        assert _gated(G, cfg, y_type=2, **bad) == 4


def test_products_of_no_tokens(G):
    cfg = ctypes.byref(G.make_config(bits=4))
    assert _matmul(G, cfg, n=0, codes=None, xs=None, Y=None) == 0
    assert _gated(G, cfg, n=0, codes=None, xs=None, Y=None) == 0


def test_binding_refuses_host_tensors(G):
    x = torch.zeros(2, 64)
    codes, scales = G.alloc_codes(2, 64, device="cpu")
    layer = G.alloc_outputs(16, 64, G.make_config(), device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        G.gptq_rmsnorm_quant8(x, None)
    with pytest.raises(ValueError, match="CUDA"):
        G.gptq_w4a8_matmul(*layer, G.make_config(), codes, scales)
    with pytest.raises(ValueError, match="CUDA"):
        G.gptq_w4a8_gated(layer, layer, G.make_config(), codes, scales)


def test_alloc_codes_pitch(G):
    codes, scales = G.alloc_codes(3, 200, device="cpu")
    assert codes.shape == (3, 200) and codes.stride() == (208, 1) and scales.shape == (3, 2)
    assert G.alloc_codes(3, 200, 0, device="cpu")[1].shape == (3, 1)


def test_binding_shape_checks(G):
    """The checks that stand behind the device check."""
    t = torch.zeros(4, 64)
    f32 = (torch.float32,)
    assert G._rows("t", t, f32, 4, 64, -1) == 64
    assert G._rows("t", t[:, :32], f32, 4, 32, -1) == 64
    assert G._rows("t", t[:1, :32], f32, 1, 32, -1) == 64
    for bad in (t.T, t.bfloat16(), t[:, ::2], t[:1].expand(4, 64), t[:2]):
        with pytest.raises(ValueError):
            G._rows("t", bad, f32, 4, 64, -1)
    with pytest.raises(ValueError):
        G._rows("t", t, f32, 4, 64, 0)  # another device
    with pytest.raises(ValueError):
        G._dense("t", t[:, :32], f32, (4, 32), -1)


@pytest.mark.parametrize("bad", [
    dict(X=off(256), out=off(256), x_type=0), dict(X=off(256), out=off(256), ldx=72),
    dict(X=off(256), out=off(256), r_type=0), dict(res=off(256), out=off(256), ldo=72),
], ids=str)
def test_norm_refuses_half_in_place(G, bad):
    """residual_out in X's or the residual's memory needs its stride and type."""
    good = dict(X=FAKE, res=off(1 << 20), out=off(1 << 21))
    assert G.load_library().gptq_rmsnorm_quant8(*{**NORM, **good, **bad}.values()) == 1
