"""The norm with 8-bit output against its 64-bit form; the bounds are derived
in act8_reference.py."""
import numpy as np
import pytest
import torch

import act8_reference as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_26_b200 import build, gptq
    build.build()
    gptq.load_library()
    return gptq


def inputs(n, d, x_dtype, r_dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * d + n)
    x = torch.randn(n, d, generator=gen)
    x[:, torch.rand(d, generator=gen) < 0.02] *= 20.0
    res = None if r_dtype is None else (3.0 * torch.randn(n, d, generator=gen)).to(r_dtype).cuda()
    weight = (1.0 + 0.2 * torch.randn(d, generator=gen)).cuda()
    return x.to(x_dtype).cuda(), res, weight


def check(got, x, res, weight, eps, group):
    codes, scales = got[0].cpu().numpy(), got[1].cpu().numpy()
    stored = None
    if res is not None:
        want = (x.float() + res.float()).to(res.dtype)
        assert torch.equal(got[2], want)
        stored = want.double().cpu().numpy()
    y, dy = R.norm(x.double().cpu().numpy(), stored,
                   None if weight is None else weight.double().cpu().numpy(), eps)
    R.check_codes(codes, scales, y, dy, group)


# widths: one column, short, odd, off the 8- and 16-byte vectors, ragged last
# group, each capacity of the register routes and beyond them
@pytest.mark.parametrize("d", [1, 2, 31, 127, 128, 129, 136, 200, 1000, 1024, 2047, 2048, 2056,
                               4096, 8192, 8200, 11008, 16384, 16392, 22016, 32768, 65536])
@pytest.mark.parametrize("group", [0, 128])
def test_widths(G, d, group):
    x, res, w = inputs(3, d, BF, BF)
    check(G.gptq_rmsnorm_quant8(x, w, 1e-5, residual=res, group=group), x, res, w, 1e-5, group)


@pytest.mark.parametrize("x_dtype", [BF, F32])
@pytest.mark.parametrize("r_dtype", [BF, F32, None])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("d", [192, 1001, 4096])
def test_types(G, x_dtype, r_dtype, group, d):
    x, res, w = inputs(5, d, x_dtype, r_dtype, seed=1)
    check(G.gptq_rmsnorm_quant8(x, w, 1e-6, residual=res, group=group), x, res, w, 1e-6, group)
    check(G.gptq_rmsnorm_quant8(x, None, 0.0, residual=res, group=group), x, res, None, 0.0, group)


@pytest.mark.parametrize("n", [1, 2, 147, 1000, 5000])
@pytest.mark.parametrize("group", [0, 128])
def test_token_counts(G, n, group):
    x, res, w = inputs(n, 2048, BF, F32, seed=2)
    check(G.gptq_rmsnorm_quant8(x, w, 1e-6, residual=res, group=group), x, res, w, 1e-6, group)


def test_no_tokens(G):
    codes, scales, r = G.gptq_rmsnorm_quant8(torch.empty(0, 64, device="cuda"), None,
                                             residual=torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0, 1) and r.shape == (0, 64)


@pytest.mark.parametrize("pad,shift", [(16, 0), (8, 0), (3, 0), (16, 1), (16, 8)])
@pytest.mark.parametrize("group", [0, 128])
def test_strides_and_what_lies_between(G, pad, shift, group):
    """Rows inside wider arrays, aligned and not; the columns beside them and
    the rows behind the last stay as they were."""
    n, d = 6, 1152
    x, res, w = inputs(n, d, BF, BF, seed=3)

    def inside(t, fill):
        big = torch.full((n + 1, d + pad + shift), fill, dtype=t.dtype, device="cuda")
        view = big[:n, shift:shift + d]
        view.copy_(t)
        return big, view

    _, xv = inside(x, 9.0)
    _, rv = inside(res, 9.0)
    ob, ov = inside(torch.zeros_like(res), 5.0)
    cb, cv = inside(torch.zeros(n, d, dtype=torch.int8, device="cuda"), 77)
    scales = torch.empty(n, 9 if group else 1, device="cuda")
    got = G.gptq_rmsnorm_quant8(xv, w, 1e-5, residual=rv, group=group, residual_out=ov,
                                out=(cv, scales))
    check(got, x, res, w, 1e-5, group)
    for big, fill in ((ob, 5.0), (cb, 77)):
        assert (big[n] == fill).all() and (big[:, :shift] == fill).all()
        assert (big[:, shift + d:] == fill).all()


@pytest.mark.parametrize("d", [1024, 1001, 40000])
@pytest.mark.parametrize("onto", ["residual", "x"])
def test_in_place(G, d, onto):
    x, res, w = inputs(4, d, BF, BF, seed=4)
    want = G.gptq_rmsnorm_quant8(x, w, residual=res)
    x2, r2 = x.clone(), res.clone()
    got = G.gptq_rmsnorm_quant8(x2, w, residual=r2, residual_out=r2 if onto == "residual" else x2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [1024, 1001, 40000])
def test_zero_rows_and_tiny_values(G, d):
    x, _, _ = inputs(4, d, F32, None, seed=5)
    x[0] = 0.0
    x[1] *= 1e-36   # below the range of 127 / max
    x[2, :128] = 0.0
    x[3] *= 1e30    # the squares overflow: y = 0
    for group in (0, 128):
        codes, scales = G.gptq_rmsnorm_quant8(x[:3], None, 1.0, group=group)
        assert (codes[0] == 0).all() and (scales[0] == 0).all()
        check((codes, scales), x[:3], None, None, 1.0, group)
        codes, scales = G.gptq_rmsnorm_quant8(x[3:], None, 1.0, group=group)
        assert (codes == 0).all() and (scales == 0).all()
    codes, scales = G.gptq_rmsnorm_quant8(x[:3], None, 1.0, group=128)
    assert scales[2, 0] == 0 and (codes[2, :128] == 0).all()


@pytest.mark.parametrize("d", [1024, 1001, 40000])
def test_nan_and_infinity(G, d):
    """A NaN reaches every scale of its token; an infinite value makes its own
    group NaN and the others zero; other tokens are untouched."""
    x, _, w = inputs(3, d, F32, None, seed=6)
    clean = G.gptq_rmsnorm_quant8(x, w)
    x[0, 300] = float("nan")
    x[1, 300] = -float("inf")
    codes, scales = G.gptq_rmsnorm_quant8(x, w)
    assert torch.isnan(scales[0]).all() and (codes[:2] == 0).all()
    assert torch.isnan(scales[1, 2]) and (scales[1, :2] == 0).all()
    assert torch.equal(codes[2], clean[0][2]) and torch.equal(scales[2], clean[1][2])
    _, scales = G.gptq_rmsnorm_quant8(x, w, group=0)
    assert torch.isnan(scales[:2]).all()


def test_awq_scale_in_the_weight(G):
    """Dividing the weight by s divides the norm's output by s."""
    x, _, w = inputs(4, 512, BF, None, seed=8)
    s = torch.rand(512, device="cuda") + 0.5
    codes, scales = G.gptq_rmsnorm_quant8(x, w / s, 1e-6)
    y, dy = R.norm(x.double().cpu().numpy(), None, w.double().cpu().numpy(), 1e-6)
    sd = s.double().cpu().numpy()
    # the quotient w / s is rounded once more to fp32
    R.check_codes(codes.cpu().numpy(), scales.cpu().numpy(), y / sd, dy / sd + R.U * np.abs(y / sd),
                  128)


def test_repeats_and_streams(G):
    """The same bits on every call, on another stream and from a replayed graph."""
    x, res, w = inputs(70, 4096, BF, BF, seed=9)
    want = G.gptq_rmsnorm_quant8(x, w, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = G.gptq_rmsnorm_quant8(x, w, residual=res, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    x2 = x.clone()
    with torch.cuda.graph(graph):
        got = G.gptq_rmsnorm_quant8(x2, w, residual=res)
    for k in range(3):
        x2.copy_(x * (k + 1))
        graph.replay()
        want = G.gptq_rmsnorm_quant8(x2, w, residual=res)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(G):
    x, res, w = inputs(4, 64, BF, BF)
    for bad in (dict(residual=res[:3]), dict(residual=res.half()), dict(residual_out=res),
                dict(residual=res, residual_out=res.float()), dict(weight=w.bfloat16()),
                dict(weight=w[:32]), dict(out=G.alloc_codes(4, 60)),
                dict(out=(G.alloc_codes(4, 64)[0], torch.empty(4, 2, device="cuda"))),
                dict(residual=res.cpu()), dict(residual=res.T.contiguous().T)):
        with pytest.raises(ValueError):
            G.gptq_rmsnorm_quant8(x, bad.pop("weight", w), **bad)
    with pytest.raises(ValueError):
        G.gptq_rmsnorm_quant8(x.half(), w)
    with pytest.raises(G.GptqError):
        G.gptq_rmsnorm_quant8(x, w, eps=-1.0)
    with pytest.raises(G.GptqError):
        G.gptq_rmsnorm_quant8(x, w, group=64)
