"""The feed-forward block as a decoder layer runs it, on layers that the
quantizer packed: norm, gate and up, down, and the next norm's residual."""
import numpy as np
import pytest
import torch

import act8_reference as R
from post_weight_quantization_26_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_26_b200 import build, gptq
    build.build()
    gptq.load_library()
    return gptq


@pytest.fixture(scope="module")
def block(G):
    """Three layers of a block with width 256 and 640 inner columns, quantized
    from their calibration inputs."""
    cfg = G.make_config(bits=4, group_size=128)
    out = {"cfg": cfg, "dense": {}}
    for k, (name, rows, cols) in enumerate((("gate", 640, 256), ("up", 640, 256), ("down", 256, 640))):
        spec = synth.tiny_spec(rows, cols, 2048, seed=20 + k).with_(group=128)
        w = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(k)) * cols ** -0.5).cuda()
        h = torch.zeros((cols, cols), device="cuda")
        G.gptq_hessian_accumulate(h, synth.gen_tokens(spec).cuda())
        ws = G.alloc_workspace(rows, cols, cfg)
        f, dead = torch.empty_like(h), torch.empty(cols, dtype=torch.uint8, device="cuda")
        out[name] = G.alloc_outputs(rows, cols, cfg)
        G.gptq_prepare_factor(h, 0.01, f, dead, ws)
        G.gptq_quantize_layer_factor(w, f, dead, cfg, *out[name], ws)
        w_hat = torch.empty_like(w)
        G.gptq_dequant_check(*out[name], w, h, cfg, W_hat=w_hat, ws=ws)
        out["dense"][name] = w_hat.double().cpu().numpy()
    assert G.gptq_device_status() == 0
    return out


def forward(G, b, x, res, w, w2, xg=128):
    codes, scales, r = G.gptq_rmsnorm_quant8(x, w, 1e-5, residual=res, group=xg)
    h, hs = G.gptq_w4a8_gated(b["gate"], b["up"], b["cfg"], codes, scales, dtype=torch.int8)
    y = G.gptq_w4a8_matmul(*b["down"], b["cfg"], h, hs, dtype=torch.bfloat16)
    return (codes, scales, r, h, hs, y, *G.gptq_rmsnorm_quant8(y, w2, 1e-5, residual=r, group=xg))


def inputs(n, seed=0):
    gen = torch.Generator().manual_seed(seed + n)
    x = torch.randn(n, 256, generator=gen).bfloat16().cuda()
    res = torch.randn(n, 256, generator=gen).bfloat16().cuda()
    return x, res, *(1.0 + 0.1 * torch.randn(2, 256, generator=gen)).cuda()


@pytest.mark.parametrize("n", [1, 7, 16, 50, 129, 400])
@pytest.mark.parametrize("xg", [0, 128])
def test_steps_and_whole(G, block, n, xg):
    x, res, w, w2 = inputs(n)
    codes, scales, r, h, hs, y, codes2, scales2, r2 = forward(G, block, x, res, w, w2, xg)
    assert G.gptq_device_status() == 0
    a = {k: v.double().cpu().numpy() for k, v in dict(
        x=x, r=r, w=w, w2=w2, codes=codes, scales=scales, h=h, hs=hs, y=y, r2=r2).items()}
    np_layers = {k: tuple(t.cpu().numpy() for t in block[k]) for k in ("gate", "up", "down")}
    # every step against the 64-bit form of its own inputs
    assert torch.equal(r, x + res) and torch.equal(r2, y + r)
    R.check_codes(a["codes"], a["scales"], *R.norm(a["x"], a["r"], a["w"], 1e-5), xg)
    R.check_codes(a["h"], a["hs"], *R.gated(np_layers["gate"], np_layers["up"], 128, a["codes"],
                                            a["scales"]), 128)
    R.check_float(a["y"], *R.product(*np_layers["down"], 128, a["h"], a["hs"]), bf16=True)
    R.check_codes(codes2.cpu().numpy(), scales2.cpu().numpy(),
                  *R.norm(a["y"], a["r2"], a["w2"], 1e-5), xg)
    # the whole against the block without 8-bit steps: each 8-bit form is off
    # by at most s / 2 a value, carried through with the weights' magnitudes
    d = block["dense"]
    yn, dyn = R.norm(a["x"], a["r"], a["w"], 1e-5)
    dyn = dyn + R.activation_scales(a["scales"], 256) * (0.5 + 127 * 4 * R.U)
    g, u = yn @ d["gate"].T, yn @ d["up"].T
    dg, du = dyn @ np.abs(d["gate"]).T, dyn @ np.abs(d["up"]).T
    silu = g / (1 + np.exp(-g))
    dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du
    dh = dh + R.activation_scales(a["hs"], 640) * (0.5 + 127 * 4 * R.U)
    ref = (silu * u) @ d["down"].T
    dy = dh @ np.abs(d["down"]).T
    slack = 1e-3 * dy + 1e-6  # fp32 sums, far below the 8-bit steps
    assert np.all(np.abs(a["y"] - ref) <= dy + 2.0 ** -8 * np.abs(ref) + slack)


def test_eager_graph_and_streams(G, block):
    """The block captured once and replayed on other inputs, beside the same
    block on another stream, gives the eager call's bits."""
    x, res, w, w2 = inputs(33)
    graph = torch.cuda.CUDAGraph()
    forward(G, block, x, res, w, w2)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = forward(G, block, x, res, w, w2)
    side = torch.cuda.Stream()
    for seed in (1, 2):
        nx, nres, _, _ = inputs(33, seed)
        x.copy_(nx)
        res.copy_(nres)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = forward(G, block, nx, nres, w, w2)
        torch.cuda.synchronize()
        want = forward(G, block, nx, nres, w, w2)
        assert all(torch.equal(p, q) and torch.equal(p, o) for p, q, o in zip(want, held, other))


def test_padded_batch(G, block):
    """Tokens do not touch one another: a batch's rows are those of the batch
    with other tokens behind them, within the bounds of another split."""
    x, res, w, w2 = inputs(40)
    whole = forward(G, block, x, res, w, w2)
    part = forward(G, block, x[:12], res[:12], w, w2)
    assert torch.equal(whole[0][:12], part[0]) and torch.equal(whole[1][:12], part[1])
    d = (whole[5][:12].double() - part[5].double()).abs().cpu().numpy()
    h, hs = (t[:12].double().cpu().numpy() for t in (whole[3], whole[4]))
    # h may differ by one code where a sum's last bits differ
    step = (R.activation_scales(hs, 640) + 1e-6 * np.abs(h * R.activation_scales(hs, 640)))
    tol = step @ np.abs(block["dense"]["down"]).T
    assert np.all(d <= tol * 1.001 + 2.0 ** -7 * np.abs(part[5].double().cpu().numpy()) + 1e-6)
