"""The gated feed-forward block of a decoder layer on packed 4-bit weights,
with the activations between its steps in 8 bits, as measurable cases.

    norm    residual addition, root-mean-square norm, 8-bit codes and scales
    gated   silu(X Wg^T) * (X Wu^T) from two packed 4-bit layers
    matmul  X W^T from one packed 4-bit layer

Codes are int8, x = s * q with one fp32 scale a token, or a token and 128
columns.  ``run`` computes a case in plain torch operations, or, where ``own``
is true, through the library's entry points.
"""
from __future__ import annotations

import torch

own = False

DEV = "cuda"
GROUP = 128  # columns of a token that share a scale, where a token has several
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    def norm(name, n, d, x, res, group):
        return {"name": name, "op": "norm", "n": n, "d": d, "x": x, "res": res, "group": group}

    def matmul(name, n, rows, cols, wgroup, group, out):
        return {"name": name, "op": "matmul", "n": n, "rows": rows, "cols": cols,
                "wgroup": wgroup, "group": group, "out": out}

    def gated(name, n, rows, cols, wgroup, group, out):
        return dict(matmul(name, n, rows, cols, wgroup, group, out), op="gated")

    return [
        # one token of a generation: a launch and its latency
        norm("norm_1x8192", 1, 8192, "bf16", "bf16", GROUP),
        # a small batch of a generation: the product comes as fp32, one scale a token
        norm("norm_8x4096_token", 8, 4096, "fp32", "bf16", 0),
        # a prompt of odd length at the head of a stack, no residual yet
        norm("norm_777x4096_plain", 777, 4096, "fp32", "none", 0),
        # a long prompt: bound by memory
        norm("norm_16384x8192", 16384, 8192, "bf16", "bf16", GROUP),
        # one token through the down projection: every weight read for one row
        matmul("matmul_1_8192x22016", 1, 8192, 22016, 128, GROUP, "fp32"),
        # a batch of eight through a small layer with one scale a channel
        matmul("matmul_8_4096x4096_channel", 8, 4096, 4096, 0, 0, "bf16"),
        # a ragged batch between generation and prompt, fine weight groups
        matmul("matmul_61_11008x4096_g64", 61, 11008, 4096, 64, GROUP, "fp32"),
        # a long prompt through the down projection: bound by arithmetic
        matmul("matmul_4096_8192x22016", 4096, 8192, 22016, 128, GROUP, "bf16"),
        # one token through gate and up projection, 8-bit for the down projection
        gated("gated_1_22016x8192", 1, 22016, 8192, 128, GROUP, "8bit"),
        # a batch of sixteen, one scale a token, bf16 out
        gated("gated_16_11008x4096_token", 16, 11008, 4096, 128, 0, "bf16"),
        # a short prompt of odd length, the finest weight groups
        gated("gated_333_11008x4096_g32", 333, 11008, 4096, 32, GROUP, "8bit"),
        # a long prompt through gate and up projection
        gated("gated_2048_22016x8192", 2048, 22016, 8192, 128, GROUP, "8bit"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def draw(rng):
    op = rng.choice(["norm", "matmul", "gated"])
    group = rng.choice([0, GROUP])
    if op == "norm":
        return {"op": op, "n": _spread(rng, 1, 16384), "d": 32 * _spread(rng, 8, 256),
                "x": rng.choice(["bf16", "fp32"]), "res": rng.choice(["bf16", "fp32", "none"]),
                "group": group}
    wgroup = rng.choice([0, 32, 64, 128, 256])
    step = max(32, wgroup)
    cols = step * max(1, _spread(rng, 512, 22016 if op == "matmul" else 8192) // step)
    rows = _spread(rng, 500, 8192 if op == "matmul" else 22016)
    return {"op": op, "n": _spread(rng, 1, 4096 if op == "matmul" else 2048), "rows": rows,
            "cols": cols, "wgroup": wgroup, "group": group,
            "out": rng.choice(["bf16", "fp32", "8bit"] if op == "gated" else ["bf16", "fp32"])}


def work(case):
    def groups(cols, group):
        return -(-cols // group) if group else 1

    size = {"bf16": 2, "fp32": 4, "none": 0}
    n = case["n"]
    if case["op"] == "norm":
        d = case["d"]
        b = n * d * (size[case["x"]] + 2 * size[case["res"]] + 1) + 4 * d
        return {"bytes": b + 4 * n * groups(d, case["group"]), "flops": 8 * n * d}
    rows, cols = case["rows"], case["cols"]
    layers = 2 if case["op"] == "gated" else 1
    b = layers * rows * (cols // 2 + 5 * groups(cols, case["wgroup"]))
    b += n * cols + 4 * n * groups(cols, case["group"])
    if case["out"] == "8bit":
        b += n * rows + 4 * n * groups(rows, GROUP)
    else:
        b += n * rows * size[case["out"]]
    return {"bytes": b, "flops": 2 * layers * n * rows * cols}


# ------------------------------------------------------------------ inputs
def _activations(gen, n, d):
    """Normal values with one channel of a hundred twenty times as large."""
    x = torch.randn(n, d, generator=gen, device=DEV)
    big = torch.rand(d, generator=gen, device=DEV) < 0.01
    return torch.where(big, 20.0 * x, x)


def _layer(gen, rows, cols, group):
    """A normal weight matrix as packed min-max codes: (words, scales, zeros)."""
    w = torch.randn(rows, cols, generator=gen, device=DEV) * cols ** -0.5
    w = w.view(rows, -1, group if group else cols)
    lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
    s = (hi - lo) / 15.0
    z = torch.round(-lo / s)
    q = (torch.round(w / s[:, :, None]) + z[:, :, None]).clamp_(0, 15)
    q = q.view(rows, cols // 8, 8).to(torch.int32)
    words = q[:, :, 0].clone()
    for k in range(1, 8):
        words |= q[:, :, k] << (4 * k)
    return words, s.contiguous(), z.to(torch.uint8).contiguous()


def _codes(x, group):
    """8-bit codes and scales of x, for the inputs of the products."""
    n, d = x.shape
    g = group if group else d
    pad = torch.nn.functional.pad(x, (0, -d % g)).view(n, -1, g)
    top = pad.abs().amax(2)
    q = torch.round(pad * torch.where(top > 0, 127.0 / top, 0.0)[:, :, None])
    return q.view(n, -1)[:, :d].to(torch.int8).contiguous(), (top / 127.0).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = case["n"]
    if case["op"] == "norm":
        d = case["d"]
        return {"case": case, "eps": 1e-5,
                "x": _activations(gen, n, d).to(DTYPES[case["x"]]),
                "res": None if case["res"] == "none" else
                (3.0 * torch.randn(n, d, generator=gen, device=DEV)).to(DTYPES[case["res"]]),
                "weight": 1.0 + 0.2 * torch.randn(d, generator=gen, device=DEV)}
    rows, cols, wgroup = case["rows"], case["cols"], case["wgroup"]
    layers = [_layer(gen, rows, cols, wgroup) for _ in range(2 if case["op"] == "gated" else 1)]
    codes, scales = _codes(_activations(gen, n, cols), case["group"])
    return {"case": case, "layers": layers, "codes": codes, "scales": scales}


# -------------------------------------------------------------------- plain
def _values(codes, scales, group):
    """What 8-bit codes stand for, as bf16."""
    n, d = codes.shape
    out = torch.empty(n, d, dtype=torch.bfloat16, device=codes.device)
    if group and d % group:
        torch.mul(codes, scales.repeat_interleave(group, 1)[:, :d], out=out)
    else:
        g = group if group else d
        torch.mul(codes.view(n, -1, g), scales[:, :, None], out=out.view(n, -1, g))
    return out


def _plain_codes(y, group):
    """The values of y's 8-bit codes and their scales, y in fp32."""
    n, d = y.shape
    g = group if group else d
    rows = torch.nn.functional.pad(y, (0, -d % g)).view(n, -1, g)
    top = rows.abs().amax(2)
    inverse = torch.where(top > 0, 127.0 / top, torch.zeros_like(top))
    q = torch.round(rows * inverse[:, :, None])
    s = top / 127.0
    return (q * s[:, :, None]).view(n, -1)[:, :d].to(torch.bfloat16), s


def _plain_layer(words, scales, zeros, cols):
    """W = s * (q - z) in fp32."""
    rows = words.shape[0]
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)
    q = (words[:, :, None] >> shifts) & 15
    w = q.view(rows, scales.shape[1], -1).float() - zeros[:, :, None].float()
    return (w * scales[:, :, None]).view(rows, cols)


def _plain_activations(codes, scales, group):
    n, d = codes.shape
    if not group:
        return codes.float() * scales
    return codes.float() * scales.repeat_interleave(group, 1)[:, :d]


def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "norm":
        r = state["x"].float()
        out = {}
        if state["res"] is not None:
            out["residual"] = (r + state["res"].float()).to(state["res"].dtype)
            r = out["residual"].float()
        y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + state["eps"]) * state["weight"]
        out["values"], out["scales"] = _plain_codes(y, case["group"])
        return out
    x = _plain_activations(state["codes"], state["scales"], case["group"])
    w = [_plain_layer(*layer, case["cols"]) for layer in state["layers"]]
    if case["op"] == "matmul":
        return {"y": (x @ w[0].T).to(DTYPES[case["out"]])}
    g = x @ w[0].T
    h = g / (1.0 + torch.exp(-g)) * (x @ w[1].T)
    if case["out"] != "8bit":
        return {"h": h.to(DTYPES[case["out"]])}
    values, scales = _plain_codes(h, GROUP)
    return {"values": values, "scales": scales}


def _run_own(state, case):
    from post_weight_quantization_26_b200 import gptq as G
    if case["op"] == "norm":
        got = G.gptq_rmsnorm_quant8(state["x"], state["weight"], state["eps"],
                                    residual=state["res"], group=case["group"])
        out = {"values": _values(got[0], got[1], case["group"]), "scales": got[1]}
        if state["res"] is not None:
            out["residual"] = got[2]
        return out
    if "config" not in state:  # a program makes it once, with the layers
        state["config"] = G.make_config(bits=4, group_size=case["wgroup"])
    if case["op"] == "matmul":
        return {"y": G.gptq_w4a8_matmul(*state["layers"][0], state["config"], state["codes"],
                                        state["scales"], dtype=DTYPES[case["out"]])}
    if case["out"] != "8bit":
        return {"h": G.gptq_w4a8_gated(*state["layers"], state["config"], state["codes"],
                                       state["scales"], dtype=DTYPES[case["out"]])}
    codes, scales = G.gptq_w4a8_gated(*state["layers"], state["config"], state["codes"],
                                      state["scales"], dtype=torch.int8)
    return {"values": _values(codes, scales, GROUP), "scales": scales}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    state = prepare(case, seed)

    def spread(s, group, d):  # one value a group -> one a column
        index = torch.arange(d, device=DEV) // (group if group else d)
        return s.double()[:, index]

    def eight(y, group):
        d = y.shape[1]
        index = torch.arange(d, device=DEV) // (group if group else d)
        top = torch.zeros(y.shape[0], int(index[-1]) + 1, dtype=torch.float64, device=DEV)
        top.index_reduce_(1, index, y.abs(), "amax")
        s = top / 127.0
        each = s[:, index]
        return torch.where(each > 0, torch.round(y / each) * each, 0.0), s

    if case["op"] == "norm":
        r, out = state["x"].double(), {}
        if state["res"] is not None:
            out["residual"] = r + state["res"].double()
            # the norm is of the sum as it is stored
            r = (state["x"].float() + state["res"].float()).to(state["res"].dtype).double()
        mean = torch.einsum("td,td->t", r, r) / r.shape[1]
        y = r / torch.sqrt(mean + state["eps"])[:, None] * state["weight"].double()
        out["values"], out["scales"] = eight(y, case["group"])
        return out
    cols = case["cols"]
    x = state["codes"].double() * spread(state["scales"], case["group"], cols)

    def product(layer):
        words, s, z = layer
        w = torch.empty(words.shape[0], cols, dtype=torch.float64, device=DEV)
        for k in range(8):
            w[:, k::8] = (words.long() >> (4 * k)) % 16
        w -= spread(z, case["wgroup"], cols)
        w *= spread(s, case["wgroup"], cols)
        return x @ w.T

    if case["op"] == "matmul":
        return {"y": product(state["layers"][0])}
    g = product(state["layers"][0])
    h = g * torch.sigmoid(g) * product(state["layers"][1])
    if case["out"] != "8bit":
        return {"h": h}
    values, scales = eight(h, GROUP)
    return {"values": values, "scales": scales}
