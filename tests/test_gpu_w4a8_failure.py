"""Waits of the W4A8 kernels that run out, without faulting the GPU.

The fault-injection switch makes the producer of the kernels' rings issue no
loads (the readers' first waits run out, with nothing in flight), or the ring's
readers hand nothing back (the producer's own wait runs out, with a ring of
copies and products behind it).  Every wait has a limit of 20 ms.  The call
returns, the status word says so once, and the next call on the same context
gives the bits of the call before, so tensor memory, barriers and the cluster's
shared memory were left in order.
"""
import pytest
import torch

from post_weight_quantization_26_b200 import synth

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
TIMEOUT = 6
LIMIT_NS = 20_000_000


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_weight_quantization_26_b200 import build, gptq
    build.build()
    gptq.load_library()
    yield gptq
    gptq.gptq_fault_inject(gptq.FAULT_NONE, 0)


def layer(d_row, d_col, group, seed):
    return tuple(t.cuda() for t in synth.gen_packed_layer(d_row, d_col, group, seed))


def acts(n, d, xg):
    gen = torch.Generator().manual_seed(n + d)
    codes = torch.randint(-127, 128, (n, d), generator=gen, dtype=I8).cuda()
    return codes, (0.01 + torch.rand(n, -(-d // 128) if xg else 1, generator=gen)).cuda()


# (tokens, rows, columns, weight group, scales of tokens): the row kernel for up to 8
# and 16 tokens, with scales that come with the stages and without; the tile kernel's
# small shapes, whose columns are split over a cluster; the persistent shape (a tile
# for every SM), where two MMA warps take turns, where runs span chunks, and where a
# chunk has four runs.  All have more stages a CTA than the ring holds.
CASES = [(1, 96, 8192, 128, 128), (5, 96, 8192, 256, 0), (16, 96, 8192, 32, 128),
         (40, 256, 16384, 128, 128), (30, 200, 16384, 0, 0), (100, 256, 16384, 64, 128),
         (60, 256, 16384, 32, 0), (148 * 256, 128, 1024, 128, 128), (148 * 256, 100, 1024, 0, 0),
         (148 * 256 + 9, 128, 1024, 32, 128)]


def stalled_between(G, fault, call):
    before = call()
    assert G.gptq_device_status() == 0
    G.gptq_fault_inject(fault, LIMIT_NS)
    try:
        call()
        status = G.gptq_device_status()
    finally:
        G.gptq_fault_inject(G.FAULT_NONE, 0)
    assert status == TIMEOUT
    assert G.gptq_device_status() == 0
    for _ in range(2):
        after = call()
        assert G.gptq_device_status() == 0
        for a, b in zip(before, after):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fault", ["FAULT_W4A8_LOADS", "FAULT_W4A8_STAGES"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_product_wait_runs_out(G, case, fault):
    n, rows, cols, group, xg = case
    L, cfg = layer(rows, cols, group, 1), G.make_config(group_size=group)
    codes, scales = acts(n, cols, xg)
    stalled_between(G, getattr(G, fault),
                    lambda: (G.gptq_w4a8_matmul(*L, cfg, codes, scales, dtype=BF),))


@pytest.mark.parametrize("fault", ["FAULT_W4A8_LOADS", "FAULT_W4A8_STAGES"])
@pytest.mark.parametrize("dtype", [F32, I8])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_gated_wait_runs_out(G, case, dtype, fault):
    n, rows, cols, group, xg = case
    gate, up = layer(rows, cols, group, 1), layer(rows, cols, group, 2)
    cfg = G.make_config(group_size=group)
    codes, scales = acts(n, cols, xg)
    scales *= 1e-3  # gates of ordinary size

    def call():
        out = G.gptq_w4a8_gated(gate, up, cfg, codes, scales, dtype=dtype)
        return out if dtype == I8 else (out,)

    stalled_between(G, getattr(G, fault), call)


def test_a_captured_call_reports_its_stall(G):
    """The switch holds for the launches made under it: a graph captured under it
    stalls at each replay, one captured without it never does."""
    L, cfg = layer(256, 16384, 128, 1), G.make_config(group_size=128)
    codes, scales = acts(40, 16384, 128)
    want = G.gptq_w4a8_matmul(*L, cfg, codes, scales)
    good, bad = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(good):
        got = G.gptq_w4a8_matmul(*L, cfg, codes, scales)
    G.gptq_fault_inject(G.FAULT_W4A8_LOADS, LIMIT_NS)
    try:
        with torch.cuda.graph(bad):
            G.gptq_w4a8_matmul(*L, cfg, codes, scales)
    finally:
        G.gptq_fault_inject(G.FAULT_NONE, 0)
    for graph, status in ((good, 0), (bad, TIMEOUT), (bad, TIMEOUT), (good, 0)):
        graph.replay()
        assert G.gptq_device_status() == status
    assert torch.equal(got, want)
