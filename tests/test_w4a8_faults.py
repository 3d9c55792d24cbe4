"""The switches that make waits of the W4A8 kernels run out, without a GPU."""
import os
import re

import pytest

from post_weight_quantization_26_b200 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gptq.h")


@pytest.fixture(scope="module")
def G():
    B.build()
    from post_weight_quantization_26_b200 import gptq
    gptq.load_library()
    yield gptq
    gptq.gptq_fault_inject(gptq.FAULT_NONE, 0)


def test_switches(G):
    f = G.load_library().gptq_fault_inject
    named = dict(re.findall(r"GPTQ_(FAULT_\w+) = (\d+)", open(HEADER).read()))
    assert len(named) == 5
    for name, value in named.items():  # the binding's names are the header's
        assert getattr(G, name) == int(value)
        assert f(int(value), 20_000_000) == 0
    for unknown in (3, 6, -1):
        assert f(unknown, 0) == 1
    assert f(G.FAULT_W4A8_LOADS, 999_999) == 1 and f(G.FAULT_W4A8_STAGES, 10_000_000_001) == 1
    assert f(G.FAULT_NONE, 0) == 0
