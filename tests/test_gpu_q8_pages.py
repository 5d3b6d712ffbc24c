"""moe_tree_attention_q8 on tensor cores with pages and blocks that are no powers of two."""
import pytest

import test_gpu_attention_q8 as attend

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("aware_expert_routing_gb300")


@pytest.fixture(scope="module", autouse=True)
def built():
    from aware_expert_routing_gb300 import build as b
    b.build()
    moe.load()


# rows a key head: 8, 24, 128, 320
@pytest.mark.parametrize("n", [[1, 1], [3, 2], [16, 15], [40, 33]])
@pytest.mark.parametrize("D,page,block", [(128, 384, 3), (64, 384, 96), (128, 384, 384), (64, 640, 5), (128, 128, 2)])
def test_pages_and_blocks_that_are_no_powers_of_two(n, D, page, block):
    c = attend.Case([1000, 383], n, 16, 2, D, page, block, "bf16", n[0] > 1, 47 + page)
    out, l, flags = c.run()
    assert flags == 0
    c.check(out, l)
