"""What the calls of normed heads and of the cache in 8 bits refuse, without a GPU."""
import pytest

import test_q8_abi as abi
from test_q8_abi import lib, moe  # noqa: F401


@pytest.mark.parametrize("eps,D", [(3e36, 128), (3e38, 16), (1.4e36, 256)])
def test_q8_append_refuses_an_eps_whose_sum_passes_fp32(lib, eps, D):  # noqa: F811
    """Its exact root counts with eps * head_dim."""
    c = abi.cache(page_table=None, n_requests=0, max_pages=0, head_dim=D)
    assert abi.append(lib, c, n=abi.norm(eps=eps), rot=0) == moe.MOE_ERR_ARG
    assert b"eps" in lib.moe_last_error()
    assert abi.append(lib, c, n=abi.norm(eps=1e36), rot=0, T=0) == moe.MOE_OK
