"""What the calls of normed heads and of the cache in 8 bits refuse, without a GPU."""
import ctypes

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


def handle(kind):
    """An object of a kind of descriptor, over no tensors (the calls below end before they look at any)."""
    x = kind.__new__(kind)
    x.zeros = ctypes.create_string_buffer(256)
    setattr(x, {moe.KvCache: "_at", moe.KvCacheQ8: "_at8"}[kind], ctypes.addressof(x.zeros))
    return x


@pytest.mark.parametrize("wrong", ["cache", "cache q8", "norm", "none", "number"])
def test_another_kind_of_descriptor_is_refused_by_name(lib, wrong):  # noqa: F811
    """Each call that takes a cache or a norm says which argument is of the wrong kind, and reads nothing of it."""
    x = {"cache": handle(moe.KvCache), "cache q8": handle(moe.KvCacheQ8), "norm": moe.HeadNorm(), "none": None, "number": 5}[wrong]
    plain, q8, norm = handle(moe.KvCache), handle(moe.KvCacheQ8), moe.HeadNorm()
    n6 = [None] * 6
    calls = []
    if wrong != "cache":
        calls += [(lambda: moe.moe_kv_append(*n6, x, None, None), "cache", "KvCache"),
                  (lambda: moe.moe_kv_append_norm(*n6, norm, x, None, None), "cache", "KvCache"),
                  (lambda: moe.moe_tree_attention(*[None] * 4, x, None, None, None), "cache", "KvCache")]
    if wrong != "cache q8":
        calls += [(lambda: moe.moe_kv_append_q8(*n6, norm, x, None, None), "cache", "KvCacheQ8"),
                  (lambda: moe.moe_kv_read_q8(None, x, None, None, None), "cache", "KvCacheQ8"),
                  (lambda: moe.moe_tree_attention_q8(*[None] * 4, x, None, None, None), "cache", "KvCacheQ8")]
    if wrong != "norm":
        calls += [(lambda: moe.moe_kv_append_norm(*n6, x, plain, None, None), "norm", "HeadNorm")]
        if wrong != "none":
            calls += [(lambda: moe.moe_kv_append_q8(*n6, x, q8, None, None), "norm", "HeadNorm")]
    for call, name, kind in calls:
        with pytest.raises(ValueError, match=f"{name} must be a {kind}, not a "):
            call()
