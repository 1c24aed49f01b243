"""Limits of the cache operators that are checked before a GPU is touched."""
import ctypes

import pytest
import torch

import bit_ternary_matmul_gb300 as q


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


P = 0x100000  # never dereferenced: validation fails first


def test_reordering_refuses_more_kv_heads_than_its_counters_hold(L):
    """A page of 256 tokens of 2^19 heads of 128 has 2^31 pieces of 16 bytes, which are counted in 32 bits."""
    def call(n_kv, page=256):
        c = q._KvCacheStruct(k=P, v=P, n_pages=4, n_layers=1, n_kv=n_kv, page=page, dim=128, type=q.Q2_0_TYPE_F16)
        return L.q2_0_beam_reorder(ctypes.addressof(c), P, 1, 2, P, P, 3, P, P, P, P, None)
    for n_kv in ((1 << 16) + 1, 1 << 19, 1 << 21):
        assert call(n_kv) == q.Q2_0_EINVAL, n_kv
    assert call(1 << 20, 16) == q.Q2_0_EINVAL


def test_a_plan_refuses_prefix_lengths_without_their_pages():
    """They would be passed over, and the sequences would attend to their own tokens alone."""
    class Cache:
        k, dim = torch.zeros(1, dtype=torch.float16), 64
    x = torch.zeros((4, 2, 64), dtype=torch.float16)
    ids = torch.zeros((4, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="prefix_table"):
        q.AttnPlan(Cache, x, x, ids, ids[:, 0], prefix_len=torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):   # (a prefix's table is looked at first)
        q.AttnPlan(Cache, x, x, ids, ids[:, 0], prefix_table=ids[:1], prefix_len=torch.ones(1, dtype=torch.int32))
