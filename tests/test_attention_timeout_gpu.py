"""The attention kernels' waits are bounded: q2_0_test_stall_attention makes every block of one execute stop
copying keys some tiles into its share. The waits run out (after a second), the execute records
Q2_0_DEVERR_TIMEOUT (info 301 to 314), the join that follows it stays inside the plan's scratch, whatever
that memory held before the plan, and the next executes are correct."""
import math
import time

import pytest
import torch

import bit_ternary_matmul_gb300 as q
from test_cache_ops_gpu import BF16, F16, Attn

pytestmark = pytest.mark.gpu

CASES = [
    # prefix lengths, own lengths, n_q, n_kv, dim, dtype: 200 to 900 tiles of 128 keys
    ([0], [700 + 30 * i for i in range(30)], 8, 2, 128, F16),       # own tokens, 4 rows a product
    ([15000], [40, 0, 300, 7], 16, 4, 128, BF16),                   # a prefix of 16 rows
    ([9000, 8000], [200] * 20, 16, 4, 64, F16),                     # prefixes of 40 rows
    ([0], [1500] * 20, 96, 2, 64, BF16),                            # own tokens, 48 rows
    ([15000], [150] * 30, 16, 4, 128, F16),                         # a prefix of 120 rows: launches of their own
    ([15000], [130] * 70, 16, 4, 64, BF16),                         # and of 280
]


@pytest.fixture(scope="module", autouse=True)
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    q.build()
    torch.cuda.set_device(0)
    assert q.q2_0_device_check() == q.Q2_0_OK
    q.q2_0_get_error()


@pytest.mark.parametrize("stage", [0, 2])
@pytest.mark.parametrize("plens,lens,n_q,n_kv,dim,dtype", CASES)
def test_stalled_attention_times_out_and_recovers(plens, lens, n_q, n_kv, dim, dtype, stage):
    c = Attn(plens, lens, n_q, n_kv, dim, 64, dtype, seed=3)
    dirt = [torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del dirt
    torch.cuda.empty_cache()        # a new plan's scratch may be this memory
    plan = c.plan()
    q.q2_0_test_stall_attention(stage)
    t0 = time.perf_counter()
    plan.execute(0)
    code, info = q.q2_0_get_error()     # synchronises
    assert code == q.Q2_0_DEVERR_TIMEOUT and 301 <= info <= 314, (code, info)
    assert time.perf_counter() - t0 < 15.0
    for _ in range(2):
        c.out.fill_(math.nan)
        plan.execute(0)
        assert q.q2_0_get_error() == (0, 0)
        c.check("after the stall")
    if stage == 2:      # now with an earlier execute's records
        q.q2_0_test_stall_attention(stage)
        plan.execute(0)
        code, info = q.q2_0_get_error()
        assert code == q.Q2_0_DEVERR_TIMEOUT and 301 <= info <= 314, (code, info)
        plan.execute(0)
        assert q.q2_0_get_error() == (0, 0)
        c.check("after the second stall")
    plan.close()


@pytest.mark.parametrize("plens,lens,n_q,n_kv,dim,dtype", [
    ([0], [100 + i % 150 for i in range(400)], 8, 2, 128, F16),         # 5 or more segments a block: the next one's
    ([0], [100 + i % 150 for i in range(200)], 96, 2, 64, BF16),        # queries are copied ahead, or behind the last
    ([300] * 90, [5] * 90 * 32, 16, 4, 64, F16)])                       # prefixes of 128 rows
def test_stalled_attention_with_queries_in_flight(plens, lens, n_q, n_kv, dim, dtype):
    test_stalled_attention_times_out_and_recovers(plens, lens, n_q, n_kv, dim, dtype, 0)
    test_stalled_attention_times_out_and_recovers(plens, lens, n_q, n_kv, dim, dtype, 8)
