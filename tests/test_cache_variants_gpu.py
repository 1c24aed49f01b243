"""The decode step's operators in every variant that a plan may take: moving references, launches, captured
graphs that follow the lengths, and side streams."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_ternary_matmul_gb300 as q
from test_cache_ops_gpu import BF16, F16, Attn, _ints, _no_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    q.build()
    torch.cuda.set_device(0)
    assert q.q2_0_device_check() == q.Q2_0_OK
    q.q2_0_get_error()


VARIANTS = [
    # sequences, n_q, n_kv, dim, dtype; query rows of a prefix's product = sequences * n_q / n_kv
    (4, 8, 2, 64, F16),        # 16
    (8, 8, 2, 128, BF16),      # 32
    (12, 8, 2, 128, F16),      # 48
    (16, 16, 4, 64, BF16),     # 64
    (17, 16, 4, 128, F16),     # 68
    (32, 8, 2, 64, BF16),      # 128
    (33, 8, 2, 128, BF16),     # 132
    (70, 8, 2, 64, F16),       # 280
    (3, 48, 1, 64, F16),       # 48 a sequence, 144
]


@pytest.mark.parametrize("n,n_q,n_kv,dim,dtype", VARIANTS)
def test_launches(n, n_q, n_kv, dim, dtype):
    """Three where a prefix is shared by more than 64 query heads of a kv head, else two."""
    c = Attn([100], [5] * n, n_q, n_kv, dim, 16, dtype)
    plan = c.plan()
    assert plan.launches == (3 if n * n_q // n_kv > 64 else 2)
    assert c.plan(shared=False).launches == 2


@pytest.mark.parametrize("how", ["rising", "falling", "late_peak", "flat", "steep", "steps"])
@pytest.mark.parametrize("n,n_q,n_kv,dim,dtype", VARIANTS)
def test_moving_references(n, n_q, n_kv, dim, dtype, how):
    """Scores whose maximum moves from tile to tile, sits in one key, or rises by a step in every tile."""
    def k_of(k):
        t = torch.arange(k.shape[1], device="cuda")[None, :, None]
        m = max(1, k.shape[1])
        if how == "rising":
            return k * (0.05 + 6.0 * t / m)
        if how == "falling":
            return k * (0.05 + 6.0 * (m - t) / m)
        if how == "late_peak":
            return torch.where(t == m - 3, k * 20, k * 0.1)
        if how == "flat":
            return k * 0
        if how == "steep":
            return k * 12
        return torch.full_like(k, dim ** -0.5) * (10.0 * (t // 128) + 1) + 0.02 * k
    # two prefixes, long enough that a block has several tiles of one
    plens, lens = ([26000, 24100] if n < 64 else [14000, 9001]), [(57 * i) % 400 for i in range(2 * n)]
    c = Attn(plens, lens, n_q, n_kv, dim, 128, dtype, seed=41, k_of=k_of)
    if how == "steps":
        c.q.copy_(torch.ones_like(c.q) + 0.02 * c.q)
    plan = c.plan()
    plan.execute(0)
    _no_error()
    c.check(how)
    first = c.out.clone()
    for _ in range(3):
        plan.execute(0)
        assert torch.equal(c.out, first), "the same inputs gave other outputs"


def _shorter(c, full, plen, lens):
    c.t_plen.copy_(_ints([plen]))
    c.t_len.copy_(_ints(lens))
    c.plens, c.lens = [plen], lens
    c.ks = [full[0][0][:, :plen]] + [full[0][1 + i][:, :n] for i, n in enumerate(lens)]
    c.vs = [full[1][0][:, :plen]] + [full[1][1 + i][:, :n] for i, n in enumerate(lens)]
    c.out.fill_(math.nan)


@pytest.mark.parametrize("n,n_q,n_kv,dim,dtype", VARIANTS)
def test_a_captured_execute_follows_the_lengths(n, n_q, n_kv, dim, dtype):
    c = Attn([3000], [300] * n, n_q, n_kv, dim, 16, dtype, seed=43)
    full = c.ks, c.vs
    plan = c.plan()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.execute(0)
    side.synchronize()
    _no_error()
    c.check("on a side stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):      # executes one behind the other, as the layers of a step
            plan.execute(0)
    for plen, lens in ((3000, [300] * n), (77, [(i * 13) % 301 for i in range(n)]), (0, [i % 3 for i in range(n)]),
                       (2999, [0] * n), (129, [1] * n)):
        _shorter(c, full, plen, lens)
        g.replay()
        torch.cuda.synchronize()
        _no_error()
        c.check(f"{plen} {lens[:3]}")


def test_a_captured_step_of_append_selection_and_reordering():
    """One graph of the three calls, replayed on new contents; compared with the calls one by one."""
    g = torch.Generator(device="cuda").manual_seed(9)
    layers, pages, n_kv, page, dim, W, V = 2, 64, 2, 16, 64, 6, 20011
    k = torch.randn((layers, pages, n_kv, page, dim), generator=g, device="cuda").half()
    v = torch.randn((layers, pages, n_kv, page, dim), generator=g, device="cuda").half()
    cache = q.KvCache(k, v)
    qkv = torch.randn((W, (4 + 2 * n_kv), dim), generator=g, device="cuda")
    rope = torch.randn((100, dim), generator=g, device="cuda")
    logits, scores = torch.empty((1, W, V), device="cuda"), torch.empty((1, W), device="cuda")
    table, place, length = _ints(np.arange(3 * W).reshape(W, 3)), _ints([0] * W), _ints([0] * W)
    fresh = _ints(np.arange(3 * W, 4 * W))

    def step():
        a = q.q2_0_kv_append(cache, 1, qkv[:, :4], qkv[:, 4:4 + n_kv], qkv[:, 4 + n_kv:], place, place, table, rope)
        s, p, t = q.q2_0_beam_select(logits, scores, W)
        return (a, s, p, t) + q.q2_0_beam_reorder(cache, p, table, length, fresh)

    def contents(i):
        r = torch.Generator(device="cuda").manual_seed(100 + i)
        logits.copy_(torch.randn(logits.shape, generator=r, device="cuda") * 3)
        scores.copy_(-torch.rand(scores.shape, generator=r, device="cuda") * 4)
        qkv.copy_(torch.randn(qkv.shape, generator=r, device="cuda"))
        place.fill_(7 * i + 2)
        length.fill_(7 * i + 3)
    contents(0)
    step()
    torch.cuda.synchronize()
    k0, v0 = k.clone(), v.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = step()
    for i in range(5):
        contents(i)
        k.copy_(k0), v.copy_(v0)
        want = [x.clone() for x in step()] + [k.clone(), v.clone()]
        for x in made:
            x.zero_()
        k.copy_(k0), v.copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(list(made) + [k, v], want):
            assert torch.equal(a, b), i
    _no_error()


def test_a_plan_that_finds_no_memory_leaves_no_error_behind():
    """Scratch for 65535 sequences of 4096 heads and their prefix does not fit any GPU: the plan is refused, and
    the next call is not."""
    k = torch.zeros((1, 1, 64, 16, 128), dtype=F16, device="cuda")
    cache, some = q.KvCache(k, torch.zeros_like(k)), torch.zeros(64, dtype=F16, device="cuda")
    ids = torch.zeros(64, dtype=torch.int32, device="cuda")
    p, i = some.data_ptr(), ids.data_ptr()
    d = q._AttnDesc(cache._c, p, p, 1, 65535, 4096, 0.1, i, i, 1, i, i, 1)
    h = ctypes.c_void_p()
    assert q.lib().q2_0_attn_plan_create(ctypes.byref(d), ctypes.byref(h)) == q.Q2_0_ECUDA and not h.value
    x = torch.ones((1, 64, 128), device="cuda")
    q.q2_0_kv_append(cache, 0, None, x, x, None, ids[:1], ids[:1].reshape(1, 1), None)
    _no_error()
    assert (k[0, 0, :, 0] == 1).all()
