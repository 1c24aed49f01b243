"""Calls on a stream that is not the current one: what they allocate for themselves belongs to the
stream they run on, and their results do not depend on what the current stream does meanwhile."""
import numpy as np
import pytest
import torch

import bit_ternary_matmul_gb300 as q

pytestmark = pytest.mark.gpu

N, K = 192, 512


@pytest.fixture(scope="module", autouse=True)
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    q.build()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    assert q.q2_0_device_check() == q.Q2_0_OK
    q.q2_0_get_error()
    return d


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.fixture(scope="module")
def calls(dev):
    """name: (call of a stream, the tensors that it changes and their contents before), of every call that
    allocates something."""
    g = torch.Generator(device="cuda").manual_seed(1)
    src = torch.randn((N, K), generator=g, device="cuda") * 0.1
    w = q.q2_0_quantize_ref(src, N, K)
    experts = torch.cat([w, q.q2_0_quantize_ref(-src, N, K)])
    chosen = _ints([[0], [1], [1], [0], [1], [0]])
    zeros = torch.zeros(30, dtype=torch.int32, device="cuda")
    split = q.q2_0_split_layout(w, N, K)
    x = torch.randn((40, K), generator=g, device="cuda")
    one, h, ids = x[:1].contiguous(), x.half(), _ints([3, 0, 191, 7])
    w128 = torch.randint(0, 256, (N * (K // 128), 34), generator=g, device="cuda", dtype=torch.uint8)
    w128[:, 0], w128[:, 1] = 0, 0x2C            # finite scales
    w128 = w128.reshape(-1)
    ws = torch.empty(q.q2_0_mul_mat_vec_workspace_size(K, 1), dtype=torch.uint8, device="cuda")
    kc, vc = (torch.randn((2, 40, 2, 16, 64), generator=g, device="cuda").half() for _ in range(2))
    cache, k0, v0 = q.KvCache(kc, vc), kc.clone(), vc.clone()
    qkv = torch.randn((30, 8, 64), generator=g, device="cuda")
    rope = torch.randn((50, 64), generator=g, device="cuda")
    place, row = _ints(np.arange(30)), _ints([[4, 9]])
    logits = torch.randn((3, 5, 30011), generator=g, device="cuda") * 3
    scores = -torch.rand((3, 5), generator=g, device="cuda")
    table = _ints(np.arange(20).reshape(10, 2))
    parent, length, fresh = _ints([[0, 0, 1, 1, 4], [2, 2, 2, 0, 1]]), _ints([21] * 10), _ints(np.arange(20, 30))
    kv = ((kc, k0), (vc, v0))
    return {
        "quantize_ref": (lambda s: q.q2_0_quantize_ref(src, N, K, stream=s), ()),
        "mul_mat_vec": (lambda s: q.q2_0_mul_mat_vec(w, one, N, K, stream=s), ()),
        "mul_mat_vec_f16": (lambda s: q.q2_0_mul_mat_vec_f16(w, h[:2], N, K, stream=s), ()),
        "mul_mat_vec_ws": (lambda s: q.q2_0_mul_mat_vec_ws(w, one, N, K, 1, ws, stream=s), ()),
        "mul_mat_vec_noalloc": (lambda s: q.q2_0_mul_mat_vec_noalloc(w, one, N, K, stream=s), ()),
        "mul_mat": (lambda s: q.q2_0_mul_mat(w, x, N, K, stream=s), ()),
        "mul_mat_f16": (lambda s: q.q2_0_mul_mat_f16(w, h, N, K, stream=s), ()),
        "get_rows": (lambda s: q.q2_0_get_rows(w, N, K, ids, stream=s), ()),
        "mul_mat_id": (lambda s: q.q2_0_mul_mat_id(experts, 2, N, K, x[:6], chosen, stream=s), ()),
        "split_layout": (lambda s: q.q2_0_split_layout(w, N, K, stream=s), ()),
        "join_layout": (lambda s: q.q2_0_join_layout(split, N, K, stream=s), ()),
        "mul_mat_vec_split": (lambda s: q.q2_0_mul_mat_vec_split(split, one, N, K, stream=s), ()),
        "g128_to_g64": (lambda s: q.q2_0_g128_to_g64(w128, N, K, stream=s), ()),
        "g128_get_rows": (lambda s: q.q2_0_g128_get_rows(w128, N, K, ids, stream=s), ()),
        "g128_mul_mat_vec": (lambda s: q.q2_0_g128_mul_mat_vec(w128, one, N, K, stream=s), ()),
        "kv_append": (lambda s: q.q2_0_kv_append(cache, 1, qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], place, place, row, rope,
                                                 seq=zeros, stream=s), kv),
        "beam_select": (lambda s: q.q2_0_beam_select(logits, scores, 6, stream=s), ()),
        "beam_reorder": (lambda s: q.q2_0_beam_reorder(cache, parent, table, length, fresh, stream=s), kv),
    }


NAMES = ["quantize_ref", "mul_mat_vec", "mul_mat_vec_f16", "mul_mat_vec_ws", "mul_mat_vec_noalloc", "mul_mat", "mul_mat_f16",
         "get_rows", "mul_mat_id", "split_layout", "join_layout", "mul_mat_vec_split", "g128_to_g64", "g128_get_rows",
         "g128_mul_mat_vec", "kv_append", "beam_select", "beam_reorder"]


class _NoCalls:
    """A library whose calls do nothing, but for the sizes."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name.endswith(("_size", "_bytes", "_launches")):
            return getattr(self.real, name)
        return lambda *a: q.Q2_0_OK


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_buffers_belong_to_the_stream_of_the_call(name, handle, calls, monkeypatch):
    """No kernel runs here: the stream that is current at each allocation."""
    side = torch.cuda.Stream()
    seen, empty, empty_like = [], torch.empty, torch.empty_like

    def note(f):
        def g(*a, **k):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return f(*a, **k)
        return g
    call = calls[name][0]
    real = q.lib()
    monkeypatch.setattr(q, "lib", lambda: _NoCalls(real))
    monkeypatch.setattr(torch, "empty", note(empty))
    monkeypatch.setattr(torch, "empty_like", note(empty_like))
    out = call(side.cuda_stream if handle else side)
    assert out is not None
    assert seen and set(seen) == {side.cuda_stream}, (name, seen)
    seen.clear()
    call(None)
    assert set(seen) == {torch.cuda.current_stream().cuda_stream}


def _flat(out):
    return [t.clone() for t in (out if isinstance(out, tuple) else (out,))]


@pytest.mark.parametrize("name", NAMES)
def test_results_beside_a_busy_current_stream(name, calls):
    """The current stream has work queued that fills memory it has freed since; two other streams call."""
    call, changed = calls[name]

    def restore():
        for t, before in changed:
            t.copy_(before)
    restore()
    want = _flat(call(None)) + [t.clone() for t, _ in changed]
    restore()
    torch.cuda.synchronize()
    # (one alone where two calls at a time would share a cache or a workspace)
    one = changed or name.endswith(("_ws", "_noalloc"))
    sides = [torch.cuda.Stream() for _ in range(1 if one else 2)]
    for _ in range(3):
        restore()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)              # about 10 ms
        junk = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 20) for _ in range(4)]
        del junk
        got = [call(s) for s in sides]
        for s in sides:
            s.synchronize()
        torch.cuda.synchronize()
        for out in got:
            for a, b in zip(_flat(out) + [t for t, _ in changed], want):
                assert torch.equal(a, b), name
    assert q.q2_0_get_error() == (0, 0)
