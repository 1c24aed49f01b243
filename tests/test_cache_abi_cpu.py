"""Host-side checks of the cache operators' arguments: what the C entry points and
the binding refuse before a GPU is touched."""
import ctypes

import pytest
import torch

import bit_ternary_matmul_gb300 as q


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


P = 0x100000  # never dereferenced: validation fails first


def _cache(**over):
    f = dict(k=P, v=P, n_pages=10, n_layers=2, n_kv=2, page=16, dim=64, type=q.Q2_0_TYPE_F16)
    f.update(over)
    return q._KvCacheStruct(**f)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=P + 8), dict(n_pages=0), dict(n_layers=0), dict(n_kv=0), dict(page=8),
              dict(page=24), dict(page=512), dict(dim=96), dict(dim=256), dict(type=2), dict(type=-1),
              dict(n_pages=1 << 27), dict(n_kv=1 << 30, n_pages=1 << 30)]


def _append(L, c, **over):
    a = dict(layer=0, q=P, qs=256, k=P, ks=128, v=P, vs=128, T=3, n_q=4, pos=P, slot=P, seq=None, table=P, n_seq=3, width=4,
             rope=P, n_pos=10, rot=64, style=0, qo=P)
    a.update(over)
    return L.q2_0_kv_append(ctypes.addressof(c) if c is not None else None, a["layer"], a["q"], a["qs"], a["k"], a["ks"],
                            a["v"], a["vs"], a["T"], a["n_q"], a["pos"], a["slot"], a["seq"], a["table"], a["n_seq"],
                            a["width"], a["rope"], a["n_pos"], a["rot"], a["style"], a["qo"], None)


def test_append_refusals(L):
    assert _append(L, None) == q.Q2_0_EINVAL
    for over in BAD_CACHES:
        assert _append(L, _cache(**over)) == q.Q2_0_EINVAL, over
    c = _cache()
    for over in (dict(layer=-1), dict(layer=2), dict(q=None), dict(k=None), dict(v=None), dict(slot=None), dict(table=None),
                 dict(T=-1), dict(n_q=-1), dict(qs=255), dict(ks=127), dict(vs=100), dict(pos=None), dict(rope=None),
                 dict(n_pos=0), dict(rot=66), dict(rot=7), dict(rot=-2), dict(style=2), dict(style=-1), dict(qo=None),
                 dict(n_seq=0), dict(n_seq=2), dict(width=0), dict(T=1 << 31)):
        assert _append(L, c, **over) == q.Q2_0_EINVAL, over
    assert _append(L, c, T=0, k=None, q=None) == q.Q2_0_OK


def _desc(c=None, **over):
    a = dict(cache=c or _cache(), q=P, out=P, n_groups=2, n_seq=3, n_q=4, scale=0.1, prefix_table=P, prefix_len=P,
             prefix_width=3, table=P, len=P, width=5)
    a.update(over)
    return q._AttnDesc(**a)


def test_attention_refusals(L):
    h = ctypes.c_void_p()
    assert L.q2_0_attn_plan_create(None, ctypes.byref(h)) == q.Q2_0_EINVAL
    assert L.q2_0_attn_plan_create(ctypes.byref(_desc()), None) == q.Q2_0_EINVAL
    for d in [_desc(_cache(**o)) for o in BAD_CACHES] + [_desc(**o) for o in (
            dict(q=None), dict(out=None), dict(q=P + 4), dict(out=P + 2), dict(table=None), dict(len=None), dict(n_groups=0),
            dict(n_seq=0), dict(n_groups=300, n_seq=300), dict(n_q=0), dict(n_q=3), dict(n_q=130), dict(width=0),
            dict(prefix_width=-1), dict(prefix_table=None), dict(prefix_len=None), dict(width=1 << 27),
            dict(prefix_width=1 << 27), dict(scale=float("inf")), dict(scale=float("nan")),
            dict(n_groups=255, n_seq=255, n_q=8192, cache=_cache(n_kv=512, n_pages=1)))]:
        assert L.q2_0_attn_plan_create(ctypes.byref(d), ctypes.byref(h)) == q.Q2_0_EINVAL
        assert not h.value
    assert L.q2_0_attn_plan_execute(None, 0, None) == q.Q2_0_EINVAL
    assert L.q2_0_attn_plan_launches(None) == 0
    L.q2_0_attn_plan_destroy(None)


def test_select_refusals(L):
    def call(**over):
        a = dict(x=P, stride=100, score=P, done=None, G=2, W=3, V=100, n=3, so=P, po=P, to=P, ws=None, wb=0)
        a.update(over)
        return L.q2_0_beam_select(a["x"], a["stride"], a["score"], a["done"], 0, a["G"], a["W"], a["V"], a["n"], a["so"],
                                  a["po"], a["to"], a["ws"], a["wb"], None)
    for over in (dict(x=None), dict(score=None), dict(so=None), dict(po=None), dict(to=None), dict(stride=99), dict(G=-1),
                 dict(W=0), dict(W=65), dict(V=0), dict(V=1 << 31, stride=1 << 31), dict(n=0), dict(n=33), dict(G=30000)):
        assert call(**over) == q.Q2_0_EINVAL, over
    assert call(G=0, x=None) == q.Q2_0_OK
    need = L.q2_0_beam_select_workspace_size(2, 3, 100, 3)
    assert need > 0 and need % 256 == 0
    assert call(ws=P, wb=need - 1) == q.Q2_0_EINVAL
    assert call(ws=P + 16, wb=need) == q.Q2_0_EINVAL
    assert L.q2_0_beam_select_workspace_size(2, 3, 100, 33) == 0
    assert L.q2_0_beam_select_workspace_size(2, 3, 200000, 3) > need


def test_reorder_refusals(L):
    def call(c=_cache(), **over):
        a = dict(parent=P, G=2, W=4, table=P, len=P, width=3, fresh=P, to=P, lo=P, used=P)
        a.update(over)
        return L.q2_0_beam_reorder(ctypes.addressof(c) if c is not None else None, a["parent"], a["G"], a["W"], a["table"],
                                   a["len"], a["width"], a["fresh"], a["to"], a["lo"], a["used"], None)
    assert call(None) == q.Q2_0_EINVAL
    for over in BAD_CACHES:
        assert call(_cache(**over)) == q.Q2_0_EINVAL, over
    for over in (dict(parent=None), dict(table=None), dict(len=None), dict(fresh=None), dict(to=None), dict(lo=None),
                 dict(used=None), dict(G=-1), dict(W=0), dict(W=1025), dict(width=0), dict(width=1 << 31), dict(G=1 << 30)):
        assert call(**over) == q.Q2_0_EINVAL, over
    assert call(G=0, parent=None) == q.Q2_0_OK


def test_binding_refuses_tensors_that_do_not_fit():
    f16 = torch.zeros((1, 2, 1, 16, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        q.KvCache(f16, f16)                      # not on a GPU
    with pytest.raises(ValueError):
        q.KvCache(f16.float(), f16.float())
    with pytest.raises(ValueError):
        q.KvCache(f16, f16[:, :1])
    with pytest.raises(TypeError):
        q.KvCache(f16, None)
    with pytest.raises(ValueError):
        q.q2_0_beam_select(torch.zeros((1, 2, 5)), torch.zeros((1, 2)))
    with pytest.raises(TypeError):
        q.q2_0_beam_select(None, torch.zeros((1, 2)))
