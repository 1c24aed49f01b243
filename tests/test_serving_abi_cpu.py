"""What routing, verification and the calls on rows of pages refuse before a GPU is touched."""
import ctypes

import pytest
import torch

import bit_ternary_matmul_gb300 as q


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


P = 0x1000000  # never dereferenced: validation fails first
Q = P + (1 << 20)
EINVAL = q.Q2_0_EINVAL


def _passes(call, **over):
    """The arguments themselves are accepted. (Without a GPU alone: nothing is launched then.)"""
    if not torch.cuda.is_available():
        assert call(**over) in (q.Q2_0_ECUDA, q.Q2_0_EUNSUPPORTED), over


def _cache(**over):
    f = dict(k=P, v=P, n_pages=10, n_layers=2, n_kv=2, page=16, dim=64, type=q.Q2_0_TYPE_F16)
    f.update(over)
    return q._KvCacheStruct(**f)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=P + 8), dict(n_pages=0), dict(n_layers=0), dict(n_kv=0), dict(page=8),
              dict(page=24), dict(page=512), dict(dim=96), dict(type=2), dict(n_pages=1 << 27)]


def _rows(**over):
    f = dict(refs=P, table=P + 4096, len=P + 8192, n_rows=4, width=3)
    f.update(over)
    return q._KvRowsStruct(**f)


BAD_ROWS = [dict(refs=None), dict(table=None), dict(len=None), dict(n_rows=0), dict(n_rows=(1 << 20) + 1), dict(width=0),
            dict(width=1 << 27)]
# beside _rows(): 40 bytes of counts, 48 of a table, 16 of lengths
BAD_OUT = [dict(refs=None), dict(n_rows=5), dict(width=4), dict(refs=P + 36), dict(refs=P - 36), dict(table=P + 4096 + 44),
           dict(table=P + 4096 - 44), dict(len=P + 8192 + 12), dict(len=P), dict(refs=P + 4096), dict(table=P + 8192)]


def _ref(x):
    return None if x is None else ctypes.addressof(x)


def test_route_refusals(L):
    def call(router=True, x=P, stride=8, T=3, ids=Q, w=Q + 4096, **over):
        f = dict(n_expert=8, n_used=2, score=0, n_group=1, n_group_used=1, group_top=1, norm=1, scale=1.0, bias=None)
        f.update(over)
        r = q._RouterStruct(**f)
        return L.q2_0_moe_route(_ref(r) if router else None, x, stride, T, ids, w, None)
    for over in (dict(router=False), dict(x=None), dict(ids=None), dict(w=None), dict(stride=7), dict(T=-1), dict(T=1 << 31),
                 dict(n_expert=0), dict(n_expert=1025, stride=1025), dict(n_used=0), dict(n_used=9), dict(score=2),
                 dict(score=-1), dict(n_group=0), dict(n_group=3), dict(n_group_used=0), dict(n_group_used=2),
                 dict(n_group=4, n_group_used=2, n_used=5), dict(group_top=0), dict(group_top=3), dict(scale=float("inf")),
                 dict(scale=float("nan")), dict(n_expert=66, stride=66, n_group=33, n_group_used=33),
                 dict(n_expert=64, stride=64, n_used=33)):
        assert call(**over) == EINVAL, over
    assert call(T=0, x=None) == q.Q2_0_OK
    for over in (dict(), dict(n_expert=1024, stride=1024, n_used=32), dict(n_group=4, n_group_used=2, n_used=4, group_top=2)):
        _passes(call, **over)


def test_route_refuses_outputs_that_overlap(L):
    """3 rows of 8 logits, 10 apart, end 112 bytes on; a row's 2 outputs take 24 bytes; a bias 32."""
    def call(x=P, ids=Q, w=Q + 4096, bias=None, T=3, stride=10):
        r = q._RouterStruct(8, 2, 0, 1, 1, 1, 1, 1.0, bias)
        return L.q2_0_moe_route(_ref(r), x, stride, T, ids, w, None)
    for over in (dict(w=Q), dict(w=Q + 20), dict(w=Q - 20), dict(ids=P), dict(ids=P + 108), dict(ids=P - 20), dict(w=P + 108),
                 dict(bias=Q + 20), dict(bias=Q + 4096 - 28), dict(ids=P + 4096, stride=1 << 61)):
        assert call(**over) == EINVAL, over
    for over in (dict(w=Q + 24), dict(ids=P + 112), dict(ids=P - 24), dict(bias=Q + 24), dict(bias=Q + 4096 - 32),
                 dict(x=Q + 4096 + 24), dict(T=1, stride=1 << 61)):
        _passes(call, **over)


def test_verify_refusals(L):
    def call(**over):
        a = dict(t=P, ts=100, d=P, ds=100, tok=P, count=None, rand=P, n=2, k=3, V=100, acc=Q, out=Q + 4096)
        a.update(over)
        return L.q2_0_draft_verify(a["t"], a["ts"], a["d"], a["ds"], a["tok"], a["count"], a["rand"], a["n"], a["k"], a["V"],
                                   a["acc"], a["out"], None)
    for over in (dict(t=None), dict(ts=99), dict(ds=99), dict(tok=None), dict(rand=None), dict(n=-1), dict(n=65536),
                 dict(k=-1), dict(k=1025), dict(V=0), dict(V=1 << 31, ts=1 << 31, ds=1 << 31), dict(acc=None),
                 dict(out=None)):
        assert call(**over) == EINVAL, over
    assert call(n=0, t=None) == q.Q2_0_OK
    for over in (dict(), dict(d=None, ds=0), dict(k=0, tok=None, d=None), dict(count=P)):
        _passes(call, **over)


def test_verify_refuses_outputs_that_overlap(L):
    """2 sequences of 3 drafts over 100 tokens: 8 rows, 104 apart, end 3312 bytes on, the drafts' 6 2480; the drafts
    take 24 bytes, counts 8, numbers 32, the outputs 8 and 32."""
    at = dict(t=P, d=P + (1 << 16), tok=P + (2 << 16), count=P + (3 << 16), rand=P + (4 << 16))
    ends = dict(t=3312, d=2480, tok=24, count=8, rand=32)

    def call(acc=Q, out=Q + 4096, k=3, d=at["d"], tok=at["tok"]):
        return L.q2_0_draft_verify(at["t"], 104, d, 104, tok, at["count"], at["rand"], 2, k, 100, acc, out, None)
    for name, p in at.items():
        for over in (dict(acc=p), dict(acc=p - 4), dict(acc=p + ends[name] - 4), dict(out=p), dict(out=p - 28),
                     dict(out=p + ends[name] - 4)):
            assert call(**over) == EINVAL, (name, over)
        for over in (dict(acc=p - 8), dict(acc=p + ends[name]), dict(out=p - 32), dict(out=p + ends[name])):
            _passes(call, **over)
    for over in (dict(out=Q), dict(out=Q + 4), dict(out=Q - 28)):
        assert call(**over) == EINVAL, over
    for over in (dict(out=Q + 8), dict(out=Q - 32), dict(out=at["tok"], k=0), dict(out=at["d"], d=None)):
        _passes(call, **over)


def test_copy_refusals(L):
    def call(c=_cache(), src=P, dst=P, count=None, n=3):
        return L.q2_0_kv_copy(_ref(c), src, dst, count, n, None)
    assert call(c=None) == EINVAL
    for over in BAD_CACHES:
        assert call(c=_cache(**over)) == EINVAL, over
    for over in (dict(src=None), dict(dst=None), dict(n=-1), dict(n=1 << 31)):
        assert call(**over) == EINVAL, over
    assert call(n=0, src=None) == q.Q2_0_OK


def _each_rows(call):
    assert call(c=None) == EINVAL
    assert call(r=None) == EINVAL
    for over in BAD_CACHES:
        assert call(c=_cache(**over)) == EINVAL, over
    for over in BAD_ROWS:
        assert call(r=_rows(**over)) == EINVAL, over
    for over in BAD_OUT:
        assert call(out=_rows(**over)) == EINVAL, over


def _each_workspace(call, need):
    """A workspace beside the rows, where their outcome goes, and the cache: 81920 bytes of keys, and of values."""
    rows, far = _rows(), 1 << 24
    for name in ("refs", "table", "len"):
        p = getattr(rows, name)
        for over in (dict(ws=p, wb=need), dict(ws=p + 256 - need, wb=need)):
            assert call(c=_cache(k=P + far, v=P + far), **over) == EINVAL, (name, over)
            out = _rows(**{n: getattr(rows, n) + far for n in ("refs", "table", "len")})
            assert call(c=_cache(k=P + 2 * far, v=P + 2 * far), out=out, ws=over["ws"] + far, wb=need) == EINVAL, (name, over)
    for k, v in ((P + far, P + 2 * far), (P + 2 * far, P + far)):
        for at in (0, 81920 - 256, 256 - need):
            assert call(c=_cache(k=k, v=v), ws=P + far + at, wb=need) == EINVAL, at
        for at in (81920, -need):
            _passes(call, c=_cache(k=k, v=v), ws=P + far + at, wb=need)


def test_fork_refusals(L):
    def call(c=_cache(), r=_rows(), parent=Q, child=Q, n=2, out=None):
        return L.q2_0_kv_fork(_ref(c), _ref(r), parent, child, n, _ref(out), None)
    _each_rows(call)
    for over in (dict(parent=None), dict(child=None), dict(n=-1), dict(n=4097), dict(parent=P + 32), dict(child=P + 4096),
                 dict(child=P + 8192 - 4), dict(parent=Q, out=_rows(len=Q + 4))):
        assert call(**over) == EINVAL, over
    for over in (dict(), dict(n=0, parent=None), dict(out=_rows()), dict(out=_rows(refs=P - 40, len=P + 8192 + 16))):
        _passes(call, **over)


def test_resize_refusals(L):
    need = L.q2_0_kv_resize_workspace_size(10, 4)

    def call(c=_cache(), r=_rows(), new=Q, out=None, ws=None, wb=0):
        return L.q2_0_kv_resize(_ref(c), _ref(r), new, _ref(out), ws, wb, None)
    _each_rows(call)
    up = (need + 255) // 256 * 256
    assert up == need
    _each_workspace(call, need)
    for over in (dict(new=None), dict(ws=Q, wb=need - 1), dict(ws=Q + 16, wb=need), dict(new=P), dict(new=P + 8192 + 4),
                 dict(new=P + 4096 - 12), dict(out=_rows(len=Q)), dict(out=_rows(table=Q - 44)), dict(ws=Q, wb=need),
                 dict(ws=Q + 512 - up, wb=need, new=Q + 508)):
        assert call(**over) == EINVAL, over
    for over in (dict(), dict(new=P + 8192), dict(new=P + 8192, out=_rows(refs=Q)), dict(out=_rows(len=Q + 16)),
                 dict(ws=Q + 256, wb=need), dict(ws=Q + 512 - up, wb=need, new=Q + 512)):
        _passes(call, **over)
    for bad in ((0, 4), (10, 0), (1 << 31, 4), (10, (1 << 20) + 1)):
        assert L.q2_0_kv_resize_workspace_size(*bad) == 0
        assert L.q2_0_kv_compact_workspace_size(*bad) == 0


def test_compact_refusals(L):
    need = L.q2_0_kv_compact_workspace_size(10, 4)

    def call(c=_cache(), r=_rows(), out=None, place=Q, live=Q + 64, ws=None, wb=0):
        return L.q2_0_kv_compact(_ref(c), _ref(r), _ref(out), place, live, ws, wb, None)
    _each_rows(call)
    _each_workspace(call, need)
    for over in (dict(place=None), dict(live=None), dict(ws=Q, wb=need - 1), dict(ws=Q + 16, wb=need), dict(live=Q + 36),
                 dict(ws=Q, wb=need), dict(ws=Q + 256, wb=need, live=Q + 256 + need - 4),
                 dict(ws=Q + 256, wb=need, place=Q + 256 - 36),
                 dict(place=P), dict(place=P + 4096 - 36), dict(live=P + 8192 + 12), dict(out=_rows(refs=Q + 8))):
        assert call(**over) == EINVAL, over
    for over in (dict(), dict(ws=Q + 256, wb=need), dict(ws=Q + 256, wb=need, live=Q + 256 + need), dict(out=_rows(table=Q + 128))):
        _passes(call, **over)


def _calls_on_rows(L):
    """(name, call) of every call on rows, with arguments that are accepted."""
    c = _cache(k=Q + (1 << 20), v=Q + (1 << 20))
    return [("fork", lambda r, out=None: L.q2_0_kv_fork(_ref(c), _ref(r), Q, Q, 2, _ref(out), None)),
            ("resize", lambda r, out=None: L.q2_0_kv_resize(_ref(c), _ref(r), Q, _ref(out), None, 0, None)),
            ("compact", lambda r, out=None: L.q2_0_kv_compact(_ref(c), _ref(r), _ref(out), Q, Q + 64, None, 0, None))]


def test_rows_whose_arrays_overlap_one_another_are_refused(L):
    """Of rows before a call, and of two new arrays for their outcome: 40 bytes of counts, 48 of a table, 16 of lengths."""
    bad = [dict(refs=P, table=P), dict(refs=P, len=P), dict(table=P, len=P), dict(refs=P, table=P + 36), dict(refs=P, table=P - 44),
           dict(refs=P, len=P + 36), dict(refs=P, len=P - 12), dict(table=P, len=P + 44), dict(table=P, len=P - 12)]
    good = [dict(refs=P, table=P + 40), dict(refs=P, table=P - 48), dict(refs=P, len=P + 40), dict(refs=P, len=P - 16),
            dict(table=P, len=P + 48), dict(table=P, len=P - 16), dict(refs=P, table=P + 40, len=P + 88)]
    far = 1 << 18

    def at(over, by=0):
        f = {n: P + (i + 5) * 4096 for i, n in enumerate(("refs", "table", "len"))}
        f.update(over)
        return {n: x + by for n, x in f.items()}
    for name, call in _calls_on_rows(L):
        for over in bad:
            assert call(_rows(**at(over))) == EINVAL, (name, over)                      # in place
            assert call(_rows(**at(over)), _rows(**at(over))) == EINVAL, (name, over)
            assert call(_rows(), _rows(**at(over, far))) == EINVAL, (name, over)        # new arrays
            assert call(_rows(**at(over)), _rows(**at({}, far))) == EINVAL, (name, over)
        for over in good:
            _passes(lambda r: call(r), r=_rows(**at(over)))
            _passes(lambda out: call(_rows(), out), out=_rows(**at(over, far)))


def test_numbers_in_the_pages_that_a_call_writes_are_refused(L):
    """Keys of 81920 bytes at P, values behind a gap."""
    k, v, far = P, P + (1 << 18), P + (1 << 19)
    c, r = _cache(k=k, v=v), _rows(refs=far + 4096, table=far + 8192, len=far + 12288)

    def copy(src=far, dst=far + 64, count=far + 128):
        return L.q2_0_kv_copy(_ref(c), src, dst, count, 3, None)

    def compact(place=far, live=far + 64):
        return L.q2_0_kv_compact(_ref(c), _ref(r), None, place, live, None, 0, None)
    for call, sizes in ((copy, dict(src=12, dst=12, count=12)), (compact, dict(place=40, live=4))):
        for name, size in sizes.items():
            for base in (k, v):
                for p in (base, base - size + 4, base + 81920 - 4):
                    assert call(**{name: p}) == EINVAL, (name, p)
                for p in (base - size, base + 81920):
                    _passes(call, **{name: p})
    _passes(copy, count=None)


def test_new_lengths_in_the_cache_are_refused(L):
    """Pages of keys and values are written by a change of lengths; the lengths themselves may be given, wherever they are."""
    k, v, far = P, P + (1 << 18), P + (1 << 19)
    c, r = _cache(k=k, v=v), _rows(refs=far + 4096, table=far + 8192, len=far + 12288)

    def call(new):
        return L.q2_0_kv_resize(_ref(c), _ref(r), new, None, None, 0, None)
    for base in (k, v):
        for p in (base, base - 12, base + 81920 - 4):
            assert call(p) == EINVAL, p
        for p in (base - 16, base + 81920, far + 12288):
            _passes(call, new=p)


def test_binding_refuses_tensors_that_do_not_fit():
    f, i = torch.zeros((2, 3, 5)), torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        q.q2_0_moe_route(q.Router(5, 2), f[0])
    with pytest.raises(TypeError):
        q.q2_0_moe_route(q.Router(5, 2), None)
    with pytest.raises(ValueError, match="CUDA"):
        q.Router(5, 2, bias=torch.zeros(5))
    with pytest.raises(ValueError, match="CUDA"):
        q.q2_0_draft_verify(f, i, f[:, :, 0])
    with pytest.raises(ValueError, match="tokens"):
        q.q2_0_draft_verify(f, i[0], f[:, :, 0])
    with pytest.raises(TypeError):
        q.q2_0_draft_verify(f, None, f[:, :, 0])
    with pytest.raises(ValueError, match="CUDA"):
        q.KvRows(i[0], i, i[0])
