"""GPU checks of the decode step's cache operators against plain implementations
in 64 bits: q2_0_kv_append, q2_0_attn_plan_*, q2_0_beam_select, q2_0_beam_reorder.

Tolerances. u is the unit roundoff of the cache's type (2^-11 or 2^-8).
  append: one rounding of an f32 result: u |e| + 3 * 2^-24 (|a c| + |b s|), and half
    a spacing of f16's subnormals (2^-25).
  attention: A = sum p|v|. The weights are rounded to the cache's type (u A); a
    score's error ds = 2^-23 (dim + 4) max_t sum |q k| scale (the products' sum, the
    scale) turns into 2 ds A; the sums over the keys are f32 additions, at most one per
    16 keys and 64 more, each 2^-23 A; weights below f16's normal range lose at
    most 2^-32 max|v| each; the output is rounded once, u |out| (f16: + 2^-25).
  selection: score within 2^-22 (|score| + |x| + |lse|) + 2^-20 of the exact one.
Reordering moves values: bit-exact.
"""
import math

import numpy as np
import pytest
import torch

import bit_ternary_matmul_gb300 as q

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    q.build()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    assert q.q2_0_device_check() == q.Q2_0_OK
    q.q2_0_get_error()
    return d


def _no_error():
    assert q.q2_0_get_error() == (0, 0)


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ---- append ----------------------------------------------------------------------
def _rope_table(n_pos, rot, base=1e4):
    f = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n_pos)[:, None] * f
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def _rotated(x, pos, rope, style):
    """(exact in 64 bits, |a c| + |b s|) of x f32 [T][heads][dim]."""
    x = x.double()
    mag = torch.zeros_like(x)
    if rope is None:
        return x, mag
    rot = rope.shape[1]
    h = rot // 2
    i = torch.arange(h, device=x.device)
    ia, ib = (i, i + h) if style == q.Q2_0_ROPE_HALVES else (2 * i, 2 * i + 1)
    cs = rope.double()[pos.long()][:, None]
    c, s = cs[..., :h], cs[..., h:]
    a, b = x[..., ia], x[..., ib]
    y = x.clone()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (a * s).abs() + (b * c).abs()
    return y, mag


def _near(got, exact, mag, dtype, what):
    tol = U[dtype] * exact.abs() * (1 + 2.0 ** -10) + 3 * 2.0 ** -24 * mag + 2.0 ** -25
    bad = (got.double() - exact).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside tolerance"


APPEND = [
    # tokens, seqs, n_q, n_kv, dim, page, rot, style, dtype, layers, fused, odd
    (1, 1, 16, 8, 128, 64, 128, 0, torch.float16, 1, True, 0),
    (8, 8, 16, 8, 128, 16, 128, 0, torch.bfloat16, 2, True, 0),
    (61, 3, 12, 4, 64, 16, 64, 1, torch.float16, 1, False, 0),
    (61, 3, 6, 2, 64, 32, 32, 0, torch.bfloat16, 1, True, 0),
    (33, 5, 5, 1, 128, 256, 48, 1, torch.float16, 3, True, 0),
    (33, 5, 5, 5, 128, 128, 0, 0, torch.float16, 1, True, 0),
    (40, 2, 4, 2, 64, 16, 22, 0, torch.float16, 1, True, 0),   # a rotation in no units of 16
    (40, 2, 4, 2, 64, 16, 2, 1, torch.bfloat16, 1, True, 0),
    (40, 2, 4, 2, 128, 16, 64, 0, torch.float16, 1, True, 1),  # rows off 16-byte alignment
    (40, 2, 4, 2, 128, 16, 64, 1, torch.float16, 1, True, 3),
    (700, 9, 32, 8, 128, 16, 128, 0, torch.float16, 1, False, 0),
    (17, 17, 1, 3, 64, 64, 64, 0, torch.float16, 1, True, 0),
]


@pytest.mark.parametrize("T,S,n_q,n_kv,dim,page,rot,style,dtype,layers,fused,odd", APPEND)
def test_append(T, S, n_q, n_kv, dim, page, rot, style, dtype, layers, fused, odd):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + dim + rot)
    r = np.random.RandomState(T + page)
    layer = layers - 1
    seq = np.sort(r.randint(0, S, T)) if T != S else np.arange(S)
    slot = np.zeros(T, int)
    for b in range(S):
        n = int((seq == b).sum())
        slot[seq == b] = r.randint(0, 2 * page) + np.arange(n)
    width = int(slot.max()) // page + 2
    n_pages = S * width + 2
    table = r.permutation(n_pages)[: S * width].reshape(S, width)
    slot[:: 7] = np.where(np.arange(0, T, 7) % 2 == 1, -1, slot[:: 7])  # some padding
    k_cache = torch.full((layers, n_pages, n_kv, page, dim), 7.0, dtype=dtype, device="cuda")
    v_cache = torch.full_like(k_cache, -3.0)
    cache = q.KvCache(k_cache, v_cache)
    heads = n_q + 2 * n_kv
    if fused:  # slices of one product's rows
        all_ = torch.randn((T, heads * dim + odd), generator=g, device="cuda")
        part = all_[:, odd:].unflatten(1, (heads, dim))
        xq, xk, xv = part[:, :n_q], part[:, n_q: n_q + n_kv], part[:, n_q + n_kv:]
    else:
        xq, xk, xv = (torch.randn((T, h, dim), generator=g, device="cuda") for h in (n_q, n_kv, n_kv))
    n_pos = 5000
    pos = r.randint(0, n_pos, T)
    rope = _rope_table(n_pos, rot) if rot else None
    seq_t = None if T == S else _ints(seq)
    got = q.q2_0_kv_append(cache, layer, xq, xk, xv, _ints(pos) if rot else None, _ints(slot),
                           _ints(table), rope, style=style, seq=seq_t)
    _no_error()
    pos_t = _ints(pos)
    e, mag = _rotated(xq, pos_t, rope, style)
    _near(got, e, mag, dtype, "q")
    e, mag = _rotated(xk, pos_t, rope, style)
    st = np.nonzero(slot >= 0)[0]
    page_of, at = table[seq[st], slot[st] // page], slot[st] % page
    _near(k_cache[layer][page_of, :, at], e[st], mag[st], dtype, "k")
    _near(v_cache[layer][page_of, :, at], xv.double()[st], torch.zeros_like(e[st]), dtype, "v")
    # nothing else was written
    for c, fill in ((k_cache, 7.0), (v_cache, -3.0)):
        rest = c.clone()
        rest[layer][page_of, :, at] = fill
        assert (rest == fill).all()


def test_append_out_of_range_indices_store_nothing():
    T, n_kv, dim, page = 6, 2, 64, 16
    k_cache = torch.full((1, 4, n_kv, page, dim), 5.0, dtype=torch.float16, device="cuda")
    v_cache = torch.full_like(k_cache, 5.0)
    cache = q.KvCache(k_cache, v_cache)
    x = torch.randn((T, n_kv, dim), device="cuda")
    rope = _rope_table(10, dim)
    table = _ints([[0, 1], [2, 9], [-1, 3]])
    ok = dict(pos=[1] * T, slot=[0, 1, 2, 3, 4, 5], seq=[0] * T)
    for name, at, val in (("pos", 3, 10), ("pos", 2, -1), ("slot", 4, 32), ("seq", 5, 3), ("seq", 1, -1),
                          ("seq", 0, 2), ("slot17", 2, 17)):
        a = {k: list(v) for k, v in ok.items()}
        if name == "slot17":
            a["slot"][at], a["seq"][at] = 17, 1  # the table names page 9 of 4
        else:
            a[name][at] = val
        k_cache.fill_(5.0)
        qo = torch.full((T, n_kv, dim), 9.0, dtype=torch.float16, device="cuda")
        q.q2_0_kv_append(cache, 0, x, x, x, _ints(a["pos"]), _ints(a["slot"]), table, rope, seq=_ints(a["seq"]), q_out=qo)
        assert q.q2_0_get_error() == (q.Q2_0_DEVERR_BAD_ID, at), name
        assert (qo[at] == 9.0).all()
        assert int((k_cache != 5.0).any(-1).any(2).sum()) == T - 1  # the other tokens' places
    _no_error()


def test_append_nothing_and_only_keys():
    cache = q.KvCache(*(torch.zeros((1, 2, 1, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2)))
    x = torch.ones((0, 1, 64), device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert q.q2_0_kv_append(cache, 0, None, x, x, None, none, _ints([[0]]), None) is None
    x = torch.ones((1, 1, 64), device="cuda")
    assert q.q2_0_kv_append(cache, 0, None, x, 2 * x, None, _ints([15]), _ints([[1]]), None) is None
    assert (cache.k[0, 1, 0, 15] == 1).all() and (cache.v[0, 1, 0, 15] == 2).all()
    assert float(cache.k.sum()) == 64
    _no_error()


# ---- attention -------------------------------------------------------------------
class Attn:
    """A case's inputs; every place that no sequence owns holds NaN."""

    def __init__(self, plens, lens, n_q, n_kv, dim, page, dtype, seed=0, layers=1, layer=0, qs=1.5, k_of=None,
                 spare=2, scale=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.RandomState(seed)
        self.plens, self.lens, self.layer, self.dtype, self.page = plens, lens, layer, dtype, page
        n, groups = len(lens), len(plens)
        width, pwidth = (max(1, -(-max(x) // page)) + 1 for x in (lens, plens))
        need = sum(-(-x // page) for x in plens + lens)
        ids = r.permutation(need + spare)
        n_pages = need + spare
        shape = (layers, n_pages, n_kv, page, dim)
        self.k = torch.full(shape, math.nan, dtype=dtype, device="cuda")
        self.v = torch.full(shape, math.nan, dtype=dtype, device="cuda")
        self.table = np.full((n, width), -7, np.int32)  # columns past a length are not read
        self.ptable = np.full((groups, pwidth), -7, np.int32)
        at = 0
        self.ks, self.vs = [], []
        for t, ls in ((self.ptable, plens), (self.table, lens)):
            for i, x in enumerate(ls):
                m = -(-x // page)
                t[i, :m] = ids[at: at + m]
                kk = torch.randn((n_kv, x, dim), generator=g, device="cuda")
                if k_of is not None:
                    kk = k_of(kk)
                kk = kk.to(dtype)
                vv = torch.randn((n_kv, x, dim), generator=g, device="cuda").to(dtype)
                for j in range(m):
                    c = min(page, x - j * page)
                    self.k[layer, ids[at + j], :, :c] = kk[:, j * page: j * page + c]
                    self.v[layer, ids[at + j], :, :c] = vv[:, j * page: j * page + c]
                self.ks.append(kk)
                self.vs.append(vv)
                at += m
        self.q = (torch.randn((n, n_q, dim), generator=g, device="cuda") * qs).to(dtype)
        self.out = torch.full_like(self.q, math.nan)
        self.scale = dim ** -0.5 if scale is None else scale
        self.cache = q.KvCache(self.k, self.v)
        self.t_table, self.t_ptable = _ints(self.table), _ints(self.ptable)
        self.t_len, self.t_plen = _ints(lens), _ints(plens)

    def plan(self, shared=True):
        if not shared:
            return q.AttnPlan(self.cache, self.q, self.out, self.t_table, self.t_len, scale=self.scale)
        return q.AttnPlan(self.cache, self.q, self.out, self.t_table, self.t_len, self.t_ptable, self.t_plen,
                          scale=self.scale)

    def exact(self):
        """(out, tolerance) in 64 bits."""
        groups, n = len(self.plens), len(self.lens)
        n_q, dim = self.q.shape[1:]
        n_kv = self.k.shape[2]
        share = n_q // n_kv
        out = torch.zeros((n, n_q, dim), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        u = U[self.dtype]
        for b in range(n):
            gi = b // (n // groups)
            kk = torch.cat([self.ks[gi], self.ks[groups + b]], 1).double()
            vv = torch.cat([self.vs[gi], self.vs[groups + b]], 1).double()
            L = kk.shape[1]
            if L == 0:
                continue
            qq = self.q[b].double().reshape(n_kv, share, dim)
            s = qq @ kk.transpose(1, 2) * self.scale
            p = torch.softmax(s, -1)
            o = p @ vv
            a = p @ vv.abs()
            ds = 2.0 ** -23 * (dim + 4) * abs(self.scale) * (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1, keepdim=True)
            t = a * (u + 2 * ds + 2.0 ** -23 * (L / 16 + 64)) + L * 2.0 ** -32 * vv.abs().amax(1, keepdim=True) \
                + u * o.abs() + 2.0 ** -25
            out[b], tol[b] = o.reshape(n_q, dim), t.reshape(n_q, dim)
        return out, tol

    def check(self, what=""):
        e, tol = self.exact()
        assert torch.isfinite(self.out).all(), f"{what}: not finite"
        bad = (self.out.double() - e).abs() > tol
        assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside tolerance, first at "
                               f"{tuple(bad.nonzero()[0].tolist())}, worst {float(((self.out.double() - e).abs() / tol).max()):.3g} times")


F16, BF16 = torch.float16, torch.bfloat16
ATTN = [
    # prefix lengths, own lengths, n_q, n_kv, dim, page, dtype
    ([0], [1], 1, 1, 64, 16, F16),
    ([0], [1], 16, 8, 128, 64, F16),
    ([1], [0], 16, 8, 128, 64, BF16),
    ([1], [1], 2, 1, 128, 16, F16),
    ([0], [0, 1, 15, 16, 17, 127, 128, 129], 8, 2, 128, 16, F16),
    ([0], [255, 256, 257, 0, 31], 4, 4, 64, 32, BF16),
    ([128], [0], 4, 1, 128, 128, F16),
    ([129], [127, 1], 4, 1, 128, 128, F16),
    ([517], [37, 37, 37, 37], 16, 8, 128, 16, F16),
    ([1000], [5, 0, 300, 64, 1, 200, 77, 128], 32, 8, 128, 64, F16),
    ([999], [10] * 5, 3, 3, 64, 256, BF16),                      # one query head per kv head
    ([333], [0] * 7, 24, 8, 128, 16, F16),                       # three query heads per kv head
    ([64, 0, 257], [3, 4, 0, 0, 200, 130], 6, 2, 64, 16, BF16),  # groups, one without a prefix
    ([0, 0], [0, 0, 0, 0], 4, 2, 128, 16, F16),                  # nothing to attend to
    ([700, 650], [20 + 7 * i for i in range(26)], 10, 2, 64, 32, F16),
    ([1500], [i for i in range(40)], 32, 8, 128, 16, F16),       # 160 rows on a kv head
    ([2100], [(37 * i) % 300 for i in range(70)], 8, 2, 128, 64, BF16),
    ([400], [90, 3, 0], 64, 1, 128, 16, F16),                    # one kv head for all
    ([300], [140, 9], 64, 1, 64, 64, BF16),
    ([70], [5, 6, 7], 60, 20, 64, 16, F16),
    ([5003], [1, 2], 4, 2, 128, 16, BF16),
    ([3], [1] * 200, 8, 4, 64, 16, F16),
    ([9001], [1] * 16, 16, 4, 128, 64, F16),                     # 64 rows, long
    ([5000], [200, 0, 33] * 4, 8, 2, 64, 16, BF16),              # 48 rows
    ([12000], [17] * 12, 8, 2, 128, 128, BF16),
    ([9000, 4100], [i * 50 for i in range(60)], 4, 2, 64, 32, F16),
    ([8000], [130] * 32, 8, 2, 64, 64, F16),                     # 128 rows, narrow heads
    ([20000], [3] * 30, 4, 1, 128, 256, F16),
]


@pytest.mark.parametrize("plens,lens,n_q,n_kv,dim,page,dtype", ATTN)
def test_attention(plens, lens, n_q, n_kv, dim, page, dtype):
    c = Attn(plens, lens, n_q, n_kv, dim, page, dtype, seed=len(lens) * 100 + dim + page)
    plan = c.plan()
    assert plan.launches >= 1
    plan.execute(0)
    _no_error()
    c.check("first")
    first = c.out.clone()
    c.out.fill_(math.nan)
    plan.execute(0)
    assert torch.equal(c.out, first), "the same inputs gave other outputs"
    plan.close()


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (128, F16)])
def test_attention_without_prefix_tables(dim, dtype):
    c = Attn([0], [70, 0, 300], 4, 2, dim, 16, dtype, seed=3)
    plan = c.plan(shared=False)  # kept until it has run
    plan.execute(0)
    _no_error()
    c.check()


def test_attention_scratch_of_an_earlier_plan():
    """Plans made one after another get the same scratch, with the earlier ones' results in it."""
    for i in range(3):
        for plens, lens, n_q, n_kv, dim, page, dtype in ATTN[4::3]:
            c = Attn(plens, lens, n_q, n_kv, dim, page, dtype, seed=i)
            plan = c.plan()
            plan.execute(0)
            _no_error()
            c.check(f"{plens} {len(lens)}")
            plan.close()


@pytest.mark.parametrize("how", ["rising", "falling", "late_peak", "flat", "steep"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_score_ranges(how, dtype):
    """Scores whose maximum keeps moving from tile to tile, or sits in one key."""
    def k_of(k):
        t = torch.arange(k.shape[1], device="cuda")[None, :, None]
        n = max(1, k.shape[1])
        if how == "rising":
            return k * (0.05 + 6.0 * t / n)
        if how == "falling":
            return k * (0.05 + 6.0 * (n - t) / n)
        if how == "late_peak":
            return torch.where(t == n - 3, k * 20, k * 0.1)
        if how == "flat":
            return k * 0
        return k * 12
    c = Attn([1111], [400, 3, 129, 0], 8, 2, 128, 16, dtype, seed=11, k_of=k_of)
    plan = c.plan()
    plan.execute(0)
    _no_error()
    c.check(how)


def test_attention_large_negative_and_zero_scale():
    for scale, k_of in ((0.0, None), (1.0, lambda k: -k.abs() * 30), (-0.3, None)):
        c = Attn([260], [130, 1], 4, 2, 64, 16, F16, seed=5, scale=scale, k_of=k_of)
        if k_of is not None:
            c.q.copy_(c.q.abs())
        plan = c.plan()
        plan.execute(0)
        _no_error()
        c.check(f"scale {scale}")


RAISES = [
    # prefix lengths, own lengths, n_q, n_kv, dim, dtype: variants by the query rows of a product; 300 runs of
    # tiles or more, so that a block's share of the tiles holds whole ones
    ([0], [260 + i for i in range(100)], 16, 4, 128, F16),                # own tokens, 4 rows
    ([0], [300 + 3 * i for i in range(90)], 4, 4, 64, BF16),              # own tokens, 1 row
    ([0], [290 + i for i in range(160)], 128, 2, 128, F16),               # own tokens, 64 rows
    ([0], [390 + i for i in range(160)], 96, 2, 64, BF16),                # own tokens, 48 rows
    ([300 + 9 * i for i in range(40)], [0] * 400, 16, 8, 128, F16),       # prefixes of 20 rows
    ([300 + 9 * i for i in range(40)], [3] * 480, 32, 8, 64, F16),        # prefixes of 48 rows
    ([385] * 40, [1] * 640, 32, 8, 128, BF16),                            # prefixes of 64 rows
]


@pytest.mark.parametrize("plens,lens,n_q,n_kv,dim,dtype", RAISES)
def test_attention_references_rise_to_the_last_tile(plens, lens, n_q, n_kv, dim, dtype):
    """Every tile of 128 keys raises every reference, a segment's last one too: outputs and sums so far are
    scaled down by the tile's factors and by nothing else."""
    def k_of(k):  # scores rise by 12 or more (log2 units) from tile to tile
        t = torch.arange(k.shape[1], device="cuda")[None, :, None]
        return torch.full_like(k, dim ** -0.5) * (10.0 * (t // 128) + 1) + 0.02 * k
    c = Attn(plens, lens, n_q, n_kv, dim, 64, dtype, seed=31, k_of=k_of)
    c.q.copy_(torch.ones_like(c.q) + 0.02 * c.q)
    plan = c.plan()
    plan.execute(0)
    _no_error()
    c.check("rising")
    first = c.out.clone()
    for _ in range(20):
        plan.execute(0)
        assert torch.equal(c.out, first), "the same inputs gave other outputs"


HUGE = [
    ([0], [1, 129, 300, 700], 8, 2, 128, F16), ([400], [1, 129, 0, 200], 8, 2, 64, BF16),
    ([0], [300, 500], 64, 1, 64, F16), ([400], [5] * 12, 8, 2, 128, BF16), ([400], [140, 0, 5] * 10, 8, 2, 128, F16),
    ([400], [140, 0] * 40, 8, 2, 64, BF16)]


@pytest.mark.parametrize("size", [26, 29, 33])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("plens,lens,n_q,n_kv,dim,dtype", HUGE)
def test_attention_huge_finite_scores(plens, lens, n_q, n_kv, dim, dtype, sign, size):
    """Scores of about +-2^size (log2 units) in which one key is ahead by far: the output is its value. The
    weight and the output are rounded to the cache's type once each: 2 u |v|."""
    _one_key_ahead(plens, lens, n_q, n_kv, dim, dtype, sign, size)


def _one_key_ahead(plens, lens, n_q, n_kv, dim, dtype, sign, size):
    c_k = 1.37 * 2.0 ** ((size + 2.97 - math.log2(dim)) / 2)   # of elements: dim c_k^2 / sqrt(dim) is the score's size
    groups, calls, win = len(plens), [], []

    def k_of(k):
        g = torch.Generator(device="cuda").manual_seed(len(calls))
        n = k.shape[1]
        m = 0.3 + 0.3 * torch.rand((k.shape[0], n, 1), generator=g, device="cuda")
        best = 0.8 if len(calls) < groups else 0.9     # a sequence's own winner is ahead of its prefix's
        if sign < 0:
            m, best = 1.3 - m, 1 - best
        calls.append(n)
        win.append((7 * len(calls) + n // 2) % max(1, n))
        if n:
            m[:, win[-1]] = best
        return m.expand_as(k) * (sign * c_k)
    c = Attn(plens, lens, n_q, n_kv, dim, 16, dtype, seed=17, k_of=k_of)
    c.q.fill_(c_k)
    plan = c.plan()
    plan.execute(0)
    _no_error()
    share = n_q // n_kv
    for b, n in enumerate(lens):
        i = groups + b if n else b // (len(lens) // groups)
        if calls[i]:
            e = c.vs[i][:, win[i]].double().repeat_interleave(share, 0)
            tol = 2 * U[dtype] * (1 + 2.0 ** -8) * e.abs() + 2.0 ** -25
            assert ((c.out[b].double() - e).abs() <= tol).all(), (b, n)


@pytest.mark.parametrize("plens,lens,n_q,n_kv,dim,dtype", [h for h in HUGE if h[-1] is BF16])
def test_attention_scores_near_the_largest_float(plens, lens, n_q, n_kv, dim, dtype):
    for sign in (1, -1):
        _one_key_ahead(plens, lens, n_q, n_kv, dim, dtype, sign, 119)


@pytest.mark.parametrize("plens,lens,n_q,n_kv", [([0], [128] * 3, 8, 2), ([0], [128] * 2, 64, 1), ([128], [0] * 40, 8, 2)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_small_weights_behind_a_sink(plens, lens, n_q, n_kv, dtype):
    """One key takes nearly all the weight and has no value; the others lie 2^-24.349 below it. F16 weights this
    small have a fixed spacing: in it theirs is 100.49, so that rounding moves them all by 0.49 of it. The bound is
    the declared one: u (sum p|v| + |out|), F16: 2^-32 sum |v| more, and f32 rounding."""
    c = Attn(plens, lens, n_q, n_kv, 64, 64, dtype, seed=23, scale=24.349 * math.log(2), k_of=lambda k: k * 0)
    c.q.zero_()
    c.q[..., 0] = 1
    c.v.mul_(1000)
    rows = [(c.ptable[0], plens[0], 0)] + [(c.table[b], n, 1 + b) for b, n in enumerate(lens)]
    for row, n, i in rows:
        if n:
            c.vs[i] = c.vs[i] * 1000
            c.vs[i][:, 0] = 0
            c.ks[i][:, 0, 0] = 1
            c.k[0, int(row[0]), :, 0, 0] = 1
            c.v[0, int(row[0]), :, 0] = 0
    plan = c.plan()
    plan.execute(0)
    _no_error()
    u, worst = U[dtype], 0.0
    for b, n in enumerate(lens):
        i = 1 + b if n else 0
        s = c.ks[i][:, :, 0].double() * c.scale
        p, v = torch.softmax(s, -1), c.vs[i].double()
        e, a = (torch.einsum("ht,htd->hd", p, x).repeat_interleave(n_q // n_kv, 0) for x in (v, v.abs()))
        err = (c.out[b].double() - e).abs()
        # f32: the scores' one product and its scaling (2^-23 of 24.4, as in the head of this file), 64 additions
        plain = u * (1 + 2.0 ** -8) * (a + e.abs()) + 2.0 ** -23 * (2 * 3 * 17 + 64) * a + 2.0 ** -25
        more = 2.0 ** -32 * v.abs().sum(1).repeat_interleave(n_q // n_kv, 0) if dtype is F16 else 0.0
        assert (err <= plain + more).all()
        worst = max(worst, float((err / plain).max()))
    assert dtype is BF16 or worst > 1, "the small weights' own term is not needed"


def test_attention_layers_and_streams():
    c = Attn([300], [40, 50], 8, 4, 64, 32, F16, seed=6, layers=3, layer=2)
    plan = c.plan()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan.execute(2, stream=s)
    s.synchronize()
    _no_error()
    c.check("layer 2 on a side stream")


def test_attention_in_a_graph_follows_the_lengths():
    c = Attn([200], [128, 128], 8, 2, 128, 16, F16, seed=7)
    plan = c.plan()
    plan.execute(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.execute(0)
    full = c.ks, c.vs
    for plen, lens in ((200, [128, 128]), (77, [1, 64]), (0, [17, 0]), (160, [0, 0])):
        c.t_plen.copy_(_ints([plen]))
        c.t_len.copy_(_ints(lens))
        c.plens, c.lens = [plen], lens
        c.ks = [full[0][0][:, :plen]] + [full[0][1 + i][:, :n] for i, n in enumerate(lens)]
        c.vs = [full[1][0][:, :plen]] + [full[1][1 + i][:, :n] for i, n in enumerate(lens)]
        c.out.fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        _no_error()
        c.check(str(lens))


def test_attention_bad_lengths_and_pages_are_reported():
    c = Attn([64], [32, 32, 32], 4, 2, 64, 16, F16, seed=8)
    # finite everywhere: page 0 stands in for a bad one
    c.k.nan_to_num_()
    c.v.nan_to_num_()
    plan = c.plan()
    good = (c.t_len.clone(), c.t_plen.clone(), c.t_table.clone(), c.t_ptable.clone())
    for i, (t, at, val, info) in enumerate(((c.t_len, (1,), -1, 1), (c.t_len, (2,), 1 << 20, 2), (c.t_plen, (0,), -5, 3),
                                            (c.t_table, (0, 1), 10 ** 6, 0), (c.t_ptable, (0, 2), -1, 3))):
        for a, b in zip((c.t_len, c.t_plen, c.t_table, c.t_ptable), good):
            a.copy_(b)
        if val == 1 << 20:  # the length is cut to the row: give the row pages
            c.t_table[2] = 0
        t[at] = val
        plan.execute(0)
        assert q.q2_0_get_error() == (q.Q2_0_DEVERR_BAD_ID, info), i
    for a, b in zip((c.t_len, c.t_plen, c.t_table, c.t_ptable), good):
        a.copy_(b)
    plan.execute(0)
    _no_error()
    c.check("after the errors")


# ---- selection -------------------------------------------------------------------
def _select_ref(logits, scores, done, done_token, n_out):
    """(score, parent, token) from the definition, in 64 bits; equal logits and equal scores tie."""
    G, W, V = logits.shape
    out = []
    for g in range(G):
        cands = []
        for b in range(W):
            s0 = float(scores[g, b])
            if done is not None and done[g, b]:
                if s0 > -math.inf:
                    cands.append((-s0, b, 0.0, 0, done_token))
                continue
            x = logits[g, b].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
            ok = np.nonzero(x > -np.inf)[0]
            if not len(ok) or not s0 > -math.inf:
                continue
            m = x[ok].max()
            lse = m + math.log(np.exp(x[ok] - m).sum())
            best = ok[np.lexsort((ok, -x[ok]))][:n_out]
            cands += [(-(s0 + (x[t] - lse)), b, -x[t], t, t) for t in best]
        cands.sort()
        rows = [(-c[0], c[1], c[4]) for c in cands[:n_out]]
        out.append(rows + [(-math.inf, 0, -1)] * (n_out - len(rows)))
    a = np.array(out, dtype=np.float64)
    return a[..., 0], a[..., 1].astype(np.int64), a[..., 2].astype(np.int64)


def _check_select(logits, scores, n_out, done=None, done_token=2, what=""):
    lt = torch.from_numpy(logits).cuda()
    s, p, t = q.q2_0_beam_select(lt, torch.from_numpy(scores).cuda(), n_out,
                                 done=None if done is None else torch.from_numpy(done).cuda(), done_token=done_token)
    _no_error()
    rs, rp, rt = _select_ref(logits, scores, done, done_token, n_out)
    s, p, t = s.cpu().numpy().astype(np.float64), p.cpu().numpy(), t.cpu().numpy()
    assert np.array_equal(p, rp) and np.array_equal(t, rt), f"{what}: {p} {rp} {t} {rt}"
    fin = np.isfinite(rs)
    assert np.array_equal(fin, np.isfinite(s))
    mag = np.abs(rs[fin]) + (np.abs(logits[np.isfinite(logits)].astype(np.float64)).max() if np.isfinite(logits).any() else 0) * 2 + 14
    assert (np.abs(s[fin] - rs[fin]) <= 2.0 ** -22 * mag + 2.0 ** -20).all(), what


@pytest.mark.parametrize("G,W,V,n_out", [(1, 1, 1, 1), (1, 1, 5, 3), (1, 4, 151936, 4), (3, 5, 32003, 10), (2, 8, 4096, 8),
                                         (2, 3, 4097, 32), (7, 2, 4095, 1), (1, 64, 1001, 32), (4, 16, 333, 31),
                                         (2, 2, 12289, 17)])
def test_select(G, W, V, n_out):
    r = np.random.RandomState(V + W)
    logits = (r.standard_normal((G, W, V)) * 3).astype(np.float32)
    scores = (-r.random((G, W)) * 9).astype(np.float32)
    _check_select(logits, scores, n_out, what="plain")
    done = (r.random((G, W)) < 0.4).astype(np.uint8)
    logits[:, :, r.random(V) < 0.1] = -np.inf
    _check_select(logits, scores, n_out, done=done, what="banned and done")


def test_select_ties_go_to_the_lowest():
    # equal logits everywhere: more survivors than are kept in shared memory
    for V in (3, 64, 5000, 20000):
        logits = np.zeros((2, 3, V), np.float32)
        scores = np.array([[0, -1, -2], [-7, -7.5, -7.25]], np.float32)
        _check_select(logits, scores, 8, what=str(V))
    # a few values many times over; rows of a multiple of 4 tokens are summed alike, so equal rows tie exactly
    r = np.random.RandomState(1)
    logits = r.randint(0, 4, (1, 4, 8192)).astype(np.float32)
    logits[0, 2] = logits[0, 1]
    logits[0, 3] = -logits[0, 3] * 0.0  # zeros of both signs
    _check_select(logits, np.array([[-1, -0.5, -0.5, -30]], np.float32), 32)
    logits = np.zeros((1, 2, 400), np.float32)
    logits[0, 0, 100:120] = -0.0
    _check_select(logits, np.zeros((1, 2), np.float32), 32)


def test_select_masks_and_odd_values():
    r = np.random.RandomState(2)
    V = 9001
    base = (r.standard_normal((1, 4, V)) * 2).astype(np.float32)
    none = base.copy()
    none[0, 1] = -np.inf                       # a row whose mask leaves nothing
    _check_select(none, np.full((1, 4), -1, np.float32), 6, what="empty row")
    none[:] = -np.inf
    _check_select(none, np.zeros((1, 4), np.float32), 6, what="all empty")
    few = np.full((1, 4, V), -np.inf, np.float32)
    few[0, 2, 8999], few[0, 0, 3], few[0, 0, 4100] = 1.5, -2, 0.25
    _check_select(few, np.array([[-3, 0, -1, 0]], np.float32), 6, what="few")
    low = np.full((1, 2, V), np.finfo(np.float32).min, np.float32)   # the type's lowest value is a value
    low[0, 0, 77] = 3
    _check_select(low[:, :1], np.zeros((1, 1), np.float32), 3, what="lowest")
    _check_select(low, np.zeros((1, 2), np.float32), 4, what="lowest alone")
    nan = base.copy()
    nan[0, 0, ::3] = np.nan
    _check_select(nan, np.zeros((1, 4), np.float32), 6, what="nan")
    inf = base.copy()
    inf[0, 3, 55] = np.inf
    _check_select(inf, np.array([[0, 0, 0, -0.5]], np.float32), 4, what="inf")
    first = base.copy()                        # a search's first step: one beam alive
    _check_select(first, np.array([[0, -np.inf, -np.inf, np.nan]], np.float32), 4, what="first step")
    wide = base * 1000
    _check_select(wide, np.zeros((1, 4), np.float32), 4, what="wide")


def test_select_many_rows_of_odd_shapes():
    """Enough rows for the long pieces: sorted both ways, masked ranges, plateaus, one value far out."""
    r = np.random.RandomState(5)
    G, W, V = 5, 16, 151937
    logits = (r.standard_normal((G, W, V)) * 2).astype(np.float32)
    logits[0, :4] = np.sort(logits[0, :4], axis=-1)
    logits[0, 4:8] = np.sort(logits[0, 4:8], axis=-1)[..., ::-1]
    logits[1, :, : 140000] = -np.inf
    logits[1, 3, 140000:] = -np.inf
    logits[2, 0] = np.float32(0.5)
    logits[2, 1:8] = np.round(logits[2, 1:8] / 4)
    logits[2, 8, 100001] = 300.0
    logits[2, 9, 100003] = 3e38
    logits[2, 10] = np.finfo(np.float32).min
    logits[2, 11, ::2] = np.finfo(np.float32).min
    logits[3, :, ::5] = np.nan
    scores = (-r.random((G, W)) * 3).astype(np.float32)
    scores[2, 9:11] = -40
    _check_select(logits, scores, 16, what="shapes")
    _check_select(logits, scores, 32, what="shapes, 32")


def test_select_strided_rows_workspace_and_outputs():
    r = np.random.RandomState(3)
    G, W, V = 2, 3, 1003
    wide = torch.from_numpy((r.standard_normal((G * W, 1024)) * 3).astype(np.float32)).cuda()
    rows = wide[:, 5: 5 + V].unflatten(0, (G, W))
    scores = torch.from_numpy((-r.random((G, W))).astype(np.float32)).cuda()
    a = q.q2_0_beam_select(rows, scores, 6)
    b = q.q2_0_beam_select(rows.contiguous(), scores, 6)
    need = q.q2_0_beam_select_workspace_size(G, W, V, 6)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = (torch.empty((G, 6), device="cuda"),) + tuple(torch.empty((G, 6), dtype=torch.int32, device="cuda") for _ in range(2))
    c = q.q2_0_beam_select(rows, scores, 6, workspace=ws, out=out)
    assert c[0] is out[0]
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    for x, y in zip(a, c):
        assert torch.equal(x, y)
    rs, rp, rt = _select_ref(rows.cpu().numpy(), scores.cpu().numpy(), None, 0, 6)
    assert np.array_equal(a[1].cpu().numpy(), rp) and np.array_equal(a[2].cpu().numpy(), rt)
    e = q.q2_0_beam_select(torch.empty((0, 3, 50), device="cuda"), torch.empty((0, 3), device="cuda"), 2)
    assert e[0].shape == (0, 2)
    _no_error()


# ---- reordering ------------------------------------------------------------------
def _reorder_ref(parent, table, length, fresh, page, k, v):
    G, W = parent.shape
    t, n, u = np.empty_like(table), np.empty_like(length), np.zeros(len(length), np.int32)
    k, v = k.clone(), v.clone()
    src_k, src_v = k.clone(), v.clone()
    for g in range(G):
        seen = set()
        for j in range(W):
            p, i = g * W + parent[g, j], g * W + j
            t[i], n[i] = table[p], length[p]
            last, fill = divmod(int(length[p]), page)
            if fill and parent[g, j] in seen:
                k[:, fresh[i], :, :fill] = src_k[:, table[p, last], :, :fill]
                v[:, fresh[i], :, :fill] = src_v[:, table[p, last], :, :fill]
                t[i, last], u[i] = fresh[i], 1
            elif not fill and last < table.shape[1]:
                t[i, last], u[i] = fresh[i], 1
            seen.add(parent[g, j])
    return t, n, u, k, v


@pytest.mark.parametrize("G,W,layers,n_kv,dim,page,dtype,lens", [
    (1, 1, 1, 1, 64, 16, F16, [0]), (1, 8, 3, 2, 128, 16, F16, [37]), (2, 4, 2, 3, 64, 32, BF16, [32, 95]),
    (3, 5, 1, 1, 128, 256, F16, [0, 1, 255]), (4, 2, 5, 8, 64, 16, F16, [15, 16, 17, 48]),
    (1, 300, 1, 1, 64, 16, BF16, [9])])
def test_reorder(G, W, layers, n_kv, dim, page, dtype, lens):
    r = np.random.RandomState(G * 10 + W)
    n = G * W
    width = max(lens) // page + 1
    n_pages = n * (width + 1)
    ids = r.permutation(n_pages).astype(np.int32)
    table, fresh = ids[: n * width].reshape(n, width), ids[n * width:]
    length = np.repeat(np.array(lens, np.int32), W)
    if W == 4:
        length = length + np.tile(np.array([0, -1, -2, -32], np.int32), G)  # beams of different lengths
    parent = r.randint(0, W, (G, W)).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(9)
    k = torch.randn((layers, n_pages, n_kv, page, dim), generator=g, device="cuda").to(dtype)
    v = torch.randn((layers, n_pages, n_kv, page, dim), generator=g, device="cuda").to(dtype)
    rt, rn, ru, rk, rv = _reorder_ref(parent, table, length, fresh, page, k, v)
    t, ln, u = q.q2_0_beam_reorder(q.KvCache(k, v), _ints(parent), _ints(table), _ints(length), _ints(fresh))
    _no_error()
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(ln.cpu().numpy(), rn)
    assert np.array_equal(u.cpu().numpy(), ru)
    assert torch.equal(k, rk) and torch.equal(v, rv)


def test_reorder_full_rows_and_bad_indices():
    page = 16
    k = torch.randn((2, 12, 1, page, 64), device="cuda").half()
    v = torch.randn((2, 12, 1, page, 64), device="cuda").half()
    cache, k0 = q.KvCache(k, v), k.clone()
    table = np.arange(8, dtype=np.int32).reshape(4, 2)
    # a full row has no column for a next page
    t, n, u = q.q2_0_beam_reorder(cache, _ints([[1, 1, 0, 3]]), _ints(table), _ints([32] * 4), _ints([8, 9, 10, 11]))
    assert np.array_equal(t.cpu().numpy(), table[[1, 1, 0, 3]]) and int(u.sum()) == 0
    _no_error()
    for parent, length, fresh, bad in (([1, 4, 0, 0], [20] * 4, [8, 9, 10, 11], 1), ([1, -1, 0, 2], [20] * 4, [8, 9, 10, 11], 1),
                                       ([1, 0, 2, 3], [20, 20, 33, 20], [8, 9, 10, 11], 2),
                                       ([1, 0, 2, 3], [20, 20, 20, -1], [8, 9, 10, 11], 3),
                                       ([1, 0, 0, 3], [20] * 4, [8, 9, 12, 11], 2)):
        out = (torch.full((4, 2), -5, dtype=torch.int32, device="cuda"),) + tuple(
            torch.full((4,), -5, dtype=torch.int32, device="cuda") for _ in range(2))
        q.q2_0_beam_reorder(cache, _ints([parent]), _ints(table), _ints(length), _ints(fresh), out=out)
        assert q.q2_0_get_error() == (q.Q2_0_DEVERR_BAD_ID, bad)
        assert (out[0][bad] == -5).all() and int(out[1][bad]) == -5 and int(out[2][bad]) == -5
        assert int((out[1] == -5).sum()) == 1
    rest = [i for i in range(12) if i != 11]  # 11: the fourth beam's copy of the first case
    assert torch.equal(k[:, rest], k0[:, rest])
    e = q.q2_0_beam_reorder(cache, torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                            torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                            torch.empty(0, dtype=torch.int32, device="cuda"))
    assert e[0].shape == (0, 2)
    _no_error()


@pytest.mark.parametrize("n_seq", [1, 65])
def test_attention_lengths_up_to_32_bits(n_seq):
    """The longest row that a plan takes, 2^31 - 32 tokens, as a sequence of its own or a prefix: its one page
    over and over, but for the last place. Equal weights give the mean, a large last score the last value."""
    width, page = (1 << 27) - 2, 16
    k = torch.zeros((1, 2, 1, page, 64), dtype=F16, device="cuda")
    v = torch.ones_like(k)
    v[0, 1, 0, 15] = torch.arange(64, device="cuda") - 20.0
    k[0, 1, 0, 15, 0] = 40 * 8                      # a score of 40: e^40 is 10^8 times the other weights' sum
    long = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    long[0, -1] = 1
    short = torch.zeros((n_seq, 1), dtype=torch.int32, device="cuda")
    n, none = _ints([width * page]), _ints([0] * n_seq)
    qq = torch.zeros((n_seq, 1, 64), dtype=F16, device="cuda")
    out = torch.full_like(qq, math.nan)
    cache = q.KvCache(k, v)
    plan = q.AttnPlan(cache, qq, out, short, none, long, n) if n_seq > 1 else q.AttnPlan(cache, qq, out, long, n)
    plan.execute(0)
    _no_error()
    assert ((out - 1).abs() <= 2.0 ** -10).all()
    qq[..., 0] = 1
    plan.execute(0)
    _no_error()
    e = v[0, 1, 0, 15].double()
    assert ((out.double() - e).abs() <= 2.0 ** -10 * e.abs() + 2.0 ** -20).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: its last pages are appended to, attended over and copied."""
    n_kv, page, dim = 8, 256, 128
    n_pages = (1 << 32) // (n_kv * page * dim) + 40
    k = torch.empty((1, n_pages, n_kv, page, dim), dtype=F16, device="cuda")
    v = torch.empty((1, n_pages, n_kv, page, dim), dtype=F16, device="cuda")
    cache = q.KvCache(k, v)
    last = n_pages - 1
    T = 300
    g = torch.Generator(device="cuda").manual_seed(4)
    xq, xk, xv = (torch.randn((T, h, dim), generator=g, device="cuda") for h in (16, n_kv, n_kv))
    table = _ints([[last, last - 1, 0]])
    seq = torch.zeros(T, dtype=torch.int32, device="cuda")
    qr = q.q2_0_kv_append(cache, 0, xq, xk, xv, None, _ints(np.arange(T)), table, None, seq=seq)
    assert torch.equal(k[0, last], xk[:256].half().transpose(0, 1))
    assert torch.equal(v[0, last - 1, :, :44], xv[256:].half().transpose(0, 1))
    out = torch.empty_like(qr[:1])
    plan = q.AttnPlan(cache, qr[:1], out, table, _ints([T]))
    plan.execute(0)
    kk, vv = xk.half().double().transpose(0, 1), xv.half().double().transpose(0, 1)
    s = qr[0].double().reshape(n_kv, 2, dim) @ kk.transpose(1, 2) * dim ** -0.5
    e = (torch.softmax(s, -1) @ vv).reshape(16, dim)
    a = (torch.softmax(s, -1) @ vv.abs()).reshape(16, dim)
    ds = 2.0 ** -23 * (dim + 4) * 40.0  # max sum |q k| scale is below 40 for these inputs
    assert ((out[0].double() - e).abs() <= a * (2.0 ** -11 + 2 * ds + 1e-5) + 2.0 ** -11 * e.abs() + 2.0 ** -25).all()
    t, n, u = q.q2_0_beam_reorder(cache, _ints([[0, 0]]), _ints([[last, last - 1, 0]] * 2), _ints([T, T]), _ints([5, last - 2]))
    assert u.tolist() == [0, 1] and t.tolist() == [[last, last - 1, 0], [last, last - 2, 0]]
    assert torch.equal(k[0, last - 2, :, :44], k[0, last - 1, :, :44])
    assert torch.equal(v[0, last - 2, :, :44], v[0, last - 1, :, :44])
    _no_error()
