"""The operators of a decode step on a paged key/value cache, as cases that can be timed and compared.

Four operators: appending keys and values with the position rotation ("append"), attention of sequences that share a
prefix ("attn"), the selection step of a beam search ("select") and the reordering of the beams' page tables ("reorder").
`run` computes them with elementary torch operations in 32 bits, or, where `own` is true, by the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------------
def listed():
    return [
        # eight beams (the most columns of the decode mat-vec) take one token each, 1.7B-class heads: latency
        dict(name="append_step", op="append", tokens=8, seqs=8, n_q=16, n_kv=8, dim=128, page=64, rot=128, pairs=False,
             dtype="f16", start=200),
        # several ragged prompts stored at once in short pages, narrow heads, half of each head rotated in pairs
        dict(name="append_ragged", op="append", tokens=1003, seqs=7, n_q=12, n_kv=4, dim=64, page=16, rot=32, pairs=True,
             dtype="bf16", start=5),
        # a long prompt, 8B-class heads
        dict(name="append_prompt", op="append", tokens=16384, seqs=2, n_q=32, n_kv=8, dim=128, page=16, rot=128,
             pairs=False, dtype="bf16", start=0),
        # four beams a few tokens after a short prompt: latency
        dict(name="attn_beam4", op="attn", groups=1, seqs=4, n_q=16, n_kv=8, dim=128, page=16, dtype="f16", prefix=517,
             suffix=37, even=True),
        # eight beams far behind a long document, 8B-class heads
        dict(name="attn_beam8_long", op="attn", groups=1, seqs=8, n_q=32, n_kv=8, dim=128, page=64, dtype="f16",
             prefix=50021, suffix=200, even=True),
        # a server: four system prompts, sixteen users on each at different lengths; narrow heads, no sharing of kv heads
        dict(name="attn_serve", op="attn", groups=4, seqs=16, n_q=16, n_kv=16, dim=64, page=16, dtype="bf16", prefix=4099,
             suffix=1500, even=False),
        # many users on one very long prompt, 8B-class heads
        dict(name="attn_serve_long", op="attn", groups=1, seqs=64, n_q=32, n_kv=8, dim=128, page=128, dtype="bf16",
             prefix=131072, suffix=3000, even=False),
        # one request of four beams over the head's vocabulary: latency
        dict(name="select_beam4", op="select", groups=1, beams=4, vocab=151936, n_out=4, done=0),
        # odd small vocabulary, twice as many candidates as beams, some beams finished
        dict(name="select_small", op="select", groups=6, beams=5, vocab=32003, n_out=10, done=4),
        # a batch of requests, eight beams each
        dict(name="select_batch", op="select", groups=32, beams=8, vocab=151936, n_out=8, done=20),
        # eight beams of one request, 1.7B-class layers and heads
        dict(name="reorder_beam8", op="reorder", groups=1, beams=8, layers=28, n_kv=8, dim=128, page=16, dtype="f16",
             length=137),
        # a batch of requests, 8B-class layers, longer pages
        dict(name="reorder_batch", op="reorder", groups=16, beams=8, layers=36, n_kv=8, dim=128, page=64, dtype="bf16",
             length=450),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges; no case costs more than the largest listed one of its operator."""
    op = rng.choice(["append", "attn", "attn", "select", "reorder"])
    n_kv = rng.choice([1, 2, 4, 8, 16])
    share = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    if op == "append":
        most = 16384 * 48 * 128 // ((share + 2) * n_kv * dim)
        tokens = _log_int(rng, 1, min(16384, most))
        return dict(op=op, tokens=tokens, seqs=min(tokens, _log_int(rng, 1, 64)), n_q=n_kv * share, n_kv=n_kv, dim=dim,
                    page=page, rot=rng.choice([dim, dim // 2, 0]), pairs=rng.random() < 0.5, dtype=dtype,
                    start=rng.randrange(0, 300))
    if op == "attn":
        groups = rng.choice([1, 1, 2, 4])
        seqs = _log_int(rng, 1, 64)
        # no more cached bytes and no more products than the largest listed case
        kv = 320000 * 8 * 128 // (n_kv * dim)
        prefix = min(_log_int(rng, 100, 131072), kv // (2 * groups), 131072 * 64 * 32 * 128 // (groups * seqs * n_kv * share * dim))
        if rng.random() < 0.1:
            prefix = 0
        suffix = max(1, min(_log_int(rng, 1, 3000), kv // (2 * groups * seqs)))
        return dict(op=op, groups=groups, seqs=seqs, n_q=n_kv * share, n_kv=n_kv, dim=dim, page=page, dtype=dtype,
                    prefix=prefix, suffix=suffix, even=rng.random() < 0.5)
    if op == "select":
        beams = _log_int(rng, 1, 16)
        vocab = _log_int(rng, 1000, 151936)
        groups = max(1, min(_log_int(rng, 1, 64), 32 * 8 * 151936 // (beams * vocab)))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, n_out=beams * rng.choice([1, 2]),
                    done=rng.randrange(0, max(1, groups * beams // 3)))
    beams = _log_int(rng, 2, 16)
    layers = rng.choice([1, 12, 28, 36])
    groups = max(1, min(_log_int(rng, 1, 32), 16 * 8 * 36 * 8 * 128 * 64 // (beams * layers * n_kv * dim * page)))
    return dict(op=op, groups=groups, beams=beams, layers=layers, n_kv=n_kv, dim=dim, page=page, dtype=dtype,
                length=_log_int(rng, 1, 1000))


def _lens(case):
    """The sequences' own lengths: part of the case, not of the seed."""
    n = case["groups"] * case["seqs"]
    if case["even"]:
        return [case["suffix"]] * n
    r = random.Random(case["suffix"] * 1000003 + n)
    return [r.randint(0, case["suffix"]) for _ in range(n)]


def _prefix_lens(case):
    """The groups' prefixes: the first is the longest."""
    return [case["prefix"] - (case["prefix"] * g) // (3 * case["groups"]) for g in range(case["groups"])]


def _append_rows(case):
    """(sequence, place in it) of each token: the tokens split as evenly as they go, in order."""
    t, s = case["tokens"], case["seqs"]
    seq = [i * s // t for i in range(t)]
    first = {}
    for i, b in enumerate(seq):
        first.setdefault(b, i)
    return seq, [case["start"] + 3 * b + i - first[b] for i, b in enumerate(seq)]


# ---- inputs ----------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 31))
    state = {"append": _prepare_append, "attn": _prepare_attn, "select": _prepare_select,
             "reorder": _prepare_reorder}[case["op"]](case, g, r)
    return {"case": case, **state}


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _lib():
    import bit_ternary_matmul_gb300 as q
    return q


def _cache(case, g, layers, n_pages):
    """Keys have a few large channels, as trained ones do."""
    shape = (layers, n_pages, case["n_kv"], case["page"], case["dim"])
    dt = DTYPES[case["dtype"]]
    wide = torch.ones(case["dim"], device="cuda")
    wide[:4] = 3.0
    k = torch.empty(shape, dtype=dt, device="cuda")
    v = torch.empty(shape, dtype=dt, device="cuda")
    for i in range(layers):
        k[i] = (torch.randn(shape[1:], generator=g, device="cuda") * wide).to(dt)
        v[i] = torch.randn(shape[1:], generator=g, device="cuda").to(dt)
    return k, v


def _prepare_append(case, g, r):
    seq, slot = _append_rows(case)
    page = case["page"]
    width = (max(slot) + 1 + page - 1) // page + 1
    n_pages = case["seqs"] * width + 3
    table = r.permutation(n_pages)[: case["seqs"] * width].reshape(case["seqs"], width)
    dt = DTYPES[case["dtype"]]
    shape = (1, n_pages, case["n_kv"], page, case["dim"])
    k_cache, v_cache = torch.zeros(shape, dtype=dt, device="cuda"), torch.zeros(shape, dtype=dt, device="cuda")
    heads = case["n_q"] + 2 * case["n_kv"]
    # the three projections' outputs side by side, as one product over the stacked weights leaves them
    qkv = torch.randn((case["tokens"], heads, case["dim"]), generator=g, device="cuda")
    pos = np.asarray(slot) + 1000  # behind a shared prefix
    rope = None
    if case["rot"]:
        f = 1e6 ** (-np.arange(0, case["rot"], 2) / case["rot"])
        a = np.arange(int(pos.max()) + 1)[:, None] * f
        rope = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    state = dict(q=qkv[:, : case["n_q"]], k=qkv[:, case["n_q"]: case["n_q"] + case["n_kv"]],
                 v=qkv[:, case["n_q"] + case["n_kv"]:], k_cache=k_cache, v_cache=v_cache, table=_ints(table),
                 seq=_ints(seq), slot=_ints(slot), pos=_ints(pos), rope=rope,
                 q_out=torch.empty((case["tokens"], case["n_q"], case["dim"]), dtype=dt, device="cuda"))
    if own:
        state["cache"] = _lib().KvCache(k_cache, v_cache)
    return state


def _prepare_attn(case, g, r):
    page, lens, plens = case["page"], _lens(case), _prefix_lens(case)
    n = len(lens)
    width = max(1, -(-max(lens) // page))
    pwidth = max(1, -(-max(plens) // page))
    need = sum(-(-x // page) for x in lens + plens) + 1
    ids = r.permutation(need)
    table, ptable = np.zeros((n, width), np.int32), np.zeros((case["groups"], pwidth), np.int32)
    at = 0
    for t, ls in ((ptable, plens), (table, lens)):
        for i, x in enumerate(ls):
            m = -(-x // page)
            t[i, :m] = ids[at: at + m]
            at += m
    k, v = _cache(case, g, 1, need)
    dt = DTYPES[case["dtype"]]
    q = (torch.randn((n, case["n_q"], case["dim"]), generator=g, device="cuda") * 1.5).to(dt)
    state = dict(q=q, k_cache=k, v_cache=v, table=_ints(table), length=_ints(lens), prefix_table=_ints(ptable),
                 prefix_len=_ints(plens), scale=case["dim"] ** -0.5, out=torch.empty_like(q))
    if own:
        lib = _lib()
        state["plan"] = lib.AttnPlan(lib.KvCache(k, v), q, state["out"], state["table"], state["length"],
                                     state["prefix_table"], state["prefix_len"], scale=state["scale"])
    return state


def _prepare_select(case, g, r):
    n = case["groups"] * case["beams"]
    logits = torch.randn((case["groups"], case["beams"], case["vocab"]), generator=g, device="cuda") * 2.5
    # some tokens may not be chosen (a grammar, a banned word)
    ban = torch.rand(case["vocab"], generator=g, device="cuda") < 0.01
    logits.masked_fill_(ban, -math.inf)
    scores = -torch.rand((case["groups"], case["beams"]), generator=g, device="cuda") * 6 - 2
    done = torch.zeros(n, dtype=torch.uint8, device="cuda")
    done[torch.from_numpy(r.permutation(n)[: case["done"]]).cuda()] = 1
    return dict(logits=logits, scores=scores, done=done.reshape(case["groups"], case["beams"]), done_token=2)


def _prepare_reorder(case, g, r):
    w, page = case["beams"], case["page"]
    n = case["groups"] * w
    # lengths differ from group to group, and are one within a group
    length = np.repeat([max(0, case["length"] - 5 * i) for i in range(case["groups"])], w)
    width = case["length"] // page + 2
    n_pages = 3 * n + 8
    ids = r.permutation(n_pages)
    table = r.randint(0, n_pages, (n, width))
    table[np.arange(n), length // page] = ids[:n]  # each beam's last page is its own
    fresh = ids[n: 2 * n]
    parent = np.sort(r.randint(0, w, (case["groups"], w)) // 2, axis=1)  # the best beams have several children
    k, v = _cache(case, g, case["layers"], n_pages)
    state = dict(parent=_ints(parent), table=_ints(table), length=_ints(length), fresh=_ints(fresh), k_cache=k, v_cache=v)
    if own:
        state["cache"] = _lib().KvCache(k, v)
    return state


# ---- one pass --------------------------------------------------------------------
def run(state):
    return {"append": _run_append, "attn": _run_attn, "select": _run_select, "reorder": _run_reorder}[state["case"]["op"]](state)


def _rotate(x, c, s, rot, pairs):
    """x [T][heads][dim] in 32 bits; c, s [T][1][rot / 2]."""
    h = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :h], x[..., h:rot])
    y = x.clone()
    if pairs:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        y[..., :h], y[..., h:rot] = a * c - b * s, a * s + b * c
    return y


def _run_append(st):
    case = st["case"]
    if own:
        lib = _lib()
        q_out = lib.q2_0_kv_append(st["cache"], 0, st["q"], st["k"], st["v"], st["pos"], st["slot"], st["table"], st["rope"],
                                   style=lib.Q2_0_ROPE_PAIRS if case["pairs"] else lib.Q2_0_ROPE_HALVES, seq=st["seq"],
                                   q_out=st["q_out"])
        return {"q": q_out, "k": st["k_cache"], "v": st["v_cache"]}
    dt, page = DTYPES[case["dtype"]], case["page"]
    q, k, rot = st["q"], st["k"], case["rot"]
    if rot:
        cs = st["rope"][st["pos"].long()][:, None]
        c, s = cs[..., : rot // 2], cs[..., rot // 2:]
        q, k = _rotate(q, c, s, rot, case["pairs"]), _rotate(k, c, s, rot, case["pairs"])
    slot = st["slot"].long()
    at = st["table"][st["seq"].long(), slot // page].long()
    st["k_cache"][0][at, :, slot % page] = k.to(dt)
    st["v_cache"][0][at, :, slot % page] = st["v"].to(dt)
    return {"q": q.to(dt), "k": st["k_cache"], "v": st["v_cache"]}


def _pages(cache, table):
    """[n][heads][tokens][dim] in 32 bits, of the pages that a table [n][width] names."""
    x = cache[0][table.long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1]).float()


def _run_attn(st):
    if own:
        st["plan"].execute(0)
        return st["out"]
    case = st["case"]
    gr, n_kv, d = case["groups"], case["n_kv"], case["dim"]
    n = gr * case["seqs"]
    share = case["n_q"] // n_kv
    q = st["q"].float().reshape(n, n_kv, share, d) * st["scale"]
    # the shared part: the rows of a group's sequences side by side
    qg = q.reshape(gr, case["seqs"], n_kv, share, d).transpose(1, 2).reshape(gr, n_kv, case["seqs"] * share, d)
    kp, vp = _pages(st["k_cache"], st["prefix_table"]), _pages(st["v_cache"], st["prefix_table"])
    inp = torch.arange(kp.shape[2], device="cuda") < st["prefix_len"][:, None]
    sp = (qg @ kp.transpose(2, 3)).masked_fill(~inp[:, None, None], -math.inf)
    # each sequence's own part
    ks, vs = _pages(st["k_cache"], st["table"]), _pages(st["v_cache"], st["table"])
    ins = torch.arange(ks.shape[2], device="cuda") < st["length"][:, None]
    ss = (q @ ks.transpose(2, 3)).masked_fill(~ins[:, None, None], -math.inf)
    back = lambda x: x.reshape(gr, n_kv, case["seqs"], share, -1).transpose(1, 2).reshape(n, n_kv, share, -1)  # noqa: E731
    fwd = lambda x: x.reshape(gr, case["seqs"], n_kv, share, -1).transpose(1, 2).reshape(gr, n_kv, case["seqs"] * share, -1)  # noqa: E731
    m = torch.maximum(back(sp.amax(-1, keepdim=True)), ss.amax(-1, keepdim=True))
    m = m.masked_fill(m == -math.inf, 0.0)
    pp, ps = torch.exp(sp - fwd(m)), torch.exp(ss - m)
    total = back(pp.sum(-1, keepdim=True)) + ps.sum(-1, keepdim=True)
    o = back(pp @ vp) + ps @ vs
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.reshape(n, case["n_q"], d).to(st["q"].dtype)


def _run_select(st):
    case = st["case"]
    if own:
        s, p, t = _lib().q2_0_beam_select(st["logits"], st["scores"], case["n_out"], done=st["done"], done_token=st["done_token"])
        return {"score": s, "parent": p, "token": t}
    gr, w, n_out = case["groups"], case["beams"], case["n_out"]
    x = st["logits"]
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    # the best of each beam by its logits, the lowest token first among equals; then over the beams by score, the lowest beam first
    keep = min(n_out, case["vocab"])
    top, token = torch.sort(x, dim=-1, descending=True, stable=True)
    top, token = top[..., :keep], token[..., :keep]
    score = st["scores"][..., None] + (top - lse)
    done = st["done"].bool()[..., None]
    first = torch.arange(keep, device="cuda") == 0
    score = torch.where(done, torch.where(first, st["scores"][..., None], -math.inf), score)
    token = torch.where(done, st["done_token"], token)
    best, at = torch.sort(score.reshape(gr, w * keep), dim=-1, descending=True, stable=True)
    at, best = at[:, :n_out], best[:, :n_out].contiguous()
    parent, token = at // keep, torch.gather(token.reshape(gr, w * keep), 1, at)
    return {"score": best, "parent": parent.int(), "token": token.int()}


def _run_reorder(st):
    case = st["case"]
    if own:
        t, n, u = _lib().q2_0_beam_reorder(st["cache"], st["parent"], st["table"], st["length"], st["fresh"])
        return {"table": t, "length": n, "used": u, "k": st["k_cache"], "v": st["v_cache"]}
    w, page = case["beams"], case["page"]
    n = case["groups"] * w
    base = torch.arange(case["groups"], device="cuda")[:, None] * w
    p = (st["parent"] + base).reshape(-1).long()
    # the first child of a beam keeps its last page
    again = (p[:, None] == p[None, :]).tril(-1).any(1)
    length = st["length"][p]
    fill, last = length % page, (length // page).long()
    used = again | (fill == 0)
    table = st["table"][p]
    rows = torch.arange(n, device="cuda")
    old = table[rows, last].long()
    table[rows, last] = torch.where(used, st["fresh"], table[rows, last])
    keep = (torch.arange(page, device="cuda") < fill[:, None]) & used[:, None]
    keep = keep[None, :, None, :, None]
    to = st["fresh"].long()
    for c in (st["k_cache"], st["v_cache"]):
        c[:, to] = torch.where(keep, c[:, old], c[:, to])
    return {"table": table, "length": length, "used": used.int(), "k": st["k_cache"], "v": st["v_cache"]}


# ---- what a pass cannot do without ------------------------------------------------
def work(case):
    if case["op"] == "append":
        t, d = case["tokens"], case["dim"]
        heads = case["n_q"] + 2 * case["n_kv"]
        return {"bytes": t * heads * d * 6 + t * case["rot"] * 4 + t * 16,
                "flops": t * (case["n_q"] + case["n_kv"]) * case["rot"] * 3}
    if case["op"] == "attn":
        lens, plens = _lens(case), _prefix_lens(case)
        d, n = case["dim"], len(lens)
        kept = (sum(lens) + sum(plens)) * case["n_kv"] * d * 4
        pages = sum(-(-x // case["page"]) for x in lens + plens)
        seen = sum(lens) + case["seqs"] * sum(plens)
        return {"bytes": kept + n * case["n_q"] * d * 4 + pages * 4 + (n + len(plens)) * 4, "flops": 4 * d * case["n_q"] * seen}
    if case["op"] == "select":
        n = case["groups"] * case["beams"]
        return {"bytes": n * case["vocab"] * 4 + n * 5 + case["groups"] * case["n_out"] * 12, "flops": n * case["vocab"] * 4}
    n = case["groups"] * case["beams"]
    width = case["length"] // case["page"] + 2
    fill = sum(max(0, case["length"] - 5 * g) % case["page"] for g in range(case["groups"])) * case["beams"]
    # of the beams' children about half are second ones, whose pages are read and written
    moved = fill // 2 * case["layers"] * case["n_kv"] * case["dim"] * 2 * 2 * 2
    return {"bytes": n * (width * 8 + 5 * 4) + moved, "flops": 0}


# ---- the same in 64 bits, from the definitions --------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "attn":
        return _exact_attn(case, st)
    if case["op"] == "select":
        return _exact_select(case, st)
    return _exact_reorder(case, st)


def _exact_append(case, st):
    rot, d = case["rot"], case["dim"]
    out = []
    for x in (st["q"], st["k"]):
        y = x.double()
        if rot:
            i = torch.arange(rot // 2, device="cuda")
            a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + rot // 2)
            cs = st["rope"].double()[st["pos"].long()]
            z = torch.complex(y[..., a], y[..., b]) * torch.complex(cs[:, : rot // 2], cs[:, rot // 2:])[:, None]
            y = y.clone()
            y[..., a], y[..., b] = z.real, z.imag
        out.append(y)
    flat = []
    where = (st["table"].gather(1, (st["slot"] // case["page"]).long()[None].expand(case["seqs"], -1))
             .gather(0, st["seq"].long()[None])[0].long() * case["page"] + (st["slot"] % case["page"]).long())
    for cache, x in ((st["k_cache"], out[1]), (st["v_cache"], st["v"].double())):
        c = cache[0].double().transpose(1, 2).reshape(-1, case["n_kv"], d).clone()
        c[where] = x
        flat.append(c.reshape(1, -1, case["page"], case["n_kv"], d).transpose(2, 3).contiguous())
    return {"q": out[0], "k": flat[0], "v": flat[1]}


def _exact_attn(case, st):
    lens, plens = _lens(case), _prefix_lens(case)
    share, s = case["n_q"] // case["n_kv"], case["seqs"]
    k, v = st["k_cache"][0], st["v_cache"][0]
    if 4 * case["dim"] * case["n_q"] * (sum(lens) + s * sum(plens)) > 4e11 or case["groups"] * s * case["n_kv"] > 4096:
        return None
    take = lambda c, ids, n, h: c[ids.long(), h].reshape(-1, case["dim"])[:n].double()  # noqa: E731
    out = torch.zeros((case["groups"] * s, case["n_q"], case["dim"]), dtype=torch.float64, device="cuda")
    for h in range(case["n_kv"]):
        hs = slice(h * share, (h + 1) * share)
        for g in range(case["groups"]):
            kp, vp = take(k, st["prefix_table"][g], plens[g], h), take(v, st["prefix_table"][g], plens[g], h)
            for b in range(g * s, (g + 1) * s):
                kk = torch.cat([kp, take(k, st["table"][b], lens[b], h)])
                if len(kk):
                    p = torch.softmax(st["q"][b, hs].double() @ kk.T * st["scale"], -1)
                    out[b, hs] = p @ torch.cat([vp, take(v, st["table"][b], lens[b], h)])
    return out


def _exact_select(case, st):
    w, n_out = case["beams"], case["n_out"]
    res = []
    for g in range(case["groups"]):
        x = st["logits"][g].double()
        s = torch.log_softmax(x, -1) + st["scores"][g].double()[:, None]
        one = torch.full_like(s, -math.inf)
        one[:, 0] = st["scores"][g].double()
        s = torch.where(st["done"][g].bool()[:, None], one, s)
        res.append(torch.topk(s.reshape(-1), n_out).values)
    return {"score": torch.stack(res), "parent": None, "token": None}


def _exact_reorder(case, st):
    w, page = case["beams"], case["page"]
    parent, table = st["parent"].tolist(), st["table"].tolist()
    length, fresh = st["length"].tolist(), st["fresh"].tolist()
    k, v = st["k_cache"].clone(), st["v_cache"].clone()
    for g in range(case["groups"]):
        seen = set()
        for j, p in enumerate(parent[g]):
            n = length[g * w + p]
            if p in seen and n % page:
                src = table[g * w + p][n // page]
                for c in (k, v):
                    c[:, fresh[g * w + j], :, : n % page] = c[:, src, :, : n % page]
            seen.add(p)
    return {"table": None, "length": None, "used": None, "k": k, "v": v}
